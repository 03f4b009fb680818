"""What a call on a stream of its own still reads is not handed out again: inputs of a load that
are gone on the host, weights dropped while a product runs.  The streams are held up by a wait of
some milliseconds, so that the kernels run after the memory could have been reused."""

import pytest
import torch

pytestmark = pytest.mark.gpu

from draft_sampling_lossless_gb300 import layer  # noqa: E402
from test_gpu_layer import DEV, Matrix, activations, check_linear, run_linear  # noqa: E402

WAIT = 40_000_000  # cycles: some 20 ms


def overwrite(n, stream=None):
    """Allocates and fills memory of n bytes: blocks that were freed come first."""
    with torch.cuda.stream(stream):
        return [torch.full((n,), 0x77, dtype=torch.uint8, device=DEV) for _ in range(4)]


@pytest.mark.parametrize("quantize", (False, True))
def test_inputs_of_a_load_on_another_stream_may_be_temporary(quantize):
    m = Matrix(512, 1024, lo=120, hi=126)
    host = m.m.cpu().float().bfloat16(), m.codes, m.scales
    x = activations(20, 1024)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(WAIT)
    if quantize:
        t = (host[0].to(DEV),)
    else:
        t = (m.codes.to(DEV), m.scales.to(DEV))
    s.wait_stream(torch.cuda.current_stream())
    q = layer.Weights4.quantize(*t, stream=s) if quantize else layer.Weights4.load(*t, stream=s)
    sizes = [v.nbytes for v in t]
    del t
    kept = [overwrite(n) for n in sizes]
    torch.cuda.current_stream().wait_stream(s)
    check_linear(x, m, run_linear(x, q))
    del kept


@pytest.mark.parametrize("gated", (False, True))
def test_weights_may_be_dropped_while_a_product_runs_on_another_stream(gated):
    """Loaded on one stream, used on another, dropped at once: the store's stream hands its
    memory out again only after the product."""
    m = Matrix(512, 1024, lo=118, hi=122)
    x = activations(20, 1024)
    run = (lambda q, o, ws: layer.gated4(x, q, q, o, ws)) if gated else (
        lambda q, o, ws: layer.linear4(x, q, o, ws))
    outs = [torch.empty(20, 512, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    ws = layer.workspace(20, 1024)
    run(m.load(), outs[0], ws)
    s = torch.cuda.Stream()
    codes, scales = m.codes.to(DEV), m.scales.to(DEV)
    torch.cuda.synchronize()
    q = layer.Weights4.load(codes, scales, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(WAIT)
    run(q, outs[1], ws)
    n = q.store.nbytes
    del q
    kept = overwrite(n, s)
    torch.cuda.synchronize()
    assert torch.equal(*outs)
    del kept


def test_weights_made_here_and_used_on_a_given_stream():
    m = Matrix(512, 1024)
    x, s = activations(20, 1024), torch.cuda.Stream()
    out = torch.empty(20, 512, dtype=torch.bfloat16, device=DEV)
    q = m.load()
    s.wait_stream(torch.cuda.current_stream())
    ws = layer.workspace(20, 1024, stream=s)
    with torch.cuda.stream(s):
        torch.cuda._sleep(WAIT)
    layer.linear4(x, q, out, ws, stream=s)
    n = q.store.nbytes
    del q
    kept = overwrite(n)
    torch.cuda.synchronize()
    check_linear(x, m, out)
    assert layer.status(ws) == 0
    del kept


def test_a_stream_is_noted_once_and_a_capture_may_be_the_first_use():
    m = Matrix(130, 256)
    x = activations(9, 256)
    q = m.load()
    s = torch.cuda.Stream()
    out, ws = torch.empty(9, 130, dtype=torch.bfloat16, device=DEV), layer.workspace(9, 256)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        layer.linear4(x, q, out, ws)
    assert q._streams >= {s.cuda_stream} and len(q._streams) == 2
    g.replay()
    check_linear(x, m, out)
    layer.linear4(x, q, out, ws, stream=s)
    assert len(q._streams) == 2
    torch.cuda.synchronize()
    check_linear(x, m, out)
    g.replay()
    torch.cuda.synchronize()
