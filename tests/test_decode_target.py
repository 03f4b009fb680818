"""What the decoder asks of a target and what becomes of device status words, on the host: no
GPU needed."""

import pytest
import torch

from draft_sampling_lossless_gb300 import decode, layer


class Words:
    """Stands for whatever has a status() of its own."""

    def __init__(self, word=0):
        self.word = word

    def status(self, ws=None):
        return self.word


def decoder(target, step=0):
    d = object.__new__(decode.Decoder)
    d.t, d.step_, d.caches, d.ws = target, Words(step), [Words()], {}
    return d


def test_a_target_without_a_status_of_its_own_is_accepted():
    class Plain:
        def forward(self, tokens, attention):
            return None

    decoder(Plain()).check()
    with pytest.raises(RuntimeError, match="0x10"):
        decoder(Plain(), step=0x10).check()


def test_a_targets_status_is_looked_at():
    decoder(Words()).check()
    with pytest.raises(RuntimeError, match="0x10"):
        decoder(Words(0x10)).check()


def test_a_status_word_outlives_its_workspace(lib, monkeypatch):
    """Target4 takes a larger workspace when a pass has more rows than the last: what the kernels
    wrote into the first one's status word is still reported."""
    def empty(*args, **kw):
        return None

    for name in ("norm", "linear4", "gated4"):
        monkeypatch.setattr(layer, name, empty)
    monkeypatch.setattr(layer.Weights4, "quantize", classmethod(lambda cls, src: src))
    monkeypatch.setattr(layer, "status", lambda ws: int(ws[:4].view(torch.int32)))

    t = decode.Target4(V=16, d=32, Hq=2, Hkv=1, D=32, layers=1, F=32, device="cpu")

    def attention(i, q, k, v):
        return torch.zeros(q.shape, dtype=torch.bfloat16)

    assert t.status() == 0
    t.forward(torch.zeros(2, dtype=torch.long), attention)
    assert t.status() == 0
    t.ws[0][0] = 0x10
    t.forward(torch.zeros(500, dtype=torch.long), attention)
    assert t.status() == 0x10
    t.forward(torch.zeros(2, dtype=torch.long), attention)
    assert t.status() == 0x10


def test_workspaces_are_few(lib, monkeypatch):
    """Passes of more and more rows keep all their workspaces: a few, which add up to less than four
    times what the largest pass needs."""
    monkeypatch.setattr(layer, "norm", lambda *a, **kw: None)
    monkeypatch.setattr(layer, "linear4", lambda *a, **kw: None)
    monkeypatch.setattr(layer, "gated4", lambda *a, **kw: None)
    monkeypatch.setattr(layer.Weights4, "quantize", classmethod(lambda cls, src: src))
    t = decode.Target4(V=16, d=32, Hq=2, Hkv=1, D=32, layers=1, F=32, device="cpu")
    for n in range(0, 300):
        t.forward(torch.zeros(n, dtype=torch.long),
                  lambda i, q, k, v: torch.zeros(q.shape, dtype=torch.bfloat16))
        assert t.ws[-1].numel() >= layer.workspace_bytes(n, 64)
    assert len(t.ws) <= 11
    assert sum(w.numel() for w in t.ws) <= 4 * layer.workspace_bytes(300, 64)


@pytest.mark.gpu
def test_the_prompts_pass_is_checked():
    """A status word that the prompts' pass sets is an error before any step."""
    class Bad(decode.Target):
        def status(self):
            return 0x10

    with pytest.raises(RuntimeError, match="0x10"):
        decode.Decoder(Bad(), [[1, 2, 3]])
    decode.Decoder(Bad(), [[1]])  # no pass for prompts of one token
