"""Speculative decoding over the paged cache (draft_sampling_lossless_gb300.decode):
every token of a greedy run is the argmax of a plain 64-bit forward pass over the
whole sequence, up to what the cache's and the operators' roundings can move."""

import pytest
import torch

pytestmark = pytest.mark.gpu

from draft_sampling_lossless_gb300.decode import Decoder, Target  # noqa: E402


def plain_logits(t, tokens, e4m3):
    """Logits of every position in 64 bits, and a bound of what roundings move; e4m3:
    keys and values as such a cache holds them."""
    def q8(x):  # the cache's e4m3: one power-of-two scale for each row of D values
        amax = x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -140)
        e = torch.ceil(torch.log2(amax / 448)).clamp(min=-100)
        e = torch.where(448 * 2.0 ** (e - 1) >= amax, e - 1, e).clamp(min=-100)
        s = torch.exp2(e)
        return (x / s).to(torch.float32).to(torch.float8_e4m3fn).double() * s

    x = t.emb.double()[torch.tensor(tokens, device=t.emb.device)]
    n = len(tokens)
    err = torch.zeros(n, dtype=torch.float64, device=x.device)  # of x, Euclidean
    causal = torch.ones(n, n, dtype=torch.bool, device=x.device).tril()
    if t.window:
        causal &= ~torch.ones_like(causal).tril(-t.window)
    for wqkv, wo in zip(t.wqkv, t.wo):
        h = t.norm(x)
        y = (h @ wqkv.double()).bfloat16().double().view(n, -1, t.D)
        q, k, v = y.split([t.Hq, t.Hkv, t.Hkv], dim=1)
        if e4m3:
            k, v = q8(k), q8(v)
        rep = t.Hq // t.Hkv
        k, v = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
        s = torch.einsum("ihd,jhd->hij", q, k) / t.D ** 0.5
        p = s.masked_fill(~causal, -torch.inf).softmax(-1)
        o = torch.einsum("hij,jhd->ihd", p, v).reshape(n, -1)
        # a relative 2^-8 of q, k, v and of o each (bf16; e4m3: a code's step of 2^-3 where
        # that turns a rounding over), and x's own error once more through norm and the
        # projection; s moves o by twice its change
        size = x.norm(dim=1) / t.d ** 0.5
        dh = err / size + 2.0 ** -20
        gain = torch.linalg.matrix_norm(wqkv.double(), 2)
        qk = dh * gain + 2.0 ** (-3 if e4m3 else -8) * y.flatten(1).norm(dim=1)
        worst = torch.cummax(qk, 0).values
        qn = q.norm(dim=2).amax(1)
        kn = torch.cummax(k.norm(dim=2).amax(1), 0).values
        vn = torch.cummax(v.norm(dim=2).amax(1), 0).values
        ds = (worst * (qn + kn)) / t.D ** 0.5
        do = t.Hq ** 0.5 * (2 * ds * vn + worst + 2.0 ** -7 * vn)
        err = err + torch.linalg.matrix_norm(wo.double(), 2) * do
        x = x + o @ wo.double()
    size = x.norm(dim=1) / t.d ** 0.5
    bound = err / size * t.unemb.double().norm(dim=1).amax()
    return t.norm(x) @ t.unemb.double().T, bound


@pytest.mark.parametrize("e4m3,window,page", [(False, 0, 16), (True, 0, 32), (False, 24, 16)])
def test_tokens_are_the_targets(e4m3, window, page):
    g = torch.Generator().manual_seed(5)
    prompts = [torch.randint(0, 512, (n,), generator=g).tolist() for n in (1, 2, 33, 90)]
    t = Target(window=window, seed=3)
    d = Decoder(t, prompts, page=page, e4m3=e4m3)
    gained = sum(len(x) for _ in range(8) for x in d.step())
    assert gained >= 8 * len(prompts)
    near = total = 0
    for p, seq in zip(prompts, d.tokens):
        logits, bound = plain_logits(t, seq, e4m3)
        at = torch.arange(len(p) - 1, len(seq) - 1, device=logits.device)
        got = logits[at, torch.tensor(seq[len(p):], device=logits.device)]
        top = logits[at].amax(1)
        assert (top - got <= 2 * bound[at]).all(), (top - got).max().item()
        near += int((top != got).sum())
        total += len(at)
    assert near <= total // 10  # the bound is wide; nearly all are the argmax itself


def test_more_than_a_token_a_step():
    """The drafter shares the target's tables: some drafted tokens are accepted."""
    prompts = [[i, 7 * i + 1] for i in range(8)]
    d = Decoder(Target(layers=1, seed=1), prompts)
    n = sum(len(x) for _ in range(6) for x in d.step())
    assert n > 8 * 6


def test_move_between_formats():
    """Pools moved bf16 -> bf16 on other pages change nothing."""
    prompts = [[3, 1, 4], list(range(50)), [9]]
    a, b = (Decoder(Target(seed=4), prompts) for _ in range(2))
    for i in range(6):
        if i == 3:
            b.move(e4m3=False)
        assert a.step() == b.step()
    b.move(e4m3=True)
    b.step()


def test_sampling_runs():
    d = Decoder(Target(seed=6), [[1, 2, 3], [4]], T=1.0)
    gained = [d.step() for _ in range(4)]
    assert all(1 <= len(x) <= 8 for s in gained for x in s)
