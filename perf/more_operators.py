"""The target's layers around its attention: products with 4-bit weights, the
gated product of a feed-forward block, the norms between the blocks.  Cases,
inputs, plain forms and counts.

A 4-bit matrix W [N][K] is kept as codes [N][K / 2] (two a byte, the even column
in the low half) and one scale byte for 32 columns, [N][K / 32].  A code is a sign
bit over three bits that stand for 0, 0.5, 1, 1.5, 2, 3, 4, 6; a scale byte b
stands for 2^(b - 127).

  linear  out = x W^T
  gated   out = act(x G^T) * (x U^T), act silu or gelu (tanh form)
  norm    x' = x + alpha * gate * rms(y) * post,  h = rms(x') * pre, where
          rms(v) = v / sqrt(mean v^2 + eps); without post: x' = x + alpha * gate * y
          (without gate: 1), without y: x' = x

x, y, gate, out and h are bf16, the stream x of the norm bf16 or fp32.
"""

import math
import random

import torch

own = False

_FIELDS = dict(kind="linear", T=1, N=0, K=0, act="", dt="", post=False, gate="", y=True, apart=0)
_EPS = 1e-6


def _case(name=None, **kw):
    c = dict(_FIELDS, **kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    # hidden size 2560, 32 query heads over 8 key/value heads of 128 and 151936 tokens: the
    # qwen3_4b workload and the attention's cases; hidden size 7168: the deepseek workload;
    # a feed-forward width of four hidden sizes.  122 rows: what the scheduler lets through
    # of that workload's 64 requests and 7 drafted tokens each.
    return [
        # one user, one new token: queries, keys and values of one layer; latency alone
        _case("linear one token", T=1, N=6144, K=2560),
        # a few users' tokens through the second half of a feed-forward block
        _case("linear few down", T=6, N=2560, K=10240),
        # the verified rows of a step through the attention's output product
        _case("linear verify", T=122, N=2560, K=4096),
        # the logits of a batch's single tokens
        _case("linear logits", T=64, N=151936, K=2560),
        # prompts through queries, keys and values
        _case("linear prompts", T=4100, N=6144, K=2560),
        # one user's token through the first half of a feed-forward block
        _case("gated one token", kind="gated", T=1, N=10240, K=2560, act="silu"),
        # the verified rows of a step
        _case("gated verify", kind="gated", T=122, N=10240, K=2560, act="silu"),
        # a narrow expert of odd sizes, its rows gathered into a wider buffer
        _case("gated odd", kind="gated", T=37, N=1000, K=2080, act="gelu", apart=24),
        # prompts
        _case("gated prompts", kind="gated", T=4100, N=10240, K=2560, act="silu"),
        # one token between two blocks: latency alone
        _case("norm one token", kind="norm", T=1, K=2560, dt="bf16"),
        # the verified rows of a large model whose blocks have norms and gates of their own
        _case("norm verify", kind="norm", T=300, K=7168, dt="bf16", post=True, gate="rows"),
        # prompts, the stream between the blocks in fp32
        _case("norm prompts", kind="norm", T=16000, K=2560, dt="f32", post=True, gate="one"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["linear", "linear", "gated", "gated", "norm"])
    c = _case(kind=kind)
    c["apart"] = 8 * rng.choice([0, 0, 1, 5, 64])
    if kind == "norm":
        c["T"], c["K"] = _log_int(rng, 1, 16000), 8 * _log_int(rng, 8, 1024)
        c["dt"] = rng.choice(["bf16", "f32"])
        c["y"] = rng.random() < 0.85
        if c["y"]:
            c["post"], c["gate"] = rng.random() < 0.5, rng.choice(["", "one", "rows"])
    else:
        c["T"] = _log_int(rng, 1, 5000) if rng.random() < 0.5 else _log_int(rng, 1, 200)
        c["K"] = 32 * _log_int(rng, 2, 320)
        c["N"] = _log_int(rng, 16, 20000) if rng.random() < 0.85 else _log_int(rng, 20000, 150000)
        if kind == "gated":
            c["act"] = rng.choice(["silu", "gelu"])
    # no more than the largest listed cases
    top = [work(x) for x in listed() if x["kind"] == kind]
    while work(c)["flops"] > max(w["flops"] for w in top):
        c["T"] //= 2
    while work(c)["bytes"] > max(w["bytes"] for w in top):
        c["T" if kind == "norm" else "N"] //= 2
    return c


def work(case):
    T, N, K = case["T"], case["N"], case["K"]
    if case["kind"] == "norm":
        size = 4 if case["dt"] == "f32" else 2
        row = (size + 2) * K  # the stream in, h out
        if case["y"]:
            row += (size + 2) * K + (2 * K if case["gate"] == "rows" else 0)
        return {"bytes": T * row + 4 * K * (1 + case["post"]) + 2 * K * (case["gate"] == "one"),
                "flops": 0}
    mats = 2 if case["kind"] == "gated" else 1
    return {"bytes": mats * N * (K // 2 + K // 32) + 2 * T * (K + N), "flops": 2 * mats * T * N * K}


def _weights(g, N, K):
    """Codes and scales of a matrix of normal values, rows of different sizes, each group of
    32 scaled so that its largest value is at most 6."""
    dev = g.device
    w = torch.randn((N, K // 32, 32), generator=g, device=dev)
    w *= torch.exp(0.5 * torch.randn((N, 1, 1), generator=g, device=dev)) / math.sqrt(K)
    e = torch.ceil(torch.log2(w.abs().amax(-1) / 6)).clamp(min=-100)
    a = w.abs() * torch.exp2(-e).unsqueeze(-1)
    code = torch.zeros(w.shape, dtype=torch.uint8, device=dev)
    for border in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):  # to the nearest value
        code += a > border
    code += 8 * (w < 0).to(torch.uint8)
    code = code.view(N, K)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e + 127).to(torch.uint8)


def _inputs(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 29)
    kind, T, N, K = (case[k] for k in ("kind", "T", "N", "K"))
    s = dict(case=case)
    # hidden states: channels of different sizes, a few far larger than the others
    size = torch.exp(0.5 * torch.randn(K, generator=g, device=dev))
    size[torch.randint(0, K, (max(1, K // 512),), generator=g, device=dev)] *= 30
    x = torch.randn((T, K + case["apart"]), generator=g, device=dev)
    x[:, :K] *= size
    if kind != "norm":
        s["x"] = x.bfloat16()[:, :K]
        for name in ("w",) if kind == "linear" else ("gate", "up"):
            s[name] = _weights(g, N, K)
        return s
    s["x"] = (x if case["dt"] == "f32" else x.bfloat16())[:, :K]
    s["y"] = s["post"] = s["gate"] = None
    s["alpha"] = 1.0
    if case["y"]:
        s["y"] = torch.randn((T, K + case["apart"]), generator=g, device=dev).bfloat16()[:, :K]
        s["alpha"] = 0.7
        if case["post"]:
            s["post"] = 1 + 0.2 * torch.randn(K, generator=g, device=dev)
        if case["gate"]:
            rows = T if case["gate"] == "rows" else 1
            s["gate"] = torch.sigmoid(torch.randn((rows, K), generator=g, device=dev)).bfloat16()
    s["pre"] = 1 + 0.2 * torch.randn(K, generator=g, device=dev)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    T, N, K = case["T"], case["N"], case["K"]
    dev = s["x"].device
    if case["kind"] == "norm":
        s["h"] = torch.empty((T, K), dtype=torch.bfloat16, device=dev)
        s["x_out"] = torch.empty((T, K), dtype=s["x"].dtype, device=dev) if case["y"] else None
        return s
    s["out"] = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
    if own:
        from draft_sampling_lossless_gb300.layer import Weights4, workspace

        for name in ("w", "gate", "up"):
            if name in s:
                s[name] = Weights4.load(*s[name])
        s["ws"] = workspace(T, K, device=dev)
    return s


def _matrix(w):
    """fp32 values of codes and scales."""
    codes, scales = w
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    values = torch.cat([values, -values])
    both = torch.stack([codes & 15, codes >> 4], dim=-1)
    m = values[both.int()].view(codes.shape[0], -1, 32)
    return (m * torch.exp2(scales.float() - 127).unsqueeze(-1)).view(codes.shape[0], -1)


def _rms(v):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + _EPS)


def run(state):
    s, case = state, state["case"]
    if own:
        from draft_sampling_lossless_gb300 import layer

        if case["kind"] == "linear":
            layer.linear4(s["x"], s["w"], s["out"], s["ws"])
            return s["out"]
        if case["kind"] == "gated":
            layer.gated4(s["x"], s["gate"], s["up"], s["out"], s["ws"], act=case["act"])
            return s["out"]
        layer.norm(s["x"], s["h"], s["pre"], y=s["y"], x_out=s["x_out"], post=s["post"],
                   gate=s["gate"], alpha=s["alpha"], eps=_EPS)
        return s["h"] if s["x_out"] is None else (s["h"], s["x_out"])
    x = s["x"].float()
    if case["kind"] == "linear":
        return (x @ _matrix(s["w"]).T).bfloat16()
    if case["kind"] == "gated":
        a, b = x @ _matrix(s["gate"]).T, x @ _matrix(s["up"]).T
        if case["act"] == "silu":
            a = a / (1 + torch.exp(-a))
        else:
            a = 0.5 * a * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a * a * a)))
        return (a * b).bfloat16()
    if s["y"] is None:
        return (_rms(x) * s["pre"]).bfloat16()
    u = s["y"].float()
    if s["post"] is not None:
        u = _rms(u) * s["post"]
    if s["gate"] is not None:
        u = u * s["gate"].float()
    x = x + s["alpha"] * u
    return (_rms(x) * s["pre"]).bfloat16(), x.to(s["x"].dtype)


def _exact_matrix(codes, scales):
    """64-bit values: a code's fields are a sign, 2 bits of exponent (bias 1) and 1 of fraction."""
    c = torch.zeros((codes.shape[0], 2 * codes.shape[1]), dtype=torch.int64, device=codes.device)
    c[:, 0::2], c[:, 1::2] = (codes % 16).long(), (codes // 16).long()
    e, f = (c // 2) % 4, (c % 2).double() / 2
    v = torch.where(e == 0, f, torch.ldexp(1 + f, e - 1))
    v = torch.where(c >= 8, -v, v)
    return torch.ldexp(v, scales.long().repeat_interleave(32, 1) - 127)


def _exact_product(x, w):
    """x W^T in 64 bits, some rows of W at a time."""
    step = max(1, (1 << 26) // x.shape[1])
    return torch.cat([x @ _exact_matrix(w[0][n:n + step], w[1][n:n + step]).T
                      for n in range(0, w[0].shape[0], step)], dim=1)


def exact(case, seed):
    if work(case)["flops"] > 4e12:
        return None
    s = _inputs(case, seed)
    x = s["x"].double()
    if case["kind"] == "linear":
        return _exact_product(x, s["w"])
    if case["kind"] == "gated":
        a, b = _exact_product(x, s["gate"]), _exact_product(x, s["up"])
        if case["act"] == "silu":
            return a * torch.sigmoid(a) * b
        t = torch.tanh((2 / math.pi) ** 0.5 * (a + 0.044715 * a ** 3))
        return a * (1 + t) / 2 * b
    if s["y"] is not None:
        u = s["y"].double()
        if s["post"] is not None:
            u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + _EPS) * s["post"].double()
        if s["gate"] is not None:
            u = s["gate"].double() * u
        x = x + s["alpha"] * u
    h = x / torch.sqrt((x * x).mean(-1, keepdim=True) + _EPS) * s["pre"].double()
    return h if s["y"] is None else (h, x)
