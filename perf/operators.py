"""Attention over a paged key/value cache, and the cache's writing and reading:
cases, inputs, plain forms and counts.

Request n brings the rows row_off[n] .. row_off[n+1]-1 of a packed batch; its
row j sits at position ctx[n] + j.  Position p of request n is kept in page
pages[n][p // page] at slot p % page of the pools k and v, [pages][Hkv][page][D]:
bf16 values, or e4m3 codes with one exponent byte for each (page, head, slot).
The value of a code c is c * 2^(byte - 127); a row's exponent is the smallest
e >= -100 with max |x| <= 448 * 2^e.

  attend  o = softmax(scale * q k^T) v over the visible positions, and the
          natural logarithm of each row's sum of exponentials
  write   the new rows' keys and values go into the pools; the pools (bf16),
          or the new rows read back (e4m3), come out
  read    a range of positions of every request as bf16 rows
"""

import math
import random

import torch

own = False

_FIELDS = dict(kind="attend", fmt="bf16", R=1, Hq=32, Hkv=8, D=128, page=16, rows_lo=1, rows_hi=1,
               ctx_lo=0, ctx_hi=0, causal=True, window=0)


def _case(name=None, **kw):
    c = dict(_FIELDS, **kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    # 32 query heads over 8 key/value heads of 128: the attention of the 4B model whose
    # vocabulary and hidden size the qwen3_4b workload has; 64 requests and up to 8 rows
    # (7 drafted positions and the anchor) are that workload's step.
    return [
        # one user, one new token, a short conversation: latency alone
        _case("attend one token", R=1, ctx_lo=700, ctx_hi=700),
        # a full serving batch that generates without drafts, 8-bit cache
        _case("attend tokens e4m3", fmt="fp8", R=256, ctx_lo=60, ctx_hi=2100, page=32),
        # the verification of a drafted block: ragged lengths that the scheduler chose
        _case("attend verify", R=64, rows_lo=1, rows_hi=8, ctx_lo=500, ctx_hi=8000),
        # the same over an 8-bit cache
        _case("attend verify e4m3", fmt="fp8", R=64, rows_lo=1, rows_hi=8, ctx_lo=500, ctx_hi=8000),
        # a few very long documents: the long axis has to be split
        _case("attend long", R=3, rows_lo=5, rows_hi=8, ctx_lo=90000, ctx_hi=180000, page=64),
        # prompts in chunks, the earlier chunks already cached
        _case("attend chunk", R=2, rows_lo=1900, rows_hi=2100, ctx_lo=1000, ctx_hi=7000, page=64),
        # prompts in chunks for a model of sliding-window layers, 8-bit cache
        _case("attend chunk e4m3", fmt="fp8", R=3, Hq=40, Hkv=8, rows_lo=700, rows_hi=1500,
              ctx_lo=0, ctx_hi=6000, window=2048, page=32),
        # the drafter's block: its positions see each other both ways; small heads
        _case("attend block", R=64, Hq=16, Hkv=8, D=64, rows_lo=7, rows_hi=7, ctx_lo=100,
              ctx_hi=4000, causal=False),
        # the verified rows' keys and values go into the cache
        _case("write rows", kind="write", R=64, rows_lo=1, rows_hi=8, ctx_lo=100, ctx_hi=900),
        # the same quantised, and read back
        _case("write rows e4m3", kind="write", fmt="fp8", R=64, rows_lo=1, rows_hi=8, ctx_lo=100,
              ctx_hi=900),
        # prompts quantised as they are written, and read back for the drafter
        _case("write prompts e4m3", kind="write", fmt="fp8", R=9, rows_lo=1500, rows_hi=6000,
              ctx_lo=0, ctx_hi=3000, page=64),
        # cached prefixes read out to be moved to another pool
        _case("read prefixes", kind="read", R=24, rows_lo=500, rows_hi=8000, page=32),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "attend", "attend", "write", "read"])
    fmt = rng.choice(["bf16", "fp8"])
    Hkv = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 80, 96, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    c = _case(kind=kind, fmt=fmt, Hkv=Hkv, Hq=Hkv * group, D=D, page=page)
    if kind == "attend":
        shape = rng.choice(["tokens", "verify", "verify", "long", "chunk"])
        c["R"] = _log_int(rng, 1, 256)
        c["ctx_hi"] = _log_int(rng, 50, 9000)
        if shape == "verify":
            c["rows_hi"] = rng.randint(2, 17)
            c["causal"] = rng.random() < 0.8
            c["rows_lo"] = 1
        elif shape == "long":
            c["R"] = rng.randint(1, 3)
            c["ctx_hi"] = _log_int(rng, 30000, 150000)
            c["rows_lo"], c["rows_hi"] = 1, rng.randint(1, 8)
        elif shape == "chunk":
            c["R"] = rng.randint(1, 3)
            c["rows_hi"] = _log_int(rng, 50, 2000)
            c["rows_lo"] = max(1, c["rows_hi"] // 2)
            c["ctx_hi"] = _log_int(rng, 50, 6000)
        c["ctx_lo"] = int(c["ctx_hi"] * rng.uniform(0.05, 0.9))
        if c["causal"] and rng.random() < 0.25:
            c["window"] = _log_int(rng, 16, 4096)
    else:
        c["R"] = _log_int(rng, 1, 100)
        c["rows_hi"] = _log_int(rng, 1, 8000)
        c["rows_lo"] = max(1, c["rows_hi"] // 5)
        c["ctx_hi"] = _log_int(rng, 1, 2000) if kind == "write" else 0
    # no more than the largest listed cases
    top = [work(x) for x in listed() if x["kind"] == kind]
    while any(work(c)[k] > max(w[k] for w in top) for k in ("bytes", "flops")):
        at = "R" if c["R"] > 1 else "rows_hi" if c["rows_hi"] > 64 else "ctx_hi"
        c[at] //= 2
        c["rows_lo"], c["ctx_lo"] = min(c["rows_lo"], c["rows_hi"]), min(c["ctx_lo"], c["ctx_hi"])
    return c


def _sizes(case):
    """Rows and cached positions of each request: by the case alone."""
    rng = random.Random(":".join(str(case[k]) for k in _FIELDS))
    rows = [rng.randint(case["rows_lo"], case["rows_hi"]) for _ in range(case["R"])]
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["R"])]
    return rows, ctx


def _visible(case, m, ctx):
    """(rows' visible positions in all, positions that any row sees)."""
    if not case["causal"]:
        return m * (ctx + m), ctx + m
    w = case["window"] or ctx + m
    return sum(min(ctx + j + 1, w) for j in range(m)), ctx + m - max(0, ctx + 1 - w)


def work(case):
    rows, ctx = _sizes(case)
    T, D, Hq, Hkv = sum(rows), case["D"], case["Hq"], case["Hkv"]
    held = 2 * D if case["fmt"] == "bf16" else D + 1
    if case["kind"] == "attend":
        seen = [_visible(case, m, c) for m, c in zip(rows, ctx)]
        return {"bytes": 2 * Hkv * held * sum(s[1] for s in seen) + 2 * T * Hq * D * 2 + 4 * T * Hq,
                "flops": 4 * D * Hq * sum(s[0] for s in seen)}
    if case["kind"] == "read":
        return {"bytes": 2 * T * Hkv * (held + 2 * D), "flops": 0}
    back = 0 if case["fmt"] == "bf16" else held + 2 * D
    return {"bytes": 2 * T * Hkv * (2 * D + held + back), "flops": 0}


def _pow2(e):
    """2^e in fp32 (-126 <= e <= 127), from its bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantised(x):
    """e4m3 codes (as bytes) and exponent bytes of rows of x, along the last axis."""
    amax = x.float().abs().amax(-1)
    f, e = torch.frexp(amax)
    e = torch.where(f <= 0.875, e - 9, e - 8).clamp(min=-100)
    y = x.float() * _pow2(-e).unsqueeze(-1)
    return y.to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _values(codes, byte):
    """fp32 values of a pool's entries."""
    if byte is None:
        return codes.float()
    return codes.view(torch.float8_e4m3fn).float() * _pow2(byte.int() - 127).unsqueeze(-1)


def _inputs(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 17)
    rows, ctx = _sizes(case)
    R, Hq, Hkv, D, P = (case[k] for k in ("R", "Hq", "Hkv", "D", "page"))
    T = sum(rows)
    s = dict(case=case, scale=1.0 / math.sqrt(D))
    off = [0]
    for m in rows:
        off.append(off[-1] + m)
    s["row_off"] = torch.tensor(off, dtype=torch.int32, device=dev)
    s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
    s["max_rows"] = max(rows)
    # pages of a pool in use for a while: any order, some left over
    need = [-(-(c + m) // P) for m, c in zip(rows, ctx)]
    n_pages = sum(need) + 5
    ids = torch.randperm(n_pages, generator=g, device=dev).int()
    start = torch.tensor([sum(need[:n]) for n in range(R)], device=dev)
    at = torch.arange(max(need), device=dev)
    table = ids[(start.unsqueeze(1) + at).clamp(max=n_pages - 1)]
    used = torch.tensor(need, device=dev).unsqueeze(1) > at
    s["pages"] = torch.where(used, table, torch.full_like(table, -1))
    # the rows as one projection leaves them: queries, keys and values side by side
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device=dev).bfloat16()
    qkv[:, :Hq] *= 1.5
    s["q"], s["k_new"], s["v_new"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    # keys and values of heads and positions differ in size
    size = torch.exp(0.5 * torch.randn((2, n_pages, Hkv, P, 1), generator=g, device=dev))
    k, v = (torch.randn((n_pages, Hkv, P, D), generator=g, device=dev).mul_(x).bfloat16()
            for x in size)
    s["k_exp"] = s["v_exp"] = None
    if case["fmt"] == "fp8":
        k, s["k_exp"] = _quantised(k)
        v, s["v_exp"] = _quantised(v)
    s["k"], s["v"] = k, v
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    T, Hq, Hkv, D = s["q"].shape[0], case["Hq"], case["Hkv"], case["D"]
    if own:
        from draft_sampling_lossless_gb300.cache import PagedCache

        s["cache"] = PagedCache(s["k"], s["v"], s["k_exp"], s["v_exp"])
        s["ws"] = s["cache"].workspace(case["R"], T, Hq)
    dev = s["q"].device
    if case["kind"] == "attend":
        s["out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty((T, Hq), dtype=torch.float32, device=dev)
    else:
        s["k_out"], s["v_out"] = (torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=dev)
                                  for _ in range(2))
    return s


def _places(s, first):
    """Page and slot of every row: request n's row j at position first[n] + j."""
    t = torch.arange(s["q"].shape[0], device=first.device)
    n = torch.searchsorted(s["row_off"][1:].contiguous(), t.int(), right=True)
    p = first[n] + t - s["row_off"][n]
    P = s["case"]["page"]
    return s["pages"][n, p // P].long(), p % P


def _plain_write(s):
    page, slot = _places(s, s["ctx"])
    for pool, byte, new in (("k", "k_exp", "k_new"), ("v", "v_exp", "v_new")):
        if s[byte] is None:
            s[pool][page, :, slot] = s[new]
        else:
            s[pool][page, :, slot], s[byte][page, :, slot] = _quantised(s[new])


def _plain_read(s, first):
    page, slot = _places(s, first)
    return [_values(s[pool][page, :, slot], None if s[byte] is None else s[byte][page, :, slot])
            .bfloat16() for pool, byte in (("k", "k_exp"), ("v", "v_exp"))]


def _plain_attend(s):
    case, off, ctx = s["case"], s["row_off"], s["ctx"]
    R, Hq, Hkv, D = (case[k] for k in ("R", "Hq", "Hkv", "D"))
    G, dev = Hq // Hkv, off.device
    j = torch.arange(s["max_rows"], device=dev)
    m = (off[1:] - off[:-1]).unsqueeze(1)
    live = j < m  # [R, M]: the requests' rows, padded to the longest
    t = (off[:-1].unsqueeze(1) + j).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][t].float().view(R, -1, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hkv, -1, D)
    table = s["pages"].clamp(min=0).long()
    k, v = (_values(s[pool][table], None if s[byte] is None else s[byte][table])
            .transpose(1, 2).reshape(R, Hkv, -1, D) for pool, byte in (("k", "k_exp"), ("v", "v_exp")))
    c = torch.arange(k.shape[2], device=dev)
    pos = ctx.unsqueeze(1) + j  # [R, M]
    if case["causal"]:
        see = c <= pos.unsqueeze(-1)
        if case["window"]:
            see &= c > pos.unsqueeze(-1) - case["window"]
    else:
        see = (c < ctx.unsqueeze(1) + m).unsqueeze(1).expand(-1, j.numel(), -1)
    hide = ~(see & live.unsqueeze(-1)).repeat_interleave(G, 1).unsqueeze(1)  # [R, 1, M * G, L]
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).masked_fill_(hide, -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / total.clamp(min=1e-38)
    lse = (top + total.log()).squeeze(-1)
    o = o.view(R, Hkv, -1, G, D).permute(0, 2, 1, 3, 4).reshape(R, -1, Hq, D)
    lse = lse.view(R, Hkv, -1, G).permute(0, 2, 1, 3).reshape(R, -1, Hq)
    return o[live].bfloat16(), lse[live]


def run(state):
    s, kind = state, state["case"]["kind"]
    if kind == "attend":
        if not own:
            return _plain_attend(s)
        s["cache"].attend(s["q"], s["row_off"], s["ctx"], s["pages"], s["out"], lse=s["lse"],
                          scale=s["scale"], causal=s["case"]["causal"], window=s["case"]["window"],
                          max_rows=s["max_rows"], ws=s["ws"])
        return s["out"], s["lse"]
    if kind == "write":
        if own:
            s["cache"].append(s["k_new"], s["v_new"], s["row_off"], s["ctx"], s["pages"], s["ws"])
        else:
            _plain_write(s)
        if s["k_exp"] is None:
            return s["k"], s["v"]
    if not own:
        return _plain_read(s, s["ctx"])
    s["cache"].read(s["row_off"], s["ctx"], s["pages"], s["k_out"], s["v_out"], s["ws"])
    return s["k_out"], s["v_out"]


def _exact_pow2(e):
    """2^e in 64 bits, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values(codes, byte):
    """64-bit values: e4m3 by its fields, sign, 4 bits of exponent (bias 7), 3 of fraction."""
    if byte is None:
        return codes.double()
    u = codes.long()
    e, f = (u >> 3) & 15, (u & 7).double()
    mag = torch.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * _exact_pow2(e - 7))
    mag = mag * _exact_pow2(byte.long() - 127).unsqueeze(-1)
    return torch.where(u >= 128, -mag, mag)


def _exact_round(x):
    """What stands in the cache for the rows x, along the last axis."""
    x = x.double()
    amax = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448)).clamp(min=-100)
    e = torch.where(448 * _exact_pow2(e - 1) >= amax, e - 1, e).clamp(min=-100)
    e = torch.where(448 * _exact_pow2(e) < amax, e + 1, e)
    y = x / _exact_pow2(e)
    step = _exact_pow2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * _exact_pow2(e)


def exact(case, seed):
    if work(case)["flops"] > 4e12:
        return None
    s = _inputs(case, seed)
    rows, ctx = _sizes(case)
    Hkv, P, kind = case["Hkv"], case["page"], case["kind"]
    G = case["Hq"] // Hkv
    dev = s["q"].device
    o, lse, ks, vs, a = [], [], [], [], 0
    for n, (m, c0) in enumerate(zip(rows, ctx)):
        p = torch.arange(0 if kind == "attend" else c0, c0 + m, device=dev)
        page, slot = s["pages"][n].long()[p // P], p % P
        if kind == "write":
            new = [s[x][a:a + m] for x in ("k_new", "v_new")]
            if s["k_exp"] is None:
                s["k"][page, :, slot], s["v"][page, :, slot] = new
            else:
                ks.append(_exact_round(new[0]))
                vs.append(_exact_round(new[1]))
            a += m
            continue
        k, v = (_exact_values(s[x][page, :, slot], None if s[y] is None else s[y][page, :, slot])
                for x, y in (("k", "k_exp"), ("v", "v_exp")))
        if kind == "read":
            ks.append(k)
            vs.append(v)
            continue
        q = s["q"][a:a + m].double()
        a += m
        at = torch.arange(c0, c0 + m, device=dev).unsqueeze(1)
        hide = p > at
        if case["window"]:
            hide |= p <= at - case["window"]
        if not case["causal"]:
            hide = torch.zeros_like(hide)
        oh, lh = [], []
        for h in range(case["Hq"]):
            x = (q[:, h] @ k[:, h // G].T) * s["scale"]
            x = torch.where(hide, torch.full_like(x, -math.inf), x)
            z = torch.logsumexp(x, -1, keepdim=True)
            oh.append(torch.exp(x - z) @ v[:, h // G])
            lh.append(z[:, 0])
        o.append(torch.stack(oh, 1))
        lse.append(torch.stack(lh, 1))
    if kind == "attend":
        return torch.cat(o), torch.cat(lse)
    if kind == "write" and s["k_exp"] is None:
        return s["k"].double(), s["v"].double()
    return torch.cat(ks), torch.cat(vs)
