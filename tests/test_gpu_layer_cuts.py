"""The 4-bit products in every form that a call can take, and at large sizes, against a 64-bit form
of codes and scales that this file made: nothing of the library is in the reference.

A product is cut by a rule on its sizes: rows of x a tile, one or two row tiles of W a block,
both of x's terms in one MMA or one each, K over 1 to 8 blocks, x split by the blocks or by a kernel
before, one tile a block or several.  LINEAR and GATED have one size, ragged where it can be,
for each combination that the rule takes among 3 million drawn sizes (T to 5000, N to 160000,
K to 12800) on 152 SMs, and one for each form of the kernel of a few rows.

x has 8 bits in every value, the weights' partial sums are whole numbers of halves: of random
signs, K of at most 255 * 6 * 2, they pass 2^22 with a chance below 2 exp(-2^44 / (2 K 3060^2)),
1e-30 at K = 13000 (where K is larger the scales are 1: K of 255 * 6, K to 65536, 1e-24).  So fp32
sums are exact in any order, and a product is the exact one, rounded once.  The gated product's
factors are exact alike; act in fp32 is off by 2^-15 at most (the exponential's argument is
below 96 and carries 5 roundings), the result is rounded once."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

from draft_sampling_lossless_gb300 import layer  # noqa: E402
from test_gpu_layer import DEV, VALUES, act64, run_gated, run_linear  # noqa: E402

LINEAR = ((1, 131, 32), (9, 131, 32), (17, 133, 32), (33, 131, 32), (33, 138, 704), (33, 137, 992),
          (1249, 131, 32), (2484, 131, 32), (9, 132, 9504), (17, 139, 5056), (19, 137, 5312),
          (18, 131, 7200), (1, 17162, 1184), (2451, 269, 32), (1, 7311, 3520), (1, 7322, 3808),
          (1, 104733, 288), (3662, 265, 32), (50, 19457, 32), (1, 12249, 2720), (61, 20053, 32),
          (97, 14604, 32), (17, 107225, 32), (65, 29881, 32), (82, 29737, 32), (17, 34014, 160),
          (2568, 132, 288), (2449, 259, 160), (33, 97771, 32), (4899, 139, 160), (1327, 266, 416),
          (17, 4945, 1760), (97, 49099, 32), (17, 10241, 928), (113, 49975, 32), (17, 1999, 5728),
          (614, 135, 2528), (290, 134, 5440), (636, 270, 1344), (1320, 133, 1440), (725, 257, 1504),
          (282, 131, 7776), (132, 68115, 32), (50, 2314, 2528), (24, 5393, 2336), (23, 4777, 2784),
          (81, 13434, 288), (29, 20877, 544), (52, 4902, 1440), (68, 2319, 2336), (34, 19614, 576),
          (484, 29329, 32), (22, 4837, 4384), (1441, 131, 2880), (2486, 148, 1504),
          (19, 9793, 3168), (458, 146, 10144), (4949, 261, 544), (3167, 131, 1760),
          (34, 5025, 5440), (199, 146062, 32), (36, 10246, 2976), (1906, 132, 5536),
          (243, 6434, 928), (15, 10209, 11072), (3737, 134, 3520), (15, 22505, 5408),
          (133, 13046, 1056), (2092, 131, 7104), (54, 20495, 1760), (4262, 132, 3808),
          (53, 4885, 10144), (2437, 158, 7616), (4900, 162, 4000), (49, 10017, 6720),
          (50, 60138, 1184), (165, 13159, 2272), (70, 19836, 4512), (161, 7230, 6848),
          (69, 10817, 12192), (207, 20910, 2912), (90, 59692, 11328), (123, 98121, 11872),
          (129, 109163, 12544))
GATED = ((1, 131, 32), (9, 132, 32), (17, 132, 32), (34, 132, 32), (36, 132, 672), (33, 140, 928),
         (1235, 137, 32), (17, 133, 4672), (1, 85758, 160), (3695, 131, 32), (33, 19542, 32),
         (66, 10031, 32), (22, 140, 8224), (65, 13250, 32), (18, 14613, 160), (18, 2509, 1344),
         (1256, 131, 448), (17, 5020, 928), (33, 6639, 416), (2574, 134, 288), (50, 68411, 32),
         (299, 135, 3040), (65, 68705, 32), (99, 45642, 32), (24, 2550, 2464), (613, 150, 1760),
         (1240, 137, 1184), (49, 10103, 416), (23, 4924, 1888), (81, 108194, 32), (250, 134, 10816),
         (4957, 161, 544), (908, 134, 3744), (53, 30201, 288), (17, 4657, 6560), (1995, 138, 1952),
         (4925, 273, 448), (2548, 132, 2016), (1390, 133, 3872), (65, 29886, 416),
         (15, 12557, 5088), (146, 68987, 160), (242, 16497, 416), (131, 13644, 1120),
         (81, 10857, 2336), (3077, 140, 5024), (1604, 141, 9632), (3901, 132, 8352),
         (92, 29282, 1600), (2472, 143, 12352), (4997, 159, 6336), (114, 12959, 6816))
# rows of the workloads, a vocabulary, the longest rows
LARGE = ((64, 151936, 2560), (9, 32000, 2560), (33, 151936, 640), (1500, 2560, 10240),
         (4100, 6144, 2560), (1, 300, 65536), (5, 130, 65280), (40, 130, 65280), (200, 130, 65280))
LARGE_GATED = ((1, 10240, 2560), (122, 10240, 2560), (2300, 10240, 640), (4100, 10240, 2560))


class Codes:
    """Random codes, and scales of shift and shift + 1 (K to 20000), on the GPU."""

    def __init__(self, N, K, seed, shift=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.N, self.K = N, K
        self.c = torch.randint(0, 16, (N, K), generator=g, device=DEV, dtype=torch.uint8)
        self.s = (127 - shift + torch.randint(0, 2 if K <= 20000 else 1, (N, K // 32), generator=g,
                                              device=DEV)).to(torch.uint8)

    def load(self):
        return layer.Weights4.load(self.c[:, 0::2] | (self.c[:, 1::2] << 4), self.s)

    def product(self, x):
        """x W^T in 64 bits, some rows of W at a time."""
        x, values, parts = x.double(), VALUES.to(DEV), []
        step = max(1, (1 << 26) // self.K)
        for n in range(0, self.N, step):
            w = values[self.c[n:n + step].int()].view(-1, self.K // 32, 32)
            w *= torch.exp2(self.s[n:n + step].double() - 127).unsqueeze(-1)
            parts.append(x @ w.view(-1, self.K).T)
        return torch.cat(parts, 1)


def rows(T, K, apart, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = 2 * torch.randint(64, 128, (T, K + apart), generator=g, device=DEV) + 1
    x *= 2 * torch.randint(0, 2, x.shape, generator=g, device=DEV) - 1
    return x.bfloat16()[:, :K]


@pytest.mark.parametrize("T,N,K", LINEAR + LARGE)
def test_linear(T, N, K):
    w = Codes(N, K, T + N)
    x = rows(T, K, 8 * (T % 3), T + K)
    o = w.product(x)
    assert o.abs().max() < 2 ** 22
    assert torch.equal(run_linear(x, w.load(), apart=(0, 3, 8)[(T + N) % 3]), o.float().bfloat16())


@pytest.mark.parametrize("T,N,K", GATED + LARGE_GATED)
def test_gated(T, N, K):
    # sums of some +-2: a product's size is 255 / 1.3 * 3 * 1.6 sqrt(K)
    shift = round(math.log2(470 * math.sqrt(K)))
    g, u = Codes(N, K, T + N, shift), Codes(N, K, T + N + 1, shift)
    x = rows(T, K, 8 * (T % 3), T + K)
    a, b = g.product(x), u.product(x)
    assert max(a.abs().max(), b.abs().max()) < 2.0 ** (22 - shift)
    act = ("silu", "gelu")[(T + N + K // 32) % 2]
    want = act64(act, a) * b
    got = run_gated(x, g.load(), u.load(), act, apart=(0, 3, 8)[(T + N) % 3])
    assert ((got.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -14) * want.abs() + 1e-36).all()


@pytest.mark.parametrize("N,K,dt", ((20001, 2560, torch.bfloat16), (1000, 10240, torch.float32),
                                    (151936, 640, torch.bfloat16), (130, 65280, torch.float32)))
def test_quantize(N, K, dt):
    """Codes by search over the values (ties to the even code) and scales by the rule, laid out by
    load: the store that quantize fills."""
    g = torch.Generator(device=DEV).manual_seed(N + K)
    w = torch.randn((N, K), generator=g, device=DEV).mul_(0.02).to(dt)
    mag, codes, scales = VALUES[:8].to(DEV), [], []
    step = max(1, (1 << 24) // K)
    for n in range(0, N, step):
        v = w[n:n + step].double().view(-1, K // 32, 32)
        m, e = torch.frexp(v.abs().amax(-1))  # the largest is m 2^e, 1/2 <= m < 1; 6 = 3/4 2^3
        e = torch.where(m <= 0.75, e - 3, e - 2).clamp(-100, 125)
        y = torch.ldexp(v, -e.unsqueeze(-1)).view(-1, K).abs()
        code = torch.zeros(y.shape, dtype=torch.uint8, device=DEV)
        for i in range(7):
            border = (mag[i] + mag[i + 1]) / 2
            code += (y >= border) if i % 2 else (y > border)
        codes.append(code + 8 * torch.signbit(w[n:n + step]).to(torch.uint8))
        scales.append((e + 127).to(torch.uint8))
    c, s = torch.cat(codes), torch.cat(scales)
    a = layer.Weights4.load(c[:, 0::2] | (c[:, 1::2] << 4), s)
    assert torch.equal(a.store, layer.Weights4.quantize(w).store)
