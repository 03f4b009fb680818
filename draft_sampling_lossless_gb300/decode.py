"""Speculative decoding of a small target model, its attention over a paged
key/value cache: the draft, confidence, scheduling and verification calls of a
step with the target's forward pass between them.

In every layer the scheduled rows' keys and values are appended to the cache
and the rows attend to all that is cached before them.  A step's rejected rows
are not undone: the next step's context is shorter and its rows overwrite
them.  `Decoder.move` carries the sequences over to other pools (read, then
append), say from bf16 to e4m3.

The target is synthetic: random embeddings, a few attention layers on top of
them, an output table.  The drafter is the Markov head alone on the same two
tables, so that it agrees with the target most of the time.  The projections are
plain fp32 torch products; the attention, the cache and the four stages run in
the CUDA library.

    python -m draft_sampling_lossless_gb300.decode
"""

from __future__ import annotations

import math

import torch

from .cache import PagedCache
from .pipeline import DSparkStep


class Target:
    """x = emb[token]; per layer x += wo attention(norm(x) wq, wk, wv); then
    logits = norm(x) unemb^T.  Tokens have no positions but their order."""

    def __init__(self, V=512, d=64, Hq=8, Hkv=2, D=32, layers=2, window=0, device="cuda", seed=0):
        g = torch.Generator(device="cpu").manual_seed(seed)

        def w(*shape, std):
            return (torch.randn(shape, generator=g) * std).to(device)

        self.V, self.d, self.Hq, self.Hkv, self.D, self.window = V, d, Hq, Hkv, D, window
        self.emb = w(V, d, std=1.0)
        self.unemb = w(V, d, std=1.0)
        self.wqkv = [w(d, (Hq + 2 * Hkv) * D, std=1.5 / math.sqrt(d)) for _ in range(layers)]
        self.wo = [w(Hq * D, d, std=0.7 / math.sqrt(Hq * D)) for _ in range(layers)]

    @staticmethod
    def norm(x):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)

    def qkv(self, layer, x):
        """q [T, Hq, D], k and v [T, Hkv, D] in bf16: slices of one product."""
        y = (self.norm(x) @ self.wqkv[layer]).bfloat16().view(x.shape[0], -1, self.D)
        return y.split([self.Hq, self.Hkv, self.Hkv], dim=1)

    def forward(self, tokens, attention):
        """Logits [T, V] fp32; attention(layer, q, k, v) gives [T, Hq, D]."""
        x = self.emb[tokens]
        for i in range(len(self.wqkv)):
            x = x + attention(i, *self.qkv(i, x)).reshape(len(tokens), -1).float() @ self.wo[i]
        return self.norm(x) @ self.unemb.T


class Decoder:
    """R sequences decoded greedily (T = 0) or by sampling, gamma drafted tokens
    a step; pages of `page` positions out of one table for all layers."""

    def __init__(self, target, prompts, gamma=7, T=0.0, max_len=512, page=16, e4m3=False, seed=1):
        self.t, self.gamma, self.T, self.page = target, gamma, T, page
        self.R = R = len(prompts)
        self.dev = dev = target.emb.device
        self.max_pages = -(-(max_len + gamma + 1) // page)
        self.gen = torch.Generator(device=dev).manual_seed(seed)
        self._new_pools(e4m3)
        self.step_ = DSparkStep(R, gamma, target.V, target.d, R * (gamma + 1) + 1, device=dev)
        self.z = torch.zeros((R, gamma, target.V), device=dev)
        self.sps = 1.0 / (1.0 + torch.arange(R * (gamma + 1) + 1, device=dev) / (8.0 * R))
        self.c_in = torch.full((R, gamma), 0.8, device=dev)
        self.sts = torch.ones(gamma, device=dev)
        # the prompts, all but their last tokens, in one ragged call
        lens = [len(p) - 1 for p in prompts]
        row_off = torch.tensor([0] + lens, dtype=torch.int32, device=dev).cumsum(0).int()
        self.ctx = torch.zeros(R, dtype=torch.int32, device=dev)
        flat = torch.tensor([t for p in prompts for t in p[:-1]], dtype=torch.int64, device=dev)
        if len(flat):
            self._forward(flat, row_off, max(lens))
        self.ctx += torch.tensor(lens, dtype=torch.int32, device=dev)
        self.anchor = torch.tensor([p[-1] for p in prompts], dtype=torch.int32, device=dev)
        self.tokens = [list(p) for p in prompts]

    def _new_pools(self, e4m3):
        t, n = self.t, self.R * self.max_pages
        self.caches = [PagedCache.empty(n, t.Hkv, self.page, t.D, e4m3=e4m3, device=self.dev)
                       for _ in t.wqkv]
        ids = torch.randperm(n, generator=self.gen, device=self.dev)
        self.pages = ids.int().view(self.R, self.max_pages)
        # workspaces by the rows of a call
        self.ws = {}

    def _workspace(self, rows):
        if rows not in self.ws:
            self.ws[rows] = self.caches[0].workspace(self.R, rows, self.t.Hq)
        return self.ws[rows]

    def _forward(self, tokens, row_off, max_rows):
        ws = self._workspace(len(tokens))

        def attention(i, q, k, v):
            c = self.caches[i]
            c.append(k, v, row_off, self.ctx, self.pages, ws)
            out = torch.zeros(q.shape, dtype=torch.bfloat16, device=q.device)
            c.attend(q, row_off, self.ctx, self.pages, out, window=self.t.window,
                     max_rows=max_rows, ws=ws)
            return out

        return self.t.forward(tokens, attention)

    def step(self):
        """One speculative step; returns the tokens that each sequence gained."""
        s, t, R, G = self.step_, self.t, self.R, self.gamma
        u = None
        if self.T > 0:
            u = [torch.rand(n, generator=self.gen, device=self.dev) for n in ((R, G), (R, G), (R,))]
        u_draft, u_acc, u_fin = u or (None, None, None)
        s.draft(self.z, t.emb, t.unemb, self.anchor, u_draft, self.T)
        s.confidence(None, None, t.emb, self.anchor, self.sts, c_in=self.c_in)
        s.schedule(self.sps)
        # the scheduled rows: each sequence's last token, then its drafted ones
        row = torch.arange(R * (G + 1), dtype=torch.int32, device=self.dev)
        n = (torch.searchsorted(s.row_off, row, right=True) - 1).clamp(max=R - 1)
        j = (row - s.row_off[n]).clamp(max=G)
        drafted = s.tokens[n, (j - 1).clamp(min=0).long()]
        rows = torch.where(j == 0, self.anchor[n], drafted).long()
        logits = self._forward(rows, s.row_off, G + 1)
        s.verify(self.z, t.emb, t.unemb, self.anchor, logits, u_acc, u_fin, self.T)
        self.ctx += s.n_acc + 1
        self.anchor = s.out_tokens.gather(1, s.n_acc.long().view(R, 1)).view(R)
        out, n_acc = s.out_tokens.tolist(), s.n_acc.tolist()
        gained = [out[i][:n_acc[i] + 1] for i in range(R)]
        for i in range(R):
            self.tokens[i] += gained[i]
        self.check()
        return gained

    def move(self, e4m3):
        """The sequences in new pools of the given format, on other pages."""
        old, old_pages = self.caches, self.pages
        row_off = torch.cat([self.ctx.new_zeros(1), self.ctx.cumsum(0).int()])
        rows = int(row_off[-1])
        start = torch.zeros_like(self.ctx)
        ws = old[0].workspace(self.R, rows, self.t.Hq)
        kv = [torch.empty((rows, self.t.Hkv, self.t.D), dtype=torch.bfloat16, device=self.dev)
              for _ in range(2)]
        self._new_pools(e4m3)
        for a, b in zip(old, self.caches):
            a.read(row_off, start, old_pages, *kv, ws)
            b.append(*kv, row_off, start, self.pages, ws)
        if a.status(ws) != 0:
            raise RuntimeError(f"device status {a.status(ws):#x}")

    def check(self):
        for word in [self.step_.status()] + [self.caches[0].status(w) for w in self.ws.values()]:
            if word != 0:
                raise RuntimeError(f"device status {word:#x}")


def main():
    g = torch.Generator().manual_seed(2)
    prompts = [torch.randint(0, 512, (n,), generator=g).tolist() for n in (1, 5, 40, 150)]
    d = Decoder(Target(), prompts)
    steps = 24
    for i in range(steps):
        if i == steps // 2:
            d.move(e4m3=True)
        d.step()
    for p, t in zip(prompts, d.tokens):
        print(f"prompt of {len(p):3d}: {len(t) - len(p):3d} tokens in {steps} steps "
              f"({(len(t) - len(p)) / steps:.2f} a step): {t[len(p):len(p) + 12]} ..")


if __name__ == "__main__":
    main()
