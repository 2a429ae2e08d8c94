"""Batches over a paged key/value cache and their values in 64 bits, for the
tests of fp8_rope_append_kv and fp8_paged_attention.  The reference walks the
sequences one by one, reads every key through the page table and keeps only
the visible ones; it shares nothing with the kernels."""
import numpy as np
import torch

import fp8_fine_grained_x128_gb300 as fg

KINDS = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}


class Case:
    """`lens`: (new, kv_len) of every sequence, kv_len counting the new tokens."""

    def __init__(self, lens, kind="bf16", heads=2, group=4, dim=128, page=16, layout="hnd", seed=0, spare_tokens=0,
                 first=0, pool_extra=3, stale=float("nan"), q_std=2.0):
        g = torch.Generator(device="cuda").manual_seed(1000 + seed)
        self.lens, self.kind, self.heads, self.group, self.dim, self.page = lens, kind, heads, group, dim, page
        need = [-(-kv // page) for _, kv in lens]
        pool = sum(need) + pool_extra
        order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
        width = max(need + [1])
        table = torch.full((len(lens), width), -7, dtype=torch.int32, device="cuda")   # unused entries: no page
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = table
        news = [first] + [n for n, _ in lens]
        self.q_offsets = torch.tensor(np.cumsum(news), dtype=torch.int32, device="cuda")
        self.kv_lens = torch.tensor([kv for _, kv in lens], dtype=torch.int32, device="cuda")
        self.first, self.tokens = first, int(sum(news)) + spare_tokens
        self.max_new = max([n for n, _ in lens] + [0])

        def pool_tensor():
            if layout == "nhd":
                t = torch.empty((pool, page, heads, dim), dtype=KINDS[kind], device="cuda").transpose(1, 2)
            elif layout == "padded":   # rows, heads and pages further apart than they are long
                t = torch.empty((pool, heads + 1, page + 1, dim + 32), dtype=KINDS[kind], device="cuda")
                t = t[:, :heads, :page, :dim]
            else:
                t = torch.empty((pool, heads, page, dim), dtype=KINDS[kind], device="cuda")
            return t

        self.k_scale = self.v_scale = None
        if kind != "bf16":
            self.k_scale = torch.tensor([5.1 / FMAX[kind]], device="cuda")
            self.v_scale = torch.tensor([4.3 / FMAX[kind]], device="cuda")
        if layout == "joint":   # keys and values of a page side by side in one allocation
            both = torch.empty((pool, 2, heads, page, dim), dtype=KINDS[kind], device="cuda")
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k, self.v = pool_tensor(), pool_tensor()
        for t, s in ((self.k, self.k_scale), (self.v, self.v_scale)):
            x = torch.randn(t.shape, generator=g, device="cuda")
            if s is not None:
                x = (x / s).clamp(-FMAX[kind], FMAX[kind])
            t.copy_(x.to(t.dtype))
        if stale is not None:   # whatever no sequence holds: pages of nobody and the rest of last pages
            self.fill_stale(stale)
        H = heads * group
        self.q = (torch.randn((self.tokens, H, dim), generator=g, device="cuda") * q_std).bfloat16()

    def fill_stale(self, value):
        used = torch.zeros((self.k.shape[0], self.page), dtype=torch.bool, device="cuda")
        for b, (_, kv) in enumerate(self.lens):
            j = torch.arange(kv, device="cuda")
            used[self.table[b, j // self.page].long(), j % self.page] = True
        for t in (self.k, self.v):
            x = t.float()
            x = torch.where(used[:, None, :, None], x, torch.full_like(x, value))
            t.copy_(x.to(t.dtype))

    def cache(self):
        return fg.PagedKV(self.k, self.v, self.k_scale, self.v_scale)

    def batch(self):
        return fg.PagedBatch(self.q_offsets, self.kv_lens, self.table, self.max_new)

    def keys(self, b):
        """[heads, kv_len, dim] keys and values of sequence b in 64 bits."""
        kv = self.lens[b][1]
        j = torch.arange(kv, device="cuda")
        pg, r = self.table[b, j // self.page].long(), j % self.page
        out = []
        for t, s in ((self.k, self.k_scale), (self.v, self.v_scale)):
            x = t.float()[pg, :, r].double()
            out.append((x if s is None else x * s.double()).transpose(0, 1))
        return out

    def reference(self, scale=None):
        """out, lse and the per-element error bounds of both, in 64 bits (rows of no sequence: NaN)."""
        H, D, G = self.heads * self.group, self.dim, self.group
        scale = D ** -0.5 if scale is None else scale
        out = torch.full((self.tokens, H, D), float("nan"), dtype=torch.float64, device="cuda")
        lse = torch.full((self.tokens, H), float("nan"), dtype=torch.float64, device="cuda")
        tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
        at = self.first
        for b, (new, kv) in enumerate(self.lens):
            k, v = self.keys(b)
            for i in range(new):
                p = kv - new + i
                t = at + i
                if p < 0:
                    out[t], lse[t] = 0.0, -float("inf")
                    continue
                kk, vv = k[:, :p + 1], v[:, :p + 1]
                q = self.q[t].double().view(self.heads, G, D)
                x = scale * q @ kk.transpose(1, 2)
                w = torch.softmax(x, -1)
                out[t] = (w @ vv).reshape(H, D)
                lse[t] = torch.logsumexp(x, -1).reshape(H)
                # FP32 scores: D products whose sum is rounded (at most one ulp an addition on the
                # tensor cores); FP32 sums over p + 1 keys; the exponential's and logarithm's own error
                mag = (scale * q.abs() @ kk.abs().transpose(1, 2)).amax(-1).reshape(H)
                e32 = 2 * (D * 2.0 ** -23 * mag + (p + 1) * 2.0 ** -24 + 2.0 ** -20)
                # probabilities rounded to BF16 (2^-9 each), then the output's own rounding
                mean_abs = (w @ vv.abs()).reshape(H, D)
                half_ulp = 2.0 ** (torch.floor(torch.log2(out[t].abs().clamp(min=2.0 ** -126))) - 8)
                tol[t] = mean_abs * (2.0 ** -9 + e32[:, None]) * 1.01 + half_ulp
                ltol[t] = e32 + 2.0 ** -22 * lse[t].abs()
            at += new
        return out, lse, tol, ltol
