"""Helpers of the attention tests: a batch over a paged cache on the device, and its 64-bit results."""
from __future__ import annotations

import numpy as np

from oracle import attention as oa


class Batch:
    """Sequences of lens[b] tokens in the cache, the last ns[b] of them the call's own."""

    def __init__(self, ns, lens, Hq, Hkv, P, seed=0, extra_pages=3, slack=1, spread=1.0):
        import torch
        self.ns, self.lens, self.Hq, self.Hkv, self.P = list(ns), list(lens), Hq, Hkv, P
        self.B, self.N, self.G = len(self.ns), sum(self.ns), Hq // Hkv
        rng = self.rng = np.random.default_rng(seed)
        used = [-(-L // P) for L in self.lens]
        self.width = max(1, max(used)) + slack
        self.n_pages = sum(used) + extra_pages
        order = rng.permutation(self.n_pages)
        self.table = np.full((self.B, self.width), 1 << 30, np.int32)   # unused entries are never read
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = order[at:at + u]
            at += u
        shape = (self.n_pages, Hkv, P, 128)
        # any code but NaN in what is held; stale slots hold anything, NaN included
        self.k, self.v = (rng.integers(0, 256, shape).astype(np.uint8) for _ in range(2))
        self.ks, self.vs = (2.0 ** rng.integers(-7, -3, shape[:2]).astype(np.float32) for _ in range(2))
        for codes in (self.k, self.v):
            x = oa.e4m3_codes(rng.normal(0, 30 * spread, shape))
            live = np.zeros(shape[:3], bool)
            for b in range(self.B):
                for t in range(self.lens[b]):
                    live[self.table[b, t // P], :, t % P] = True
            codes[live] = x[live]
        self.q_start = np.concatenate([[0], np.cumsum(self.ns)]).astype(np.int32)
        self.kv_len = np.array(self.lens, np.int32)
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        self.d = {n: dev(getattr(self, n)) for n in ("k", "v", "ks", "vs", "table", "q_start", "kv_len")}

    def dims(self, **kw):
        import gated_delta_ssm_gb300 as gdn
        d = dict(n_seq=self.B, n_q_heads=self.Hq, n_kv_heads=self.Hkv, page_size=self.P,
                 n_pages=self.n_pages, max_pages=self.width, n_tokens=self.N, max_q=max(self.ns))
        d.update(kw)
        return gdn.AttnDims(**d)

    def cache(self):
        import gated_delta_ssm_gb300 as gdn
        return gdn.KvCache(self.d["k"], self.d["v"], self.d["ks"], self.d["vs"], self.d["table"])

    def make_q(self, std=1.0):
        import torch
        self.q = torch.from_numpy(self.rng.normal(0, std, (self.N, self.Hq, 128))).to(torch.bfloat16).cuda()
        return self.q

    def expected(self, scale, softcap=0.0, window=0):
        """(out, bound): the 64-bit result of attention and how far a correct kernel may be from it.

        bound: the output's rounding, 2^-8 |out|; each weight rounded to no fewer bits than bf16 has,
        2^-8, and an absolute floor of 2^-18 of the largest of 128 keys, 2^-11 together; sums and scores
        in 32 bits, at most 2^-16 of the sum of |products| of a score (128 terms and the factors)."""
        q = self.q.double().cpu().numpy()
        out, bound = np.zeros(q.shape), np.zeros(q.shape)
        for b in range(self.B):
            r0, r1 = self.q_start[b], self.q_start[b + 1]
            for h in range(self.Hkv):
                hs = slice(h * self.G, (h + 1) * self.G)
                k = oa.held(self.k, self.ks, self.table[b], self.lens[b], h)
                v = oa.held(self.v, self.vs, self.table[b], self.lens[b], h)
                o, mass, size = oa.attend(q[r0:r1, hs], k, v, scale, softcap, window)
                out[r0:r1, hs] = o
                bound[r0:r1, hs] = (2.0 ** -8 * np.abs(o) +
                                    (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16 * (1 + size[..., None])) * mass)
        return out, bound


def check(got, want, bound):
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.isfinite(err).all()
    over = err > bound
    assert not over.any(), f"{over.sum()} of {over.size} over; worst {np.max(err / np.maximum(bound, 1e-30)):.3g}"
