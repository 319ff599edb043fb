"""The softmax-attention layer of a hybrid model over the paged 8-bit cache, as a server runs it.

Two prompts are prefilled in chunks, then both sequences decode token by token, and at the end a draft of three
tokens is verified, two of which are rejected and overwritten by the next step. Every step is an append and an
attention call; the page table grows as the sequences do. The outputs are compared with plain attention over
the same keys and values in 32 bits.

    python examples/attention_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_ssm_gb300 as gdn  # noqa: E402

HQ, HKV, D, PAGE, ROT = 16, 4, 128, 64, 64
MAX_PAGES, N_PAGES = 16, 24


class Layer:
    """One layer's cache and what a server keeps beside it: page table, lengths, rotation table, workspaces."""

    def __init__(self, n_seq: int, dev):
        code = torch.float8_e4m3fn
        self.k, self.v = (torch.empty(N_PAGES, HKV, PAGE, D, dtype=code, device=dev) for _ in range(2))
        self.ks, self.vs = (torch.empty(N_PAGES, HKV, device=dev) for _ in range(2))
        self.table = torch.zeros(n_seq, MAX_PAGES, dtype=torch.int32, device=dev)
        self.cache = gdn.KvCache(self.k, self.v, self.ks, self.vs, self.table)
        self.rope = gdn.Rope.table(MAX_PAGES * PAGE, ROT, device=dev)
        self.free = list(range(N_PAGES))
        self.pages = [[] for _ in range(n_seq)]
        self.lens = [0] * n_seq
        self.n_seq, self.dev = n_seq, dev

    def step(self, qkv, counts, drop=0):
        """Append and attend counts[b] tokens of each sequence (rows of a fused q|k|v projection), after dropping
        the last `drop` tokens of every sequence (rejected drafts)."""
        for b, n in enumerate(counts):
            self.lens[b] += n - drop
            while len(self.pages[b]) * PAGE < self.lens[b]:
                page = self.free.pop()
                self.table[b, len(self.pages[b])] = page
                self.pages[b].append(page)
        dims = gdn.AttnDims(n_seq=self.n_seq, n_q_heads=HQ, n_kv_heads=HKV, page_size=PAGE, n_pages=N_PAGES,
                            max_pages=MAX_PAGES, n_tokens=qkv.shape[0], max_q=max(counts))
        starts = torch.tensor([0, *counts], device=self.dev).cumsum(0).to(torch.int32)
        lens = torch.tensor(self.lens, dtype=torch.int32, device=self.dev)
        q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([HQ * D, HKV * D, HKV * D], 1))
        rotated = torch.empty(q.shape, dtype=torch.bfloat16, device=self.dev)
        out = torch.empty_like(rotated)
        gdn.attn_append(q, k, v, self.cache, starts, lens, self.rope, rotated, dims)
        few = max(counts) * (HQ // HKV) <= 64
        (gdn.attn_decode if few else gdn.attn_prefill)(rotated, self.cache, starts, lens, out, dims)
        return out


def plain(rope, qkv, n_new):
    """Plain causal attention of a sequence's last n_new tokens; qkv [L][(HQ + 2 HKV) * D]."""
    L = qkv.shape[0]
    q, k, v = (t.float().unflatten(1, (-1, D)) for t in qkv.split([HQ * D, HKV * D, HKV * D], 1))
    c, s = rope.cos[:L, None], rope.sin[:L, None]

    def rotate(x):
        a, b, rest = x[..., :ROT // 2], x[..., ROT // 2:ROT], x[..., ROT:]
        return torch.cat([a * c - b * s, b * c + a * s, rest], -1)

    q, k = rotate(q)[L - n_new:], rotate(k)
    k, v = (x.repeat_interleave(HQ // HKV, 1) for x in (k, v))
    w = torch.einsum("ihd,jhd->hij", q, k) * D ** -0.5
    seen = torch.arange(L, device=qkv.device)[None] <= torch.arange(L - n_new, L, device=qkv.device)[:, None]
    return torch.einsum("hij,jhd->ihd", w.masked_fill(~seen, -torch.inf).softmax(-1), v)


def main() -> float:
    """Runs the layer; returns the largest root mean square error of a step, relative to its outputs'."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(0)
    rows = lambda n: torch.randn(n, (HQ + 2 * HKV) * D, generator=gen, device=dev).bfloat16()
    layer = Layer(2, dev)
    history = [rows(0), rows(0)]
    worst = 0.0

    def run(counts, drop=0):
        nonlocal worst
        qkv = rows(sum(counts))
        out = layer.step(qkv, counts, drop)
        for b, (new, got) in enumerate(zip(qkv.split(counts), out.split(counts))):
            history[b] = torch.cat([history[b][:len(history[b]) - drop], new])
            want = plain(layer.rope, history[b], counts[b])
            worst = max(worst, float((got.float() - want).norm() / want.norm()))

    run([300, 37])             # prompts, the first in two chunks
    run([200, 1])
    for _ in range(5):         # token by token
        run([1, 1])
    run([3, 3])                # a draft of three tokens
    run([1, 1], drop=2)        # of which one was accepted
    assert gdn.check_device() == 0
    return worst


if __name__ == "__main__":
    err = main()
    print(f"error {err:.3f} of the outputs (root mean square, worst step; keys and values are held in 8 bits)")
