"""Run by tests/test_gpu_checked_attn.py in a child process with GDN_CHECKED=1: the attention calls of the checked
library (index range checks compiled in) over the smallest, ragged, shared-out, windowed and masked batches. Exits 0
when no check fired and the results match the oracle."""
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import gated_delta_ssm_gb300 as gdn  # noqa: E402
from oracle import attention as oa  # noqa: E402
from tests._attn import Batch, check  # noqa: E402

SCALE = 128 ** -0.5


def expect(code, what):
    torch.cuda.synchronize()
    got = gdn.check_device()
    if got != code:
        raise SystemExit(f"{what}: device error word {got}, expected {code}")


def attend(form, t, code=0, **kw):
    t.make_q()
    out = torch.full((t.N, t.Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    (gdn.attn_decode if form == "decode" else gdn.attn_prefill)(
        t.q, t.cache(), t.d["q_start"], t.d["kv_len"], out, t.dims(), scale=SCALE, **kw)
    expect(code, f"{form} {t.ns[:4]} {t.lens[:4]} {kw}")
    if code == 0:
        check(out, *t.expected(SCALE, **kw))


def append(t, dtype, rot, interleaved):
    mk = lambda h: torch.from_numpy(t.rng.normal(0, 1, (t.N, h, 128))).to(dtype).cuda()
    q, k, v = mk(t.Hq), mk(t.Hkv), mk(t.Hkv)
    rope = gdn.Rope.table(max(max(t.lens), 1), rot, 10000.0, interleaved)
    qo = torch.empty(t.N, t.Hq, 128, dtype=torch.bfloat16, device="cuda")
    gdn.attn_append(q, k, v, t.cache(), t.d["q_start"], t.d["kv_len"], rope, qo, t.dims())
    expect(0, f"append {t.ns} {t.lens} {rot}")
    for b in range(t.B):
        oa.append(t.v, t.vs, t.table[b], v[t.q_start[b]:t.q_start[b + 1]].double().cpu().numpy(), t.lens[b])
    assert np.array_equal(t.d["v"].cpu().numpy(), t.v) and np.array_equal(t.d["vs"].cpu().numpy(), t.vs)


def main():
    assert os.path.basename(gdn.library_path()) == "libgdn_checked.so", gdn.library_path()
    assert gdn.check_device() == 0
    for P in (16, 32, 64, 128):
        for dtype in (torch.bfloat16, torch.float32):
            append(Batch([1], [1], 1, 1, P), dtype, 16, False)
            append(Batch([1, 5, 70, 0, 3, 1], [1, 200, 70, 12, 2, 0], 6, 2, P, seed=P), dtype, 128, P == 32)
            append(Batch([4, 1, 2], [4, 65, 130], 16, 1, P, seed=P + 1), dtype, 64, P != 32)
        for form in ("decode", "prefill"):
            attend(form, Batch([1], [1], 1, 1, P))
            attend(form, Batch([4, 1, 0, 3, 2], [700, 129, 50, 2, 128], 16, 1, P, seed=P))
            attend(form, Batch([2, 1], [300, 77], 10, 2, P, seed=P), window=65)
        attend("prefill", Batch([300, 1, 129], [400, 17, 129], 6, 2, P, seed=P))
    rng = np.random.default_rng(0)
    for form in ("decode", "prefill"):
        attend(form, Batch([1], [40000], 8, 1, 64, seed=1))                  # shared out over the whole GPU
        attend(form, Batch([8, 8], [3000, 900], 8, 1, 32, seed=2), softcap=30.0)
        attend(form, Batch([1] * 300, rng.integers(0, 60, 300).tolist(), 2, 1, 16, seed=3))   # counted by whole CTAs
        t = Batch([2, 2], [100, 200], 4, 2, 16, seed=4)                      # a page outside the cache
        t.d["table"][1, 3] = t.n_pages
        attend(form, t, code=256)
    attend("prefill", Batch([2000, 300], [2000, 1500], 3, 1, 64, seed=5))
    attend("prefill", Batch([2000], [2000], 1, 1, 64, seed=6), window=100)
    print("checked attention clean")


if __name__ == "__main__":
    main()
