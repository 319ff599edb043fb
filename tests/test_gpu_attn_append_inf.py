"""Infinite elements inside the rotated part of a key or of q: the rotation's formula gives infinities there, which
are held as +-448 scales, or NaN where it has infinity times zero or less infinity, which is held as 0."""
import numpy as np
import pytest

from oracle import attention as oa
from tests._attn import Batch

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import gated_delta_ssm_gb300 as gdn  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,rot,interleaved", [(2, 128, False), (2, 64, True), (40, 64, False), (40, 128, True)])
def test_infinities_turn_as_the_formula_turns_them(dtype, n, rot, interleaved):
    t = Batch([n], [n + 5], 2, 1, 16, seed=n + rot)
    mk = lambda h: torch.from_numpy(t.rng.normal(0, 1, (n, h, 128))).to(dtype).cuda()
    q, k, v = mk(2), mk(1), mk(1)
    half = rot // 2
    a, b = (6, 7) if interleaved else (3, 3 + half)     # a pair, infinite on either side, and on both
    for x in (q, k):
        x[0, 0, a], x[1, 0, b] = float("inf"), float("-inf")
        if n > 2:
            x[7, 0, a], x[7, 0, b] = float("-inf"), float("inf")
            x[20, 0, a] = float("nan")
            x[33, 0, 127] = float("inf")
    rope = gdn.Rope.table(64, rot, 100.0, interleaved)
    qo = torch.empty(n, 2, 128, dtype=torch.bfloat16, device="cuda")
    gdn.attn_append(q, k, v, t.cache(), t.d["q_start"], t.d["kv_len"], rope, qo, t.dims())
    assert gdn.check_device() == 512
    cos, sin = rope.cos.cpu().numpy(), rope.sin.cpu().numpy()
    pos = np.arange(5, n + 5)
    with np.errstate(invalid="ignore"):
        want_q = oa.rotate(q.double().cpu().numpy(), pos, cos, sin, interleaved)
        want_k = oa.rotate(k.double().cpu().numpy(), pos, cos, sin, interleaved)
    oa.append(t.k, t.ks, t.table[0], want_k, n + 5)
    got = oa.held(t.d["k"].cpu().numpy(), t.d["ks"].cpu().numpy(), t.table[0], n + 5, 0)
    ref = oa.held(t.k, t.ks, t.table[0], n + 5, 0)
    assert np.array_equal(t.d["ks"].cpu().numpy(), t.ks)
    assert np.array_equal(got[5:], ref[5:])
    assert (np.abs(got[5]) == 448 * np.repeat(t.ks[t.table[0, 0], 0], 128)).sum() >= 2   # both members of the pair
    got_q = qo.double().cpu().numpy()
    assert np.array_equal(np.isnan(got_q), np.isnan(want_q))
    far = np.isinf(want_q)
    assert far.any() and np.array_equal(got_q[far], want_q[far])
    rest = np.isfinite(want_q)
    assert np.all(np.abs(got_q[rest] - want_q[rest]) <= 2.0 ** -8 * np.abs(want_q[rest]) + 2.0 ** -18)
