"""Keys that the rotation turns to just beside a rounding border: the codes and scales are those of the exact
rotation, not of its value in 32 bits, which lies on the border."""
import numpy as np
import pytest

from oracle import attention as oa
from tests._attn import Batch

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import gated_delta_ssm_gb300 as gdn  # noqa: E402

# cos 1 and sin 2^-30: (a, b) becomes a - b 2^-30 exactly, which 32 bits round to a for a of about 1
TINY = 2.0 ** -30


def _append(t, k, rope):
    v = torch.zeros_like(k)
    gdn.attn_append(None, k, v, t.cache(), t.d["q_start"], t.d["kv_len"], rope, None, t.dims())
    torch.cuda.synchronize()
    cos, sin = rope.cos.cpu().numpy(), rope.sin.cpu().numpy()
    x = oa.rotate(k.double().cpu().numpy(), np.arange(t.lens[0] - t.ns[0], t.lens[0]), cos, sin, rope.interleaved)
    oa.append(t.k, t.ks, t.table[0], x, t.lens[0])
    assert np.array_equal(t.d["ks"].cpu().numpy(), t.ks)
    codes, scales = t.d["k"].cpu().numpy(), t.d["ks"].cpu().numpy()
    for h in range(t.Hkv):   # values: a zero may have either sign
        assert np.array_equal(oa.held(codes, scales, t.table[0], t.lens[0], h),
                              oa.held(t.k, t.ks, t.table[0], t.lens[0], h))
    assert gdn.check_device() == 0
    return x


def _rope(n, rot, interleaved):
    return gdn.Rope(torch.full((n, rot // 2), 1.0, device="cuda"), torch.full((n, rot // 2), TINY, device="cuda"),
                    interleaved=interleaved)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,P,rot,interleaved", [(1, 16, 128, False), (4, 16, 32, True), (70, 64, 128, False),
                                                 (33, 32, 64, True), (129, 128, 96, False)])
def test_codes_beside_a_midpoint(dtype, n, P, rot, interleaved):
    t = Batch([n], [n], 2, 2, P, seed=n)
    a = np.zeros((n, 2, 128))
    i = np.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    # midpoints between the eight codes of [1, 2), times powers of two down to the scale's smallest step, of either
    # sign, turned up or down by a partner of either sign; the scale is that of the largest value, 1
    token, head = np.arange(n)[:, None, None], np.arange(2)[None, :, None]
    mid = (1 + (2 * ((i + token) % 8) + 1) / 16) * 2.0 ** -(1 + (i + token + head) % 12) * (-1.0) ** (i // 2 + head)
    a[..., ia] = mid
    a[..., ib] = (-1.0) ** (i + token) + 0 * head
    x = _append(t, torch.from_numpy(a).to(dtype).cuda(), _rope(n, rot, interleaved))
    s = float(t.ks[t.table[0, 0], 0])
    held = [oa.e4m3_codes(y / s) for y in (x, x.astype(np.float32).astype(np.float64))]
    assert (held[0] != held[1]).sum() > rot // 8     # the borders are met


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_a_scale_beside_its_border(dtype, sign):
    # 1.75 (448 times a power of two) turned up needs the next scale, turned down it does not
    for partner, scale in ((-1.0, 2.0 ** -7), (1.0, 2.0 ** -8)):
        t = Batch([3], [3], 1, 1, 16, seed=2)
        a = np.zeros((3, 1, 128))
        a[1, 0, 5], a[1, 0, 69] = sign * 1.75, sign * partner
        _append(t, torch.from_numpy(a).to(dtype).cuda(), _rope(3, 128, False))
        assert float(t.ks[t.table[0, 0], 0]) == scale


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_codes_of_many_keys_are_the_exact_rotations(dtype, interleaved):
    # about one code in a million lies beside a border in 32 bits
    t = Batch([3000], [3001], 8, 8, 64, seed=4)
    k = torch.from_numpy(t.rng.normal(0, 1, (3000, 8, 128))).to(dtype).cuda()
    _append(t, k, gdn.Rope.table(3001, 128, 10000.0, interleaved))
