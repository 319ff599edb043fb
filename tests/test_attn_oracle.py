"""The 64-bit attention oracle against closed forms, and its e4m3 codec against torch's."""
import numpy as np
import pytest

from oracle import attention as oa

torch = pytest.importorskip("torch")


def test_codec_matches_torch_on_every_code_and_on_ties():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(v, oa.e4m3_values().astype(np.float32), equal_nan=True)
    p = oa.e4m3_values()[:127]
    mid = (p[1:] + p[:-1]) / 2
    x = np.concatenate([p, mid, mid * (1 + 1e-6), mid * (1 - 1e-6), np.random.default_rng(0).normal(0, 30, 4000)])
    x = np.concatenate([x, -x])
    x = x[np.abs(x) <= 448]
    x32 = torch.from_numpy(x).float()
    mine = oa.e4m3_codes(x32.double().numpy())
    assert np.array_equal(mine, x32.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert np.array_equal(oa.e4m3_codes(np.array([1e9, -1e9, np.inf])), [126, 254, 126])


def test_scale_is_the_smallest_power_of_two_that_fits():
    for a in (448.0, 448.0 * (1 + 1e-9), 1.0, 0.875, 0.8750001, 1e-20, 3e30):
        s = oa.pow2_scale(a)
        assert a <= 448 * s and np.log2(s) == int(np.log2(s)) and a > 448 * s / 2
    assert oa.pow2_scale(0.0) == 2.0 ** -100


def test_rotation_keeps_norms_and_depends_on_the_distance_alone():
    rng = np.random.default_rng(1)
    a = np.arange(50)[:, None] * 100.0 ** (-np.arange(0, 64, 2) / 64)
    for inter in (False, True):
        x, y = rng.normal(size=(1, 1, 128)), rng.normal(size=(1, 1, 128))
        r = lambda z, p: oa.rotate(z, np.array([p]), np.cos(a), np.sin(a), inter)
        assert np.allclose(np.linalg.norm(r(x, 31)), np.linalg.norm(x))
        assert np.allclose((r(x, 31) * r(y, 11)).sum(), (r(x, 40) * r(y, 20)).sum())
        assert np.array_equal(r(x, 31)[..., 64:], x[..., 64:])


def test_appending_token_by_token_holds_the_same_values_when_the_first_is_largest():
    # no growth after the first token: the scale and every code equal those of one call
    rng = np.random.default_rng(2)
    x = rng.normal(size=(20, 2, 128))
    x[0, :, 0] = 100.0
    x[16, :, 0] = 100.0
    table = np.array([2, 0])
    one = np.zeros((3, 2, 16, 128), np.uint8), np.zeros((3, 2), np.float32)
    many = np.zeros((3, 2, 16, 128), np.uint8), np.zeros((3, 2), np.float32)
    oa.append(*one, table, x, 20)
    for i in range(20):
        oa.append(*many, table, x[i:i + 1], i + 1)
    assert np.array_equal(one[0], many[0]) and np.array_equal(one[1], many[1])
    got = oa.held(*one, table, 20, 1)
    assert np.all(np.abs(got - x[:, 1]) <= np.maximum(np.abs(x[:, 1]) * 2.0 ** -4, 0.25 * 2.0 ** -10))


def test_attention_closed_forms():
    k, v = np.zeros((6, 128)), np.random.default_rng(3).normal(size=(6, 128))
    q = np.ones((2, 3, 128))
    out, _, _ = oa.attend(q, k, v, 0.1)                       # equal scores: the mean of what is seen
    assert np.allclose(out[0], v[:5].mean(0)) and np.allclose(out[1], v.mean(0))
    out, _, _ = oa.attend(q, k, v, 0.1, window=2)
    assert np.allclose(out[0], v[3:5].mean(0)) and np.allclose(out[1], v[4:].mean(0))
    out, _, _ = oa.attend(np.ones((3, 1, 128)), k[:1], v[:1], 0.1)   # two padding rows
    assert not out[:2].any() and np.allclose(out[2], v[0])
    k[2] = 1.0                                                # one dominant score, capped
    out, _, _ = oa.attend(q, k, v, 1.0)
    assert np.allclose(out[1], v[2])
    out, _, _ = oa.attend(q, k, v, 1.0, softcap=np.log(4.0))
    w = np.ones(6)
    w[2] = 4.0 ** np.tanh(128 / np.log(4.0))
    assert np.allclose(out[1], w @ v / w.sum())
