"""Values at the ends of the ranges that gdn.h states for the attention calls, under scores that rise steeply."""
import numpy as np
import pytest

from tests._attn import Batch, check

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import gated_delta_ssm_gb300 as gdn  # noqa: E402


def _run(form, t, scale, **kw):
    out = torch.full((t.N, t.Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    (gdn.attn_decode if form == "decode" else gdn.attn_prefill)(
        t.q, t.cache(), t.d["q_start"], t.d["kv_len"], out, t.dims(), scale=scale, **kw)
    torch.cuda.synchronize()
    assert gdn.check_device() == 0
    return out


def _steps(ns, lens, Hq, steps, seed=0):
    """Every key of tile i scores steps[i]: keys of one value in all dimensions, q of ones, scale 1 / 128."""
    t = Batch(ns, lens, Hq, 1, 64, seed=seed)
    for b in range(t.B):
        for blk in range(-(-t.lens[b] // 64)):
            v = float(steps(blk // 2))
            t.k[t.table[b, blk]] = torch.tensor([v]).to(torch.float8_e4m3fn).view(torch.uint8).item()
    t.ks[:] = 1.0
    t.d["k"].copy_(torch.from_numpy(t.k)), t.d["ks"].copy_(torch.from_numpy(t.ks))
    t.q = torch.ones(t.N, Hq, 128, dtype=torch.bfloat16, device="cuda")
    return t


def _values(t, exponent, zero=lambda blk: False):
    """Values of pages of scale 2^exponent, zeros (as an append of zeros leaves them) in the pages that `zero` says."""
    t.vs[:] = 2.0 ** exponent
    for b in range(t.B):
        for blk in range(-(-t.lens[b] // 64)):
            if zero(blk):
                t.v[t.table[b, blk]], t.vs[t.table[b, blk]] = 0, 2.0 ** -100
    t.d["v"].copy_(torch.from_numpy(t.v)), t.d["vs"].copy_(torch.from_numpy(t.vs))


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_values_of_zero_everywhere(form):
    # three steps of e^20 within each CTA's share, and shares e^192 apart
    t = _steps([1], [131072], 1, lambda i: 20 * (i % 3) if i < 900 else 192)
    _values(t, 0, zero=lambda blk: True)
    assert not _run(form, t, 1 / 128).any()


@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("top", [20, 40, 112])
def test_pages_of_zeros_among_others(form, top):
    t = _steps([1, 4], [40000, 900], 2, lambda i: top * (i % 3) / 2)
    _values(t, -8, zero=lambda blk: blk % 4 == 1)
    check(_run(form, t, 1 / 128), *t.expected(1 / 128))


@pytest.mark.parametrize("exponent", [-75, -40, 0, 60, 100])
@pytest.mark.parametrize("top", [20, 40, 112])
def test_decode(exponent, top):
    t = _steps([1, 4], [131072, 900], 2, lambda i: top * (i % 3) / 2)
    _values(t, exponent)
    out, (want, bound) = _run("decode", t, 1 / 128), t.expected(1 / 128)
    check(out, want, bound)
    assert np.abs(want).max() > 2.0 ** exponent      # nothing but rounding separates zeros from these


@pytest.mark.parametrize("exponent", [-50, 0, 48])      # 448 * 2^48 * 6000 keys < 2^70
@pytest.mark.parametrize("top", [20, 40, 112])
def test_prefill(exponent, top):
    t = _steps([300, 2], [6000, 1000], 2, lambda i: top * (i % 3) / 2)
    _values(t, exponent)
    check(_run("prefill", t, 1 / 128), *t.expected(1 / 128))


@pytest.mark.parametrize("softcap", [30.0, 50.0, 55.0])
@pytest.mark.parametrize("exponent", [-50, 0, 23])      # 448 * 2^23 * 6000 keys < 2^45
@pytest.mark.parametrize("score", [-448, 448])
def test_prefill_with_a_cap(softcap, exponent, score):
    t = _steps([300, 2], [6000, 1000], 2, lambda i: score)
    _values(t, exponent)
    check(_run("prefill", t, 1 / 128, softcap=softcap), *t.expected(1 / 128, softcap))


@pytest.mark.parametrize("form,P", [("decode", 16), ("decode", 64), ("prefill", 16)])
@pytest.mark.parametrize("low,high", [(-75, -5), (-35, 35), (30, 100), (-50, 20)])
def test_pages_of_very_different_scales(form, P, low, high):
    if form == "prefill" and (low < -50 or high > 45):
        pytest.skip("past the prefill's range")
    t = Batch([1, 4], [9000, 900], 2, 1, P, seed=P)
    t.make_q()
    t.vs[:] = 2.0 ** np.where(t.rng.random(t.vs.shape) < 0.5, low, high)
    t.d["vs"].copy_(torch.from_numpy(t.vs))
    out = torch.zeros(t.N, t.Hq, 128, dtype=torch.bfloat16, device="cuda")
    (gdn.attn_decode if form == "decode" else gdn.attn_prefill)(
        t.q, t.cache(), t.d["q_start"], t.d["kv_len"], out, t.dims())
    torch.cuda.synchronize()
    check(out, *t.expected(128 ** -0.5))
