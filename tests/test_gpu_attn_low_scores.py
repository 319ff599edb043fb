"""Rows all of whose scores lie far below zero, in blocks that several CTAs share: a part in which such a row sees no
key (the tiles past its own position, or ahead of its window) must not outweigh the part that holds its keys."""
import pytest

from tests._attn import Batch, check

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import gated_delta_ssm_gb300 as gdn  # noqa: E402

SCALE = 128 ** -0.5


def _low(ns, lens, Hq, Hkv, P, seed, level=25.0):
    """Keys of positive values, 0.75 in the mean, and q rows near -level: scores near -8.5 level."""
    t = Batch(ns, lens, Hq, Hkv, P, seed=seed)
    t.k &= 0x7f
    t.k[t.k == 0x7f] = 0
    t.ks[:] = 2.0 ** -5
    t.d["k"].copy_(torch.from_numpy(t.k)), t.d["ks"].copy_(torch.from_numpy(t.ks))
    t.make_q()
    t.q = (-(t.q.float().abs() * 0.1 + 1) * level).to(torch.bfloat16)
    return t


def _run(form, t, **kw):
    out = torch.full((t.N, t.Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    (gdn.attn_decode if form == "decode" else gdn.attn_prefill)(
        t.q, t.cache(), t.d["q_start"], t.d["kv_len"], out, t.dims(), scale=SCALE, **kw)
    torch.cuda.synchronize()
    assert gdn.check_device() == 0
    check(out, *t.expected(SCALE, **kw))


@pytest.mark.parametrize("level", [8.0, 12.0, 25.0])     # natural scores near -68, -102 and -213
def test_causal_blocks_cut_inside_the_diagonal(level):
    _run("prefill", _low([2048], [2048], 1, 1, 64, seed=1, level=level))
    _run("prefill", _low([700, 300], [700, 2300], 4, 2, 32, seed=2, level=level))


@pytest.mark.parametrize("window", [1, 100, 400])
def test_windows(window):
    _run("prefill", _low([1500], [2000], 1, 1, 16, seed=3), window=window)


@pytest.mark.parametrize("softcap", [50.0, 100.0, 300.0])
def test_caps(softcap):
    _run("prefill", _low([1500], [1500], 1, 1, 64, seed=4), softcap=softcap)


@pytest.mark.parametrize("window", [0, 300])
def test_drafts(window):
    _run("decode", _low([4, 1, 4], [9000, 3, 700], 4, 1, 64, seed=5), window=window)
    _run("prefill", _low([4, 1, 4], [9000, 3, 700], 4, 1, 64, seed=5), window=window)
