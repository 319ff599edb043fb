"""Score caps and scales at the ends of the ranges that the calls accept."""
import pytest

from tests._attn import Batch, check

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import gated_delta_ssm_gb300 as gdn  # noqa: E402

SCALE = 128 ** -0.5


def _run(form, scale=SCALE, std=1.0, zero_rows=(), **kw):
    t = Batch([2, 1], [300, 77], 8, 2, 32, seed=4)
    t.make_q(std)
    for r in zero_rows:
        t.q[r] = 0
    out = torch.full((t.N, t.Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    (gdn.attn_decode if form == "decode" else gdn.attn_prefill)(
        t.q, t.cache(), t.d["q_start"], t.d["kv_len"], out, t.dims(), scale=scale, **kw)
    torch.cuda.synchronize()
    assert gdn.check_device() == 0
    check(out, *t.expected(scale, **kw))


@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("softcap", [1.5e-45, 1e-39, 1e-30, 1e-7, 55.4, 55.5, 1e20, 2.9e38, 3e38])
def test_caps(form, softcap):
    _run(form, softcap=softcap, zero_rows=(1,))


@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("scale,std", [(3e38, 1e-36), (-3e38, 1e-36), (1e-38, 1e38 / 8), (0.0, 1e30)])
def test_scales(form, softcap, scale, std):
    _run(form, scale=scale, std=std, softcap=softcap, zero_rows=(1,))
