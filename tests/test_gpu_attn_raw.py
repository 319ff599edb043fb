"""Raw device addresses in place of tensors, with the binding's own workspace."""
import pytest

from tests._attn import Batch, check

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import gated_delta_ssm_gb300 as gdn  # noqa: E402


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_every_argument_may_be_an_address(form):
    t = Batch([1, 2], [300, 200], 8, 2, 64, seed=2)
    t.make_q()
    out = torch.full((t.N, t.Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    cache = gdn.KvCache(*(t.d[n].data_ptr() for n in ("k", "v", "ks", "vs", "table")))
    (gdn.attn_decode if form == "decode" else gdn.attn_prefill)(
        t.q.data_ptr(), cache, t.d["q_start"].data_ptr(), t.d["kv_len"].data_ptr(), out.data_ptr(), t.dims())
    torch.cuda.synchronize()
    check(out, *t.expected(128 ** -0.5))
    assert gdn.check_device() == 0
