"""A q row that holds a NaN or an infinity gives NaN in every dimension of its output, whatever the score cap, and
leaves the other rows right; a row that sees nothing gives zeros whatever its q holds."""
import numpy as np
import pytest

from tests._attn import Batch, check

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import gated_delta_ssm_gb300 as gdn  # noqa: E402

SCALE = 128 ** -0.5
CALLS = {"decode": gdn.attn_decode, "prefill": gdn.attn_prefill}


def _attend(form, t, q, **kw):
    out = torch.full((t.N, t.Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    CALLS[form](q, t.cache(), t.d["q_start"], t.d["kv_len"], out, t.dims(), scale=SCALE, **kw)
    torch.cuda.synchronize()
    assert gdn.check_device() == 0
    return out


@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("softcap", [0.0, 1e-7, 1e-3, 30.0, 50.0, 100.0])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("Hq,Hkv,window", [(4, 2, 0), (16, 1, 70)])
def test_rows_that_are_not_finite(form, softcap, bad, Hq, Hkv, window):
    # drafts in 3 sequences, the first long enough to be shared out, the last with a padding row
    t = Batch([4, 2, 3], [3000, 130, 2], Hq, Hkv, 32, seed=Hq)
    t.make_q()
    want, bound = t.expected(SCALE, softcap, window)
    q = t.q.clone()
    rows = [(0, 0, 5), (3, Hq - 1, 127), (5, 1, 64), (8, 0, 0)]
    for row, head, d in rows:
        q[row, head, d] = bad
    q[6, 2, 9] = bad                  # the padding row
    got = _attend(form, t, q, softcap=softcap, window=window)
    hit = np.zeros((t.N, Hq), bool)
    for row, head, _ in rows:
        hit[row, head] = True
    hit = torch.from_numpy(hit).cuda()
    assert torch.isnan(got[hit]).all()
    rest = ~hit.cpu().numpy()
    check(got[~hit], want[rest], bound[rest])
    assert not got[6].any()


@pytest.mark.parametrize("softcap", [0.0, 30.0, 100.0])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_of_prompts_that_are_not_finite(softcap, bad):
    t = Batch([600, 90], [600, 400], 4, 2, 64, seed=2)
    t.make_q()
    want, bound = t.expected(SCALE, softcap)
    q = t.q.clone()
    hit = torch.zeros(t.N, t.Hq, dtype=torch.bool, device="cuda")
    hit[::37, 1] = True
    hit[0, 2] = hit[599, 3] = hit[600, 0] = True
    q[..., 77][hit] = bad
    got = _attend("prefill", t, q, softcap=softcap)
    assert torch.isnan(got[hit]).all()
    rest = ~hit.cpu().numpy()
    check(got[~hit], want[rest], bound[rest])
