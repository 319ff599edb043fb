"""Bounded waits of the attention kernels: a wait that runs out is reported, and the next call is correct.

The limit of each CTA's first wait for keys is set to 1 ns through the test hook of include/gdn_testing.h. The
kernels must set their bit of the device error word, let their copies and products end, free their tensor
memory and return. The waits end by their own limits: nothing here faults or hangs the GPU.
"""
import pytest

from tests._attn import Batch, check

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import gated_delta_ssm_gb300 as gdn  # noqa: E402

BIT_ATTN_WAIT = 1024


@pytest.mark.parametrize("form,ns,lens,Hq", [
    ("decode", [1, 1, 1], [300, 2000, 64], 4), ("decode", [4, 4], [700, 90], 8), ("decode", [8, 8], [700, 3000], 8),
    ("prefill", [300, 40], [300, 900], 4),
])
def test_wait_expiry_is_reported_and_the_next_call_is_correct(form, ns, lens, Hq):
    call = gdn.attn_decode if form == "decode" else gdn.attn_prefill
    t = Batch(ns, lens, Hq, 1, 32, seed=len(lens) + Hq)
    t.make_q()
    want, bound = t.expected(128 ** -0.5)
    out = torch.zeros(t.N, t.Hq, 128, dtype=torch.bfloat16, device="cuda")
    args = (t.q, t.cache(), t.d["q_start"], t.d["kv_len"], out, t.dims())
    assert gdn.check_device() == 0
    gdn.testing_set_first_wait_ns(1)
    try:
        call(*args)
        code = gdn.check_device()
    finally:
        gdn.testing_set_first_wait_ns(0)
    assert code == BIT_ATTN_WAIT
    call(*args)
    torch.cuda.synchronize()
    assert gdn.check_device() == 0
    check(out, want, bound)
