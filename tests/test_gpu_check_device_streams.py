"""gdn_check_device waits for work on every stream, those that do not wait for the default stream among them."""
import pytest

from tests._attn import Batch

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import gated_delta_ssm_gb300 as gdn  # noqa: E402


@pytest.mark.parametrize("call", ["append", "decode", "prefill"])
def test_an_error_of_a_call_still_queued_on_another_stream(call):
    t = Batch([2, 2], [100, 200], 4, 2, 16, seed=1)
    t.make_q()
    t.d["table"][1, 12] = t.n_pages          # the page of the last tokens is outside the cache
    out, cache, rope = torch.empty_like(t.q), t.cache(), gdn.Rope.table(200, 64)
    k, v = (torch.randn(t.N, 2, 128, device="cuda").bfloat16() for _ in range(2))
    ws = torch.empty(gdn.attn_workspace_bytes(t.dims(), True), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()

    def run():
        if call == "append":
            gdn.attn_append(None, k, v, cache, t.d["q_start"], t.d["kv_len"], rope, None, t.dims())
        else:
            (gdn.attn_decode if call == "decode" else gdn.attn_prefill)(
                t.q, cache, t.d["q_start"], t.d["kv_len"], out, t.dims(), workspace=ws)

    run()                                    # a kernel's first launch may wait for the device by itself
    torch.cuda.synchronize()
    assert gdn.check_device() == 256 and gdn.check_device() == 0
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)       # some 50 ms
        run()
    try:
        assert gdn.check_device() == 256
    finally:
        torch.cuda.synchronize()
        gdn.check_device()
