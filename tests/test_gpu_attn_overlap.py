"""q_start entries that run backwards, so that many valid sequences share the same rows: their blocks and tiles are
more than 32 bits count. The call reports the entries and ends without touching anything."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import gated_delta_ssm_gb300 as gdn  # noqa: E402


@pytest.mark.parametrize("n_seq", [131, 200, 256, 280])      # counted by one warp, and by the whole CTA
def test_more_work_than_the_rows_can_hold_is_not_started(n_seq):
    # each even sequence: 65536 tokens of 16 heads behind a million, 32 million pairs of row block and key tile
    N, L, P = 65536, 1 << 20, 128
    dev = "cuda"
    codes = [torch.zeros(1, 1, P, 128, dtype=torch.uint8, device=dev) for _ in range(2)]
    scales = [torch.ones(1, 1, device=dev) for _ in range(2)]
    table = torch.zeros(n_seq, L // P, dtype=torch.int32, device=dev)
    cache = gdn.KvCache(*codes, *scales, table)
    starts = torch.zeros(n_seq + 1, dtype=torch.int32, device=dev)
    starts[1::2] = N
    lens = torch.full((n_seq,), L, dtype=torch.int32, device=dev)
    dims = gdn.AttnDims(n_seq=n_seq, n_q_heads=16, n_kv_heads=1, page_size=P, n_pages=1, max_pages=L // P, n_tokens=N,
                        max_q=N)
    q = torch.zeros(N, 16, 128, dtype=torch.bfloat16, device=dev)
    out = torch.full_like(q, 7.0)
    gdn.attn_prefill(q, cache, starts, lens, out, dims)
    assert gdn.check_device() == 256
    assert bool((out == 7.0).all())
