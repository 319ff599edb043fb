"""A sequence's results in whatever company: alone, among others (which moves the borders of the CTAs' shares, so sums
are joined in another order), beside calls on other streams and from other host threads."""
import threading

import pytest

from tests._attn import Batch, check

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import gated_delta_ssm_gb300 as gdn  # noqa: E402

SCALE = 128 ** -0.5
CALLS = {"decode": gdn.attn_decode, "prefill": gdn.attn_prefill}


@pytest.mark.parametrize("form,n", [("decode", 1), ("decode", 8), ("prefill", 2), ("prefill", 300)])
def test_the_rest_of_the_batch(form, n):
    others = [(n, 5000), (1, 17), (n, n), (n, 20000), (1, 0), (n, 600)]
    t = Batch([n] + [o[0] for o in others], [4000] + [o[1] for o in others], 8, 2, 32, seed=n)
    t.make_q()
    want, bound = t.expected(SCALE)
    cache, q, table = t.cache(), t.q, t.d["table"]
    for company in ([0], [0, 1], [2, 0], [0, 3, 4, 5], list(range(7)), [6, 5, 4, 3, 2, 1, 0] * 20):
        rows = torch.cat([torch.arange(t.q_start[b], t.q_start[b + 1]) for b in company]).cuda()
        starts = torch.tensor([0] + [t.ns[b] for b in company]).cumsum(0).int().cuda()
        some = gdn.KvCache(cache.k, cache.v, cache.k_scale, cache.v_scale, table[company].contiguous())
        lens = torch.tensor([t.lens[b] for b in company], dtype=torch.int32, device="cuda")
        out = torch.full((len(rows), 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        dims = t.dims(n_seq=len(company), n_tokens=len(rows))
        CALLS[form](q[rows], some, starts, lens, out, dims)
        torch.cuda.synchronize()
        assert gdn.check_device() == 0
        check(out, want[rows.cpu()], bound[rows.cpu()])


def _batches():
    for i, (form, ns, lens) in enumerate([("decode", [1] * 8, [9000 + 700 * b for b in range(8)]),
                                          ("prefill", [700, 90], [700, 5000]), ("decode", [8, 3], [30000, 40]),
                                          ("prefill", [1500], [2500])]):
        t = Batch(ns, lens, 8, 2, 64, seed=i)
        t.make_q()
        out = torch.zeros(t.N, 8, 128, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(gdn.attn_workspace_bytes(t.dims(), form == "prefill"), dtype=torch.uint8, device="cuda")
        yield t, out, (t.q, t.cache(), t.d["q_start"], t.d["kv_len"], out, t.dims()), CALLS[form], ws


def test_calls_in_flight_on_several_streams():
    work = list(_batches())
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    for _ in range(20):
        for (_, _, args, call, ws), s in zip(work, streams):
            call(*args, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert gdn.check_device() == 0
    for t, out, *_ in work:
        check(out, *t.expected(SCALE))


def test_calls_from_several_host_threads():
    work = list(_batches())
    torch.cuda.synchronize()
    failed = []

    def run(args, call):
        try:
            stream = torch.cuda.Stream()
            for _ in range(20):
                call(*args, stream=stream)      # each with a workspace of its own
            stream.synchronize()
        except Exception as e:                  # reported by the main thread
            failed.append(e)

    threads = [threading.Thread(target=run, args=(args, call)) for _, _, args, call, _ in work]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not failed and gdn.check_device() == 0
    for t, out, *_ in work:
        check(out, *t.expected(SCALE))
