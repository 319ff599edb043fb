"""gdn_attn_append against the 64-bit oracle: rotation, scales, codes, growth of a page's scale."""
import numpy as np
import pytest

from oracle import attention as oa
from tests._attn import Batch

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import gated_delta_ssm_gb300 as gdn  # noqa: E402


def _inputs(t: Batch, dtype, std=1.0, fused=False):
    rng = t.rng
    mk = lambda h: torch.from_numpy(rng.normal(0, std, (t.N, h, 128))).to(dtype).cuda()
    if not fused:
        return mk(t.Hq), mk(t.Hkv), mk(t.Hkv)
    row = torch.from_numpy(rng.normal(0, std, (t.N, (t.Hq + 2 * t.Hkv + 1) * 128))).to(dtype).cuda()
    q, k, v, _ = row.split([t.Hq * 128, t.Hkv * 128, t.Hkv * 128, 128], 1)
    return (x.unflatten(1, (-1, 128)) for x in (q, k, v))


def _run_and_check(t: Batch, q, k, v, rope, stream=None):
    qo = torch.full((t.N, t.Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    gdn.attn_append(q, k, v, t.cache(), t.d["q_start"], t.d["kv_len"], rope, qo, t.dims(), stream=stream)
    torch.cuda.synchronize()
    _check_result(t, q, k, v, rope, qo)


def _check_result(t, q, k, v, rope, qo):
    cos, sin = rope.cos.cpu().numpy(), rope.sin.cpu().numpy()
    f64 = lambda x: x.double().cpu().numpy()
    got = {n: t.d[n].cpu().numpy() for n in ("k", "v", "ks", "vs")}
    for b in range(t.B):
        n, L, r0 = t.ns[b], t.lens[b], t.q_start[b]
        pos = np.arange(L - n, L)
        at = np.maximum(pos, 0)
        want = oa.rotate(f64(q[r0:r0 + n]), at, cos, sin, rope.interleaved)
        # one rounding to bf16, and the rotation in 32 bits
        err = np.abs(f64(qo[r0:r0 + n]) - want)
        assert np.all(err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * np.abs(f64(q[r0:r0 + n])).max(initial=0))
        for codes, scales, x in (("k", "ks", oa.rotate(f64(k[r0:r0 + n]), at, cos, sin, rope.interleaved)),
                                 ("v", "vs", f64(v[r0:r0 + n]))):
            ref_c, ref_s = getattr(t, codes), getattr(t, scales)
            oa.append(ref_c, ref_s, t.table[b], x, L)
            mine = np.stack([oa.held(got[codes], got[scales], t.table[b], L, h) for h in range(t.Hkv)], 1)
            ref = np.stack([oa.held(ref_c, ref_s, t.table[b], L, h) for h in range(t.Hkv)], 1)
            if codes == "v":
                assert np.array_equal(mine, ref, equal_nan=True)
                continue
            # old tokens: the same values; new ones: half a step of e4m3, or of its smallest step
            old = max(L - n, 0)
            assert np.array_equal(mine[:old], ref[:old], equal_nan=True)
            s = np.stack([np.repeat(ref_s[t.table[b, :-(-L // t.P)], h], t.P)[:L] for h in range(t.Hkv)], 1)[old:]
            new = x[n - (L - old):] if n else x
            step = np.maximum(2.0 ** -4 * np.abs(new), 2.0 ** -10 * s[..., None])
            top = np.abs(new).max() if new.size else 0.0
            assert np.all(np.abs(mine[old:] - new) <= step + 2.0 ** -21 * top)
    # scales equal, and nothing outside the touched pages changed
    assert np.array_equal(got["ks"], t.ks) and np.array_equal(got["vs"], t.vs)
    assert np.array_equal(got["v"], t.v)
    touched = np.zeros(t.n_pages, bool)
    for b in range(t.B):
        for blk in range(max(t.lens[b] - t.ns[b], 0) // t.P, -(-t.lens[b] // t.P)):
            touched[t.table[b, blk]] = True
    assert np.array_equal(got["k"][~touched], t.k[~touched])
    assert gdn.check_device() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("P,rot,interleaved", [(16, 128, False), (32, 64, True), (64, 32, False), (128, 128, True),
                                               (64, 0, False), (32, 16, False), (16, 112, False)])
def test_append_matches_the_oracle(dtype, P, rot, interleaved):
    t = Batch([1, 5, 70, 1, 129, 2, 0], [1, 200, 70, 64, 300, 130, 40], 6, 2, P, seed=P + rot)
    rope = gdn.Rope.table(400, rot, 10000.0, interleaved) if rot else gdn.Rope(
        torch.empty(1000, 0, device="cuda"), torch.empty(1000, 0, device="cuda"))
    _run_and_check(t, *_inputs(t, dtype), rope)


@pytest.mark.parametrize("Hq,Hkv,fused", [(1, 1, False), (16, 1, True), (20, 4, True), (9, 3, False)])
def test_append_head_layouts_and_fused_rows(Hq, Hkv, fused):
    t = Batch([3, 1, 33], [3, 17, 80], Hq, Hkv, 32, seed=Hq)
    _run_and_check(t, *_inputs(t, torch.bfloat16, fused=fused), gdn.Rope.table(100, 128))


def test_a_growing_scale_moves_the_pages_codes():
    # token after token, each larger than the last: every append raises the scale of its page
    t = Batch([1, 1], [20, 33], 2, 2, 32, seed=5)
    rope = gdn.Rope.table(64, 64)
    for i in range(12):
        t.lens = [20 + i, 33 + i]
        t.d["kv_len"].copy_(torch.tensor(t.lens, dtype=torch.int32))
        if t.lens[0] > 32:
            break
        _run_and_check(t, *_inputs(t, torch.float32, std=4.0 ** i), rope)


def test_the_largest_and_smallest_values():
    t = Batch([4, 4], [4, 20], 1, 1, 16, seed=6)
    q, k, v = _inputs(t, torch.float32)
    k[0], v[0] = 3e38, -3e38
    v[1] = 1e-44
    k[4:], v[4:] = 0.0, 1e-38
    _run_and_check(t, q, k, v, gdn.Rope(torch.empty(64, 0, device="cuda"), torch.empty(64, 0, device="cuda")))


def test_values_at_the_borders_of_a_scale():
    for top in (448.0, 447.9, 448.1, 224.0, 7.0, 0.875, 0.8751):
        t = Batch([2], [2], 1, 1, 16, seed=7)
        q, k, v = _inputs(t, torch.float32)
        v.clamp_(-0.8, 0.8)
        v[1, 0, 5] = -top
        _run_and_check(t, q, k, v, gdn.Rope.table(8, 128))


def test_values_that_are_not_finite_are_reported_and_do_not_spoil_the_page():
    t = Batch([3], [19], 2, 1, 32, seed=8)
    q, k, v = _inputs(t, torch.float32)
    v[1, 0, 3], v[2, 0, 9], v[0, 0, 0] = float("inf"), float("nan"), float("-inf")
    gdn.attn_append(q, k, v, t.cache(), t.d["q_start"], t.d["kv_len"], gdn.Rope.table(32, 0 or 16),
                    torch.empty(3, 2, 128, dtype=torch.bfloat16, device="cuda"), t.dims())
    assert gdn.check_device() == 512
    oa.append(t.v, t.vs, t.table[0], v.double().cpu().numpy(), 19)
    assert np.array_equal(t.d["v"].cpu().numpy(), t.v) and np.array_equal(t.d["vs"].cpu().numpy(), t.vs)
    got = oa.held(t.v, t.vs, t.table[0], 19, 0)
    assert got[17, 3] == 448 * t.vs[t.table[0, 0], 0] and got[18, 9] == 0


def test_padding_rows_are_not_appended():
    # an idle slot (length 0), and a sequence with more rows than tokens
    t = Batch([1, 4, 1], [0, 2, 5], 2, 1, 16, seed=9)
    _run_and_check(t, *_inputs(t, torch.bfloat16), gdn.Rope.table(16, 64))


def test_keys_and_values_alone():
    t = Batch([2], [6], 2, 1, 16, seed=10)
    q, k, v = _inputs(t, torch.bfloat16)
    other = Batch([2], [6], 2, 1, 16, seed=10)
    gdn.attn_append(None, k, v, t.cache(), t.d["q_start"], t.d["kv_len"], gdn.Rope.table(16, 64), None, t.dims())
    qo = torch.empty(2, 2, 128, dtype=torch.bfloat16, device="cuda")
    gdn.attn_append(q, k, v, other.cache(), other.d["q_start"], other.d["kv_len"], gdn.Rope.table(16, 64), qo,
                    other.dims())
    torch.cuda.synchronize()
    assert all(torch.equal(t.d[n], other.d[n]) for n in ("k", "v", "ks", "vs"))


@pytest.mark.parametrize("spoil", ["page", "negative page", "len", "negative len", "starts", "rows", "max_q", "table"])
def test_bad_batch_entries_are_reported_and_skipped(spoil):
    t = Batch([2, 2, 2], [10, 20, 30], 2, 1, 16, seed=11)
    q, k, v = _inputs(t, torch.bfloat16)
    before = t.d["k"].clone()
    dims, rope = t.dims(), gdn.Rope.table(64, 64)
    if spoil == "page":
        t.d["table"][1, 1] = t.n_pages
    elif spoil == "negative page":
        t.d["table"][1, 1] = -1
    elif spoil == "len":
        t.d["kv_len"][1] = t.width * 16 + 1
    elif spoil == "negative len":
        t.d["kv_len"][1] = -1
    elif spoil == "starts":
        t.d["q_start"][1] = 5                      # sequence 1 would end before it starts
    elif spoil == "rows":
        t.d["q_start"][2:] = 1 << 30
    elif spoil == "max_q":
        dims = t.dims(max_q=1)
    else:
        rope = gdn.Rope.table(15, 64)              # positions 18 and 19 are past the table
    qo = torch.empty(6, 2, 128, dtype=torch.bfloat16, device="cuda")
    gdn.attn_append(q, k, v, t.cache(), t.d["q_start"], t.d["kv_len"], rope, qo, dims)
    assert gdn.check_device() == 256
    assert torch.equal(t.d["k"][t.table[1, 1]], before[t.table[1, 1]])


def test_append_on_another_stream_and_in_a_graph():
    t = Batch([1, 1], [9, 33], 4, 2, 16, seed=12)
    q, k, v = _inputs(t, torch.bfloat16)
    rope, side = gdn.Rope.table(64, 128), torch.cuda.Stream()
    qo = torch.empty(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    cache, dims = t.cache(), t.dims()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        gdn.attn_append(q, k, v, cache, t.d["q_start"], t.d["kv_len"], rope, qo, dims)
    g.replay()
    torch.cuda.synchronize()
    _check_result(t, q, k, v, rope, qo)
    t = Batch([1, 1], [9, 33], 4, 2, 16, seed=13)
    q, k, v = _inputs(t, torch.bfloat16)
    torch.cuda.synchronize()
    _run_and_check(t, q, k, v, rope, stream=side)


def test_codes_past_4_gib_of_cache():
    P, Hkv = 128, 8
    n_pages = (1 << 32) // (P * Hkv * 128) + 8
    k, v = (torch.zeros(n_pages, Hkv, P, 128, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(n_pages, Hkv, device="cuda") for _ in range(2))
    table = torch.tensor([[n_pages - 1]], dtype=torch.int32, device="cuda")
    x = torch.randn(2, Hkv, 128, device="cuda")
    dims = gdn.AttnDims(n_seq=1, n_q_heads=Hkv, n_kv_heads=Hkv, page_size=P, n_pages=n_pages, max_pages=1, n_tokens=2,
                        max_q=2)
    at, ln = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([0, 2], [2]))
    gdn.attn_append(None, x, x, gdn.KvCache(k, v, ks, vs, table), at, ln, gdn.Rope.table(4, 128), None, dims)
    torch.cuda.synchronize()
    held = v[-1, :, :2].view(torch.float8_e4m3fn).float() * vs[-1][:, None, None]
    assert (held.transpose(0, 1) - x).abs().max() <= 2 ** -4 * x.abs().max()
    assert not v[:-1].any() and not k[:-1].any()
