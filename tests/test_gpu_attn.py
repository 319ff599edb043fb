"""gdn_attn_decode and gdn_attn_prefill against the 64-bit oracle."""
import numpy as np
import pytest

from tests._attn import Batch, check

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import gated_delta_ssm_gb300 as gdn  # noqa: E402

CALLS = {"decode": gdn.attn_decode, "prefill": gdn.attn_prefill}
SCALE = 128 ** -0.5


def _attend(form, t, q=None, scale=SCALE, dims=None, stream=None, **kw):
    q = t.q if q is None else q
    out = torch.full((t.N, t.Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    dims = dims or t.dims()
    # a workspace of NaN: nothing may depend on what it held
    ws = torch.full((gdn.attn_workspace_bytes(dims, form == "prefill"),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    CALLS[form](q, t.cache(), t.d["q_start"], t.d["kv_len"], out, dims, scale=scale, workspace=ws, stream=stream, **kw)
    torch.cuda.synchronize()
    return out


def _run(form, t, scale=SCALE, std=1.0, **kw):
    t.make_q(std)
    out = _attend(form, t, scale=scale, **kw)
    assert gdn.check_device() == 0
    check(out, *t.expected(scale, **kw))


LENS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 400, 513]


@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (6, 2), (16, 1), (8, 4)])
def test_one_token_at_every_kind_of_length(form, P, Hq, Hkv):
    _run(form, Batch([1] * len(LENS), LENS, Hq, Hkv, P, seed=P + Hq))


@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("n,Hq,Hkv", [(2, 10, 2), (4, 16, 1), (8, 8, 1), (64, 1, 1), (3, 14, 2), (7, 9, 1)])
def test_drafts_of_several_tokens(form, n, Hq, Hkv):
    # ragged: fewer tokens than max_q, as many tokens as the sequence has, none at all
    ns = [n, 1, max(1, n - 1), n, 0, n]
    lens = [n, 300, 129 + n, 128, 77, 257]
    _run(form, Batch(ns, lens, Hq, Hkv, 32, seed=n))


@pytest.mark.parametrize("n,Hq,Hkv,P", [(100, 4, 2, 16), (128, 2, 2, 64), (129, 3, 1, 32), (257, 16, 2, 128), (300, 5, 1, 64),
                                        (33, 16, 1, 16)])
def test_prompts(n, Hq, Hkv, P):
    ns = [n, n // 2 + 1, 1, n - 1]
    lens = [n, n // 2 + 1 + 130, 200, n + 383]
    _run("prefill", Batch(ns, lens, Hq, Hkv, P, seed=n))


@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("window", [1, 2, 100, 128, 129, 1000, 2 ** 31 - 1])
def test_sliding_windows(form, window):
    _run(form, Batch([4, 1, 4], [600, 129, 4], 8, 2, 64, seed=window % 1000), window=window)


@pytest.mark.parametrize("window", [1, 60, 128, 300])
def test_sliding_windows_of_prompts(window):
    _run("prefill", Batch([257, 40], [600, 40], 4, 1, 32, seed=window), window=window)


@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("softcap,std", [(30.0, 1.0), (5.0, 4.0), (1e-3, 1.0), (1e30, 0.5)])
def test_softcap(form, softcap, std):
    _run(form, Batch([2, 1], [300, 77], 8, 2, 32, seed=3), softcap=softcap, std=std)


@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("scale,std", [(0.0, 1.0), (-SCALE, 1.0), (1.0, 1.0), (SCALE, 1e-30), (SCALE, 30.0), (1e-30, 1e30)])
def test_scales_of_scores(form, scale, std):
    _run(form, Batch([2, 1], [300, 77], 8, 2, 32, seed=4), scale=scale, std=std)


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_one_key_holds_almost_all_of_the_weight(form):
    # the first key scores far above thousands of others, whose weights are small but many
    t = Batch([2], [6000], 4, 1, 64, seed=5)
    t.make_q()
    page = t.table[0, 0]
    t.k[:, 0] = 0
    t.k[page, 0, 0] = 0x38                       # 1.0 in every dimension
    t.ks[:] = 1.0
    t.q.fill_(10.0 / 128 / SCALE)                # score 10 for the first key, 0 for the others
    t.d["k"].copy_(torch.from_numpy(t.k)), t.d["ks"].copy_(torch.from_numpy(t.ks))
    out = _attend(form, t)
    check(out, *t.expected(SCALE))


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_scores_that_keep_rising(form):
    # every tile's largest score is above all before it
    t = Batch([1, 3], [1500, 900], 2, 1, 32, seed=6)
    for b in range(2):
        for blk in range(-(-t.lens[b] // 32)):
            t.ks[t.table[b, blk]] = 2.0 ** min(3, blk // 6 - 5)
            t.vs[t.table[b, blk]] = 2.0 ** (blk % 40 - 20)
    t.d["ks"].copy_(torch.from_numpy(t.ks)), t.d["vs"].copy_(torch.from_numpy(t.vs))
    t.k &= 0x7f
    t.k[t.k == 0x7f] = 0
    t.d["k"].copy_(torch.from_numpy(t.k))
    t.make_q()
    t.q.abs_()
    check(_attend(form, t), *t.expected(SCALE))


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_rows_that_see_nothing_give_zeros(form):
    t = Batch([1, 3, 1, 2], [0, 1, 40, 0], 4, 2, 16, seed=7)
    t.make_q()
    out = _attend(form, t)
    check(out, *t.expected(SCALE))
    assert not out[:3].any() and not out[5:].any()
    assert gdn.check_device() == 0


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_one_sequence_split_over_the_whole_gpu(form):
    _run(form, Batch([1], [40000], 8, 1, 64, seed=8))
    _run(form, Batch([4, 4, 1], [9000, 100, 17000], 8, 2, 16, seed=9))


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_many_short_sequences(form):
    rng = np.random.default_rng(10)
    lens = rng.integers(0, 60, 700).tolist()
    _run(form, Batch([1] * 700, lens, 2, 1, 16, seed=10))


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_results_do_not_depend_on_the_rest_of_the_batch_or_the_run(form):
    t = Batch([2, 2, 2], [500, 90, 3000], 8, 2, 32, seed=11)
    t.make_q()
    assert torch.equal(_attend(form, t), _attend(form, t))


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_q_rows_of_a_wider_array(form):
    t = Batch([2, 1], [70, 30], 6, 2, 16, seed=12)
    t.make_q()
    wide = torch.full((t.N, (t.Hq + 3) * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 128:-256] = t.q.flatten(1)
    q = wide[:, 128:-256].unflatten(1, (t.Hq, 128))
    assert torch.equal(_attend(form, t), _attend(form, t, q=q))


@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("spoil", ["page", "negative page", "len", "negative len", "starts", "rows", "max_q"])
def test_bad_batch_entries_are_reported_and_skipped(form, spoil):
    t = Batch([2, 2, 2], [100, 200, 300], 4, 2, 16, seed=13)
    t.make_q()
    want, bound = t.expected(SCALE)
    dims = t.dims()
    skipped = slice(2, 4)
    if spoil == "page":
        t.d["table"][1, 3] = t.n_pages
    elif spoil == "negative page":
        t.d["table"][1, 3] = -5
    elif spoil == "len":
        t.d["kv_len"][1] = t.width * 16 + 1
    elif spoil == "negative len":
        t.d["kv_len"][1] = -1
    elif spoil == "starts":
        t.d["q_start"][1] = 5
        skipped = slice(0, 4)
    elif spoil == "rows":
        t.d["q_start"][2:] = 1 << 30
        skipped = slice(2, 6)
    else:
        dims = t.dims(max_q=1)
        skipped = slice(0, 6)
    out = _attend(form, t, dims=dims)
    assert gdn.check_device() == 256
    if "page" in spoil:                           # the page's 16 tokens are not seen
        P, page = t.P, t.table[1, 3]
        got = out[2:4].double().cpu().numpy()
        keep = np.r_[0:48, 64:200]
        from oracle import attention as oa
        for h in range(2):
            k, v = (oa.held(c, s, t.table[1], 200, h)[keep] for c, s in ((t.k, t.ks), (t.v, t.vs)))
            o, mass, size = oa.attend(t.q[2:4, 2 * h:2 * h + 2].double().cpu().numpy(), k, v, SCALE)
            lim = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16 * (1 + size[..., None])) * mass
            assert np.all(np.abs(got[:, 2 * h:2 * h + 2] - o) <= lim)
    else:
        assert torch.all(out[skipped] == 7.0)
    rest = np.ones(t.N, bool)
    rest[skipped] = False
    check(out[torch.from_numpy(rest).cuda()], want[rest], bound[rest])


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_another_stream_and_a_graph(form):
    t = Batch([1, 2], [3000, 200], 8, 2, 64, seed=14)
    t.make_q()
    want = _attend(form, t)
    side = torch.cuda.Stream()
    assert torch.equal(_attend(form, t, stream=side), want)
    out = torch.zeros_like(want)
    cache, dims = t.cache(), t.dims()
    ws = torch.empty(gdn.attn_workspace_bytes(dims, form == "prefill"), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        CALLS[form](t.q, cache, t.d["q_start"], t.d["kv_len"], out, dims, workspace=ws)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    # the graph follows the lengths on the device
    t.lens = [2000, 111]
    t.kv_len[:] = t.lens
    t.d["kv_len"].copy_(torch.from_numpy(t.kv_len))
    g.replay()
    torch.cuda.synchronize()
    check(out, *t.expected(SCALE))


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_pages_past_4_gib_of_cache(form):
    P, Hkv = 128, 8
    far = (1 << 32) // (P * Hkv * 128) + 8
    small = Batch([2], [300], 16, Hkv, P, seed=15, extra_pages=0, slack=0)
    small.make_q()
    want = _attend(form, small)
    k, v = (torch.full((far + 3, Hkv, P, 128), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((far + 3, Hkv), float("nan"), device="cuda") for _ in range(2))
    for big, name in ((k, "k"), (v, "v"), (ks, "ks"), (vs, "vs")):
        big[far:] = small.d[name]
    cache = gdn.KvCache(k, v, ks, vs, small.d["table"] + far)
    out = torch.empty_like(want)
    dims = small.dims(n_pages=far + 3)
    CALLS[form](small.q, cache, small.d["q_start"], small.d["kv_len"], out, dims)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
