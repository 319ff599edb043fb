"""Refusals of the attention calls that need no GPU: the C ABI's host checks and the binding's."""
import ctypes as ct

import pytest

import gated_delta_ssm_gb300 as gdn
from gated_delta_ssm_gb300 import build as gbuild

torch = pytest.importorskip("torch")

FAKE = 1 << 40      # well aligned, never dereferenced: every call below is refused first
BAD, UNSUPPORTED = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdn.load()


def _dims(**kw):
    d = dict(n_seq=2, n_q_heads=8, n_kv_heads=2, n_pages=10, max_pages=4, n_tokens=2, max_q=1)
    d.update(kw)
    return gdn.AttnDims(**d)


def _cache(**kw):
    p = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, page_table=FAKE)
    p.update(kw)
    return gdn._CKvCache(*p.values())


def _append(lib, dims=None, cache=None, rope=None, dtype=gdn.GDN_BF16, **kw):
    p = dict(q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, starts=FAKE, lens=FAKE, qo=FAKE)
    p.update(kw)
    dims = dims or _dims()
    r = gdn._CRope(FAKE, FAKE, 100, 64, 0, 0) if rope is None else rope
    return lib.gdn_attn_append(p["q"], p["qs"], p["k"], p["ks"], p["v"], p["vs"], dtype,
                               ct.byref(cache or _cache()), p["starts"], p["lens"], ct.byref(r) if r else None,
                               p["qo"], dims._ref, None)


def _attend(lib, form, dims=None, cache=None, **kw):
    p = dict(q=FAKE, qs=1024, starts=FAKE, lens=FAKE, out=FAKE, scale=0.1, cap=0.0, window=0, ws=FAKE, nbytes=1 << 40)
    p.update(kw)
    dims = dims or _dims()
    return getattr(lib, "gdn_attn_" + form)(p["q"], p["qs"], ct.byref(cache or _cache()), p["starts"], p["lens"],
                                            p["out"], dims._ref, p["scale"], p["cap"], p["window"], p["ws"],
                                            p["nbytes"], None)


BAD_DIMS = [
    (dict(n_seq=0), BAD), (dict(n_seq=65536), BAD), (dict(n_q_heads=7), BAD), (dict(n_q_heads=0), BAD),
    (dict(n_kv_heads=0), BAD), (dict(n_pages=0), BAD), (dict(max_pages=0), BAD), (dict(n_tokens=0), BAD),
    (dict(max_q=0), BAD), (dict(head_dim=0), BAD), (dict(page_size=0), BAD),
    (dict(max_pages=1 << 25), BAD),                                  # positions past 2^30
    (dict(n_tokens=1 << 26), UNSUPPORTED),                           # 2^28 (token, head of a group) rows
    (dict(head_dim=64), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED),
    (dict(n_q_heads=34, n_kv_heads=2), UNSUPPORTED),                 # 17 q heads per KV head
]


@pytest.mark.parametrize("kw,status", BAD_DIMS)
def test_bad_dims(lib, kw, status):
    dims = _dims(**kw)
    assert _append(lib, dims, qs=1 << 20) == status
    assert _attend(lib, "decode", dims, qs=1 << 20) == status
    assert _attend(lib, "prefill", dims, qs=1 << 20) == status
    assert gdn.attn_workspace_bytes(dims) == gdn.attn_workspace_bytes(dims, True) == 0


@pytest.mark.parametrize("field", ["k", "v", "k_scale", "v_scale", "page_table"])
def test_missing_or_misaligned_cache_parts(lib, field):
    for bad in (None, FAKE + (8 if field in "kv" else 2)):
        cache = _cache(**{field: bad})
        assert _append(lib, cache=cache) == _attend(lib, "decode", cache=cache) == BAD
        assert _attend(lib, "prefill", cache=cache) == BAD


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(q=None), dict(qo=None), dict(starts=None), dict(lens=None),
    dict(k=FAKE + 8), dict(v=FAKE + 2), dict(q=FAKE + 4), dict(qo=FAKE + 8), dict(lens=FAKE + 1),
    dict(ks=255), dict(ks=260), dict(vs=128), dict(qs=1023), dict(qs=1028), dict(dtype=2),
    dict(rope=gdn._CRope(None, FAKE, 10, 64, 0, 0)), dict(rope=gdn._CRope(FAKE, FAKE + 4, 10, 64, 0, 0)),
    dict(rope=gdn._CRope(FAKE, FAKE, -1, 64, 0, 0)), dict(rope=gdn._CRope(FAKE, FAKE, 10, 144, 0, 0)),
    dict(rope=gdn._CRope(FAKE, FAKE, 10, 64, 2, 0)), dict(rope=gdn._CRope(FAKE, FAKE, 10, 64, 0, 1)),
    dict(rope=False),
])
def test_append_refuses(lib, kw):
    assert _append(lib, **kw) == BAD


def test_append_refuses_what_it_has_no_kernel_for(lib):
    assert _append(lib, rope=gdn._CRope(FAKE, FAKE, 10, 24, 0, 0)) == UNSUPPORTED


@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("kw", [
    dict(q=None), dict(out=None), dict(ws=None), dict(starts=None), dict(lens=None), dict(q=FAKE + 8),
    dict(out=FAKE + 2), dict(ws=FAKE + 8), dict(qs=1000), dict(qs=1028), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(cap=-1.0), dict(cap=float("nan")), dict(cap=float("inf")), dict(window=-1),
    dict(nbytes=0),
])
def test_attention_refuses(lib, form, kw):
    assert _attend(lib, form, **kw) == BAD


def test_decode_refuses_more_rows_than_it_takes(lib):
    dims = _dims(n_tokens=100, max_q=17)                              # 4 heads x 17 tokens > 64
    assert _attend(lib, "decode", dims) == UNSUPPORTED
    assert gdn.attn_workspace_bytes(dims) == 0 and gdn.attn_workspace_bytes(dims, True) > 0
    assert gdn.attn_workspace_bytes(_dims(n_tokens=100, max_q=16)) > 0


# ------------------------------------------------------------------ the binding
def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def _handle():
    return gdn.KvCache(FAKE, FAKE, FAKE, FAKE, FAKE)


def _rope():
    r = gdn.Rope.__new__(gdn.Rope)
    r._c = gdn._CRope(FAKE, FAKE, 100, 64, 0, 0)
    r._ref = ct.byref(r._c)
    return r


def _py_append(**kw):
    a = dict(q=FAKE, k=_t(2, 2, 128), v=FAKE, cache=_handle(), q_start=FAKE, kv_len=FAKE, rope=_rope(), q_out=FAKE,
             dims=_dims())
    a.update(kw)
    gdn.attn_append(**a)


@pytest.mark.parametrize("kw,error,text", [
    (dict(k=_t(2, 2, 128, dtype=torch.float16)), TypeError, "k: dtype torch.float16"),
    (dict(k=_t(3, 2, 128)), ValueError, "k: shape"),
    (dict(k=_t(2, 2, 256)[..., ::2]), ValueError, "k: elements of a row must be contiguous"),
    (dict(k=_t(2, 128, 2).transpose(1, 2)), ValueError, "k: elements of a row must be contiguous"),
    (dict(k=_t(2, 2, 128)), ValueError, "k: tensor is on cpu"),
    (dict(k=[1, 2]), TypeError, "k: expected a torch tensor"),
])
def test_binding_refuses_inputs(lib, kw, error, text):
    with pytest.raises(error, match=text):
        _py_append(**kw)


def test_binding_refuses_outputs_and_counts(lib):
    args = (_handle(), FAKE, FAKE)
    with pytest.raises(TypeError, match="out: dtype torch.float32"):
        gdn.attn_decode(FAKE, *args, _t(2, 8, 128, dtype=torch.float32), _dims(), workspace=_t(1))
    with pytest.raises(ValueError, match="out: rows must be dense"):
        gdn.attn_decode(FAKE, *args, _t(2, 16, 128)[:, :8], _dims(), workspace=_t(1))
    with pytest.raises(TypeError, match="q: dtype torch.float32"):
        gdn.attn_prefill(_t(2, 8, 128, dtype=torch.float32), *args, FAKE, _dims(), workspace=_t(1))
    with pytest.raises(ValueError, match="q_start: 2 entries, expected 3"):
        gdn.attn_decode(FAKE, _handle(), _t(2, dtype=torch.int32), FAKE, FAKE, _dims(), workspace=_t(1))
    with pytest.raises(TypeError, match="kv_len: dtype torch.int64"):
        gdn.attn_decode(FAKE, _handle(), FAKE, _t(2, dtype=torch.int64), FAKE, _dims(), workspace=_t(1))


def test_binding_refuses_a_cache_of_other_sizes():
    with pytest.raises(TypeError, match="cache.k: dtype torch.bfloat16"):
        gdn.KvCache(_t(1, 2, 64, 128), FAKE, FAKE, FAKE, FAKE)
    with pytest.raises(ValueError, match="cache.k: tensor is on cpu"):
        gdn.KvCache(_t(1, 2, 64, 128, dtype=torch.uint8), FAKE, FAKE, FAKE, FAKE)
    c = _handle()
    c._shape = (10, 2, 64, 128, 2, 4)
    c._for(_dims())
    with pytest.raises(ValueError, match="cache: sizes"):
        c._for(_dims(n_pages=11))
