"""A cache or a rotation table on another device than the call's is refused, before anything is launched."""
import ctypes as ct

import pytest

import gated_delta_ssm_gb300 as gdn

torch = pytest.importorskip("torch")

FAKE = 1 << 40      # never dereferenced
DIMS = gdn.AttnDims(n_seq=2, n_q_heads=8, n_kv_heads=2, n_pages=10, max_pages=4, n_tokens=2, max_q=1)


class _Tensor(torch.Tensor):
    """A host tensor that says it is a contiguous one on CUDA device `at`."""
    at = 0
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.at))

    def get_device(self):
        return self.at


def _t(*shape, dtype=torch.uint8, at=0):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(_Tensor)
    t.at = at
    return t


class _NoLaunch:
    def __getattr__(self, name):
        def call(*args):
            raise AssertionError(f"{name} was called")
        return call


@pytest.fixture
def on(monkeypatch):
    """Sets the current device; a call into the library fails the test."""
    def use(dev):
        monkeypatch.setattr(torch.cuda, "current_device", lambda: dev)
        gdn._load_torch()
        monkeypatch.setattr(gdn, "_current_device", lambda: dev)
        monkeypatch.setattr(gdn, "_raw_stream", lambda d: 0)
        monkeypatch.setattr(gdn, "_lib", _NoLaunch())
    return use


def _cache(at):
    f32 = torch.float32
    return gdn.KvCache(_t(10, 2, 64, 128, at=at), _t(10, 2, 64, 128, at=at), _t(10, 2, dtype=f32, at=at),
                       _t(10, 2, dtype=f32, at=at), _t(2, 4, dtype=torch.int32, at=at))


def _rope(at):
    return gdn.Rope(_t(100, 32, dtype=torch.float32, at=at), _t(100, 32, dtype=torch.float32, at=at))


def test_a_cache_of_another_device_is_refused(on):
    on(0)
    cache, rope = _cache(0), _rope(0)
    with pytest.raises(AssertionError, match="gdn_attn_decode was called"):      # accepted where it is at home
        gdn.attn_decode(FAKE, cache, FAKE, FAKE, FAKE, DIMS, workspace=_t(64))
    on(1)
    for call in (gdn.attn_decode, gdn.attn_prefill):
        with pytest.raises(ValueError, match="cache: its tensors are on cuda:0, the current device is cuda:1"):
            call(FAKE, cache, FAKE, FAKE, FAKE, DIMS, workspace=_t(64, at=1))
    k = _t(2, 2, 128, dtype=torch.bfloat16, at=1)
    with pytest.raises(ValueError, match="cache: its tensors are on cuda:0"):
        gdn.attn_append(FAKE, k, FAKE, cache, FAKE, FAKE, _rope(1), FAKE, DIMS)
    with pytest.raises(ValueError, match="rope: its tensors are on cuda:0"):
        gdn.attn_append(FAKE, k, FAKE, _cache(1), FAKE, FAKE, rope, FAKE, DIMS)


def test_the_device_is_looked_at_in_every_call(on):
    on(0)
    cache = _cache(0)
    cache._for(DIMS, 0)
    with pytest.raises(ValueError, match="cache: its tensors are on cuda:0"):
        cache._for(DIMS, 1)
    cache._for(DIMS, 0)


def test_raw_addresses_stay_unchecked(on):
    on(3)
    cache = gdn.KvCache(FAKE, FAKE, FAKE, FAKE, FAKE)
    assert ct.addressof(cache._for(DIMS, 3)._obj) == ct.addressof(cache._c)


def test_the_sizes_are_looked_at_in_every_call():
    cache = gdn.KvCache(*[FAKE] * 5)
    cache._shape = (10, 2, 64, 128, 2, 4)
    assert cache._for(DIMS) is cache._ref
    cache._shape = (10, 2, 64, 128, 2, 5)
    with pytest.raises(ValueError, match="cache: sizes"):
        cache._for(DIMS)
