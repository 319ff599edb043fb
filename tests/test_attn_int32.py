"""Sizes and windows past 32 bits reach the library as what they mean, or not at all: ctypes would wrap them."""
import ctypes as ct

import pytest

import gated_delta_ssm_gb300 as gdn

pytest.importorskip("torch")

FAKE = 1 << 40      # never dereferenced
DIMS = dict(n_seq=2, n_q_heads=8, n_kv_heads=2, n_pages=10, max_pages=4, n_tokens=2, max_q=1)


@pytest.mark.parametrize("field", [*DIMS, "head_dim", "page_size"])
@pytest.mark.parametrize("value", [(1 << 32) + 1, 1 << 31, -(1 << 32) + 1])
def test_sizes(field, value):
    with pytest.raises(ValueError, match=f"{field}: {value} "):
        gdn.AttnDims(**{**DIMS, field: value})


@pytest.mark.parametrize("window,passed", [(0, 0), (7, 7), ((1 << 31) - 1, (1 << 31) - 1), (1 << 31, (1 << 31) - 1),
                                           ((1 << 32) + 5, (1 << 31) - 1), (-1, -1), (-(1 << 32) + 5, -1)])
def test_windows(monkeypatch, window, passed):
    got = []

    class Lib:
        def __getattr__(self, name):
            return lambda *args: got.append(ct.c_int32(args[9]).value) or 0

    class Workspace:
        is_contiguous = lambda self: True
        get_device = lambda self: 0
        data_ptr = numel = element_size = lambda self: 16

    gdn._load_torch()
    monkeypatch.setattr(gdn, "_current_device", lambda: 0)
    monkeypatch.setattr(gdn, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(gdn, "_lib", Lib())
    cache = gdn.KvCache(*[FAKE] * 5)
    for call in (gdn.attn_decode, gdn.attn_prefill):
        call(FAKE, cache, FAKE, FAKE, FAKE, gdn.AttnDims(**DIMS), window=window, workspace=Workspace())
    assert got == [passed, passed]
