"""The attention workspace can be sized once: for the longest draft, whatever the tokens of the call."""
import pytest

import gated_delta_ssm_gb300 as gdn
from gated_delta_ssm_gb300 import build as gbuild


@pytest.fixture(scope="module", autouse=True)
def _built():
    gbuild.build()


def _bytes(G, max_q, prefill=False, n_tokens=4096, n_seq=2):
    return gdn.attn_workspace_bytes(gdn.AttnDims(n_seq=n_seq, n_q_heads=2 * G, n_kv_heads=2, n_pages=10, max_pages=4,
                                                 n_tokens=n_tokens, max_q=max_q), prefill)


@pytest.mark.parametrize("G", range(1, 17))
def test_a_longer_draft_never_needs_less(G):
    sizes = [_bytes(G, n) for n in range(1, 64 // G + 1)]
    assert sizes[0] > 0 and sizes == sorted(sizes)
    assert _bytes(G, 64 // G + 1) == 0
    assert len({_bytes(G, n, True) for n in (1, 2, 100, 4096)}) == 1


@pytest.mark.parametrize("G,max_q", [(1, 1), (1, 64), (4, 3), (8, 8), (16, 4), (5, 12)])
def test_the_size_does_not_depend_on_the_tokens_or_the_sequences(G, max_q):
    for prefill in (False, True):
        want = _bytes(G, max_q, prefill)
        for n_tokens in (1, 2, 7, 100000):
            for n_seq in (1, 300):
                assert _bytes(G, max_q, prefill, n_tokens, n_seq) == want


def test_dims_sized_for_any_draft_serve_a_call_of_few_tokens():
    # max_q beyond what a decode takes is accepted where the call has few tokens in all
    assert _bytes(8, 100, n_tokens=8) == _bytes(8, 8)
    assert _bytes(8, 100, n_tokens=9) == 0
