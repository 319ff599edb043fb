"""A rotation table without positions is refused: a padding row would read its position 0."""
import ctypes as ct

import pytest

import gated_delta_ssm_gb300 as gdn
from gated_delta_ssm_gb300 import build as gbuild

FAKE = 1 << 40      # well aligned, never dereferenced: a call that passes the checks fails at the launch, without a GPU


def _append(n_positions, rotary_dim):
    gbuild.build()
    dims = gdn.AttnDims(n_seq=2, n_q_heads=8, n_kv_heads=2, n_pages=10, max_pages=4, n_tokens=2, max_q=1)
    cache = gdn._CKvCache(*[FAKE] * 5)
    rope = gdn._CRope(FAKE, FAKE, n_positions, rotary_dim, 0, 0)
    return gdn.load().gdn_attn_append(FAKE, 1024, FAKE, 256, FAKE, 256, gdn.GDN_BF16, ct.byref(cache), FAKE, FAKE,
                                      ct.byref(rope), FAKE, dims._ref, None)


@pytest.mark.parametrize("rotary_dim", [16, 64, 128])
def test_no_positions_to_rotate_by(rotary_dim):
    assert _append(0, rotary_dim) == gdn.GDN_ERR_INVALID_ARG
