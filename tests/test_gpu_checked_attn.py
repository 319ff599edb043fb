"""The attention calls under the checked build (libgdn_checked.so, -DGDN_CHECKS), in a fresh process that loads it: no
range check fires, and the results match the oracle."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_checked_build_runs_the_attention_calls_clean():
    from gated_delta_ssm_gb300 import build as gbuild
    gbuild.build()
    r = subprocess.run([sys.executable, "-m", "tests._checked_attn_child"], cwd=ROOT,
                       env=dict(os.environ, GDN_CHECKED="1"), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "checked attention clean" in r.stdout
