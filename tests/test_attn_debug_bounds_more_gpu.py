"""More of the attention-layer, page and sampling tests through the
bounds-checking build (see test_attn_debug_bounds_gpu.py)."""
import os
import subprocess
import sys

import pytest
import torch

from speculative_decode_hybrid_gb300 import build as B

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_more_calls_stay_in_bounds():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    env = dict(os.environ, GDNSPEC_LIB=B.build(debug=True))
    files = [os.path.join(ROOT, "tests", f) for f in ("test_attn_values_gpu.py", "test_sample_pages_more_gpu.py", "test_hybrid_parts_gpu.py")]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", *files], cwd=ROOT, env=env, capture_output=True, text=True,
                       timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
