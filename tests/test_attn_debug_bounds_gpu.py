"""The attention-layer, cache-page and sampled-acceptance tests through the
bounds-checking build: every access that would fall outside its buffer sets
GDN_DEV_BOUNDS, and those tests want a status word without it."""
import os
import subprocess
import sys

import pytest
import torch

from speculative_decode_hybrid_gb300 import build as B

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_new_calls_stay_in_bounds():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    lib = B.build(debug=True)
    env = dict(os.environ, GDNSPEC_LIB=lib)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-k", "not far_into and not full_vocabulary",
                        os.path.join(ROOT, "tests", "test_attn_gpu.py"), os.path.join(ROOT, "tests", "test_sample_pages_gpu.py")],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
