"""Values that are no numbers, compared in full with the plain form: a drafted
node's infinities and NaN reach the paths that see the node and no other row,
column or tile, in calls of one and of two blocks of rows, over contexts whose
drafted slots lie in one tile, across two, and in a split piece."""
import numpy as np
import pytest
import torch

import attn_reference as R
from gpu_helpers import ensure_built
from test_attn_gpu import attend, f64, make
from speculative_decode_hybrid_gb300 import gdnspec as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()


def check_all(cache, q, parents, out, scale):
    """Numbers within their bounds, and what is none where the plain form has it."""
    B, T, _, d = q.shape
    some = 0
    for b, n in enumerate(cache.ctx):
        k, v = (f64(x) for x in cache.rows(b, np.arange(n + T)))
        parent = R.chain(T + 1) if parents is None else parents[b]
        with np.errstate(invalid="ignore"):
            want, mass, big = R.attention(f64(q[b]), k, v, parent, n, scale)
            bound = R.attention_bound(want, mass, big, d, n + T, cache.dtype == G.GDN_BF16)
        got, fine = f64(out[b]), np.isfinite(want)
        some += np.count_nonzero(~fine)
        assert np.all(np.abs(got[fine] - want[fine]) <= bound[fine]), b
        np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
        np.testing.assert_array_equal(got[np.isinf(want)], want[np.isinf(want)])
        assert np.isfinite(got).sum() == fine.sum()
    return some


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,h_q,h_kv,n,page", [
    (20, 16, 2, 50, 16),      # 160 rows
    (20, 16, 2, 3001, 16),    # ... in pieces
    (12, 4, 2, 120, 32),      # 24 rows, drafted slots in two tiles
    (12, 4, 2, 2999, 64),
    (40, 6, 2, 0, 16),        # 120 rows, nothing committed
    (64, 8, 2, 700, 256)])    # 256 rows
def test_values_that_are_no_numbers(dtype, d, T, h_q, h_kv, n, page):
    g = np.random.default_rng(T * d + n)
    cache, q, _ = make(g, [n, 33], T, h_q, h_kv, d, page, dtype, True)
    parents = np.stack([R.random_tree(g, T + 1, 0.3) for _ in range(2)])
    bad = [(2, 0, "inf"), (3, 5, "-inf"), (3, 4, "nan"), (7, 5, "inf"), (9, d - 1, "nan"), (10, 63, "-inf"), (11, 8, "inf"),
           (T, 7, "nan"), (T, d - 2, "inf")]
    for b, base in enumerate(cache.ctx):
        for node, col, x in bad[b:]:
            at, off = cache.where(b, [base + node - 1])
            cache.v[at, :, off, col] = float(x)
    out, st = attend(cache, q, parents, d ** -0.5)
    assert check_all(cache, q, parents, out, d ** -0.5) > 0 and int(st.item()) == 0
    # a drafted key that is no number spoils the rows that see it, whole
    at, off = cache.where(0, [n + 6 - 1])
    cache.k[at, :, off, 3] = float("nan")
    out, st = attend(cache, q, parents, d ** -0.5)
    check_all(cache, q, parents, out, d ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,h_q", [(1, 4), (6, 4), (33, 16)])
def test_committed_values_that_are_no_numbers_reach_every_row(dtype, T, h_q):
    g = np.random.default_rng(T)
    cache, q, parents = make(g, [200, 90], T, h_q, 2, 128, 16, dtype, T > 1)
    for slot, col, x in ((17, 9, "nan"), (88, 70, "inf")):
        at, off = cache.where(1, [slot])
        cache.v[at, :, off, col] = float(x)
    out, st = attend(cache, q, parents, 0.1)
    assert check_all(cache, q, parents, out, 0.1) == 2 * T * h_q and int(st.item()) == 0
