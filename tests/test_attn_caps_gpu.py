"""Capped scores whose cap is far above the scores, and near them, on the GPU: the
result is the uncapped one but for z - z^3 / (3 cap^2) + ..., so its error is held to
the scores' size and not to the cap's."""
import numpy as np
import pytest
import torch

import attn_reference as R
from gpu_helpers import ensure_built
from speculative_decode_hybrid_gb300 import gdnspec as G
from attn_reference import U16, U32
from test_attn_ex_gpu import attend, slopes_of
from test_attn_gpu import f64, make
from test_attn_shared_gpu import SHAPES, Forest, plan_for, queries
from test_attn_shared_gpu import attend as attend_shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()


def expected(q, k, v, parent, n, scale, cap, slopes, bf16):
    """q [T][Hq][D], k, v [n + T][Hkv][D] in 64 bits; the result and the bound on its
    error. A score's error: its sum's, D roundings relative to sum |q_i k_i|; the
    exponential's, 2^-21; the cap's. An exponential, a reciprocal and the roundings
    between them are off by 2^-20 of the cap, which is allowed up to a cap of 128
    (1 / 16 of the half step of a bf16 weight, 2^-9). Above, where |z| is below a quarter
    of the cap, a series has half a dozen roundings relative to z, below 2^-21; where it
    is not, tanh is above 0.244 and 2^-20 of the cap are 2^-18 of the result. The bias's
    2^-21. From there as attn_reference.attention_bound."""
    T, Hq, D = q.shape
    Hk = k.shape[1]
    out, bound = np.zeros_like(q), np.zeros_like(q)
    for t in range(T):
        path = R.path_of(parent, t + 1)
        seen = np.r_[np.arange(n), [n + i - 1 for i in path]].astype(int)
        far = np.r_[n + len(path) - 1 - np.arange(n), len(path) - 1 - np.arange(len(path))]
        for h in range(Hq):
            kk, vv = k[seen, h * Hk // Hq], v[seen, h * Hk // Hq]
            z, big = scale * (kk @ q[t, h]), scale * (np.abs(kk) @ np.abs(q[t, h]))
            z = cap * np.tanh(z / cap)
            delta = 2 * (D + 2) * U32 * big + 2.0 ** -21 + min(cap, 128.0) * 2.0 ** -20 + 2.0 ** -18 * np.abs(z)
            if slopes is not None:
                bias = float(slopes[h]) * far
                delta = delta + 2.0 ** -21 * (np.abs(bias) + np.abs(z))
                z = z - bias
            p = np.exp(z - z.max())
            p /= p.sum()
            out[t, h], mass = p @ vv, p @ np.abs(vv)
            bound[t, h] = 2 * ((p * delta) @ np.abs(vv) + (p @ delta) * mass) + (4 * len(seen) * U32 + (U16 if bf16 else 0.0)) * mass
    return out, bound + (U16 if bf16 else 4 * U32) * np.abs(out) + 1e-30


def check(cache, q, parents, out, scale, cap, slopes=None):
    T = q.shape[1]
    for b, n in enumerate(cache.ctx):
        k, v = (f64(x) for x in cache.rows(b, np.arange(n + T)))
        parent = R.chain(T + 1) if parents is None else parents[b]
        want, bound = expected(f64(q[b]), k, v, parent, n, scale, cap, slopes, cache.dtype == G.GDN_BF16)
        err = np.abs(f64(out[b]) - want)
        assert np.all(err <= bound), (b, float((err / bound).max()))


CAPS = [100.0, 127.9, 128.1, 200.0, 1e3, 1e5, 1e6, 1e8, 1e30]
SIZES = [(1, 4, 2, 256, 64, False), (5, 6, 3, 64, 32, True), (22, 16, 2, 128, 16, True)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("T,h_q,h_kv,d,page,tree", SIZES)
def test_caps_above_the_scores(dtype, cap, T, h_q, h_kv, d, page, tree):
    g = np.random.default_rng(d)
    cache, q, parents = make(g, [37, 0, 300], T, h_q, h_kv, d, page, dtype, tree, spread=3.0)
    for slopes in (None, slopes_of(h_q)):
        out, st = attend(cache, q, parents, d ** -0.5, cap=cap, slopes=slopes)
        check(cache, q, parents, out, d ** -0.5, cap, slopes)
        assert st == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cap", [129.0, 200.0, 1e3])
def test_scores_of_the_caps_size(dtype, cap):
    """Scores below a quarter of the cap, above it and beyond the cap in one row."""
    g = np.random.default_rng(int(cap))
    cache, q, parents = make(g, [200, 63], 9, 8, 2, 128, 16, dtype, True, spread=0.5 * cap)
    out, st = attend(cache, q, parents, 128 ** -0.5, cap=cap)
    check(cache, q, parents, out, 128 ** -0.5, cap)
    assert st == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cap", [1e3, 1e7])
def test_large_caps_over_shared_prefixes(dtype, cap):
    g = np.random.default_rng(2)
    f = Forest(g, SHAPES["system_prompt"], 5, 2, 128, 32, dtype)
    plan, size = plan_for(f, f.dims(6))
    q = queries(g, f, 5, 6)
    parents = np.stack([R.random_tree(g, 6) for _ in f.ctx])
    out, st = attend_shared(f, q, parents, 0.1, plan, size, cap=cap)
    check(f, q, parents, out, 0.1, cap)
    assert st == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_numbers_under_a_large_cap(dtype):
    """A key that is no number in a drafted node: NaN on the paths that see it, nothing changed on the others."""
    g = np.random.default_rng(4)
    T = 22
    cache, q, parents = make(g, [100, 257], T, 4, 2, 128, 16, dtype, True)
    clean, _ = attend(cache, q, parents, 0.1, cap=1e4)
    for b, n in enumerate(cache.ctx):
        page, off = cache.where(b, [n + 6])
        cache.k[page, :, off, 3] = float("nan")
    out, st = attend(cache, q, parents, 0.1, cap=1e4)
    assert st == 0
    for b in range(2):
        for t in range(T):
            if 7 in R.path_of(parents[b], t + 1):
                assert torch.isnan(out[b, t]).all()
            else:
                assert torch.equal(out[b, t], clean[b, t])
