"""Sampled acceptance of single requests, whose probabilities need no margin, and
page tables of thousands of entries."""
import numpy as np
import pytest
import torch

import attn_reference as R
from gpu_helpers import ensure_built
from test_sample_pages_gpu import accept, dev, dims_of, inputs
from speculative_decode_hybrid_gb300 import gdnspec as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("N,V", [(2, 1), (2, 33), (23, 4097), (65, 3001), (65, 20011)])
def test_single_requests(drawn, tree, N, V):
    """Each seed's probabilities of drafted tokens are compared whatever the walk
    did, and the walk wherever no decision was closer than f32's rounding."""
    sure = 0
    for seed in range(8):
        g = np.random.default_rng(1000 * N + V + seed)
        logits, q, tokens, parent, temperature, u, noise = inputs(g, 1, N, V, tree, drawn)
        ints, prob, st = accept(logits, q, tokens, parent if tree else None, temperature, u, noise, shift=seed & 1)
        T = float(temperature[0])
        length, node, token, want, margin = R.sample(logits[0], None if q is None else q[0].astype(np.float64), tokens[0], parent[0], T,
                                                     u[0].astype(np.float64), noise[0].astype(np.float64))
        rel = R.prob_bound(logits[0], T, V)
        assert st == 0
        np.testing.assert_allclose(prob[0, 1:], want[1:], rtol=rel, atol=1e-37)
        if margin > 1e-4:
            sure += 1
            assert (int(ints[0, 0]), int(ints[1, 0]), int(ints[2, 0])) == (length, node, token), (seed, margin)
            np.testing.assert_allclose(prob[0, 0], want[0], rtol=rel, atol=1e-37)
    assert sure >= 6


@pytest.mark.parametrize("drawn", [True, False])
def test_a_uniform_of_zero_accepts_whatever_the_target_can_say(drawn):
    """Node 1 with uniform 0: accepted however improbable, unless it is impossible."""
    g = np.random.default_rng(3)
    B, N, V = 5, 6, 2000
    logits, q, tokens, parent, temperature, u, noise = inputs(g, B, N, V, True, drawn)
    temperature[:] = 1.0
    u[:, 1] = 0.0
    tokens[:, 1] = logits[:, 0].argmin(-1)
    logits[np.arange(B), 0, tokens[:, 1]] = -60.0          # p of some 1e-30
    logits[4, 0, tokens[4, 1]] = -np.inf                   # p of 0
    ints, prob, st = accept(logits, q, tokens, parent, temperature, u, noise)
    assert st == 0
    assert np.all(ints[0, :4] >= 1) and np.all((prob[:4, 1] > 0) & (prob[:4, 1] < 1e-25))
    for b in range(4):
        assert R.path_of(parent[b], int(ints[1, b]))[0] == 1
    assert prob[4, 1] == 0 and (ints[1, 4] == 0 or R.path_of(parent[4], int(ints[1, 4]))[0] != 1)


def resized(table, ref, want, page):
    """A table and its counts after kv_pages_resize, with enough free pages."""
    table, ref = table.copy(), ref.copy()
    keep = np.where(want < 0, -1, -(-want // page))
    columns = np.arange(table.shape[1])
    for b in np.flatnonzero(keep >= 0):
        gone = (columns >= keep[b]) & (table[b] >= 0)
        np.subtract.at(ref, table[b, gone], 1)
        table[b, gone] = -1
    free = iter(np.flatnonzero(ref == 0))
    for b in np.flatnonzero(keep >= 0):
        for c in np.flatnonzero((columns < keep[b]) & (table[b] < 0)):
            table[b, c] = next(free)
            ref[table[b, c]] += 1
    return table, ref


@pytest.mark.parametrize("B,width,page", [(64, 4000, 16), (3, 32768, 16), (1100, 70, 64)])
def test_resize_wide_tables(B, width, page):
    g = np.random.default_rng(width)
    n_pages = B * width + 77
    length = g.integers(1, width - 40, B)
    ids = g.permutation(n_pages)[:int(length.sum())].astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    table[np.arange(width)[None] < length[:, None]] = ids
    ref = np.zeros(n_pages, np.int32)
    ref[ids] = 1
    t, r = dev(table), dev(ref)
    dims = dims_of(B, 1, 1, 64, page, n_pages, width)
    wsb = G.kv_pages_workspace_bytes(dims)
    ws = torch.full((wsb,), 255, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    held = length * page
    grow = held + 1                                              # every request by a page
    mixed = np.where(g.random(B) < 0.3, -1, np.where(g.random(B) < 0.5, held // 3, held + g.integers(1, 30 * page, B)))
    for want in (grow, mixed, np.zeros(B, np.int64)):
        G.kv_pages_resize(dims, dev(want.astype(np.int32)), t, r, ws, wsb, st)
        table, ref = resized(table, ref, want, page)
        np.testing.assert_array_equal(t.cpu().numpy(), table)
        np.testing.assert_array_equal(r.cpu().numpy(), ref)
    assert int(st.item()) == 0
