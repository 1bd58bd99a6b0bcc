"""The attention layers' calls on the GPU against 64-bit plain forms: norm and
rotary into the paged cache, chain and tree attention, where they can go wrong
(page and tile edges, empty contexts, shared heads, rubbish in masked places)."""
import numpy as np
import pytest
import torch

import attn_reference as R
from gpu_helpers import ensure_built
from speculative_decode_hybrid_gb300 import gdnspec as G

pytestmark = pytest.mark.gpu
TYPES = {"bf16": (torch.bfloat16, G.GDN_BF16), "f32": (torch.float32, G.GDN_F32)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()


def f64(t):
    return t.double().cpu().numpy()


class Cache:
    """A pool with rubbish in every row that no slot in use lies in."""

    def __init__(self, g, ctx, new, h_kv, d, page, dtype, spare=3, width=None, rubbish=float("nan")):
        self.ctx, self.page, self.h_kv, self.d = list(ctx), page, h_kv, d
        need = [-(-(n + new) // page) for n in ctx]
        self.width = width or max(need)
        n_pages = sum(need) + spare
        order = g.permutation(n_pages)
        self.table = np.full((len(ctx), self.width), 2 ** 30, np.int32)   # entries that no slot needs are not read
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[at:at + k]
            at += k
        self.n_pages, self.dt = n_pages, TYPES[dtype][0]
        shape = (n_pages, h_kv, page, d)
        self.k = torch.full(shape, rubbish, dtype=self.dt, device="cuda")
        self.v = torch.full(shape, rubbish, dtype=self.dt, device="cuda")
        self.table_dev = torch.from_numpy(self.table).cuda()
        self.ctx_dev = torch.tensor(self.ctx, dtype=torch.int32, device="cuda")
        self.dtype = TYPES[dtype][1]

    def dims(self, h_q, batch=None, layers=1):
        return G.make_attn_dims(batch or len(self.ctx), layers, h_q, self.h_kv, self.d, self.page, self.n_pages, self.width,
                                self.dtype)

    def where(self, b, slots):
        s = np.asarray(slots)
        return torch.from_numpy(self.table[b, s // self.page].astype(np.int64)).cuda(), torch.from_numpy(s % self.page).cuda()

    def put(self, b, slots, k, v):
        page, off = self.where(b, slots)
        self.k[page, :, off] = k.to(self.dt)
        self.v[page, :, off] = v.to(self.dt)

    def rows(self, b, slots):
        page, off = self.where(b, slots)
        return self.k[page, :, off], self.v[page, :, off]


def attend(cache, q, parents, scale, stream=None, status=None):
    B, T, Hq, _ = q.shape
    dims = cache.dims(Hq, B)
    wsb = G.attn_workspace_bytes(dims, T)
    ws = torch.full((wsb,), 255, dtype=torch.uint8, device="cuda")   # any contents
    out = torch.full_like(q, float("nan"))
    st = torch.zeros(1, dtype=torch.int32, device="cuda") if status is None else status
    if parents is None:
        G.attn_verify_span(dims, T, q, cache.k, cache.v, cache.table_dev, cache.ctx_dev, scale, out, ws, wsb, st, stream)
    else:
        G.attn_tree_verify(dims, T + 1, parents, torch.from_numpy(np.ascontiguousarray(parents)).cuda(), q, cache.k, cache.v,
                           cache.table_dev, cache.ctx_dev, scale, out, ws, wsb, st, stream)
    return out, st


def make(g, ctx, T, h_q, h_kv, d, page, dtype, tree, spread=1.0, **kw):
    cache = Cache(g, ctx, T, h_kv, d, page, dtype, **kw)
    gen = torch.Generator("cuda").manual_seed(int(g.integers(1 << 30)))
    for b, n in enumerate(ctx):
        kv = torch.randn((2, n + T, h_kv, d), device="cuda", generator=gen)
        cache.put(b, np.arange(n + T), kv[0], kv[1])
    q = (spread * torch.randn((len(ctx), T, h_q, d), device="cuda", generator=gen)).to(cache.dt)
    parents = np.stack([R.random_tree(g, T + 1) for _ in ctx]) if tree else None
    return cache, q, parents


def check(cache, q, parents, out, scale, skip=()):
    B, T, Hq, d = q.shape
    for b, n in enumerate(cache.ctx):
        if b in skip:
            continue
        k, v = cache.rows(b, np.arange(n + T))
        parent = R.chain(T + 1) if parents is None else parents[b]
        want, mass, big = R.attention(f64(q[b]), f64(k), f64(v), parent, n, scale)
        bound = R.attention_bound(want, mass, big, d, n + T, cache.dtype == G.GDN_BF16)
        err = np.abs(f64(out[b]) - want)
        assert np.all(err <= bound), (b, float((err / bound).max()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,h_q,h_kv,page,tree", [
    (1, 4, 4, 16, False), (1, 8, 1, 32, False), (3, 6, 2, 16, True), (5, 7, 1, 64, False), (22, 16, 2, 16, True),
    (33, 12, 3, 128, True), (64, 8, 2, 256, True), (64, 5, 5, 64, False)])
def test_attention_heads_and_spans(dtype, d, T, h_q, h_kv, page, tree):
    g = np.random.default_rng(T * 1000 + d)
    cache, q, parents = make(g, [37, 0, 130], T, h_q, h_kv, d, page, dtype, tree)
    out, st = attend(cache, q, parents, d ** -0.5)
    check(cache, q, parents, out, d ** -0.5)
    assert int(st.item()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_attention_context_lengths_at_every_edge(dtype, page):
    g = np.random.default_rng(page)
    ctx = [0, 1, 15, 16, 17, 63, 64, 65, 106, 107, 127, 128, 129, 255, 256, 257, 383]
    for d in (128, 256):
        cache, q, parents = make(g, ctx, 22, 4, 2, d, page, dtype, True)
        out, st = attend(cache, q, parents, d ** -0.5)
        check(cache, q, parents, out, d ** -0.5)
        assert int(st.item()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_many_requests_of_different_lengths(dtype):
    g = np.random.default_rng(3)
    ctx = [int(x) for x in np.r_[g.integers(0, 60, 60), 1500, 3, 700]]
    cache, q, parents = make(g, ctx, 7, 6, 2, 64, 16, dtype, True)
    out, st = attend(cache, q, parents, 0.2)
    check(cache, q, parents, out, 0.2)
    assert int(st.item()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 256])
def test_attention_peaks_and_a_rising_maximum(dtype, d):
    """Scores of hundreds, their maximum rising along the slots: the softmax's
    reference has to follow, and what was summed before to be scaled down."""
    g = np.random.default_rng(d)
    n, T = 900, 4
    cache, q, parents = make(g, [n], T, 4, 2, d, 32, dtype, True)
    k, v = cache.rows(0, np.arange(n + T))
    cache.put(0, np.arange(n + T), k.float() * torch.linspace(0.05, 12.0, n + T, device="cuda")[:, None, None], v)
    out, st = attend(cache, q, parents, d ** -0.5)
    check(cache, q, parents, out, d ** -0.5)
    assert int(st.item()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_values_that_are_no_numbers_stay_on_their_paths(dtype):
    g = np.random.default_rng(8)
    T, n, d = 20, 50, 128
    cache, q, parents = make(g, [n], T, 16, 2, d, 16, dtype, True)
    parents[0] = R.random_tree(np.random.default_rng(1), T + 1, 0.3)
    bad = {4: float("inf"), 9: float("nan")}
    for node, x in bad.items():
        page, off = cache.where(0, [n + node - 1])
        cache.v[page, :, off, 5] = x
    page, off = cache.where(0, [n + 11 - 1])
    cache.k[page, :, off, 7] = float("nan")
    out, st = attend(cache, q, parents, d ** -0.5)
    assert int(st.item()) == 0
    k, v = (f64(x) for x in cache.rows(0, np.arange(n + T)))
    for t in range(T):
        path = R.path_of(parents[0], t + 1)
        got = f64(out[0, t])
        if 11 in path:
            assert np.isnan(got).all(), t
            continue
        want, mass, big = R.attention(f64(q[0])[t:t + 1], k[list(range(n)) + [n + i - 1 for i in path]],
                                      v[list(range(n)) + [n + i - 1 for i in path]],
                                      R.chain(len(path) + 1), n, d ** -0.5) if len(path) == 1 else (None, None, None)
        finite = np.ones(d, bool)
        finite[5] = not any(i in bad for i in path)
        assert np.isfinite(got[:, finite]).all(), t
        if 9 in path:
            assert np.isnan(got[:, 5]).all(), t
        elif 4 in path:
            assert np.isposinf(got[:, 5]).all(), t


def test_attention_far_into_a_large_pool():
    """Pages whose rows lie more than 2^32 bytes into the pool."""
    d, page, h_kv, T = 128, 64, 8, 3
    n_pages = 2 ** 32 // (page * h_kv * d * 2) + 40
    g = np.random.default_rng(2)
    cache = Cache(g, [100], T, h_kv, d, page, "bf16", spare=1)
    cache.n_pages = n_pages
    cache.k = torch.empty((n_pages, h_kv, page, d), dtype=torch.bfloat16, device="cuda")
    cache.v = torch.empty_like(cache.k)
    cache.table = np.array([[n_pages - 1, n_pages - 30]], np.int32)
    cache.table_dev = torch.from_numpy(cache.table).cuda()
    kv = torch.randn((2, 103, h_kv, d), device="cuda")
    cache.put(0, np.arange(103), kv[0], kv[1])
    q = torch.randn((1, T, 16, d), device="cuda").bfloat16()
    out, st = attend(cache, q, None, d ** -0.5)
    check(cache, q, None, out, d ** -0.5)
    assert int(st.item()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_leaves_out_lengths_and_flags_pages(dtype):
    g = np.random.default_rng(5)
    T, d = 4, 64
    cache, q, _ = make(g, [40, 40, 40], T, 4, 2, d, 16, dtype, False)
    cache.ctx_dev[1] = cache.width * 16 - T + 1
    out, st = attend(cache, q, None, d ** -0.5)
    check(cache, q, None, out, d ** -0.5, skip=(1,))
    assert torch.count_nonzero(out[1]).item() == 0
    assert int(st.item()) == G.GDN_DEV_LENGTH
    cache.ctx_dev[1] = -1
    out, st = attend(cache, q, None, d ** -0.5)
    assert torch.count_nonzero(out[1]).item() == 0 and int(st.item()) == G.GDN_DEV_LENGTH
    # a page outside the pool reads as zeros
    cache.ctx_dev[1] = 40
    cache.table_dev[1, 1] = cache.n_pages + 5
    out, st = attend(cache, q, None, d ** -0.5)
    assert int(st.item()) == G.GDN_DEV_PAGE
    k, v = (f64(x) for x in cache.rows(1, np.arange(44)))
    k[16:32], v[16:32] = 0, 0
    want, mass, big = R.attention(f64(q[1]), k, v, R.chain(T + 1), 40, d ** -0.5)
    assert np.all(np.abs(f64(out[1]) - want) <= R.attention_bound(want, mass, big, d, 44, dtype == "bf16"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,h_q,h_kv,n", [(17, 3, 3, 2900), (8, 4, 1, 3000), (25, 8, 2, 2111), (16, 8, 1, 1500), (64, 24, 3, 700)])
def test_attention_many_rows_over_long_contexts(dtype, d, T, h_q, h_kv, n):
    """17 to 512 rows of a key/value head, each over many tiles, their maximum
    rising along the slots, beside a request that has hardly any."""
    g = np.random.default_rng(T * d + n)
    cache, q, parents = make(g, [n, 1, 333], T, h_q, h_kv, d, 16, dtype, True)
    k, v = cache.rows(0, np.arange(n + T))
    cache.put(0, np.arange(n + T), k.float() * torch.linspace(0.2, 4.0, n + T, device="cuda")[:, None, None], v)
    out, st = attend(cache, q, parents, d ** -0.5)
    check(cache, q, parents, out, d ** -0.5)
    assert int(st.item()) == 0
    again, _ = attend(cache, q, parents, d ** -0.5)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,h_q,h_kv", [(1, 2, 2), (2, 3, 3), (1, 6, 2), (4, 1, 1), (3, 4, 2), (2, 8, 2), (10, 2, 2)])
def test_attention_few_rows_over_long_contexts(dtype, d, T, h_q, h_kv):
    g = np.random.default_rng(T * d + h_q)
    ctx = [2741, 0, 127, 1030]
    cache, q, parents = make(g, ctx, T, h_q, h_kv, d, 32, dtype, T > 1)
    n = ctx[0] + T
    k, v = cache.rows(0, np.arange(n))
    cache.put(0, np.arange(n), k.float() * torch.linspace(0.2, 4.0, n, device="cuda")[:, None, None], v)
    out, st = attend(cache, q, parents, d ** -0.5)
    check(cache, q, parents, out, d ** -0.5)
    assert int(st.item()) == 0
    again, _ = attend(cache, q, parents, d ** -0.5)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 256])
def test_attention_many_rows_leave_out_lengths_and_flag_pages(dtype, d):
    g = np.random.default_rng(15)
    T, n = 20, 300
    cache, q, _ = make(g, [n, n, n], T, 16, 2, d, 16, dtype, False)
    cache.ctx_dev[1] = cache.width * 16 - T + 1
    out, st = attend(cache, q, None, d ** -0.5)
    check(cache, q, None, out, d ** -0.5, skip=(1,))
    assert torch.count_nonzero(out[1]).item() == 0 and int(st.item()) == G.GDN_DEV_LENGTH
    cache.ctx_dev[1] = n
    cache.table_dev[1, 9], cache.table_dev[1, 19] = cache.n_pages, -3   # 19: the last page, where drafted nodes lie
    out, st = attend(cache, q, None, d ** -0.5)
    assert int(st.item()) == G.GDN_DEV_PAGE
    k, v = (f64(x) for x in cache.rows(1, np.arange(n + T)))
    for j in (9, 19):
        k[j * 16:j * 16 + 16], v[j * 16:j * 16 + 16] = 0, 0
    want, mass, big = R.attention(f64(q[1]), k, v, R.chain(T + 1), n, d ** -0.5)
    assert np.all(np.abs(f64(out[1]) - want) <= R.attention_bound(want, mass, big, d, n + T, dtype == "bf16"))


def test_attention_device_parent_is_checked_again():
    g = np.random.default_rng(6)
    cache, q, parents = make(g, [70], 6, 4, 2, 64, 16, "bf16", True)
    good = R.chain(7)[None].copy()
    bad = torch.from_numpy(good.copy()).cuda()
    bad[0, 3], bad[0, 5] = 99, -7       # taken as i - 1: the chain again
    dims = cache.dims(4)
    wsb = G.attn_workspace_bytes(dims, 6)
    ws = torch.zeros(wsb, dtype=torch.uint8, device="cuda")
    out, st = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    G.attn_tree_verify(dims, 7, good, bad, q, cache.k, cache.v, cache.table_dev, cache.ctx_dev, 0.125, out, ws, wsb, st)
    check(cache, q, good, out, 0.125)
    assert int(st.item()) == G.GDN_DEV_TREE


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_chain_is_the_tree_of_a_chain_and_runs_repeat(dtype):
    g = np.random.default_rng(7)
    cache, q, _ = make(g, [500, 90], 16, 8, 2, 128, 32, dtype, False)
    chains = np.stack([R.chain(17)] * 2)
    a, _ = attend(cache, q, None, 0.1)
    b, _ = attend(cache, q, chains, 0.1)
    c, _ = attend(cache, q, None, 0.1)
    assert torch.equal(a, b) and torch.equal(a, c)


def test_attention_on_another_stream_and_in_a_graph():
    g = np.random.default_rng(9)
    cache, q, parents = make(g, [300, 20], 9, 8, 2, 128, 16, "bf16", True)
    want, _ = attend(cache, q, parents, 0.1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, _ = attend(cache, q, parents, 0.1)
    explicit, _ = attend(cache, q, parents, 0.1, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(want, got) and torch.equal(want, explicit)
    dims = cache.dims(8)
    wsb = G.attn_workspace_bytes(dims, 9)
    ws, out = torch.zeros(wsb, dtype=torch.uint8, device="cuda"), torch.zeros_like(q)
    pd = torch.from_numpy(parents).cuda()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        G.attn_tree_verify(dims, 10, parents, pd, q, cache.k, cache.v, cache.table_dev, cache.ctx_dev, 0.1, out, ws, wsb)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    # the lengths are read by the kernel: a replay follows them
    cache.ctx_dev[0] = 250
    cache.ctx[0] = 250
    graph.replay()
    torch.cuda.synchronize()
    check(cache, q, parents, out, 0.1)


# ---------------------------------------------------------------- norm and rotary

def rope_table(n, rot):
    inv = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(n)[:, None] * inv
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot", [(64, 0), (64, 16), (64, 64), (128, 32), (128, 128), (256, 64), (256, 256)])
@pytest.mark.parametrize("T,h_q,h_kv,tree,pairs,pad", [(1, 1, 1, False, False, 0), (7, 6, 2, True, True, 32),
                                                       (64, 8, 8, True, False, 0), (203, 5, 1, False, True, 8)])
def test_norm_rope(dtype, d, rot, T, h_q, h_kv, tree, pairs, pad):
    g = np.random.default_rng(T + d + rot)
    ctx, page, eps, offset = [13, 0, 31], 16, 1e-6, 1.0
    dt = TYPES[dtype][0]
    cache = Cache(g, ctx, T, h_kv, d, page, dtype, rubbish=7.0)
    heads = h_q + 2 * h_kv
    qkv = (3.0 * torch.randn((3, T, heads * d + pad), device="cuda")).to(dt)
    qkv[1, 0, :d] = 0.0                                  # a head of zeros stays one
    qn, kn = ((0.2 * torch.randn(d, device="cuda")).to(dt) for _ in range(2))
    rope = rope_table(max(ctx) + T, rot) if rot else None
    parents = np.stack([R.random_tree(g, T + 1) for _ in ctx]) if tree else None
    out = torch.full((3, T, h_q, d), float("nan"), dtype=dt, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = cache.k.clone()
    G.attn_qk_norm_rope(cache.dims(h_q), T, qkv, heads * d + pad, qn, kn, eps, offset,
                        None if rope is None else torch.from_numpy(rope).cuda(), rot, 0 if rope is None else len(rope),
                        None if parents is None else torch.from_numpy(parents).cuda(), cache.ctx_dev, cache.table_dev, out,
                        cache.k, cache.v, st, flags=G.GDN_ROPE_PAIRS if pairs else 0)
    assert int(st.item()) == 0
    x, q, bf = f64(qkv[:, :, :heads * d]).reshape(3, T, heads, d), f64(out), dtype == "bf16"
    written = torch.zeros(cache.k.shape[:3], dtype=torch.bool, device="cuda")
    for b, n in enumerate(ctx):
        k, v = (f64(t) for t in cache.rows(b, n + np.arange(T)))
        pg, off = cache.where(b, n + np.arange(T))
        written[pg, :, off] = True
        for t in range(T):
            pos = n + (len(R.path_of(parents[b], t + 1)) if tree else t + 1) - 1
            w = np.concatenate([np.tile(f64(qn), (h_q, 1)), np.tile(f64(kn), (h_kv, 1))])
            y = R.norm_rope(x[b, t, :h_q + h_kv], w, eps, offset, None if rope is None else rope.astype(np.float64), rot, pos, pairs)
            got = np.concatenate([q[b, t], k[t]])
            assert np.all(np.abs(got - y) <= R.norm_bound(y, d, bf)), (b, t)
            np.testing.assert_array_equal(v[t], x[b, t, h_q + h_kv:])
    assert torch.equal(cache.k[~written], before[~written])      # nothing else is touched


def test_norm_rope_leaves_out_lengths_and_flags_pages():
    g = np.random.default_rng(1)
    T, d = 5, 64
    cache = Cache(g, [10, 10, 10], T, 2, d, 16, "f32", rubbish=7.0)
    qkv = torch.randn((3, T, 8 * d), device="cuda")
    w, rope = torch.ones(d, device="cuda"), torch.from_numpy(rope_table(15, d)).cuda()
    cache.ctx_dev[1] = cache.width * 16
    cache.table_dev[2, 0] = -1
    out = torch.full((3, T, 4, d), 9.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    want_k = cache.k.clone()
    G.attn_qk_norm_rope(cache.dims(4), T, qkv, 8 * d, w, w, 1e-6, 0.0, rope, d, 15, None, cache.ctx_dev, cache.table_dev, out,
                        cache.k, cache.v, st)
    assert int(st.item()) == G.GDN_DEV_LENGTH | G.GDN_DEV_PAGE
    assert torch.all(out[1] == 9.0) and not torch.any(out[2] == 9.0)
    pg, off = cache.where(0, 10 + np.arange(T))
    want_k[pg, :, off] = cache.k[pg, :, off]
    assert torch.equal(cache.k, want_k)                           # only request 0 wrote
    # a rotary table too short leaves a request out as well
    st.zero_()
    cache.ctx_dev[:] = torch.tensor([11, 10, 10], device="cuda")
    cache.table_dev[2, 0] = int(cache.table[2, 0])
    G.attn_qk_norm_rope(cache.dims(4), T, qkv, 8 * d, w, w, 1e-6, 0.0, rope, d, 15, None, cache.ctx_dev, cache.table_dev, out,
                        cache.k, cache.v, st)
    assert int(st.item()) == G.GDN_DEV_LENGTH
