"""Sampled acceptance and the cache pages on the GPU against plain forms."""
import numpy as np
import pytest
import torch

import attn_reference as R
from gpu_helpers import ensure_built
from speculative_decode_hybrid_gb300 import gdnspec as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()


def dev(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


def accept(logits, q, tokens, parent, temperature, uniforms, noise, shift=0):
    """shift: the arrays begin that many floats past an aligned address."""
    B, N, V = logits.shape

    def at(x):
        if x is None:
            return None
        t = torch.empty(x.size + 4, device="cuda")[shift:shift + x.size]
        t.copy_(dev(x.astype(np.float32)).flatten())
        return t
    keep = [at(logits), at(q), at(uniforms), at(noise), dev(tokens.astype(np.int32)), dev(parent),
            dev(None if temperature is None else temperature.astype(np.float32))]
    ints = torch.full((3, B), -9, dtype=torch.int32, device="cuda")
    prob = torch.full((B, N), -9.0, device="cuda")
    wsb = G.spec_accept_sample_workspace_bytes(B, N)
    ws = torch.full((wsb,), 255, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    G.spec_accept_sample(B, N, V, keep[0], keep[1], keep[4], keep[5], keep[6], keep[2], keep[3], ints[0], ints[1], ints[2], prob,
                         ws, wsb, st)
    torch.cuda.synchronize()
    return ints.cpu().numpy(), prob.double().cpu().numpy(), int(st.item())


def inputs(g, B, N, V, tree, drawn, hot=3.0):
    logits = (hot * g.standard_normal((B, N, V))).astype(np.float32)
    parent = np.stack([R.random_tree(g, N) if tree else R.chain(N) for _ in range(B)])
    temperature = g.uniform(0.5, 1.5, B).astype(np.float32)
    tokens = np.zeros((B, N), np.int32)
    q = None
    if drawn:
        z = (logits[:, :max(N - 1, 1)] + 0.7 * g.standard_normal((B, max(N - 1, 1), V))) / temperature[:, None, None]
        e = np.exp(z - z.max(-1, keepdims=True))
        q = (e / e.sum(-1, keepdims=True)).astype(np.float32)
    for b in range(B):
        for i in range(1, N):
            row = logits[b, parent[b, i]] / temperature[b] if q is None else np.log(np.maximum(q[b, parent[b, i]], 1e-30))
            tokens[b, i] = np.argmax(row - np.log(g.exponential(size=V)))
    u = g.random((B, N)).astype(np.float32)
    noise = (g.exponential(size=(B, V)) + 1e-9).astype(np.float32)
    return logits, q, tokens, parent, temperature, u, noise


def check(args, got, tree):
    logits, q, tokens, parent, temperature, u, noise = args
    ints, prob, st = got
    B, N, V = logits.shape
    sure = 0
    for b in range(B):
        T = 1.0 if temperature is None else float(temperature[b])
        length, node, token, want, margin = R.sample(logits[b], None if q is None else q[b].astype(np.float64), tokens[b], parent[b],
                                                     T, u[b].astype(np.float64), noise[b].astype(np.float64))
        # f32 decides as 64 bits do unless a test or a race is closer than its own rounding
        if margin > 1e-4:
            sure += 1
            assert (int(ints[0, b]), int(ints[1, b]), int(ints[2, b])) == (length, node, token), (b, margin)
            rel = R.prob_bound(logits[b], T, V)
            np.testing.assert_allclose(prob[b], want, rtol=rel, atol=1e-37)
    assert sure >= B - max(1, B // 4)


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("B,N,V", [(1, 1, 7), (1, 2, 1), (3, 5, 1000), (2, 23, 4097), (9, 17, 513), (1, 65, 3001), (40, 9, 66)])
def test_sample_matches_the_definition(drawn, tree, B, N, V):
    if drawn and N == 1:
        pytest.skip("no drafted token")
    g = np.random.default_rng(B * 7 + N + V)
    for shift in (0, 1):
        args = inputs(g, B, N, V, tree, drawn)
        got = accept(args[0], args[1], args[2], args[3] if tree else None, *args[4:], shift=shift)
        check(args, got, tree)
        assert got[2] == 0


def test_sample_full_vocabulary():
    g = np.random.default_rng(0)
    for tree, drawn in ((False, True), (True, False), (True, True)):
        args = inputs(g, 2, 17, 151936, tree, drawn)
        check(args, accept(args[0], args[1], args[2], args[3] if tree else None, *args[4:]), tree)


def test_sample_siblings_that_repeat_a_token():
    g = np.random.default_rng(4)
    N, V = 9, 50
    args = list(inputs(g, 6, N, V, True, False, hot=1.0))
    args[3] = np.tile(np.array([-1] + [0] * 8, np.int32), (6, 1))       # a root with eight children
    args[2] = np.tile(np.array([0, 3, 3, 4, 3, 4, 5, 5, 3], np.int32), (6, 1))
    args[5][:] = 0.999
    check(args, accept(args[0], None, args[2], args[3], *args[4:]), True)
    # every token of the vocabulary rejected: p itself is drawn from
    V = 4
    args = list(inputs(g, 3, 5, V, True, False, hot=0.1))
    args[3] = np.tile(np.array([-1, 0, 0, 0, 0], np.int32), (3, 1))
    args[2] = np.tile(np.array([0, 0, 1, 2, 3], np.int32), (3, 1))
    args[5][:] = 1.0 - 2.0 ** -24
    ints, prob, st = accept(args[0], None, args[2], args[3], *args[4:])
    assert np.all((ints[2] >= 0) & (ints[2] < V)) and st == 0


def test_sample_draft_equal_to_the_target_accepts_everything():
    g = np.random.default_rng(5)
    logits, _, tokens, parent, temperature, u, noise = inputs(g, 4, 12, 2000, False, False)
    e = np.exp((logits - logits.max(-1, keepdims=True)).astype(np.float64) / temperature[:, None, None])
    q = (e / e.sum(-1, keepdims=True))[:, :-1].astype(np.float32)
    u = np.minimum(u, 0.999).astype(np.float32)
    ints, _, st = accept(logits, q, tokens, None, temperature, u, noise)
    assert np.all(ints[0] == 11) and st == 0


@pytest.mark.parametrize("drawn", [True, False])
def test_sample_cold_masked_and_undefined_rows(drawn):
    g = np.random.default_rng(6)
    B, N, V = 6, 6, 999
    logits, q, tokens, parent, temperature, u, noise = inputs(g, B, N, V, False, drawn)
    temperature[:] = [0.0, 0.0, 1.0, 1.0, 1.0, 1.0]
    logits[1] = np.round(logits[1])                        # ties at temperature 0: uniform over them
    tokens[0, 1:] = logits[0, :-1].argmax(-1)              # the greedy chain is accepted whole
    if drawn:
        q[0] = 1.0 / V
        u[0] = 0.9
    logits[2, :, 100:] = -np.inf                           # a masked vocabulary
    tokens[2, 1:] %= 100
    logits[3, 0, 17] = np.nan
    logits[4, 0, 5] = np.inf
    logits[5, 0] = -np.inf
    args = (logits, q, tokens, parent, temperature, u, noise)
    ints, prob, st = accept(logits, q, tokens, None, temperature, u, noise)
    assert st == G.GDN_DEV_NAN_LOGIT
    assert ints[0, 0] == 5 and ints[2, 0] == logits[0, 5].argmax()
    assert logits[1, ints[1, 1], ints[2, 1]] == logits[1, ints[1, 1]].max()
    assert ints[2, 2] < 100
    for b in (3, 4, 5):
        assert ints[0, b] == 0 and ints[2, b] == 0 and np.isnan(prob[b, 0])
    sure = [0, 2]
    check(tuple(None if x is None else x[sure] for x in args), (ints[:, sure], prob[sure], st), False)


def test_sample_tokens_and_parents_out_of_range():
    g = np.random.default_rng(7)
    args = list(inputs(g, 2, 8, 300, True, False))
    args[2][0, 3], args[2][1, 2] = 300, -1
    ints, prob, st = accept(args[0], None, args[2], args[3], *args[4:])
    assert st == G.GDN_DEV_TOKEN_RANGE
    check(args, (ints, prob, st), True)
    args[3][0, 4], args[3][1, 1] = 6, -3
    ints, prob, st = accept(args[0], None, args[2], args[3], *args[4:])
    assert st == G.GDN_DEV_TOKEN_RANGE | G.GDN_DEV_TREE
    check(args, (ints, prob, st), True)


def test_sample_statistics():
    """The committed token is a sample of the target, whatever the draft."""
    g = np.random.default_rng(8)
    V, B = 5, 20000
    p = np.array([0.1, 0.4, 0.05, 0.25, 0.2])
    q = np.array([0.5, 0.1, 0.2, 0.1, 0.1])
    logits = np.tile(np.log(p).astype(np.float32), (B, 2, 1))
    draft = g.choice(V, B, p=q)
    tokens = np.stack([np.zeros(B), draft], 1).astype(np.int32)
    ints, _, _ = accept(logits, np.tile(q.astype(np.float32), (B, 1, 1)), tokens, None, None, g.random((B, 2)), g.exponential(size=(B, V)) + 1e-9)
    first = np.where(ints[0] > 0, draft, ints[2])
    counts = np.bincount(first, minlength=V) / B
    assert np.all(np.abs(counts - p) < 5 * np.sqrt(p * (1 - p) / B))   # five standard deviations


# ---------------------------------------------------------------- pages

def dims_of(B, layers, h_kv, d, page, n_pages, width, f32=False):
    return G.make_attn_dims(B, layers, h_kv, h_kv, d, page, n_pages, width, G.GDN_F32 if f32 else G.GDN_BF16)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("B,N,layers,h_kv,page", [(1, 2, 1, 1, 16), (3, 23, 3, 2, 16), (2, 65, 2, 3, 128), (5, 9, 1, 8, 256)])
def test_commit_path(f32, d, B, N, layers, h_kv, page):
    g = np.random.default_rng(d + N)
    ctx = g.integers(0, 70, B)
    width = -(-(70 + N) // page)
    n_pages = B * width + 2
    table = g.permutation(n_pages)[:B * width].reshape(B, width).astype(np.int32)
    dt = torch.float32 if f32 else torch.bfloat16
    k, v = (torch.randn((layers, n_pages, h_kv, page, d), device="cuda").to(dt) for _ in range(2))
    for case in range(3):
        parent = np.stack([R.random_tree(g, N, (0.3, 0.8, 0.0)[case]) for _ in range(B)])
        node = np.array([(N - 1, 0, int(g.integers(0, N)))[case]] * B, np.int32)
        want = [k.clone(), v.clone()]
        for b in range(B):
            for j, i in enumerate(R.path_of(parent[b], int(node[b]))):
                s, z = int(ctx[b]) + i - 1, int(ctx[b]) + j
                for pool in want:
                    pool[:, table[b, z // page], :, z % page] = pool[:, table[b, s // page], :, s % page].clone()
        out = torch.zeros(B, dtype=torch.int32, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        G.kv_commit_path(dims_of(B, layers, h_kv, d, page, n_pages, width, f32), N, dev(parent), dev(node), dev(ctx.astype(np.int32)),
                         dev(table), k, v, out, st)
        assert torch.equal(k, want[0]) and torch.equal(v, want[1])
        np.testing.assert_array_equal(out.cpu().numpy(), ctx + [len(R.path_of(parent[b], int(node[b]))) for b in range(B)])
        assert int(st.item()) == 0


def test_commit_chain_and_refusals_on_the_device():
    d = dims_of(4, 1, 1, 64, 16, 20, 4)
    ctx = torch.tensor([5, 6, 7, 62], dtype=torch.int32, device="cuda")
    node = torch.tensor([3, 0, 9, 1], dtype=torch.int32, device="cuda")
    out = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.arange(16, dtype=torch.int32, device="cuda").view(4, 4)
    G.kv_commit_path(d, 5, None, node, ctx, table, None, None, out, st)
    assert out.tolist() == [8, 6, 7, 62]
    assert int(st.item()) == G.GDN_DEV_NODE_RANGE | G.GDN_DEV_LENGTH
    # a tree over a page that is not there: flagged, the row left over
    k = torch.randn((1, 20, 1, 16, 64), device="cuda").bfloat16()
    before = k.clone()
    st.zero_()
    table[0, 0] = 77
    parent = torch.tensor([[-1, 0, 0, 2, 1]] * 4, dtype=torch.int32, device="cuda")
    G.kv_commit_path(d, 5, parent, torch.tensor([3, 0, 0, 0], dtype=torch.int32, device="cuda"),
                     torch.tensor([5, 6, 7, 8], dtype=torch.int32, device="cuda"), table, k, k.clone(), out, st)
    assert torch.equal(k, before) and int(st.item()) == G.GDN_DEV_PAGE and out.tolist() == [7, 6, 7, 8]


class Pool:
    """The pages in plain Python."""

    def __init__(self, table, ref, ctx, page):
        self.table, self.ref, self.ctx, self.page, self.flags = [list(r) for r in table], list(ref), list(ctx), page, 0

    def take(self):
        if 0 not in self.ref:
            self.flags |= G.GDN_DEV_POOL
            return -1
        i = self.ref.index(0)
        self.ref[i] = 1
        return i

    def resize(self, want):
        keep = []
        for row, w in zip(self.table, want):
            n = -(-w // self.page) if w >= 0 else -1
            if n > len(row):
                self.flags |= G.GDN_DEV_LENGTH
                n = -1
            keep.append(n)
            for j in range(n if n >= 0 else len(row), len(row)):
                if row[j] >= 0:
                    self.ref[row[j]] -= 1
                    row[j] = -1
        for row, n in zip(self.table, keep):
            for j in range(max(n, 0)):
                if row[j] < 0:
                    row[j] = self.take()

    def fork(self, src, dst, pools):
        fresh = {}
        for i, (a, z) in enumerate(zip(src, dst)):       # the pages first, in order
            if not (0 <= a < len(self.table) and 0 <= z < len(self.table)):
                self.flags |= G.GDN_DEV_NODE_RANGE
            elif self.ctx[a] < 0 or self.ctx[a] > len(self.table[a]) * self.page:
                self.flags |= G.GDN_DEV_LENGTH
            else:
                fresh[i] = self.take() if self.ctx[a] % self.page else None
        for i, new in fresh.items():
            a, z = src[i], dst[i]
            full, tail = divmod(self.ctx[a], self.page)
            if new == -1:
                self.table[z], self.ctx[z] = [-1] * len(self.table[z]), 0
                continue
            self.table[z] = self.table[a][:full] + [-1] * (len(self.table[a]) - full)
            for p in self.table[a][:full]:
                self.ref[p] += 1
            if tail:
                self.table[z][full] = new
                for pool in pools:
                    pool[:, new, :, :tail] = pool[:, self.table[a][full], :, :tail]
            self.ctx[z] = self.ctx[a]


@pytest.mark.parametrize("B,width,page,n_pages", [(4, 5, 16, 13), (40, 9, 32, 200), (70, 40, 16, 6000), (3, 300, 16, 500)])
def test_pages_random_life(B, width, page, n_pages):
    """Requests grown, cut, forked and freed at random, the pool often empty."""
    g = np.random.default_rng(B + width)
    layers, h_kv, d = 2, 2, 64
    k, v = (torch.randn((layers, n_pages, h_kv, page, d), device="cuda").bfloat16() for _ in range(2))
    mirror = [k.clone(), v.clone()]
    pool = Pool(np.full((B, width), -1).tolist(), [0] * n_pages, [0] * B, page)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    ref = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
    dims = dims_of(B, layers, h_kv, d, page, n_pages, width)
    wsb = G.kv_pages_workspace_bytes(dims)
    ws = torch.full((wsb,), 255, dtype=torch.uint8, device="cuda")
    for step in range(12):
        pool.flags = 0
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        want = np.where(g.random(B) < 0.3, -1, g.integers(0, width * page + 1, B) // (1 if step % 3 else 4))
        if step == 5:
            want[0] = width * page + 1
        if step == 7:
            want[:] = 0
        G.kv_pages_resize(dims, dev(want.astype(np.int32)), table, ref, ws, wsb, st)
        pool.resize(want.tolist())
        held = [sum(x >= 0 for x in row) * page for row in pool.table]
        pool.ctx = [int(g.integers(0, h + 1)) if h else 0 for h in held]
        ctx.copy_(torch.tensor(pool.ctx, dtype=torch.int32))
        assert table.tolist() == pool.table and ref.tolist() == pool.ref, step
        n = int(g.integers(1, B // 2 + 1))
        order = g.permutation(B).tolist()
        src, dst = [order[0]] * n if step % 4 == 1 else order[:n], order[B - n:]
        if B >= 3 and src[0] in dst:
            continue
        free = np.zeros(B, np.int64) - 1
        free[dst] = 0
        G.kv_pages_resize(dims, dev(free.astype(np.int32)), table, ref, ws, wsb, st)
        pool.resize(free.tolist())
        G.kv_pages_fork(dims, n, dev(np.array(src, np.int32)), dev(np.array(dst, np.int32)), table, ctx, ref, k, v, ws, wsb, st)
        pool.fork(src, dst, mirror)
        assert table.tolist() == pool.table and ref.tolist() == pool.ref and ctx.tolist() == pool.ctx, step
        assert torch.equal(k, mirror[0]) and torch.equal(v, mirror[1]), step
        assert int(st.item()) == pool.flags, step


def test_fork_leaves_out_what_is_out_of_range():
    page, n_pages, width, B = 16, 12, 3, 5
    table = np.full((B, width), -1, np.int32)
    table[0, :2], table[1, :3] = [4, 7], [1, 2, 3]
    ref = np.zeros(n_pages, np.int32)
    ref[[4, 7, 1, 2, 3]] = 1
    ctx = np.array([20, 49, 0, 0, 0], np.int32)       # request 1's length is past its table
    k = torch.randn((1, n_pages, 1, page, 64), device="cuda").bfloat16()
    v = k.clone()
    mirror, pool = [k.clone(), v.clone()], Pool(table.tolist(), ref.tolist(), ctx.tolist(), page)
    src, dst = [0, 1, 9, 0], [2, 3, 4, -1]
    t, r, c, st = dev(table), dev(ref), dev(ctx), torch.zeros(1, dtype=torch.int32, device="cuda")
    dims = dims_of(B, 1, 1, 64, page, n_pages, width)
    wsb = G.kv_pages_workspace_bytes(dims)
    ws = torch.zeros(wsb, dtype=torch.uint8, device="cuda")
    G.kv_pages_fork(dims, 4, dev(np.array(src, np.int32)), dev(np.array(dst, np.int32)), t, c, r, k, v, ws, wsb, st)
    pool.fork(src, dst, mirror)
    assert t.tolist() == pool.table and r.tolist() == pool.ref and c.tolist() == pool.ctx
    assert torch.equal(k, mirror[0]) and int(st.item()) == pool.flags == G.GDN_DEV_NODE_RANGE | G.GDN_DEV_LENGTH
