"""CPU-only checks of the attention-layer, cache-page and sampled-acceptance
calls: what they refuse, they refuse on the host, before anything is queued."""
import ctypes

import numpy as np
import pytest

import attn_reference as R
from speculative_decode_hybrid_gb300 import build as B
from speculative_decode_hybrid_gb300 import gdnspec as G

FAKE = 0x10000  # an aligned non-NULL address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    B.build()
    return G.load()


def dims(**kw):
    d = dict(batch=2, layers=3, h_q=8, h_kv=2, d_head=128, page_tokens=32, n_pages=40, table_width=9, dtype=G.GDN_BF16)
    d.update(kw)
    return G.make_attn_dims(*d.values())


BAD_DIMS = [dict(batch=0), dict(batch=70000), dict(layers=0), dict(layers=70000), dict(h_kv=0), dict(h_q=1), dict(h_q=7),
            dict(h_q=2048), dict(d_head=96), dict(d_head=32), dict(d_head=512), dict(page_tokens=8), dict(page_tokens=48),
            dict(page_tokens=512), dict(n_pages=0), dict(n_pages=2 ** 31 - 1), dict(table_width=0),
            dict(table_width=2 ** 26), dict(batch=65535, table_width=2 ** 16)]


def rope(lib, d, **kw):
    a = dict(n_tok=5, qkv=FAKE, stride=12 * 128, qn=FAKE, kn=FAKE, eps=1e-6, off=1.0, rope=FAKE, rot=64, max_pos=100, parent=None,
             ctx=FAKE, table=FAKE, q=FAKE, k=FAKE, v=FAKE, st=FAKE, flags=0)
    a.update(kw)
    return lib.attn_qk_norm_rope(ctypes.byref(d) if d is not None else None, *a.values(), None)


def span(lib, d, **kw):
    a = dict(n_tok=5, q=FAKE, k=FAKE, v=FAKE, table=FAKE, ctx=FAKE, scale=0.1, out=FAKE, ws=FAKE, wsb=1 << 40, st=FAKE)
    a.update(kw)
    return lib.attn_verify_span(ctypes.byref(d) if d is not None else None, *a.values(), None)


def tree(lib, d, parent, **kw):
    a = dict(n_nodes=6, ph=None if parent is None else parent.ctypes.data, pd=FAKE, q=FAKE, k=FAKE, v=FAKE, table=FAKE, ctx=FAKE,
             scale=0.1, out=FAKE, ws=FAKE, wsb=1 << 40, st=FAKE)
    a.update(kw)
    return lib.attn_tree_verify(ctypes.byref(d), *a.values(), None)


def commit(lib, d, **kw):
    a = dict(n_nodes=6, parent=FAKE, node=FAKE, ctx=FAKE, table=FAKE, k=FAKE, v=FAKE, out=FAKE, st=FAKE)
    a.update(kw)
    return lib.kv_commit_path(ctypes.byref(d) if d is not None else None, *a.values(), None)


def resize(lib, d, **kw):
    a = dict(want=FAKE, table=FAKE, ref=FAKE, ws=FAKE, wsb=1 << 40, st=FAKE)
    a.update(kw)
    return lib.kv_pages_resize(ctypes.byref(d) if d is not None else None, *a.values(), None)


def fork(lib, d, **kw):
    a = dict(n=1, src=FAKE, dst=FAKE, table=FAKE, ctx=FAKE, ref=FAKE, k=FAKE, v=FAKE, ws=FAKE, wsb=1 << 40, st=FAKE)
    a.update(kw)
    return lib.kv_pages_fork(ctypes.byref(d) if d is not None else None, *a.values(), None)


def sample(lib, **kw):
    a = dict(batch=2, n=5, vocab=100, logits=FAKE, q=FAKE, tokens=FAKE, parent=None, temp=None, u=FAKE, noise=FAKE, al=FAKE, an=FAKE,
             nt=FAKE, prob=None, ws=FAKE, wsb=1 << 40, st=None)
    a.update(kw)
    return lib.spec_accept_sample(*a.values(), None)


@pytest.mark.parametrize("bad", BAD_DIMS, ids=str)
def test_dims_out_of_range(lib, bad):
    d = dims(**bad)
    for call in (rope, span, commit, resize, fork):
        assert call(lib, d) == G.GDN_ERR_DIMS, call.__name__
    assert G.attn_workspace_bytes(d, 4) == 0 and G.kv_pages_workspace_bytes(d) == 0


def test_null_dims_and_types(lib):
    for call in (rope, span, commit, resize, fork):
        assert call(lib, None) == G.GDN_ERR_NULL
        assert call(lib, dims(dtype=5)) == G.GDN_ERR_DTYPE


def test_norm_rope_refuses(lib):
    d = dims()
    for bad in (dict(n_tok=0), dict(n_tok=2 ** 30), dict(parent=FAKE, n_tok=65), dict(stride=12 * 128 - 8), dict(stride=12 * 128 + 4),
                dict(rot=-16), dict(rot=8), dict(rot=24), dict(rot=144), dict(max_pos=0), dict(eps=0.0), dict(eps=float("nan")),
                dict(off=float("inf"))):
        assert rope(lib, d, **bad) == G.GDN_ERR_DIMS, bad
    for name in ("qkv", "qn", "kn", "rope", "ctx", "table", "q", "k", "v"):
        assert rope(lib, d, **{name: None}) == G.GDN_ERR_NULL, name
    for name in ("qkv", "qn", "kn", "rope", "q", "k", "v"):
        assert rope(lib, d, **{name: FAKE + 8}) == G.GDN_ERR_ALIGN, name
    for name in ("parent", "ctx", "table", "st"):
        assert rope(lib, d, **{name: FAKE + 2}) == G.GDN_ERR_ALIGN, name
    assert rope(lib, d, flags=2) == G.GDN_ERR_FLAGS


def test_attention_refuses(lib):
    d = dims()
    for bad in (dict(n_tok=0), dict(n_tok=65), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert span(lib, d, **bad) == G.GDN_ERR_DIMS, bad
    assert span(lib, dims(batch=40000)) == G.GDN_ERR_DIMS       # batch * h_kv
    for name in ("q", "k", "v", "table", "ctx", "out"):
        assert span(lib, d, **{name: None}) == G.GDN_ERR_NULL, name
    for name in ("q", "k", "v", "out"):
        assert span(lib, d, **{name: FAKE + 8}) == G.GDN_ERR_ALIGN, name
    for name in ("table", "ctx", "st"):
        assert span(lib, d, **{name: FAKE + 1}) == G.GDN_ERR_ALIGN, name
    need = G.attn_workspace_bytes(d, 5)
    assert need > 0
    for bad in (dict(ws=None), dict(ws=FAKE + 128), dict(wsb=need - 1)):
        assert span(lib, d, **bad) == G.GDN_ERR_WORKSPACE, bad


def test_tree_attention_refuses_geometry(lib):
    d = dims()
    good = np.stack([R.chain(6), R.chain(6)])
    for b, i, x, code in ((0, 0, 0, G.GDN_ERR_TREE_ROOT), (1, 3, 3, G.GDN_ERR_TREE_PARENT), (1, 2, -1, G.GDN_ERR_TREE_PARENT),
                          (0, 4, 9, G.GDN_ERR_TREE_PARENT)):
        p = good.copy()
        p[b, i] = x
        assert tree(lib, d, p) == code
    assert tree(lib, d, good, n_nodes=1) == G.GDN_ERR_TREE_TRUNCATED
    assert tree(lib, d, good, n_nodes=66) == G.GDN_ERR_DIMS
    assert tree(lib, d, None) == G.GDN_ERR_NULL
    assert tree(lib, d, good, pd=None) == G.GDN_ERR_NULL
    assert tree(lib, d, good, ws=None) == G.GDN_ERR_WORKSPACE


def test_commit_and_pages_refuse(lib):
    d = dims()
    for n in (0, 1, 66):
        assert commit(lib, d, n_nodes=n) == G.GDN_ERR_DIMS
    many = dims(layers=2048, h_q=1024, h_kv=1024)
    assert commit(lib, many) == G.GDN_ERR_DIMS and fork(lib, many) == G.GDN_ERR_DIMS
    for name in ("node", "ctx", "table", "k", "v", "out"):
        assert commit(lib, d, **{name: None}) == G.GDN_ERR_NULL, name
    for name in ("k", "v"):
        assert commit(lib, d, **{name: FAKE + 4}) == G.GDN_ERR_ALIGN, name
        assert fork(lib, d, **{name: FAKE + 4}) == G.GDN_ERR_ALIGN, name
        assert fork(lib, d, **{name: None}) == G.GDN_ERR_NULL, name
    for name in ("parent", "node", "ctx", "table", "out", "st"):
        assert commit(lib, d, **{name: FAKE + 2}) == G.GDN_ERR_ALIGN, name
    for name in ("want", "table", "ref"):
        assert resize(lib, d, **{name: None}) == G.GDN_ERR_NULL, name
        assert resize(lib, d, **{name: FAKE + 2}) == G.GDN_ERR_ALIGN, name
    for name in ("src", "dst", "table", "ctx", "ref"):
        assert fork(lib, d, **{name: None}) == G.GDN_ERR_NULL, name
        assert fork(lib, d, **{name: FAKE + 2}) == G.GDN_ERR_ALIGN, name
    for n in (0, 3):
        assert fork(lib, d, n=n) == G.GDN_ERR_DIMS
    need = G.kv_pages_workspace_bytes(d)
    for call in (resize, fork):
        for bad in (dict(ws=None), dict(ws=FAKE + 16), dict(wsb=need - 1)):
            assert call(lib, d, **bad) == G.GDN_ERR_WORKSPACE, bad
        assert call(lib, d, st=FAKE + 1) == G.GDN_ERR_ALIGN


def test_sample_refuses(lib):
    for bad in (dict(batch=0), dict(batch=70000), dict(n=0), dict(n=66), dict(vocab=0)):
        assert sample(lib, **bad) == G.GDN_ERR_DIMS, bad
    for name in ("logits", "tokens", "u", "noise", "al", "an", "nt"):
        assert sample(lib, **{name: None}) == G.GDN_ERR_NULL, name
    for name in ("logits", "q", "tokens", "parent", "temp", "u", "noise", "al", "an", "nt", "prob", "st"):
        assert sample(lib, **{name: FAKE + 2}) == G.GDN_ERR_ALIGN, name
    need = G.spec_accept_sample_workspace_bytes(2, 5)
    for bad in (dict(ws=None), dict(ws=FAKE + 16), dict(wsb=need - 1)):
        assert sample(lib, **bad) == G.GDN_ERR_WORKSPACE, bad
    assert G.spec_accept_sample_workspace_bytes(0, 5) == 0 and G.spec_accept_sample_workspace_bytes(1, 66) == 0


def test_binding_raises(lib):
    with pytest.raises(G.GdnError) as e:
        G.attn_verify_span(dims(), 0, FAKE, FAKE, FAKE, FAKE, FAKE, 1.0, FAKE, FAKE, 1 << 30, None, 0)
    assert e.value.status == G.GDN_ERR_DIMS


def test_reference_forms_agree_with_each_other():
    """The tests' own plain forms: a tree's node sees what the chain of its root
    path sees, and the closed rest of a row is the rest taken step by step."""
    g = np.random.default_rng(0)
    T, n, d = 9, 5, 8
    p = R.random_tree(g, T + 1)
    q, k, v = (g.standard_normal(s) for s in ((T, 2, d), (n + T, 1, d), (n + T, 1, d)))
    out, _, _ = R.attention(q, k, v, p, n, 0.3)
    for t in range(T):
        path = R.path_of(p, t + 1)
        rows = list(range(n)) + [n + i - 1 for i in path]
        one, _, _ = R.attention(q[[i - 1 for i in path]], k[rows], v[rows], R.chain(len(path) + 1), n, 0.3)
        np.testing.assert_allclose(one[-1], out[t], rtol=1e-12)
    pr, dr = (x / x.sum() for x in g.random((2, 50)))
    rest, c, mass = pr.copy(), 0.0, 1.0
    for _ in range(4):
        c, rest = c + mass, np.maximum(rest - dr, 0) / max(np.maximum(rest - dr, 0).sum(), 1e-300)
        mass = np.maximum(pr - c * dr, 0).sum()
        np.testing.assert_allclose(np.maximum(pr - c * dr, 0) / mass, rest, atol=1e-12)
