"""Where the attention-layer, page and sampling calls stop: sizes at which an
index of a kernel would leave its range, and arguments that overlap, are refused
on the host. A size that fits is recognised by the refusal of the (missing)
workspace, which comes last, so nothing is queued either way."""
import ctypes

import pytest

from speculative_decode_hybrid_gb300 import build as B
from speculative_decode_hybrid_gb300 import gdnspec as G

FAKE = 0x10000  # an aligned non-NULL address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    B.build()
    return G.load()


def sample(lib, vocab, **kw):
    a = dict(batch=1, n=1, vocab=vocab, logits=FAKE, q=FAKE, tokens=FAKE, parent=None, temp=None, u=FAKE, noise=FAKE, al=FAKE,
             an=FAKE, nt=FAKE, prob=None, ws=None, wsb=0, st=None)
    a.update(kw)
    return lib.spec_accept_sample(*a.values(), None)


@pytest.mark.parametrize("batch,n", [(1, 1), (1, 65), (40, 9)])
def test_sample_vocabulary_limit(lib, batch, n):
    """Up to 2^30 a row's slices, their rounding to whole pieces and the last
    step past the end stay in 31 bits; the number of pieces stays within the
    workspace's places."""
    assert sample(lib, 2 ** 30, batch=batch, n=n) == G.GDN_ERR_WORKSPACE
    for v in (2 ** 30 + 1, 2 ** 31 - 2 ** 14, 2 ** 31 - 39, 2 ** 31 - 8, 2 ** 31 - 1):
        assert sample(lib, v, batch=batch, n=n) == G.GDN_ERR_DIMS, v


def dims(**kw):
    d = dict(batch=1, layers=1, h_q=8, h_kv=8, d_head=64, page_tokens=256, n_pages=40, table_width=9, dtype=G.GDN_BF16)
    d.update(kw)
    return G.make_attn_dims(*d.values())


def span(lib, d, n_tok=1):
    return lib.attn_verify_span(ctypes.byref(d), n_tok, *[FAKE] * 5, 0.1, FAKE, None, 0, None, None)


@pytest.mark.parametrize("n_tok,fits,over", [
    # a request's tiles of 64 slots x heads x 128-row groups reach 2^31 (a table may repeat a page)
    (1, dict(h_q=1024, h_kv=512, table_width=2 ** 20 - 1), dict(h_q=1024, h_kv=512, table_width=2 ** 20)),
    (64, dict(h_q=1024, h_kv=1, table_width=2 ** 20 - 1), dict(h_q=1024, h_kv=1, table_width=2 ** 20)),
    # the requests' together reach 2^34
    (1, dict(batch=31, h_q=1024, h_kv=1024, table_width=2 ** 17), dict(batch=32, h_q=1024, h_kv=1024, table_width=2 ** 17)),
    (8, dict(batch=65535, h_q=64, h_kv=1, table_width=2 ** 14), dict(batch=65535, h_q=256, h_kv=1, table_width=2 ** 14))])
def test_bf16_attention_tile_limit(lib, n_tok, fits, over):
    assert span(lib, dims(**fits), n_tok) == G.GDN_ERR_WORKSPACE and G.attn_workspace_bytes(dims(**fits), n_tok) > 0
    assert span(lib, dims(**over), n_tok) == G.GDN_ERR_DIMS and G.attn_workspace_bytes(dims(**over), n_tok) == 0
    f32 = dims(**dict(over, dtype=G.GDN_F32))       # counts in 64 bits where it has to
    assert span(lib, f32, n_tok) == G.GDN_ERR_WORKSPACE


@pytest.mark.parametrize("parent", [None, FAKE])
def test_commit_refuses_lengths_in_place(lib, parent):
    """Blocks of a request would read the length that another has replaced."""
    d = dims(batch=6)
    for out in (FAKE, FAKE + 4, FAKE + 20, FAKE - 4, FAKE - 20):
        assert lib.kv_commit_path(ctypes.byref(d), 4, parent, FAKE, FAKE, FAKE, FAKE, FAKE, out, None, None) == G.GDN_ERR_OVERLAP
    assert "overlap" in G.status_str(G.GDN_ERR_OVERLAP)
