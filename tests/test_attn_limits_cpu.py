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
