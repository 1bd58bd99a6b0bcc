"""HybridStep.fork without a GPU: what it queues and where, by a step whose tensors
have no memory (torch's meta device) and a library that only notes its calls."""
import contextlib

import numpy as np
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from speculative_decode_hybrid_gb300 import hybrid as H


class Notes:
    """The library's calls, in the place of hybrid.G."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append((name, a))


class Holder:
    pass


def meta(*shape, dtype=torch.int32):
    return torch.empty(shape, dtype=dtype, device="meta")


def step(monkeypatch, B=4, tree=False):
    h = H.HybridStep.__new__(H.HybridStep)
    g = h.gdn = Holder()
    g.ssm_state, g.conv_state, g.tokens, g.logits = meta(B, 2, 3), meta(B, 2, 3), meta(B, 5), meta(B, 5, 7)
    g.tree = tree
    g.parent_host = np.tile(np.arange(-1, 4, dtype=np.int32), (B, 1)) if tree else None
    g.parent = meta(B, 5) if tree else None
    h.shape = Holder()
    h.shape.batch, h.shape.n_tok = B, 4
    h.dims, h.status = None, meta(1)
    h.want, h.ctx, h.table, h.page_ref = meta(B), meta(B), meta(B, 9), meta(30)
    h.every = meta(B, dtype=torch.long)
    h.page_ws, h.k_pages, h.v_pages = meta(64), meta(8), meta(8)
    notes = Notes()
    monkeypatch.setattr(H, "G", notes)
    return h, notes


class Where(TorchDispatchMode):
    """Notes which torch operations run outside of on_stream."""

    def __init__(self, monkeypatch):
        super().__init__()
        self.inside, self.outside, self.streams = 0, [], []
        monkeypatch.setattr(H, "on_stream", self.on_stream)

    @contextlib.contextmanager
    def on_stream(self, stream):
        self.streams.append(stream)
        self.inside += 1
        yield
        self.inside -= 1

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if not self.inside and any(t.device.type == "meta" for t in (out if isinstance(out, (tuple, list)) else [out]) if isinstance(t, torch.Tensor)):
            self.outside.append(str(func))
        return out


def test_all_that_a_fork_makes_is_on_its_stream(monkeypatch):
    """The request numbers are read by what is queued on the given stream: made on another, their memory could be
    given away and written again before it has been read."""
    h, notes = step(monkeypatch)
    with Where(monkeypatch) as w:
        h.fork([0, 0], [1, 3], stream=77)
    assert w.outside == [] and set(w.streams) == {77}
    assert [n for n, _ in notes.calls] == ["kv_pages_resize", "kv_pages_fork", "kv_pages_resize"]
    assert all(a[-1] == 77 for _, a in notes.calls)


@pytest.mark.parametrize("src,dst", [([0], [0]), ([0, 1], [1, 2]), ([0, 2], [1, 1]), ([0], [4]), ([4], [0]), ([-1], [1]), ([0], [-1]),
                                     ([0], [1, 2]), ([0, 0], [1])], ids=str)
def test_requests_that_cannot_be_forked(monkeypatch, src, dst):
    """A copy of itself or of one that is being replaced, the same place twice, numbers that are none of the batch, lists
    of different lengths: refused before anything is queued or given back."""
    h, notes = step(monkeypatch)
    with Where(monkeypatch) as w, pytest.raises(ValueError):
        h.fork(src, dst)
    assert notes.calls == [] and w.streams == []


def test_the_tree_goes_with_its_tokens(monkeypatch):
    """A tree of each request: the copy has its source's, in the host's array too; the array that was given is left as it was."""
    h, _ = step(monkeypatch, tree=True)
    g = h.gdn
    g.parent_host[0] = [-1, 0, 0, 1, 1]
    given, before = g.parent_host, g.parent_host.copy()
    copied = []
    monkeypatch.setattr(torch.Tensor, "__setitem__", lambda self, i, v: copied.append(self))
    h.fork([0, 0], [1, 3])
    np.testing.assert_array_equal(g.parent_host, before[[0, 0, 2, 0]])
    np.testing.assert_array_equal(given, before)
    assert any(t is g.parent for t in copied) and any(t is g.tokens for t in copied)
