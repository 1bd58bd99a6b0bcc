"""The hybrid step's own parts on the GPU: streams other than the current one."""
import pytest
import torch

from gpu_helpers import ensure_built
from speculative_decode_hybrid_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()


def small(seed=2, ctx=(40, 3, 0), **kw):
    from speculative_decode_hybrid_gb300.hybrid import AttnShape, HybridStep
    shape = AttnShape(layers=2, h_q=4, h_kv=2, d_head=64, rot_dim=32, page_tokens=16, max_tokens=192)
    return HybridStep(W.make_workload(3, seed=5, batch=len(ctx), layers=2, vocab=512), shape, list(ctx), seed=seed, **kw)


@pytest.mark.parametrize("handle", [False, True])
def test_room_is_made_on_the_stream_that_is_given(handle):
    """The lengths grow on a side stream while the current one is busy: the room
    is that of the new lengths, and nothing of it waits for the current stream."""
    h = small()
    T = h.shape.n_tok
    side = torch.cuda.Stream()
    more = torch.tensor([50, 0, 17], dtype=torch.int32, device="cuda")
    h.ctx.add_(more).sub_(more)             # what is loaded or allocated at first use is there
    h.make_room(side)
    h.table.cpu()
    torch.cuda.synchronize()
    before = torch.cuda.Event()
    torch.cuda._sleep(400_000_000)          # some 0.2 s
    before.record()
    with torch.cuda.stream(side):
        h.ctx.add_(more)
    h.make_room(side.cuda_stream if handle else side)
    with torch.cuda.stream(side):
        table, ref = h.table.cpu(), h.page_ref.cpu()
    assert not before.query()               # the current stream is still at it
    want = [-(-(n + T) // 16) for n in (90, 3, 17)]
    assert [(row >= 0).sum().item() for row in table] == want
    assert int(ref.sum()) == sum(want) and int(h.status.item()) == 0


def test_the_next_token_begins_the_next_span():
    """Node 1 is the token sampled last, row 0 the row it was drawn from, and it
    is not tested a second time."""
    h = small(ctx=(40, 3, 0, 9), temperature=0.5)
    for step in range(6):
        h.draw()
        tokens, length = h.gdn.tokens.clone(), h.ctx.clone()
        rows = h.gdn.logits.clone()
        h.step()
        assert int(h.status.item()) == 0
        node, taken = h.accept_node.tolist(), h.accept_len.tolist()
        for b in range(4):
            assert taken[b] >= 1, step
            i = node[b]
            while h.gdn.parent_host[b][i] > 0:
                i = int(h.gdn.parent_host[b][i])
            assert i == 1                                      # the root's first child is on the path
            assert int(h.ctx[b]) == int(length[b]) + taken[b]
            assert torch.equal(h.gdn.logits[b, 0], rows[b, node[b]])
            assert torch.equal(h.gdn.logits[b, 1:], rows[b, 1:])
        assert torch.equal(h.gdn.tokens[:, 1], h.next_token) and torch.equal(h.gdn.tokens[:, 2:], tokens[:, 2:])
        # the next step's probability of node 1 is what the token was drawn with
        drawn = h.token_prob[:, 0].clone()
        h.accept()
        torch.testing.assert_close(h.token_prob[:, 1], drawn, rtol=1e-5, atol=0)


def test_room_on_the_current_and_the_default_stream():
    h = small()
    for stream in (None, 0, torch.cuda.default_stream()):
        h.ctx.add_(16)
        h.make_room(stream)
        assert [(row >= 0).sum().item() for row in h.table.cpu()] == [-(-(n + h.shape.n_tok) // 16) for n in h.ctx.tolist()]
    assert int(h.status.item()) == 0
