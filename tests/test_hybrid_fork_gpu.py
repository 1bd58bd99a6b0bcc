"""HybridStep.fork on the GPU: on a stream other than the current one."""
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


def small(wid=4, ctx=(130, 3, 0, 40), **kw):
    from speculative_decode_hybrid_gb300.hybrid import AttnShape, HybridStep
    shape = AttnShape(layers=2, h_q=4, h_kv=2, d_head=64, rot_dim=32, page_tokens=16, max_tokens=256)
    return HybridStep(W.make_workload(wid, seed=5, batch=len(ctx), layers=2, vocab=512), shape, list(ctx), temperature=0.7, seed=2, **kw)


def held(h):
    """What a fork leaves, the pages' contents by request."""
    rows = [h.k_pages[:, h.table[b, :(n + 15) // 16].long()] for b, n in enumerate(h.ctx.tolist())]
    return [h.ctx, h.table, h.page_ref, h.gdn.ssm_state, h.gdn.conv_state, h.gdn.tokens, h.gdn.logits] + rows


@pytest.mark.parametrize("handle", [False, True])
def test_forks_on_the_stream_that_is_given(handle):
    """Beside a busy current stream that takes and writes small tensors as soon as the fork has returned."""
    want, h = small(), small()
    for src, dst in (([0, 3], [1, 2]), ([1], [3])):
        want.fork(src, dst)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = torch.cuda.Event()
    torch.cuda._sleep(400_000_000)          # some 0.2 s
    busy.record()
    kept = []
    for src, dst in (([0, 3], [1, 2]), ([1], [3])):
        h.fork(src, dst, stream=side.cuda_stream if handle else side)
        kept += [torch.full((2,), 0, dtype=torch.int32, device="cuda") for _ in range(64)]
    side.synchronize()
    assert not busy.query()                 # nothing of it waited for the current stream
    torch.cuda.synchronize()
    assert int(h.status.item()) == 0
    for x, y in zip(held(want), held(h)):
        assert torch.equal(x, y)


def test_forked_trees():
    """Each request has a tree of its own: a copy's acceptance with its source's random numbers is its source's."""
    h = small(wid=3)
    assert not (h.gdn.parent[0] == h.gdn.parent[2]).all()
    h.fork([0, 0], [2, 3])
    for _ in range(2):
        h.draw()
        for x in (h.uniforms, h.noise):
            x[2:] = x[0]
        h.step()
        torch.cuda.synchronize()
        assert int(h.status.item()) == 0
        for x in (h.gdn.parent, h.accept_len, h.accept_node, h.next_token, h.ctx, h.gdn.tokens, h.token_prob):
            assert torch.equal(x[2], x[0]) and torch.equal(x[3], x[0])
        assert (h.gdn.parent.cpu().numpy() == h.gdn.parent_host).all()
