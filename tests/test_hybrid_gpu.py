"""The hybrid step: GDN layers, attention layers, sampled acceptance and commit
together, against what plain decoding of the accepted tokens would leave."""
import numpy as np
import pytest
import torch

import attn_reference as R
from gpu_helpers import ensure_built
from speculative_decode_hybrid_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()


def rows(h, pool, y, b, slots):
    page = h.attn.page_tokens
    t = h.table[b].tolist()
    return torch.stack([pool[y, t[s // page], :, s % page] for s in slots]) if len(slots) else pool[y, :0, :, 0]


@pytest.mark.parametrize("wid", [0, 3])
def test_hybrid_step_commits_what_plain_decoding_would(wid):
    from speculative_decode_hybrid_gb300.hybrid import AttnShape, HybridStep
    wl = W.make_workload(wid, seed=3, batch=3, layers=2, vocab=1024)
    shape = AttnShape(layers=2, h_q=4, h_kv=2, d_head=64, rot_dim=32, page_tokens=16, max_tokens=192)
    h = HybridStep(wl, shape, [30, 0, 17], seed=1)
    T, bf16 = wl.shape.n_tok, wl.shape.dtype == W.GDN_BF16
    rope = h.rope.double().cpu().numpy()
    for step in range(3):
        h.draw()
        ctx = h.ctx.tolist()
        before = [rows(h, h.k_pages, y, b, range(n)).clone() for y in range(2) for b, n in enumerate(ctx)]
        h.gdn.verify()
        for y in range(2):
            h.attend(y)
        out = h.attn_out.double().cpu().numpy()
        parents = [R.chain(T + 1) if wl.parent is None else wl.parent[b] for b in range(3)]
        for y in range(2):            # the span's attention, from the cache as it stands
            for b, n in enumerate(ctx):
                k, v = (rows(h, p, y, b, range(n + T)).double().cpu().numpy() for p in (h.k_pages, h.v_pages))
                x = h.qkv[y, b].double().cpu().numpy().reshape(T, 8, 64)
                q = np.stack([R.norm_rope(x[t, :4].copy(), h.q_norm[y].double().cpu().numpy(), 1e-6, 1.0, rope, 32,
                                          n + len(R.path_of(parents[b], t + 1)) - 1, False) for t in range(T)])
                qq = torch.from_numpy(q).to(h.q.dtype).double().numpy()      # as the attention gets it
                want, mass, big = R.attention(qq, k, v, parents[b], n, 64 ** -0.5)
                bound = R.attention_bound(want, mass, big, 64, n + T, bf16)
                # a q within its bound may round to the other side: one unit of the type more
                bound = bound + 2 * (R.U16 if bf16 else 8 * R.U32) * big * mass
                assert np.all(np.abs(out[y, b] - want) <= bound), (step, y, b)
        span = [[rows(h, p, y, b, range(n, n + T)).clone() for p in (h.k_pages, h.v_pages)] for y in range(2) for b, n in enumerate(ctx)]
        state = h.gdn.ssm_state.clone()
        h.accept()
        h.commit()
        h.ctx.copy_(h.ctx_next)
        h.make_room()
        assert int(h.status.item()) == 0
        for b, n in enumerate(ctx):
            node = int(h.accept_node[b])
            path = R.path_of(parents[b], node)
            assert int(h.accept_len[b]) == len(path) and int(h.ctx[b]) == n + len(path)
            want = state[b] if node == 0 else h.gdn.ssm_ckpt[b, :, node - 1]
            assert torch.equal(h.gdn.ssm_state[b], want)
            for y in range(2):
                at = [i - 1 for i in path]
                k, v = span[y * 3 + b]
                assert torch.equal(rows(h, h.k_pages, y, b, range(n, n + len(path))), k[at])
                assert torch.equal(rows(h, h.v_pages, y, b, range(n, n + len(path))), v[at])
                assert torch.equal(rows(h, h.k_pages, y, b, range(n)), before[y * 3 + b])   # the past stays
        need = sum(-(-(int(n) + T) // 16) for n in h.ctx.tolist())
        assert int(h.page_ref.sum()) == need == int((h.table >= 0).sum())


def test_hybrid_step_runs_in_a_graph():
    from speculative_decode_hybrid_gb300.hybrid import AttnShape, HybridStep
    shape = AttnShape(layers=2, h_q=4, h_kv=2, d_head=128, rot_dim=128, page_tokens=32, max_tokens=512)

    def fresh():
        return HybridStep(W.make_workload(4, seed=5, batch=2, layers=2, vocab=4096), shape, [40, 100], seed=2)
    a, b = fresh(), fresh()
    for _ in range(3):
        a.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    b.step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        b.step()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert a.ctx.tolist() == b.ctx.tolist() and a.next_token.tolist() == b.next_token.tolist()
    assert torch.equal(a.attn_out, b.attn_out) and torch.equal(a.k_pages, b.k_pages)
    assert torch.equal(a.gdn.ssm_state, b.gdn.ssm_state)
