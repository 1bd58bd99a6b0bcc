"""The sampled next token as node 1 of the next span: two steps in a row commit
a sample of the target's chain. The rule (node 1 with uniform 0, row 0 the row
that the token was drawn from) is tried on the plain form, where breaking it is
seen, and on the library."""
import numpy as np
import pytest

import attn_reference as R

V = 4
# rows: the target's next-token distribution after each token, the last after the prompt
P = np.array([[0.55, 0.2, 0.15, 0.1], [0.05, 0.15, 0.1, 0.7], [0.3, 0.4, 0.2, 0.1], [0.1, 0.1, 0.6, 0.2], [0.4, 0.1, 0.3, 0.2]])
PARENT = np.array([-1, 0, 1, 1, 2], np.int32)      # node 1 has two children, the first has one


def plain(logits, q, tokens, parent, uniforms, noise):
    got = [R.sample(logits[b], None if q is None else q[b].astype(np.float64), tokens[b], parent, 1.0, uniforms[b], noise[b])[:3]
           for b in range(len(logits))]
    return np.array(got).T


def committed(accept, B, drawn, rule, seed):
    """The first three tokens that B requests commit in two steps."""
    g = np.random.default_rng(seed)
    draft = np.array([[0.1, 0.3, 0.3, 0.3], [0.4, 0.2, 0.2, 0.2], [0.25, 0.25, 0.25, 0.25], [0.3, 0.3, 0.1, 0.3], [0.25] * 4])
    pick = lambda p: np.array([g.choice(V, p=x) for x in p])
    last = pick(np.tile(P[V], (B, 1)))             # the prompt's own sample
    row0 = np.tile(P[V], (B, 1))
    out = [[int(x)] for x in last]                 # every token counts once, when it is first drawn or accepted
    N = len(PARENT)
    for _ in range(2):
        tokens = np.zeros((B, N), np.int32)
        tokens[:, 1] = last
        for i in range(2, N):
            above = tokens[:, PARENT[i]]
            tokens[:, i] = pick(draft[above]) if drawn else (above + i) % V
        rows = np.stack([row0] + [P[tokens[:, n]] for n in range(1, N)], 1)
        q = np.stack([np.tile(draft[V], (B, 1))] + [draft[tokens[:, n]] for n in range(1, N - 1)], 1) if drawn else None
        u = g.random((B, N)).astype(np.float32)
        if rule:
            u[:, 1] = 0.0
        noise = (g.exponential(size=(B, V)) + 1e-9).astype(np.float32)
        length, node, token = accept(np.log(rows).astype(np.float32), None if q is None else q.astype(np.float32), tokens, PARENT, u,
                                     noise)
        for b in range(B):
            path = R.path_of(PARENT, int(node[b]))
            if 1 not in path:
                out[b].pop()                       # the token that was drawn is tested again and lost
            out[b] += [int(tokens[b, i]) for i in path if i != 1] + [int(token[b])]
        last, row0 = np.asarray(token), rows[np.arange(B), np.asarray(node)]
    return np.array([x[:3] if len(x) >= 3 else x + [-1] * (3 - len(x)) for x in out])


def deviation(seq):
    """The largest deviation of a triple's frequency, in standard deviations."""
    seq = seq[(seq >= 0).all(1)]
    p = np.einsum("a,ab,bc->abc", P[V], P[:V], P[:V]).ravel()
    n = len(seq)
    counts = np.bincount((seq[:, 0] * V + seq[:, 1]) * V + seq[:, 2], minlength=V ** 3)
    return float(np.max(np.abs(counts - n * p) / np.sqrt(n * p * (1 - p))))


@pytest.mark.parametrize("drawn", [False, True])
def test_plain_form_two_steps(drawn):
    assert deviation(committed(plain, 8000, drawn, True, 1)) < 5          # 64 cells: five standard deviations
    assert deviation(committed(plain, 8000, drawn, False, 1)) > 10        # a second test of the token shows


@pytest.mark.gpu
@pytest.mark.parametrize("drawn", [False, True])
def test_library_two_steps(drawn):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from gpu_helpers import ensure_built
    from speculative_decode_hybrid_gb300 import gdnspec as G
    ensure_built()

    def accept(logits, q, tokens, parent, uniforms, noise):
        B, N, _ = logits.shape
        dev = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()
        ints = torch.zeros((3, B), dtype=torch.int32, device="cuda")
        wsb = G.spec_accept_sample_workspace_bytes(B, N)
        ws = torch.zeros(wsb, dtype=torch.uint8, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        keep = [dev(x) for x in (logits, q, tokens, np.tile(parent, (B, 1)), uniforms, noise)]
        G.spec_accept_sample(B, N, V, keep[0], keep[1], keep[2], keep[3], None, keep[4], keep[5], ints[0], ints[1], ints[2], None, ws,
                             wsb, st)
        assert int(st.item()) == 0
        length, node, token = ints.cpu().numpy()
        assert np.all(length >= 1)                # node 1 is never refused
        return length, node, token
    assert deviation(committed(accept, 40000, drawn, True, 2)) < 5
