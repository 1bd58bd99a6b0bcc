"""Plain 64-bit forms of the attention-layer, cache-page and sampled-acceptance
calls, written from their definitions in numpy, and the error bounds that the
GPU results are held to. Nothing here uses the library."""
import numpy as np

U16 = 2.0 ** -8    # unit roundoff of bf16: 8 significant bits, half of a unit in the last (7th) fraction place
U32 = 2.0 ** -24   # unit roundoff of f32


def path_of(parent, i):
    """Nodes from below the root to i."""
    got = []
    while i > 0:
        got.append(i)
        i = int(parent[i])
    return got[::-1]


def chain(n_nodes):
    return np.arange(-1, n_nodes - 1, dtype=np.int32)


def random_tree(g, n_nodes, straight=0.4):
    p = chain(n_nodes)
    for i in range(2, n_nodes):
        if g.random() >= straight:
            p[i] = g.integers(0, i)
    return p


def attention(q, k, v, parent, ctx, scale):
    """q [T][Hq][D], k, v [slots][Hkv][D] (slots = ctx + T), all float64.
    Returns out and, per element, sum p |v| and the largest sum |q_i k_i| of a
    row's scores: what the bounds are made of."""
    T, Hq, D = q.shape
    Hk = k.shape[1]
    out, mass, big = np.zeros_like(q), np.zeros_like(q), np.zeros((T, Hq, 1))
    for t in range(T):
        seen = list(range(ctx)) + [ctx + i - 1 for i in path_of(parent, t + 1)]
        for h in range(Hq):
            kk, vv = k[seen, h * Hk // Hq], v[seen, h * Hk // Hq]
            s = scale * (kk @ q[t, h])
            with np.errstate(invalid="ignore", over="ignore"):
                p = np.exp(s - s.max())
                p /= p.sum()
                out[t, h], mass[t, h] = p @ vv, p @ np.abs(vv)
            big[t, h] = scale * np.max(np.abs(kk) @ np.abs(q[t, h]))
    return out, mass, big


def attention_bound(out, mass, big, D, slots, bf16):
    """A score's rounding errors, D of them relative to sum |q_i k_i|, and the
    exponential's (argument and result: 2^-21) move each weight by a factor
    1 +- delta; a weighted mean of v then moves by 2 delta sum p |v|, and its f32
    sums over the slots by 2 slots u. bf16: each weight is rounded to u16 once
    more (not the divisor), and so is the result. Twice u32 for sums, whose order
    and rounding on the tensor cores is not f32's."""
    delta = 2 * (D + 2) * U32 * big + 2.0 ** -21
    bound = (2 * delta + 4 * slots * U32 + (U16 if bf16 else 0.0)) * mass
    return bound + (U16 if bf16 else 4 * U32) * np.abs(out) + 1e-30


def norm_rope(x, w, eps, offset, rope, rot, pos, pairs):
    """x [heads][D] of one token."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (w + offset)
    if rot:
        c, s = rope[pos, :rot // 2], rope[pos, rot // 2:]
        i = np.arange(rot // 2) * (2 if pairs else 1)
        j = i + (1 if pairs else rot // 2)
        yi, yj = y[:, i].copy(), y[:, j].copy()
        y[:, i], y[:, j] = yi * c - yj * s, yj * c + yi * s
    return y


def norm_bound(y, D, bf16):
    """Relative to a head's largest value: the sum of D squares (D u, halved by
    the root), the reciprocal root's two units, and a rotation's six roundings;
    bf16: the result's rounding, relative to itself."""
    top = np.abs(y).max(-1, keepdims=True)
    return (0.5 * (D + 2) * U32 + 12 * U32) * top + (U16 if bf16 else U32) * np.abs(y) + 1e-30


def sample(logits, q, tokens, parent, temperature, uniforms, noise):
    """One request. Returns accept_len, accept_node, next_token, token_prob and
    the smallest relative margin of a decision it took."""
    n, v = logits.shape
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        z = logits.astype(np.float64)
        z = z - z.max(-1, keepdims=True)
        e = np.exp(z / temperature) if temperature > 0 else (z == 0).astype(np.float64)
        p = e / e.sum(-1, keepdims=True)
    prob = np.zeros(n)
    for i in range(1, n):
        ok = 0 <= parent[i] < i and 0 <= tokens[i] < v
        prob[i] = p[parent[i], tokens[i]] if ok else 0.0
    at = depth = 0
    margin = np.inf
    while True:
        rest, hit = p[at].copy(), None
        dead = np.isnan(rest).any()
        for i in [j for j in range(1, n) if parent[j] == at]:
            x = int(tokens[i])
            if not dead and 0 <= x < v:
                share = rest[x] / max(rest.sum(), 1e-300)
                a, b = (uniforms[i], share) if q is None else (uniforms[i] * q[at, x], share)
                margin = min(margin, abs(a - b) / max(a, b, 1e-300))
                if a < b:
                    hit = i
                    break
                if q is None:
                    rest[x] = 0.0
            if q is not None and not dead:
                rest = np.maximum(rest / max(rest.sum(), 1e-300) - q[at], 0.0)
        if hit is None:
            break
        at, depth = hit, depth + 1
    if dead:
        return depth, at, 0, prob, margin
    if not rest.max() > 0:
        rest = p[at]
    score = rest / noise
    token = int(np.argmax(score))
    two = np.sort(score)[-2:] if v > 1 else [0.0, 1.0]
    margin = min(margin, (two[1] - two[0]) / two[1])
    prob[0] = p[at, token]
    return depth, at, token, prob, margin


def prob_bound(logits, temperature, V):
    """Relative error of p: the exponential's argument (its rounding relative to
    its size, and the division by T), its result, and a row's sum, taken by 256
    threads and more and joined pairwise."""
    z = np.abs(logits - logits.max()).max() / max(temperature, 1e-6)
    return 4 * U32 * min(z, 200.0) + (V / 256 + 64) * U32 + 2.0 ** -20
