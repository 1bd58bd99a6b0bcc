"""A bias by distance whose slopes are below zero, with a window or a document that
begins far into the context: the weight lies where the row begins to see, and the
result's error is held to distances from there."""
import numpy as np
import pytest
import torch

import attn_reference as R
from attn_reference import U16, U32
from gpu_helpers import ensure_built
from speculative_decode_hybrid_gb300 import gdnspec as G
from test_attn_ex_gpu import attend
from test_attn_gpu import TYPES, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()


class Late:
    """Requests of any length of which only the slots from `since` on have pages."""

    def __init__(self, g, ctx, since, T, h_kv, d, page, dtype):
        self.ctx, self.page, self.h_kv = list(ctx), page, h_kv
        self.dt, self.dtype = TYPES[dtype]
        self.width = max(-(-(n + T) // page) for n in ctx)
        self.table = np.full((len(ctx), self.width), -1, np.int32)
        at = 0
        for b, (n, s) in enumerate(zip(ctx, since)):
            k = -(-(n + T) // page) - s // page
            self.table[b, s // page:s // page + k] = np.arange(at, at + k)
            at += k
        self.n_pages, self.d = at, d
        gen = torch.Generator("cuda").manual_seed(int(g.integers(1 << 30)))
        self.k, self.v = (torch.randn((at, h_kv, page, d), device="cuda", generator=gen).to(self.dt) for _ in range(2))
        self.table_dev = torch.from_numpy(self.table).cuda()
        self.ctx_dev = torch.tensor(self.ctx, dtype=torch.int32, device="cuda")

    def dims(self, h_q, batch=None):
        return G.make_attn_dims(len(self.ctx), 1, h_q, self.h_kv, self.d, self.page, self.n_pages, self.width, self.dtype)

    def rows(self, b, slots):
        page, off = torch.from_numpy(self.table[b, slots // self.page].astype(np.int64)).cuda(), torch.from_numpy(slots % self.page).cuda()
        return f64(self.k[page, :, off]), f64(self.v[page, :, off])


def check(cache, q, parents, out, scale, slopes, window, first):
    """A score's error: its sum's (D roundings), the exponential's (2^-21), the bias's, a few
    roundings of its distance from the place where the bias is zero: the node's own position, or for
    a slope below 0 the first slot that the row sees, at most a tile's 64 slots aside. From there as
    attn_reference.attention_bound."""
    T, Hq, D = q.shape[1:]
    bf16 = cache.dtype == G.GDN_BF16
    for b, n in enumerate(cache.ctx):
        since = max(first[b] if first else 0, n + 1 - window if window else 0)
        k, v = cache.rows(b, np.arange(since, n + T))
        parent = R.chain(T + 1) if parents is None else parents[b]
        for t in range(T):
            path = R.path_of(parent, t + 1)
            own = n + len(path) - 1
            slot = np.r_[np.arange(since, n), [n + i - 1 for i in path]].astype(int)
            place = np.r_[np.arange(since, n), n + np.arange(len(path))]
            if window:
                keep = own - place < window
                slot, place = slot[keep], place[keep]
            for h in range(Hq):
                kk, vv = k[slot - since, h * cache.h_kv // Hq], v[slot - since, h * cache.h_kv // Hq]
                qq = f64(q[b, t, h])
                z, big = scale * (kk @ qq), scale * (np.abs(kk) @ np.abs(qq))
                zero = place[0] if slopes[h] < 0 else own
                bias = float(slopes[h]) * (place - zero)
                delta = 2 * (D + 2) * U32 * big + 2.0 ** -21 + 2.0 ** -21 * (np.abs(float(slopes[h])) * (np.abs(place - zero) + 64) + np.abs(z))
                z = z + bias
                p = np.exp(z - z.max())
                p /= p.sum()
                want, mass = p @ vv, p @ np.abs(vv)
                bound = 2 * ((p * delta) @ np.abs(vv) + (p @ delta) * mass) + (4 * len(slot) * U32 + (U16 if bf16 else 0.0)) * mass
                bound += (U16 if bf16 else 4 * U32) * np.abs(want) + 1e-30
                err = np.abs(f64(out[b, t, h]) - want)
                assert np.all(err <= bound), (b, t, h, float((err / bound).max()))


SLOPES = np.array([-1.0, 0.5, -0.25, -2.0 ** -8, 0.0, -0.03], np.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,late", [(200, False), (1500, False), (0, True), (300, True)], ids=str)
@pytest.mark.parametrize("T,tree,d", [(1, False, 256), (5, False, 64), (22, True, 128)])
def test_slopes_below_zero_far_into_the_context(dtype, window, late, T, tree, d):
    g = np.random.default_rng(T)
    ctx = [8_000_000, 100_001, 1_000_077]
    first = [n - x for n, x in zip(ctx, (400, 33, 1000))] if late else None
    since = [max(first[b] if late else 0, n + 1 - window if window else 0) for b, n in enumerate(ctx)]
    cache = Late(g, ctx, since, T, 2, d, 32, dtype)
    q = torch.randn((3, T, 6, d), device="cuda", generator=torch.Generator("cuda").manual_seed(T)).to(cache.dt)
    parents = np.stack([R.random_tree(g, T + 1) for _ in ctx]) if tree else None
    out, st = attend(cache, q, parents, d ** -0.5, window=window, slopes=SLOPES, first=first)
    assert st == 0
    check(cache, q, parents, out, d ** -0.5, SLOPES, window, first)
