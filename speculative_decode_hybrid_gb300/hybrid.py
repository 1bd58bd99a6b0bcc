"""One sampled speculative step of a hybrid target: its Gated DeltaNet layers
and its full-attention layers together.

    python -m speculative_decode_hybrid_gb300.hybrid [--batch 4] [--attn-layers 16] [--steps 8]

`HybridStep` adds to a workload's `SpecStep` (the GDN layers) the attention
layers' caches in pages and queues, on one stream and with no host
synchronisation, what such a target does with a drafted span:

    kv_pages_resize        room for the span
    gdn_verify_span / gdn_tree_verify          every GDN layer
    attn_qk_norm_rope, attn_verify_span / attn_tree_verify   per attention layer
    spec_accept_sample     acceptance from given random numbers
    gdn_rollback_restore   GDN states of the accepted node
    kv_commit_path         cache rows of the accepted path, the new lengths
    (carry)                the next token as node 1 of the next span

With limits (top_k, top_p, min_p) the target's rows are cut by spec_sample before the
acceptance; with drawn drafts spec_sample draws the span's tokens from a draft's logits
and gives their distributions. `fork` makes requests copies of others (several samples
of a prompt); with `share`, kv_prefix_plan finds what their tables share and the
attention reads it once (attn_*_shared). Layers with capped scores, a window or a bias
by distance use attn_*_ex.

Node 1 of every span is a token that has been sampled (by the step before, for
the first step by the prompt's last row) but not processed yet: it is accepted
without another test (uniform 0), and a step commits one token at least. The first
span's is whatever the workload begins with: a step that cuts it (limits, temperature
0) refuses it and goes on from the root.

The model around the calls (projections, feed-forward layers, the draft) is
the caller's: inputs here are seeded random numbers of its shapes, as the
workloads' are.
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass

import numpy as np
import torch

from . import gdnspec as G
from .pipeline import SpecStep
from .workloads import GDN_BF16, Workload


@dataclass(frozen=True)
class AttnShape:
    """The attention layers of a hybrid target and their cache."""
    layers: int = 16
    h_q: int = 16
    h_kv: int = 2
    d_head: int = 256
    rot_dim: int = 64
    page_tokens: int = 64
    max_tokens: int = 4096      # slots a request's page table holds
    softcap: float = 0.0        # scores capped by softcap * tanh(score / softcap)
    window: int = 0             # positions a node sees back, itself included (0: all)
    bias: bool = False          # scores less slope * distance, slopes 2^(-8 (h + 1) / h_q)


def on_stream(stream):
    """Context in which torch queues where the library's calls do: on the current
    stream (None), a torch stream, or the stream of a handle."""
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


class HybridStep:
    def __init__(self, wl: Workload, attn: AttnShape, ctx_len, temperature: float = 1.0, seed: int = 0, device="cuda",
                 top_k: int = 0, top_p: float = 1.0, min_p: float = 0.0, drafts: bool = False, share: bool = False):
        """ctx_len: committed tokens of each request (their cache rows are
        filled with random keys and values). top_k, top_p, min_p: limits of the
        target's and the draft's distributions (0, 1, 0: none). drafts: the span's
        tokens past node 1 are drawn from a draft's logits (chains). share:
        requests that share pages in front read them once; not with a window. It
        pays for prefixes of tens of thousands of slots (attn_verify_span_shared's
        figures); below, the attention without it is as fast or faster."""
        if drafts and wl.parent is not None:
            raise ValueError("drafts are drawn for chains only")
        if share and attn.window:
            raise ValueError("layers with a window do not share prefixes")
        self.gdn = SpecStep(wl, device=device)
        self.shape, self.attn = wl.shape, attn
        s, a, dev = wl.shape, attn, self.gdn.device
        B, T = s.batch, s.n_tok
        gen = torch.Generator(dev).manual_seed(seed)
        dt = torch.bfloat16 if s.dtype == GDN_BF16 else torch.float32
        width = -(-a.max_tokens // a.page_tokens)
        n_pages = B * width
        self.dims = G.make_attn_dims(B, a.layers, a.h_q, a.h_kv, a.d_head, a.page_tokens, n_pages, width, s.dtype)

        def normal(*shape, dtype=torch.float32):
            return torch.randn(shape, generator=gen, device=dev, dtype=dtype)

        pool = (a.layers, n_pages, a.h_kv, a.page_tokens, a.d_head)
        self.k_pages, self.v_pages = normal(*pool, dtype=dt), normal(*pool, dtype=dt)
        self.table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
        self.page_ref = torch.zeros((n_pages,), dtype=torch.int32, device=dev)
        self.ctx = torch.as_tensor(list(ctx_len), dtype=torch.int32).to(dev)
        self.ctx_next, self.want = torch.empty_like(self.ctx), torch.empty_like(self.ctx)
        # per layer and token the projected row [q | k | v], the norm weights
        self.row = (a.h_q + 2 * a.h_kv) * a.d_head
        self.qkv = normal(a.layers, B, T, self.row, dtype=dt)
        self.q_norm, self.k_norm = (0.1 * normal(a.layers, a.d_head)).to(dt), (0.1 * normal(a.layers, a.d_head)).to(dt)
        self.q = torch.empty((B, T, a.h_q, a.d_head), dtype=dt, device=dev)
        self.attn_out = torch.empty((a.layers, B, T, a.h_q, a.d_head), dtype=dt, device=dev)
        if a.rot_dim:
            inv = 10000.0 ** (-np.arange(0, a.rot_dim, 2) / a.rot_dim)
            angle = np.arange(a.max_tokens)[:, None] * inv
            self.rope = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).to(dev)
        else:
            self.rope = None
        # acceptance: fixed candidates, one set of random numbers (draw() makes new ones)
        self.temperature = torch.full((B,), float(temperature), device=dev)
        self.generator = gen
        self.uniforms = torch.empty((B, s.n_nodes), device=dev)
        self.noise = torch.empty((B, s.vocab), device=dev)
        self.accept_len, self.accept_node, self.next_token = (torch.zeros((B,), dtype=torch.int32, device=dev) for _ in range(3))
        self.token_prob = torch.zeros((B, s.n_nodes), device=dev)
        self.every = torch.arange(B, device=dev)
        self.limits = (torch.full((B,), int(top_k), dtype=torch.int32, device=dev) if top_k > 0 else None,
                       torch.full((B,), float(top_p), device=dev) if top_p < 1 else None,
                       torch.full((B,), float(min_p), device=dev) if min_p > 0 else None)
        limited = any(x is not None for x in self.limits)
        self.cut_logits = torch.empty((B, s.n_nodes, s.vocab), device=dev) if limited else None
        if drafts:      # one row per node that has a child, the draft's own noise, what it drew
            self.draft_logits = normal(B, T, s.vocab)
            self.draft_noise = torch.empty((B, T, s.vocab), device=dev)
            self.draft_tokens = torch.zeros((B, T), dtype=torch.int32, device=dev)
            self.draft_probs = torch.empty((B, T, s.vocab), device=dev)
        else:
            self.draft_logits = self.draft_probs = None
        slopes = 2.0 ** (-8.0 * torch.arange(1, a.h_q + 1, device=dev) / a.h_q) if a.bias else None
        self.mods = G.make_attn_mods(a.softcap, a.window, slopes) if a.softcap or a.window or a.bias else None
        self.share = share
        self.status = torch.zeros((1,), dtype=torch.int32, device=dev)

        def workspace(n):
            return torch.zeros((n,), dtype=torch.uint8, device=dev)
        size = G.attn_shared_workspace_bytes if share else G.attn_ex_workspace_bytes if self.mods else G.attn_workspace_bytes
        self.attn_ws = workspace(size(self.dims, T))
        self.plan_ws = workspace(G.kv_prefix_plan_bytes(self.dims)) if share else None
        self.page_ws = workspace(G.kv_pages_workspace_bytes(self.dims))
        self.accept_ws = workspace(G.spec_accept_sample_workspace_bytes(B, s.n_nodes))
        self.draw()
        self.make_room()

    def draw(self):
        """New random numbers for the next acceptance."""
        self.uniforms.uniform_(generator=self.generator)
        self.uniforms[:, 1] = 0.0       # node 1 is a sample already
        self.noise.exponential_(generator=self.generator).clamp_(min=1e-10)
        if self.draft_logits is not None:
            self.draft_noise.exponential_(generator=self.generator).clamp_(min=1e-10)

    def draft(self, stream=None):
        """The span's tokens past node 1 (which is a sample already) from the draft's
        logits, and the distributions that they were drawn from. Row n of both is
        node n's: its child is node n + 1."""
        if self.draft_logits is None:
            return
        s = self.shape
        G.spec_sample(s.batch * s.n_tok, s.vocab, s.n_tok, self.draft_logits, self.temperature, *self.limits, self.draft_noise,
                      self.draft_tokens, None, self.draft_probs, None, self.status, stream)
        with on_stream(stream):
            self.gdn.tokens[:, 2:] = self.draft_tokens[:, 1:]

    def fork(self, src, dst, stream=None):
        """Requests dst become copies of src: cache pages shared (tails copied), GDN
        states, the span so far (its tree and tokens, node 1 with them, and the target's
        rows); room for their next spans. The caller's inputs and the requests' limits
        stay. The dst differ from each other and from every src."""
        src, dst = ([int(b) for b in x] for x in (src, dst))
        if len(src) != len(dst) or len(set(dst)) != len(dst) or set(src) & set(dst):
            raise ValueError("a fork needs a source for each of its destinations, which differ from each other and from every source")
        if not all(0 <= b < self.shape.batch for b in src + dst):
            raise ValueError("a fork's requests lie in [0, %d)" % self.shape.batch)
        g = self.gdn
        if g.tree:      # (the workload's own array stays)
            g.parent_host = g.parent_host.copy()
            g.parent_host[dst] = g.parent_host[src]
        with on_stream(stream):      # the request numbers are made where they are read
            of, to = (torch.as_tensor(x, dtype=torch.int32).to(self.every.device) for x in (src, dst))
            self.want.fill_(-1)
            self.want[to.long()] = 0
        G.kv_pages_resize(self.dims, self.want, self.table, self.page_ref, self.page_ws, self.page_ws.numel(), self.status, stream)
        G.kv_pages_fork(self.dims, len(dst), of, to, self.table, self.ctx, self.page_ref, self.k_pages, self.v_pages, self.page_ws,
                        self.page_ws.numel(), self.status, stream)
        with on_stream(stream):
            for x in (g.ssm_state, g.conv_state, g.tokens, g.logits) + ((g.parent,) if g.tree else ()):
                x[to.long()] = x[of.long()]
        self.make_room(stream)

    def plan(self, stream=None):
        """What the requests' tables share in front, for the attention of every layer."""
        if self.share:
            G.kv_prefix_plan(self.dims, self.table, self.ctx, self.plan_ws, self.plan_ws.numel(), self.status, stream)

    def make_room(self, stream=None):
        """Pages for the committed tokens and the next span."""
        with on_stream(stream):      # the lengths are summed where they are used
            torch.add(self.ctx, self.shape.n_tok, out=self.want)
        G.kv_pages_resize(self.dims, self.want, self.table, self.page_ref, self.page_ws, self.page_ws.numel(), self.status, stream)

    def attend(self, y: int, stream=None):
        """Attention layer y over the span: norm and rotary, then attention."""
        a, g, T = self.attn, self.gdn, self.shape.n_tok
        k, v = self.k_pages[y], self.v_pages[y]
        G.attn_qk_norm_rope(self.dims, T, self.qkv[y], self.row, self.q_norm[y], self.k_norm[y], 1e-6, 1.0, self.rope, a.rot_dim,
                            a.max_tokens, g.parent, self.ctx, self.table, self.q, k, v, self.status, stream)
        scale, out = a.d_head ** -0.5, self.attn_out[y]
        where = (self.q, k, v, self.table, self.ctx)
        rest = (out, self.attn_ws, self.attn_ws.numel(), self.status, stream)
        if self.share:
            where += (self.plan_ws, self.plan_ws.numel(), scale, self.mods)
            tree, span = G.attn_tree_verify_shared, G.attn_verify_span_shared
        elif self.mods:
            where += (scale, self.mods)
            tree, span = G.attn_tree_verify_ex, G.attn_verify_span_ex
        else:
            where += (scale,)
            tree, span = G.attn_tree_verify, G.attn_verify_span
        if g.tree:
            tree(self.dims, T + 1, g.parent_host, g.parent, *where, *rest)
        else:
            span(self.dims, T, *where, *rest)

    def accept(self, stream=None):
        s, g = self.shape, self.gdn
        logits = g.logits
        if self.cut_logits is not None:
            logits = self.cut_logits
            G.spec_sample(s.batch * s.n_nodes, s.vocab, s.n_nodes, g.logits, self.temperature, *self.limits, None, None, None, None,
                          logits, self.status, stream)
        G.spec_accept_sample(s.batch, s.n_nodes, s.vocab, logits, self.draft_probs, g.tokens, g.parent, self.temperature, self.uniforms,
                             self.noise, self.accept_len, self.accept_node, self.next_token, self.token_prob, self.accept_ws,
                             self.accept_ws.numel(), self.status, stream)

    def commit(self, stream=None):
        """The GDN states and the cache rows of the accepted node's path."""
        g, s = self.gdn, self.shape
        G.gdn_rollback_restore(g.dims, g.n_tok, self.accept_node, g.ssm_ckpt, g.conv_ckpt, g.ssm_state, g.conv_state, self.status,
                               stream)
        G.kv_commit_path(self.dims, s.n_nodes, g.parent, self.accept_node, self.ctx, self.table, self.k_pages, self.v_pages,
                         self.ctx_next, self.status, stream)

    def carry(self, stream=None):
        """The next span's node 1, the next token, and its row 0, the accepted
        node's. The other nodes' tokens and rows are the caller's to make."""
        with on_stream(stream):
            self.gdn.tokens[:, 1] = self.next_token
            self.gdn.logits[:, 0] = self.gdn.logits[self.every, self.accept_node.long()]

    def step(self):
        """One step on the current stream; afterwards ctx holds the new lengths
        and the next span begins with the sampled next token."""
        self.draft()
        self.plan()
        self.gdn.verify()
        for y in range(self.attn.layers):
            self.attend(y)
        self.accept()
        self.commit()
        self.carry()
        self.ctx.copy_(self.ctx_next)
        self.make_room()


def main(argv=None):
    from . import workloads as W
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--gdn-layers", type=int, default=48)
    ap.add_argument("--attn-layers", type=int, default=16)
    ap.add_argument("--ctx", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--samples", action="store_true", help="the requests are samples of one prompt, whose pages they share")
    ap.add_argument("--drafts", action="store_true", help="the span's tokens drawn from a draft's logits")
    ap.add_argument("--top-k", type=int, default=0)
    ap.add_argument("--top-p", type=float, default=1.0)
    ap.add_argument("--min-p", type=float, default=0.0)
    ap.add_argument("--softcap", type=float, default=0.0)
    ap.add_argument("--window", type=int, default=0)
    a = ap.parse_args(argv)
    wl = W.make_workload(4, seed=0, batch=a.batch, layers=a.gdn_layers)
    h = HybridStep(wl, AttnShape(layers=a.attn_layers, softcap=a.softcap, window=a.window), [a.ctx] * a.batch, temperature=0.3,
                   top_k=a.top_k, top_p=a.top_p, min_p=a.min_p, drafts=a.drafts, share=a.samples)
    if a.samples and a.batch > 1:
        h.fork([0] * (a.batch - 1), range(1, a.batch))
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    h.step()
    for i in range(a.steps):
        h.draw()
        start.record()
        h.step()
        stop.record()
        torch.cuda.synchronize()
        print("step %d: %.2f ms, accepted %s, next %s, lengths %s, flags %d" % (
            i, start.elapsed_time(stop), h.accept_len.tolist(), h.next_token.tolist(), h.ctx.tolist(), int(h.status.item())))


if __name__ == "__main__":
    main()
