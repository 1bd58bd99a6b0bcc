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

Node 1 of every span is a token that has been sampled (by the step before, for
the first step by the prompt's last row) but not processed yet: it is accepted
without another test (uniform 0), and a step commits one token at least.

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


def on_stream(stream):
    """Context in which torch queues where the library's calls do: on the current
    stream (None), a torch stream, or the stream of a handle."""
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


class HybridStep:
    def __init__(self, wl: Workload, attn: AttnShape, ctx_len, temperature: float = 1.0, seed: int = 0, device="cuda"):
        """ctx_len: committed tokens of each request (their cache rows are
        filled with random keys and values)."""
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
        self.status = torch.zeros((1,), dtype=torch.int32, device=dev)

        def workspace(n):
            return torch.zeros((n,), dtype=torch.uint8, device=dev)
        self.attn_ws = workspace(G.attn_workspace_bytes(self.dims, T))
        self.page_ws = workspace(G.kv_pages_workspace_bytes(self.dims))
        self.accept_ws = workspace(G.spec_accept_sample_workspace_bytes(B, s.n_nodes))
        self.draw()
        self.make_room()

    def draw(self):
        """New random numbers for the next acceptance."""
        self.uniforms.uniform_(generator=self.generator)
        self.uniforms[:, 1] = 0.0       # node 1 is a sample already
        self.noise.exponential_(generator=self.generator).clamp_(min=1e-10)

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
        if g.tree:
            G.attn_tree_verify(self.dims, T + 1, g.parent_host, g.parent, self.q, k, v, self.table, self.ctx, scale, out,
                               self.attn_ws, self.attn_ws.numel(), self.status, stream)
        else:
            G.attn_verify_span(self.dims, T, self.q, k, v, self.table, self.ctx, scale, out, self.attn_ws, self.attn_ws.numel(),
                               self.status, stream)

    def accept(self, stream=None):
        s, g = self.shape, self.gdn
        G.spec_accept_sample(s.batch, s.n_nodes, s.vocab, g.logits, None, g.tokens, g.parent, self.temperature, self.uniforms,
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
    a = ap.parse_args(argv)
    wl = W.make_workload(4, seed=0, batch=a.batch, layers=a.gdn_layers)
    h = HybridStep(wl, AttnShape(layers=a.attn_layers), [a.ctx] * a.batch, temperature=0.3)
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
