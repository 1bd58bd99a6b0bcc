"""Python binding of libgdnspec (the C ABI declared in include/gdnspec.h).

Argument marshalling only: every step of the path runs in the library's
CUDA kernels. Device arrays are torch CUDA tensors (PyTorch provides the
memory and the stream); the functions keep the C names and raise GdnError on
a non-zero status. There is no CPU fallback: if the library is missing or
cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
# GDNSPEC_LIB selects another build of the library (e.g. the bounds-checking
# _lib/libgdnspec_debug.so) for the whole process.
LIB_PATH = os.environ.get("GDNSPEC_LIB") or os.path.join(_HERE, "_lib", "libgdnspec.so")

GDN_F32 = 0
GDN_BF16 = 1

GDN_OK = 0
GDN_ERR_NULL = 1
GDN_ERR_DIMS = 2
GDN_ERR_ALIGN = 3
GDN_ERR_DTYPE = 4
GDN_ERR_TREE_ROOT = 5
GDN_ERR_TREE_PARENT = 6
GDN_ERR_TREE_DEPTH = 7
GDN_ERR_TREE_TRUNCATED = 8
GDN_ERR_TREE_NOT_CHAIN = 9
GDN_ERR_WORKSPACE = 10
GDN_ERR_CUDA = 11
GDN_ERR_FLAGS = 12
GDN_ERR_OVERLAP = 13

GDN_VERIFY_STATE_READY = 0x1
GDN_ROPE_PAIRS = 0x1

GDN_DEV_TOKEN_RANGE = 0x1
GDN_DEV_NAN_LOGIT = 0x2
GDN_DEV_NODE_RANGE = 0x4
GDN_DEV_TREE = 0x8
GDN_DEV_SCHED = 0x10
GDN_DEV_BOUNDS = 0x20
GDN_DEV_LENGTH = 0x40
GDN_DEV_PAGE = 0x80
GDN_DEV_POOL = 0x100

GDN_MAX_TOKENS = 64
GDN_MAX_CONV_K = 8
GDN_MAX_TOPK = 32
GDN_WY_MAX_TOKENS = 16

EXPORTED = ("gdn_verify_span", "gdn_tree_verify", "spec_accept_greedy",
            "spec_accept_workspace_bytes", "gdn_rollback_restore", "gdn_tree_check",
            "gdn_status_str", "gdn_verify_span_nockpt", "gdn_commit_replay", "spec_topk",
            "spec_topk_workspace_bytes", "gdn_verify_span_wy", "gdn_commit_wy", "gdn_verify_span_ex",
            "gdn_tree_verify_ex", "gdn_verify_span_pipelined", "gdn_tree_verify_pipelined",
            "attn_qk_norm_rope", "attn_verify_span", "attn_tree_verify", "attn_workspace_bytes",
            "spec_accept_sample", "spec_accept_sample_workspace_bytes", "kv_commit_path",
            "kv_pages_resize", "kv_pages_fork", "kv_pages_workspace_bytes")


class GdnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: status {status} ({status_str(status)})")


class gdn_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("layers", ctypes.c_int32),
                ("h_k", ctypes.c_int32), ("h_v", ctypes.c_int32),
                ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("conv_ch", ctypes.c_int32), ("conv_k", ctypes.c_int32),
                ("in_dtype", ctypes.c_int32), ("q_scale", ctypes.c_float)]


def make_dims(batch, layers, h_k, h_v, d_k, d_v, conv_k, in_dtype, q_scale=1.0, conv_ch=None) -> gdn_dims:
    if conv_ch is None:
        conv_ch = 2 * h_k * d_k + h_v * d_v
    return gdn_dims(batch, layers, h_k, h_v, d_k, d_v, conv_ch, conv_k, in_dtype, float(q_scale))


class attn_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("layers", ctypes.c_int32),
                ("h_q", ctypes.c_int32), ("h_kv", ctypes.c_int32),
                ("d_head", ctypes.c_int32), ("page_tokens", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("table_width", ctypes.c_int32),
                ("in_dtype", ctypes.c_int32)]


def make_attn_dims(batch, layers, h_q, h_kv, d_head, page_tokens, n_pages, table_width, in_dtype) -> attn_dims:
    return attn_dims(batch, layers, h_q, h_kv, d_head, page_tokens, n_pages, table_width, in_dtype)


_lock = threading.Lock()
_lib = None


def load(path: Optional[str] = None):
    """Load libgdnspec.so (built by speculative_decode_hybrid_gb300.build)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                f"libgdnspec.so not found at {p}: build it first "
                "(python -m speculative_decode_hybrid_gb300.build); there is no fallback path")
        lib = ctypes.CDLL(p)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        dp = ctypes.POINTER(gdn_dims)
        lib.gdn_verify_span.argtypes = [dp, i32] + [vp] * 9 + [vp, vp]
        lib.gdn_tree_verify.argtypes = [dp, i32, vp, vp] + [vp] * 9 + [vp, vp]
        u32 = ctypes.c_uint32
        lib.gdn_verify_span_ex.argtypes = [dp, i32] + [vp] * 9 + [vp, u32, vp]
        lib.gdn_tree_verify_ex.argtypes = [dp, i32, vp, vp] + [vp] * 9 + [vp, u32, vp]
        lib.gdn_verify_span_pipelined.argtypes = [dp, i32] + [vp] * 9 + [vp, u32, vp, vp]
        lib.gdn_tree_verify_pipelined.argtypes = [dp, i32, vp, vp] + [vp] * 9 + [vp, u32, vp, vp]
        lib.spec_accept_greedy.argtypes = [i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
        lib.spec_accept_workspace_bytes.argtypes = [i32, i32]
        lib.spec_accept_workspace_bytes.restype = sz
        lib.gdn_rollback_restore.argtypes = [dp, i32, vp, vp, vp, vp, vp, vp, vp]
        lib.spec_topk.argtypes = [i32, i32, i32, vp, vp, vp, vp, sz, vp, vp]
        lib.spec_topk_workspace_bytes.argtypes = [i32, i32]
        lib.spec_topk_workspace_bytes.restype = sz
        lib.gdn_verify_span_nockpt.argtypes = [dp, i32] + [vp] * 7 + [vp, vp]
        lib.gdn_commit_replay.argtypes = [dp, i32] + [vp] * 9
        lib.gdn_verify_span_wy.argtypes = [dp, i32] + [vp] * 7 + [vp, vp]
        lib.gdn_commit_wy.argtypes = [dp, i32] + [vp] * 9
        ap, f32, i64 = ctypes.POINTER(attn_dims), ctypes.c_float, ctypes.c_int64
        lib.attn_qk_norm_rope.argtypes = [ap, i32, vp, i64, vp, vp, f32, f32, vp, i32, i32] + [vp] * 6 + [vp, u32, vp]
        lib.attn_verify_span.argtypes = [ap, i32] + [vp] * 5 + [f32, vp, vp, sz, vp, vp]
        lib.attn_tree_verify.argtypes = [ap, i32, vp, vp] + [vp] * 5 + [f32, vp, vp, sz, vp, vp]
        lib.attn_workspace_bytes.argtypes = [ap, i32]
        lib.spec_accept_sample.argtypes = [i32, i32, i32] + [vp] * 11 + [vp, sz, vp, vp]
        lib.spec_accept_sample_workspace_bytes.argtypes = [i32, i32]
        lib.kv_commit_path.argtypes = [ap, i32] + [vp] * 7 + [vp, vp]
        lib.kv_pages_resize.argtypes = [ap] + [vp] * 3 + [vp, sz, vp, vp]
        lib.kv_pages_fork.argtypes = [ap, i32] + [vp] * 7 + [vp, sz, vp, vp]
        lib.kv_pages_workspace_bytes.argtypes = [ap]
        for f in ("attn_workspace_bytes", "spec_accept_sample_workspace_bytes", "kv_pages_workspace_bytes"):
            getattr(lib, f).restype = sz
        lib.gdn_tree_check.argtypes = [vp, i32, i32, i32, i32]
        lib.gdn_status_str.argtypes = [ctypes.c_int]
        lib.gdn_status_str.restype = ctypes.c_char_p
        for f in ("gdn_verify_span", "gdn_tree_verify", "gdn_verify_span_ex", "gdn_tree_verify_ex",
                  "gdn_verify_span_pipelined", "gdn_tree_verify_pipelined", "spec_accept_greedy",
                  "gdn_rollback_restore", "gdn_tree_check", "gdn_verify_span_nockpt",
                  "gdn_commit_replay", "spec_topk", "gdn_verify_span_wy", "gdn_commit_wy",
                  "attn_qk_norm_rope", "attn_verify_span", "attn_tree_verify", "spec_accept_sample",
                  "kv_commit_path", "kv_pages_resize", "kv_pages_fork"):
            getattr(lib, f).restype = ctypes.c_int
        _lib = lib
        return lib


def status_str(status: int) -> str:
    try:
        return load().gdn_status_str(int(status)).decode()
    except Exception:  # library missing: still describe the code
        return "status %d" % status


def _ptr(t) -> Optional[int]:
    """Raw pointer of a tensor / numpy array / int / None."""
    if t is None:
        return None
    try:
        return t.data_ptr()
    except AttributeError:
        pass
    if isinstance(t, int):
        return t
    if hasattr(t, "ctypes"):
        return t.ctypes.data
    raise TypeError(f"cannot take a pointer of {type(t)}")


_raw_stream = None


def _current_stream() -> int:
    """Handle of the current stream, without the Stream object that
    torch.cuda.current_stream() builds (3 us, a third of a small call) where
    this PyTorch has the getter its own compiled code uses."""
    global _raw_stream
    import torch
    if _raw_stream is None:
        raw, dev = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
        torch.cuda.init()
        _raw_stream = (lambda: raw(dev())) if raw and dev else (lambda: torch.cuda.current_stream().cuda_stream)
    return _raw_stream()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ok(rc: int, what: str):
    if rc != GDN_OK:
        raise GdnError(rc, what)


def gdn_verify_span(dims: gdn_dims, n_tok: int, x, a, b, conv_w, ssm_in, conv_in,
                    ssm_ckpt, conv_ckpt, out, dev_status=None, stream=None, flags: int = 0,
                    x_ready=None) -> None:
    """gdn_verify_span; gdn_verify_span_ex when flags (GDN_VERIFY_*) are given;
    gdn_verify_span_pipelined when x_ready (device int32 [batch][layers]) is."""
    args = (ctypes.byref(dims), int(n_tok), _ptr(x), _ptr(a), _ptr(b), _ptr(conv_w), _ptr(ssm_in),
            _ptr(conv_in), _ptr(ssm_ckpt), _ptr(conv_ckpt), _ptr(out), _ptr(dev_status))
    if x_ready is not None:
        _ok(load().gdn_verify_span_pipelined(*args, int(flags), _ptr(x_ready), _stream(stream)),
            "gdn_verify_span_pipelined")
    elif flags:
        _ok(load().gdn_verify_span_ex(*args, int(flags), _stream(stream)), "gdn_verify_span_ex")
    else:
        _ok(load().gdn_verify_span(*args, _stream(stream)), "gdn_verify_span")


def gdn_tree_verify(dims: gdn_dims, n_nodes: int, parent_host, parent_dev, x, a, b, conv_w, ssm_in,
                    conv_in, ssm_ckpt, conv_ckpt, out, dev_status=None, stream=None, flags: int = 0,
                    x_ready=None) -> None:
    """gdn_tree_verify; gdn_tree_verify_ex when flags (GDN_VERIFY_*) are given;
    gdn_tree_verify_pipelined when x_ready (device int32 [batch][layers]) is."""
    import numpy as np
    ph = None
    if parent_host is not None:
        ph = np.ascontiguousarray(parent_host, dtype=np.int32)
    args = (ctypes.byref(dims), int(n_nodes), _ptr(ph), _ptr(parent_dev), _ptr(x), _ptr(a), _ptr(b),
            _ptr(conv_w), _ptr(ssm_in), _ptr(conv_in), _ptr(ssm_ckpt), _ptr(conv_ckpt), _ptr(out),
            _ptr(dev_status))
    if x_ready is not None:
        _ok(load().gdn_tree_verify_pipelined(*args, int(flags), _ptr(x_ready), _stream(stream)),
            "gdn_tree_verify_pipelined")
    elif flags:
        _ok(load().gdn_tree_verify_ex(*args, int(flags), _stream(stream)), "gdn_tree_verify_ex")
    else:
        _ok(load().gdn_tree_verify(*args, _stream(stream)), "gdn_tree_verify")


def spec_accept_workspace_bytes(batch: int, n_nodes: int) -> int:
    return int(load().spec_accept_workspace_bytes(int(batch), int(n_nodes)))


def spec_accept_greedy(batch: int, n_nodes: int, vocab: int, logits, tokens, parent_dev,
                       argmax_out, accept_len, accept_node, workspace, workspace_bytes: int,
                       dev_status=None, stream=None) -> None:
    rc = load().spec_accept_greedy(int(batch), int(n_nodes), int(vocab), _ptr(logits), _ptr(tokens),
                                   _ptr(parent_dev), _ptr(argmax_out), _ptr(accept_len),
                                   _ptr(accept_node), _ptr(workspace), int(workspace_bytes),
                                   _ptr(dev_status), _stream(stream))
    _ok(rc, "spec_accept_greedy")


def gdn_rollback_restore(dims: gdn_dims, n_tok: int, accept_node_dev, ssm_ckpt, conv_ckpt,
                         ssm_state, conv_state, dev_status=None, stream=None) -> None:
    rc = load().gdn_rollback_restore(ctypes.byref(dims), int(n_tok), _ptr(accept_node_dev),
                                     _ptr(ssm_ckpt), _ptr(conv_ckpt), _ptr(ssm_state),
                                     _ptr(conv_state), _ptr(dev_status), _stream(stream))
    _ok(rc, "gdn_rollback_restore")


def gdn_verify_span_nockpt(dims: gdn_dims, n_tok: int, x, a, b, conv_w, ssm_in, conv_in, out,
                           dev_status=None, stream=None) -> None:
    rc = load().gdn_verify_span_nockpt(ctypes.byref(dims), int(n_tok), _ptr(x), _ptr(a), _ptr(b),
                                       _ptr(conv_w), _ptr(ssm_in), _ptr(conv_in), _ptr(out),
                                       _ptr(dev_status), _stream(stream))
    _ok(rc, "gdn_verify_span_nockpt")


def gdn_commit_replay(dims: gdn_dims, n_tok: int, accept_len_dev, x, a, b, conv_w, ssm_state,
                      conv_state, dev_status=None, stream=None) -> None:
    rc = load().gdn_commit_replay(ctypes.byref(dims), int(n_tok), _ptr(accept_len_dev), _ptr(x), _ptr(a),
                                  _ptr(b), _ptr(conv_w), _ptr(ssm_state), _ptr(conv_state),
                                  _ptr(dev_status), _stream(stream))
    _ok(rc, "gdn_commit_replay")


def gdn_verify_span_wy(dims: gdn_dims, n_tok: int, x, a, b, conv_w, ssm_in, conv_in, out,
                       dev_status=None, stream=None) -> None:
    rc = load().gdn_verify_span_wy(ctypes.byref(dims), int(n_tok), _ptr(x), _ptr(a), _ptr(b),
                                   _ptr(conv_w), _ptr(ssm_in), _ptr(conv_in), _ptr(out),
                                   _ptr(dev_status), _stream(stream))
    _ok(rc, "gdn_verify_span_wy")


def gdn_commit_wy(dims: gdn_dims, n_tok: int, accept_len_dev, x, a, b, conv_w, ssm_state,
                  conv_state, dev_status=None, stream=None) -> None:
    rc = load().gdn_commit_wy(ctypes.byref(dims), int(n_tok), _ptr(accept_len_dev), _ptr(x), _ptr(a),
                              _ptr(b), _ptr(conv_w), _ptr(ssm_state), _ptr(conv_state),
                              _ptr(dev_status), _stream(stream))
    _ok(rc, "gdn_commit_wy")


def spec_topk_workspace_bytes(rows: int, k: int) -> int:
    return int(load().spec_topk_workspace_bytes(int(rows), int(k)))


def spec_topk(rows: int, vocab: int, k: int, logits, idx_out, val_out, workspace, workspace_bytes: int,
              dev_status=None, stream=None) -> None:
    rc = load().spec_topk(int(rows), int(vocab), int(k), _ptr(logits), _ptr(idx_out), _ptr(val_out),
                          _ptr(workspace), int(workspace_bytes), _ptr(dev_status), _stream(stream))
    _ok(rc, "spec_topk")


def gdn_tree_check(parent_host, batch: int, n_nodes: int, require_chain: bool = False,
                   max_depth: int = 0) -> int:
    """Host-only geometry check; returns the status code (does not raise)."""
    import numpy as np
    ph = None if parent_host is None else np.ascontiguousarray(parent_host, dtype=np.int32)
    return int(load().gdn_tree_check(_ptr(ph), int(batch), int(n_nodes), int(bool(require_chain)),
                                     int(max_depth)))


# -- the attention layers: norm + rotary, span attention, the paged cache ----

def attn_qk_norm_rope(dims: attn_dims, n_tok: int, qkv, qkv_stride: int, q_norm, k_norm, eps: float,
                      norm_offset: float, rope, rot_dim: int, max_pos: int, parent_dev, ctx_len, page_table,
                      q_out, k_pages, v_pages, dev_status=None, stream=None, flags: int = 0) -> None:
    """Per-head RMS norm and rotary embedding of q and k; k and v into the
    cache. parent_dev: None for chains; flags: GDN_ROPE_PAIRS."""
    rc = load().attn_qk_norm_rope(ctypes.byref(dims), int(n_tok), _ptr(qkv), int(qkv_stride), _ptr(q_norm),
                                  _ptr(k_norm), float(eps), float(norm_offset), _ptr(rope), int(rot_dim),
                                  int(max_pos), _ptr(parent_dev), _ptr(ctx_len), _ptr(page_table), _ptr(q_out),
                                  _ptr(k_pages), _ptr(v_pages), _ptr(dev_status), int(flags), _stream(stream))
    _ok(rc, "attn_qk_norm_rope")


def attn_workspace_bytes(dims: attn_dims, n_tok: int) -> int:
    return int(load().attn_workspace_bytes(ctypes.byref(dims), int(n_tok)))


def attn_verify_span(dims: attn_dims, n_tok: int, q, k_pages, v_pages, page_table, ctx_len, scale: float, out,
                     workspace, workspace_bytes: int, dev_status=None, stream=None) -> None:
    """Attention of a drafted chain over the paged cache (n_tok 1: decoding)."""
    rc = load().attn_verify_span(ctypes.byref(dims), int(n_tok), _ptr(q), _ptr(k_pages), _ptr(v_pages),
                                 _ptr(page_table), _ptr(ctx_len), float(scale), _ptr(out), _ptr(workspace),
                                 int(workspace_bytes), _ptr(dev_status), _stream(stream))
    _ok(rc, "attn_verify_span")


def attn_tree_verify(dims: attn_dims, n_nodes: int, parent_host, parent_dev, q, k_pages, v_pages, page_table,
                     ctx_len, scale: float, out, workspace, workspace_bytes: int, dev_status=None,
                     stream=None) -> None:
    """Attention of a drafted tree over the paged cache."""
    import numpy as np
    ph = None if parent_host is None else np.ascontiguousarray(parent_host, dtype=np.int32)
    rc = load().attn_tree_verify(ctypes.byref(dims), int(n_nodes), _ptr(ph), _ptr(parent_dev), _ptr(q),
                                 _ptr(k_pages), _ptr(v_pages), _ptr(page_table), _ptr(ctx_len), float(scale),
                                 _ptr(out), _ptr(workspace), int(workspace_bytes), _ptr(dev_status),
                                 _stream(stream))
    _ok(rc, "attn_tree_verify")


def spec_accept_sample_workspace_bytes(batch: int, n_nodes: int) -> int:
    return int(load().spec_accept_sample_workspace_bytes(int(batch), int(n_nodes)))


def spec_accept_sample(batch: int, n_nodes: int, vocab: int, logits, draft_probs, tokens, parent_dev,
                       temperature, uniforms, noise, accept_len, accept_node, next_token, token_prob,
                       workspace, workspace_bytes: int, dev_status=None, stream=None) -> None:
    """Acceptance by sampling from given random numbers. draft_probs: None for
    fixed candidates; parent_dev: None for chains; temperature: None for 1."""
    rc = load().spec_accept_sample(int(batch), int(n_nodes), int(vocab), _ptr(logits), _ptr(draft_probs),
                                   _ptr(tokens), _ptr(parent_dev), _ptr(temperature), _ptr(uniforms),
                                   _ptr(noise), _ptr(accept_len), _ptr(accept_node), _ptr(next_token),
                                   _ptr(token_prob), _ptr(workspace), int(workspace_bytes), _ptr(dev_status),
                                   _stream(stream))
    _ok(rc, "spec_accept_sample")


def kv_commit_path(dims: attn_dims, n_nodes: int, parent_dev, accept_node, ctx_len, page_table, k_pages,
                   v_pages, ctx_out, dev_status=None, stream=None) -> None:
    """The accepted path's cache rows moved together; ctx_out = ctx_len + its
    length. parent_dev: None for chains."""
    rc = load().kv_commit_path(ctypes.byref(dims), int(n_nodes), _ptr(parent_dev), _ptr(accept_node),
                               _ptr(ctx_len), _ptr(page_table), _ptr(k_pages), _ptr(v_pages), _ptr(ctx_out),
                               _ptr(dev_status), _stream(stream))
    _ok(rc, "kv_commit_path")


def kv_pages_workspace_bytes(dims: attn_dims) -> int:
    return int(load().kv_pages_workspace_bytes(ctypes.byref(dims)))


def kv_pages_resize(dims: attn_dims, want, page_table, page_ref, workspace, workspace_bytes: int,
                    dev_status=None, stream=None) -> None:
    """Every request's table row cut or grown to want[b] tokens (< 0: as it is)."""
    rc = load().kv_pages_resize(ctypes.byref(dims), _ptr(want), _ptr(page_table), _ptr(page_ref),
                                _ptr(workspace), int(workspace_bytes), _ptr(dev_status), _stream(stream))
    _ok(rc, "kv_pages_resize")


def kv_pages_fork(dims: attn_dims, n_fork: int, src, dst, page_table, ctx_len, page_ref, k_pages, v_pages,
                  workspace, workspace_bytes: int, dev_status=None, stream=None) -> None:
    """Requests dst become copies of src: full pages shared, tails copied."""
    rc = load().kv_pages_fork(ctypes.byref(dims), int(n_fork), _ptr(src), _ptr(dst), _ptr(page_table),
                              _ptr(ctx_len), _ptr(page_ref), _ptr(k_pages), _ptr(v_pages), _ptr(workspace),
                              int(workspace_bytes), _ptr(dev_status), _stream(stream))
    _ok(rc, "kv_pages_fork")


GDN_STATIC_SCRATCH_BYTES = 1 << 20


def spec_accept_greedy_static(batch: int, n_nodes: int, vocab: int, logits, tokens, parent_dev,
                              argmax_out, accept_len, accept_node, dev_status=None, stream=None) -> None:
    """spec_accept_greedy without a workspace argument, for callers that
    cannot allocate device memory: the library's fixed 1 MiB device scratch
    is used instead. All calls share that scratch, so calls that may overlap
    on the GPU must be serialised by the caller; make the first call on a
    device before any stream capture (it looks up the scratch's address)."""
    lib = load()
    f = lib.spec_accept_greedy_static
    if not getattr(f, "_gdn_typed", False):
        vp, i32 = ctypes.c_void_p, ctypes.c_int32
        f.argtypes = [i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp]
        f.restype = ctypes.c_int
        f._gdn_typed = True
    rc = f(int(batch), int(n_nodes), int(vocab), _ptr(logits), _ptr(tokens), _ptr(parent_dev),
           _ptr(argmax_out), _ptr(accept_len), _ptr(accept_node), _ptr(dev_status), _stream(stream))
    _ok(rc, "spec_accept_greedy_static")
