/*
 * gdnspec — target-side verify and rollback of a speculative span over the
 * Gated DeltaNet (GDN) linear-attention layers of a hybrid model, on one
 * GB300 (sm_103a).
 *
 * A step of DFlash / DDTree speculative decoding on a Qwen3.5/3.6 hybrid
 * target feeds the drafted tokens through the target, keeps an F32 SSM and
 * conv checkpoint after every drafted token, accepts the longest prefix (or
 * root path) whose tokens equal the target's greedy argmax, and restores the
 * recurrent state at the accepted token on the device, with no replay:
 *   - lucebox PR #506 "perf(dflash): split-chain fast rollback with F32 SSM
 *     checkpoints", Summary and Memory trade-off (per-token F32 checkpoints,
 *     fast rollback);
 *   - lucebox PR #533 "feat: DFlash support for tensor-parallel Qwen3.6
 *     targets", Changes (restore SSM and convolution state on-device; DDTree);
 *   - openinfer PR #626 "feat(qwen35): add opt-in DFlash speculative
 *     decoding", Summary and What Changed (greedy verify; recurrent state,
 *     conv state).
 *
 * Per GDN layer the pages name the recurrent (SSM) state and the conv state
 * but do not print the equations; this library computes, per request, layer
 * and processed node t (in node-index order):
 *   conv:  y[c] = SiLU( sum_{j<K} w[c][j] * win_t[c][j] ),  win_t[c][K-1] = x_t[c]
 *          and win_t[c][0..K-2] the K-1 previous inputs on the node's root
 *          path (the initial conv state above the root), oldest first;
 *   split: y = [ q (H_k*d_k) | k (H_k*d_k) | v (H_v*d_v) ];
 *          q, k L2-normalised per key head: u / sqrt(sum u^2 + 1e-6); q *= q_scale;
 *   rule:  value head h uses key head g = floor(h * H_k / H_v) and
 *          S_t = a_t S_p (I - b_t k_t k_t^T) + b_t v_t k_t^T,   o_t = S_t q_t
 *          with S_p the state after the parent node (the initial state for
 *          children of the root); S is [d_v][d_k] (row = value index).
 *
 * Conventions for every call:
 *   - Node 0 is the committed root. Its effect is already in the initial
 *     state; a span processes nodes 1..N-1 (n_tok = N-1 tokens). Row t-1 of
 *     every per-token array belongs to node t.
 *   - All arrays are row-major, contiguous, in the layouts given below, and
 *     owned by the caller. Device arrays live on the current CUDA device.
 *     The library allocates nothing.
 *   - Every call validates its arguments on the host first and returns a
 *     non-zero status with NOTHING queued when a check fails (fail-closed).
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL is the legacy
 *     default stream); the library never synchronises the host with the
 *     device. Launch failures return GDN_ERR_CUDA.
 *   - Problems that only the device can see (a draft token outside the
 *     vocabulary, an accepted node out of range, a NaN logit) never trap:
 *     they are OR-ed into *dev_status (nullable) as GDN_DEV_* bits.
 *   - Calls are stateless; concurrent calls on distinct buffers are safe.
 */
#ifndef GDNSPEC_H
#define GDNSPEC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t, passed as an opaque pointer (NULL = legacy default stream). */
typedef void *gdn_stream_t;

/* Element type of the inputs x, a, b and conv_w. States, checkpoints, outputs
 * and logits are always float32. */
#define GDN_F32 0
#define GDN_BF16 1

/* Status codes returned by every call. */
#define GDN_OK 0
#define GDN_ERR_NULL 1            /* a required pointer is NULL */
#define GDN_ERR_DIMS 2            /* a size is out of the supported range, see gdn_dims, attn_dims */
#define GDN_ERR_ALIGN 3           /* a float state/checkpoint/output pointer is not 16-byte aligned */
#define GDN_ERR_DTYPE 4           /* in_dtype is neither GDN_F32 nor GDN_BF16 */
#define GDN_ERR_TREE_ROOT 5       /* parent[0] != -1 (malformed root) */
#define GDN_ERR_TREE_PARENT 6     /* parent[i] outside [0, i) for i >= 1: forward, cyclic,
                                     self, out-of-range or second-root parent */
#define GDN_ERR_TREE_DEPTH 7      /* a node deeper than the allowed maximum */
#define GDN_ERR_TREE_TRUNCATED 8  /* fewer than 2 nodes: nothing to verify */
#define GDN_ERR_TREE_NOT_CHAIN 9  /* a sibling / skipped parent where a pure chain is required */
#define GDN_ERR_WORKSPACE 10      /* workspace NULL, misaligned or smaller than required */
#define GDN_ERR_CUDA 11           /* a CUDA launch or query failed */
#define GDN_ERR_FLAGS 12          /* a flags argument has a bit this library does not define */
#define GDN_ERR_OVERLAP 13        /* an output overlaps an input that it must not */

/* Device-side status bits, OR-ed into *dev_status (int32, device memory). */
#define GDN_DEV_TOKEN_RANGE 0x1   /* a draft token id outside [0, vocab): counted as a mismatch */
#define GDN_DEV_NAN_LOGIT 0x2     /* a NaN logit was seen: it ranks above every number */
#define GDN_DEV_NODE_RANGE 0x4    /* accepted node outside [0, n_tok]: nothing restored for it */
#define GDN_DEV_TREE 0x8          /* a device parent array broke parent[i] in [0, i): the kernel
                                     used parent i-1 for that node (verify) or left it unmatched
                                     (acceptance) instead of reading out of bounds */
#define GDN_DEV_SCHED 0x10        /* verify, attention: a CTA gave up waiting for an asynchronous
                                     hardware operation (the answer to a work-stealing request,
                                     a copy, a tensor-core product, or (the _pipelined calls) an
                                     input flag); its outputs are incomplete */
#define GDN_DEV_BOUNDS 0x20       /* debug builds of the library only (GDN_DEBUG_BOUNDS): a kernel
                                     skipped a global access that fell outside its buffer */
#define GDN_DEV_LENGTH 0x40       /* a context length, or a count of tokens asked for, that its row of
                                     the page table (or the rotary table) cannot hold: the request
                                     is left out */
#define GDN_DEV_PAGE 0x80         /* a page id outside [0, n_pages) where a page is needed: read as
                                     zeros, never written */
#define GDN_DEV_POOL 0x100        /* no free page was left: what needed one is left out */

/* Limits of this library. */
#define GDN_MAX_TOKENS 64         /* n_tok (= N - 1) per span */
#define GDN_MAX_CONV_K 8
#define GDN_MAX_TOPK 32           /* k of spec_topk */
#define GDN_MAX_SAMPLE_VOCAB 368640 /* vocab of spec_sample: a row lies in a cluster's shared memory */
#define GDN_WY_MAX_TOKENS 16      /* n_tok of the chunked-form calls */
#define GDN_MAX_PREFIX_BATCH 4096 /* requests of kv_prefix_plan and attn_*_shared */

/*
 * Model and batch dimensions shared by the verify and restore calls.
 *   batch    B  >= 1 requests
 *   layers   Y  >= 1 GDN layers (B * Y <= 65535)
 *   h_k, h_v    key and value heads, h_v % h_k == 0
 *   d_k         key head size: 64 or 128
 *   d_v         value head size: a multiple of 16, 16..1024
 *   conv_ch  C  = 2 * h_k * d_k + h_v * d_v (channels of the [q | k | v] conv)
 *   conv_k   K  conv kernel width, 1..GDN_MAX_CONV_K (4 for Qwen3.5/3.6)
 *   in_dtype    GDN_F32 or GDN_BF16 for x, a, b, conv_w
 *   q_scale     multiplies the normalised q (1.0 keeps o_t = S_t q_t as written)
 */
typedef struct gdn_dims {
    int32_t batch, layers, h_k, h_v, d_k, d_v, conv_ch, conv_k;
    int32_t in_dtype;
    float q_scale;
} gdn_dims;

/*
 * gdn_verify_span — verify a drafted CHAIN of n_tok tokens over every layer
 * and request, writing an F32 checkpoint after every token.
 * (lucebox PR #506, Summary: F32 SSM checkpoint capture; pure-chain path.)
 *
 * Inputs (device):
 *   x        [B][Y][n_tok][C]        pre-conv channels [q | k | v], in_dtype
 *   a, b     [B][Y][n_tok][h_v]      decay a_t and write strength b_t, in_dtype
 *   conv_w   [Y][C][K]               conv taps; tap K-1 multiplies the current token, in_dtype
 *   ssm_in   [B][Y][h_v][d_v][d_k]   f32 state before the span (read only)
 *   conv_in  [B][Y][C][K-1]          f32 last K-1 conv inputs before the span, oldest first
 *                                    (may be NULL only when K == 1)
 * Outputs (device, fully overwritten):
 *   ssm_ckpt  [B][Y][n_tok][h_v][d_v][d_k]  f32 state after each token
 *   conv_ckpt [B][Y][n_tok][C][K-1]         f32 conv window after each token
 *                                           (may be NULL only when K == 1)
 *   out       [B][Y][n_tok][h_v][d_v]       f32 o_t
 * The live state (ssm_in, conv_in) is never written: rejecting every token
 * needs no work. Outputs must not overlap inputs.
 *   dev_status  nullable, device int32 for device-side findings, as in
 *               gdn_tree_verify (a chain defines none today; it is accepted so
 *               both verify calls take the same arguments).
 * Returns GDN_OK or GDN_ERR_{NULL,DIMS,ALIGN,DTYPE,CUDA}.
 */
int gdn_verify_span(const gdn_dims *dims, int32_t n_tok,
                    const void *x, const void *a, const void *b, const void *conv_w,
                    const float *ssm_in, const float *conv_in,
                    float *ssm_ckpt, float *conv_ckpt, float *out,
                    int32_t *dev_status, gdn_stream_t stream);

/*
 * Flags of gdn_verify_span_ex and gdn_tree_verify_ex.
 *
 * GDN_VERIFY_STATE_READY — the caller promises that ssm_in, conv_in, conv_w
 * and (trees) parent_dev are not written by any work on `stream` that may
 * still be running when this call's kernel starts: with programmatic
 * dependent launch that is the kernel queued just before the call, whose
 * tail the verify overlaps (earlier work has completed). The verify then
 * loads those inputs, and builds its tree tables, before it waits for that
 * kernel, and only x, a and b (which the previous kernel may produce) after
 * it. Typical use: the verify of layer y + 1 queued right after the verify
 * of layer y, as a model whose layers run in sequence calls it; the
 * previous call writes only layer y's checkpoints and outputs. Not for the
 * first verify after a restore or commit, which writes the live state. The
 * results are the same with or without the flag; if the promise is broken,
 * the verify may read stale state.
 */
#define GDN_VERIFY_STATE_READY 0x1u

/*
 * gdn_verify_span_ex — gdn_verify_span with a flags word (GDN_VERIFY_*;
 * 0 = gdn_verify_span). Returns, in addition, GDN_ERR_FLAGS for an unknown
 * bit.
 */
int gdn_verify_span_ex(const gdn_dims *dims, int32_t n_tok,
                       const void *x, const void *a, const void *b, const void *conv_w,
                       const float *ssm_in, const float *conv_in,
                       float *ssm_ckpt, float *conv_ckpt, float *out,
                       int32_t *dev_status, uint32_t flags, gdn_stream_t stream);

/*
 * gdn_tree_verify — verify a DDTree of n_nodes nodes (node 0 = committed
 * root, T = n_nodes - 1 processed nodes) per request. Node i starts from the
 * state of parent(i) and its conv window follows its root path.
 * (lucebox PR #533, Changes and Verification: DDTree verify; lucebox PR #506,
 * Safety boundary: malformed geometry is rejected before execution.)
 *
 *   parent_host [B][n_nodes] int32, host memory: validated before anything is
 *               queued (GDN_ERR_TREE_* as for gdn_tree_check, depth <= T).
 *   parent_dev  [B][n_nodes] int32, device memory, the same contents; read by
 *               the kernel, which re-checks parent[i] in [0, i) and flags
 *               GDN_DEV_TREE in *dev_status (nullable) instead of reading out
 *               of bounds if the two copies differ.
 * Other arguments and layouts are those of gdn_verify_span with n_tok = T.
 */
int gdn_tree_verify(const gdn_dims *dims, int32_t n_nodes,
                    const int32_t *parent_host, const int32_t *parent_dev,
                    const void *x, const void *a, const void *b, const void *conv_w,
                    const float *ssm_in, const float *conv_in,
                    float *ssm_ckpt, float *conv_ckpt, float *out,
                    int32_t *dev_status, gdn_stream_t stream);

/* gdn_tree_verify_ex — gdn_tree_verify with a flags word, as gdn_verify_span_ex. */
int gdn_tree_verify_ex(const gdn_dims *dims, int32_t n_nodes,
                       const int32_t *parent_host, const int32_t *parent_dev,
                       const void *x, const void *a, const void *b, const void *conv_w,
                       const float *ssm_in, const float *conv_in,
                       float *ssm_ckpt, float *conv_ckpt, float *out,
                       int32_t *dev_status, uint32_t flags, gdn_stream_t stream);

/*
 * gdn_verify_span_pipelined / gdn_tree_verify_pipelined — the _ex calls (the
 * same operation, the same bytes) for inputs that are still landing when the
 * kernel starts: a step whose x, a and b arrive over the host link while
 * the verify already runs the layers that are there. This is an interface
 * of this library, not of the pages.
 *
 *   x_ready [B][layers] int32, device memory, nullable (null: the _ex call).
 *           The kernel reads the x, a and b rows of (request b, layer y) only
 *           after x_ready[b * layers + y] != 0. It waits for that (bounded,
 *           about a quarter second; a wait that gives up sets GDN_DEV_SCHED in
 *           *dev_status and the item reads whatever is there). Everything
 *           else (ssm_in, conv_in, conv_w, parent_dev) must be in place when
 *           the call's kernel starts, as for the _ex calls.
 *           The caller sets a flag only after that (request, layer)'s rows
 *           have landed, with a copy-engine write queued behind them (a
 *           host-to-device cudaMemcpyAsync on the stream that copied the
 *           rows), never from a kernel: a kernel could be waiting for an SM
 *           that this launch holds. The kernel reads the flags and never
 *           clears them: the caller zeroes them before the next call's
 *           copies set them again.
 * Returns as the _ex calls, and GDN_ERR_ALIGN for an x_ready not 4-byte
 * aligned.
 */
int gdn_verify_span_pipelined(const gdn_dims *dims, int32_t n_tok,
                              const void *x, const void *a, const void *b, const void *conv_w,
                              const float *ssm_in, const float *conv_in,
                              float *ssm_ckpt, float *conv_ckpt, float *out,
                              int32_t *dev_status, uint32_t flags, const int32_t *x_ready,
                              gdn_stream_t stream);
int gdn_tree_verify_pipelined(const gdn_dims *dims, int32_t n_nodes,
                              const int32_t *parent_host, const int32_t *parent_dev,
                              const void *x, const void *a, const void *b, const void *conv_w,
                              const float *ssm_in, const float *conv_in,
                              float *ssm_ckpt, float *conv_ckpt, float *out,
                              int32_t *dev_status, uint32_t flags, const int32_t *x_ready,
                              gdn_stream_t stream);

/*
 * spec_accept_greedy — greedy acceptance for a batch of requests.
 * (openinfer PR #626, Summary: single greedy request whose speculative output
 * matches plain greedy decoding; lucebox PR #533, Changes: top-K / argmax on
 * the GPU's logits.)
 *
 *   logits     [B][N][V] f32 (device): row n is the target's prediction after node n
 *   tokens     [B][N] int32 (device): tokens[b][n] = drafted token of node n (n >= 1;
 *              entry 0 is ignored)
 *   parent_dev [B][N] int32 (device) for trees, NULL for chains (parent[i] = i-1)
 * Outputs (device):
 *   argmax_out [B][N] int32: argmax of each row, lowest index on ties, the first
 *              NaN ranking above every number (flagged GDN_DEV_NAN_LOGIT)
 *   accept_len [B] int32: depth of the accepted node (chain: k in [0, N-1])
 *   accept_node[B] int32: the accepted node = the deepest node whose root path
 *              matches (tokens[i] == argmax[parent(i)] all along); among equally
 *              deep ones the lower node index at the first divergence wins.
 *              The bonus token is argmax_out[b][accept_node[b]].
 *   workspace  device scratch of at least spec_accept_workspace_bytes(B, N)
 *              bytes, 256-byte aligned, ZERO-FILLED before its first use; every
 *              call leaves every byte it used zero again, so one workspace serves
 *              calls of any shape. Calls that overlap in time must not share it.
 *   dev_status nullable, device int32: GDN_DEV_TOKEN_RANGE / NAN_LOGIT / TREE bits.
 * Limits: 1 <= N <= GDN_MAX_TOKENS + 1, 1 <= V < 2^31, B * N <= 2^20.
 * Returns GDN_OK or GDN_ERR_{NULL,DIMS,WORKSPACE,CUDA}.
 */
int spec_accept_greedy(int32_t batch, int32_t n_nodes, int32_t vocab,
                       const float *logits, const int32_t *tokens,
                       const int32_t *parent_dev,
                       int32_t *argmax_out, int32_t *accept_len, int32_t *accept_node,
                       void *workspace, size_t workspace_bytes,
                       int32_t *dev_status, gdn_stream_t stream);

/* Bytes of workspace spec_accept_greedy needs for (batch, n_nodes); 0 if the
 * sizes are out of range. */
size_t spec_accept_workspace_bytes(int32_t batch, int32_t n_nodes);

/* Size of the fixed device scratch behind spec_accept_greedy_static (1 MiB). */
#define GDN_STATIC_SCRATCH_BYTES (1 << 20)

/*
 * spec_accept_greedy_static — spec_accept_greedy without a caller-supplied
 * workspace, for callers that cannot allocate device memory: code that runs
 * where cudaMalloc is unavailable or forbidden (for example inside an
 * allocator-less runtime, a plugin host that owns all device memory, or a
 * hot loop that must never reach the allocator). The pages have no
 * counterpart of this call; it is a convenience of this library.
 *
 * Arguments, outputs and results are those of spec_accept_greedy, minus the
 * workspace. The scratch is a fixed GDN_STATIC_SCRATCH_BYTES array in the
 * library's device memory, present on every GPU that loads the library until
 * the process exits. The first call on a device (with that device current)
 * looks up the array's device address; make that first call before any
 * stream capture. If the lookup fails, that call returns GDN_ERR_CUDA and
 * the next call looks again; once found, the address is kept for the life
 * of the process, so cudaDeviceReset is not supported with this call. Every
 * call zeroes the part of the array that must start at zero (a small
 * cudaMemsetAsync on `stream`) and allocates nothing.
 * All calls share the one array: calls that may overlap on the GPU (other
 * streams, other host threads) race and must be serialised by the caller.
 * Returns GDN_ERR_WORKSPACE when spec_accept_workspace_bytes(batch, n_nodes)
 * exceeds GDN_STATIC_SCRATCH_BYTES (8 bytes per logit row plus 4 per
 * request: about 130,000 rows, e.g. batch 2,000 with n_nodes 65 fits), and
 * the other codes of spec_accept_greedy.
 */
int spec_accept_greedy_static(int32_t batch, int32_t n_nodes, int32_t vocab,
                              const float *logits, const int32_t *tokens,
                              const int32_t *parent_dev,
                              int32_t *argmax_out, int32_t *accept_len, int32_t *accept_node,
                              int32_t *dev_status, gdn_stream_t stream);

/*
 * gdn_rollback_restore — restore, on the device, the live SSM and conv state
 * of every request and layer to the checkpoint of its accepted node.
 * (lucebox PR #533, Changes: restore split SSM and convolution state
 * on-device; lucebox PR #506, Summary: fast rollback from F32 checkpoints.)
 *
 *   accept_node_dev [B] int32 (device), e.g. spec_accept_greedy's accept_node:
 *       node 0 leaves the state untouched; node in [1, n_tok] copies slot
 *       node-1; anything else copies nothing and sets GDN_DEV_NODE_RANGE.
 *   ssm_ckpt, conv_ckpt  as written by gdn_verify_span / gdn_tree_verify
 *   ssm_state [B][Y][h_v][d_v][d_k], conv_state [B][Y][C][K-1]: the live state
 *       (normally the verify call's ssm_in / conv_in buffers), overwritten
 *       bit-exactly with the chosen slot.
 * Returns GDN_OK or GDN_ERR_{NULL,DIMS,ALIGN,CUDA}.
 */
int gdn_rollback_restore(const gdn_dims *dims, int32_t n_tok,
                         const int32_t *accept_node_dev,
                         const float *ssm_ckpt, const float *conv_ckpt,
                         float *ssm_state, float *conv_state,
                         int32_t *dev_status, gdn_stream_t stream);

/*
 * Replay commit (the conservative alternative to checkpoints): verify without
 * writing any checkpoint, then, once the accepted length is known, re-run
 * only the accepted tokens from the live state and update it in place.
 * (openinfer PR #626, What Changed: commit restores the canonical state and
 * replays the accepted target span; Future Work: a lower-overhead commit.)
 * Restoring checkpoint k and replaying the first k tokens give the same
 * bytes. Chains only: a tree's branches need the per-node states.
 *
 * gdn_verify_span_nockpt — gdn_verify_span writing only `out` (no ssm or
 * conv checkpoints); the live state is read, never written.
 */
int gdn_verify_span_nockpt(const gdn_dims *dims, int32_t n_tok,
                           const void *x, const void *a, const void *b, const void *conv_w,
                           const float *ssm_in, const float *conv_in, float *out,
                           int32_t *dev_status, gdn_stream_t stream);

/*
 * gdn_commit_replay — for every request b with k = accept_len_dev[b] in
 * [1, n_tok], re-run conv + recurrence over tokens 0..k-1 of the span (the
 * same x, a, b, conv_w as the verify call, layouts of gdn_verify_span) from
 * ssm_state / conv_state and overwrite both with the state after token k-1.
 * k = 0 leaves the request untouched; k outside [0, n_tok] changes nothing
 * and sets GDN_DEV_NODE_RANGE in *dev_status (nullable). Two kernels on
 * `stream` (the state replay, then the conv-state update).
 * Returns GDN_OK or GDN_ERR_{NULL,DIMS,ALIGN,DTYPE,CUDA}.
 */
int gdn_commit_replay(const gdn_dims *dims, int32_t n_tok, const int32_t *accept_len_dev,
                      const void *x, const void *a, const void *b, const void *conv_w,
                      float *ssm_state, float *conv_state, int32_t *dev_status,
                      gdn_stream_t stream);

/*
 * gdn_verify_span_wy — gdn_verify_span_nockpt computed in chunked (WY) form:
 * per (request, layer, value head) the span's tokens are solved together
 * (one S_0 [K | Q] product, a shared T x T unit lower triangular forward
 * substitution) instead of one rank-1 update per token. Same arguments,
 * layouts and results (up to rounding order) as gdn_verify_span_nockpt.
 * (lucebox PR #506, Summary: the span's gated delta rule; openinfer PR #626,
 * Summary: the conservative commit this verify pairs with.)
 * Limits: n_tok <= GDN_WY_MAX_TOKENS; x and conv_w 16-byte aligned.
 * Returns GDN_OK or GDN_ERR_{NULL,DIMS,ALIGN,DTYPE,CUDA}.
 */
int gdn_verify_span_wy(const gdn_dims *dims, int32_t n_tok,
                       const void *x, const void *a, const void *b, const void *conv_w,
                       const float *ssm_in, const float *conv_in, float *out,
                       int32_t *dev_status, gdn_stream_t stream);

/*
 * gdn_commit_wy — gdn_commit_replay in chunked form: for every request b with
 * k = accept_len_dev[b] in [1, n_tok], the live state becomes
 * A_{k-1} S + sum_{j<k} D[k-1][j] b_j u_j k_j^T (the state after token k-1,
 * u from the same forward substitution as gdn_verify_span_wy) and the live
 * conv state the last K-1 inputs; k = 0 leaves the request untouched; k
 * outside [0, n_tok] changes nothing and sets GDN_DEV_NODE_RANGE. Same
 * arguments and layouts as gdn_commit_replay; two kernels on `stream`.
 * Limits: n_tok <= GDN_WY_MAX_TOKENS; x and conv_w 16-byte aligned.
 * Returns GDN_OK or GDN_ERR_{NULL,DIMS,ALIGN,DTYPE,CUDA}.
 */
int gdn_commit_wy(const gdn_dims *dims, int32_t n_tok, const int32_t *accept_len_dev,
                  const void *x, const void *a, const void *b, const void *conv_w,
                  float *ssm_state, float *conv_state, int32_t *dev_status,
                  gdn_stream_t stream);

/*
 * spec_topk — the k best logits of each row in the greedy order: larger value
 * first, lower index among equal values, every NaN above every number (the
 * first NaN first; flagged GDN_DEV_NAN_LOGIT), -0.0 equal to +0.0. For
 * draft-side tree construction (lucebox PR #533, Changes: draft top-K on the
 * GPU's logits).
 *   logits  [rows][V] f32 (device, 16-byte aligned)
 *   idx_out [rows][k] int32, val_out [rows][k] f32 (device): the k indices and
 *           their logits, best first
 *   workspace: at least spec_topk_workspace_bytes(rows, k) bytes of device
 *           memory, 256-byte aligned, zero-filled before first use; every call
 *           leaves it zero-filled. Overlapping calls must not share it.
 * Limits: 1 <= k <= GDN_MAX_TOPK, k <= V, 1 <= rows <= 65535.
 * Returns GDN_OK or GDN_ERR_{NULL,DIMS,ALIGN,WORKSPACE,CUDA}.
 */
int spec_topk(int32_t rows, int32_t vocab, int32_t k, const float *logits,
              int32_t *idx_out, float *val_out, void *workspace, size_t workspace_bytes,
              int32_t *dev_status, gdn_stream_t stream);

/* Bytes of workspace spec_topk needs; 0 if the sizes are out of range. */
size_t spec_topk_workspace_bytes(int32_t rows, int32_t k);

/*
 * The full-attention layers of a hybrid target: their drafted span, their
 * paged key/value cache, and the sampled form of the acceptance. These calls
 * stand beside the GDN calls above in the same step (verify, accept, restore):
 * attn_qk_norm_rope and attn_verify_span / attn_tree_verify per attention
 * layer, spec_accept_sample in the place of spec_accept_greedy, kv_commit_path
 * beside gdn_rollback_restore, and kv_pages_resize / kv_pages_fork between
 * steps. The pages name the hybrid's attention layers and their KV cache
 * (lucebox PR #506, Summary; openinfer PR #626, What Changed: committed KV)
 * without printing equations; each call states its own.
 *
 * Cache of one layer: k_pages, v_pages [n_pages][h_kv][page_tokens][d_head],
 * in_dtype. Token slot s of request b lies in page page_table[b][s /
 * page_tokens] at row s % page_tokens. ctx_len[b] committed tokens lie in
 * slots 0..ctx_len-1; the span's node t (t >= 1) has slot ctx_len + t - 1.
 * Entries of page_table that no slot in use needs are not read. A request
 * with ctx_len < 0 or ctx_len + n_tok > table_width * page_tokens is left
 * out (GDN_DEV_LENGTH), a needed page id outside [0, n_pages) reads as zeros
 * and is never written (GDN_DEV_PAGE).
 *
 *   batch        B >= 1 requests, B <= 65535
 *   layers       Y >= 1 layers of the kv_* calls' caches [Y][n_pages]...
 *                (Y * h_kv * h_kv < 2^31 there, Y <= 65535); the attn_* calls
 *                work on one layer and ignore it
 *   h_q, h_kv    query and key/value heads, h_q % h_kv == 0, query head h
 *                reads key/value head floor(h * h_kv / h_q); at most 1024
 *   d_head       64, 128 or 256
 *   page_tokens  16, 32, 64, 128 or 256
 *   n_pages      pages of one layer's pool; n_pages * h_kv < 2^31
 *   table_width  entries of a request's page table row;
 *                table_width * page_tokens < 2^30, batch * table_width < 2^31
 *   in_dtype     GDN_F32 or GDN_BF16: q, k, v, norm weights and out
 */
typedef struct attn_dims {
    int32_t batch, layers, h_q, h_kv, d_head, page_tokens, n_pages, table_width;
    int32_t in_dtype;
} attn_dims;

/*
 * attn_qk_norm_rope — RMS norm of every query and key head, rotary embedding,
 * and the span's keys and values into the cache, in one pass.
 *
 * For each new token t = 1..n_tok of each request, with x one head's d_head
 * values of q or k and w that kind's norm weights,
 *   y_i = x_i / sqrt(mean(x^2) + eps) * (w_i + norm_offset)
 * then, on the first rot_dim values, with the position p = ctx_len +
 * depth(t) - 1 and (c, s) = (cos, sin) of its row of the rotary table,
 *   (y_i, y_j) <- (y_i c_m - y_j s_m,  y_j c_m + y_i s_m),   m < rot_dim / 2,
 * for the pairs (i, j) = (m, m + rot_dim / 2), or (2m, 2m + 1) with
 * GDN_ROPE_PAIRS. v is copied. Arithmetic in f32, rounded once at the store.
 *
 *   qkv         [B][n_tok] rows of qkv_stride elements (a multiple of 16 bytes),
 *               each starting with q (h_q * d_head) | k (h_kv * d_head) | v (h_kv * d_head)
 *   q_norm, k_norm [d_head] in_dtype; norm_offset 0, or 1 for weights stored
 *               around zero; eps > 0
 *   rope        [max_pos][rot_dim] f32: rot_dim / 2 cosines, then the sines.
 *               May be NULL when rot_dim == 0 (no rotation)
 *   rot_dim     0 or a multiple of 16, at most d_head
 *   parent_dev  [B][n_tok + 1] for trees (n_tok <= GDN_MAX_TOKENS), NULL for
 *               chains of any length (depth(t) = t). A parent outside [0, i)
 *               is flagged GDN_DEV_TREE and taken as i - 1
 *   q_out       [B][n_tok][h_q][d_head]
 *   k_pages, v_pages  one layer's cache; slots ctx_len..ctx_len+n_tok-1 written
 * A request with ctx_len + n_tok > max_pos is left out too (GDN_DEV_LENGTH;
 * rot_dim 0: no such limit). Limits: n_tok >= 1, B * n_tok < 2^31. All
 * pointers but the integer ones 16-byte aligned.
 * Returns GDN_OK or GDN_ERR_{NULL,DIMS,ALIGN,DTYPE,FLAGS,CUDA}.
 */
#define GDN_ROPE_PAIRS 0x1u
int attn_qk_norm_rope(const attn_dims *dims, int32_t n_tok, const void *qkv, int64_t qkv_stride,
                      const void *q_norm, const void *k_norm, float eps, float norm_offset,
                      const float *rope, int32_t rot_dim, int32_t max_pos,
                      const int32_t *parent_dev, const int32_t *ctx_len, const int32_t *page_table,
                      void *q_out, void *k_pages, void *v_pages, int32_t *dev_status,
                      uint32_t flags, gdn_stream_t stream);

/*
 * attn_verify_span / attn_tree_verify — attention of a drafted chain or tree
 * over the paged cache: for node t of 1..n_tok and each query head
 *   o_t = sum_s softmax_s(scale q_t . k_s) v_s
 * over the committed slots and the slots of the node's root path (chain: the
 * nodes 1..t). One token (n_tok = 1) is plain decoding. Slots outside that set
 * do not touch the result, whatever they hold; rows of a page past the last
 * slot are not read as numbers.
 *
 *   q          [B][n_tok][h_q][d_head]
 *   out        [B][n_tok][h_q][d_head], in_dtype; zeros for a request left out
 *   workspace  at least attn_workspace_bytes(dims, n_tok) bytes, 256-byte
 *              aligned, any contents; overlapping calls must not share it
 *   parent_host, parent_dev as for gdn_tree_verify ([B][n_nodes], n_tok =
 *              n_nodes - 1); a device parent outside [0, i) is flagged
 *              GDN_DEV_TREE and taken as i - 1
 * bf16: products on the tensor cores with f32 accumulation, softmax in f32, its
 * weights rounded to bf16 for the second product; f32: all in f32.
 * Limits: 1 <= n_tok <= GDN_MAX_TOKENS, batch * h_kv <= 65535,
 * scale finite and above 0; bf16: ceil(table_width * page_tokens / 64) * h_kv *
 * ceil(n_tok * (h_q / h_kv) / 128), a request's most tiles of 64 slots and 128
 * rows, below 2^31, and times batch below 2^34.
 * Returns GDN_OK or GDN_ERR_{NULL,DIMS,ALIGN,DTYPE,TREE_*,WORKSPACE,CUDA}.
 */
int attn_verify_span(const attn_dims *dims, int32_t n_tok, const void *q, const void *k_pages,
                     const void *v_pages, const int32_t *page_table, const int32_t *ctx_len,
                     float scale, void *out, void *workspace, size_t workspace_bytes,
                     int32_t *dev_status, gdn_stream_t stream);
int attn_tree_verify(const attn_dims *dims, int32_t n_nodes, const int32_t *parent_host,
                     const int32_t *parent_dev, const void *q, const void *k_pages,
                     const void *v_pages, const int32_t *page_table, const int32_t *ctx_len,
                     float scale, void *out, void *workspace, size_t workspace_bytes,
                     int32_t *dev_status, gdn_stream_t stream);

/* Bytes of workspace attn_verify_span (n_tok) or attn_tree_verify (n_tok =
 * n_nodes - 1) needs; 0 if the sizes are out of range. */
size_t attn_workspace_bytes(const attn_dims *dims, int32_t n_tok);

/*
 * attn_verify_span_ex / attn_tree_verify_ex — attn_verify_span and
 * attn_tree_verify for layers that change their scores or see less than the
 * whole context. With p the positions (a committed slot's is its number, node
 * t's ctx_len + depth(t) - 1), query head h's score of slot s for node t is
 *   z = scale q_t . k_s
 *   z <- softcap tanh(z / softcap)           softcap > 0
 *   z <- z - slopes[h] (p_t - p_s)           slopes given
 * and of the slots that attn_verify_span sees, node t sees those with
 *   p_t - p_s < window                       window > 0 (its own slot is always seen)
 *   s >= first[b]                            first given: the request's document
 *                                            begins at slot first[b] of its row
 * Slots that no node sees are not read, nor are their pages' table entries: a
 * caller that keeps its own tables may have given those pages away (kv_pages_resize
 * does not do it: it takes back the end of a row, and takes a new page for an entry
 * that is missing in front). first[b] outside [0, ctx_len[b]] leaves the request out
 * (GDN_DEV_LENGTH). Where an NaN or infinity lies in a slot that a node does not
 * see, the node's result does not change.
 *
 *   mods       host memory, read before the call returns; NULL: nothing changed.
 *              slopes [h_q] f32 and first [B] int32 are device memory, nullable
 *   workspace  at least attn_ex_workspace_bytes(dims, n_tok)
 * All else as attn_verify_span / attn_tree_verify. softcap 0, or 1e-30 to 1e30
 * (a cap that overflows scale / softcap is refused); window >= 0.
 * Returns as they do.
 */
typedef struct attn_mods {
    float softcap;         /* 0: none */
    int32_t window;        /* 0: none */
    const float *slopes;   /* NULL: none */
    const int32_t *first;  /* NULL: none */
} attn_mods;

int attn_verify_span_ex(const attn_dims *dims, int32_t n_tok, const void *q, const void *k_pages,
                        const void *v_pages, const int32_t *page_table, const int32_t *ctx_len,
                        float scale, const attn_mods *mods, void *out, void *workspace,
                        size_t workspace_bytes, int32_t *dev_status, gdn_stream_t stream);
int attn_tree_verify_ex(const attn_dims *dims, int32_t n_nodes, const int32_t *parent_host,
                        const int32_t *parent_dev, const void *q, const void *k_pages,
                        const void *v_pages, const int32_t *page_table, const int32_t *ctx_len,
                        float scale, const attn_mods *mods, void *out, void *workspace,
                        size_t workspace_bytes, int32_t *dev_status, gdn_stream_t stream);
size_t attn_ex_workspace_bytes(const attn_dims *dims, int32_t n_tok);

/*
 * Shared prefixes: requests whose tables name the same pages in front
 * (kv_pages_fork's) read those pages once for all.
 *
 * kv_prefix_plan — finds the sharing from the tables: requests with the same
 * first page are compared with the first of them; of the lengths that they have in
 * common with it (full pages of committed tokens, whole multiples of 128 slots)
 * the one that saves the most reading makes a group of those that have it. The
 * others, and requests with an invalid length, stand alone.
 *   plan       at least kv_prefix_plan_bytes(dims) bytes of device memory,
 *              256-byte aligned, any contents before; batch at most
 *              GDN_MAX_PREFIX_BATCH. Calls that overlap in time may read one plan
 *              together, but not write it
 * A plan serves every layer's attention, until page_table or ctx_len change (a
 * ctx_len that only grows, and table rows that only get more entries, keep it
 * good). With any other table or length the attention's results are undefined, but
 * it stays within its buffers.
 *
 * attn_verify_span_shared / attn_tree_verify_shared — attn_verify_span_ex and
 * attn_tree_verify_ex with such a plan, of the same dims, table and lengths. The
 * results are theirs up to the order of sums. mods may change scores (softcap,
 * slopes); window and first must be none (GDN_ERR_DIMS).
 * They read less and launch more, and what they save is read from L2 while it
 * fits there. Plan included, against attn_verify_span_ex, in us: bf16, 8 single
 * tokens, 16 heads on 2, 128 wide: 21 and 16 over 2,000 shared slots, 25 and 24 over
 * 10,000, 27 and 32 over 20,000; 256 wide over 32,000, a layer of four 35 and 66; 2 x
 * 8 trees of 22 over 16,000, a layer of two 120 and 134 (attn_tree_verify 115). f32: no
 * gain below some 50,000 slots, and its time grows with the square of the batch (512
 * tokens of 256 prompts over 2,000 slots 1,693 and 330).
 *   workspace  at least attn_shared_workspace_bytes(dims, n_tok)
 * Limits: theirs, batch at most GDN_MAX_PREFIX_BATCH, and for bf16 their tile
 * limit with batch * n_tok in the place of n_tok. Returns as they do
 * (GDN_ERR_WORKSPACE for a plan that is NULL, misaligned or too small, too).
 */
int kv_prefix_plan(const attn_dims *dims, const int32_t *page_table, const int32_t *ctx_len,
                   void *plan, size_t plan_bytes, int32_t *dev_status, gdn_stream_t stream);
size_t kv_prefix_plan_bytes(const attn_dims *dims);
int attn_verify_span_shared(const attn_dims *dims, int32_t n_tok, const void *q, const void *k_pages,
                            const void *v_pages, const int32_t *page_table, const int32_t *ctx_len,
                            const void *plan, size_t plan_bytes, float scale, const attn_mods *mods,
                            void *out, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                            gdn_stream_t stream);
int attn_tree_verify_shared(const attn_dims *dims, int32_t n_nodes, const int32_t *parent_host,
                            const int32_t *parent_dev, const void *q, const void *k_pages,
                            const void *v_pages, const int32_t *page_table, const int32_t *ctx_len,
                            const void *plan, size_t plan_bytes, float scale, const attn_mods *mods,
                            void *out, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                            gdn_stream_t stream);
size_t attn_shared_workspace_bytes(const attn_dims *dims, int32_t n_tok);

/*
 * spec_accept_sample — acceptance of drafted tokens by sampling, so that what
 * is committed is distributed as the target's own samples. Random numbers are
 * inputs. With p_n = softmax(logits row n / temperature) and the children of a
 * node tried in index order, starting at the root:
 *   draft_probs given (row n: the distribution q the children of n were drawn
 *     from, independently): r = p_n; child i with token x is accepted if
 *     uniforms[i] * q(x) < r(x), else r <- max(r - q, 0) normalised;
 *   draft_probs NULL (fixed candidates): child i is accepted if uniforms[i] <
 *     r(x), else r <- r without x, normalised;
 *   accepted: continue at that child. No child left: the next token is the
 *     largest r(v) / noise[v] (lowest index on ties), a sample of r when the
 *     noise is exponential with mean 1. If r is zero everywhere, p_n is taken.
 * Temperature 0 is the limit: p uniform over the largest logits. A NaN or +inf
 * among a row's logits, or a row with none above -inf, makes its p NaN: its
 * children are rejected, the next token after it is 0, and GDN_DEV_NAN_LOGIT
 * is set. A token outside [0, vocab) is rejected (GDN_DEV_TOKEN_RANGE), a
 * parent outside [0, i) leaves its node out (GDN_DEV_TREE).
 *
 *   logits      [B][N][V] f32, 4-byte aligned
 *   draft_probs [B][N-1][V] f32 or NULL, 4-byte aligned
 *   tokens      [B][N] int32, entry 0 ignored
 *   parent_dev  [B][N] int32 for trees, NULL for chains
 *   temperature [B] f32 (>= 0) or NULL (all 1)
 *   uniforms    [B][N] f32 in [0, 1), entry 0 ignored
 *   noise       [B][V] f32 > 0
 * The next token in the next step: it is a sample already and must not be tested
 * again (a refusal would undo it, and what is committed would no longer be
 * distributed as the target's samples). It has neither a recurrent state nor a
 * cache row yet, so it is node 1 of the next span, whose row 0 is the accepted
 * node's; the caller gives that node uniforms[b][1] = 0. With it node 1, the
 * root's first child, is accepted at once (0 < p), the root's other children are
 * not tried, and the drafts proper are the nodes below node 1. The same goes for
 * the token that was sampled from a prompt's last row.
 * Outputs: accept_len [B], accept_node [B] as spec_accept_greedy;
 *   next_token [B] int32; token_prob [B][N] f32 (nullable): entry n >= 1 the
 *   target's p(tokens[n]) after its parent, entry 0 p(next_token) after the
 *   accepted node.
 *   workspace  at least spec_accept_sample_workspace_bytes(B, N) bytes,
 *              256-byte aligned, any contents; overlapping calls must not share it
 * Limits: 1 <= N <= GDN_MAX_TOKENS + 1, 1 <= V <= 2^30, B <= 65535.
 * Returns GDN_OK or GDN_ERR_{NULL,DIMS,ALIGN,WORKSPACE,CUDA}.
 */
int spec_accept_sample(int32_t batch, int32_t n_nodes, int32_t vocab, const float *logits,
                       const float *draft_probs, const int32_t *tokens, const int32_t *parent_dev,
                       const float *temperature, const float *uniforms, const float *noise,
                       int32_t *accept_len, int32_t *accept_node, int32_t *next_token,
                       float *token_prob, void *workspace, size_t workspace_bytes,
                       int32_t *dev_status, gdn_stream_t stream);
size_t spec_accept_sample_workspace_bytes(int32_t batch, int32_t n_nodes);

/*
 * spec_sample — tokens sampled from rows of logits with temperature, top-k,
 * top-p and min-p. Random numbers are inputs. It draws a draft's tokens and
 * gives their distribution (the draft_probs of spec_accept_sample), draws the
 * token after a prompt, and cuts the target's rows for an acceptance under the
 * same limits. With w_v = exp((x_v - max) / T) and a row's tokens in the greedy
 * order (larger logit first, lower index among equals, -0.0 equal to +0.0),
 * token j of that order is kept if
 *   j < top_k,   w_j >= min_p,   and  sum_{i<j} w_i < top_p * (the sum of the first top_k w);
 * the first one always. p = w / (sum of the kept w), 0 for the others; the token
 * is the largest p(v) / noise[v] (lowest index on ties), a sample of p when the
 * noise is exponential with mean 1. The sums that place a border, and weights next
 * to min_p, are integers in units of 2^-44, so that a border is off by at most
 * 2^-28 + V 2^-42 of the first top_k's sum (or 2^-44 in a weight); the sum that p is divided by is f32, its
 * terms added in a fixed order (off by less than 5e-6 at V = 151,936). Results are
 * the same from call to call.
 * Temperature 0 (or below, or NaN) is the limit: w = 1 for the largest logits, 0
 * for the others (logits less than 5e-37 below the largest count as it). A NaN or
 * +inf among a row's logits, or a row with none above -inf: token 0, its probability
 * and its row of probs NaN, its logits kept as they are, GDN_DEV_NAN_LOGIT.
 *
 *   logits      [rows][V] f32
 *   temperature, top_p, min_p [ceil(rows / rows_per_request)] f32, top_k the
 *               same, int32: row i uses entry i / rows_per_request. Each NULL
 *               for no limit (temperature: 1), as are top_k <= 0 or >= V, top_p
 *               >= 1 and min_p <= 0 (NaN too)
 *   noise       [rows][V] f32 > 0; may be NULL when token is
 * Outputs, each nullable, one of token, probs and kept_logits at least:
 *   token       [rows] int32;  token_prob [rows] f32: p(token) (with token only)
 *   probs       [rows][V] f32: p
 *   kept_logits [rows][V] f32: the logits, -inf where not kept; softmax(kept_logits
 *               / T) = p. May be `logits` itself. No other output may overlap an
 *               input or another output (checked for the [rows][V] arrays).
 * Limits: 1 <= rows <= 2^20, 1 <= V <= GDN_MAX_SAMPLE_VOCAB, rows_per_request >= 1.
 * All arrays 4-byte aligned. No workspace.
 * Returns GDN_OK or GDN_ERR_{NULL,DIMS,ALIGN,OVERLAP,CUDA}.
 */
int spec_sample(int32_t rows, int32_t vocab, int32_t rows_per_request, const float *logits,
                const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                const float *noise, int32_t *token, float *token_prob, float *probs, float *kept_logits,
                int32_t *dev_status, gdn_stream_t stream);

/*
 * kv_commit_path — after the acceptance, the accepted root path's keys and
 * values moved together in every layer: the path's j-th node (j = 1..k, k =
 * depth of accept_node) goes from slot ctx_len + node - 1 to ctx_len + j - 1,
 * and ctx_out[b] = ctx_len[b] + k. What lies past the new length is left over.
 *   parent_dev   [B][n_nodes] for trees; NULL for chains, whose path is in
 *                place already (only ctx_out is written; the pools may be NULL)
 *   accept_node  [B]; outside [0, n_nodes): the request keeps its length
 *                (GDN_DEV_NODE_RANGE). A parent outside [0, i) is flagged
 *                GDN_DEV_TREE and taken as i - 1
 *   k_pages, v_pages [Y][n_pages][h_kv][page_tokens][d_head]
 *   ctx_out      [B]; must not overlap ctx_len
 * Limits: 2 <= n_nodes <= GDN_MAX_TOKENS + 1.
 * Returns GDN_OK or GDN_ERR_{NULL,DIMS,ALIGN,DTYPE,OVERLAP,CUDA}.
 */
int kv_commit_path(const attn_dims *dims, int32_t n_nodes, const int32_t *parent_dev,
                   const int32_t *accept_node, const int32_t *ctx_len, const int32_t *page_table,
                   void *k_pages, void *v_pages, int32_t *ctx_out, int32_t *dev_status,
                   gdn_stream_t stream);

/*
 * Pages of the cache. page_ref[n_pages] int32 counts the table entries that
 * name a page; a page is free while its count is 0, and the free page with the
 * lowest id is taken first, so results do not depend on timing. A request's
 * valid entries (>= 0) stand at the start of its row; the others are -1.
 *
 * kv_pages_resize — for every request b with want[b] >= 0 the row is made
 * ceil(want[b] / page_tokens) entries long: first every request's entries
 * beyond that are given back (count - 1, entry -1), then missing ones are
 * taken, requests in order, each from its first missing entry on. want[b] < 0
 * leaves the row as it is. A want[b] beyond the table is left out
 * (GDN_DEV_LENGTH); an entry for which no page is free stays -1
 * (GDN_DEV_POOL). want 0 frees a request; ctx_len trims a rejected span;
 * ctx_len + n_tok makes room for the next.
 *
 * kv_pages_fork — request dst[i] becomes a copy of src[i], i = 0..n_fork-1 in
 * order: pages full up to ctx_len[src] are shared (count + 1), a tail page's
 * ctx_len % page_tokens live rows are copied in every layer into a page taken
 * for it, the other entries become -1, and ctx_len[dst] = ctx_len[src]. What
 * dst's row held before is overwritten, not given back: resize it to 0 first.
 * The dst must differ from each other and from every src. An index outside
 * [0, B), or a length that the table cannot hold, leaves out that fork
 * (GDN_DEV_NODE_RANGE, GDN_DEV_LENGTH); one whose tail finds no free page
 * makes dst empty: length 0, all entries -1 (GDN_DEV_POOL).
 *
 * workspace: at least kv_pages_workspace_bytes(dims) bytes, 256-byte aligned,
 * any contents; overlapping calls must not share it.
 * Return GDN_OK or GDN_ERR_{NULL,DIMS,ALIGN,DTYPE,WORKSPACE,CUDA}.
 */
int kv_pages_resize(const attn_dims *dims, const int32_t *want, int32_t *page_table,
                    int32_t *page_ref, void *workspace, size_t workspace_bytes,
                    int32_t *dev_status, gdn_stream_t stream);
int kv_pages_fork(const attn_dims *dims, int32_t n_fork, const int32_t *src, const int32_t *dst,
                  int32_t *page_table, int32_t *ctx_len, int32_t *page_ref,
                  void *k_pages, void *v_pages, void *workspace, size_t workspace_bytes,
                  int32_t *dev_status, gdn_stream_t stream);
size_t kv_pages_workspace_bytes(const attn_dims *dims);

/*
 * gdn_tree_check — host-only geometry check of B parent arrays of n_nodes
 * nodes each (the pure-chain guard of lucebox PR #506, Safety boundary).
 *   require_chain != 0: additionally require parent[i] == i-1 (no sibling or
 *   skipped parent). max_depth > 0 bounds every node's depth.
 * Returns GDN_OK, GDN_ERR_NULL, GDN_ERR_DIMS (batch < 1),
 * GDN_ERR_TREE_{TRUNCATED,ROOT,PARENT,DEPTH,NOT_CHAIN}. Touches no GPU.
 */
int gdn_tree_check(const int32_t *parent_host, int32_t batch, int32_t n_nodes,
                   int32_t require_chain, int32_t max_depth);

/* A static, human-readable name for a status code. */
const char *gdn_status_str(int status);

#ifdef __cplusplus
}
#endif

#endif /* GDNSPEC_H */
