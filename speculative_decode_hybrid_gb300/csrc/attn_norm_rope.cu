// attn_qk_norm_rope: RMS norm of every query and key head, rotary embedding,
// and the span's keys and values into the paged cache, in one pass over the
// projected rows (the hybrid's attention layers of lucebox PR #506, Summary;
// openinfer PR #626, What Changed).
//
// A head of D values is D / 8 lanes of two runs of four values: under the
// rotation the second run is the first's partner, rot_dim / 2 values on, so that
// a pair never leaves its lane (with GDN_ROPE_PAIRS the runs are neighbours and
// the pairs within them); the sum of squares is a butterfly over the head's
// lanes. A warp takes a token's heads in turn, 32 / (D / 8) at a time, the
// queries, the keys and the values each in a loop of its own, with the token's
// cosines and sines and the norm weights in registers: what is done per head is
// its loads, its arithmetic (two values an instruction) and its stores. A first
// form that chose between the three kinds head by head took 210 instructions a
// step and was bound by issuing them: 56 us for 8,002 tokens of 48 bf16 heads of
// 128 (201 MB). This one takes 146, and 42.5 us: 4.7 TB/s, 0.70 of the measured
// copy rate, bound by issue slots (59 % used) and the latency of a step's loads
// together. f32, with half the arithmetic per byte: 18.9 us for 4,000 tokens of
// 24 heads of 128, 0.77 of that rate.
#include <cuda_runtime.h>

#include <cmath>
#include <initializer_list>
#include <type_traits>

#include "attn_device.cuh"
#include "gdn_host.h"
#include "gdnspec.h"

namespace {

using gdndev::Buf;
using gdndev::fma2;
using gdndev::mul2;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// What the registers leave room for: with a fourth block the f32 form spills (31 us
// instead of 19 for 4,000 tokens of 24 heads of 128).
constexpr int blocks_per_sm(bool bf16) { return bf16 ? 4 : 3; }

struct RopeArgs {
    int n_tok, h_q, h_kv, page_shift, n_pages, width, rot, max_pos, warps_per_token;
    int64_t tokens, stride;
    const void *qkv, *q_norm, *k_norm;
    float eps, offset;
    const float *rope;
    const int32_t *parent, *ctx, *table;
    void *q_out, *k_pages, *v_pages;
    int32_t *status;
    int batch;
    bool pairs;
};

// Four values as they are stored.
template <bool BF16>
struct Run {
    unsigned u[BF16 ? 2 : 4];
};

template <bool BF16>
__device__ __forceinline__ Run<BF16> load_run(const char *p) {
    Run<BF16> r;
    if constexpr (BF16) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        r.u[0] = v.x, r.u[1] = v.y;
    } else {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        r.u[0] = v.x, r.u[1] = v.y, r.u[2] = v.z, r.u[3] = v.w;
    }
    return r;
}

template <bool BF16>
__device__ __forceinline__ void store_run(char *p, const Run<BF16> &r) {
    if constexpr (BF16)
        *reinterpret_cast<uint2 *>(p) = make_uint2(r.u[0], r.u[1]);
    else
        *reinterpret_cast<uint4 *>(p) = make_uint4(r.u[0], r.u[1], r.u[2], r.u[3]);
}

template <bool BF16>
__device__ __forceinline__ void widen(const Run<BF16> &r, float2 (&x)[2]) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
        x[j] = BF16 ? make_float2(__uint_as_float(r.u[j] << 16), __uint_as_float(r.u[j] & 0xffff0000u))
                    : make_float2(__uint_as_float(r.u[BF16 ? 0 : 2 * j]), __uint_as_float(r.u[BF16 ? 0 : 2 * j + 1]));
}

template <bool BF16>
__device__ __forceinline__ Run<BF16> narrow(const float2 (&x)[2]) {
    Run<BF16> r;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if constexpr (BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[j].x, x[j].y);
            r.u[j] = *reinterpret_cast<const unsigned *>(&h);
        } else {
            r.u[2 * j] = __float_as_uint(x[j].x), r.u[2 * j + 1] = __float_as_uint(x[j].y);
        }
    }
    return r;
}

// grid (token blocks, parts): a block's eight warps are 8 / warps_per_token
// tokens; with several parts a token's warps are spread over as many blocks.
template <bool BF16, int D, bool PAIRS>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(BF16)) qk_norm_rope(RopeArgs a) {
    constexpr int kLanes = D / 8, kGroups = 32 / kLanes, kElem = BF16 ? 2 : 4, kRun = 4 * kElem, kHead = D * kElem;
    constexpr int kAhead = BF16 ? 4 : 2;  // steps whose loads are in flight together
    const int lane = threadIdx.x % kLanes, group = threadIdx.x % 32 / kLanes, warp = threadIdx.x / 32;
    const int64_t token = (int64_t)blockIdx.x * (kWarps / a.warps_per_token) + warp / a.warps_per_token;
    const int warps = a.warps_per_token * gridDim.y, mine = warp % a.warps_per_token + a.warps_per_token * blockIdx.y;
    int32_t *st = a.status;
    const size_t B = a.batch, pool_bytes = ((size_t)a.n_pages * a.h_kv << a.page_shift) * kHead;
    const Buf bx{a.qkv, ((size_t)(a.tokens - 1) * a.stride + (size_t)(a.h_q + 2 * a.h_kv) * D) * kElem},
        bq{a.q_out, (size_t)a.tokens * a.h_q * kHead}, bk{a.k_pages, pool_bytes}, bv{a.v_pages, pool_bytes},
        bpar{a.parent, B * (a.n_tok + 1) * 4}, btab{a.table, B * (size_t)a.width * 4},
        brope{a.rope, (size_t)a.max_pos * a.rot * 4};
    // this lane's two runs of a head, in bytes, and whether they turn
    const int half = a.rot / 2;
    const bool turned = PAIRS ? lane * 8 < a.rot : lane * 4 < half;
    const int d0 = (turned && !PAIRS ? lane * 4 : lane * 8) * kElem, d1 = (turned && !PAIRS ? half + lane * 4 : lane * 8 + 4) * kElem;
    gdndev::pdl_wait();
    gdndev::pdl_launch_dependents();
    if (token >= a.tokens) return;
    const int b = (int)((unsigned)token / (unsigned)a.n_tok), t = (int)token - b * a.n_tok + 1;
    const int ctx = a.ctx[b];
    int depth = t;
    if (a.parent) {
        depth = 0;
        const int32_t *row = a.parent + (size_t)b * (a.n_tok + 1);
        for (int i = t; i > 0; ++depth) {
            int up = GDN_IN(row + i, 4, bpar, st) ? row[i] : i - 1;
            if (up < 0 || up >= i) {
                up = i - 1;
                if (threadIdx.x % 32 == 0 && st) atomicOr(st, GDN_DEV_TREE);
            }
            i = up;
        }
    }
    // a chain's last position bounds a tree's; a request is left out as a whole
    if (ctx < 0 || (int64_t)ctx + a.n_tok > (int64_t)a.width << a.page_shift ||
        (a.rot > 0 && (int64_t)ctx + a.n_tok > a.max_pos)) {
        if (threadIdx.x % 32 == 0 && st) atomicOr(st, GDN_DEV_LENGTH);
        return;
    }
    const int pos = ctx + depth - 1, slot = ctx + t - 1;
    const int32_t *entry = a.table + (size_t)b * a.width + (slot >> a.page_shift);
    const int page = GDN_IN(entry, 4, btab, st) ? *entry : -1;
    const bool page_ok = page >= 0 && page < a.n_pages;
    float2 cs[2] = {make_float2(1.f, 1.f), make_float2(1.f, 1.f)}, sn[2] = {};  // no turn: cosine 1, sine 0
    if (turned) {
        const float *row = a.rope + (size_t)pos * a.rot + lane * 4;
        if (GDN_IN(row, 16, brope, st) && GDN_IN(row + half, 16, brope, st)) {
            const float4 c = gdndev::ld4(row), s = gdndev::ld4(row + half);
            cs[0] = make_float2(c.x, c.y), cs[1] = make_float2(c.z, c.w);
            sn[0] = make_float2(s.x, s.y), sn[1] = make_float2(s.z, s.w);
        }
    }
    if (!page_ok && threadIdx.x % 32 == 0 && st) atomicOr(st, GDN_DEV_PAGE);
    const char *src = static_cast<const char *>(a.qkv) + token * a.stride * kElem;
    const size_t page_at = ((((size_t)(page_ok ? page : 0) * a.h_kv) << a.page_shift) + (slot & ((1 << a.page_shift) - 1))) * kHead;
    const int kv_step = kHead << a.page_shift;  // from a page's head to its next

    // heads `first`, first + warps * kGroups, ... of one kind; from: its first
    // head in the row; to, to_step: its first head's place and the way to the next
    auto kind = [&](auto norm, int first_step, int count, const char *from, char *to, int to_step, const void *weights, Buf bto) {
        float2 w[4];
        if constexpr (norm) {
            if (first_step * kGroups >= count) return;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float2 x[2];
                widen<BF16>(load_run<BF16>(static_cast<const char *>(weights) + (j ? d1 : d0)), x);
                w[2 * j] = make_float2(x[0].x + a.offset, x[0].y + a.offset);
                w[2 * j + 1] = make_float2(x[1].x + a.offset, x[1].y + a.offset);
            }
        }
        for (int h0 = first_step * kGroups + group; h0 - group < count; h0 += kAhead * warps * kGroups) {
            Run<BF16> raw[kAhead][2];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int h = h0 + k * warps * kGroups;
                const char *p = from + h * kHead;
                if (h < count && GDN_IN(p + d0, kRun, bx, st) && GDN_IN(p + d1, kRun, bx, st))
                    raw[k][0] = load_run<BF16>(p + d0), raw[k][1] = load_run<BF16>(p + d1);
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int h = h0 + k * warps * kGroups;
                if (h - group >= count) break;  // the whole warp; a group past the end goes along
                Run<BF16> out[2] = {raw[k][0], raw[k][1]};
                if constexpr (norm) {
                    float2 x[2], y[2];
                    widen<BF16>(raw[k][0], x);
                    widen<BF16>(raw[k][1], y);
                    float2 s2 = mul2(x[0], x[0]);
                    s2 = fma2(x[1], x[1], s2);
                    s2 = fma2(y[0], y[0], s2);
                    s2 = fma2(y[1], y[1], s2);
                    float s = s2.x + s2.y;
#pragma unroll
                    for (int o = kLanes / 2; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
                    const float r = rsqrtf(fmaf(s, 1.0f / D, a.eps));
                    const float2 rr = make_float2(r, r);
#pragma unroll
                    for (int j = 0; j < 2; ++j) x[j] = mul2(mul2(x[j], rr), w[j]), y[j] = mul2(mul2(y[j], rr), w[2 + j]);
                    if constexpr (PAIRS) {
                        const float c4[4] = {cs[0].x, cs[0].y, cs[1].x, cs[1].y}, s4[4] = {sn[0].x, sn[0].y, sn[1].x, sn[1].y};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float2 &z = j < 2 ? x[j] : y[j - 2];
                            z = make_float2(z.x * c4[j] - z.y * s4[j], z.y * c4[j] + z.x * s4[j]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float2 u = x[j], v = y[j], minus = make_float2(-sn[j].x, -sn[j].y);
                            x[j] = fma2(v, minus, mul2(u, cs[j]));
                            y[j] = fma2(u, sn[j], mul2(v, cs[j]));
                        }
                    }
                    out[0] = narrow<BF16>(x);
                    out[1] = narrow<BF16>(y);
                }
                char *p = to + h * to_step;
                if (h < count && GDN_IN(p + d0, kRun, bto, st) && GDN_IN(p + d1, kRun, bto, st))
                    store_run<BF16>(p + d0, out[0]), store_run<BF16>(p + d1, out[1]);
            }
        }
    };
    // the kinds' steps in one row, dealt out to the token's warps in turn
    const int q_steps = (a.h_q + kGroups - 1) / kGroups, kv_steps = (a.h_kv + kGroups - 1) / kGroups;
    auto start = [&](int steps_before) { return (mine + warps - steps_before % warps) % warps; };
    kind(std::true_type{}, mine, a.h_q, src, static_cast<char *>(a.q_out) + token * a.h_q * kHead, kHead, a.q_norm, bq);
    if (!page_ok) return;
    kind(std::true_type{}, start(q_steps), a.h_kv, src + a.h_q * kHead, static_cast<char *>(a.k_pages) + page_at, kv_step, a.k_norm, bk);
    kind(std::false_type{}, start(q_steps + kv_steps), a.h_kv, src + (a.h_q + a.h_kv) * kHead, static_cast<char *>(a.v_pages) + page_at,
         kv_step, nullptr, bv);
}

template <bool BF16, int D>
int launch(RopeArgs a, cudaStream_t st) {
    constexpr int kGroups = 32 / (D / 8);
    // many tokens: a warp each, as long as that fills the GPU; few: up to a warp
    // for every step
    const int sms = gdnhost::sm_count(), resident = blocks_per_sm(BF16) * kWarps * (sms > 0 ? sms : 152);
    const int steps = (a.h_q + kGroups - 1) / kGroups + 2 * ((a.h_kv + kGroups - 1) / kGroups);
    int64_t want = 8LL * resident / a.tokens;  // warps a token: eight rounds and more even out the last one
    if (want > steps) want = steps;
    a.warps_per_token = want >= 8 ? 8 : want >= 4 ? 4 : want >= 2 ? 2 : 1;
    const int parts = want > 8 ? (int)((want + 7) / 8) : 1;
    const int64_t per_block = kWarps / a.warps_per_token, blocks = (a.tokens + per_block - 1) / per_block;
    return gdndev::launch_pdl(a.pairs ? qk_norm_rope<BF16, D, true> : qk_norm_rope<BF16, D, false>, dim3((unsigned)blocks, parts),
                              dim3(kThreads), 0, st, a) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

extern "C" int attn_qk_norm_rope(const attn_dims *dims, int32_t n_tok, const void *qkv, int64_t qkv_stride,
                                 const void *q_norm, const void *k_norm, float eps, float norm_offset,
                                 const float *rope, int32_t rot_dim, int32_t max_pos, const int32_t *parent_dev,
                                 const int32_t *ctx_len, const int32_t *page_table, void *q_out, void *k_pages,
                                 void *v_pages, int32_t *dev_status, uint32_t flags, gdn_stream_t stream) {
    if (const int rc = gdnhost::check_attn(dims)) return rc;
    if (flags & ~GDN_ROPE_PAIRS) return GDN_ERR_FLAGS;
    const int d = dims->d_head;
    const int64_t row = (int64_t)(dims->h_q + 2 * dims->h_kv) * d, e = (int64_t)gdnhost::attn_elem_bytes(dims);
    if (n_tok < 1 || (parent_dev && n_tok > GDN_MAX_TOKENS) || (int64_t)dims->batch * n_tok > 0x7fffffffLL) return GDN_ERR_DIMS;
    if (qkv_stride < row || qkv_stride > (1LL << 40) || qkv_stride * e % 16 != 0) return GDN_ERR_DIMS;
    if (rot_dim < 0 || rot_dim > d || rot_dim % 16 != 0 || (rot_dim > 0 && max_pos < 1)) return GDN_ERR_DIMS;
    if (!std::isfinite(eps) || eps <= 0.f || !std::isfinite(norm_offset)) return GDN_ERR_DIMS;
    if (!qkv || !q_norm || !k_norm || (rot_dim > 0 && !rope) || !ctx_len || !page_table || !q_out || !k_pages || !v_pages)
        return GDN_ERR_NULL;
    using gdnhost::aligned_to;
    for (const void *p : {qkv, q_norm, k_norm, (const void *)rope, (const void *)q_out, (const void *)k_pages, (const void *)v_pages})
        if (!aligned_to(p, 16)) return GDN_ERR_ALIGN;
    for (const int32_t *p : {parent_dev, ctx_len, page_table, (const int32_t *)dev_status})
        if (!aligned_to(p, 4)) return GDN_ERR_ALIGN;
    int shift = 0;
    while ((1 << shift) < dims->page_tokens) ++shift;
    RopeArgs a{n_tok, dims->h_q, dims->h_kv, shift, dims->n_pages, dims->table_width, rot_dim, max_pos, 1,
               (int64_t)dims->batch * n_tok, qkv_stride, qkv, q_norm, k_norm, eps, norm_offset, rope, parent_dev, ctx_len,
               page_table, q_out, k_pages, v_pages, dev_status, dims->batch,
               rot_dim > 0 && (flags & GDN_ROPE_PAIRS) != 0};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dims->in_dtype == GDN_BF16)
        return d == 64 ? launch<true, 64>(a, st) : d == 128 ? launch<true, 128>(a, st) : launch<true, 256>(a, st);
    return d == 64 ? launch<false, 64>(a, st) : d == 128 ? launch<false, 128>(a, st) : launch<false, 256>(a, st);
}
