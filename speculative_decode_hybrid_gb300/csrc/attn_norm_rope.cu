// attn_qk_norm_rope: RMS norm of every query and key head, rotary embedding,
// and the span's keys and values into the paged cache, in one pass over the
// projected rows (the hybrid's attention layers of lucebox PR #506, Summary;
// openinfer PR #626, What Changed).
//
// A head of D values is D / 8 lanes with 8 consecutive values each (16 bytes
// of bf16, twice 16 of f32). The sum of squares is a butterfly over the head's
// lanes; the partner of a value under the rotation lies rot_dim / 2 values on,
// which is a fixed number of lanes (rot_dim is a multiple of 16), so the
// rotation is eight shuffles; with GDN_ROPE_PAIRS it is the neighbour in the
// same lane. Every input is read once, every output written once, and a
// token's cosines and sines are held in registers over its heads: the kernel is
// bound by the bytes of qkv, q and the cache rows.
#include <cuda_runtime.h>

#include <cmath>
#include <initializer_list>

#include "gdn_device.cuh"
#include "gdn_host.h"
#include "gdnspec.h"

namespace {

using gdndev::Buf;

constexpr int kThreads = 256;

struct RopeArgs {
    int n_tok, h_q, h_kv, page_shift, n_pages, width, rot, max_pos, tokens_per_block;
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

template <bool BF16>
__device__ __forceinline__ void load8(const void *p, size_t i, float (&x)[8]) {
    if constexpr (BF16) {
        const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + i);
        const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(w[j] << 16);
            x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    } else {
        const float4 *f = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        const float4 a = f[0], b = f[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
}

template <bool BF16>
__device__ __forceinline__ void store8(void *p, size_t i, const float (&x)[8]) {
    if constexpr (BF16) {
        unsigned w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
            w[j] = *reinterpret_cast<const unsigned *>(&h);
        }
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        float4 *f = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
        f[0] = make_float4(x[0], x[1], x[2], x[3]);
        f[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// grid (token blocks, head parts). A block's lane groups are dealt out to
// tokens_per_block tokens; a token's groups take its heads in turn.
template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads) qk_norm_rope(RopeArgs a) {
    constexpr int kLanes = D / 8, kGroups = kThreads / kLanes, kElem = BF16 ? 2 : 4;
    const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    const int per_token = kGroups / a.tokens_per_block;
    const int64_t token = (int64_t)blockIdx.x * a.tokens_per_block + group / per_token;
    const bool live_token = token < a.tokens;
    int32_t *st = a.status;
    const size_t B = a.batch, pool_bytes = ((size_t)a.n_pages * a.h_kv << a.page_shift) * D * kElem;
    const Buf bx{a.qkv, ((size_t)(a.tokens - 1) * a.stride + (size_t)(a.h_q + 2 * a.h_kv) * D) * kElem},
        bq{a.q_out, (size_t)a.tokens * a.h_q * D * kElem}, bk{a.k_pages, pool_bytes}, bv{a.v_pages, pool_bytes},
        bpar{a.parent, B * (a.n_tok + 1) * 4}, btab{a.table, B * (size_t)a.width * 4},
        brope{a.rope, (size_t)a.max_pos * a.rot * 4};
    gdndev::pdl_wait();
    if (!live_token) return;  // whole lane groups: no shuffle below crosses one
    const int b = (int)(token / a.n_tok), t = (int)(token % a.n_tok) + 1;
    const int ctx = a.ctx[b];
    int depth = t;
    if (a.parent) {
        depth = 0;
        const int32_t *row = a.parent + (size_t)b * (a.n_tok + 1);
        for (int i = t; i > 0; ++depth) {
            int p = GDN_IN(row + i, 4, bpar, st) ? row[i] : i - 1;
            if (p < 0 || p >= i) {
                p = i - 1;
                if (lane == 0 && st) atomicOr(st, GDN_DEV_TREE);
            }
            i = p;
        }
    }
    // a chain's last position bounds a tree's; a request is left out as a whole
    const bool fits = ctx >= 0 && (int64_t)ctx + a.n_tok <= (int64_t)a.width << a.page_shift &&
                      (a.rot == 0 || (int64_t)ctx + a.n_tok <= a.max_pos);
    if (!fits) {
        if (lane == 0 && st) atomicOr(st, GDN_DEV_LENGTH);
        return;
    }
    const int pos = ctx + depth - 1, slot = ctx + t - 1;
    const int32_t *entry = a.table + (size_t)b * a.width + (slot >> a.page_shift);
    const int page = GDN_IN(entry, 4, btab, st) ? *entry : -1;
    const bool page_ok = page >= 0 && page < a.n_pages;
    if (!page_ok && lane == 0 && st) atomicOr(st, GDN_DEV_PAGE);

    const int half = a.rot / 2, d0 = lane * 8;
    // this lane's cosines and sines: of its values' pair indices
    float cs[8], sn[8];
    const bool turned = d0 < a.rot;
    if (turned && a.pairs) {
        const float *row = a.rope + (size_t)pos * a.rot + d0 / 2;
        if (GDN_IN(row, 16, brope, st) && GDN_IN(row + half, 16, brope, st)) {
            const float4 c = gdndev::ld4(row), s = gdndev::ld4(row + half);
            cs[0] = cs[1] = c.x, cs[2] = cs[3] = c.y, cs[4] = cs[5] = c.z, cs[6] = cs[7] = c.w;
            sn[0] = sn[1] = s.x, sn[2] = sn[3] = s.y, sn[4] = sn[5] = s.z, sn[6] = sn[7] = s.w;
        }
    } else if (turned) {
        const float *row = a.rope + (size_t)pos * a.rot + (d0 < half ? d0 : d0 - half);
        if (GDN_IN(row, 32, brope, st)) load8<false>(row, 0, cs);
        if (GDN_IN(row + half, 32, brope, st)) load8<false>(row + half, 0, sn);
    }
    float wq[8], wk[8];
    load8<BF16>(a.q_norm, d0, wq);
    load8<BF16>(a.k_norm, d0, wk);
    const int heads = a.h_q + 2 * a.h_kv, stride = per_token * gridDim.y;
    const unsigned mask = kLanes == 32 ? ~0u : ((1u << kLanes) - 1) << (threadIdx.x % 32 / kLanes * kLanes);
    for (int h = group % per_token + per_token * blockIdx.y; h < heads; h += stride) {
        const size_t from = (size_t)token * a.stride + (size_t)h * D + d0;
        float x[8] = {};
        if (GDN_IN(static_cast<const char *>(a.qkv) + from * kElem, 8 * kElem, bx, st)) load8<BF16>(a.qkv, from, x);
        if (h < a.h_q + a.h_kv) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) s = fmaf(x[j], x[j], s);
#pragma unroll
            for (int o = kLanes / 2; o; o >>= 1) s += __shfl_xor_sync(mask, s, o);
            const float r = rsqrtf(s * (1.0f / D) + a.eps);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= r * ((h < a.h_q ? wq[j] : wk[j]) + a.offset);
            if (a.pairs) {
                if (turned) {
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        const float u = x[j], v = x[j + 1];
                        x[j] = u * cs[j] - v * sn[j];
                        x[j + 1] = v * cs[j] + u * sn[j];
                    }
                }
            } else if (a.rot > 0) {
                // the partner lane: rot / 2 values away
                const int hop = half / 8, src = turned ? (d0 < half ? lane + hop : lane - hop) : lane;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float y = __shfl_sync(mask, x[j], src, kLanes);
                    if (turned) x[j] = d0 < half ? x[j] * cs[j] - y * sn[j] : x[j] * cs[j] + y * sn[j];
                }
            }
        }
        if (h < a.h_q) {
            const size_t to = ((size_t)token * a.h_q + h) * D + d0;
            if (GDN_IN(static_cast<char *>(a.q_out) + to * kElem, 8 * kElem, bq, st)) store8<BF16>(a.q_out, to, x);
        } else if (page_ok) {
            const int kv = h < a.h_q + a.h_kv ? h - a.h_q : h - a.h_q - a.h_kv;
            void *pool = h < a.h_q + a.h_kv ? a.k_pages : a.v_pages;
            const size_t to = ((((size_t)page * a.h_kv + kv) << a.page_shift) + (slot & ((1 << a.page_shift) - 1))) * D + d0;
            if (GDN_IN(static_cast<char *>(pool) + to * kElem, 8 * kElem, (h < a.h_q + a.h_kv ? bk : bv), st))
                store8<BF16>(pool, to, x);
        }
    }
}

template <bool BF16, int D>
int launch(RopeArgs a, cudaStream_t st) {
    constexpr int kGroups = kThreads / (D / 8);
    const int heads = a.h_q + 2 * a.h_kv;
    // few heads: several tokens share a block; few tokens: several blocks share
    // a token's heads, until every lane group has one head
    a.tokens_per_block = 1;
    while (a.tokens_per_block * 2 <= kGroups && heads * a.tokens_per_block * 2 <= kGroups) a.tokens_per_block *= 2;
    const int64_t blocks = (a.tokens + a.tokens_per_block - 1) / a.tokens_per_block;
    const int sms = gdnhost::sm_count();
    int parts = (heads * a.tokens_per_block + kGroups - 1) / kGroups;
    const int64_t want = (2 * (sms > 0 ? sms : 152) + blocks - 1) / blocks;
    if (parts > want) parts = (int)want;
    return gdndev::launch_pdl(qk_norm_rope<BF16, D>, dim3((unsigned)blocks, parts < 1 ? 1 : parts), dim3(kThreads), 0, st,
                              a) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
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
