// Attention of a drafted span over the paged cache, in f32 arithmetic
// throughout (attn_verify_span / attn_tree_verify with GDN_F32).
//
// One pass over the keys with the running maximum and sum of each row's
// softmax. A block takes 32 query rows (nodes x query heads of one key/value
// head) and a part of the slots; a warp takes 8 of the rows, a lane one of a
// tile's 32 slots for the scores and D / 32 of the columns for the sums. Parts
// are joined by a second kernel. Bound by the f32 pipe: 4 D operations per row
// and slot.
#include <cuda_runtime.h>

#include "attn_common.cuh"
#include "attn_host.h"
#include "gdn_host.h"
#include "gdnspec.h"

namespace {

using gdnattn::AttnArgs;
using gdndev::Buf;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kRowsPerWarp = 8;
constexpr int kRows = kWarps * kRowsPerWarp;
constexpr int kTile = 32;
constexpr int kMaxParts = 64;

template <bool BF16, int D>
__device__ __forceinline__ void load_row4(const void *p, size_t i, float4 &x) {
    if constexpr (BF16) {
        const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p) + i);
        x = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                        __uint_as_float(u.y & 0xffff0000u));
    } else {
        x = gdndev::ld4(static_cast<const float *>(p) + i);
    }
}

template <int D>
struct Shared {
    float q[kRows][D];
    float k[kTile][D + 4];
    float v[kTile][D];
    float p[kRows][kTile];
    unsigned long long path[GDN_MAX_TOKENS];
    int parent[GDN_MAX_TOKENS + 1];
};

// grid (row blocks, B * h_kv, parts); partial results [B][n_tok][h_q][parts]
// of D sums (relative to the maximum) and of (maximum, sum) in powers of two.
template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads) attend(AttnArgs a, int parts, float *part_o, float2 *part_ms) {
    extern __shared__ __align__(16) char raw[];
    Shared<D> &s = *reinterpret_cast<Shared<D> *>(raw);
    constexpr int kElem = BF16 ? 2 : 4, kCols = D / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.y / a.h_kv, kv = blockIdx.y % a.h_kv, part = blockIdx.z;
    const int group = a.h_q / a.h_kv, rows = a.n_tok * group, row0 = blockIdx.x * kRows;
    int32_t *st = a.status;
    const size_t B = a.batch, pool = ((size_t)a.n_pages * a.h_kv << a.page_shift) * D * kElem,
                 heads = B * a.n_tok * a.h_q;
    const Buf bq{a.q, heads * D * kElem}, bk{a.k_pages, pool}, bv{a.v_pages, pool}, bt{a.table, B * (size_t)a.width * 4},
        bo{part_o, heads * parts * D * 4}, bms{part_ms, heads * parts * 8};
    gdndev::pdl_launch_dependents();
    gdndev::pdl_wait();
    const int slots = gdnattn::slots_of(a, b), ctx = slots - a.n_tok;
    if (slots == 0 && tid == 0 && st) atomicOr(st, GDN_DEV_LENGTH);
    const int per = ((slots + parts - 1) / parts + kTile - 1) / kTile * kTile;
    const int s0 = min(slots, part * per), s1 = min(slots, s0 + per);
    gdnattn::root_paths(a, b, s.path, s.parent, tid, kThreads, part == 0, [] { __syncthreads(); });
    for (int i = tid; i < kRows * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row0 + r < rows) {
            const int t = (row0 + r) / group, h = kv * group + (row0 + r) % group;
            const size_t at = (((size_t)b * a.n_tok + t) * a.h_q + h) * D + c;
            if (GDN_IN(static_cast<const char *>(a.q) + at * kElem, 4 * kElem, bq, st)) load_row4<BF16, D>(a.q, at, x);
        }
        *reinterpret_cast<float4 *>(&s.q[r][c]) = x;
    }
    float m[kRowsPerWarp], l[kRowsPerWarp], o[kRowsPerWarp][kCols];
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
        m[r] = -INFINITY, l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < kCols; ++c) o[r][c] = 0.f;
    }
    for (int base = s0; base < s1; base += kTile) {
        __syncthreads();
        for (int i = tid; i < kTile * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = i % (D / 4) * 4, slot = base + r;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
            if (slot < s1) {
                const int32_t *e = a.table + (size_t)b * a.width + (slot >> a.page_shift);
                const int page = GDN_IN(e, 4, bt, st) ? *e : -1;
                if (page >= 0 && page < a.n_pages) {
                    const size_t at = ((((size_t)page * a.h_kv + kv) << a.page_shift) + (slot & ((1 << a.page_shift) - 1))) * D + c;
                    if (GDN_IN(static_cast<const char *>(a.k_pages) + at * kElem, 4 * kElem, bk, st)) load_row4<BF16, D>(a.k_pages, at, x);
                    if (GDN_IN(static_cast<const char *>(a.v_pages) + at * kElem, 4 * kElem, bv, st)) load_row4<BF16, D>(a.v_pages, at, y);
                } else if (c == 0 && st) {
                    atomicOr(st, GDN_DEV_PAGE);
                }
            }
            *reinterpret_cast<float4 *>(&s.k[r][c]) = x;
            *reinterpret_cast<float4 *>(&s.v[r][c]) = y;
        }
        __syncthreads();
        float sc[kRowsPerWarp] = {};
#pragma unroll 4
        for (int c = 0; c < D; c += 4) {
            const float4 kk = *reinterpret_cast<const float4 *>(&s.k[lane][c]);
#pragma unroll
            for (int r = 0; r < kRowsPerWarp; ++r)
                sc[r] = gdndev::dot4(*reinterpret_cast<const float4 *>(&s.q[warp * kRowsPerWarp + r][c]), kk, sc[r]);
        }
        const int slot = base + lane;
#pragma unroll
        for (int r = 0; r < kRowsPerWarp; ++r) {
            const int row = row0 + warp * kRowsPerWarp + r;
            const unsigned long long path = row < rows ? s.path[row / group] : ~0ull;
            const bool seen = slot < s1 && (slot < ctx || (path >> (slot - ctx) & 1));
            const float x = seen ? sc[r] * a.scale_log2 : -INFINITY;
            float top = x;
#pragma unroll
            for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
            const float m2 = fmaxf(m[r], top), mm = m2 == -INFINITY ? 0.f : m2;
            const float scale = exp2f(m[r] - mm), p = exp2f(x - mm);
            m[r] = m2;
            l[r] = l[r] * scale + p;
#pragma unroll
            for (int c = 0; c < kCols; ++c) o[r][c] *= scale;
            s.p[warp * kRowsPerWarp + r][lane] = seen ? p : -1.f;  // below zero: not in the sum, whatever v holds
        }
        __syncwarp();
        const int n = min(kTile, s1 - base);
        for (int j = 0; j < n; ++j) {
            float vv[kCols];
#pragma unroll
            for (int c = 0; c < kCols; ++c) vv[c] = s.v[j][lane + c * 32];
#pragma unroll
            for (int r = 0; r < kRowsPerWarp; ++r) {
                const float p = s.p[warp * kRowsPerWarp + r][j];
                if (p >= 0.f || p != p)
#pragma unroll
                    for (int c = 0; c < kCols; ++c) o[r][c] = fmaf(p, vv[c], o[r][c]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
        float sum = l[r];
#pragma unroll
        for (int w = 16; w; w >>= 1) sum += __shfl_xor_sync(~0u, sum, w);
        const int row = row0 + warp * kRowsPerWarp + r;
        if (row < rows) {
            const int t = row / group, h = kv * group + row % group;
            const size_t at = (((size_t)b * a.n_tok + t) * a.h_q + h) * parts + part;
            if (lane == 0 && GDN_IN(part_ms + at, 8, bms, st)) part_ms[at] = make_float2(m[r], sum);
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                float *to = part_o + at * D + lane + c * 32;
                if (GDN_IN(to, 4, bo, st)) *to = o[r][c];
            }
        }
    }
}

// One warp per output row: the parts' maxima, then their sums on that scale.
template <bool BF16, int D>
__global__ void __launch_bounds__(256) join_parts(AttnArgs a, int parts, const float *part_o, const float2 *part_ms) {
    const int64_t rows = (int64_t)a.batch * a.n_tok * a.h_q, row = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    constexpr int kCols = D / 32, kElem = BF16 ? 2 : 4;
    int32_t *st = a.status;
    const Buf bo{part_o, (size_t)rows * parts * D * 4}, bms{part_ms, (size_t)rows * parts * 8}, bout{a.out, (size_t)rows * D * kElem};
    gdndev::pdl_wait();
    gdndev::pdl_launch_dependents();
    if (row >= rows) return;
    float m = -INFINITY;
    for (int p = lane; p < parts; p += 32) {
        const float2 *f = part_ms + row * parts + p;
        if (GDN_IN(f, 8, bms, st)) m = fmaxf(m, f->x);
    }
#pragma unroll
    for (int w = 16; w; w >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, w));
    const float mm = m == -INFINITY ? 0.f : m;
    float sum = 0.f, o[kCols] = {};
    for (int p = 0; p < parts; ++p) {
        const float2 *f = part_ms + row * parts + p;
        const float2 ms = GDN_IN(f, 8, bms, st) ? *f : make_float2(-INFINITY, 0.f);
        if (ms.x == -INFINITY && ms.y == 0.f) continue;  // this part held nothing that the row sees
        const float w = exp2f(ms.x - mm);
        sum += ms.y * w;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
            const float *g = part_o + (row * parts + p) * D + lane + c * 32;
            if (GDN_IN(g, 4, bo, st)) o[c] = fmaf(*g, w, o[c]);
        }
    }
    // a request that is left out has no sum and gets zeros
    const bool empty = m == -INFINITY && sum == 0.f;
    const float inv = 1.f / sum;
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
        const float x = empty ? 0.f : o[c] * inv;
        const size_t at = (size_t)row * D + lane + c * 32;
        if (GDN_IN(static_cast<char *>(a.out) + at * kElem, kElem, bout, st)) {
            if constexpr (BF16) static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(x);
            else static_cast<float *>(a.out)[at] = x;
        }
    }
}

template <bool BF16, int D>
int launch(const AttnArgs &a, int parts, void *ws, cudaStream_t st) {
    constexpr size_t kSmem = sizeof(Shared<D>);
    static bool set[256] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return GDN_ERR_CUDA;
    if (!set[dev]) {
        if (cudaFuncSetAttribute(attend<BF16, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) != cudaSuccess)
            return GDN_ERR_CUDA;
        set[dev] = true;
    }
    const int64_t out_rows = (int64_t)a.batch * a.n_tok * a.h_q;
    float2 *ms = static_cast<float2 *>(ws);
    float *o = reinterpret_cast<float *>(static_cast<char *>(ws) + ((size_t)out_rows * parts * 8 + 255) / 256 * 256);
    const int rows = a.n_tok * (a.h_q / a.h_kv);
    // batch * h_kv goes to gridDim.y: 65535 of them a launch
    if ((int64_t)a.batch * a.h_kv > 65535) return GDN_ERR_DIMS;
    if (gdndev::launch_pdl(attend<BF16, D>, dim3((rows + kRows - 1) / kRows, a.batch * a.h_kv, parts), dim3(kThreads), kSmem,
                           st, a, parts, o, ms) != cudaSuccess)
        return GDN_ERR_CUDA;
    return gdndev::launch_pdl(join_parts<BF16, D>, dim3((unsigned)((out_rows + 7) / 8)), dim3(256), 0, st, a, parts,
                              (const float *)o, (const float2 *)ms) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

namespace gdnattn {

// Parts a request's slots are cut into: enough blocks for the GPU, and no part
// under 128 slots of the longest request that the table holds.
int simt_parts(const attn_dims *d, int n_tok) {
    const int rows = n_tok * (d->h_q / d->h_kv);
    const int64_t blocks = (int64_t)((rows + kRows - 1) / kRows) * d->batch * d->h_kv;
    const int64_t slots = (int64_t)d->table_width * d->page_tokens;
    int64_t parts = (2 * 152 + blocks - 1) / blocks;
    if (parts > (slots + 127) / 128) parts = (slots + 127) / 128;
    return (int)(parts < 1 ? 1 : parts > kMaxParts ? kMaxParts : parts);
}

size_t simt_workspace(const attn_dims *d, int n_tok) {
    const size_t heads = (size_t)d->batch * n_tok * d->h_q * simt_parts(d, n_tok);
    return (heads * 8 + 255) / 256 * 256 + heads * d->d_head * 4;
}

int simt_launch(const attn_dims *d, const AttnArgs &a, void *ws, cudaStream_t st) {
    const int parts = simt_parts(d, a.n_tok);
    if (d->in_dtype == GDN_BF16)
        return a.d == 64 ? launch<true, 64>(a, parts, ws, st) : a.d == 128 ? launch<true, 128>(a, parts, ws, st)
                                                                           : launch<true, 256>(a, parts, ws, st);
    return a.d == 64 ? launch<false, 64>(a, parts, ws, st) : a.d == 128 ? launch<false, 128>(a, parts, ws, st)
                                                                        : launch<false, 256>(a, parts, ws, st);
}

}  // namespace gdnattn
