// Attention of a drafted span over the paged cache, in f32 arithmetic
// throughout (attn_verify_span / attn_tree_verify with GDN_F32).
//
// One pass over the keys with the running maximum and sum of each row's
// softmax. A block takes 8 R query rows (nodes x query heads of one key/value
// head) and a part of the slots; a warp takes R of the rows, a lane one of a
// tile's 32 slots for the scores and D / 32 of the columns for the sums. The
// next tile is copied into shared memory while one is worked on. R is 1, 2, 4 or
// 8: the least that takes all rows in one block, so that a single token's few
// heads do not carry empty rows along. Parts are joined by a second kernel.
// Bound by the f32 pipe and the shared-memory reads that feed it (4 D operations
// per row and slot) with many rows, by the copies with few.
#include <cuda_runtime.h>

#include "attn_common.cuh"
#include "attn_host.h"
#include "gdn_host.h"
#include "gdnspec.h"

namespace {

using gdnattn::AttnArgs;
using gdndev::Buf;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 32;
constexpr int kMaxParts = 128;

template <int D, int R>
struct Shared {
    float q[kWarps * R][D];
    float k[2][kTile][D + 4];  // rows 16 bytes apart in the banks
    float v[2][kTile][D];
    float p[kWarps * R][kTile];
    unsigned long long path[GDN_MAX_TOKENS];
    int parent[GDN_MAX_TOKENS + 1];
};

__device__ __forceinline__ void copy16(void *to, const void *from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((unsigned)__cvta_generic_to_shared(to)), "l"(from),
                 "r"(there ? 16 : 0)
                 : "memory");  // zeros where there is nothing to copy
}

// grid (row blocks, B * h_kv, parts); partial results [B][n_tok][h_q][parts]
// of D sums (relative to the maximum) and of (maximum, sum) in powers of two.
template <int D, int R>
__global__ void __launch_bounds__(kThreads) attend(AttnArgs a, int parts, float *part_o, float2 *part_ms) {
    extern __shared__ __align__(16) char raw[];
    Shared<D, R> &s = *reinterpret_cast<Shared<D, R> *>(raw);
    constexpr int kCols = D / 32, kRows = kWarps * R;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.y / a.h_kv, kv = blockIdx.y % a.h_kv, part = blockIdx.z;
    const int group = a.h_q / a.h_kv, rows = a.n_tok * group, row0 = blockIdx.x * kRows;
    int32_t *st = a.status;
    const size_t B = a.batch, pool = ((size_t)a.n_pages * a.h_kv << a.page_shift) * D * 4, heads = B * a.n_tok * a.h_q;
    const Buf bq{a.q, heads * D * 4}, bk{a.k_pages, pool}, bv{a.v_pages, pool}, bt{a.table, B * (size_t)a.width * 4},
        bo{part_o, heads * parts * D * 4}, bms{part_ms, heads * parts * 8};
    gdndev::pdl_launch_dependents();
    gdndev::pdl_wait();
    const int slots = gdnattn::slots_of(a, b), ctx = slots - a.n_tok;
    if (slots == 0 && tid == 0 && st) atomicOr(st, GDN_DEV_LENGTH);
    const int per = ((slots + parts - 1) / parts + kTile - 1) / kTile * kTile;
    const int s0 = min(slots, part * per), s1 = min(slots, s0 + per);
    const float *kp = static_cast<const float *>(a.k_pages), *vp = static_cast<const float *>(a.v_pages);
    // a warp copies four rows of a tile; their pages are looked up first
    auto fetch = [&](int base, int buf) {
#pragma unroll
        for (int i = 0; i < kTile / kWarps; ++i) {
            const int r = warp * (kTile / kWarps) + i, slot = base + r;
            size_t at = 0;
            bool there = false;
            if (slot < s1) {
                const int32_t *e = a.table + (size_t)b * a.width + (slot >> a.page_shift);
                const int page = GDN_IN(e, 4, bt, st) ? *e : -1;
                there = page >= 0 && page < a.n_pages;
                if (!there && lane == 0 && st) atomicOr(st, GDN_DEV_PAGE);
                at = ((((size_t)(there ? page : 0) * a.h_kv + kv) << a.page_shift) + (slot & ((1 << a.page_shift) - 1))) * D;
            }
#pragma unroll
            for (int c = lane * 4; c < D; c += 128) {
                copy16(&s.k[buf][r][c], kp + at + c, there && GDN_IN(kp + at + c, 16, bk, st));
                copy16(&s.v[buf][r][c], vp + at + c, there && GDN_IN(vp + at + c, 16, bv, st));
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (s0 < s1) fetch(s0, 0);
    for (int i = tid; i < kRows * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row0 + r < rows) {
            const int t = (row0 + r) / group, h = kv * group + (row0 + r) % group;
            const float *f = static_cast<const float *>(a.q) + (((size_t)b * a.n_tok + t) * a.h_q + h) * D + c;
            if (GDN_IN(f, 16, bq, st)) x = gdndev::ld4(f);
        }
        *reinterpret_cast<float4 *>(&s.q[r][c]) = x;
    }
    if (s1 > ctx) gdnattn::root_paths(a, b, s.path, s.parent, tid, kThreads, part == parts - 1, [] { __syncthreads(); });
    float m[R], l[R], o[R][kCols];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY, l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < kCols; ++c) o[r][c] = 0.f;
    }
    for (int base = s0, buf = 0; base < s1; base += kTile, buf ^= 1) {
        if (base + kTile < s1) {
            fetch(base + kTile, buf ^ 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();
        if (row0 + warp * R < rows) {
            float sc[R] = {};
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                const float4 kk = *reinterpret_cast<const float4 *>(&s.k[buf][lane][c]);
#pragma unroll
                for (int r = 0; r < R; ++r)
                    sc[r] = gdndev::dot4(*reinterpret_cast<const float4 *>(&s.q[warp * R + r][c]), kk, sc[r]);
            }
            const int slot = base + lane;
            const bool edge = base + kTile > ctx;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int row = row0 + warp * R + r;
                const bool seen = !edge || (slot < s1 && (slot < ctx || (row < rows && (s.path[row / group] >> (slot - ctx) & 1))));
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
                s.p[warp * R + r][lane] = seen ? p : -1.f;  // below zero: not in the sum, whatever v holds
            }
            __syncwarp();
#pragma unroll 1
            for (int j = 0; j < kTile; j += 4) {
                float4 p[R];
#pragma unroll
                for (int r = 0; r < R; ++r) p[r] = *reinterpret_cast<const float4 *>(&s.p[warp * R + r][j]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float vv[kCols];
#pragma unroll
                    for (int c = 0; c < kCols; ++c) vv[c] = s.v[buf][j + i][lane + c * 32];
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float w = i == 0 ? p[r].x : i == 1 ? p[r].y : i == 2 ? p[r].z : p[r].w;
                        if (!edge || w >= 0.f || w != w)
#pragma unroll
                            for (int c = 0; c < kCols; ++c) o[r][c] = fmaf(w, vv[c], o[r][c]);
                    }
                }
            }
        }
        __syncthreads();  // the buffer is fetched into again
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float sum = l[r];
#pragma unroll
        for (int w = 16; w; w >>= 1) sum += __shfl_xor_sync(~0u, sum, w);
        const int row = row0 + warp * R + r;
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
template <int D>
__global__ void __launch_bounds__(256) join_parts(AttnArgs a, int parts, const float *part_o, const float2 *part_ms) {
    const int64_t rows = (int64_t)a.batch * a.n_tok * a.h_q, row = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    constexpr int kCols = D / 32;
    int32_t *st = a.status;
    const Buf bo{part_o, (size_t)rows * parts * D * 4}, bms{part_ms, (size_t)rows * parts * 8}, bout{a.out, (size_t)rows * D * 4};
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
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
        const float2 *f = part_ms + row * parts + p;
        const float2 ms = GDN_IN(f, 8, bms, st) ? *f : make_float2(-INFINITY, 0.f);
        const float w = exp2f(ms.x - mm);  // 0 for a part that held nothing that the row sees: its sums are zeros
        sum = fmaf(ms.y, w, sum);
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
        float *to = static_cast<float *>(a.out) + row * D + lane + c * 32;
        if (GDN_IN(to, 4, bout, st)) *to = empty ? 0.f : o[c] * inv;
    }
}

int rows_per_warp(int rows) { return rows <= kWarps ? 1 : rows <= 2 * kWarps ? 2 : rows <= 4 * kWarps ? 4 : 8; }

template <int D, int R>
int launch(const AttnArgs &a, int parts, void *ws, cudaStream_t st) {
    constexpr size_t kSmem = sizeof(Shared<D, R>);
    static bool set[256] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return GDN_ERR_CUDA;
    if (!set[dev]) {
        if (cudaFuncSetAttribute(attend<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) != cudaSuccess)
            return GDN_ERR_CUDA;
        set[dev] = true;
    }
    const int64_t out_rows = (int64_t)a.batch * a.n_tok * a.h_q;
    float2 *ms = static_cast<float2 *>(ws);
    float *o = reinterpret_cast<float *>(static_cast<char *>(ws) + ((size_t)out_rows * parts * 8 + 255) / 256 * 256);
    const int rows = a.n_tok * (a.h_q / a.h_kv);
    if (gdndev::launch_pdl(attend<D, R>, dim3((rows + kWarps * R - 1) / (kWarps * R), a.batch * a.h_kv, parts), dim3(kThreads),
                           kSmem, st, a, parts, o, ms) != cudaSuccess)
        return GDN_ERR_CUDA;
    return gdndev::launch_pdl(join_parts<D>, dim3((unsigned)((out_rows + 7) / 8)), dim3(256), 0, st, a, parts, (const float *)o,
                              (const float2 *)ms) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <int D>
int launch_rows(const AttnArgs &a, int parts, void *ws, cudaStream_t st) {
    switch (rows_per_warp(a.n_tok * (a.h_q / a.h_kv))) {
        case 1: return launch<D, 1>(a, parts, ws, st);
        case 2: return launch<D, 2>(a, parts, ws, st);
        case 4: return launch<D, 4>(a, parts, ws, st);
        default: return launch<D, 8>(a, parts, ws, st);
    }
}

// Parts a request's slots are cut into: enough blocks for the GPU, and no part
// under four tiles of the longest request that the table holds.
int parts_of(const attn_dims *d, int n_tok) {
    const int rows = n_tok * (d->h_q / d->h_kv), block = kWarps * rows_per_warp(rows);
    const int64_t blocks = (int64_t)((rows + block - 1) / block) * d->batch * d->h_kv;
    const int64_t slots = (int64_t)d->table_width * d->page_tokens;
    int64_t parts = (4 * 152 + blocks - 1) / blocks;
    if (parts > (slots + 4 * kTile - 1) / (4 * kTile)) parts = (slots + 4 * kTile - 1) / (4 * kTile);
    return (int)(parts < 1 ? 1 : parts > kMaxParts ? kMaxParts : parts);
}

}  // namespace

namespace gdnattn {

size_t simt_workspace(const attn_dims *d, int n_tok) {
    const size_t heads = (size_t)d->batch * n_tok * d->h_q * parts_of(d, n_tok);
    return (heads * 8 + 255) / 256 * 256 + heads * d->d_head * 4;
}

int simt_launch(const attn_dims *d, const AttnArgs &a, void *ws, cudaStream_t st) {
    const int parts = parts_of(d, a.n_tok);
    return a.d == 64 ? launch_rows<64>(a, parts, ws, st) : a.d == 128 ? launch_rows<128>(a, parts, ws, st)
                                                                      : launch_rows<256>(a, parts, ws, st);
}

}  // namespace gdnattn
