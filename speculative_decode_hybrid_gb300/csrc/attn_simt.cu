// Attention of a drafted span over the paged cache, in f32 arithmetic
// throughout (attn_verify_span / attn_tree_verify with GDN_F32).
//
// One pass over the keys with the running maximum and sum of each row's
// softmax. A row is a node's query head of one key/value head.
//
// Few rows (attend(): single tokens, short chains): a block takes 8 R rows and a
// part of the slots; a warp takes R of the rows, a lane one of a tile's 32 slots
// for the scores and D / 32 of the columns for the sums. The next tile is copied
// into shared memory while one is worked on. R is 1, 2 or 4: the least that takes
// all rows in one block, so that a single token's few heads do not carry empty
// rows along. Bound by the copies' latency: 8 requests' single tokens, 16 heads of
// 128 over 2,000 slots take 20.6 us with the join (the bytes alone 4.1).
//
// Many rows: attend_many(), below. Parts are joined by a second kernel.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

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

// Many rows: a warp takes 4 R rows and its own tile of 32 slots, a lane R rows by
// four slots of the scores and R rows by D / 8 columns of the sums, so that a
// value read from shared memory goes into four to R products. The block's eight
// warps are `row_warps` by kWarps / row_warps: those in a row of warps share a tile,
// the others have tiles, and partial results, of their own. The next tile's keys
// are copied while the weights multiply the values, its values during the scores.
// Bound by the f32 pipe (4 D operations per row and slot) and by the shared-memory
// reads that feed it: a lane reads 48 numbers for 128 products of the scores (at
// 32 lanes' numbers a cycle that is 2/3 of the pipe's rate) and 24 for 128 of the
// sums. Measured, with a warp of R rows and a slot a lane for comparison:
// 8 requests, 64 nodes, 32 heads of 128 over 4,000 slots 704 us (1,217; the pipe
// alone 417); 4 spans of 16, 32 heads of 128 over 4,000 131 us (196; 52); 22 nodes,
// 16 heads of 256 over 8,000 115 us (183; 36); 8 trees of 40, 8 heads of 64 over
// 3,000 107 us (113; 24: 40 rows fill 64). Pairs of f32 products in one
// instruction in the sums took 8 % off; in the scores, whose reads bound them,
// nothing, nor did a rescaling left out where no maximum moved.
constexpr int kLaneSlots = 4;

template <int D, int R>
struct Many {
    static constexpr int kRows = 4 * R;  // of a warp
    static constexpr int kKRow = D + 4, kPRow = kRows + 4;  // rows 16 bytes apart in the banks
    static __host__ __device__ constexpr size_t floats(int row_warps) {
        return (size_t)(kWarps / row_warps) * kTile * (kKRow + D) + (size_t)row_warps * kRows * kKRow + kWarps * kTile * kPRow;
    }
    static constexpr size_t bytes(int row_warps) {
        return floats(row_warps) * 4 + GDN_MAX_TOKENS * 8 + (GDN_MAX_TOKENS + 1) * 4;
    }
};

template <int D, int R>
__global__ void __launch_bounds__(kThreads, 1)
attend_many(AttnArgs a, int parts, int row_warps_log, float *part_o, float2 *part_ms) {
    using M = Many<D, R>;
    extern __shared__ __align__(16) char raw[];
    constexpr int kChunks = D / 32, kJ = kLaneSlots;
    const int row_warps = 1 << row_warps_log, slot_warps = kWarps >> row_warps_log;
    const int step = kTile * slot_warps;  // slots that the block takes at a time
    float *ks = reinterpret_cast<float *>(raw), *vs = ks + step * M::kKRow, *qs = vs + step * D,
          *ps = qs + row_warps * M::kRows * M::kKRow;
    unsigned long long *path = reinterpret_cast<unsigned long long *>(ps + kWarps * kTile * M::kPRow);
    int *parent = reinterpret_cast<int *>(path + GDN_MAX_TOKENS);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 3, e = lane & 7;
    const int row_warp = warp & (row_warps - 1), slot_warp = warp >> row_warps_log;
    const int b = blockIdx.y / a.h_kv, kv = blockIdx.y % a.h_kv, part = blockIdx.z;
    const int group = a.h_q / a.h_kv, rows = a.n_tok * group, row0 = blockIdx.x * row_warps * M::kRows;
    int32_t *st = a.status;
    const size_t B = a.batch, pool = ((size_t)a.n_pages * a.h_kv << a.page_shift) * D * 4, heads = B * a.n_tok * a.h_q;
    const size_t pieces = (size_t)parts * slot_warps;
    const Buf bq{a.q, heads * D * 4}, bk{a.k_pages, pool}, bv{a.v_pages, pool}, bt{a.table, B * (size_t)a.width * 4},
        bo{part_o, heads * pieces * D * 4}, bms{part_ms, heads * pieces * 8};
    gdndev::pdl_launch_dependents();
    gdndev::pdl_wait();
    const int slots = gdnattn::slots_of(a, b), ctx = slots - a.n_tok;
    if (slots == 0 && tid == 0 && st) atomicOr(st, GDN_DEV_LENGTH);
    const int per = ((slots + parts - 1) / parts + step - 1) / step * step;
    const int s0 = (int)min((long long)slots, (long long)part * per), s1 = (int)min((long long)slots, (long long)s0 + per);
    const float *kp = static_cast<const float *>(a.k_pages), *vp = static_cast<const float *>(a.v_pages);
    // A warp copies 4 slot_warps rows of the block's tiles; lane i knows the page of the i-th.
    const int mine = 4 * slot_warps, first = warp * mine;
    auto page_of = [&](int base) {
        const int slot = base + first + lane;
        if (lane >= mine || slot >= s1) return -2;  // nothing there
        const int32_t *f = a.table + (size_t)b * a.width + (slot >> a.page_shift);
        return GDN_IN(f, 4, bt, st) ? *f : -1;
    };
    auto place_of = [&](int base, int page) {
        const int slot = base + first + lane;
        if (page >= 0 && page < a.n_pages)
            return (long long)((((size_t)page * a.h_kv + kv) << a.page_shift) + (slot & ((1 << a.page_shift) - 1))) * D;
        if (page != -2 && st) atomicOr(st, GDN_DEV_PAGE);
        return -1ll;
    };
    auto fetch = [&](long long place, const float *from, const Buf &bf, float *to, int stride) {
#pragma unroll 4
        for (int i = 0; i < mine; ++i) {
            const long long at = __shfl_sync(~0u, place, i);
#pragma unroll
            for (int c = lane * 4; c < D; c += 128) {
                const float *f = from + (at < 0 ? 0 : at) + c;
                copy16(to + (first + i) * stride + c, f, at >= 0 && GDN_IN(f, 16, bf, st));
            }
        }
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
    auto all_but_one = [] { asm volatile("cp.async.wait_group 1;" ::: "memory"); };
    if (s0 < s1) {
        const long long place = place_of(s0, page_of(s0));
        fetch(place, kp, bk, ks, M::kKRow);
        commit();
        fetch(place, vp, bv, vs, D);
        commit();
    }
    for (int i = tid; i < row_warps * M::kRows * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row0 + r < rows) {
            const int t = (row0 + r) / group, h = kv * group + (row0 + r) % group;
            const float *f = static_cast<const float *>(a.q) + (((size_t)b * a.n_tok + t) * a.h_q + h) * D + c;
            if (GDN_IN(f, 16, bq, st)) x = gdndev::ld4(f);
        }
        *reinterpret_cast<float4 *>(qs + r * M::kKRow + c) = x;
    }
    if (s1 > ctx) gdnattn::root_paths(a, b, path, parent, tid, kThreads, part == parts - 1, [] { __syncthreads(); });
    // a lane's rows are row0 + row_warp * kRows + 4 r + g
    const int lane_row = row0 + row_warp * M::kRows + g;
    const bool rows_here = row0 + row_warp * M::kRows < rows;
    const float *kw = ks + (slot_warp * kTile + e) * M::kKRow, *vw = vs + slot_warp * kTile * D + e * 4,
                *qw = qs + (row_warp * M::kRows + g) * M::kKRow;
    float *pw = ps + warp * kTile * M::kPRow + g * R;
    float m[R], l[R];
    float2 o[R][kChunks * 2];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY, l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < kChunks * 2; ++c) o[r][c] = make_float2(0.f, 0.f);
    }
    // the sums take a tile's weights; with `edge` a weight below zero is no part of them, whatever v holds
    auto add = [&](auto edge) {
#pragma unroll 2
        for (int j = 0; j < kTile; ++j) {
            float p[R];
            float4 v[kChunks];
#pragma unroll
            for (int r = 0; r < R; r += 4)
                *reinterpret_cast<float4 *>(p + r) = *reinterpret_cast<const float4 *>(pw + j * M::kPRow + r);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) v[c] = *reinterpret_cast<const float4 *>(vw + j * D + c * 32);
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (!decltype(edge)::value || p[r] >= 0.f || p[r] != p[r])
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        const float2 pp = make_float2(p[r], p[r]);
                        o[r][c * 2] = gdndev::fma2(pp, make_float2(v[c].x, v[c].y), o[r][c * 2]);
                        o[r][c * 2 + 1] = gdndev::fma2(pp, make_float2(v[c].z, v[c].w), o[r][c * 2 + 1]);
                    }
        }
    };
    for (int base = s0; base < s1; base += step) {
        const int own = base + slot_warp * kTile;  // this warp's tile
        const bool active = rows_here && own < s1, edge = own + kTile > ctx;
        const int next = base + step < s1 ? page_of(base + step) : -2;
        float sc[R][kJ] = {};
        all_but_one();
        __syncthreads();  // the keys are there
        if (active) {
#pragma unroll 2
            for (int c = 0; c < D; c += 4) {
                float4 k[kJ];
#pragma unroll
                for (int j = 0; j < kJ; ++j) k[j] = *reinterpret_cast<const float4 *>(kw + j * 8 * M::kKRow + c);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float4 q = *reinterpret_cast<const float4 *>(qw + r * 4 * M::kKRow + c);
#pragma unroll
                    for (int j = 0; j < kJ; ++j) sc[r][j] = gdndev::dot4(q, k[j], sc[r][j]);
                }
            }
        }
        __syncthreads();  // the keys have been read
        const long long place = place_of(base + step, next);
        if (base + step < s1) fetch(place, kp, bk, ks, M::kKRow);
        commit();
        if (active) {
            unsigned seen = ~0u;  // bit 4 r + j
            if (edge) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int row = lane_row + 4 * r;
                    const unsigned long long bits = row < rows && s1 > ctx ? path[row / group] : 0ull;
#pragma unroll
                    for (int j = 0; j < kJ; ++j) {
                        const int slot = own + j * 8 + e;
                        if (slot >= s1 || (slot >= ctx && !(bits >> (slot - ctx) & 1))) seen &= ~(1u << (4 * r + j));
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
                    sc[r][j] = seen >> (4 * r + j) & 1 ? sc[r][j] * a.scale_log2 : -INFINITY;
                    top = fmaxf(top, sc[r][j]);
                }
#pragma unroll
                for (int w = 4; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
                const float m2 = fmaxf(m[r], top), mm = m2 == -INFINITY ? 0.f : m2, scale = exp2f(m[r] - mm);
                m[r] = m2;
                l[r] *= scale;
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
                    const float p = exp2f(sc[r][j] - mm);
                    l[r] += p;
                    sc[r][j] = seen >> (4 * r + j) & 1 ? p : -1.f;
                }
#pragma unroll
                for (int c = 0; c < kChunks * 2; ++c) o[r][c] = gdndev::mul2(o[r][c], make_float2(scale, scale));
            }
#pragma unroll
            for (int j = 0; j < kJ; ++j)
#pragma unroll
                for (int r = 0; r < R; r += 4)
                    *reinterpret_cast<float4 *>(pw + (j * 8 + e) * M::kPRow + r) =
                        make_float4(sc[r][j], sc[r + 1][j], sc[r + 2][j], sc[r + 3][j]);
        }
        all_but_one();
        __syncthreads();  // the values are there, and the warp's weights
        if (active) {
            if (edge)
                add(std::true_type{});
            else
                add(std::false_type{});
        }
        __syncthreads();  // the values have been read
        if (base + step < s1) fetch(place, vp, bv, vs, D);
        commit();
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float sum = l[r];
#pragma unroll
        for (int w = 4; w; w >>= 1) sum += __shfl_xor_sync(~0u, sum, w);
        const int row = lane_row + 4 * r;
        if (row < rows) {
            const int t = row / group, h = kv * group + row % group;
            const size_t at = (((size_t)b * a.n_tok + t) * a.h_q + h) * pieces + part * slot_warps + slot_warp;
            if (e == 0 && GDN_IN(part_ms + at, 8, bms, st)) part_ms[at] = make_float2(m[r], sum);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                float *to = part_o + at * D + e * 4 + c * 32;
                if (GDN_IN(to, 16, bo, st))
                    *reinterpret_cast<float4 *>(to) = make_float4(o[r][c * 2].x, o[r][c * 2].y, o[r][c * 2 + 1].x, o[r][c * 2 + 1].y);
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

int rows_per_warp(int rows) { return rows <= kWarps ? 1 : rows <= 2 * kWarps ? 2 : 4; }

// Whether attend_many() takes a call, and how: a lane's rows (R), the warps side
// by side in rows, the parts that a request's slots are cut into by blocks, and
// the partial results of a row.
struct Cut {
    int lane_rows, row_warps, row_blocks, parts, pieces;
};

// attend_many() from one row more on than the other kernel's warps hold with two
// each; heads of 256, whose tiles leave it no room for less than 64 rows, from 33 on.
Cut cut_of(const attn_dims *dims, int n_tok) {
    const int batch = dims->batch, h_kv = dims->h_kv, d = dims->d_head;
    const int rows = n_tok * (dims->h_q / h_kv), few = d == 256 ? 4 * kWarps : 2 * kWarps;
    const int64_t slots = (int64_t)dims->table_width * dims->page_tokens;
    Cut c{};
    if (rows <= few) {
        // enough blocks for the GPU, and no part under four tiles of the longest request that the table holds
        const int block = kWarps * rows_per_warp(rows);
        const int64_t blocks = (int64_t)((rows + block - 1) / block) * batch * h_kv;
        const int64_t most = (slots + 4 * kTile - 1) / (4 * kTile), parts = (4 * 152 + blocks - 1) / blocks;
        c.row_blocks = (rows + block - 1) / block;
        c.parts = (int)(parts > most ? most : parts);
        c.parts = c.parts > kMaxParts ? kMaxParts : c.parts < 1 ? 1 : c.parts;
        c.pieces = c.parts;
        return c;
    }
    c.lane_rows = d == 256 || rows <= 32 ? 4 : 8;
    // the fewest rows of padding, then the fewest copies of a tile
    for (int w = kWarps; w >= (d == 256 ? 4 : 2); w /= 2) {
        const int block = w * 4 * c.lane_rows, blocks = (rows + block - 1) / block;
        if (!c.row_warps || blocks * w < c.row_blocks * c.row_warps) c.row_warps = w, c.row_blocks = blocks;
    }
    // one block of an SM at a time: the parts whose rounds of blocks take the fewest tiles, half a
    // tile counted for a block's start and end
    const int slot_warps = kWarps / c.row_warps;
    const int64_t tiles = (slots + kTile * slot_warps - 1) / (kTile * slot_warps), units = (int64_t)c.row_blocks * batch * h_kv;
    int64_t best = INT64_MAX;
    for (int p = 1; p <= kMaxParts / slot_warps && (p == 1 || 2 * p <= tiles); ++p) {
        const int64_t cost = (units * p + 151) / 152 * (2 * ((tiles + p - 1) / p) + 1);
        if (cost < best) best = cost, c.parts = p;
    }
    c.pieces = c.parts * slot_warps;
    return c;
}

// Lets a kernel have `bytes` of shared memory, once for each device.
template <typename Kernel>
bool allow_smem(Kernel kernel, size_t bytes, bool (&set)[256]) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return false;
    if (!set[dev]) set[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess;
    return set[dev];
}

template <int D, int R>
bool launch_few(const AttnArgs &a, const Cut &c, float *o, float2 *ms, cudaStream_t st) {
    constexpr size_t kSmem = sizeof(Shared<D, R>);
    static bool set[256] = {};
    return allow_smem(attend<D, R>, kSmem, set) &&
           gdndev::launch_pdl(attend<D, R>, dim3(c.row_blocks, a.batch * a.h_kv, c.parts), dim3(kThreads), kSmem, st, a, c.parts, o,
                              ms) == cudaSuccess;
}

template <int D, int R>
bool launch_many(const AttnArgs &a, const Cut &c, float *o, float2 *ms, cudaStream_t st) {
    using M = Many<D, R>;
    constexpr int kFew = D == 256 ? 4 : 2;
    constexpr size_t kMost = M::bytes(kFew) > M::bytes(kWarps) ? M::bytes(kFew) : M::bytes(kWarps);
    static_assert(kMost <= 227 * 1024 && M::bytes(4) <= kMost, "shared memory of a block");
    static bool set[256] = {};
    const int log = c.row_warps == 8 ? 3 : c.row_warps == 4 ? 2 : 1;
    return allow_smem(attend_many<D, R>, kMost, set) &&
           gdndev::launch_pdl(attend_many<D, R>, dim3(c.row_blocks, a.batch * a.h_kv, c.parts), dim3(kThreads),
                              M::bytes(c.row_warps), st, a, c.parts, log, o, ms) == cudaSuccess;
}

template <int D>
int launch(const AttnArgs &a, const Cut &c, void *ws, cudaStream_t st) {
    const int64_t out_rows = (int64_t)a.batch * a.n_tok * a.h_q;
    float2 *ms = static_cast<float2 *>(ws);
    float *o = reinterpret_cast<float *>(static_cast<char *>(ws) + ((size_t)out_rows * c.pieces * 8 + 255) / 256 * 256);
    bool ok;
    if constexpr (D == 256) {
        const int r = rows_per_warp(a.n_tok * (a.h_q / a.h_kv));
        ok = c.lane_rows ? launch_many<D, 4>(a, c, o, ms, st) : r == 1 ? launch_few<D, 1>(a, c, o, ms, st)
           : r == 2 ? launch_few<D, 2>(a, c, o, ms, st) : launch_few<D, 4>(a, c, o, ms, st);
    } else {
        ok = c.lane_rows == 8 ? launch_many<D, 8>(a, c, o, ms, st) : c.lane_rows == 4 ? launch_many<D, 4>(a, c, o, ms, st)
           : rows_per_warp(a.n_tok * (a.h_q / a.h_kv)) == 1 ? launch_few<D, 1>(a, c, o, ms, st) : launch_few<D, 2>(a, c, o, ms, st);
    }
    if (!ok) return GDN_ERR_CUDA;
    return gdndev::launch_pdl(join_parts<D>, dim3((unsigned)((out_rows + 7) / 8)), dim3(256), 0, st, a, c.pieces, (const float *)o,
                              (const float2 *)ms) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

namespace gdnattn {

size_t simt_workspace(const attn_dims *d, int n_tok) {
    const size_t heads = (size_t)d->batch * n_tok * d->h_q * cut_of(d, n_tok).pieces;
    return (heads * 8 + 255) / 256 * 256 + heads * d->d_head * 4;
}

int simt_launch(const attn_dims *d, const AttnArgs &a, void *ws, cudaStream_t st) {
    const Cut c = cut_of(d, a.n_tok);
    return a.d == 64 ? launch<64>(a, c, ws, st) : a.d == 128 ? launch<128>(a, c, ws, st) : launch<256>(a, c, ws, st);
}

}  // namespace gdnattn
