// Attention of a drafted span over the paged cache, in f32 arithmetic
// throughout (attn_verify_span / attn_tree_verify with GDN_F32).
//
// One pass over the keys with the running maximum and sum of each row's
// softmax. A row is a node's query head of one key/value head.
//
// Few rows (single tokens, short chains): attend(). Many rows: attend_many(). Parts
// of a request's slots are joined by a second kernel.
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

// Few rows: R of them a block, each warp with slots of its own, U at a time (2 U
// where half a warp spans a head). A lane holds its columns of the queries, keys,
// values and sums in registers; the next keys are asked for once the products with
// the last are made, the next values once the sums are. Nothing but weights goes
// through shared memory, whose reads bound a form with shared tiles (in brackets):
// 4 requests' single tokens, 16 heads of 256 over 5,000 slots 41 us (100; the bytes
// alone 21); 8 requests', 16 heads of 128 over 2,000 15.3 us with the join (20.6;
// 4.1); one over 777 10.8 us (14.7), two launches. Bound by the wait for the loads,
// 64 KB of them in flight on an SM, and by about as many operations for the sums
// over lanes as for the products. Two blocks an SM leave 128 registers a thread:
// with four rows some 212 bytes of a thread spill (128 and 64 wide), with one or
// two, and in the one-block forms, none.
template <int D, int R>
struct Few {
    static constexpr int kLanes = D == 64 ? 16 : 32, kGroups = 32 / kLanes, kC = D / (4 * kLanes);
    static constexpr int kU = D == 256 && R == 8 ? 4 : 8, kStep = kU * kGroups;  // slots a warp takes at a time
    static constexpr int kScores = R * kU;                                       // of a group of lanes
    static constexpr int kOwn = kScores >= kLanes ? kScores / kLanes : 1;        // of them a lane has in the end
    static constexpr int kSame = kScores >= kLanes ? 1 : kLanes / kScores;       // lanes that have the same
    struct Smem {
        float o[kWarps][R][D];
        float p[kWarps][kGroups][kScores];
        float scale[kWarps][R], m[kWarps][R], l[kWarps][R];
        unsigned long long path[GDN_MAX_TOKENS];
        int parent[GDN_MAX_TOKENS + 1];
    };
};

// x[N] summed over `kLanes` lanes; lane i is left with the sums of its kOwn places
// from i * N / kLanes on (N < kLanes: of place i * N / kLanes). Halves are exchanged,
// so that N sums take N shuffles and not 5 N.
template <int N, int kW>
__device__ __forceinline__ void sum_apart(float *x, int lane) {
    if constexpr (kW > 0) {
        if constexpr (N > 1) {
            const bool upper = lane & kW;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const float keep = upper ? x[i + N / 2] : x[i], send = upper ? x[i] : x[i + N / 2];
                x[i] = keep + __shfl_xor_sync(~0u, send, kW);
            }
            sum_apart<N / 2, kW / 2>(x, lane);
        } else {
            x[0] += __shfl_xor_sync(~0u, x[0], kW);
            sum_apart<1, kW / 2>(x, lane);
        }
    }
}

// grid (row blocks, B * h_kv, parts); partial results [B][n_tok][h_q][parts]
// of D sums (relative to the maximum) and of (maximum, sum) in powers of two.
template <int D, int R>
__global__ void __launch_bounds__(kThreads, R == 8 || D == 256 ? 1 : 2) attend(AttnArgs a, int parts, float *part_o, float2 *part_ms) {
    using F = Few<D, R>;
    constexpr int kC = F::kC, kU = F::kU, kG = F::kGroups, kOwn = F::kOwn;
    extern __shared__ __align__(16) char raw[];
    typename F::Smem &s = *reinterpret_cast<typename F::Smem *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = lane % F::kLanes, grp = lane / F::kLanes;
    const int b = blockIdx.y / a.h_kv, kv = blockIdx.y % a.h_kv, part = blockIdx.z;
    const int group = a.h_q / a.h_kv, rows = a.n_tok * group, row0 = blockIdx.x * R;
    int32_t *st = a.status;
    const size_t B = a.batch, pool = ((size_t)a.n_pages * a.h_kv << a.page_shift) * D * 4, heads = B * a.n_tok * a.h_q;
    const Buf bq{a.q, heads * D * 4}, bk{a.k_pages, pool}, bv{a.v_pages, pool}, bt{a.table, B * (size_t)a.width * 4},
        bo{part_o, heads * parts * D * 4}, bms{part_ms, heads * parts * 8};
    gdndev::pdl_launch_dependents();
    gdndev::pdl_wait();
    const int slots = gdnattn::slots_of(a, b), ctx = slots - a.n_tok;
    if (slots == 0 && tid == 0 && st) atomicOr(st, GDN_DEV_LENGTH);
    constexpr int kBlock = kWarps * F::kStep;
    const int per = ((slots + parts - 1) / parts + kBlock - 1) / kBlock * kBlock;
    const int s0 = (int)min((long long)slots, (long long)part * per), s1 = (int)min((long long)slots, (long long)s0 + per);
    const float *kp = static_cast<const float *>(a.k_pages), *vp = static_cast<const float *>(a.v_pages);
    // lane i knows the page of the warp's i-th slot
    auto page_of = [&](int base) {
        const int slot = base + lane;
        if (lane >= F::kStep || slot >= s1) return -2;  // nothing there
        const int32_t *f = a.table + (size_t)b * a.width + (slot >> a.page_shift);
        return GDN_IN(f, 4, bt, st) ? *f : -1;
    };
    auto place_of = [&](int base, int page) {
        const int slot = base + lane;
        if (page >= 0 && page < a.n_pages)
            return (long long)((((size_t)page * a.h_kv + kv) << a.page_shift) + (slot & ((1 << a.page_shift) - 1))) * D;
        if (page != -2 && st) atomicOr(st, GDN_DEV_PAGE);
        return -1ll;
    };
    auto load = [&](float4 (&x)[kU][kC], const float *from, const Buf &bf, long long place) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const long long at = __shfl_sync(~0u, place, u * kG + grp);
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const float *f = from + at + c * 128 + sub * 4;
                x[u][c] = at >= 0 && GDN_IN(f, 16, bf, st) ? gdndev::ld4(f) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
    };
    float4 q[R][kC], o[R][kC], k[kU][kC], v[kU][kC];
    int base = s0 + warp * F::kStep, next = page_of(base);
    long long place = place_of(base, next);
    next = page_of(base + kBlock);
    load(k, kp, bk, place);
    load(v, vp, bv, place);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int t = (row0 + r) / group, h = kv * group + (row0 + r) % group;
        const float *f = static_cast<const float *>(a.q) + (((size_t)b * a.n_tok + t) * a.h_q + h) * D + sub * 4;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            q[r][c] = row0 + r < rows && GDN_IN(f + c * 128, 16, bq, st) ? gdndev::ld4(f + c * 128) : make_float4(0.f, 0.f, 0.f, 0.f);
            o[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    if (s1 > ctx) gdnattn::root_paths(a, b, s.path, s.parent, tid, kThreads, part == parts - 1, [] { __syncthreads(); });
    // this lane's scores of a step: places own0 + i, slot place / R, row place % R
    const int own0 = F::kScores >= F::kLanes ? sub * kOwn : sub / F::kSame;
    float m[kOwn], l[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) m[i] = -INFINITY, l[i] = 0.f;
    float *pw = s.p[warp][grp];
#pragma unroll 1
    for (; base < s1; base += kBlock) {
        float x[F::kScores];
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                x[u * R + r] = 0.f;
#pragma unroll
                for (int c = 0; c < kC; ++c) x[u * R + r] = gdndev::dot4(q[r][c], k[u][c], x[u * R + r]);
            }
        place = place_of(base + kBlock, next);
        next = page_of(base + 2 * kBlock);
        load(k, kp, bk, place);
        sum_apart<F::kScores, F::kLanes / 2>(x, lane);
        const bool edge = base + F::kStep > ctx;
        float scale[kOwn];
        bool moved = false;
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            const int r = (own0 + i) % R, slot = base + (own0 + i) / R * kG + grp, row = row0 + r;
            const bool seen = !edge || (slot < s1 && (slot < ctx || (row < rows && (s.path[row / group] >> (slot - ctx) & 1))));
            const float score = seen ? x[i] * a.scale_log2 : -INFINITY;
            float top = score;
#pragma unroll
            for (int w = F::kSame * R / kOwn; w < 32; w *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
            const float m2 = fmaxf(m[i], top), mm = m2 == -INFINITY ? 0.f : m2, p = exp2f(score - mm);
            scale[i] = exp2f(m[i] - mm);
            moved |= m2 != m[i];
            m[i] = m2;
            l[i] = l[i] * scale[i] + p;
            pw[own0 + i] = seen ? p : -1.f;  // below zero: not in the sum, whatever v holds
        }
        if (__any_sync(~0u, moved)) {
#pragma unroll
            for (int i = 0; i < kOwn; ++i) s.scale[warp][(own0 + i) % R] = scale[i];
            __syncwarp();
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float f = s.scale[warp][r];
#pragma unroll
                for (int c = 0; c < kC; ++c) o[r][c] = make_float4(o[r][c].x * f, o[r][c].y * f, o[r][c].z * f, o[r][c].w * f);
            }
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float w = pw[u * R + r];
                if (!edge || w >= 0.f || w != w)
#pragma unroll
                    for (int c = 0; c < kC; ++c) {
                        o[r][c].x = fmaf(w, v[u][c].x, o[r][c].x);
                        o[r][c].y = fmaf(w, v[u][c].y, o[r][c].y);
                        o[r][c].z = fmaf(w, v[u][c].z, o[r][c].z);
                        o[r][c].w = fmaf(w, v[u][c].w, o[r][c].w);
                    }
            }
        __syncwarp();  // the weights' and scales' places are written again
        load(v, vp, bv, place);
    }
    // the warps' sums on one scale
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        float sum = l[i];
#pragma unroll
        for (int w = F::kSame * R / kOwn; w < 32; w *= 2) sum += __shfl_xor_sync(~0u, sum, w);
        s.m[warp][(own0 + i) % R] = m[i];
        s.l[warp][(own0 + i) % R] = sum;
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            if (kG == 2) {
                o[r][c].x += __shfl_xor_sync(~0u, o[r][c].x, 16);
                o[r][c].y += __shfl_xor_sync(~0u, o[r][c].y, 16);
                o[r][c].z += __shfl_xor_sync(~0u, o[r][c].z, 16);
                o[r][c].w += __shfl_xor_sync(~0u, o[r][c].w, 16);
            }
            if (grp == 0) *reinterpret_cast<float4 *>(&s.o[warp][r][c * 128 + sub * 4]) = o[r][c];
        }
    __syncthreads();
    for (int i = tid; i < R * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = i % (D / 4) * 4, row = row0 + r;
        if (row >= rows) break;
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s.m[w][r]);
        const float mm = top == -INFINITY ? 0.f : top;
        float4 all = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2f(s.m[w][r] - mm);  // 0 for a warp that had no slot
            const float4 y = *reinterpret_cast<const float4 *>(&s.o[w][r][c]);
            sum = fmaf(s.l[w][r], f, sum);
            all = make_float4(fmaf(y.x, f, all.x), fmaf(y.y, f, all.y), fmaf(y.z, f, all.z), fmaf(y.w, f, all.w));
        }
        const int t = row / group, h = kv * group + row % group;
        const size_t at = (((size_t)b * a.n_tok + t) * a.h_q + h) * parts + part;
        if (c == 0 && GDN_IN(part_ms + at, 8, bms, st)) part_ms[at] = make_float2(top, sum);
        float *to = part_o + at * D + c;
        if (GDN_IN(to, 16, bo, st)) *reinterpret_cast<float4 *>(to) = all;
    }
}

__device__ __forceinline__ void copy16(void *to, const void *from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((unsigned)__cvta_generic_to_shared(to)), "l"(from),
                 "r"(there ? 16 : 0)
                 : "memory");  // zeros where there is nothing to copy
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

int few_rows(int rows) { return rows <= 1 ? 1 : rows <= 2 ? 2 : rows <= 4 ? 4 : 8; }

// Whether attend_many() takes a call, and how: a lane's rows (R), the warps side
// by side in rows, the parts that a request's slots are cut into by blocks, and
// the partial results of a row.
struct Cut {
    int lane_rows, row_warps, row_blocks, parts, pieces;
};

// attend() holds eight rows in registers and reads the cache again for the next
// eight: attend_many() from nine rows on (8 requests of 16 rows, 4 heads of 128 over
// 3,000 slots: 55 us against 57); heads of 256, whose tiles leave it no room for less
// than 64 rows, from 33 on (2 requests of 28 rows over 3,000: 55 against 29).
Cut cut_of(const attn_dims *dims, int n_tok) {
    const int d = dims->d_head, rows = n_tok * (dims->h_q / dims->h_kv);
    const int64_t slots = (int64_t)dims->table_width * dims->page_tokens;  // the longest request that the table holds
    Cut c{};
    const int sms = gdnhost::sm_count();
    int tile, held = sms > 0 ? sms : 152, slot_warps = 1;  // slots that a block takes at a time, blocks that the GPU holds
    if (rows <= (d == 256 ? 32 : 8)) {
        const int block = few_rows(rows);
        c.row_blocks = (rows + block - 1) / block;
        tile = 128;
        if (block < 8 && d < 256) held *= 2;
    } else {
        c.lane_rows = d == 256 || rows <= 32 ? 4 : 8;
        // the fewest rows of padding, then the fewest copies of a tile
        for (int w = kWarps; w >= (d == 256 ? 4 : 2); w /= 2) {
            const int block = w * 4 * c.lane_rows, blocks = (rows + block - 1) / block;
            if (!c.row_warps || blocks * w < c.row_blocks * c.row_warps) c.row_warps = w, c.row_blocks = blocks;
        }
        slot_warps = kWarps / c.row_warps;
        tile = kTile * slot_warps;
    }
    // the parts whose rounds of blocks take the fewest tiles, half a tile counted for a block's start and end
    const int64_t tiles = (slots + tile - 1) / tile, units = (int64_t)c.row_blocks * dims->batch * dims->h_kv;
    int64_t best = INT64_MAX;
    for (int p = 1; p <= kMaxParts / slot_warps && (p == 1 || p <= tiles); ++p) {
        const int64_t cost = (units * p + held - 1) / held * (2 * ((tiles + p - 1) / p) + 1);
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
    constexpr size_t kSmem = sizeof(typename Few<D, R>::Smem);
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
    if (c.lane_rows) {
        if constexpr (D == 256) ok = launch_many<D, 4>(a, c, o, ms, st);
        else ok = c.lane_rows == 8 ? launch_many<D, 8>(a, c, o, ms, st) : launch_many<D, 4>(a, c, o, ms, st);
    } else {
        switch (few_rows(a.n_tok * (a.h_q / a.h_kv))) {
            case 1: ok = launch_few<D, 1>(a, c, o, ms, st); break;
            case 2: ok = launch_few<D, 2>(a, c, o, ms, st); break;
            case 4: ok = launch_few<D, 4>(a, c, o, ms, st); break;
            default: ok = launch_few<D, 8>(a, c, o, ms, st);
        }
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
