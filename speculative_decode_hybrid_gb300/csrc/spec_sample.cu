// spec_accept_sample: drafted tokens verified against the target's
// probabilities, from given random numbers (the sampled counterpart of
// spec_accept_greedy; lucebox PR #533, Changes: the acceptance runs on the
// GPU's logits).
//
// Mathematics. p_n = softmax(l_n / T). The children of a node are tried in
// index order against the rest r of its row, r = p at first. With draft rows q
// a rejection turns r into max(r - q, 0) / sum, and by induction the rest
// after j rejections is (p - c_j q)+ / S_j with
//   c_0 = 0, S_0 = 1,   c_{j+1} = c_j + S_j,   S_{j+1} = sum_v (p_v - c_{j+1} q_v)+,
// so a sibling costs one sum over the row and no row is rewritten. With fixed
// candidates a rejection removes the token, so child x is accepted when
// u (1 - sum of the removed p) < p(x). A node's index exceeds its parent's:
// one pass over the nodes in index order, with the last accepted node in hand,
// is the walk. The next token is the largest r_v / noise_v: an argmax, which
// needs neither a prefix sum nor r's normalisation.
//
// Two launches. sample_rows reads the logits once (all N rows: each drafted
// token's probability is an output), every block an equal, contiguous part of
// them all, whichever rows that cuts, with a running maximum and sum; a grid of
// whole rows or half rows leaves the last wave half empty (50 us instead of 37
// for 16 x 23 rows of 151,936). sample_pick is one cluster of blocks per request:
// all of them repeat the walk, then each takes a slice of the accepted row (and
// of q and the noise), and the first joins their candidates; what does not
// depend on the sums is read while they are still being taken. The first launch
// is bound by the logits' bytes (38 us for 224 MB, 0.87 of the measured copy rate),
// the second by latency: 14 us for the same 16 requests, in which a row's loads
// follow the walk, the walk the statistics, and those the tokens. A rejected sibling
// of a sampled draft is one more pass over its row and the draft's by the request's
// cluster: 60 us for those 16 trees with draft rows, 52 with fixed candidates. Its blocks are
// held to 64 registers: at one block an SM, only 15 of the 16 clusters of eight
// fit the GPU at once (47 us).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <initializer_list>
#include <type_traits>

#include "gdn_device.cuh"
#include "gdn_host.h"
#include "gdnspec.h"

namespace {

using gdndev::Buf;
using gdndev::key_index;
using gdndev::make_key;
using gdndev::umax64;

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 6;
constexpr int kPickThreads = 512;
constexpr int kCluster = 8;
constexpr int kAhead = 3;           // 16-byte loads of each row a thread of sample_pick has in flight
constexpr int kMaxPieces = 40;      // blocks that a row may be spread over
static_assert(kMaxPieces <= 64, "two pieces a lane");
constexpr int kMinPart = 1024;      // values a block takes at least
constexpr int kMaxNodes = GDN_MAX_TOKENS + 1;
// Indexes of a row, and what is added to them (a slice's rounding, a pass of the
// scan), are 32-bit.
constexpr int kMaxVocab = 1 << 30;
constexpr float kLog2e = 1.4426950408889634f;

// A row's maximum and the sum of exp((x - max) / T).
struct Stat {
    float m, s;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// exp((x - m) / T), c = log2(e) / T. The difference is taken first: near the
// maximum, where the weight lies, it is exact.
__device__ __forceinline__ float weight(float x, float m, float c) { return ex2((x - m) * c); }

// T == 0 is the limit: a factor that leaves weight only where x - m is 0.
__device__ __forceinline__ float coefficient(const float *temperature, int b) {
    const float t = temperature ? temperature[b] : 1.f;
    return t > 0.f ? fminf(kLog2e / t, 3e38f) : 3e38f;
}

// Join two parts' statistics. A part without a value above -inf has m = -inf
// and s = 0; NaN stays in s.
__device__ __forceinline__ Stat join(Stat a, Stat b, float c) {
    const float m = fmaxf(a.m, b.m);
    if (m == -INFINITY) return {m, a.s + b.s};
    const float wa = a.m == -INFINITY ? 0.f : weight(a.m, m, c), wb = b.m == -INFINITY ? 0.f : weight(b.m, m, c);
    return {m, a.s * wa + b.s * wb};
}

template <int K>
__device__ __forceinline__ void absorb(Stat &st, const float (&x)[K], float c) {
    float top = x[0];
#pragma unroll
    for (int i = 1; i < K; ++i) top = fmaxf(top, x[i]);
    if (top > st.m) {
        st.s = st.m == -INFINITY ? st.s : st.s * weight(st.m, top, c);
        st.m = top;
    }
    const float m = st.m == -INFINITY ? 0.f : st.m;  // all -inf so far: every weight is exp(-inf) = 0
    float s[4] = {};
#pragma unroll
    for (int i = 0; i < K; ++i) s[i & 3] += weight(x[i], m, c);
    st.s += (s[0] + s[1]) + (s[2] + s[3]);
}

// How the rows' values, one row after the other, are dealt out to the blocks.
struct Deal {
    int64_t part, total;  // values a block, a multiple of 4; all of them
    int blocks, pieces;   // at most so many of a row
};

__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
sample_rows(int n_nodes, int vocab, Deal deal, const float *__restrict__ logits, const float *__restrict__ temperature,
            const float *__restrict__ noise, Stat *__restrict__ stats, int rows, int32_t *dev_status) {
    __shared__ Stat warp_stat[2][kThreads / 32];
    const int tid = threadIdx.x;
    const Buf bl{logits, (size_t)deal.total * 4}, bs{stats, (size_t)rows * kMaxPieces * sizeof(Stat)};
    gdndev::pdl_wait();
    gdndev::pdl_launch_dependents();  // the next kernel may read this one's inputs: they are complete
    const int64_t lo = blockIdx.x * deal.part, hi = min(deal.total, lo + deal.part);
    int row = (int)(lo / vocab), flip = 0;
    for (int64_t at = lo; at < hi; ++row, flip ^= 1) {
        const int64_t begin = (int64_t)row * vocab, end = min(hi, begin + vocab);
        const float c = coefficient(temperature, row / n_nodes);
        const float *r = logits + at;
        const int n = (int)(end - at);
        Stat st{-INFINITY, 0.f};
        // scalars up to the first 16-byte boundary, 16 bytes at a time, scalars again
        const int head = min(n, (int)((16 - (reinterpret_cast<uintptr_t>(r) & 15)) & 15) / 4);
        const int body = (n - head) / 4, tail = head + body * 4;
        const float4 *r4 = reinterpret_cast<const float4 *>(r + head);
        int i = tid;
        for (; i + 3 * kThreads < body; i += 4 * kThreads) {
            float x[16];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 f = GDN_IN(r4 + i + j * kThreads, 16, bl, dev_status) ? __ldg(r4 + i + j * kThreads)
                                                                                   : make_float4(0.f, 0.f, 0.f, 0.f);
                x[4 * j] = f.x, x[4 * j + 1] = f.y, x[4 * j + 2] = f.z, x[4 * j + 3] = f.w;
            }
            absorb(st, x, c);
        }
        for (; i < body; i += kThreads) {
            const float4 f = GDN_IN(r4 + i, 16, bl, dev_status) ? __ldg(r4 + i) : make_float4(0.f, 0.f, 0.f, 0.f);
            const float x[4] = {f.x, f.y, f.z, f.w};
            absorb(st, x, c);
        }
        for (int e = tid; e < head + n - tail; e += kThreads) {
            const float *f = r + (e < head ? e : tail + e - head);
            const float x[1] = {GDN_IN(f, 4, bl, dev_status) ? *f : 0.f};
            absorb(st, x, c);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1)
            st = join(st, {__shfl_xor_sync(~0u, st.m, o), __shfl_xor_sync(~0u, st.s, o)}, c);
        if ((tid & 31) == 0) warp_stat[flip][tid >> 5] = st;
        __syncthreads();
        if (tid == 0) {
#pragma unroll
            for (int w = 1; w < kThreads / 32; ++w) st = join(st, warp_stat[flip][w], c);
            // the row's pieces in order, from the block in which it begins on; what is
            // left of their places stands for nothing
            int k = blockIdx.x - (int)(begin / deal.part);
            Stat *to = stats + (size_t)row * kMaxPieces;
            if (GDN_IN(to + k, sizeof(Stat), bs, dev_status)) to[k] = st;
            for (++k; end == begin + vocab && k < deal.pieces; ++k)
                if (GDN_IN(to + k, sizeof(Stat), bs, dev_status)) to[k] = {-INFINITY, 0.f};
        }
        at = end;
    }
    // the noise that sample_pick reads, on its way to L2
    const size_t lines = (size_t)(rows / n_nodes) * vocab * 4;
    gdndev::prefetch_l2_range(noise, lines, blockIdx.x * kThreads + tid, gridDim.x * kThreads);
}

struct PickArgs {
    int n_nodes, vocab;
    Deal deal;
    const float *logits, *draft;
    const int32_t *tokens, *parent;
    const float *temperature, *uniforms, *noise;
    int32_t *accept_len, *accept_node, *next_token;
    float *token_prob;
    const Stat *stats;
    int32_t *status;
};

// op over the cluster's threads; 0 is op's neutral value.
template <typename T, typename Op>
__device__ __forceinline__ T cluster_reduce(T v, T *warp_buf, T *cta_buf, Op op) {
    namespace cg = cooperative_groups;
    cg::cluster_group cl = cg::this_cluster();
#pragma unroll
    for (int o = 16; o; o >>= 1) v = op(v, __shfl_xor_sync(~0u, v, o));
    if ((threadIdx.x & 31) == 0) warp_buf[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = threadIdx.x < kPickThreads / 32 ? warp_buf[threadIdx.x] : T(0);
#pragma unroll
        for (int o = 16; o; o >>= 1) v = op(v, __shfl_xor_sync(~0u, v, o));
        // every CTA gets every CTA's value, in rank order: the same result everywhere
        if (threadIdx.x < kCluster) cl.map_shared_rank(cta_buf, threadIdx.x)[cl.block_rank()] = v;
    }
    cl.sync();
    v = cta_buf[0];
#pragma unroll
    for (int r = 1; r < kCluster; ++r) v = op(v, cta_buf[r]);
    return v;
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPickThreads, 2)
sample_pick(PickArgs a) {
    namespace cg = cooperative_groups;
    __shared__ float row_m[kMaxNodes], row_s[kMaxNodes];
    __shared__ float p_of[kMaxNodes], q_of[kMaxNodes], u_of[kMaxNodes];
    __shared__ int parent_of[kMaxNodes], token_of[kMaxNodes], removed[kMaxNodes], step_of[kMaxNodes], n_removed;
    __shared__ bool gone_before[kMaxNodes], more_after[kMaxNodes];
    __shared__ float sum_warp[32], sum_cta[2][kCluster];
    __shared__ unsigned long long key_warp[32], key_cta[2][kCluster];
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / kCluster, rank = (int)cl.block_rank();
    const int N = a.n_nodes, V = a.vocab;
    const size_t B = gridDim.x / kCluster;
    int32_t *st = a.status;
    const Buf bl{a.logits, B * N * (size_t)V * 4}, bq{a.draft, B * (N - 1) * (size_t)V * 4},
        bt{a.tokens, B * N * 4}, bp{a.parent, B * N * 4}, bu{a.uniforms, B * N * 4}, bn{a.noise, B * (size_t)V * 4},
        bs{a.stats, B * N * (size_t)kMaxPieces * sizeof(Stat)};
    // sample_rows lets this kernel start once its own inputs are complete, so all
    // but the statistics can be read before it ends
    cl.barrier_arrive();
    const float c = coefficient(a.temperature, b);
    if (tid < N) {
        int p = tid - 1, t = -1;
        if (a.parent) {
            const int32_t *f = a.parent + (size_t)b * N + tid;
            p = GDN_IN(f, 4, bp, st) ? *f : 0;
        }
        if (tid > 0) {
            const int32_t *f = a.tokens + (size_t)b * N + tid;
            t = GDN_IN(f, 4, bt, st) ? *f : 0;
            if (p < 0 || p >= tid) {
                p = -2;  // never reached
                if (rank == 0 && st) atomicOr(st, GDN_DEV_TREE);
            } else if (t < 0 || t >= V) {
                t = -1;
                if (rank == 0 && st) atomicOr(st, GDN_DEV_TOKEN_RANGE);
            }
            const float *fu = a.uniforms + (size_t)b * N + tid;
            u_of[tid] = GDN_IN(fu, 4, bu, st) ? *fu : 0.f;
        } else {
            p = -2;
        }
        parent_of[tid] = p;
        token_of[tid] = t;
    }
    if (tid == 0) n_removed = 0;
    __syncthreads();
    float x_token = 0.f;
    if (tid > 0 && tid < N) {
        const int p = parent_of[tid], t = token_of[tid];
        float qv = 0.f;
        bool dup = false, more = false;
        if (p >= 0 && t >= 0) {
            const float *fl = a.logits + ((size_t)b * N + p) * V + t;
            if (GDN_IN(fl, 4, bl, st)) x_token = *fl;
            if (a.draft) {
                const float *fq = a.draft + ((size_t)b * (N - 1) + p) * V + t;
                if (GDN_IN(fq, 4, bq, st)) qv = *fq;
            }
        }
        for (int j = 1; j < N; ++j)
            if (p >= 0 && parent_of[j] == p) {
                dup |= j < tid && token_of[j] == t;
                more |= j > tid;
            }
        q_of[tid] = qv;
        gone_before[tid] = dup;
        more_after[tid] = more;
    }
    gdndev::pdl_wait();
    gdndev::pdl_launch_dependents();
    for (int n = warp; n < N; n += kPickThreads / 32) {
        const Stat *row = a.stats + ((size_t)b * N + n) * kMaxPieces;
        Stat s[2];  // kMaxPieces is at most 64
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = k * 32 + lane;
            s[k] = i < a.deal.pieces && GDN_IN(row + i, sizeof(Stat), bs, st) ? row[i] : Stat{-INFINITY, 0.f};
        }
        Stat all{fmaxf(s[0].m, s[1].m), 0.f};
#pragma unroll
        for (int o = 16; o; o >>= 1) all.m = fmaxf(all.m, __shfl_xor_sync(~0u, all.m, o));
#pragma unroll
        for (int k = 0; k < 2; ++k) all.s += s[k].m == -INFINITY ? s[k].s : s[k].s * weight(s[k].m, all.m, c);
#pragma unroll
        for (int o = 16; o; o >>= 1) all.s += __shfl_xor_sync(~0u, all.s, o);
        if (lane == 0) {
            // a row with NaN, +inf or nothing above -inf has no distribution
            const bool none = all.m == -INFINITY || all.m == INFINITY || all.s != all.s;
            row_m[n] = all.m;
            row_s[n] = none ? __int_as_float(0x7fc00000) : all.s;
            if (none && rank == 0 && st) atomicOr(st, GDN_DEV_NAN_LOGIT);
        }
    }
    __syncthreads();
    if (tid > 0 && tid < N) {
        const int p = parent_of[tid];
        const float pv = p >= 0 && token_of[tid] >= 0 ? weight(x_token, row_m[p], c) / row_s[p] : 0.f;
        p_of[tid] = pv;
        if (a.token_prob && rank == 0) a.token_prob[(size_t)b * N + tid] = pv;
    }
    __syncthreads();
    if (tid > 0 && tid < N) {
        // whether the node is accepted once its turn comes; with draft rows only a
        // first child's test is known beforehand
        const int p = parent_of[tid];
        float gone = 0.f;
        if (!a.draft)
            for (int j = 1; j < tid; ++j) gone += parent_of[j] == p && !gone_before[j] ? p_of[j] : 0.f;
        const bool ok = p >= 0 && token_of[tid] >= 0 &&
                        (a.draft ? u_of[tid] * q_of[tid] < p_of[tid] : !gone_before[tid] && u_of[tid] * (1.f - gone) < p_of[tid]);
        step_of[tid] = p * 2 + ok;
    }
    __syncthreads();

    cl.barrier_wait();  // every block of the cluster runs: their shared memory may be written

    // the slice of a row that this block takes
    const int per = ((V + kCluster - 1) / kCluster + 3) & ~3;
    const int lo = min(V, rank * per), hi = min(V, lo + per);
    const float *noise = a.noise + (size_t)b * V;

    // the walk, the same in every thread of the cluster
    int node = 0, len = 0, flip = 0;
    float coef = 0.f, mass = 1.f;
#pragma unroll 8
    for (int i = 1; i < N; ++i) {
        const int step = step_of[i];
        if (step >> 1 != node) continue;
        const bool ok = coef == 0.f ? step & 1
                                    : token_of[i] >= 0 && u_of[i] * q_of[i] * mass < fmaxf(p_of[i] - coef * q_of[i], 0.f);
        if (ok) {
            node = i;
            ++len;
            coef = 0.f, mass = 1.f;
        } else if (a.draft) {
            coef += mass;
            if (more_after[i] && row_s[node] == row_s[node]) {
                const float *l = a.logits + ((size_t)b * N + node) * V, *q = a.draft + ((size_t)b * (N - 1) + node) * V;
                const float m = row_m[node], inv = 1.f / row_s[node];
                float s = 0.f;
#pragma unroll 4
                for (int v = lo + tid; v < hi; v += kPickThreads)
                    if (GDN_IN(l + v, 4, bl, st) && GDN_IN(q + v, 4, bq, st))
                        s += fmaxf(weight(l[v], m, c) * inv - coef * q[v], 0.f);
                mass = cluster_reduce(s, sum_warp, sum_cta[flip], [](float x, float y) { return x + y; });
                flip ^= 1;
            }
        }
    }

    // the next token: the largest rest / noise of the accepted row
    const float m = row_m[node], total = row_s[node], inv = 1.f / total;
    const bool defined = total == total;
    if (!a.draft && tid > node && tid < N && parent_of[tid] == node && token_of[tid] >= 0 && !gone_before[tid])
        removed[atomicAdd(&n_removed, 1)] = token_of[tid];  // in any order: only looked up
    __syncthreads();
    const int gone_tokens = n_removed;
    const float *l = a.logits + ((size_t)b * N + node) * V;
    // 16 bytes at a time where every row begins on such a boundary
    const bool wide = (V & 3) == 0 && ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.noise) |
                                        reinterpret_cast<uintptr_t>(a.draft)) & 15) == 0;
    float top, top_x;
    int at;
    // this thread's best; with_q: of (p - coef q)+ / noise, else of p / noise less
    // the removed tokens (without p's divisor, which is the same for all)
    auto scan = [&](auto with_q, int gone) {
        // the removed tokens among this thread's values: two are compared with
        // everywhere, more (a token is seldom removed at all) looked up
        int gone0 = -1, gone1 = -1;
        bool many = false;
        for (int j = 0; j < gone; ++j) {
            const int r = removed[j], i = r - lo;
            if (i < 0 || i >= hi - lo || (wide ? i / 4 : i) % kPickThreads != tid) continue;
            many |= gone1 >= 0;
            gone1 = gone0;
            gone0 = r;
        }
        const float *q = with_q ? a.draft + ((size_t)b * (N - 1) + node) * V : nullptr;
        top = 0.f, at = 0, top_x = 0.f;
        auto offer = [&](int v, float x, float e, float qv) {
            float w = weight(x, m, c);
            if constexpr (with_q) w = fmaf(-coef, qv, w * inv);
            if constexpr (!with_q) {
                if (v == gone0 || v == gone1) w = 0.f;
                if (many)
                    for (int j = 0; j < gone; ++j)
                        if (removed[j] == v) w = 0.f;
            }
            const float f = __fdividef(w, e);
            const bool more = f > top && w > 0.f;  // selected, not branched over: some lane of a warp nearly always has more
            top = more ? f : top;
            at = more ? v : at;
            top_x = more ? x : top_x;
        };
        if (wide) {
            for (int v0 = lo + tid * 4; v0 < hi; v0 += kPickThreads * 4 * kAhead) {
                float4 x[kAhead], e[kAhead], y[kAhead];
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    const int v = v0 + j * kPickThreads * 4;
                    if (v < hi) {
                        x[j] = e[j] = y[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (GDN_IN(l + v, 16, bl, st)) x[j] = gdndev::ld4(l + v);
                        if (GDN_IN(noise + v, 16, bn, st)) e[j] = gdndev::ld4(noise + v);
                        if (with_q && GDN_IN(q + v, 16, bq, st)) y[j] = gdndev::ld4(q + v);
                    }
                }
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    const int v = v0 + j * kPickThreads * 4;
                    if (v >= hi) break;
                    offer(v, x[j].x, e[j].x, y[j].x);
                    offer(v + 1, x[j].y, e[j].y, y[j].y);
                    offer(v + 2, x[j].z, e[j].z, y[j].z);
                    offer(v + 3, x[j].w, e[j].w, y[j].w);
                }
            }
        } else {
            for (int v0 = lo + tid; v0 < hi; v0 += kPickThreads * kAhead) {
                float x[kAhead], e[kAhead], y[kAhead];
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    const int v = v0 + j * kPickThreads;
                    if (v < hi) {
                        x[j] = GDN_IN(l + v, 4, bl, st) ? l[v] : 0.f;
                        e[j] = GDN_IN(noise + v, 4, bn, st) ? noise[v] : 0.f;
                        y[j] = with_q && GDN_IN(q + v, 4, bq, st) ? q[v] : 0.f;
                    }
                }
#pragma unroll
                for (int j = 0; j < kAhead; ++j)
                    if (v0 + j * kPickThreads < hi) offer(v0 + j * kPickThreads, x[j], e[j], y[j]);
            }
        }
    };
    auto larger = [](unsigned long long x, unsigned long long y) { return umax64(x, y); };
    unsigned long long key = 0ull, best = 0ull;
    if (defined) {
        if (coef > 0.f)
            scan(std::true_type{}, 0);
        else
            scan(std::false_type{}, gone_tokens);
        key = top > 0.f ? make_key(top, (unsigned)at) : 0ull;
        best = cluster_reduce(key, key_warp, key_cta[0], larger);
        if (best == 0ull) {  // nothing is left of the row: p itself
            __syncthreads();
            scan(std::false_type{}, 0);
            key = top > 0.f ? make_key(top, (unsigned)at) : 0ull;
            best = cluster_reduce(key, key_warp, key_cta[1], larger);
        }
    }
    // written by the thread that has the best, or the first where there is none
    if (best ? key == best : rank == 0 && tid == 0) {
        a.next_token[b] = best ? at : 0;
        if (a.token_prob) {
            const bool first = GDN_IN(l, 4, bl, st);
            a.token_prob[(size_t)b * N] = weight(best ? top_x : first ? l[0] : 0.f, m, c) / total;
        }
    }
    if (rank == 0 && tid == 0) {
        a.accept_len[b] = len;
        a.accept_node[b] = node;
    }
    // the last thing written into other blocks' shared memory came before the
    // reduction's barrier: a block may leave
}

// Equal parts for as many blocks as the GPU holds, none below kMinPart values,
// no row in more than kMaxPieces pieces.
Deal deal_out(int64_t rows, int vocab) {
    const int sms = gdnhost::sm_count();
    const int64_t blocks = (int64_t)kBlocksPerSm * (sms > 0 ? sms : 152), total = rows * vocab;
    int64_t part = (total + blocks - 1) / blocks;
    const int64_t by_row = (vocab + kMaxPieces - 2) / (kMaxPieces - 1);
    if (part < by_row) part = by_row;
    if (part < kMinPart) part = kMinPart;
    part = (part + 3) & ~3LL;
    return {part, total, (int)((total + part - 1) / part), (int)((vocab + part - 1) / part) + 1};
}

}  // namespace

extern "C" size_t spec_accept_sample_workspace_bytes(int32_t batch, int32_t n_nodes) {
    if (batch < 1 || batch > 65535 || n_nodes < 1 || n_nodes > kMaxNodes) return 0;
    return (size_t)batch * n_nodes * kMaxPieces * sizeof(Stat);
}

extern "C" int spec_accept_sample(int32_t batch, int32_t n_nodes, int32_t vocab, const float *logits,
                                  const float *draft_probs, const int32_t *tokens, const int32_t *parent_dev,
                                  const float *temperature, const float *uniforms, const float *noise,
                                  int32_t *accept_len, int32_t *accept_node, int32_t *next_token,
                                  float *token_prob, void *workspace, size_t workspace_bytes,
                                  int32_t *dev_status, gdn_stream_t stream) {
    if (batch < 1 || batch > 65535 || n_nodes < 1 || n_nodes > kMaxNodes || vocab < 1 || vocab > kMaxVocab)
        return GDN_ERR_DIMS;
    if (!logits || !tokens || !uniforms || !noise || !accept_len || !accept_node || !next_token) return GDN_ERR_NULL;
    using gdnhost::aligned_to;
    for (const void *p : {(const void *)logits, (const void *)draft_probs, (const void *)tokens, (const void *)parent_dev,
                          (const void *)temperature, (const void *)uniforms, (const void *)noise, (const void *)accept_len,
                          (const void *)accept_node, (const void *)next_token, (const void *)token_prob,
                          (const void *)dev_status})
        if (!aligned_to(p, 4)) return GDN_ERR_ALIGN;
    if (!workspace || workspace_bytes < spec_accept_sample_workspace_bytes(batch, n_nodes) || !aligned_to(workspace, 256))
        return GDN_ERR_WORKSPACE;
    const int rows = batch * n_nodes;
    const Deal deal = deal_out(rows, vocab);
    Stat *stats = static_cast<Stat *>(workspace);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (gdndev::launch_pdl(sample_rows, dim3(deal.blocks), dim3(kThreads), 0, st, n_nodes, vocab, deal, logits, temperature,
                           noise, stats, rows, dev_status) != cudaSuccess)
        return GDN_ERR_CUDA;
    PickArgs a{n_nodes, vocab, deal, logits, draft_probs, tokens, parent_dev, temperature, uniforms, noise,
               accept_len, accept_node, next_token, token_prob, stats, dev_status};
    return gdndev::launch_pdl(sample_pick, dim3((unsigned)batch * kCluster), dim3(kPickThreads), 0, st, a) == cudaSuccess
               ? GDN_OK
               : GDN_ERR_CUDA;
}
