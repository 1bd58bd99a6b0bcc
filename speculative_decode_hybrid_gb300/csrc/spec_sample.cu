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
// needs neither a prefix sum nor r's normalisation, and whose result does not
// depend on the order of any sum.
//
// Two launches. sample_rows reads the logits once (all N rows: each drafted
// token's probability is an output): every CTA keeps a running maximum and sum
// of its chunk of a row. sample_pick is one cluster of CTAs per request: all
// of them repeat the walk, then each takes a slice of the accepted row (and of
// q and the noise), and the first CTA joins their candidates. The first launch
// is bound by the logits' bytes, the second by latency.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <initializer_list>

#include "gdn_device.cuh"
#include "gdn_host.h"
#include "gdnspec.h"

namespace {

using gdndev::Buf;
using gdndev::key_index;
using gdndev::make_key;
using gdndev::umax64;

constexpr int kThreads = 256;
constexpr int kPickThreads = 1024;
constexpr int kCluster = 8;
constexpr int kMaxSplits = 32;
constexpr int kMaxNodes = GDN_MAX_TOKENS + 1;
constexpr float kLog2e = 1.4426950408889634f;

// A row's maximum and the sum of exp((x - max) / T) (T == 0: the number of
// values equal to the maximum).
struct Stat {
    float m, s;
};

__device__ __forceinline__ float weight(float x, float m, float c) {
    return c > 0.f ? exp2f((x - m) * c) : (x == m ? 1.f : 0.f);
}

// c = log2(e) / T, or 0 for T == 0.
__device__ __forceinline__ float coefficient(const float *temperature, int b) {
    const float t = temperature ? temperature[b] : 1.f;
    return t > 0.f ? kLog2e / t : 0.f;
}

// Join two chunks' statistics. A chunk without a value above -inf has m = -inf
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
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < K; ++i) s += c > 0.f ? exp2f((x[i] - m) * c) : (x[i] == m ? 1.f : (x[i] == x[i] ? 0.f : x[i]));
    st.s += s;
}

__global__ void __launch_bounds__(kThreads)
sample_rows(int n_nodes, int vocab, int splits, int chunk, const float *__restrict__ logits,
            const float *__restrict__ temperature, Stat *__restrict__ stats, int32_t *dev_status) {
    __shared__ Stat warp_stat[kThreads / 32];
    const int row = blockIdx.y, split = blockIdx.x, tid = threadIdx.x;
    const size_t rows = gridDim.y;
    const Buf bl{logits, rows * (size_t)vocab * 4}, bs{stats, rows * (size_t)splits * sizeof(Stat)};
    gdndev::pdl_launch_dependents();
    gdndev::pdl_wait();
    const float c = coefficient(temperature, row / n_nodes);
    const float *r = logits + (size_t)row * vocab;
    const int lo = split * chunk, hi = min(vocab, lo + chunk);
    Stat st{-INFINITY, 0.f};
    // scalars up to the first 16-byte boundary, 16 bytes at a time, scalars again
    const int head = min(hi, lo + (int)((16 - ((reinterpret_cast<uintptr_t>(r + lo)) & 15)) & 15) / 4);
    const int body = max(0, hi - head) / 4, tail = head + body * 4;
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
    for (int e = tid; e < (head - lo) + (hi - tail); e += kThreads) {
        const int at = e < head - lo ? lo + e : tail + e - (head - lo);
        const float x[1] = {GDN_IN(r + at, 4, bl, dev_status) ? r[at] : 0.f};
        absorb(st, x, c);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        st = join(st, {__shfl_xor_sync(~0u, st.m, o), __shfl_xor_sync(~0u, st.s, o)}, c);
    if ((tid & 31) == 0) warp_stat[tid >> 5] = st;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w) st = join(st, warp_stat[w], c);
        Stat *to = stats + (size_t)row * splits + split;
        if (GDN_IN(to, sizeof(Stat), bs, dev_status)) *to = st;
    }
}

struct PickArgs {
    int n_nodes, vocab, splits;
    const float *logits, *draft;
    const int32_t *tokens, *parent;
    const float *temperature, *uniforms, *noise;
    int32_t *accept_len, *accept_node, *next_token;
    float *token_prob;
    const Stat *stats;
    int32_t *status;
};

template <typename T, typename Op>
__device__ __forceinline__ T cluster_reduce(T v, T *warp_buf, T *cta_buf, Op op) {
    namespace cg = cooperative_groups;
    cg::cluster_group cl = cg::this_cluster();
#pragma unroll
    for (int o = 16; o; o >>= 1) v = op(v, __shfl_xor_sync(~0u, v, o));
    if ((threadIdx.x & 31) == 0) warp_buf[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = warp_buf[threadIdx.x];
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

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPickThreads)
sample_pick(PickArgs a) {
    namespace cg = cooperative_groups;
    __shared__ float row_m[kMaxNodes], row_s[kMaxNodes];
    __shared__ float p_of[kMaxNodes], q_of[kMaxNodes], u_of[kMaxNodes];
    __shared__ int parent_of[kMaxNodes], token_of[kMaxNodes];
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
        bs{a.stats, B * N * (size_t)a.splits * sizeof(Stat)};
    // what no kernel before this one wrote could be read earlier, but who wrote
    // it is not known here
    gdndev::pdl_wait();
    const float c = coefficient(a.temperature, b);
    for (int n = warp; n < N; n += kPickThreads / 32) {
        Stat s{-INFINITY, 0.f};
        for (int k = lane; k < a.splits; k += 32) {
            const Stat *f = a.stats + ((size_t)b * N + n) * a.splits + k;
            if (GDN_IN(f, sizeof(Stat), bs, st)) s = join(s, *f, c);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) s = join(s, {__shfl_xor_sync(~0u, s.m, o), __shfl_xor_sync(~0u, s.s, o)}, c);
        if (lane == 0) {
            // a row with NaN, +inf or nothing above -inf has no distribution
            const bool none = s.m == -INFINITY || s.m == INFINITY || s.s != s.s;
            row_m[n] = s.m;
            row_s[n] = none ? __int_as_float(0x7fc00000) : s.s;
            if (none && rank == 0 && st) atomicOr(st, GDN_DEV_NAN_LOGIT);
        }
    }
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
    __syncthreads();
    if (tid < N) {
        const int p = parent_of[tid], t = token_of[tid];
        float pv = 0.f, qv = 0.f;
        bool dup = false, more = false;
        if (tid > 0 && p >= 0) {
            if (t >= 0) {
                const float *fl = a.logits + ((size_t)b * N + p) * V + t;
                const float x = GDN_IN(fl, 4, bl, st) ? *fl : 0.f;
                pv = weight(x, row_m[p], c) / row_s[p];
                if (a.draft) {
                    const float *fq = a.draft + ((size_t)b * (N - 1) + p) * V + t;
                    qv = GDN_IN(fq, 4, bq, st) ? *fq : 0.f;
                }
            }
            for (int j = 1; j < N; ++j)
                if (parent_of[j] == p) {
                    dup |= j < tid && token_of[j] == t;
                    more |= j > tid;
                }
        }
        p_of[tid] = pv;
        q_of[tid] = qv;
        gone_before[tid] = dup;
        more_after[tid] = more;
        if (a.token_prob && rank == 0 && tid > 0) a.token_prob[(size_t)b * N + tid] = pv;
    }
    __syncthreads();

    // the slice of a row that this CTA takes
    const int per = ((V + kCluster - 1) / kCluster + 3) & ~3;
    const int lo = min(V, rank * per), hi = min(V, lo + per);
    const float *noise = a.noise + (size_t)b * V;

    // the walk, the same in every thread of the cluster
    int node = 0, len = 0, flip = 0;
    float coef = 0.f, mass = 1.f, gone = 0.f;
    for (int i = 1; i < N; ++i) {
        if (parent_of[i] != node) continue;
        const bool usable = token_of[i] >= 0 && row_s[node] == row_s[node];
        bool ok;
        if (a.draft)
            ok = usable && u_of[i] * q_of[i] * mass < fmaxf(p_of[i] - coef * q_of[i], 0.f);
        else
            ok = usable && !gone_before[i] && u_of[i] * (1.f - gone) < p_of[i];
        if (ok) {
            node = i;
            ++len;
            coef = 0.f, mass = 1.f, gone = 0.f;
            continue;
        }
        if (!a.draft) {
            if (!gone_before[i]) gone += p_of[i];
            continue;
        }
        coef += mass;
        if (more_after[i] && row_s[node] == row_s[node]) {
            const float *l = a.logits + ((size_t)b * N + node) * V, *q = a.draft + ((size_t)b * (N - 1) + node) * V;
            const float m = row_m[node], inv = 1.f / row_s[node];
            float s = 0.f;
            for (int v = lo + tid; v < hi; v += kPickThreads)
                if (GDN_IN(l + v, 4, bl, st) && GDN_IN(q + v, 4, bq, st))
                    s += fmaxf(weight(l[v], m, c) * inv - coef * q[v], 0.f);
            mass = cluster_reduce(s, sum_warp, sum_cta[flip], [](float x, float y) { return x + y; });
            flip ^= 1;
        }
    }

    // the next token: the largest rest / noise of the accepted row; the largest
    // p / noise beside it, in case the rest is zero everywhere
    const float m = row_m[node], inv = 1.f / row_s[node];
    const bool defined = row_s[node] == row_s[node];
    const bool use_q = a.draft && coef > 0.f;
    unsigned long long best = 0ull, best_p = 0ull;
    if (defined) {
        const float *l = a.logits + ((size_t)b * N + node) * V;
        const float *q = use_q ? a.draft + ((size_t)b * (N - 1) + node) * V : nullptr;
        float top = -1.f, top_p = -1.f;
        int at = 0, at_p = 0;
        for (int v = lo + tid; v < hi; v += kPickThreads) {
            if (!GDN_IN(l + v, 4, bl, st) || !GDN_IN(noise + v, 4, bn, st)) continue;
            const float p = weight(l[v], m, c) * inv, e = noise[v];
            float w = p;
            if (use_q) {
                if (GDN_IN(q + v, 4, bq, st)) w = fmaxf(p - coef * q[v], 0.f);
            } else if (!a.draft && gone > 0.f && p > 0.f) {
                for (int j = 1; j < N; ++j)
                    if (parent_of[j] == node && token_of[j] == v) w = 0.f;
            }
            const float f = w > 0.f ? w / e : 0.f, g = p > 0.f ? p / e : 0.f;
            if (f > top) top = f, at = v;
            if (g > top_p) top_p = g, at_p = v;
        }
        if (top > 0.f) best = make_key(top, (unsigned)at);
        if (top_p > 0.f) best_p = make_key(top_p, (unsigned)at_p);
    }
    best = cluster_reduce(best, key_warp, key_cta[0], [](unsigned long long x, unsigned long long y) { return umax64(x, y); });
    __syncthreads();
    if (best == 0ull)
        best = cluster_reduce(best_p, key_warp, key_cta[1], [](unsigned long long x, unsigned long long y) { return umax64(x, y); });
    if (rank == 0 && tid == 0) {
        const int next = best ? (int)key_index(best) : 0;
        a.accept_len[b] = len;
        a.accept_node[b] = node;
        a.next_token[b] = next;
        if (a.token_prob) {
            const float *f = a.logits + ((size_t)b * N + node) * V + next;
            a.token_prob[(size_t)b * N] = GDN_IN(f, 4, bl, st) ? weight(*f, m, c) / row_s[node] : 0.f;
        }
    }
    cl.sync();  // no CTA leaves while another may still write into its shared memory
}

int row_splits(int rows, int vocab) {
    const int sms = gdnhost::sm_count();
    const int target = 8 * (sms > 0 ? sms : 152);
    int s = (target + rows - 1) / rows;
    const int by_size = (vocab + 4095) / 4096;
    if (s > by_size) s = by_size;
    if (s > kMaxSplits) s = kMaxSplits;
    return s < 1 ? 1 : s;
}

}  // namespace

extern "C" size_t spec_accept_sample_workspace_bytes(int32_t batch, int32_t n_nodes) {
    if (batch < 1 || batch > 65535 || n_nodes < 1 || n_nodes > kMaxNodes) return 0;
    return (size_t)batch * n_nodes * kMaxSplits * sizeof(Stat);
}

extern "C" int spec_accept_sample(int32_t batch, int32_t n_nodes, int32_t vocab, const float *logits,
                                  const float *draft_probs, const int32_t *tokens, const int32_t *parent_dev,
                                  const float *temperature, const float *uniforms, const float *noise,
                                  int32_t *accept_len, int32_t *accept_node, int32_t *next_token,
                                  float *token_prob, void *workspace, size_t workspace_bytes,
                                  int32_t *dev_status, gdn_stream_t stream) {
    if (batch < 1 || batch > 65535 || n_nodes < 1 || n_nodes > kMaxNodes || vocab < 1) return GDN_ERR_DIMS;
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
    const int splits = row_splits(rows, vocab);
    const int chunk = ((vocab + splits - 1) / splits + 3) & ~3;
    Stat *stats = static_cast<Stat *>(workspace);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // rows go to gridDim.y, at most 65535 of them a launch
    const int per_launch = 65535 / n_nodes * n_nodes;
    for (int r0 = 0; r0 < rows; r0 += per_launch) {
        const int n = rows - r0 < per_launch ? rows - r0 : per_launch;
        if (gdndev::launch_pdl(sample_rows, dim3(splits, n), dim3(kThreads), 0, st, n_nodes, vocab, splits, chunk,
                               logits + (size_t)r0 * vocab, temperature ? temperature + r0 / n_nodes : temperature,
                               stats + (size_t)r0 * splits, dev_status) != cudaSuccess)
            return GDN_ERR_CUDA;
    }
    PickArgs a{n_nodes, vocab, splits, logits, draft_probs, tokens, parent_dev, temperature, uniforms, noise,
               accept_len, accept_node, next_token, token_prob, stats, dev_status};
    return gdndev::launch_pdl(sample_pick, dim3((unsigned)batch * kCluster), dim3(kPickThreads), 0, st, a) == cudaSuccess
               ? GDN_OK
               : GDN_ERR_CUDA;
}
