// Attention with changed scores, and over shared prefixes, on the tensor cores
// (attn_*_ex and attn_*_shared with GDN_BF16).
//
// The tiles, warps and softmax are those of attn_tc.cu; what differs:
//
// Scores. x = q k becomes, in powers of two, y = c - 2 c / (1 + 2^(x cap_in)) with
// a cap (c tanh(scale x / cap), by one exponential and one reciprocal, off by
// some 2^-20 c; caps above 128: cap_far), scale x without; a bias by distance adds
// slope (slot - r), with r the node's position, or for a slope below 0 the first slot
// that the row sees: a row's constant does not matter, and so the bias is small where
// the weight lies (from slot 0 it would have lost whole units 8 million slots in). A
// segment's tiles are taken from the last to the first, so that a bias for the near does
// not raise the maximum tile by tile. Slots before a window or a document are whole
// tiles left out, and masked in the tiles where they end; V is zeroed where no row sees
// it, and what is no number there is kept for the rows that do, as attn_tc.cu does for
// the drafted nodes.
//
// Shared prefixes. The list of work has an entry for every group of requests that
// shares its first slots, with the rows of all its members against those slots,
// and one for every request's own slots. The rows of a head's product are then
// members x nodes x query heads of the group, so that a tile read once serves all
// members. A row of a member has two parts at least: what a block has of an entry
// in full goes to a buffer with a place for each row, what it shares with other
// blocks to the blocks' pieces, and join_rows adds them up on the scale of their
// largest maximum.
//
// Weights are rounded to bf16 once for the second product, not in the divisor, as in
// attn_tc.cu, where the form in two parts and its price stand: a result is 1.8e-3 to 2.3e-3
// of its norm from the 64-bit one, of which the rounding of the result itself is 1.7e-3.
//
// Two threads a row, each with half of a tile's columns: 8 softmax warps hide more of
// each other's waits than 4, and leave registers for what changes the scores. Where the
// time goes, in cycles of a 128 x 128 x 128 tile: wait for the scores 240, their loads
// 130, maximum 160, exchange of it 110, weights 700, the reference settled 450, weights
// stored and handed over 340, of 2,300; its products take 1,024. Measured and dropped:
// tiles in turn (below), maxima exchanged by named barriers (340 cycles
// less for a softmax warp, and the scores of the next tile are waited for instead:
// 243 us instead of 246 for 2 x 8 trees, 39 instead of 37 for 22 nodes with a cap),
// weights apart from scores in tensor memory, so that scores are made earlier (246 us).
//
// Measured: 22 nodes, 256 wide, over 32,501 slots with a cap 37 us (32 us by the plain
// kernel without; the bytes 10), bound by tile latency, start and join; 16 spans of 16
// that see 4,096 of up to 16,000 slots, with a bias, 66 us, 4.1 TB/s; over up to 8,000
// slots 80 us with a bias and 89 with a cap (73 by the plain kernel), by the softmax
// warps' work: a cap is another exponential and a quarter of a reciprocal a score.
// Shared: 8 samples' tokens over 32,000 shared slots, 256 wide, 34 us a layer (66 each
// for itself; the bytes 10), 2 x 8 trees of 22 nodes over 16,000 and 12,000 slots 119 to
// 123 us (each for itself 134 by this kernel and 115 by the plain one; the products 43):
// tensor pipes 35 % busy, by the waits between a tile's scores, weights and sums, and 128
// short segments of some 11 us each. Prefixes that fit in L2 are read from there by the
// calls that do not share: 8 single tokens, 128 wide, break even at some 10,000 slots.
// Spills: none with changed scores; 30 to 34 bytes without at 64 and 128 wide, 100 in
// join_rows (64 registers, four blocks an SM).
#include <cuda.h>
#include <cuda_runtime.h>

#include "attn_ex.cuh"
#include "attn_ex_host.h"
#include "attn_tc.cuh"
#include "gdn_host.h"
#include "gdnspec.h"

namespace {

using gdnattn::AttnArgs;
using gdnattn::ExArgs;
using gdndev::add2;
using gdndev::Buf;
using gdndev::fma2;
using namespace gdnattn::tc;

constexpr int kM = 128;         // rows of an M tile
constexpr int kSoftWarps = 8;   // two threads a row, each with half of a tile's columns
constexpr int kTmemCols = 512;  // all of an SM's: one block per SM
constexpr int kNotes = 2 * kMaxBlocks / 32;

template <int D>
struct Shape {
    static constexpr int kN = D == 256 ? 64 : 128;       // slots of a tile
    static constexpr int kChunks = D / 64;               // 128-byte column chunks of a row
    static constexpr unsigned kSCol = D, kQCol = kSCol + 2 * kN;  // tensor-memory columns: O, S twice, Q
    static constexpr int kStages = D == 64 ? 6 : 3;
    static constexpr unsigned kTileBytes = kN * D * 2;   // of K, and of V
    static constexpr unsigned kPassBytes = kSoftWarps * 2048;  // a warp's 16 rows x 128 bytes of Q on their way
    static constexpr int kThreads = kSoftWarps * 32 + 96;
    static constexpr unsigned kSmem = 2 * kStages * kTileBytes + kPassBytes + 1024;
    static_assert(kQCol + D / 2 <= kTmemCols, "tensor memory");
    static_assert(gdnattn::kShareUnit % kN == 0, "a shared prefix is whole tiles");
};

struct Plan {
    int group, rows;        // query heads of a key/value head; rows of one key/value head of a request
    int m_groups, units;    // groups of P M tiles of a head; units (head, group) of a request
    int shared_units;       // of a group of requests, at most
    int blocks;             // groups of P blocks, each group on a share of its own
    int rows_pad;           // rows, a multiple of 32
    unsigned by_group, by_m_groups, by_blocks;  // 2^32 / n rounded up: x / n for x * n < 2^32
    unsigned long long by_blocks64;             // 2^64 / n rounded up: x / n for x * n < 2^64
};

// An entry of the list of work: a group's shared slots, or a request's own. Its
// units are h_kv heads of m_groups groups of M tiles. A unit counts kStart tiles more
// than it has, in front: what a block does before its first and after its last
// tile (queries, results), so that many short requests are spread over the blocks.
constexpr int kStart = 8;

struct Entry {
    int tiles, m_groups;
    gdnattn::Range range;  // of a request; a group: its slots
    int b, first, count;   // the request whose table row is read; of a group: where its members are, how many
    __device__ __forceinline__ int unit_cost() const { return tiles + kStart; }
};
template <int kN, int P>
__device__ __forceinline__ Entry request_entry(const AttnArgs &a, const ExArgs &x, const Plan &plan, int b) {
    Entry n{0, plan.m_groups, gdnattn::range_of(a, x, b), b, 0, 0};
    n.tiles = n.range.slots ? (n.range.slots - (n.range.lo & ~(kN - 1)) + kN - 1) / kN : 0;
    return n;
}
template <int kN, int P>
__device__ __forceinline__ Entry group_entry(const AttnArgs &a, const ExArgs &x, const Plan &plan, int e) {
    const gdnattn::Group g = gdnattn::group_at(a, x, e);
    return {g.count ? g.len / kN : 0, (int)(((unsigned)g.count * (unsigned)plan.rows + P * kM - 1) / (P * kM)), {g.len, 0, 0}, g.lead, g.first,
            g.count};
}

// The list of work: groups, then requests. In shared memory where it is short,
// since every role goes through it for every segment, and global memory is far.
constexpr int kKept = 64;

struct Table {
    // (the kernel's arguments once more: a function that is not inlined would read
    // its references to them from far away)
    AttnArgs a;
    ExArgs x;
    Plan plan;
    int groups;
    Entry group[kKept / 2], request[kKept];
    unsigned short order[kKept];
};

// Fills the table, by a block's threads; complete after the next barrier.
template <int kN, int P>
__device__ __forceinline__ void fill(Table &t, const AttnArgs &a, const ExArgs &x, const Plan &plan, int tid) {
    if (tid == 160) t.a = a, t.x = x, t.plan = plan;
    if (tid == 0) t.groups = gdnattn::groups_of(a, x);
    if (a.batch > kKept) return;
    if (tid < a.batch) t.request[tid] = request_entry<kN, P>(a, x, plan, tid);
    if (!x.plan) return;
    const int g = tid - 64, m = tid - 96;
    if (g >= 0 && g < a.batch / 2) t.group[g] = group_entry<kN, P>(a, x, plan, g);  // (beyond the last group: not used)
    if (m >= 0 && m < a.batch) t.order[m] = (unsigned short)gdnattn::member_at(a, x, m);
}
template <int kN, int P>
__device__ __noinline__ Entry far_entry(const Table &t, int e) {
    return e < t.groups ? group_entry<kN, P>(t.a, t.x, t.plan, e) : request_entry<kN, P>(t.a, t.x, t.plan, e - t.groups);
}
template <int kN, int P>
__device__ __forceinline__ Entry entry_at(const Table &t, int e) {
    if (t.a.batch > kKept) return far_entry<kN, P>(t, e);
    return e < t.groups ? t.group[e] : t.request[e - t.groups];
}
__device__ __forceinline__ int member_of(const Table &t, const AttnArgs &a, const ExArgs &x, int i) {
    return a.batch <= kKept ? t.order[min(i, kKept - 1)] : gdnattn::member_at(a, x, i);
}

struct Work {
    int e, off, left;  // entry, what of it has been dealt out, what is still to come for this block
};

struct Segment {
    int e, tile0, n, tiles, kv, m, m_groups;  // m: group of M tiles
    bool shared;
    int b, first, count;                      // as an Entry's
    int base;                                 // slot of tile 0
    gdnattn::Range range;
};

// n 0: there is none left. Not inlined: every role calls it, and a block's segments
// run through code that the tiles have pushed out of the instruction cache.
template <int kN, int P>
__device__ __noinline__ void next_segment(const Table &t, Work &w, Segment &s) {
    const AttnArgs &a = t.a;
    const Plan &plan = t.plan;
    s.n = 0;
    while (w.left > 0) {
        const Entry n = entry_at<kN, P>(t, w.e);
        if (n.tiles == 0) {
            if (++w.e >= t.groups + a.batch) break;
            continue;
        }
        const int cost = n.unit_cost(), unit = w.off / cost, from = w.off - unit * cost, len = min(cost - from, w.left);
        s.e = w.e;
        w.off += len;
        w.left -= len;
        if (w.off == cost * n.m_groups * a.h_kv) ++w.e, w.off = 0;
        s.tile0 = max(0, from - kStart);
        s.n = max(0, from + len - kStart) - s.tile0;
        if (s.n == 0) continue;
        s.tiles = n.tiles;
        s.shared = s.e < t.groups;
        s.m_groups = n.m_groups;
        s.kv = s.shared ? unit / n.m_groups : quotient(unit, plan.by_m_groups);
        s.m = unit - s.kv * n.m_groups;
        s.range = n.range;
        s.b = n.b, s.first = n.first, s.count = n.count;
        s.base = s.shared ? 0 : n.range.lo & ~(kN - 1);
        break;
    }
}

// Block `block`'s share, which begins at total * block / blocks, rounded down, and the
// entry in which it begins. By one warp.
template <int kN, int P>
__device__ __forceinline__ Work block_work(const Table &t, int block, bool flag) {
    const AttnArgs &a = t.a;
    const Plan &plan = t.plan;
    const int lane = threadIdx.x & 31, entries = t.groups + a.batch;
    auto cost_of = [&](int e) -> long long {
        if (e >= entries) return 0;
        const Entry n = entry_at<kN, P>(t, e);
        return n.tiles ? (long long)n.unit_cost() * n.m_groups * a.h_kv : 0;
    };
    const long long mine = cost_of(lane);
    long long total = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < entries; e0 += 32) {
        long long n = e0 ? cost_of(e0 + lane) : mine;
#pragma unroll
        for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(~0u, n, o);
        total += n;
    }
    const long long whole = plan.blocks > 1 ? (long long)__umul64hi((unsigned long long)total, plan.by_blocks64) : total;
    const int rest = (int)(total - whole * plan.blocks);
    const long long lo = whole * block + quotient(rest * block, plan.by_blocks), hi = whole * (block + 1) + quotient(rest * (block + 1), plan.by_blocks);
    Work w{0, 0, 0};
    long long before = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < entries && (lo >= before || flag); e0 += 32) {
        const int e = e0 + lane;
        const long long n = e0 ? cost_of(e) : mine;
        long long s = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(~0u, s, o);
            if (lane >= o) s += y;
        }
        const long long first = before + s - n;
        const unsigned here = __ballot_sync(~0u, lo >= first && lo < first + n);
        if (here) {
            const int from = __ffs(here) - 1;
            w = {e0 + from, (int)(lo - __shfl_sync(~0u, first, from)), (int)(hi - lo)};
        }
        if (flag && a.status && e >= t.groups && e < entries && n == 0) atomicOr(a.status, GDN_DEV_LENGTH);
        before += __shfl_sync(~0u, s, 31);
    }
    return w;
}

// The smaller, NaN if one is.
__device__ __forceinline__ float min_nan(float x, float y) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

// What changes the scores: nothing; a cap up to kMostOfNear or a bias; a cap above it (and
// a bias).
enum Scores { kPlain, kNear, kFar };

// The form of one exponential, c - 2 c / (1 + e), is a difference of two numbers as large as
// the cap, off by 2^-20 of it whatever the score: at 128 (in powers of two here) a sixteenth
// of the half step of a bf16 weight. For larger caps a score below a quarter of the cap is
// z (1 - u^2 / 3 + 2 u^4 / 15 - ...), u = z / c, its next term 10^-8; one that is not loses
// 2^-18 of itself. A kernel of its own for them: as a branch it cost the others registers
// (248 bytes of spills; 16 spans of 16 over up to 8,000 slots with a cap of 50 107 us
// instead of 89). Those spans with a cap of 200 take 104 us, 89 by the near form.
constexpr float kMostOfNear = 128.f * gdnattn::kLog2e;

template <int K>
__device__ __forceinline__ void cap_far(const ExArgs &ex, unsigned (&x)[K][32], float scale_log2) {
    const float half = ex.cap_in * 0.34657359f;  // ln 2 / 2
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 32; i += 2) top = max3(top, fabsf(__uint_as_float(x[k][i])), fabsf(__uint_as_float(x[k][i + 1])));
    auto series = [&](float s) {
        const float u = s * half, u2 = u * u;
        return s * scale_log2 * fmaf(u2, fmaf(u2, fmaf(u2, fmaf(u2, 62.f / 2835, -17.f / 315), 2.f / 15), -1.f / 3), 1.f);
    };
    if (__all_sync(~0u, top * half <= 0.25f)) {  // (a NaN is one in either form)
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 32; ++i) x[k][i] = __float_as_uint(series(__uint_as_float(x[k][i])));
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float s = __uint_as_float(x[k][i]);
                float r;
                asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(min_nan(s * ex.cap_in, 30.f))));
                x[k][i] = __float_as_uint(fabsf(s) * half <= 0.25f ? series(s) : fmaf(r, -2.f * ex.cap, ex.cap));
            }
    }
}

// Scores as they are changed: the cap, then the bias. at: the first one's slot less the
// row's reference. Four scores share a reciprocal: no NaN that is not seen may be among
// them.
template <Scores kScores, int K>
__device__ __forceinline__ void change(const ExArgs &ex, unsigned (&x)[K][32], int at, float slope, float scale_log2) {
    if (kScores == kFar) {
        cap_far(ex, x, scale_log2);
    } else if (ex.cap > 0.f) {
        const float c2 = -2.f * ex.cap;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                float e[4], r;
#pragma unroll
                for (int u = 0; u < 4; ++u)  // 2^30: 1 to the last bit of the cap
                    e[u] = 1.f + ex2(min_nan(__uint_as_float(x[k][i + u]) * ex.cap_in, 30.f));
                const float p = e[0] * e[1], q = e[2] * e[3];
                asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(p * q));
                const float rp = r * q * c2, rq = r * p * c2;
                x[k][i] = __float_as_uint(fmaf(rp, e[1], ex.cap));
                x[k][i + 1] = __float_as_uint(fmaf(rp, e[0], ex.cap));
                x[k][i + 2] = __float_as_uint(fmaf(rq, e[3], ex.cap));
                x[k][i + 3] = __float_as_uint(fmaf(rq, e[2], ex.cap));
            }
    }
    if (ex.slopes) {
        const float at0 = (float)at * slope, by = ex.cap > 0.f ? 1.f : scale_log2;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 32; ++i) x[k][i] = __float_as_uint(fmaf(__uint_as_float(x[k][i]), by, fmaf((float)(k * 32 + i), slope, at0)));
    }
}

// The bias of a tree's drafted nodes among 32 slots, the first `rel` past ctx: a node's
// place is its depth's, not its slot's, and the r-th on the path stands r - 1 past ctx.
__device__ __forceinline__ void place_nodes(unsigned (&x)[32], int rel, float slope, const gdnattn::NodePath &path) {
    if (rel >= 64 || rel <= -32) return;
    const unsigned bits = rel >= 0 ? (unsigned)(path.bits >> rel) : (unsigned)path.bits << -rel;
    int before = (rel > 0 ? __popcll(path.bits & ((1ull << rel) - 1)) : 0) + path.skipped - 1 - rel;
#pragma unroll
    for (int i = 0; i < 32; ++i, --before)
        if (bits >> i & 1) x[i] = __float_as_uint(fmaf((float)++before, slope, __uint_as_float(x[i])));
}

struct Pieces {
    float4 *o;    // [2 blocks][D / 4][P * 128]: of entries that blocks share
    float2 *ms;   // [2 blocks][P * 128]: reference maximum in powers of two, sum
    int *unit;    // [2 blocks]: number of the unit of a block's first and last piece of a shared one, -1 for none
    float4 *row_o[2];   // members' own slots, their groups': [B * h_kv][D / 4][rows_pad]
    float2 *row_ms[2];  // [B * h_kv][rows_pad]
};

__device__ __forceinline__ int unit_number(const AttnArgs &a, const Plan &plan, int m_groups, bool shared, int at, int kv, int m) {
    return shared ? a.batch * plan.units + at * plan.shared_units + kv * m_groups + m : at * plan.units + kv * m_groups + m;
}

template <int D>
struct Control {
    static constexpr int kStages = Shape<D>::kStages;
    unsigned long long k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
    unsigned long long s_full[2], p_full[2], pv_done[2], q_full, drain[2];
    unsigned long long pair[4];        // by 32 rows: maxima and sums are exchanged
    float top_of[2][2][kM], sum_of[2][kM];
    Table table;
    Work work;
    unsigned long long odd_nodes[4], odd_low[4];  // drafted nodes, and slots from range.lo on, with a value of v that is no number, by segment
    unsigned tmem;
    int quit;
};

// What is no number among the values of slots that a row sees and that were zeroed in
// shared memory (bit i of a set: slot i past its first) added to columns [k0, k1) of
// what has been written for the row: a part in f32, its 16 bytes `step` apart, or the
// result.
template <int D>
__device__ __noinline__ void restore(const Table &t, float4 *part, int step, __nv_bfloat16 *result, int k0, int k1, int b, int kv,
                                     unsigned long long set0, int first0, unsigned long long set1, int first1) {
    const AttnArgs &a = t.a;
    const Buf bt{a.table, (size_t)a.batch * a.width * 4}, bv{a.v_pages, ((size_t)a.n_pages * a.h_kv << a.page_shift) * D * 2};
    while (set0 | set1) {
        if (!set0) set0 = set1, set1 = 0, first0 = first1;
        const int at = first0 + __ffsll((long long)set0) - 1;
        set0 &= set0 - 1;
        const int32_t *e = a.table + (size_t)b * a.width + (at >> a.page_shift);
        const int page = GDN_IN(e, 4, bt, a.status) ? *e : -1;
        if (page < 0 || page >= a.n_pages) continue;
        const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v_pages) +
                                 ((((size_t)page * a.h_kv + kv) << a.page_shift) + (at & ((1 << a.page_shift) - 1))) * D;
#pragma unroll 1
        for (int k = k0; k < k1; ++k) {
            const float x = GDN_IN(v + k, 2, bv, a.status) ? __bfloat162float(v[k]) : 0.f;
            if (fabsf(x) < INFINITY) continue;
            if (result)
                result[k] = __float2bfloat16(__bfloat162float(result[k]) + x);
            else
                reinterpret_cast<float *>(part + (size_t)(k / 4) * step)[k % 4] += x;
        }
    }
}

// With a cap or a bias a kernel of its own: the code of both is longer than
// all the rest of a tile's.
template <int D, int P, Scores kScores>
__global__ void __launch_bounds__(Shape<D>::kThreads, 1)
attend_ex(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
          const __grid_constant__ AttnArgs a, const __grid_constant__ ExArgs ex, const __grid_constant__ Plan plan,
          const __grid_constant__ Pieces pieces) {
    using S = Shape<D>;
    constexpr int kN = S::kN, kStages = S::kStages;
    constexpr bool kChanged = kScores != kPlain;
    extern __shared__ char raw[];
    __shared__ Control<D> c;
    char *base = raw + ((1024 - (saddr(raw) & 1023)) & 1023);
    const unsigned k_s = saddr(base), v_s = k_s + kStages * S::kTileBytes, pass_s = v_s + kStages * S::kTileBytes;
    const int share = blockIdx.x / P, rank = blockIdx.x % P;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int32_t *st = a.status;
    constexpr int kTmaWarp = kSoftWarps, kScoreWarp = kTmaWarp + 1, kSumWarp = kTmaWarp + 2;

    if (warp == kTmaWarp && lane < 2)
        asm volatile("prefetch.tensormap [%0];" ::"l"(lane ? &v_map : &k_map) : "memory");
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            bar_init(saddr(&c.k_full[i]), 1);
            bar_init(saddr(&c.k_empty[i]), 1);
            bar_init(saddr(&c.v_full[i]), 1);
            bar_init(saddr(&c.v_empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(saddr(&c.s_full[i]), 1);
            bar_init(saddr(&c.p_full[i]), kSoftWarps);  // one arrival per softmax warp
            bar_init(saddr(&c.pv_done[i]), 1);
        }
        bar_init(saddr(&c.q_full), kSoftWarps);
        for (int i = 0; i < 4; ++i) bar_init(saddr(&c.pair[i]), 2);
        bar_init(saddr(&c.drain[0]), 1);
        bar_init(saddr(&c.drain[1]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");  // for the TMA unit
        c.quit = 0;
        for (int i = 0; i < 4; ++i) c.odd_nodes[i] = c.odd_low[i] = 0;
    }
    gdndev::pdl_launch_dependents();  // join_rows, which takes no tensor memory
    gdndev::pdl_wait();
    // All of the SM's columns, and only once nothing is waited for outside of this
    // block: the kernel before may be anybody's, and may need columns itself.
    if (warp == kScoreWarp) gdntc::tmem_alloc<kTmemCols>(&c.tmem);
    fill<kN, P>(c.table, a, ex, plan, tid);
    gdntc::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        const Work w = block_work<kN, P>(c.table, share, blockIdx.x == 0);
        if (lane == 0) c.work = w;
    }
    __syncthreads();
    gdntc::fence_after_sync();
    Work work = c.work;
    const unsigned tmem = c.tmem;
    if (tid == 0 && rank == 0) pieces.unit[2 * share] = pieces.unit[2 * share + 1] = -1;
    volatile int *quit = &c.quit;
    constexpr unsigned kSCol = S::kSCol, kQCol = S::kQCol;

    if (warp == kTmaWarp) {
        int g = 0;  // tiles so far
        const int page_rows = min(1 << a.page_shift, kN), boxes = kN / page_rows;
        const unsigned box_bytes = page_rows * 128u;
        const int mine = lane / S::kChunks, chunk = lane % S::kChunks;  // this lane's page of the tile, and its column chunk
        const Buf bt{a.table, (size_t)a.batch * a.width * 4};
        bool ok = true;
        while (work.left > 0 && ok) {
            Segment s;
            next_segment<kN, P>(c.table, work, s);
            if (s.n == 0) break;
            const int32_t *row = a.table + (size_t)s.b * a.width;
            const int slots = s.range.slots, low = s.range.lo;
            // boxes without a slot that a row sees are not loaded: their table entries may be anything
            auto wanted = [&](int slot) { return mine < boxes && slot < slots && slot + page_rows > low; };
            auto entry = [&](int slot) {
                const int32_t *f = row + (slot >> a.page_shift);
                return wanted(slot) && GDN_IN(f, 4, bt, st) ? *f : 0;
            };
            int slot = s.base + (s.tile0 + s.n - 1) * kN + mine * page_rows;
            int page = entry(slot);  // a page id is read one tile ahead
            for (int j = 0; j < s.n; ++j, ++g, slot -= kN) {
                const bool used = wanted(slot);
                const bool known = page >= 0 && page < a.n_pages;
                if (used && !known && st && chunk == 0) atomicOr(st, GDN_DEV_PAGE);
                // a page outside the pool lies outside the tensor map, which reads as zeros
                const int z = known ? page * a.h_kv + s.kv : -1, y = slot & ((1 << a.page_shift) - 1);
                const unsigned bytes = __popc(__ballot_sync(~0u, used)) * box_bytes;
                const int next = j + 1 < s.n ? entry(slot - kN) : 0;
                const int stage = g % kStages;
                const unsigned phase = (g / kStages) & 1;
                const unsigned at = stage * S::kTileBytes + (unsigned)chunk * (kN * 128u) + (unsigned)mine * box_bytes;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const unsigned full = saddr(half ? &c.v_full[stage] : &c.k_full[stage]);
                    ok = ok && wait(saddr(half ? &c.v_empty[stage] : &c.k_empty[stage]), phase ^ 1, quit);
                    ok = __all_sync(~0u, ok);
                    if (!ok) break;
                    if (lane == 0) bar_expect(full, bytes);
                    __syncwarp();
                    if (used) load_box((half ? v_s : k_s) + at, half ? &v_map : &k_map, chunk * 64, y, z, full);
                }
                if (!ok) break;
                page = next;
            }
        }
        if (!ok) {
            // copies in flight still write shared memory: wait for the last of each stage
            for (int i = 0; i < kStages; ++i) {
                const int last = g - 1 - ((g - 1 - i) % kStages + kStages) % kStages;  // last tile that used stage i
                if (last >= 0) {
                    wait(saddr(&c.k_full[i]), (last / kStages) & 1, nullptr);
                    wait(saddr(&c.v_full[i]), (last / kStages) & 1, nullptr);
                }
            }
        }
    } else if (warp == kScoreWarp) {
        // S = Q K^T. The sums have a warp of their own: each waits for its inputs
        // while the other's products run.
        if (lane == 0) {
            constexpr unsigned kIdS = gdntc::idesc_bf16(kM, kN, false);
            int g = 0;
            unsigned seg = 0;
            bool ok = true;
            while (work.left > 0 && ok) {
                Segment s;
                next_segment<kN, P>(c.table, work, s);
                if (s.n == 0) break;
                ok = wait(saddr(&c.q_full), seg & 1, quit);
                ++seg;
                gdntc::fence_after_sync();
                for (int j = 0; j < s.n && ok; ++j, ++g) {
                    const int stage = g % kStages;
                    const unsigned k = k_s + stage * S::kTileBytes;
                    ok = wait(saddr(&c.k_full[stage]), (g / kStages) & 1, quit);
                    // the weights that lay in this S buffer have been used
                    const int slot = g & 1;
                    if (g >= 2) ok = ok && wait(saddr(&c.pv_done[slot]), ((g - 2) >> 1) & 1, quit);
                    if (!ok) break;
                    gdntc::fence_after_sync();
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
                        gdntc::mma_bf16_ts(tmem + kSCol + slot * kN, tmem + kQCol + i * 8,
                                           gdntc::smem_desc_sw128(k + (i / 4) * (kN * 128) + (i % 4) * 32), kIdS, i > 0);
                    gdntc::mma_commit(saddr(&c.s_full[slot]));
                    gdntc::mma_commit(saddr(&c.k_empty[stage]));
                }
            }
            gdntc::mma_commit(saddr(&c.drain[0]));
            wait(saddr(&c.drain[0]), 0, nullptr);  // no product may run on when the columns are freed
        }
        __syncwarp();
    } else if (warp == kSumWarp) {
        // O += P V
        if (lane == 0) {
            constexpr unsigned kIdO = gdntc::idesc_bf16(kM, D, true);
            int g = 0;
            bool ok = true;
            while (work.left > 0 && ok) {
                Segment s;
                next_segment<kN, P>(c.table, work, s);
                if (s.n == 0) break;
                for (int j = 0; j < s.n && ok; ++j, ++g) {
                    const int stage = g % kStages;
                    const unsigned v = v_s + stage * S::kTileBytes;
                    ok = wait(saddr(&c.v_full[stage]), (g / kStages) & 1, quit);
                    const int slot = g & 1;
                    ok = ok && wait(saddr(&c.p_full[slot]), (g >> 1) & 1, quit);
                    if (!ok) break;
                    gdntc::fence_after_sync();
#pragma unroll
                    for (int i = 0; i < kN / 16; ++i)
                        gdntc::mma_bf16_ts(tmem, tmem + kSCol + slot * kN + i * 8, gdntc::smem_desc_sw128_mn(v + i * 2048, kN * 128),
                                           kIdO, j > 0 || i > 0);
                    gdntc::mma_commit(saddr(&c.pv_done[slot]));
                    gdntc::mma_commit(saddr(&c.v_empty[stage]));
                }
            }
            gdntc::mma_commit(saddr(&c.drain[1]));
            wait(saddr(&c.drain[1]), 0, nullptr);
        }
        __syncwarp();
    } else {
        // Warps w and w + 4 have the same 32 rows, the first half of a tile's columns and
        // the second. (Tiles in turn take longer, 289 us instead of 264 for 2 x 8 trees of 22
        // nodes over 16,000 shared slots: scores, weights and sums of a tile follow one
        // another, and there is room for two tiles' scores only.)
        const int rows_warp = warp & 3, half = warp >> 2, my_row = rows_warp * 32 + lane;
        const unsigned lane_addr = (unsigned)rows_warp << 21;  // 32 lanes each, in bits 16 and up
        unsigned exchanges = 0;
        auto exchanged = [&]() { return wait(saddr(&c.pair[rows_warp]), exchanges++ & 1, quit); };  // the other warp has arrived, too
        const Buf bq{a.q, (size_t)a.batch * a.n_tok * a.h_q * D * 2}, bout{a.out, (size_t)a.batch * a.n_tok * a.h_q * D * 2},
            bpar{a.parent, (size_t)a.batch * (a.n_tok + 1) * 4};
        const float scale = kChanged ? 1.f : a.scale_log2;  // changed scores are in powers of two before the softmax
        // The scores of tile g are issued before the sums of g - 1, so a tile's scores
        // only tell that the sums of g - 2 are done: a barrier for each S buffer
        // keeps its phases apart.
        auto sums_done = [&](int tile) { return wait(saddr(&c.pv_done[tile & 1]), (tile >> 1) & 1, quit); };
        // row r of a segment's product
        struct RowAt {
            int b, row;  // request, row of its head's
            bool live;
        };
        auto row_of = [&](const Segment &s, int r) {
            RowAt x{s.b, r, r < plan.rows};
            if (s.shared) {
                const int i = r / plan.rows;
                x.row = r - i * plan.rows;
                x.live = i < s.count;
                if (x.live) x.b = member_of(c.table, a, ex, s.first + i);
            }
            return x;
        };
        auto index_of = [&](const RowAt &x, int kv) {  // in heads; below 2^31
            const int t = quotient(x.row, plan.by_group);
            return (x.b * a.n_tok + t) * a.h_q + (kv - t) * plan.group + x.row;
        };
        int g = 0;
        unsigned seg = 0;
        bool ok = true;
        while (work.left > 0 && ok) {
            const bool first_segment = seg == 0;
            Segment s;
            next_segment<kN, P>(c.table, work, s);
            if (s.n == 0) break;
            const int kv = s.kv, row0 = (s.m * P + rank) * kM;
            const RowAt me = row_of(s, row0 + my_row);
            // the M tile's queries: a warp's 32 rows, eight lanes to 128 bytes of a
            // row; the scores of the segment before have been read, so their
            // products are done with them
            const bool live = me.live, warp_live = __any_sync(~0u, live);
            const int my_index = live ? index_of(me, kv) : -1;
            const size_t q_row = live ? (size_t)my_index * D : 0;
            const uint4 *from[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int index = __shfl_sync(~0u, my_index, i * 4 + lane / 8);
                from[i] = index >= 0 ? reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) + (size_t)index * D) + lane % 8 : nullptr;
            }
            // each of the two warps has every other 128 bytes of a row
            constexpr int kMine = (S::kChunks + 1) / 2;
            uint4 x[kMine][8];
#pragma unroll
            for (int k = 0; k < kMine; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int chunk = 2 * k + half;
                    x[k][i] = make_uint4(0, 0, 0, 0);
                    if (chunk < S::kChunks && from[i] && GDN_IN(from[i] + chunk * 8, 16, bq, st)) x[k][i] = from[i][chunk * 8];
                }
            // by way of shared memory (16 rows of 128 bytes, 16-byte units swizzled): a
            // thread's own row, far from its neighbour's, would be 32 lines a load
            char *pass = base + (pass_s - k_s) + warp * 2048;
#pragma unroll
            for (int k = 0; k < kMine; ++k) {
                const int chunk = 2 * k + half;
                if (chunk >= S::kChunks) break;
                unsigned y[32];
#pragma unroll
                for (int part = 0; part < 2; ++part) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = i * 4 + lane / 8;
                        *reinterpret_cast<uint4 *>(pass + r * 128 + (lane % 8 ^ r % 8) * 16) = x[k][part * 4 + i];
                    }
                    __syncwarp();
                    if (lane / 16 == part)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint4 u = *reinterpret_cast<const uint4 *>(pass + lane % 16 * 128 + (i ^ lane % 8) * 16);
                            y[4 * i] = u.x, y[4 * i + 1] = u.y, y[4 * i + 2] = u.z, y[4 * i + 3] = u.w;
                        }
                    __syncwarp();
                }
                gdntc::tmem_st32(tmem + lane_addr + kQCol + chunk * 32, y);
            }
            gdntc::tmem_wait_st();
            gdntc::fence_before_sync();
            if (tid == 0) c.odd_nodes[(seg + 1) & 3] = c.odd_low[(seg + 1) & 3] = 0;
            __syncwarp();
            if (lane == 0) bar_arrive(saddr(&c.q_full));
            if (work.left > 0 && half == 0) {  // the next segment's queries on their way to L2
                Work peek = work;
                Segment n;
                next_segment<kN, P>(c.table, peek, n);
                RowAt x{0, 0, false};
                if (n.n) x = row_of(n, (n.m * P + rank) * kM + my_row);
                if (x.live)
                    gdndev::prefetch_l2_range(static_cast<const __nv_bfloat16 *>(a.q) + (size_t)index_of(x, n.kv) * D, D * 2, 0, 1);
            }
            // what this row sees, and where its bias is zero
            const int ctx = s.shared ? s.range.slots : s.range.slots - a.n_tok;  // slots that no root path decides on
            gdnattn::NodePath path{0ull, 0, 0};
            int low = s.range.lo;
            float slope = 0.f;
            int ref = 0;
            if (live) {
                const int t = quotient(me.row, plan.by_group) + 1;
                if ((kChanged && ex.slopes) || ex.window || s.base + (s.tile0 + s.n) * kN > ctx)
                    path = gdnattn::node_path(a, ex, a.parent + (size_t)me.b * (a.n_tok + 1), t, bpar);
                if (ex.window && !s.shared) low = max(ex.first ? ex.first[s.b] : 0, min(ctx, ctx + path.depth - ex.window));
                if (kChanged && ex.slopes) {
                    slope = ex.slopes[kv * plan.group + me.row - (t - 1) * plan.group] * gdnattn::kLog2e;
                    ref = slope >= 0.f ? (s.shared ? a.ctx[me.b] : ctx) + path.depth - 1 : ex.plan ? 0 : low;
                }
            }
            constexpr int kCols = kN / 2, kSlices = kCols / 32;  // of a tile, this thread's
            float m = -INFINITY;
            float2 sum = make_float2(0.f, 0.f);
            for (int j = 0; j < s.n; ++j, ++g) {
                const int slot = g & 1, first_slot = s.base + (s.tile0 + s.n - 1 - j) * kN;
                const bool low_edge = first_slot < s.range.all, edge = low_edge || first_slot + kN > ctx;
                ok = wait(saddr(&c.s_full[slot]), (g >> 1) & 1, quit);
                if (edge) ok = ok && wait(saddr(&c.v_full[g % kStages]), (g / kStages) & 1, quit);
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                gdntc::fence_after_sync();
                const unsigned s_addr = tmem + lane_addr + kSCol + slot * kN;
                if (warp_live) {
                    unsigned x[kSlices][32];
#pragma unroll
                    for (int k = 0; k < kSlices; ++k) gdntc::tmem_ld32(s_addr + half * kCols + k * 32, x[k]);
                    gdntc::tmem_wait_ld();
                    const int my_first = first_slot + half * kCols;
                    auto hide = [&](unsigned as) {  // what the row does not see
#pragma unroll
                        for (int k = 0; k < kSlices; ++k) {
                            const int at = my_first + k * 32, hidden = low - at;
                            const unsigned seen = seen32(at - ctx, path.bits) & (hidden <= 0 ? ~0u : hidden >= 32 ? 0u : ~0u << hidden);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!(seen >> i & 1)) x[k][i] = as;
                        }
                    };
                    if (kChanged) {
                        if (edge && ex.cap > 0.f) hide(0u);
                        change<kScores>(ex, x, my_first - ref, slope, a.scale_log2);
                        if (edge && ex.slopes && a.parent && !s.shared)
#pragma unroll
                            for (int k = 0; k < kSlices; ++k) place_nodes(x[k], my_first + k * 32 - ctx, slope, path);
                    }
                    if (edge) hide(0xff800000u);  // -inf
                    float tops[8];  // eight chains: a single one would wait on itself
#pragma unroll
                    for (int i = 0; i < 8; ++i) tops[i] = -INFINITY;
#pragma unroll
                    for (int k = 0; k < kSlices; ++k)
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            tops[i / 2 & 7] = max3(tops[i / 2 & 7], __uint_as_float(x[k][i]), __uint_as_float(x[k][i + 1]));
                    float top = fmaxf(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])),
                                      fmaxf(fmaxf(tops[4], tops[5]), fmaxf(tops[6], tops[7])));
                    // The row's maximum over both halves. The weights are taken relative to
                    // the reference so far while the other warp's maximum is on its way, and
                    // once more where it has fallen too far behind.
                    c.top_of[g & 1][half][my_row] = top;
                    __syncwarp();
                    if (lane == 0) bar_arrive(saddr(&c.pair[rows_warp]));
                    // waits for the other's and moves the reference where it has to; whether it did
                    auto settle = [&]() {
                        ok = __all_sync(~0u, exchanged());
                        if (!ok) return false;
                        top = fmaxf(top, c.top_of[g & 1][half ^ 1][my_row]);
                        if (j == 0) {
                            m = top;
                            return false;
                        }
                        const bool far = (top - m) * scale > 8.f || (m == -INFINITY && top > m);
                        if (!__any_sync(~0u, far)) return false;
                        const float f = far ? ex2((m - top) * scale) : 1.f;
                        ok = __all_sync(~0u, sums_done(g - 1));
                        if (!ok) return false;
                        gdntc::fence_after_sync();
#pragma unroll 1
                        for (int k = half * (D / 2); k < (half + 1) * (D / 2); k += 32) {
                            unsigned o[32];
                            gdntc::tmem_ld32(tmem + lane_addr + k, o);
                            gdntc::tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            gdntc::tmem_st32(tmem + lane_addr + k, o);
                        }
                        if (far) m = top;
                        sum.x *= f;
                        sum.y *= f;
                        return true;
                    };
                    // (changed scores are in registers that taking the weights twice would ask for)
                    bool settled = kChanged || j == 0;
                    if (settled) settle();
                    unsigned p[kCols / 2];
                    float2 part[4];
                    while (ok) {
                        const float mc = m == -INFINITY ? 0.f : m * scale;  // nothing seen yet: every weight is 0
                        const float2 sc = make_float2(scale, scale), mn = make_float2(-mc, -mc);
#pragma unroll
                        for (int i = 0; i < 4; ++i) part[i] = make_float2(0.f, 0.f);
#pragma unroll
                        for (int i = 0; i < kCols / 2; ++i) {
                            const unsigned *y = &x[i / 16][i % 16 * 2];
                            float2 f = fma2(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), sc, mn);
                            f.x = ex2(f.x);
                            f.y = ex2(f.y);
                            part[i & 3] = add2(part[i & 3], f);
                            p[i] = pack_bf16(f.x, f.y);
                        }
                        if (kChanged || settled) break;
                        settled = true;
                        if (!settle()) break;
                    }
                    if (!ok) break;
                    // (both warps have read their scores, over which the weights go)
                    if constexpr (kCols == 64)
                        gdntc::tmem_st32(s_addr + half * 32, p);
                    else
                        gdntc::tmem_st16(s_addr + half * 16, p);
                    sum = add2(sum, add2(add2(part[0], part[1]), add2(part[2], part[3])));
                    gdntc::tmem_wait_st();
                }
                if (edge) {
                    // v where no row sees it becomes zeros, and so does what is no number
                    // among the values that some rows see and others do not: 0 x NaN must
                    // not reach those; the ones that see them get them back at the end
                    char *v = base + (v_s - k_s) + (g % kStages) * S::kTileBytes;
                    const int lo = low_edge ? 0 : max(0, ctx - first_slot);
                    for (int i = tid; i < (kN - lo) * S::kChunks * 8; i += kSoftWarps * 32) {
                        const int r = lo + i / (S::kChunks * 8), u = i % (S::kChunks * 8);
                        uint4 *p = reinterpret_cast<uint4 *>(v + (u / 8) * (kN * 128) + r * 128 + (u % 8) * 16);
                        const int at = first_slot + r;
                        if (at >= s.range.slots || at < s.range.lo) {
                            *p = make_uint4(0, 0, 0, 0);
                            continue;
                        }
                        if (at < ctx && at >= s.range.all) continue;
                        uint4 x = *p;
                        unsigned *y = reinterpret_cast<unsigned *>(&x);
                        bool odd = false;
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            const bool lo_odd = (y[h] & 0x7f80u) == 0x7f80u, hi_odd = (y[h] & 0x7f800000u) == 0x7f800000u;
                            if (lo_odd) y[h] &= 0xffff0000u;
                            if (hi_odd) y[h] &= 0xffffu;
                            odd |= lo_odd || hi_odd;
                        }
                        if (odd) {
                            *p = x;
                            if (at >= ctx)
                                atomicOr(&c.odd_nodes[seg & 3], 1ull << (at - ctx));
                            else
                                atomicOr(&c.odd_low[seg & 3], 1ull << (at - s.range.lo));
                        }
                    }
                    gdntc::fence_smem_to_async();
                }
                gdntc::fence_before_sync();
                __syncwarp();
                if (lane == 0) bar_arrive(saddr(&c.p_full[slot]));
            }
            if (!ok) break;
            ok = __all_sync(~0u, sums_done(g - 1));
            if (!ok) break;
            gdntc::fence_after_sync();
            if (warp_live) {
                const bool whole = s.n == s.tiles, member = s.shared || (ex.plan && s.range.lo > 0);
                const bool done = whole && !member;  // the row's result, not a part of it
                c.sum_of[half][my_row] = sum.x + sum.y;
                __syncwarp();
                if (lane == 0) bar_arrive(saddr(&c.pair[rows_warp]));
                ok = __all_sync(~0u, exchanged());
                if (!ok) break;
                const float total = c.sum_of[0][my_row] + c.sum_of[1][my_row], inv = done ? 1.f / total : 1.f;
                const unsigned long long odd = *(volatile unsigned long long *)&c.odd_nodes[seg & 3] & path.bits;
                const unsigned long long odd_low =
                    low - s.range.lo < 64 ? *(volatile unsigned long long *)&c.odd_low[seg & 3] & ~0ull << (low - s.range.lo) : 0ull;
                const size_t piece = 2 * share + (first_segment ? 0 : 1);
                const int pr = rank * kM + my_row;
                if (!whole && tid == 0 && rank == 0)
                    pieces.unit[piece] = unit_number(a, plan, s.m_groups, s.shared, s.shared ? s.e : s.b, kv, s.m);
                // a part's place: a step of rows from one 16 bytes of a row to the next
                const size_t head = (size_t)me.b * a.h_kv + kv;
                const int step = whole ? plan.rows_pad : P * kM;
                float4 *part_o = whole ? pieces.row_o[s.shared] + head * (D / 4) * plan.rows_pad + me.row
                                       : pieces.o + piece * (D / 4) * (P * kM) + pr;
                float2 *part_ms = whole ? pieces.row_ms[s.shared] + head * plan.rows_pad + me.row : pieces.ms + piece * (P * kM) + pr;
                const size_t part_rows = whole ? (size_t)a.batch * a.h_kv * plan.rows_pad : (size_t)2 * plan.blocks * P * kM;
                const Buf bo{whole ? pieces.row_o[s.shared] : pieces.o, part_rows * D * 4},
                    bms{whole ? pieces.row_ms[s.shared] : pieces.ms, part_rows * 8};
                if (!done && live && half == 0 && GDN_IN(part_ms, 8, bms, st)) *part_ms = make_float2(m == -INFINITY ? m : m * scale, total);
#pragma unroll 1
                for (int k = half * (D / 2); k < (half + 1) * (D / 2); k += 32) {
                    unsigned o[32];
                    __syncwarp();
                    gdntc::tmem_ld32(tmem + lane_addr + k, o);
                    gdntc::tmem_wait_ld();
                    if (!live) continue;
                    float f[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(o[i]) * inv;
                    if (done) {
                        __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(a.out) + q_row + k;
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            if (GDN_IN(to + i, 16, bout, st))
                                *reinterpret_cast<uint4 *>(to + i) =
                                    make_uint4(pack_bf16(f[i], f[i + 1]), pack_bf16(f[i + 2], f[i + 3]),
                                               pack_bf16(f[i + 4], f[i + 5]), pack_bf16(f[i + 6], f[i + 7]));
                    } else {
                        float4 *to = part_o + (size_t)(k / 4) * step;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (GDN_IN(to + (size_t)i * step, 16, bo, st))
                                to[(size_t)i * step] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
                    }
                }
                if (live && (odd | odd_low))
                    restore<D>(c.table, part_o, step, done ? static_cast<__nv_bfloat16 *>(a.out) + q_row : nullptr, half * (D / 2),
                               (half + 1) * (D / 2), s.b, kv, odd, ctx, odd_low, s.range.lo);
            }
            __syncwarp();
            gdntc::fence_before_sync();
            ++seg;
        }
    }
    // requests that are left out get zeros
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x)
        if ((a.batch <= kKept ? c.table.request[b].range : gdnattn::range_of(a, ex, b)).slots == 0) {
            const size_t units16 = (size_t)a.n_tok * a.h_q * D / 8;
            uint4 *to = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out)) + b * units16;
            const Buf bout{a.out, (size_t)a.batch * units16 * 16};
#pragma unroll 1
            for (size_t i = tid; i < units16; i += S::kThreads)
                if (GDN_IN(to + i, 16, bout, st)) to[i] = make_uint4(0, 0, 0, 0);
        }
    __syncthreads();
    if (c.quit && tid == 0 && st) atomicOr(st, GDN_DEV_SCHED);
    if (warp == kScoreWarp) {
        gdntc::fence_after_sync();
        gdntc::tmem_dealloc<kTmemCols>(tmem);
    }
}

// The rows' parts added up. An item is 32 rows of a request's head x 8 columns; a
// block's warps are kJoinWarps / `share` items of `share` warps, which take the item's
// parts in turn, four at a time. A row's parts are the blocks' pieces of its request's
// unit and, for a member of a group, of the group's unit in which its row lies (32 rows
// lie in two of them at most), or, where one block had a unit as a whole, the row's
// place in the buffers.
constexpr int kJoinWarps = 8;

// A row's running sums relative to its running maximum.
struct Joined {
    float m = -INFINITY, sum = 0.f;
    float4 o[2] = {};
};

template <int K>
__device__ __forceinline__ void absorb(Joined &j, const float2 (&ms)[K], const float4 (&x)[K][2]) {
    float top = j.m;
#pragma unroll
    for (int u = 0; u < K; ++u) top = fmaxf(top, ms[u].x);
    const float f0 = j.m == -INFINITY ? 0.f : ex2(j.m - top);
    j.sum *= f0;
#pragma unroll
    for (int i = 0; i < 2; ++i) j.o[i] = make_float4(j.o[i].x * f0, j.o[i].y * f0, j.o[i].z * f0, j.o[i].w * f0);
#pragma unroll
    for (int u = 0; u < K; ++u) {
        if (ms[u].x == -INFINITY && ms[u].y == 0.f) continue;  // nothing there that the row sees
        const float f = ms[u].x == top ? 1.f : ex2(ms[u].x - top);
        j.sum = fmaf(ms[u].y, f, j.sum);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            j.o[i] = make_float4(fmaf(x[u][i].x, f, j.o[i].x), fmaf(x[u][i].y, f, j.o[i].y), fmaf(x[u][i].z, f, j.o[i].z),
                                 fmaf(x[u][i].w, f, j.o[i].w));
    }
    j.m = top;
}

template <int D, int P>
__global__ void __launch_bounds__(kJoinWarps * 32, 4)
join_rows(const __grid_constant__ AttnArgs a, const __grid_constant__ ExArgs ex, const __grid_constant__ Plan plan,
          const __grid_constant__ Pieces pieces, int share, int items, int chunks) {
    constexpr int kRows = P * kM, kCols = D / 8, kAhead = 4;
    __shared__ float4 part[kJoinWarps][2][32];
    __shared__ float top[kJoinWarps][32], total[kJoinWarps][32];
    __shared__ unsigned short list[kJoinWarps][2 * kMaxBlocks];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int item = blockIdx.x * (kJoinWarps / share) + warp / share, which = warp % share;
    const int d4 = item % kCols * 2, head = item / kCols / chunks, chunk = item / kCols - head * chunks;
    const int b = item < items ? head / a.h_kv : 0, kv = item < items ? head - b * a.h_kv : 0;
    const int row = chunk * 32 + lane;
    const Buf bout{a.out, (size_t)a.batch * a.n_tok * a.h_q * D * 2};
    gdndev::pdl_wait();
    gdndev::pdl_launch_dependents();
    int note[kNotes];
#pragma unroll
    for (int i = 0; i < kNotes; ++i) {
        const int p = i * 32 + lane;
        note[i] = p < 2 * plan.blocks ? __ldcg(pieces.unit + p) : -1;
    }
    const gdnattn::Range range = gdnattn::range_of(a, ex, b);
    int g = -1, place = 0, members = 0;
    if (ex.plan) {
        const gdnattn::PrefixPlan p(ex.plan, a.batch);
        g = p.group[b], place = p.place[b], members = gdnattn::clamped(p.size[b], 1, a.batch);
        place = gdnattn::clamped(place, 0, members - 1);
        if (range.lo == 0 || g >= a.batch / 2) g = -1;
    }
    const bool there = item < items && range.slots > 0, live = there && row < plan.rows;
    // the row's units: its request's, its group's
    const int m = chunk * 32 / kRows, own = there ? unit_number(a, plan, plan.m_groups, false, b, kv, m) : -2;
    const int own_at = row - m * kRows;
    int theirs = -2, theirs_at = 0;
    if (g >= 0 && live) {
        const unsigned r = (unsigned)place * (unsigned)plan.rows + (unsigned)row;  // below 2^31
        const int m_groups = (int)(((unsigned)members * (unsigned)plan.rows + kRows - 1) / kRows);
        theirs = unit_number(a, plan, m_groups, true, g, kv, (int)(r / kRows));
        theirs_at = (int)(r % kRows);
    }
    const int low = __shfl_sync(~0u, theirs, 0);  // rows in order: lane 0 has the first unit, the others it or the next
    int n = 0, n_own = 0, n_low = 0, n_high = 0;
#pragma unroll
    for (int i = 0; i < kNotes; ++i) {
        const bool o = own >= 0 && note[i] == own, l = low >= 0 && note[i] == low, h = low >= 0 && note[i] == low + 1;
        const unsigned here = __ballot_sync(~0u, o || l || h);
        if (here == 0) continue;
        if (o || l || h) list[warp][n + __popc(here & ((1u << lane) - 1))] = (unsigned short)((i * 32 + lane) << 2 | (o ? 0 : l ? 1 : 2));
        n += __popc(here);
        n_own += __popc(__ballot_sync(~0u, o));
        n_low += __popc(__ballot_sync(~0u, l));
        n_high += __popc(__ballot_sync(~0u, h));
    }
    __syncwarp();
    const bool own_whole = n_own == 0;
    const int tag = theirs < 0 ? 3 : theirs == low ? 1 : 2;  // of its group's pieces in the list
    // one block had the whole request and has written its result
    const bool mine = live && (g >= 0 || !own_whole);
    Joined j;
#pragma unroll 1
    for (int k0 = __any_sync(~0u, mine) ? which : n; k0 < n; k0 += share * kAhead) {
        float2 ms[kAhead];
        float4 x[kAhead][2];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int k = k0 + u * share, e = k < n ? list[warp][k] : 3;
            ms[u] = make_float2(-INFINITY, 0.f);
            x[u][0] = x[u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (mine && ((e & 3) == 0 || (e & 3) == tag) && k < n) {
                const int at = (e & 3) == 0 ? own_at : theirs_at, piece = e >> 2;
                const float2 *fm = pieces.ms + piece * kRows + at;
                const float4 *fo = pieces.o + (piece * (D / 4) + d4) * kRows + at;
                const size_t all = (size_t)2 * plan.blocks * kRows;
                const Buf bms{pieces.ms, all * 8}, bo{pieces.o, all * D * 4};
                if (GDN_IN(fm, 8, bms, a.status)) ms[u] = __ldcg(fm);
                if (GDN_IN(fo, 16, bo, a.status)) x[u][0] = __ldcg(fo);
                if (GDN_IN(fo + kRows, 16, bo, a.status)) x[u][1] = __ldcg(fo + kRows);
            }
        }
        absorb(j, ms, x);
    }
    if (mine && g >= 0 && which == share - 1) {  // the buffers
        float2 ms[2];
        float4 x[2][2];
        const bool from[2] = {own_whole, (tag == 1 ? n_low : n_high) == 0};
        const size_t hd = (size_t)b * a.h_kv + kv, all = (size_t)a.batch * a.h_kv * plan.rows_pad;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            ms[u] = make_float2(-INFINITY, 0.f);
            x[u][0] = x[u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (!from[u]) continue;
            const float2 *fm = pieces.row_ms[u] + hd * plan.rows_pad + row;
            const float4 *fo = pieces.row_o[u] + (hd * (D / 4) + d4) * plan.rows_pad + row;
            const Buf bms{pieces.row_ms[u], all * 8}, bo{pieces.row_o[u], all * D * 4};
            if (GDN_IN(fm, 8, bms, a.status)) ms[u] = __ldcg(fm);
            if (GDN_IN(fo, 16, bo, a.status)) x[u][0] = __ldcg(fo);
            if (GDN_IN(fo + plan.rows_pad, 16, bo, a.status)) x[u][1] = __ldcg(fo + plan.rows_pad);
        }
        absorb(j, ms, x);
    }
    top[warp][lane] = j.m;
    total[warp][lane] = j.sum;
    part[warp][0][lane] = j.o[0];
    part[warp][1][lane] = j.o[1];
    __syncthreads();
    if (!mine || which != 0) return;
#pragma unroll 1
    for (int w = warp + 1; w < warp + share; ++w) {
        const float2 ms[1] = {make_float2(top[w][lane], total[w][lane])};
        const float4 x[1][2] = {{part[w][0][lane], part[w][1][lane]}};
        absorb(j, ms, x);
    }
    const float inv = 1.f / j.sum;
    const int t = quotient(row, plan.by_group);
    __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(a.out) +
                        (((size_t)b * a.n_tok + t) * a.h_q + (kv - t) * plan.group + row) * D + d4 * 4;
    if (GDN_IN(to, 16, bout, a.status))
        *reinterpret_cast<uint4 *>(to) =
            make_uint4(pack_bf16(j.o[0].x * inv, j.o[0].y * inv), pack_bf16(j.o[0].z * inv, j.o[0].w * inv),
                       pack_bf16(j.o[1].x * inv, j.o[1].y * inv), pack_bf16(j.o[1].z * inv, j.o[1].w * inv));
}

// Blocks side by side on the same tiles: two where a request has more than one M tile.
// A group's rows alone do not ask for it: its M tiles are at work on the same slots at
// about the same time anyway, and pairs would leave every second block idle in the
// requests' own slots (2 x 8 trees of 22 nodes over 16,000 shared slots 317 us for two
// layers instead of 340).
int pair(const attn_dims *d, int n_tok) { return (int64_t)n_tok * (d->h_q / d->h_kv) > kM ? 2 : 1; }

struct Sizes {
    int p, blocks, rows, rows_pad;
    size_t piece_rows, row_parts;  // rows of the blocks' pieces, of each of the two buffers
    Sizes(const attn_dims *d, int n_tok, bool shared) {
        p = pair(d, n_tok);
        blocks = block_count() / p;
        rows = n_tok * (d->h_q / d->h_kv);
        rows_pad = (rows + 31) / 32 * 32;
        piece_rows = (size_t)2 * blocks * p * kM;
        row_parts = shared ? (size_t)d->batch * d->h_kv * rows_pad : 0;
    }
    size_t bytes(int d) const { return (piece_rows + 2 * row_parts) * (d * 4 + 8) + 2 * (size_t)blocks * 4; }
};

template <int D, int P>
int launch(const attn_dims *d, const AttnArgs &a, const ExArgs &x, void *ws, cudaStream_t st) {
    using S = Shape<D>;
    static bool set[3][256] = {};
    const Scores scores = x.cap > kMostOfNear ? kFar : x.cap > 0.f || x.slopes ? kNear : kPlain;
    const auto kernel = scores == kFar ? attend_ex<D, P, kFar> : scores == kNear ? attend_ex<D, P, kNear> : attend_ex<D, P, kPlain>;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return GDN_ERR_CUDA;
    if (!set[scores][dev]) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem) != cudaSuccess)
            return GDN_ERR_CUDA;
        set[scores][dev] = true;
    }
    CUtensorMap k_map, v_map;
    if (!pool_map(&k_map, d, a.k_pages, S::kN) || !pool_map(&v_map, d, a.v_pages, S::kN)) return GDN_ERR_CUDA;
    const bool shared = x.plan != nullptr;
    const Sizes z(d, a.n_tok, shared);
    char *at = static_cast<char *>(ws);
    Pieces pieces{};
    auto take = [&](size_t bytes) {
        char *p = at;
        at += bytes;
        return p;
    };
    pieces.o = reinterpret_cast<float4 *>(take(z.piece_rows * D * 4));
    for (int i = 0; i < 2; ++i) pieces.row_o[i] = reinterpret_cast<float4 *>(take(z.row_parts * D * 4));
    pieces.ms = reinterpret_cast<float2 *>(take(z.piece_rows * 8));
    for (int i = 0; i < 2; ++i) pieces.row_ms[i] = reinterpret_cast<float2 *>(take(z.row_parts * 8));
    pieces.unit = reinterpret_cast<int *>(at);
    const int group = a.h_q / a.h_kv, m_groups = (z.rows + P * kM - 1) / (P * kM);
    const int shared_units = shared ? a.h_kv * (int)(((int64_t)a.batch * z.rows + P * kM - 1) / (P * kM)) : 0;
    auto by = [](int n) { return (unsigned)(((1ull << 32) + n - 1) / n); };
    const Plan plan{group, z.rows, m_groups, a.h_kv * m_groups, shared_units, z.blocks, z.rows_pad, by(group), by(m_groups), by(z.blocks), ~0ull / z.blocks + 1};
    if (gdndev::launch_pdl(kernel, dim3(z.blocks * P), dim3(S::kThreads), S::kSmem, st, k_map, v_map, a, x, plan, pieces) !=
        cudaSuccess)
        return GDN_ERR_CUDA;
    // a unit has about blocks / units pieces, and one more (fewer units where a prefix is shared)
    const int64_t units = shared ? shared_units : (int64_t)a.batch * plan.units;
    const int64_t per_unit = z.blocks / (units < z.blocks ? units : z.blocks) + 1;
    const int share = per_unit <= 4 ? 1 : per_unit <= 8 ? 2 : per_unit <= 24 ? 4 : 8;
    const int chunks = z.rows_pad / 32;
    const int items = a.batch * a.h_kv * chunks * (D / 8), per_block = kJoinWarps / share;
    return gdndev::launch_pdl(join_rows<D, P>, dim3((unsigned)((items - 1) / per_block + 1)), dim3(kJoinWarps * 32), 0, st, a, x, plan, pieces, share, items,
                              chunks) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

namespace gdnattn {

bool ex_tc_fits(const attn_dims *d, int n_tok, bool shared) {
    // tiles of 64 slots: Work::off counts an entry's cost in an int, Work::left a block's
    // share of all (16 blocks at least); units and the join's grid in 32 bits
    const int64_t rows = (int64_t)n_tok * (d->h_q / d->h_kv), all = rows * (shared ? d->batch : 1);
    const int64_t slot_tiles = ((int64_t)d->table_width * d->page_tokens + 63) / 64 + kStart;
    const int64_t tiles = slot_tiles * d->h_kv * ((all + kM - 1) / kM);
    const int64_t units = d->h_kv * (((rows + kM - 1) / kM) + (shared ? (all + kM - 1) / kM : 0));
    return (int64_t)d->batch * n_tok * d->h_q < (1LL << 31) && all < (1LL << 31) && tiles < (1LL << 31) && tiles * d->batch < (1LL << 34) && units * d->batch < (1LL << 31) &&
           (int64_t)d->batch * d->h_kv * ((rows + 31) / 32) * (d->d_head / 8) < (1LL << 31);
}

size_t ex_tc_workspace(const attn_dims *d, int n_tok, bool shared) { return Sizes(d, n_tok, shared).bytes(d->d_head); }

int ex_tc_launch(const attn_dims *d, const AttnArgs &a, const ExArgs &x, void *ws, cudaStream_t st) {
    if (pair(d, a.n_tok) == 2)
        return a.d == 64 ? launch<64, 2>(d, a, x, ws, st) : a.d == 128 ? launch<128, 2>(d, a, x, ws, st) : launch<256, 2>(d, a, x, ws, st);
    return a.d == 64 ? launch<64, 1>(d, a, x, ws, st) : a.d == 128 ? launch<128, 1>(d, a, x, ws, st) : launch<256, 1>(d, a, x, ws, st);
}

}  // namespace gdnattn
