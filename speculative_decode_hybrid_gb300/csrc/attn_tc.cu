// Attention of a drafted span over the paged cache on the tensor cores
// (attn_verify_span / attn_tree_verify with GDN_BF16).
//
// The rows of one key/value head's product are the span's nodes times the query
// heads of the group; 128 of them are an M tile, the work of one block. For each
// tile of kN slots
//   S = Q K^T        tcgen05, Q in tensor memory, K in shared memory, S in tensor memory
//   P = 2^(c S - m)  one thread per row, rounded to bf16, over S's columns
//   O += P V         tcgen05, P read from tensor memory, V MN-major in shared
//                    memory as it lies in the page
// in one pass, the softmax relative to a reference m that follows the running
// maximum only when it falls more than 2^8 behind (then O is rescaled in tensor
// memory): the weights stay below 2^8, and the final division by the sum of
// the same weights (in f32, before their rounding) makes the result independent
// of m. The rounding of P to bf16 is what feeds the second product at the tensor
// cores' 16-bit rate; it moves a result by at most 2^-8 sum p |v|: 2.0e-3 to
// 2.5e-3 of a result's norm, of which the rounding of the result itself is 1.7e-3.
// P in two bf16 parts, with a product for each, leaves that 1.7e-3 alone, takes 4 %
// longer where the cache's bytes bound (16 spans of 16 over up to 8,000 slots 77 us
// instead of 74) and 12 to 18 % elsewhere (22 nodes of 256 over 32,501 37.6 instead
// of 33.5, 512 rows over up to 8,000 50.8 instead of 43.2), and would turn an
// infinity among the committed values into NaN, 0 x inf of a part that is zero.
//
// Warps: 4 for the softmax, one that keeps the TMA loads of the next tiles in
// flight (a page's rows of one head are a box of a 3-d tensor map, so a tile is
// gathered page by page), one that issues each of the products. S is double:
// the scores of the next tile are computed while the softmax works on this one.
//
// More than 128 rows: P = 2 neighbouring blocks take an M tile each of the same
// piece of work. They load the same tiles at about the same time, each for
// itself: the second one's come from L2.
//
// Work is split over the whole flattened list of (request, head, M tiles, slot
// tile): block i of n takes the i-th n-th of it, whatever the requests'
// lengths. Pieces of a unit that several blocks share go to the workspace, and
// join_pieces adds them up on the scale of their largest maximum.
//
// Bound by the bytes of K and V while the rows are few (4 kN D bytes a tile
// against 4 x 128 x kN x D operations), by products and exponentials with full
// M tiles. Measured: 16 requests' spans of 16 over up to 8,000 slots (32 heads on
// 8, 128 wide; 378 MB read, no byte twice) 65 us, 5.8 TB/s, 0.86 of the measured
// copy rate, of which 6 us pass before the first tile has come; 22 nodes x 8 heads,
// 256 wide, over 32,501 slots (67 MB) 26 us: thirteen tiles a block, each some
// 1,850 cycles apart (1.6 us from asking for a tile to having it, three in
// flight), after 6 us until the first. Two M tiles in one block
// instead of two blocks: 55 us instead of 43 for 512 rows over up to 8,000 slots,
// as tensor memory then leaves room for single S buffers only, and a tile's
// products and softmax follow one another.
#include <cuda.h>
#include <cuda_runtime.h>

#include "attn_common.cuh"
#include "attn_host.h"
#include "attn_tc.cuh"
#include "gdn_host.h"
#include "gdnspec.h"

namespace {

using gdnattn::AttnArgs;
using gdndev::add2;
using gdndev::Buf;
using gdndev::fma2;

constexpr int kM = 128;                    // rows of an M tile
constexpr unsigned long long kGiveUpNs = 1000000000ull;  // a wait's limit

constexpr int kTmemCols = 512;  // all of an SM's: one block per SM
constexpr int kMaxBlocks = 160, kNotes = 2 * kMaxBlocks / 32;

template <int D>
struct Shape {
    static constexpr int kN = D == 256 ? 64 : 128;       // slots of a tile
    static constexpr int kChunks = D / 64;               // 128-byte column chunks of a row
    static constexpr unsigned kSCol = D, kQCol = kSCol + 2 * kN;  // tensor-memory columns: O, S twice, Q
    static constexpr int kStages = D == 64 ? 6 : 3;
    static constexpr unsigned kTileBytes = kN * D * 2;   // of K, and of V
    static constexpr unsigned kPassBytes = 4 * 4096;     // a warp's 32 rows x 128 bytes of Q on their way
    static constexpr int kThreads = 128 + 96;
    static constexpr unsigned kSmem = 2 * kStages * kTileBytes + kPassBytes + 1024;
    static_assert(kQCol + D / 2 <= kTmemCols, "tensor memory");
};

// What the host works out: divisions take a warp longer than a load from L2.
struct Plan {
    int group, rows;        // query heads of a key/value head; rows of one key/value head
    int m_groups, units;    // groups of P M tiles of a head; units (head, group) of a request
    int blocks;             // groups of P blocks, each group on a share of its own
    unsigned by_group, by_m_groups, by_blocks;  // 2^32 / n rounded up: x / n for x * n < 2^32
};

__device__ __forceinline__ int quotient(int x, unsigned by) { return by ? (int)__umulhi((unsigned)x, by) : x; }  // by 1: 2^32 is 0

struct Work {
    int b, off, left;  // request, tiles of it already dealt out, tiles of this block still to come
};

struct Segment {
    int b, unit, tile0, n, tiles, slots;
};

template <int kN>
__device__ __forceinline__ Segment next_segment(const AttnArgs &a, const Plan &plan, Work &w) {
    Segment s;
    s.b = w.b;
    s.slots = gdnattn::slots_of(a, w.b);
    while (s.slots == 0 && w.b + 1 < a.batch) s.b = ++w.b, s.slots = gdnattn::slots_of(a, w.b);
    s.tiles = (s.slots + kN - 1) / kN;
    s.unit = w.off / s.tiles;
    s.tile0 = w.off - s.unit * s.tiles;
    s.n = min(s.tiles - s.tile0, w.left);
    w.off += s.n;
    w.left -= s.n;
    if (w.off == s.tiles * plan.units) ++w.b, w.off = 0;
    return s;
}

// Block i's share of `total` tiles begins at total * i / blocks, rounded down.
struct Share {
    long long whole;
    int rest;
    __device__ __forceinline__ Share(long long total, int blocks) {
        if (total >> 31 == 0)  // the 64-bit division takes long, and totals are small
            whole = (unsigned)total / (unsigned)blocks;
        else
            whole = total / blocks;
        rest = (int)(total - whole * blocks);
    }
    __device__ __forceinline__ long long start(int i, const Plan &plan) const {
        return whole * i + quotient(rest * i, plan.by_blocks);
    }
};

// This block's share, and the request in which it begins: by each warp for
// itself, so that none waits for another.
template <int kN>
__device__ __forceinline__ Work block_work(const AttnArgs &a, const Plan &plan, int block, bool flag) {
    const int lane = threadIdx.x & 31;
    auto tiles_of = [&](int b) { return b < a.batch ? (gdnattn::slots_of(a, b) + kN - 1) / kN : 0; };
    const int mine = tiles_of(lane);
    long long total = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) total += __reduce_add_sync(~0u, b0 ? tiles_of(b0 + lane) : mine);
    const int units = plan.units;
    const Share share(total * units, plan.blocks);
    const long long lo = share.start(block, plan), hi = share.start(block + 1, plan);
    Work w{0, 0, 0};
    long long before = 0;
    for (int b0 = 0; b0 < a.batch && (lo >= before || flag); b0 += 32) {
        const int b = b0 + lane, n = b0 ? tiles_of(b) : mine;
        int x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(~0u, x, o);
            if (lane >= o) x += y;
        }
        const long long first = before + (long long)(x - n) * units;
        const unsigned here = __ballot_sync(~0u, lo >= first && lo < first + (long long)n * units);
        if (here) {
            const int from = __ffs(here) - 1;
            w = {b0 + from, (int)(lo - __shfl_sync(~0u, first, from)), (int)(hi - lo)};
        }
        if (flag && a.status && b < a.batch && n == 0) atomicOr(a.status, GDN_DEV_LENGTH);
        before += (long long)__shfl_sync(~0u, x, 31) * units;
    }
    return w;
}

__device__ __forceinline__ unsigned saddr(const void *p) { return (unsigned)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(unsigned bar, unsigned count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(unsigned bar) {
    asm volatile("{\n\t.reg .b64 t;\n\tmbarrier.arrive.shared::cta.b64 t, [%0];\n\t}" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(unsigned bar, unsigned bytes) {
    asm volatile("{\n\t.reg .b64 t;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 t, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ unsigned long long now_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}

// Wait for phase `parity`; false after a second, or once another wait of this
// block has given up (*quit). A null quit: the second alone.
__device__ __forceinline__ bool wait(unsigned bar, unsigned parity, volatile int *quit) {
    if (gdntc::mbar_wait(bar, parity, 1)) return true;
    const unsigned long long t0 = now_ns();
    while (!gdntc::mbar_wait(bar, parity, 1)) {
        if (quit && *quit) return false;
        if (now_ns() - t0 > kGiveUpNs) {
            if (quit) *quit = 1;
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ void load_box(unsigned dst, const CUtensorMap *map, int x, int y, int z, unsigned bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}
__device__ __forceinline__ unsigned pack_bf16(float lo, float hi) {
    unsigned r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Which of 32 slots, the first `rel` past the committed ones, a row with this
// root path sees.
__device__ __forceinline__ unsigned seen32(int rel, unsigned long long path) {
    if (rel >= 64) return 0u;
    if (rel >= 0) return (unsigned)(path >> rel);
    if (rel <= -32) return ~0u;
    return ((unsigned)path << -rel) | ((1u << -rel) - 1u);
}

// Row r of a key/value head's product in q and out, in heads: node r / group, the
// group's query head r % group.
__device__ __forceinline__ size_t row_offset(const AttnArgs &a, const Plan &plan, int b, int kv, int r) {
    const int t = quotient(r, plan.by_group);
    return ((size_t)b * a.n_tok + t) * a.h_q + (kv - t) * plan.group + r;
}

struct Pieces {
    float4 *o;    // [2 blocks][D / 4][P * 128]
    float2 *ms;   // [2 blocks][P * 128]: reference maximum in powers of two, sum
    int *unit;    // [2 blocks]: request * units + unit of a block's first and last piece of a shared unit, -1 for none
};

template <int D>
struct Control {
    static constexpr int kStages = Shape<D>::kStages;
    unsigned long long k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
    unsigned long long s_full[2], p_full[2], pv_done[2], q_full, drain[2];
    unsigned long long odd_nodes[4];  // drafted nodes with a value of v that is no number, by segment
    unsigned tmem;
    int quit;
};

template <int D, int P>
__global__ void __launch_bounds__(Shape<D>::kThreads, 1)
attend(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
       const __grid_constant__ AttnArgs a, const __grid_constant__ Plan plan, const __grid_constant__ Pieces pieces) {
    using S = Shape<D>;
    constexpr int kN = S::kN, kStages = S::kStages;
    extern __shared__ char raw[];
    __shared__ Control<D> c;
    char *base = raw + ((1024 - (saddr(raw) & 1023)) & 1023);
    const unsigned k_s = saddr(base), v_s = k_s + kStages * S::kTileBytes, pass_s = v_s + kStages * S::kTileBytes;
    const int share = blockIdx.x / P, rank = blockIdx.x % P;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = plan.group, rows = plan.rows;
    int32_t *st = a.status;
    constexpr int kTmaWarp = 4, kScoreWarp = 5, kSumWarp = 6;

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
            bar_init(saddr(&c.p_full[i]), 4);  // one arrival per softmax warp
            bar_init(saddr(&c.pv_done[i]), 1);
        }
        bar_init(saddr(&c.q_full), 4);
        bar_init(saddr(&c.drain[0]), 1);
        bar_init(saddr(&c.drain[1]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");  // for the TMA unit
        c.quit = 0;
        for (int i = 0; i < 4; ++i) c.odd_nodes[i] = 0;
    }
    gdndev::pdl_launch_dependents();  // join_pieces, which takes no tensor memory
    gdndev::pdl_wait();
    // All of the SM's columns, and only once nothing is waited for outside of this
    // block: the kernel before may be anybody's, and may need columns itself.
    if (warp == kScoreWarp) gdntc::tmem_alloc<kTmemCols>(&c.tmem);
    gdntc::fence_before_sync();
    Work work = block_work<kN>(a, plan, share, blockIdx.x == 0 && warp == 0);
    __syncthreads();
    gdntc::fence_after_sync();
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
            const Segment s = next_segment<kN>(a, plan, work);
            const int kv = quotient(s.unit, plan.by_m_groups);
            const int32_t *row = a.table + (size_t)s.b * a.width;
            const int32_t *e = row + ((s.tile0 * kN + mine * page_rows) >> a.page_shift);
            // a page id is read one tile ahead
            int page = mine < boxes && s.tile0 * kN + mine * page_rows < s.slots && GDN_IN(e, 4, bt, st) ? *e : 0;
            for (int j = 0; j < s.n; ++j, ++g) {
                const int slot = (s.tile0 + j) * kN + mine * page_rows;
                const bool used = mine < boxes && slot < s.slots;
                const bool known = page >= 0 && page < a.n_pages;
                if (used && !known && st && chunk == 0) atomicOr(st, GDN_DEV_PAGE);
                // a page outside the pool lies outside the tensor map, which reads as zeros
                const int z = known ? page * a.h_kv + kv : -1, y = slot & ((1 << a.page_shift) - 1);
                const unsigned bytes = __popc(__ballot_sync(~0u, used)) * box_bytes;
                int next = 0;
                if (j + 1 < s.n && mine < boxes && slot + kN < s.slots) {
                    const int32_t *f = row + ((slot + kN) >> a.page_shift);
                    if (GDN_IN(f, 4, bt, st)) next = *f;
                }
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
                const Segment s = next_segment<kN>(a, plan, work);
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
                const Segment s = next_segment<kN>(a, plan, work);
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
        const unsigned lane_addr = (unsigned)warp << 21;  // 32 lanes each, in bits 16 and up
        const Buf bq{a.q, (size_t)a.batch * a.n_tok * a.h_q * D * 2}, bout{a.out, (size_t)a.batch * a.n_tok * a.h_q * D * 2},
            bpar{a.parent, (size_t)a.batch * (a.n_tok + 1) * 4};
        const float scale = a.scale_log2;
        // The scores of tile g are issued before the sums of g - 1, so a tile's scores
        // only tell that the sums of g - 2 are done: a barrier for each S buffer
        // keeps its phases apart.
        auto sums_done = [&](int tile) { return wait(saddr(&c.pv_done[tile & 1]), (tile >> 1) & 1, quit); };
        int g = 0;
        unsigned seg = 0;
        bool ok = true;
        while (work.left > 0 && ok) {
            const bool first_segment = seg == 0;
            const Segment s = next_segment<kN>(a, plan, work);
            const int kv = quotient(s.unit, plan.by_m_groups), row0 = ((s.unit - kv * plan.m_groups) * P + rank) * kM, row = row0 + tid;
            const int ctx = s.slots - a.n_tok;
            // the M tile's queries: a warp's 32 rows, eight lanes to 128 bytes of a
            // row; the scores of the segment before have been read, so their
            // products are done with them
            const bool live = row < rows, warp_live = row0 + warp * 32 < rows;
            auto row_at = [&](int r) { return row_offset(a, plan, s.b, kv, r) * D; };
            const size_t q_row = live ? row_at(row) : 0;
            const uint4 *from[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = row0 + warp * 32 + i * 4 + lane / 8;
                from[i] = r < rows ? reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) + row_at(r)) + lane % 8
                                   : nullptr;
            }
            uint4 x[S::kChunks][8];
#pragma unroll
            for (int k = 0; k < S::kChunks; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[k][i] = make_uint4(0, 0, 0, 0);
                    if (from[i] && GDN_IN(from[i] + k * 8, 16, bq, st)) x[k][i] = from[i][k * 8];
                }
            // by way of shared memory (rows of 128 bytes, 16-byte units swizzled): a
            // thread's own row, far from its neighbour's, would be 32 lines a load
            char *pass = base + (pass_s - k_s) + warp * 4096;
#pragma unroll
            for (int k = 0; k < S::kChunks; ++k) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = i * 4 + lane / 8;
                    *reinterpret_cast<uint4 *>(pass + r * 128 + (lane % 8 ^ r % 8) * 16) = x[k][i];
                }
                __syncwarp();
                unsigned y[32];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(pass + lane * 128 + (i ^ lane % 8) * 16);
                    y[4 * i] = u.x, y[4 * i + 1] = u.y, y[4 * i + 2] = u.z, y[4 * i + 3] = u.w;
                }
                gdntc::tmem_st32(tmem + lane_addr + kQCol + k * 32, y);
                __syncwarp();
            }
            gdntc::tmem_wait_st();
            gdntc::fence_before_sync();
            if (tid == 0) c.odd_nodes[(seg + 1) & 3] = 0;
            __syncwarp();
            if (lane == 0) bar_arrive(saddr(&c.q_full));
            if (work.left > 0) {  // the next segment's queries on their way to L2
                Work peek = work;
                const Segment n = next_segment<kN>(a, plan, peek);
                const int nkv = quotient(n.unit, plan.by_m_groups), r = ((n.unit - nkv * plan.m_groups) * P + rank) * kM + tid;
                if (r < rows)
                    gdndev::prefetch_l2_range(static_cast<const __nv_bfloat16 *>(a.q) + row_offset(a, plan, n.b, nkv, r) * D, D * 2, 0, 1);
            }
            unsigned long long path = 0;
            if ((s.tile0 + s.n) * kN > ctx && live) {  // a tile with drafted slots
                const int t = quotient(row, plan.by_group) + 1;
                if (a.parent) {
                    for (int i = t; i > 0;) {
                        path |= 1ull << (i - 1);
                        const int32_t *f = a.parent + (size_t)s.b * (a.n_tok + 1) + i;
                        int p = GDN_IN(f, 4, bpar, st) ? *f : i - 1;
                        if (p < 0 || p >= i) {
                            p = i - 1;
                            if (st) atomicOr(st, GDN_DEV_TREE);
                        }
                        i = p;
                    }
                } else {
                    path = t == 64 ? ~0ull : (1ull << t) - 1;
                }
            }
            float m = -INFINITY;
            float2 sum = make_float2(0.f, 0.f);
            for (int j = 0; j < s.n; ++j, ++g) {
                const int slot = g & 1, tile = s.tile0 + j;
                const bool edge = (tile + 1) * kN > ctx;
                ok = wait(saddr(&c.s_full[slot]), (g >> 1) & 1, quit);
                if (edge) ok = ok && wait(saddr(&c.v_full[g % kStages]), (g / kStages) & 1, quit);
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                gdntc::fence_after_sync();
                const unsigned s_addr = tmem + lane_addr + kSCol + slot * kN;
                if (warp_live) {
                    unsigned x[kN / 32][32];
#pragma unroll
                    for (int k = 0; k < kN / 32; ++k) gdntc::tmem_ld32(s_addr + k * 32, x[k]);
                    gdntc::tmem_wait_ld();
                    if (edge) {
#pragma unroll
                        for (int k = 0; k < kN / 32; ++k) {
                            const unsigned seen = seen32(tile * kN + k * 32 - ctx, path);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!(seen >> i & 1)) x[k][i] = 0xff800000u;  // -inf
                        }
                    }
                    float tops[8];  // eight chains: a single one would wait on itself
#pragma unroll
                    for (int i = 0; i < 8; ++i) tops[i] = -INFINITY;
#pragma unroll
                    for (int k = 0; k < kN / 32; ++k)
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            tops[i / 2 & 7] = max3(tops[i / 2 & 7], __uint_as_float(x[k][i]), __uint_as_float(x[k][i + 1]));
                    float top = fmaxf(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])),
                                      fmaxf(fmaxf(tops[4], tops[5]), fmaxf(tops[6], tops[7])));
                    if (j == 0) {
                        m = top;
                    } else {
                        const bool far = (top - m) * scale > 8.f || (m == -INFINITY && top > m);
                        if (__any_sync(~0u, far)) {
                            const float f = far ? ex2((m - top) * scale) : 1.f;
                            ok = __all_sync(~0u, sums_done(g - 1));
                            if (!ok) break;
                            gdntc::fence_after_sync();
#pragma unroll 1
                            for (int k = 0; k < D; k += 32) {
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
                        }
                    }
                    const float mc = m == -INFINITY ? 0.f : m * scale;  // nothing seen yet: every weight is 0
                    const float2 sc = make_float2(scale, scale), mn = make_float2(-mc, -mc);
                    float2 part[4] = {};
#pragma unroll
                    for (int k = 0; k < kN / 64; ++k) {
                        unsigned p[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const unsigned *y = &x[2 * k + i / 16][i % 16 * 2];
                            float2 f = fma2(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), sc, mn);
                            f.x = ex2(f.x);
                            f.y = ex2(f.y);
                            part[i & 3] = add2(part[i & 3], f);
                            p[i] = pack_bf16(f.x, f.y);
                        }
                        gdntc::tmem_st32(s_addr + k * 32, p);
                    }
                    sum = add2(sum, add2(add2(part[0], part[1]), add2(part[2], part[3])));
                    gdntc::tmem_wait_st();
                }
                if (edge) {
                    // v past the last slot becomes zeros, and so does what is no number
                    // among the drafted nodes' values: 0 x NaN must not reach the rows
                    // that do not see them; those that do get it back at the end
                    char *v = base + (v_s - k_s) + (g % kStages) * S::kTileBytes;
                    const int lo = max(0, ctx - tile * kN);
                    for (int i = tid; i < (kN - lo) * S::kChunks * 8; i += 128) {
                        const int r = lo + i / (S::kChunks * 8), u = i % (S::kChunks * 8);
                        uint4 *p = reinterpret_cast<uint4 *>(v + (u / 8) * (kN * 128) + r * 128 + (u % 8) * 16);
                        const int node = tile * kN + r - ctx;
                        if (node >= a.n_tok) {
                            *p = make_uint4(0, 0, 0, 0);
                            continue;
                        }
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
                            atomicOr(&c.odd_nodes[seg & 3], 1ull << node);
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
                const bool whole = s.n == s.tiles;
                const float total = sum.x + sum.y, inv = whole ? 1.f / total : 1.f;
                const unsigned long long odd = *(volatile unsigned long long *)&c.odd_nodes[seg & 3] & path;
                const size_t piece = 2 * share + (first_segment ? 0 : 1);
                const int pr = rank * kM + tid;
                const Buf bo{pieces.o, (size_t)2 * plan.blocks * P * kM * D * 4}, bms{pieces.ms, (size_t)2 * plan.blocks * P * kM * 8};
                if (!whole && tid == 0 && rank == 0) pieces.unit[piece] = s.b * plan.units + s.unit;
                if (!whole && live) {
                    float2 *f = pieces.ms + piece * (P * kM) + pr;
                    if (GDN_IN(f, 8, bms, st)) *f = make_float2(m == -INFINITY ? m : m * scale, total);
                }
#pragma unroll 1
                for (int k = 0; k < D; k += 32) {
                    unsigned o[32];
                    __syncwarp();
                    gdntc::tmem_ld32(tmem + lane_addr + k, o);
                    gdntc::tmem_wait_ld();
                    if (!live) continue;
                    float f[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(o[i]) * inv;
                    if (odd) {
                        const Buf bt{a.table, (size_t)a.batch * a.width * 4},
                            bv{a.v_pages, ((size_t)a.n_pages * a.h_kv << a.page_shift) * D * 2};
                        for (unsigned long long left = odd; left; left &= left - 1) {
                            const int at = ctx + __ffsll((long long)left) - 1;
                            const int32_t *e = a.table + (size_t)s.b * a.width + (at >> a.page_shift);
                            const int page = GDN_IN(e, 4, bt, st) ? *e : -1;
                            if (page < 0 || page >= a.n_pages) continue;
                            const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v_pages) +
                                                     ((((size_t)page * a.h_kv + kv) << a.page_shift) +
                                                      (at & ((1 << a.page_shift) - 1))) * D + k;
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const float x = GDN_IN(v + i, 2, bv, st) ? __bfloat162float(v[i]) : 0.f;
                                if (!(fabsf(x) < INFINITY)) f[i] += x;
                            }
                        }
                    }
                    if (whole) {
                        __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(a.out) + q_row + k;
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            if (GDN_IN(to + i, 16, bout, st))
                                *reinterpret_cast<uint4 *>(to + i) =
                                    make_uint4(pack_bf16(f[i], f[i + 1]), pack_bf16(f[i + 2], f[i + 3]),
                                               pack_bf16(f[i + 4], f[i + 5]), pack_bf16(f[i + 6], f[i + 7]));
                    } else {
                        float4 *to = pieces.o + (piece * (D / 4) + k / 4) * (P * kM) + pr;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (GDN_IN(to + i * (P * kM), 16, bo, st))
                                to[i * (P * kM)] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
                    }
                }
            }
            __syncwarp();
            gdntc::fence_before_sync();
            ++seg;
        }
    }
    // requests that are left out get zeros
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x)
        if (gdnattn::slots_of(a, b) == 0) {
            const size_t units16 = (size_t)a.n_tok * a.h_q * D / 8;
            uint4 *to = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out)) + b * units16;
            const Buf bout{a.out, (size_t)a.batch * units16 * 16};
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

// The shared units' pieces added up. An item is 32 rows x 8 columns of one
// unit; a block's four warps are 4 / `share` items of `share` warps, which take
// the item's pieces in turn, four at a time: a piece at a time would wait for
// memory with each. Small blocks of few registers: all of them fit the GPU at
// once. 8 us for 9 to 14 MB of pieces, bound by its three round trips to memory and
// the fetching of its code. Measured and dropped: finding a unit's pieces once for
// a block of eight warps (12 us), all maxima before the first sum (19 us for 38
// pieces), the sums by the last block of attend to finish, behind an atomic count
// (the same 75 us in all for 16 requests' spans, 14.9 instead of 10.6 for one
// token). There are at most min(units, blocks - 1) shared units: with fewer units
// than blocks an item's unit is its index, otherwise it is the one cut by the
// beginning of block `index`, if that is its first cut.
constexpr int kJoinWarps = 4;

template <int D, int P>
__global__ void __launch_bounds__(kJoinWarps * 32, 8)
join_pieces(const __grid_constant__ AttnArgs a, const __grid_constant__ Plan plan, const __grid_constant__ Pieces pieces,
            int share, int items, int chunks, bool by_unit) {
    constexpr int kRows = P * kM, kCols = D / 8, kAhead = 4;
    __shared__ float4 part[kJoinWarps][2][32];
    __shared__ float top[kJoinWarps][32], total[kJoinWarps][32];
    __shared__ unsigned short list[kJoinWarps][2 * kMaxBlocks];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int item = (blockIdx.x * kJoinWarps + warp) / share, which = warp % share;
    const int d4 = item % kCols * 2, chunk = item / kCols % chunks, index = item / kCols / chunks;
    const int pr = chunk * 32 + lane;
    int32_t *st = a.status;
    const Buf bo{pieces.o, (size_t)2 * plan.blocks * kRows * D * 4}, bms{pieces.ms, (size_t)2 * plan.blocks * kRows * 8},
        bout{a.out, (size_t)a.batch * a.n_tok * a.h_q * D * 2};
    gdndev::pdl_wait();
    gdndev::pdl_launch_dependents();
    // the unit's pieces, from the blocks' notes
    int note[kNotes], unit = index;
#pragma unroll
    for (int i = 0; i < kNotes; ++i) {
        const int p = i * 32 + lane;
        note[i] = p < 2 * plan.blocks ? __ldcg(pieces.unit + p) : -1;
    }
    // (the unit's number beside the notes, not after them)
    if (!by_unit) unit = index < plan.blocks ? __ldcg(pieces.unit + 2 * index) : -1;
    int n = 0;
    if (unit >= 0) {
#pragma unroll
        for (int i = 0; i < kNotes; ++i) {
            const unsigned here = __ballot_sync(~0u, note[i] == unit);
            if (note[i] == unit) list[warp][n + __popc(here & ((1u << lane) - 1))] = (unsigned short)(i * 32 + lane);
            n += __popc(here);
        }
    }
    __syncwarp();
    // below two pieces, one block had the whole unit and has written it
    const bool mine = item < items && n >= 2 && (by_unit || list[warp][1] == 2 * index);
    const int b = mine ? unit / plan.units : 0, in_request = unit - b * plan.units, kv = mine ? in_request / plan.m_groups : 0;
    const int row = (in_request - kv * plan.m_groups) * kRows + pr;
    const bool live = mine && row < plan.rows;
    float m = -INFINITY, sum = 0.f;
    float4 o[2] = {};
    for (int k0 = live ? which : n; k0 < n; k0 += share * kAhead) {
        float2 ms[kAhead];
        float4 x[kAhead][2];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            ms[u] = make_float2(-INFINITY, 0.f);
            x[u][0] = x[u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k0 + u * share < n) {
                const size_t piece = list[warp][k0 + u * share];
                const float2 *fm = pieces.ms + piece * kRows + pr;
                const float4 *fo = pieces.o + (piece * (D / 4) + d4) * kRows + pr;
                if (GDN_IN(fm, 8, bms, st)) ms[u] = __ldcg(fm);
                if (GDN_IN(fo, 16, bo, st)) x[u][0] = __ldcg(fo);
                if (GDN_IN(fo + kRows, 16, bo, st)) x[u][1] = __ldcg(fo + kRows);
            }
        }
        float m2 = m;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) m2 = fmaxf(m2, ms[u].x);
        const float f0 = m == -INFINITY ? 0.f : ex2(m - m2);
        sum *= f0;
#pragma unroll
        for (int i = 0; i < 2; ++i) o[i] = make_float4(o[i].x * f0, o[i].y * f0, o[i].z * f0, o[i].w * f0);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (ms[u].x == -INFINITY && ms[u].y == 0.f) continue;  // nothing there that the row sees
            const float f = ms[u].x == m2 ? 1.f : ex2(ms[u].x - m2);
            sum = fmaf(ms[u].y, f, sum);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                o[i] = make_float4(fmaf(x[u][i].x, f, o[i].x), fmaf(x[u][i].y, f, o[i].y), fmaf(x[u][i].z, f, o[i].z),
                                   fmaf(x[u][i].w, f, o[i].w));
        }
        m = m2;
    }
    top[warp][lane] = m;
    total[warp][lane] = sum;
    part[warp][0][lane] = o[0];
    part[warp][1][lane] = o[1];
    __syncthreads();
    if (!live || which != 0) return;
    float mm = -INFINITY, l = 0.f;
    for (int w = warp; w < warp + share; ++w) mm = fmaxf(mm, top[w][lane]);
    o[0] = o[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = warp; w < warp + share; ++w) {
        const float tw = top[w][lane];
        if (tw == -INFINITY && total[w][lane] == 0.f) continue;
        const float f = tw == mm ? 1.f : ex2(tw - mm);
        l = fmaf(total[w][lane], f, l);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 x = part[w][i][lane];
            o[i] = make_float4(fmaf(x.x, f, o[i].x), fmaf(x.y, f, o[i].y), fmaf(x.z, f, o[i].z), fmaf(x.w, f, o[i].w));
        }
    }
    const float inv = 1.f / l;
    __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(a.out) + row_offset(a, plan, b, kv, row) * D + d4 * 4;
    if (GDN_IN(to, 16, bout, st))
        *reinterpret_cast<uint4 *>(to) = make_uint4(pack_bf16(o[0].x * inv, o[0].y * inv), pack_bf16(o[0].z * inv, o[0].w * inv),
                                                    pack_bf16(o[1].x * inv, o[1].y * inv), pack_bf16(o[1].z * inv, o[1].w * inv));
}

using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                            const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Encode encoder() {
    static Encode found = nullptr;
    if (!found) {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) == cudaSuccess &&
            r == cudaDriverEntryPointSuccess)
            found = reinterpret_cast<Encode>(f);
    }
    return found;
}

// One layer's pool as [n_pages * h_kv][page_tokens][D], in boxes of 64 columns
// and at most kN rows of one page and head.
bool pool_map(CUtensorMap *map, const attn_dims *d, const void *pool, int kn) {
    const Encode encode = encoder();
    if (!encode) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d->d_head, (cuuint64_t)d->page_tokens, (cuuint64_t)d->n_pages * d->h_kv};
    const cuuint64_t strides[2] = {(cuuint64_t)d->d_head * 2, (cuuint64_t)d->page_tokens * d->d_head * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)(d->page_tokens < kn ? d->page_tokens : kn), 1}, step[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(pool), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int block_count() {
    const int sms = gdnhost::sm_count();
    return sms <= 0 ? 152 : sms < kMaxBlocks ? sms : kMaxBlocks;
}

// Blocks side by side on the same tiles: two where there is more than one M tile.
int pair(const attn_dims *d, int n_tok) { return n_tok * (d->h_q / d->h_kv) > kM ? 2 : 1; }

template <int D, int P>
int launch(const attn_dims *d, const AttnArgs &a, void *ws, cudaStream_t st) {
    using S = Shape<D>;
    static bool set[256] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return GDN_ERR_CUDA;
    if (!set[dev]) {
        if (cudaFuncSetAttribute(attend<D, P>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem) != cudaSuccess)
            return GDN_ERR_CUDA;
        set[dev] = true;
    }
    CUtensorMap k_map, v_map;
    if (!pool_map(&k_map, d, a.k_pages, S::kN) || !pool_map(&v_map, d, a.v_pages, S::kN)) return GDN_ERR_CUDA;
    const int blocks = block_count() / P;
    char *at = static_cast<char *>(ws);
    const size_t rows_of_pieces = (size_t)2 * blocks * P * kM;
    const Pieces pieces{reinterpret_cast<float4 *>(at), reinterpret_cast<float2 *>(at + rows_of_pieces * D * 4),
                        reinterpret_cast<int *>(at + rows_of_pieces * (D * 4 + 8))};
    const int group = a.h_q / a.h_kv, rows = a.n_tok * group, m_groups = (rows + P * kM - 1) / (P * kM);
    auto by = [](int n) { return (unsigned)(((1ull << 32) + n - 1) / n); };
    const Plan plan{group, rows, m_groups, a.h_kv * m_groups, blocks, by(group), by(m_groups), by(blocks)};
    if (gdndev::launch_pdl(attend<D, P>, dim3(blocks * P), dim3(S::kThreads), S::kSmem, st, k_map, v_map, a, plan, pieces) != cudaSuccess)
        return GDN_ERR_CUDA;
    // a unit has about blocks / units pieces, and one more
    const int64_t units = (int64_t)a.batch * plan.units;
    const bool by_unit = units < blocks;
    const int indexes = by_unit ? (int)units : blocks, per_unit = blocks / indexes + 1;
    const int share = per_unit <= 4 ? 1 : per_unit <= 8 ? 2 : 4;
    const int chunks = ((rows < P * kM ? rows : P * kM) + 31) / 32, items = indexes * chunks * (D / 8);
    return gdndev::launch_pdl(join_pieces<D, P>, dim3((items * share + kJoinWarps - 1) / kJoinWarps), dim3(kJoinWarps * 32), 0, st, a, plan, pieces, share, items,
                              chunks, by_unit) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

namespace gdnattn {

bool tc_fits(const attn_dims *d, int n_tok) {
    // tiles of 64 slots (128-slot tiles and pairs of M tiles are fewer): Work::off
    // counts a request's in an int, Work::left a block's share of all (16 blocks at least)
    const int64_t rows = (int64_t)n_tok * (d->h_q / d->h_kv), slot_tiles = ((int64_t)d->table_width * d->page_tokens + 63) / 64;
    const int64_t tiles = slot_tiles * d->h_kv * ((rows + kM - 1) / kM);
    return tiles < (1LL << 31) && tiles * d->batch < (1LL << 34);
}

size_t tc_workspace(const attn_dims *d, int n_tok) {
    const size_t p = pair(d, n_tok), blocks = block_count() / p;
    return 2 * blocks * (p * kM * (d->d_head * 4 + 8) + 4);
}

int tc_launch(const attn_dims *d, const AttnArgs &a, void *ws, cudaStream_t st) {
    if (pair(d, a.n_tok) == 2)
        return a.d == 64 ? launch<64, 2>(d, a, ws, st) : a.d == 128 ? launch<128, 2>(d, a, ws, st) : launch<256, 2>(d, a, ws, st);
    return a.d == 64 ? launch<64, 1>(d, a, ws, st) : a.d == 128 ? launch<128, 1>(d, a, ws, st) : launch<256, 1>(d, a, ws, st);
}

}  // namespace gdnattn
