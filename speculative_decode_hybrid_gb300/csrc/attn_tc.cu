// Attention of a drafted span over the paged cache on the tensor cores
// (attn_verify_span / attn_tree_verify with GDN_BF16).
//
// The rows of one key/value head's product are the span's nodes times the query
// heads of the group: 128 rows are one M tile, and a block holds W of them
// (two, where the head is at most 128 wide and there are more than 128 rows).
// For each tile of kN slots
//   S = Q K^T        tcgen05, operands in shared memory, S in tensor memory
//   P = 2^(c S - m)  one thread per row, rounded to bf16, over S's columns
//   O += P V         tcgen05, P read from tensor memory, V MN-major in shared
//                    memory as it lies in the page
// in one pass, the softmax relative to a reference m that follows the running
// maximum only when it falls more than 2^8 behind (then O is rescaled in tensor
// memory): the weights stay below 2^8, and the final division by the sum of
// the same weights makes the result independent of m.
//
// Warps: 4 per M tile for the softmax, one that keeps the TMA loads of the next
// tiles in flight (a page's rows of one head are a box of a 3-d tensor map, so
// a tile is gathered page by page), one that issues the products.
//
// Work is split over the whole flattened list of (request, head, M tiles, slot
// tile): block i of n takes the i-th n-th of it, whatever the requests'
// lengths. Pieces of a unit that several blocks share go to the workspace, and
// join_pieces adds them up on the scale of their largest maximum.
//
// Bound by the bytes of K and V while the rows are few (4 kN D bytes a tile
// against 2 x 128 x kN x D x 2 W operations), and by the exponentials once two
// M tiles are full.
#include <cuda.h>
#include <cuda_runtime.h>

#include "attn_common.cuh"
#include "attn_host.h"
#include "gdn_host.h"
#include "gdn_tc.cuh"
#include "gdnspec.h"

namespace {

using gdnattn::AttnArgs;
using gdndev::Buf;

constexpr int kM = 128;                    // rows of an M tile
constexpr unsigned long long kGiveUpNs = 1000000000ull;  // a wait's limit

// Smallest power of two of tensor-memory columns: all 512, one block per SM.
constexpr int kTmemCols = 512;

template <int D, int W>
struct Shape {
    static constexpr int kN = D == 256 ? 64 : 128;       // slots of a tile
    static constexpr int kChunks = D / 64;               // 128-byte column chunks of a row
    static constexpr int kStages = D == 64 ? 4 : D == 128 && W == 1 ? 3 : 2;
    static constexpr unsigned kTileBytes = kN * D * 2;   // of K, and of V
    static constexpr unsigned kQBytes = kM * D * 2;      // of one M tile
    static constexpr int kSlots = 2;                     // S buffers: one per M tile, or two in turn
    static constexpr int kThreads = W * 128 + 64;
    static constexpr unsigned kSmem = W * kQBytes + 2 * kStages * kTileBytes + 1024;
    static_assert(W * D + kSlots * kN <= kTmemCols, "tensor memory");
};

struct Work {
    int b, off, left;  // request, tiles of it already dealt out, tiles of this block still to come
};

struct Segment {
    int b, unit, tile0, n, tiles, slots;
};

template <int kN>
__device__ __forceinline__ Segment next_segment(const AttnArgs &a, int units, Work &w) {
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
    if (w.off == s.tiles * units) ++w.b, w.off = 0;
    return s;
}

// Tiles of all requests before `upto`, times the units of one: by one warp.
template <int kN>
__device__ __forceinline__ long long tiles_before(const AttnArgs &a, int units, int upto) {
    long long n = 0;
    for (int b = threadIdx.x & 31; b < upto; b += 32) n += (gdnattn::slots_of(a, b) + kN - 1) / kN;
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(~0u, n, o);
    return n * units;
}

__device__ __forceinline__ long long range_start(long long total, int block, int blocks) { return total * block / blocks; }

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
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
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

struct Pieces {
    float4 *o;    // [2 blocks][D / 4][W * 128]
    float2 *ms;   // [2 blocks][W * 128]: reference maximum in powers of two, sum
};

template <int D, int W>
struct Control {
    static constexpr int kStages = Shape<D, W>::kStages;
    unsigned long long k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
    unsigned long long s_full[2], p_full[2], pv_done[2], q_full, drain;
    unsigned long long odd_nodes[4];  // drafted nodes with a value of v that is no number, by segment
    Work work;
    unsigned tmem;
    int quit;
};

template <int D, int W>
__global__ void __launch_bounds__(Shape<D, W>::kThreads, 1)
attend(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
       const __grid_constant__ AttnArgs a, const __grid_constant__ Pieces pieces) {
    using S = Shape<D, W>;
    constexpr int kN = S::kN, kStages = S::kStages;
    extern __shared__ char raw[];
    __shared__ Control<D, W> c;
    char *base = raw + ((1024 - (saddr(raw) & 1023)) & 1023);
    const unsigned q_s = saddr(base), k_s = q_s + W * S::kQBytes, v_s = k_s + kStages * S::kTileBytes;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = a.h_q / a.h_kv, rows = a.n_tok * group;
    const int m_groups = (rows + W * kM - 1) / (W * kM), units = a.h_kv * m_groups;
    int32_t *st = a.status;
    constexpr int kTmaWarp = W * 4, kMmaWarp = W * 4 + 1;

    if (warp == kMmaWarp) gdntc::tmem_alloc<kTmemCols>(&c.tmem);
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
        bar_init(saddr(&c.q_full), W * 4);
        bar_init(saddr(&c.drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        c.quit = 0;
        for (int i = 0; i < 4; ++i) c.odd_nodes[i] = 0;
    }
    gdndev::pdl_launch_dependents();
    gdndev::pdl_wait();
    if (warp == 0) {
        // this block's share of the list, and the request in which it begins
        const long long total = tiles_before<kN>(a, units, a.batch);
        const long long lo = range_start(total, blockIdx.x, gridDim.x), hi = range_start(total, blockIdx.x + 1, gridDim.x);
        long long before = 0;
        for (int b0 = 0; b0 < a.batch; b0 += 32) {
            const int b = b0 + lane;
            const long long n = b < a.batch ? (long long)((gdnattn::slots_of(a, b) + kN - 1) / kN) * units : 0;
            long long x = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(~0u, x, o);
                if (lane >= o) x += y;
            }
            if (lo >= before + x - n && lo < before + x) c.work = {b, (int)(lo - (before + x - n)), (int)(hi - lo)};
            before += __shfl_sync(~0u, x, 31);
            if (lo < before) break;
        }
        if (lane == 0 && hi == lo) c.work = {0, 0, 0};
        if (blockIdx.x == 0 && st)
            for (int b = lane; b < a.batch; b += 32)
                if (gdnattn::slots_of(a, b) == 0) atomicOr(st, GDN_DEV_LENGTH);
    }
    gdntc::fence_before_sync();
    __syncthreads();
    gdntc::fence_after_sync();
    const unsigned tmem = c.tmem;
    Work work = c.work;
    volatile int *quit = &c.quit;
    // tensor-memory columns: O of each M tile, then the S buffers
    constexpr unsigned kSCol = W * D;

    if (warp == kTmaWarp) {
        int g = 0;  // tiles so far
        const int page_rows = min(1 << a.page_shift, kN), boxes = kN / page_rows;
        const unsigned box_bytes = page_rows * 128u;
        const int mine = lane / S::kChunks, chunk = lane % S::kChunks;  // this lane's page of the tile, and its column chunk
        const Buf bt{a.table, (size_t)a.batch * a.width * 4};
        bool ok = true;
        while (work.left > 0 && ok) {
            const Segment s = next_segment<kN>(a, units, work);
            const int kv = s.unit / m_groups;
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
    } else if (warp == kMmaWarp) {
        if (lane == 0) {
            constexpr unsigned kIdS = gdntc::idesc_bf16(kM, kN, false), kIdO = gdntc::idesc_bf16(kM, D, true);
            int g = 0;
            unsigned seg = 0;
            bool ok = true;
            auto scores = [&](int tile, int w, int slot) {  // S = Q K^T of one M tile
                const unsigned k = k_s + (tile % kStages) * S::kTileBytes, q = q_s + w * S::kQBytes;
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    gdntc::mma_bf16_ss(tmem + kSCol + slot * kN, gdntc::smem_desc_sw128(q + (i / 4) * (kM * 128) + (i % 4) * 32),
                                       gdntc::smem_desc_sw128(k + (i / 4) * (kN * 128) + (i % 4) * 32), kIdS, i > 0);
                gdntc::mma_commit(saddr(&c.s_full[slot]));
            };
            auto sums = [&](int tile, int w, int slot, bool first) {  // O += P V
                const unsigned v = v_s + (tile % kStages) * S::kTileBytes;
#pragma unroll
                for (int i = 0; i < kN / 16; ++i)
                    gdntc::mma_bf16_ts(tmem + w * D, tmem + kSCol + slot * kN + i * 8,
                                       gdntc::smem_desc_sw128_mn(v + i * 2048, kN * 128), kIdO, !first || i > 0);
                gdntc::mma_commit(saddr(&c.pv_done[slot]));
            };
            auto k_ready = [&](int tile) { return wait(saddr(&c.k_full[tile % kStages]), (tile / kStages) & 1, quit); };
            auto v_ready = [&](int tile) { return wait(saddr(&c.v_full[tile % kStages]), (tile / kStages) & 1, quit); };
            while (work.left > 0 && ok) {
                const Segment s = next_segment<kN>(a, units, work);
                ok = wait(saddr(&c.q_full), seg & 1, quit) && k_ready(g);
                ++seg;
                if (!ok) break;
                gdntc::fence_after_sync();
                for (int w = 0; w < W; ++w) scores(g, w, W == 2 ? w : g & 1);
                gdntc::mma_commit(saddr(&c.k_empty[g % kStages]));
                for (int j = 0; j < s.n && ok; ++j, ++g) {
                    const bool more = j + 1 < s.n;
                    if (W == 1 && more) {
                        ok = k_ready(g + 1);
                        if (!ok) break;
                        gdntc::fence_after_sync();
                        scores(g + 1, 0, (g + 1) & 1);
                        gdntc::mma_commit(saddr(&c.k_empty[(g + 1) % kStages]));
                    }
                    for (int w = 0; w < W; ++w) {
                        const int slot = W == 2 ? w : g & 1;
                        ok = wait(saddr(&c.p_full[slot]), W == 2 ? g & 1 : (g >> 1) & 1, quit) && (w > 0 || v_ready(g));
                        if (!ok) break;
                        gdntc::fence_after_sync();
                        sums(g, w, slot, j == 0);
                        if (w == W - 1) gdntc::mma_commit(saddr(&c.v_empty[g % kStages]));
                        if (W == 2 && more) {
                            if (w == 0) ok = k_ready(g + 1);
                            if (!ok) break;
                            if (w == 0) gdntc::fence_after_sync();
                            scores(g + 1, w, w);
                            if (w == 1) gdntc::mma_commit(saddr(&c.k_empty[(g + 1) % kStages]));
                        }
                    }
                }
            }
            gdntc::mma_commit(saddr(&c.drain));
            wait(saddr(&c.drain), 0, nullptr);  // no product may run on when the columns are freed
        }
        __syncwarp();
    } else {
        const int w = warp / 4, row_in_tile = tid - w * 128;
        const unsigned lane_addr = (unsigned)(warp & 3) << 21;  // 32 lanes each, in bits 16 and up
        const Buf bq{a.q, (size_t)a.batch * a.n_tok * a.h_q * D * 2}, bout{a.out, (size_t)a.batch * a.n_tok * a.h_q * D * 2},
            bpar{a.parent, (size_t)a.batch * (a.n_tok + 1) * 4};
        const float scale = a.scale_log2;
        // With one M tile the scores of tile g are issued before the sums of g - 1,
        // so a tile's scores only tell that the sums of g - 2 are done: a barrier
        // for each S buffer keeps its phases apart.
        auto sums_done = [&](int tile) {
            return wait(saddr(&c.pv_done[W == 2 ? w : tile & 1]), W == 2 ? tile & 1 : (tile >> 1) & 1, quit);
        };
        int g = 0;
        unsigned seg = 0;
        bool ok = true;
        while (work.left > 0 && ok) {
            const bool first_segment = seg == 0;
            const Segment s = next_segment<kN>(a, units, work);
            const int kv = s.unit / m_groups, row0 = (s.unit % m_groups) * W * kM + w * kM, row = row0 + row_in_tile;
            const int ctx = s.slots - a.n_tok;
            // the M tile's queries, swizzled as the descriptors say; the scores of
            // the segment before have been read, so their products are done with q
            for (int i = row_in_tile; i < kM * (D / 8); i += 128) {
                const int r = i / (D / 8), u = i % (D / 8), qr = row0 + r;
                uint4 x = make_uint4(0, 0, 0, 0);
                if (qr < rows) {
                    const uint4 *f = reinterpret_cast<const uint4 *>(
                        static_cast<const __nv_bfloat16 *>(a.q) +
                        (((size_t)s.b * a.n_tok + qr / group) * a.h_q + kv * group + qr % group) * D) + u;
                    if (GDN_IN(f, 16, bq, st)) x = *f;
                }
                *reinterpret_cast<uint4 *>(base + w * S::kQBytes + (u / 8) * (kM * 128) + r * 128 + (((u % 8) ^ (r % 8)) * 16)) = x;
            }
            gdntc::fence_smem_to_async();
            if (w == 0 && row_in_tile == 0) c.odd_nodes[(seg + 1) & 3] = 0;
            __syncwarp();
            if (lane == 0) bar_arrive(saddr(&c.q_full));
            unsigned long long path = 0;
            const bool live = row < rows, warp_live = row0 + (warp & 3) * 32 < rows;
            if ((s.tile0 + s.n) * kN > ctx && live) {  // a tile with drafted slots
                const int t = row / group + 1;
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
                const int slot = W == 2 ? w : g & 1, tile = s.tile0 + j;
                const bool edge = (tile + 1) * kN > ctx;
                ok = wait(saddr(&c.s_full[slot]), W == 2 ? g & 1 : (g >> 1) & 1, quit);
                if (edge && w == 0) ok = ok && wait(saddr(&c.v_full[g % kStages]), (g / kStages) & 1, quit);
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
                    float top = -INFINITY;
#pragma unroll
                    for (int k = 0; k < kN / 32; ++k)
#pragma unroll
                        for (int i = 0; i < 32; ++i) top = fmaxf(top, __uint_as_float(x[k][i]));
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
                                gdntc::tmem_ld32(tmem + lane_addr + w * D + k, o);
                                gdntc::tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                gdntc::tmem_st32(tmem + lane_addr + w * D + k, o);
                            }
                            if (far) m = top;
                            sum.x *= f;
                            sum.y *= f;
                        }
                    }
                    const float mc = m == -INFINITY ? 0.f : m * scale;  // nothing seen yet: every weight is 0
                    const float2 sc = make_float2(scale, scale), mn = make_float2(-mc, -mc);
                    float2 part = make_float2(0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < kN / 64; ++k) {
                        unsigned p[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const unsigned *y = &x[2 * k + i / 16][i % 16 * 2];
                            float2 f = fma2(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), sc, mn);
                            f.x = ex2(f.x);
                            f.y = ex2(f.y);
                            part = add2(part, f);
                            p[i] = pack_bf16(f.x, f.y);
                        }
                        gdntc::tmem_st32(s_addr + k * 32, p);
                    }
                    sum = add2(sum, part);
                    gdntc::tmem_wait_st();
                }
                if (edge && w == 0) {
                    // v past the last slot becomes zeros, and so does what is no number
                    // among the drafted nodes' values: 0 x NaN must not reach the rows
                    // that do not see them; those that do get it back at the end
                    char *v = base + (v_s - q_s) + (g % kStages) * S::kTileBytes;
                    const int lo = max(0, ctx - tile * kN);
                    for (int i = row_in_tile; i < (kN - lo) * S::kChunks * 8; i += 128) {
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
                const size_t out_row = (((size_t)s.b * a.n_tok + row / group) * a.h_q + kv * group + row % group) * D;
                const size_t piece = 2 * blockIdx.x + (first_segment ? 0 : 1);
                const int pr = w * kM + row_in_tile;
                const Buf bo{pieces.o, (size_t)2 * gridDim.x * W * kM * D * 4}, bms{pieces.ms, (size_t)2 * gridDim.x * W * kM * 8};
                if (!whole && live) {
                    float2 *f = pieces.ms + piece * (W * kM) + pr;
                    if (GDN_IN(f, 8, bms, st)) *f = make_float2(m == -INFINITY ? m : m * scale, total);
                }
#pragma unroll 1
                for (int k = 0; k < D; k += 32) {
                    unsigned o[32];
                    __syncwarp();
                    gdntc::tmem_ld32(tmem + lane_addr + w * D + k, o);
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
                        __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(a.out) + out_row + k;
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            if (GDN_IN(to + i, 16, bout, st))
                                *reinterpret_cast<uint4 *>(to + i) =
                                    make_uint4(pack_bf16(f[i], f[i + 1]), pack_bf16(f[i + 2], f[i + 3]),
                                               pack_bf16(f[i + 4], f[i + 5]), pack_bf16(f[i + 6], f[i + 7]));
                    } else {
                        float4 *to = pieces.o + (piece * (D / 4) + k / 4) * (W * kM) + pr;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (GDN_IN(to + i * (W * kM), 16, bo, st))
                                to[i * (W * kM)] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
                    }
                }
            }
            __syncwarp();
            gdntc::fence_before_sync();
            ++seg;
        }
    }
    __syncthreads();
    if (c.quit && tid == 0 && st) atomicOr(st, GDN_DEV_SCHED);
    if (warp == kMmaWarp) {
        gdntc::fence_after_sync();
        gdntc::tmem_dealloc<kTmemCols>(tmem);
    }
}

// grid (B * units * row chunks, D / 32): 32 rows of one unit, 32 columns; the
// eight warps take its pieces in turn and their sums meet in shared memory.
template <int D, int W>
__global__ void __launch_bounds__(256) join_pieces(const __grid_constant__ AttnArgs a, const __grid_constant__ Pieces pieces, int blocks) {
    constexpr int kN = Shape<D, W>::kN, kRows = W * kM;
    __shared__ float4 part[8][8][32];
    __shared__ float top[8][32], total[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d4 = blockIdx.y * 8;
    const int group = a.h_q / a.h_kv, rows = a.n_tok * group;
    const int m_groups = (rows + kRows - 1) / kRows, units = a.h_kv * m_groups, chunks = (min(rows, kRows) + 31) / 32;
    const int chunk = blockIdx.x % chunks, unit = blockIdx.x / chunks % units, b = blockIdx.x / chunks / units;
    const int pr = chunk * 32 + lane, row = unit % m_groups * kRows + pr;
    int32_t *st = a.status;
    const Buf bo{pieces.o, (size_t)2 * blocks * kRows * D * 4}, bms{pieces.ms, (size_t)2 * blocks * kRows * 8},
        bout{a.out, (size_t)a.batch * a.n_tok * a.h_q * D * 2};
    gdndev::pdl_wait();
    const int slots = gdnattn::slots_of(a, b), tiles = (slots + kN - 1) / kN;
    const bool live = row < rows;
    __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(a.out) +
                        (((size_t)b * a.n_tok + row / group) * a.h_q + unit / m_groups * group + row % group) * D + d4 * 4 + warp * 4;
    if (tiles == 0) {  // left out
        if (live && GDN_IN(to, 8, bout, st)) *reinterpret_cast<uint2 *>(to) = make_uint2(0, 0);
        return;
    }
    const long long all = tiles_before<kN>(a, units, a.batch);
    const long long first = tiles_before<kN>(a, units, b) + (long long)unit * tiles, last = first + tiles - 1;
    const int c0 = (int)(((first + 1) * blocks - 1) / all), c1 = (int)(((last + 1) * blocks - 1) / all);
    if (c0 == c1) return;  // one block had the whole unit and has written it
    float m = -INFINITY, sum = 0.f;
    float4 o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = c0 + warp; c <= c1; c += 8) {
        const long long start = range_start(all, c, blocks);
        if (start == range_start(all, c + 1, blocks)) continue;  // no tiles
        const size_t piece = 2 * c + (start < first ? 1 : 0);    // a block's first piece, or its last
        const float2 *fm = pieces.ms + piece * kRows + pr;
        const float4 *fo = pieces.o + (piece * (D / 4) + d4) * kRows + pr;
        if (!live) continue;
        const float2 ms = GDN_IN(fm, 8, bms, st) ? __ldcg(fm) : make_float2(-INFINITY, 0.f);
        float4 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = GDN_IN(fo + i * kRows, 16, bo, st) ? __ldcg(fo + i * kRows) : make_float4(0.f, 0.f, 0.f, 0.f);
        if (ms.x == -INFINITY && ms.y == 0.f) continue;  // nothing there that the row sees
        const float m2 = fmaxf(m, ms.x), wo = m == -INFINITY ? 0.f : ex2(m - m2), wn = ms.x == m2 ? 1.f : ex2(ms.x - m2);
        m = m2;
        sum = sum * wo + ms.y * wn;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            o[i].x = o[i].x * wo + x[i].x * wn;
            o[i].y = o[i].y * wo + x[i].y * wn;
            o[i].z = o[i].z * wo + x[i].z * wn;
            o[i].w = o[i].w * wo + x[i].w * wn;
        }
    }
    top[warp][lane] = m;
    total[warp][lane] = sum;
#pragma unroll
    for (int i = 0; i < 8; ++i) part[warp][i][lane] = o[i];
    __syncthreads();
    // warp i joins the eight sums of column group i
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < 8; ++w) mm = fmaxf(mm, top[w][lane]);
    float l = 0.f;
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        const float tw = top[w][lane];
        if (tw == -INFINITY && total[w][lane] == 0.f) continue;
        const float f = tw == mm ? 1.f : ex2(tw - mm);
        const float4 x = part[w][warp][lane];
        l += total[w][lane] * f;
        r.x += x.x * f, r.y += x.y * f, r.z += x.z * f, r.w += x.w * f;
    }
    const float inv = 1.f / l;
    if (live && GDN_IN(to, 8, bout, st))
        *reinterpret_cast<uint2 *>(to) = make_uint2(pack_bf16(r.x * inv, r.y * inv), pack_bf16(r.z * inv, r.w * inv));
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
    return sms > 0 ? sms : 152;
}

int m_tiles(const attn_dims *d, int n_tok) {
    return d->d_head < 256 && n_tok * (d->h_q / d->h_kv) > kM ? 2 : 1;
}

template <int D, int W>
int launch(const attn_dims *d, const AttnArgs &a, void *ws, cudaStream_t st) {
    using S = Shape<D, W>;
    static bool set[256] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return GDN_ERR_CUDA;
    if (!set[dev]) {
        if (cudaFuncSetAttribute(attend<D, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem) != cudaSuccess)
            return GDN_ERR_CUDA;
        set[dev] = true;
    }
    CUtensorMap k_map, v_map;
    if (!pool_map(&k_map, d, a.k_pages, S::kN) || !pool_map(&v_map, d, a.v_pages, S::kN)) return GDN_ERR_CUDA;
    const int blocks = block_count();
    const Pieces pieces{static_cast<float4 *>(ws),
                        reinterpret_cast<float2 *>(static_cast<char *>(ws) + (size_t)2 * blocks * W * kM * D * 4)};
    if (gdndev::launch_pdl(attend<D, W>, dim3(blocks), dim3(S::kThreads), S::kSmem, st, k_map, v_map, a, pieces) != cudaSuccess)
        return GDN_ERR_CUDA;
    const int rows = a.n_tok * (a.h_q / a.h_kv), in_unit = rows < W * kM ? rows : W * kM;
    const int64_t units = (int64_t)a.batch * a.h_kv * ((rows + W * kM - 1) / (W * kM));
    return gdndev::launch_pdl(join_pieces<D, W>, dim3((unsigned)(units * ((in_unit + 31) / 32)), D / 32), dim3(256), 0, st, a,
                              pieces, blocks) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

namespace gdnattn {

size_t tc_workspace(const attn_dims *d, int n_tok) {
    return (size_t)2 * block_count() * m_tiles(d, n_tok) * kM * (d->d_head * 4 + 8);
}

int tc_launch(const attn_dims *d, const AttnArgs &a, void *ws, cudaStream_t st) {
    if (a.d == 256) return launch<256, 1>(d, a, ws, st);
    if (m_tiles(d, a.n_tok) == 2) return a.d == 64 ? launch<64, 2>(d, a, ws, st) : launch<128, 2>(d, a, ws, st);
    return a.d == 64 ? launch<64, 1>(d, a, ws, st) : launch<128, 1>(d, a, ws, st);
}

}  // namespace gdnattn
