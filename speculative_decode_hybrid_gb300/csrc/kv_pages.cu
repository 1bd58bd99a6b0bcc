// The paged key/value cache between steps: the accepted path's rows moved
// together (kv_commit_path), pages given back and taken (kv_pages_resize),
// requests forked (kv_pages_fork). (lucebox PR #506, Summary, and openinfer
// PR #626, What Changed: the committed context's KV beside the recurrent
// state.)
//
// All are bound by latency: a chain of lookups (lengths, parents, table entries)
// stands before the first moved byte. Commit of 16 requests' paths of 11 in 16
// layers of 8 heads of 128 bf16 (23 MB moved) 7.5 us, with slices and rows found
// by multiplications and 64 registers (13 us with divisions); a fork's copy of 16
// tails in 8 layers (13 MB) 6 us; the taking of their pages, one block and five
// dependent reads, 6 us. kv_pages_resize is one block too, whose warps walk all
// entries of their requests' rows, twice where pages are missing: 4.7 us for 32
// rows of 150 entries that grow or shrink by a page, 6.5 for 64 of 150, 12 for 64
// of 500, 69 for 64 of 4,000. A page is free while its reference count is 0 and the
// lowest free id is taken first, so that the counts are the only state of the
// pool and integer atomics, in whatever order, give the same result.
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "gdn_device.cuh"
#include "gdn_host.h"
#include "gdnspec.h"

namespace {

using gdndev::Buf;

constexpr int kMaxNodes = GDN_MAX_TOKENS + 1;

// ---------------------------------------------------------------- commit

// x / n by a multiplication with 2^32 / n rounded up (x * n < 2^32; n == 1 is 0).
__host__ __device__ __forceinline__ unsigned reciprocal(unsigned n) { return (unsigned)(((1ull << 32) + n - 1) / n); }
__device__ __forceinline__ int quotient(int x, unsigned by) { return by ? (int)__umulhi((unsigned)x, by) : x; }

// Where the slices (pool, layer, head) of the two pools lie.
struct Slices {
    uint4 *k, *v;
    int layers, h_kv;
    unsigned by_h_kv;
    size_t layer_units, head_units;  // 16-byte units of a layer's pool, of one page and head
    __device__ __forceinline__ uint4 *at(int s) const {
        const int pl = quotient(s, by_h_kv), head = s - pl * h_kv, layer = pl < layers ? pl : pl - layers;
        return (pl < layers ? k : v) + layer * layer_units + head * head_units;
    }
    // a row of page p at offset o of slice 0
    __device__ __forceinline__ size_t row(int p, int o, int row_units) const {
        return (size_t)p * h_kv * head_units + (size_t)o * row_units;
    }
};

// Whether quotient() is exact for every slice.
bool slices_fit(const attn_dims *d) { return 2ll * d->layers * d->h_kv * d->h_kv < (1ll << 32); }

Slices slices_of(const attn_dims *d, void *k, void *v) {
    const size_t head = (size_t)d->page_tokens * d->d_head * gdnhost::attn_elem_bytes(d) / 16;
    return {static_cast<uint4 *>(k), static_cast<uint4 *>(v), d->layers, d->h_kv, reciprocal(d->h_kv),
            head * d->h_kv * d->n_pages, head};
}

struct CommitArgs {
    int n_nodes, page_shift, n_pages, width, unit_shift;  // 2^unit_shift 16-byte units are a row
    Slices slices;
    const int32_t *parent, *node, *ctx, *table;
    int32_t *ctx_out, *status;
};

constexpr int kCommitThreads = 256;
constexpr int kCommitHold = 8;  // 16-byte units a thread holds between the reads and the writes

// grid (parts, B). The slices of a request (pool, layer, head) are dealt out to
// its CTAs. A path's destinations lie at or below its sources and may be other
// nodes' sources, so a slice is read whole before it is written: a round takes
// as many slices as the threads' registers hold (at least one: a path of 64
// rows of 1 KB goes in column ranges).
__global__ void __launch_bounds__(kCommitThreads, 4) commit_path(CommitArgs a) {
    __shared__ int32_t parent[kMaxNodes];
    __shared__ int depth_of_last, in_place;
    __shared__ long long src_row[GDN_MAX_TOKENS], dst_row[GDN_MAX_TOKENS];  // in units from a slice's begin; -1: no such page
    const int b = blockIdx.y, tid = threadIdx.x, N = a.n_nodes;
    const size_t B = gridDim.y;
    int32_t *st = a.status;
    const Buf bp{a.parent, B * N * 4}, bt{a.table, B * (size_t)a.width * 4};
    const int row_units = 1 << a.unit_shift;
    const Buf bk{a.slices.k, a.slices.layers * a.slices.layer_units * 16}, bv{a.slices.v, a.slices.layers * a.slices.layer_units * 16};
    gdndev::pdl_wait();
    gdndev::pdl_launch_dependents();
    const int node = a.node[b], ctx = a.ctx[b];
    const bool fits = ctx >= 0 && (int64_t)ctx + N - 1 <= (int64_t)a.width << a.page_shift;
    const bool known = node >= 0 && node < N;
    if (!fits || !known) {
        if (blockIdx.x == 0 && tid == 0) {
            a.ctx_out[b] = ctx;
            if (st) atomicOr(st, fits ? GDN_DEV_NODE_RANGE : GDN_DEV_LENGTH);
        }
        return;
    }
    if (a.parent) {
        for (int i = tid; i < N; i += kCommitThreads) {
            const int32_t *f = a.parent + (size_t)b * N + i;
            int p = GDN_IN(f, 4, bp, st) ? *f : i - 1;
            if (i > 0 && (p < 0 || p >= i)) {
                p = i - 1;
                if (blockIdx.x == 0 && st) atomicOr(st, GDN_DEV_TREE);
            }
            parent[i] = p;
        }
        __syncthreads();
        // every thread's node: its depth if it is on the accepted path
        if (tid < N) {
            bool on = false;
            int depth = 0;
            for (int i = node; i > 0; i = parent[i]) on |= i == tid;
            for (int i = tid; i > 0; i = parent[i]) ++depth;
            if (tid == node) depth_of_last = depth;
            const int s = ctx + tid - 1, d = ctx + depth - 1;
            if (on) {
                const int32_t *fs = a.table + (size_t)b * a.width + (s >> a.page_shift);
                const int32_t *fd = a.table + (size_t)b * a.width + (d >> a.page_shift);
                const int ps = GDN_IN(fs, 4, bt, st) ? *fs : -1, pd = GDN_IN(fd, 4, bt, st) ? *fd : -1;
                const int mask = (1 << a.page_shift) - 1;
                const bool okS = ps >= 0 && ps < a.n_pages, okD = pd >= 0 && pd < a.n_pages;
                if ((!okS || !okD) && blockIdx.x == 0 && st) atomicOr(st, GDN_DEV_PAGE);
                src_row[depth - 1] = okS ? (long long)a.slices.row(ps, s & mask, row_units) : -1;
                dst_row[depth - 1] = okD ? (long long)a.slices.row(pd, d & mask, row_units) : -1;
            }
        }
        __syncthreads();
        if (tid == 0) {  // the path's nodes 1..in_place are where they belong
            int j = 0;
            while (j < depth_of_last && src_row[j] == dst_row[j]) ++j;
            in_place = j;
        }
        __syncthreads();
    }
    const int k = a.parent ? depth_of_last : node;
    if (blockIdx.x == 0 && tid == 0) a.ctx_out[b] = ctx + k;
    if (!a.parent) return;
    const int first = in_place, rows = k - first;
    if (rows <= 0) return;
    const int slices = 2 * a.slices.layers * a.slices.h_kv, parts = gridDim.x;
    const int s0 = (int)((long long)slices * blockIdx.x / parts), s1 = (int)((long long)slices * (blockIdx.x + 1) / parts);
    // a round: `group` slices of 2^col_shift units of each row
    constexpr int kUnits = kCommitThreads * kCommitHold;
    int col_shift = a.unit_shift;
    while (rows << col_shift > kUnits) --col_shift;
    const int group = max(1, kUnits / (rows << col_shift));
    const unsigned by_rows = reciprocal(rows);
    for (int s = s0; s < s1; s += group)
        for (int c0 = 0; c0 < row_units; c0 += 1 << col_shift) {
            const int items = min(group, s1 - s) * rows << col_shift;
            uint4 held[kCommitHold];
            // item -> slice, row, column
            auto place = [&](int it, const long long *row_of, Buf &buf) -> uint4 * {
                const int r = it >> col_shift, sl = quotient(r, by_rows);
                const long long at = row_of[first + r - sl * rows];
                buf = s + sl < slices / 2 ? bk : bv;
                return at < 0 ? nullptr : a.slices.at(s + sl) + at + c0 + (it & ((1 << col_shift) - 1));
            };
#pragma unroll
            for (int h = 0; h < kCommitHold; ++h) {
                const int it = tid + h * kCommitThreads;
                held[h] = make_uint4(0, 0, 0, 0);
                if (it < items) {
                    Buf buf;
                    const uint4 *f = place(it, src_row, buf);
                    if (f && GDN_IN(f, 16, buf, st)) held[h] = *f;
                }
            }
            __syncthreads();
#pragma unroll
            for (int h = 0; h < kCommitHold; ++h) {
                const int it = tid + h * kCommitThreads;
                if (it < items) {
                    Buf buf;
                    uint4 *f = place(it, dst_row, buf);
                    if (f && GDN_IN(f, 16, buf, st)) *f = held[h];
                }
            }
        }
}

// ---------------------------------------------------------------- resize, fork

constexpr int kPoolThreads = 1024;
constexpr int kPoolWarps = kPoolThreads / 32;

// Exclusive prefix sum over the block of one value per thread; total returned.
__device__ __forceinline__ int block_scan(int v, int &before, int *warp_sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    const int w = warp_sum[lane];
    int s = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, s, o);
        if (lane >= o) s += y;
    }
    const int total = __shfl_sync(~0u, s, 31);
    before = x - v + __shfl_sync(~0u, s - w, warp);
    __syncthreads();
    return total;
}

// Ids of the first `wanted` free pages, in ascending order, into list; how many
// there are (at most wanted). Called by the whole block.
__device__ int find_free(const int32_t *ref, int n_pages, int wanted, int32_t *list, Buf br, Buf bl, int *warp_sum,
                         int32_t *st) {
    int found = 0;
    for (int base = 0; base < n_pages && found < wanted; base += kPoolThreads * 4) {
        const int i = base + threadIdx.x * 4;
        int r[4], n = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r[j] = i + j < n_pages && GDN_IN(ref + i + j, 4, br, st) ? __ldcg(ref + i + j) : 1;
            n += r[j] == 0;
        }
        int at;
        const int total = block_scan(n, at, warp_sum);
        at += found;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (r[j] == 0) {
                if (at < wanted && GDN_IN(list + at, 4, bl, st)) list[at] = i + j;
                ++at;
            }
        found += total;
    }
    __syncthreads();
    return min(found, wanted);
}

struct ResizeArgs {
    int batch, width, page_shift, n_pages;
    const int32_t *want;
    int32_t *table, *ref, *need, *list, *status;
};

__global__ void __launch_bounds__(kPoolThreads) resize_pages(ResizeArgs a) {
    __shared__ int warp_sum[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int32_t *st = a.status;
    const size_t B = a.batch;
    const Buf bt{a.table, B * (size_t)a.width * 4}, br{a.ref, (size_t)a.n_pages * 4}, bneed{a.need, B * 4},
        blist{a.list, (size_t)a.n_pages * 4};
    gdndev::pdl_wait();
    gdndev::pdl_launch_dependents();
    // one warp per request: entries past the wanted length are given back, the
    // missing ones below it counted
    for (int b = warp; b < a.batch; b += kPoolWarps) {
        const int want = a.want[b];
        const int keep = want < 0 ? 0 : (int)(((int64_t)want + (1 << a.page_shift) - 1) >> a.page_shift);
        int missing = 0;
        if (want >= 0 && keep > a.width) {
            if (lane == 0 && st) atomicOr(st, GDN_DEV_LENGTH);
        } else if (want >= 0) {
            for (int c = lane; c < a.width; c += 32) {
                int32_t *e = a.table + (size_t)b * a.width + c;
                const int id = GDN_IN(e, 4, bt, st) ? *e : -1;
                if (c < keep) {
                    missing += id < 0;
                } else if (id >= 0) {
                    if (id < a.n_pages) {
                        if (GDN_IN(a.ref + id, 4, br, st)) atomicSub(a.ref + id, 1);
                    } else if (st) {
                        atomicOr(st, GDN_DEV_PAGE);
                    }
                    if (GDN_IN(e, 4, bt, st)) *e = -1;
                }
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) missing += __shfl_xor_sync(~0u, missing, o);
        }
        if (lane == 0 && GDN_IN(a.need + b, 4, bneed, st)) a.need[b] = missing;
    }
    __syncthreads();
    // where each request's pages begin in the list of taken ones
    int total = 0;
    for (int base = 0; base < a.batch; base += kPoolThreads) {
        const int b = base + tid, n = b < a.batch ? a.need[b] : 0;
        int at;
        const int sum = block_scan(n, at, warp_sum);
        if (b < a.batch) a.need[b] = total + at;
        total += sum;
        if (total > a.n_pages) total = a.n_pages + 1;  // more than there can be
    }
    __syncthreads();
    if (total == 0) return;
    const int found = find_free(a.ref, a.n_pages, min(total, a.n_pages), a.list, br, blist, warp_sum, st);
    if (found < total && tid == 0 && st) atomicOr(st, GDN_DEV_POOL);
    for (int b = warp; b < a.batch; b += kPoolWarps) {
        const int want = a.want[b];
        const int keep = want < 0 ? 0 : (int)(((int64_t)want + (1 << a.page_shift) - 1) >> a.page_shift);
        if (keep > a.width) continue;
        int at = a.need[b];
        for (int c0 = 0; c0 < keep; c0 += 32) {
            const int c = c0 + lane;
            int32_t *e = a.table + (size_t)b * a.width + c;
            const bool miss = c < keep && GDN_IN(e, 4, bt, st) && *e < 0;
            const unsigned m = __ballot_sync(~0u, miss);
            const int k = at + __popc(m & ((1u << lane) - 1));
            if (miss && k < found) {
                const int id = a.list[k];
                *e = id;
                if (GDN_IN(a.ref + id, 4, br, st)) atomicAdd(a.ref + id, 1);
            }
            at += __popc(m);
        }
    }
}

struct ForkArgs {
    int batch, n_fork, width, page_shift, n_pages, row_units;
    Slices slices;
    const int32_t *src, *dst;
    int32_t *table, *ctx, *ref;
    int32_t *fresh;  // [n_fork] page taken for the tail; -1 none needed, -2 left out, -3 no page left
    int32_t *list;
    int32_t *status;
};

__global__ void __launch_bounds__(kPoolThreads) fork_take(ForkArgs a) {
    __shared__ int warp_sum[32];
    const int tid = threadIdx.x;
    int32_t *st = a.status;
    const Buf br{a.ref, (size_t)a.n_pages * 4}, blist{a.list, (size_t)a.n_pages * 4};
    gdndev::pdl_launch_dependents();
    gdndev::pdl_wait();
    int total = 0;
    for (int base = 0; base < a.n_fork; base += kPoolThreads) {
        const int i = base + tid;
        int state = -2;
        if (i < a.n_fork) {
            const int s = a.src[i], d = a.dst[i];
            if (s < 0 || s >= a.batch || d < 0 || d >= a.batch) {
                if (st) atomicOr(st, GDN_DEV_NODE_RANGE);
            } else {
                const int n = a.ctx[s];
                if (n < 0 || (int64_t)n > (int64_t)a.width << a.page_shift) {
                    if (st) atomicOr(st, GDN_DEV_LENGTH);
                } else {
                    state = (n & ((1 << a.page_shift) - 1)) ? 0 : -1;
                }
            }
        }
        int at;
        const int sum = block_scan(state == 0, at, warp_sum);
        if (i < a.n_fork) a.fresh[i] = state == 0 ? total + at : state;
        total += sum;
    }
    __syncthreads();
    const int found = total ? find_free(a.ref, a.n_pages, min(total, a.n_pages), a.list, br, blist, warp_sum, st) : 0;
    if (found < total && tid == 0 && st) atomicOr(st, GDN_DEV_POOL);
    for (int i = tid; i < a.n_fork; i += kPoolThreads) {
        int f = a.fresh[i];
        if (f == -2) continue;
        if (f >= 0) {
            f = f < found ? a.list[f] : -3;
            a.fresh[i] = f;
            if (f >= 0 && GDN_IN(a.ref + f, 4, br, st)) a.ref[f] = 1;
        }
        a.ctx[a.dst[i]] = f == -3 ? 0 : a.ctx[a.src[i]];
    }
}

constexpr int kForkThreads = 256;

// grid (parts, n_fork): the table row (first part), and the tail rows of this
// part's slices (pool, layer, head).
__global__ void __launch_bounds__(kForkThreads) fork_copy(ForkArgs a) {
    const int i = blockIdx.y, tid = threadIdx.x;
    int32_t *st = a.status;
    const size_t B = a.batch;
    const Buf bt{a.table, B * (size_t)a.width * 4}, br{a.ref, (size_t)a.n_pages * 4};
    const Buf bk{a.slices.k, a.slices.layers * a.slices.layer_units * 16}, bv{a.slices.v, a.slices.layers * a.slices.layer_units * 16};
    gdndev::pdl_wait();
    gdndev::pdl_launch_dependents();
    const int fresh = a.fresh[i];
    if (fresh == -2) return;
    const int s = a.src[i], d = a.dst[i], n = fresh == -3 ? 0 : a.ctx[s];
    const int full = n >> a.page_shift, tail = n & ((1 << a.page_shift) - 1);
    const int32_t *from = a.table + (size_t)s * a.width;
    int32_t *to = a.table + (size_t)d * a.width;
    for (int c = blockIdx.x * kForkThreads + tid; c < a.width; c += gridDim.x * kForkThreads) {
        int id = -1;
        if (c < full) {
            id = GDN_IN(from + c, 4, bt, st) ? from[c] : -1;
            if (id >= 0 && id < a.n_pages) {
                if (GDN_IN(a.ref + id, 4, br, st)) atomicAdd(a.ref + id, 1);
            } else {
                id = -1;
                if (st) atomicOr(st, GDN_DEV_PAGE);
            }
        } else if (c == full && fresh >= 0) {
            id = fresh;
        }
        if (GDN_IN(to + c, 4, bt, st)) to[c] = id;
    }
    if (fresh < 0) return;
    const int old = GDN_IN(from + full, 4, bt, st) ? from[full] : -1;
    const bool known = old >= 0 && old < a.n_pages;
    if (!known && blockIdx.x == 0 && tid == 0 && st) atomicOr(st, GDN_DEV_PAGE);
    const int slices = 2 * a.slices.layers * a.slices.h_kv, units = tail * a.row_units;
    const size_t from_row = a.slices.row(known ? old : 0, 0, a.row_units), to_row = a.slices.row(fresh, 0, a.row_units);
    for (int s = blockIdx.x; s < slices; s += gridDim.x) {
        uint4 *slice = a.slices.at(s);
        const Buf buf = s < slices / 2 ? bk : bv;
        for (int u0 = tid; u0 < units; u0 += 4 * kForkThreads) {
            uint4 x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int u = u0 + j * kForkThreads;
                x[j] = known && u < units && GDN_IN(slice + from_row + u, 16, buf, st) ? slice[from_row + u] : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int u = u0 + j * kForkThreads;
                if (u < units && GDN_IN(slice + to_row + u, 16, buf, st)) slice[to_row + u] = x[j];
            }
        }
    }
}

int log2_of(int n) {
    int s = 0;
    while ((1 << s) < n) ++s;
    return s;
}

int parts_for(int requests, int most) {
    const int sms = gdnhost::sm_count();
    const int want = (4 * (sms > 0 ? sms : 152) + requests - 1) / requests;
    return want < 1 ? 1 : want < most ? want : most;
}

constexpr size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

extern "C" int kv_commit_path(const attn_dims *dims, int32_t n_nodes, const int32_t *parent_dev,
                              const int32_t *accept_node, const int32_t *ctx_len, const int32_t *page_table,
                              void *k_pages, void *v_pages, int32_t *ctx_out, int32_t *dev_status,
                              gdn_stream_t stream) {
    if (const int rc = gdnhost::check_attn(dims)) return rc;
    if (n_nodes < 2 || n_nodes > kMaxNodes || !slices_fit(dims)) return GDN_ERR_DIMS;
    if (!accept_node || !ctx_len || !ctx_out || (parent_dev && (!page_table || !k_pages || !v_pages))) return GDN_ERR_NULL;
    using gdnhost::aligned_to;
    if (!aligned_to(k_pages, 16) || !aligned_to(v_pages, 16)) return GDN_ERR_ALIGN;
    for (const void *p : {(const void *)parent_dev, (const void *)accept_node, (const void *)ctx_len,
                          (const void *)page_table, (const void *)ctx_out, (const void *)dev_status})
        if (!aligned_to(p, 4)) return GDN_ERR_ALIGN;
    // a request's blocks read its length while the first of them writes the new one
    const uintptr_t in = reinterpret_cast<uintptr_t>(ctx_len), out = reinterpret_cast<uintptr_t>(ctx_out);
    if ((in > out ? in - out : out - in) < (uintptr_t)dims->batch * 4) return GDN_ERR_OVERLAP;
    CommitArgs a{n_nodes, log2_of(dims->page_tokens), dims->n_pages, dims->table_width,
                 log2_of((int)(dims->d_head * gdnhost::attn_elem_bytes(dims) / 16)), slices_of(dims, k_pages, v_pages),
                 parent_dev, accept_node, ctx_len, page_table, ctx_out, dev_status};
    const int64_t slices = 2LL * dims->layers * dims->h_kv;
    const int parts = parent_dev ? parts_for(dims->batch, slices < 65535 ? (int)slices : 65535) : 1;
    return gdndev::launch_pdl(commit_path, dim3(parts, dims->batch), dim3(kCommitThreads), 0,
                              static_cast<cudaStream_t>(stream), a) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

extern "C" size_t kv_pages_workspace_bytes(const attn_dims *dims) {
    if (gdnhost::check_attn(dims)) return 0;
    return round256((size_t)dims->batch * 4) + round256((size_t)dims->n_pages * 4);
}

static int check_pages(const attn_dims *dims, std::initializer_list<const void *> ints, void *workspace,
                       size_t workspace_bytes, const void *dev_status) {
    if (const int rc = gdnhost::check_attn(dims)) return rc;
    for (const void *p : ints)
        if (!p) return GDN_ERR_NULL;
    for (const void *p : ints)
        if (!gdnhost::aligned_to(p, 4)) return GDN_ERR_ALIGN;
    if (!gdnhost::aligned_to(dev_status, 4)) return GDN_ERR_ALIGN;
    if (!workspace || workspace_bytes < kv_pages_workspace_bytes(dims) || !gdnhost::aligned_to(workspace, 256))
        return GDN_ERR_WORKSPACE;
    return GDN_OK;
}

extern "C" int kv_pages_resize(const attn_dims *dims, const int32_t *want, int32_t *page_table, int32_t *page_ref,
                               void *workspace, size_t workspace_bytes, int32_t *dev_status, gdn_stream_t stream) {
    if (const int rc = check_pages(dims, {want, page_table, page_ref}, workspace, workspace_bytes, dev_status)) return rc;
    int32_t *need = static_cast<int32_t *>(workspace);
    int32_t *list = reinterpret_cast<int32_t *>(static_cast<char *>(workspace) + round256((size_t)dims->batch * 4));
    ResizeArgs a{dims->batch, dims->table_width, log2_of(dims->page_tokens), dims->n_pages, want, page_table, page_ref,
                 need, list, dev_status};
    return gdndev::launch_pdl(resize_pages, dim3(1), dim3(kPoolThreads), 0, static_cast<cudaStream_t>(stream), a) ==
                   cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

extern "C" int kv_pages_fork(const attn_dims *dims, int32_t n_fork, const int32_t *src, const int32_t *dst,
                             int32_t *page_table, int32_t *ctx_len, int32_t *page_ref, void *k_pages, void *v_pages,
                             void *workspace, size_t workspace_bytes, int32_t *dev_status, gdn_stream_t stream) {
    if (const int rc = gdnhost::check_attn(dims)) return rc;
    if (n_fork < 1 || n_fork > dims->batch || !slices_fit(dims)) return GDN_ERR_DIMS;
    if (!k_pages || !v_pages) return GDN_ERR_NULL;
    if (const int rc = check_pages(dims, {src, dst, page_table, ctx_len, page_ref}, workspace, workspace_bytes, dev_status))
        return rc;
    if (!gdnhost::aligned_to(k_pages, 16) || !gdnhost::aligned_to(v_pages, 16)) return GDN_ERR_ALIGN;
    int32_t *fresh = static_cast<int32_t *>(workspace);
    int32_t *list = reinterpret_cast<int32_t *>(static_cast<char *>(workspace) + round256((size_t)dims->batch * 4));
    ForkArgs a{dims->batch, n_fork, dims->table_width, log2_of(dims->page_tokens), dims->n_pages,
               (int)(dims->d_head * gdnhost::attn_elem_bytes(dims) / 16), slices_of(dims, k_pages, v_pages), src, dst,
               page_table, ctx_len, page_ref, fresh, list, dev_status};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (gdndev::launch_pdl(fork_take, dim3(1), dim3(kPoolThreads), 0, s, a) != cudaSuccess) return GDN_ERR_CUDA;
    const int64_t slices = 2LL * dims->layers * dims->h_kv;
    const int parts = parts_for(n_fork, slices < 65535 ? (int)slices : 65535);
    return gdndev::launch_pdl(fork_copy, dim3(parts, n_fork), dim3(kForkThreads), 0, s, a) == cudaSuccess ? GDN_OK
                                                                                                      : GDN_ERR_CUDA;
}
