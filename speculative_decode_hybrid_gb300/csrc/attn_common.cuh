// What the attention kernels share: their arguments and a node's root path as a
// bit mask.
#pragma once

#include <cstdint>

#include "attn_device.cuh"

namespace gdnattn {

constexpr float kLog2e = 1.4426950408889634f;

struct AttnArgs {
    int batch, n_tok, h_q, h_kv, d, page_shift, n_pages, width;
    float scale_log2;  // scale * log2(e): the softmax runs in powers of two
    const void *q, *k_pages, *v_pages;
    const int32_t *table, *ctx, *parent;  // parent: null for chains
    void *out;
    int32_t *status;
};

// Slots of request b that its rows see at most: ctx + n_tok, or 0 for a request
// that is left out (its length does not fit the page table).
__device__ __forceinline__ int slots_of(const AttnArgs &a, int b) {
    const int ctx = a.ctx[b];
    return ctx >= 0 && (int64_t)ctx + a.n_tok <= (int64_t)a.width << a.page_shift ? ctx + a.n_tok : 0;
}

// Root paths of the nodes 1..n_tok as bit masks (bit j: node j + 1 is on it),
// into path[n_tok]; node_parent: n_tok + 1 ints of shared memory. Called by all
// `threads` threads of a group; sync() is the group's barrier.
template <typename Sync>
__device__ __forceinline__ void root_paths(const AttnArgs &a, int b, unsigned long long *path, int *node_parent, int tid,
                                           int threads, bool flag, Sync sync) {
    const gdndev::Buf bp{a.parent, (size_t)a.batch * (a.n_tok + 1) * 4};
    if (a.parent)
        for (int i = tid; i <= a.n_tok; i += threads) {
            const int32_t *f = a.parent + (size_t)b * (a.n_tok + 1) + i;
            int p = GDN_IN(f, 4, bp, a.status) ? *f : i - 1;
            if (i > 0 && (p < 0 || p >= i)) {
                p = i - 1;
                if (flag && a.status) atomicOr(a.status, GDN_DEV_TREE);
            }
            node_parent[i] = p;
        }
    sync();
    for (int t = 1 + tid; t <= a.n_tok; t += threads) {
        unsigned long long m = 0;
        if (a.parent)
            for (int i = t; i > 0; i = node_parent[i]) m |= 1ull << (i - 1);
        else
            m = t == 64 ? ~0ull : (1ull << t) - 1;
        path[t - 1] = m;
    }
    sync();
}

}  // namespace gdnattn
