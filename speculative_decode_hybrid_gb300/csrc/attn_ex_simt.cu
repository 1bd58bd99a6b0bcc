// attn_*_ex and attn_*_shared with GDN_F32: the launches of the f32 attention with
// changed scores, and its two passes where prefixes are shared (the groups' shared
// slots with the rows of all members, then every request's own slots), joined by one
// kernel.
//
// Measured: 4 trees of 5, 64 wide, in documents of 2,001 slots with cap and bias 22 us
// (19 by the plain kernel); 64 nodes of 8 requests over 4,000 slots 735 us (714 plain).
// Shared, plan included, against each request for itself (8 heads on 2, 128 wide, 8
// requests' tokens): 64 and 60 us over 20,000 slots, whose 41 MB stay in L2, 115 and 144
// over 50,000, 325 and 541 over 200,000; 8 x 16 rows over 100,000 1,571 and 1,582, by
// the f32 pipe's work, which is the same; 4 x 5 over 3,000 58 and 31, by launches. The pass
// over the groups has blocks for half as many groups as requests, each of all requests'
// rows, most of which end at once: its grid grows with the square of the batch (single
// tokens over 2,000 slots: 64 of 8 prompts 122 and 48, 512 of 64 609 and 282, 512 of 256
// 1,693 and 330).
#include "attn_ex_host.h"
#include "attn_simt.cuh"

namespace gdnattn {

namespace {

// The cuts of the pass over the groups (one group of all requests taken for
// granted, in more parts where there are few rows to fill the GPU with; none where
// there is no plan) and of the one over the requests' slots.
struct Cuts {
    int rows, groups;
    simt::Cut shared{}, own{};
    Cuts(const attn_dims *d, int n_tok, bool plan) : rows(n_tok * (d->h_q / d->h_kv)), groups(plan ? d->batch / 2 : 0) {
        own = simt::cut_of(d, rows, d->batch);
        if (groups) shared = simt::cut_of(d, rows * d->batch, 1, rows * d->batch <= 256 ? 4 * simt::kMaxParts : simt::kMaxParts);
    }
    int pieces() const { return shared.pieces + own.pieces; }
};

template <int D>
int launch(const attn_dims *d, const AttnArgs &a, const ExArgs &x, void *ws, cudaStream_t st) {
    const Cuts c(d, a.n_tok, x.plan != nullptr);
    const simt::Results r(a, c.pieces(), ws);
    const simt::Changed shared{x, true, 0, c.pieces()}, own{x, false, c.shared.pieces, c.pieces()};
    if (c.groups && !simt::launch_parts<D>(a, shared, c.shared, c.rows * d->batch, c.groups, r.o, r.ms, st)) return GDN_ERR_CUDA;
    if (!simt::launch_parts<D>(a, own, c.own, c.rows, a.batch, r.o, r.ms, st)) return GDN_ERR_CUDA;
    return simt::launch_join<D>(a, own, c.pieces(), r.o, r.ms, st);
}

}  // namespace

size_t ex_simt_workspace(const attn_dims *d, int n_tok, bool shared) {
    return simt::Results::bytes(d, n_tok, Cuts(d, n_tok, shared).pieces());
}

int ex_simt_launch(const attn_dims *d, const AttnArgs &a, const ExArgs &x, void *ws, cudaStream_t st) {
    return a.d == 64 ? launch<64>(d, a, x, ws, st) : a.d == 128 ? launch<128>(d, a, x, ws, st) : launch<256>(d, a, x, ws, st);
}

}  // namespace gdnattn
