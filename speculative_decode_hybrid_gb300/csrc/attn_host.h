// The attention kernels behind attn_verify_span and attn_tree_verify.
#pragma once

#include <cuda_runtime.h>

#include "gdnspec.h"

namespace gdnattn {

struct AttnArgs;

// f32 arithmetic (attn_simt.cu).
size_t simt_workspace(const attn_dims *d, int n_tok);
int simt_launch(const attn_dims *d, const AttnArgs &a, void *workspace, cudaStream_t st);

// bf16 on the tensor cores (attn_tc.cu). tc_fits: whether the tiles of the longest
// requests that the page table holds can be counted in 32 bits.
bool tc_fits(const attn_dims *d, int n_tok);
size_t tc_workspace(const attn_dims *d, int n_tok);
int tc_launch(const attn_dims *d, const AttnArgs &a, void *workspace, cudaStream_t st);

}  // namespace gdnattn
