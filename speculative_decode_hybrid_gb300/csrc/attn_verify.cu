// attn_verify_span / attn_tree_verify: argument checks and the choice of the
// kernel (the hybrid's attention layers of lucebox PR #506, Summary; DDTree
// verify of lucebox PR #533, Changes).
#include <cmath>
#include <initializer_list>

#include "attn_common.cuh"
#include "attn_host.h"
#include "gdn_host.h"
#include "gdnspec.h"

namespace {

int attend(const attn_dims *dims, int32_t n_tok, const int32_t *parent_dev, const void *q, const void *k_pages,
           const void *v_pages, const int32_t *page_table, const int32_t *ctx_len, float scale, void *out,
           void *workspace, size_t workspace_bytes, int32_t *dev_status, gdn_stream_t stream) {
    if (!std::isfinite(scale) || scale <= 0.f) return GDN_ERR_DIMS;
    if (!q || !k_pages || !v_pages || !page_table || !ctx_len || !out) return GDN_ERR_NULL;
    for (const void *p : {q, k_pages, v_pages, (const void *)out})
        if (!gdnhost::aligned_to(p, 16)) return GDN_ERR_ALIGN;
    for (const int32_t *p : {parent_dev, page_table, ctx_len, (const int32_t *)dev_status})
        if (!gdnhost::aligned_to(p, 4)) return GDN_ERR_ALIGN;
    if (!workspace || workspace_bytes < attn_workspace_bytes(dims, n_tok) || !gdnhost::aligned_to(workspace, 256))
        return GDN_ERR_WORKSPACE;
    int shift = 0;
    while ((1 << shift) < dims->page_tokens) ++shift;
    const gdnattn::AttnArgs a{dims->batch, n_tok, dims->h_q, dims->h_kv, dims->d_head, shift, dims->n_pages,
                              dims->table_width, scale * gdnattn::kLog2e, q, k_pages, v_pages, page_table, ctx_len,
                              parent_dev, out, dev_status};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dims->in_dtype == GDN_BF16 ? gdnattn::tc_launch(dims, a, workspace, st) : gdnattn::simt_launch(dims, a, workspace, st);
}

int check(const attn_dims *dims, int32_t n_tok) {
    if (const int rc = gdnhost::check_attn(dims)) return rc;
    if (n_tok < 1 || n_tok > GDN_MAX_TOKENS || (int64_t)dims->batch * dims->h_kv > 65535) return GDN_ERR_DIMS;
    if (dims->in_dtype == GDN_BF16 && !gdnattn::tc_fits(dims, n_tok)) return GDN_ERR_DIMS;
    return GDN_OK;
}

}  // namespace

extern "C" size_t attn_workspace_bytes(const attn_dims *dims, int32_t n_tok) {
    if (check(dims, n_tok)) return 0;
    return dims->in_dtype == GDN_BF16 ? gdnattn::tc_workspace(dims, n_tok) : gdnattn::simt_workspace(dims, n_tok);
}

extern "C" int attn_verify_span(const attn_dims *dims, int32_t n_tok, const void *q, const void *k_pages,
                                const void *v_pages, const int32_t *page_table, const int32_t *ctx_len, float scale,
                                void *out, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                                gdn_stream_t stream) {
    if (const int rc = check(dims, n_tok)) return rc;
    return attend(dims, n_tok, nullptr, q, k_pages, v_pages, page_table, ctx_len, scale, out, workspace, workspace_bytes,
                  dev_status, stream);
}

extern "C" int attn_tree_verify(const attn_dims *dims, int32_t n_nodes, const int32_t *parent_host,
                                const int32_t *parent_dev, const void *q, const void *k_pages, const void *v_pages,
                                const int32_t *page_table, const int32_t *ctx_len, float scale, void *out,
                                void *workspace, size_t workspace_bytes, int32_t *dev_status, gdn_stream_t stream) {
    if (const int rc = gdnhost::check_attn(dims)) return rc;
    if (n_nodes < 2) return GDN_ERR_TREE_TRUNCATED;
    if (const int rc = check(dims, n_nodes - 1)) return rc;
    if (!parent_host || !parent_dev) return GDN_ERR_NULL;
    if (const int rc = gdnhost::check_tree(parent_host, dims->batch, n_nodes, false, 0)) return rc;
    return attend(dims, n_nodes - 1, parent_dev, q, k_pages, v_pages, page_table, ctx_len, scale, out, workspace,
                  workspace_bytes, dev_status, stream);
}
