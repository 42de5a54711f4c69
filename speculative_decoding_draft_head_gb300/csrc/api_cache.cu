// extern "C" entry points of the quantised cache and the attention over it:
// argument checks and launches.  Nothing here computes on the host.
#include <cmath>

#include "internal.h"

namespace dspark {
namespace {

#define fail set_last_error

dspark_status cuda_fail(cudaError_t e, const char *where) {
    return fail(DSPARK_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t dtype_bytes(dspark_dtype dt) { return dt == DSPARK_F32 ? 4 : 2; }

dspark_status check_cache(const dspark_kv_cache *c) {
    if (!c) return fail(DSPARK_ERR_INVALID_ARG, "cache is NULL");
    if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->flags)
        return fail(DSPARK_ERR_INVALID_ARG, "a pointer of the cache is NULL");
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16) ||
        !aligned(c->flags, 4))
        return fail(DSPARK_ERR_INVALID_ARG, "the cache's arrays must be 16-byte aligned");
    if (c->n_pages < 1 || c->n_kv_heads < 1)
        return fail(DSPARK_ERR_INVALID_ARG, "bad n_pages %d or n_kv_heads %d", c->n_pages, c->n_kv_heads);
    if (c->page_size < 16 || c->page_size % 16 != 0)
        return fail(DSPARK_ERR_INVALID_ARG, "page_size must be a positive multiple of 16 (got %d)", c->page_size);
    if (c->head_dim < 16 || c->head_dim % 16 != 0)
        return fail(DSPARK_ERR_INVALID_ARG, "head_dim must be a positive multiple of 16 (got %d)", c->head_dim);
    if (c->head_dim > kMaxHeadDim)
        return fail(DSPARK_ERR_UNSUPPORTED, "head_dim must be at most %d (got %d)", kMaxHeadDim, c->head_dim);
    if (c->format != DSPARK_KV_E4M3 && c->format != DSPARK_KV_INT8)
        return fail(DSPARK_ERR_INVALID_ARG, "unknown cache format %d", c->format);
    return DSPARK_OK;
}

dspark_status check_rows(const PagedRows &p, const dspark_kv_cache *c) {
    if (p.B < 1) return fail(DSPARK_ERR_INVALID_ARG, "B must be >= 1 (got %d)", p.B);
    if (p.n_rows < 0) return fail(DSPARK_ERR_INVALID_ARG, "n_rows must be >= 0 (got %d)", p.n_rows);
    if (p.max_pages < 1) return fail(DSPARK_ERR_INVALID_ARG, "max_pages must be >= 1 (got %d)", p.max_pages);
    if ((int64_t)p.max_pages * c->page_size > 0x7fffffff)
        return fail(DSPARK_ERR_INVALID_ARG, "max_pages * page_size passes 2^31 - 1 tokens");
    if (!p.row0 || !p.start || !p.block_table) return fail(DSPARK_ERR_INVALID_ARG, "a required pointer is NULL");
    return DSPARK_OK;
}

bool bad_stride(int64_t stride, int64_t width, size_t elem) {
    return stride < width || (stride * (int64_t)elem) % 16 != 0;
}

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" {

dspark_status dspark_kv_append(const dspark_kv_cache *cache, const void *k, const void *v, int64_t k_stride,
                               int64_t v_stride, dspark_dtype dtype, const int64_t *row0, int n_rows,
                               const int32_t *start, const int32_t *block_table, int max_pages, int B, void *stream) {
    dspark_status st = check_cache(cache);
    if (st != DSPARK_OK) return st;
    const PagedRows p{row0, start, block_table, max_pages, B, n_rows};
    if ((st = check_rows(p, cache)) != DSPARK_OK) return st;
    if (dtype != DSPARK_BF16 && dtype != DSPARK_F32 && dtype != DSPARK_F16)
        return fail(DSPARK_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (n_rows == 0) return DSPARK_OK;
    if (!k || !v) return fail(DSPARK_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned(k, 16) || !aligned(v, 16)) return fail(DSPARK_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
    const int64_t width = (int64_t)cache->n_kv_heads * cache->head_dim;
    if (bad_stride(k_stride, width, dtype_bytes(dtype)) || bad_stride(v_stride, width, dtype_bytes(dtype)))
        return fail(DSPARK_ERR_INVALID_ARG, "row strides must cover a row and keep rows 16-byte aligned");
    const cudaError_t e = launch_kv_append(*cache, p, k, v, k_stride, v_stride, dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "append launch");
    return DSPARK_OK;
}

dspark_status dspark_kv_read(const dspark_kv_cache *cache, const int64_t *row0, int n_rows, const int32_t *start,
                             const int32_t *block_table, int max_pages, int B, dspark_dtype dtype, void *k_out,
                             void *v_out, void *stream) {
    dspark_status st = check_cache(cache);
    if (st != DSPARK_OK) return st;
    const PagedRows p{row0, start, block_table, max_pages, B, n_rows};
    if ((st = check_rows(p, cache)) != DSPARK_OK) return st;
    if (dtype != DSPARK_BF16 && dtype != DSPARK_F32 && dtype != DSPARK_F16)
        return fail(DSPARK_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (n_rows == 0) return DSPARK_OK;
    if (!k_out && !v_out) return fail(DSPARK_ERR_INVALID_ARG, "k_out and v_out are both NULL");
    if ((k_out && !aligned(k_out, 16)) || (v_out && !aligned(v_out, 16)))
        return fail(DSPARK_ERR_INVALID_ARG, "k_out and v_out must be 16-byte aligned");
    const cudaError_t e = launch_kv_read(*cache, p, dtype, k_out, v_out, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "read launch");
    return DSPARK_OK;
}

size_t dspark_attention_workspace_bytes(int B, int n_rows, int n_q_heads, int n_kv_heads, int head_dim) {
    if (B < 1 || n_rows < 0 || n_kv_heads < 1 || n_q_heads < 1 || n_q_heads % n_kv_heads != 0 || head_dim < 16 ||
        head_dim % 16 != 0 || head_dim > kMaxHeadDim)
        return 0;
    return attention_ws_bytes(B, n_rows, n_q_heads, n_kv_heads, head_dim);
}

dspark_status dspark_block_attention(const dspark_kv_cache *cache, const void *q, int64_t q_stride, dspark_dtype dtype,
                                     int n_q_heads, const int64_t *row0, int n_rows, int B, const int32_t *block_table,
                                     int max_pages, const int32_t *kv_len, const int32_t *prefix_pages,
                                     int n_prefix_pages, int prefix_len, dspark_block_mask mask,
                                     const uint64_t *row_mask, float scale, void *out, float *lse, void *workspace,
                                     size_t workspace_bytes, void *stream) {
    dspark_status st = check_cache(cache);
    if (st != DSPARK_OK) return st;
    const PagedRows p{row0, kv_len, block_table, max_pages, B, n_rows};
    if ((st = check_rows(p, cache)) != DSPARK_OK) return st;
    if (dtype == DSPARK_F32) return fail(DSPARK_ERR_UNSUPPORTED, "q must be bf16 or fp16");
    if (dtype != DSPARK_BF16 && dtype != DSPARK_F16) return fail(DSPARK_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (n_q_heads < 1 || n_q_heads % cache->n_kv_heads != 0)
        return fail(DSPARK_ERR_INVALID_ARG, "n_q_heads must be a positive multiple of n_kv_heads (got %d, %d)", n_q_heads,
                    cache->n_kv_heads);
    if ((int64_t)n_rows * n_q_heads > 0x7fffffff / 2)
        return fail(DSPARK_ERR_UNSUPPORTED, "n_rows * n_q_heads must be below 2^30");
    if (prefix_len < 0 || n_prefix_pages < 0 || (int64_t)n_prefix_pages * cache->page_size < prefix_len)
        return fail(DSPARK_ERR_INVALID_ARG, "prefix_len %d does not fit %d pages", prefix_len, n_prefix_pages);
    if (prefix_len > 0 && !prefix_pages) return fail(DSPARK_ERR_INVALID_ARG, "prefix_pages is NULL");
    if (mask != DSPARK_MASK_CAUSAL && mask != DSPARK_MASK_FULL)
        return fail(DSPARK_ERR_INVALID_ARG, "unknown mask %d", (int)mask);
    if (!std::isfinite(scale) || scale <= 0.f) return fail(DSPARK_ERR_INVALID_ARG, "scale must be finite and > 0");
    if (n_rows == 0) return DSPARK_OK;
    if (!q || !out) return fail(DSPARK_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned(q, 16) || !aligned(out, 16)) return fail(DSPARK_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
    if (bad_stride(q_stride, (int64_t)n_q_heads * cache->head_dim, 2))
        return fail(DSPARK_ERR_INVALID_ARG, "q_stride must cover a row and keep rows 16-byte aligned");
    const size_t need = attention_ws_bytes(B, n_rows, n_q_heads, cache->n_kv_heads, cache->head_dim);
    if (!workspace) return fail(DSPARK_ERR_INVALID_ARG, "workspace is NULL");
    if (!aligned(workspace, 256)) return fail(DSPARK_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (workspace_bytes < need)
        return fail(DSPARK_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", workspace_bytes, need);
    // (the bytes from the first to the last row of q)
    const int64_t q_bytes = ((n_rows - 1) * q_stride + (int64_t)n_q_heads * cache->head_dim) * 2;
    const int64_t out_bytes = (int64_t)n_rows * n_q_heads * cache->head_dim * 2;
    const char *qb = static_cast<const char *>(q), *ob = static_cast<const char *>(out);
    if (ob < qb + q_bytes && qb < ob + out_bytes) return fail(DSPARK_ERR_INVALID_ARG, "out must not overlap q");
    const AttentionArgs a{*cache, p, q, q_stride, dtype, n_q_heads, prefix_pages, prefix_len, (int)mask, row_mask, scale,
                          out, lse, static_cast<unsigned char *>(workspace)};
    const cudaError_t e = launch_block_attention(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "attention launch");
    return DSPARK_OK;
}

}  // extern "C"
