// kda_latent_api.cu -- the C ABI of the latent attention and page pool calls (include/kda.h): argument
// validation and dispatch.  No allocation, no host synchronisation, no CUDA call before the checks pass.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/kda.h"
#include "kda_checks.h"

using namespace kda;

extern "C" {

int kda_latent_append(const kda_latent_cache *cache, int32_t layer, const kda_page_table *pt, int32_t n,
                      const int32_t *rows, const int32_t *cu_tokens, int64_t num_tokens, const void *latent,
                      int64_t latent_stride, const void *rope, int64_t rope_stride, int32_t *dev_status,
                      kda_stream_t stream) {
    clear_error();
    AppendArgs a;
    int rc = check_cache(cache, &a.c);
    if (rc == KDA_OK) rc = check_table(pt, false, &a.t);
    if (rc == KDA_OK) rc = check_same(a.c, a.t);
    if (rc != KDA_OK) return rc;
    if (layer < 0 || layer >= a.c.layers) return fail(KDA_ERR_INVALID_ARG, "latent append: layer out of range");
    if (n < 0 || n > kMaxItems || num_tokens < 0 || num_tokens >= kMaxCount)
        return fail(KDA_ERR_INVALID_ARG, "latent append: n or num_tokens out of range");
    if (n == 0 || num_tokens == 0) return KDA_OK;
    if (!cu_tokens || !latent || (a.c.rope > 0 && !rope))
        return fail(KDA_ERR_INVALID_ARG, "latent append: a required pointer is NULL");
    if (!al(latent, 16) || (a.c.rope > 0 && !al(rope, 16)) || !al(cu_tokens, 4) || (rows && !al(rows, 4)) ||
        (dev_status && !al(dev_status, 4)))
        return fail(KDA_ERR_INVALID_ARG, "latent append: latent and rope must be 16-byte aligned, the others 4-byte");
    if (bad_stride(latent_stride, num_tokens > 1 ? a.c.rank : 0, num_tokens) ||
        (a.c.rope > 0 && bad_stride(rope_stride, num_tokens > 1 ? a.c.rope : 0, num_tokens)))
        return fail(KDA_ERR_INVALID_ARG, "latent append: row strides must be multiples of 8 that hold a row");
    a.c.pages += layer * a.c.layer_stride;
    a.n = n;
    a.rows = rows;
    a.cu = cu_tokens;
    a.num_tokens = num_tokens;
    a.latent = static_cast<const uint16_t *>(latent);
    a.rope = static_cast<const uint16_t *>(rope);
    a.latent_stride = latent_stride;
    a.rope_stride = rope_stride;
    a.status = dev_status;
    return launch_latent_append(a, reinterpret_cast<cudaStream_t>(stream));
}

size_t kda_latent_decode_workspace_bytes(const kda_latent_cache *cache, int32_t H, int32_t n, int32_t max_tokens) {
    LatentCacheArgs c;
    clear_error();
    if (check_cache(cache, &c) != KDA_OK) return 0;
    if (H < 1 || H > KDA_LATENT_MAX_HEADS || n < 0 || n > 65535 || max_tokens < 1 || max_tokens > KDA_LATENT_MAX_TOKENS)
        return 0;
    return latent_decode_workspace_bytes(c.rank, H, n, max_tokens);
}

int kda_latent_decode(const kda_latent_cache *cache, int32_t layer, const kda_page_table *pt, int32_t n,
                      const int32_t *rows, const int32_t *cu_tokens, int64_t num_tokens, int32_t max_tokens, int32_t H,
                      const void *q, int64_t q_token_stride, int64_t q_head_stride, const uint64_t *tree_mask,
                      float scale, void *out, float *lse, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                      kda_stream_t stream) {
    clear_error();
    LatentDecodeArgs a;
    int rc = check_cache(cache, &a.c);
    if (rc == KDA_OK) rc = check_table(pt, false, &a.t);
    if (rc == KDA_OK) rc = check_same(a.c, a.t);
    if (rc != KDA_OK) return rc;
    if (layer < 0 || layer >= a.c.layers) return fail(KDA_ERR_INVALID_ARG, "latent decode: layer out of range");
    if (n < 0 || n > 65535 || num_tokens < 0 || max_tokens < 1 || max_tokens > KDA_LATENT_MAX_TOKENS || H < 1 ||
        H > KDA_LATENT_MAX_HEADS)
        return fail(KDA_ERR_INVALID_ARG, "latent decode: n, num_tokens, max_tokens or H out of range");
    if (!cu_tokens && num_tokens != (int64_t)n * max_tokens)
        return fail(KDA_ERR_INVALID_ARG, "latent decode: num_tokens differs from n * max_tokens without cu_tokens");
    if (num_tokens >= kMaxCount) return fail(KDA_ERR_INVALID_ARG, "latent decode: num_tokens out of range");
    if (!good_scale(scale)) return fail(KDA_ERR_INVALID_ARG, "latent decode: scale must be from 1e-30 to 1e30");
    if (n == 0 || num_tokens == 0) return KDA_OK;
    if (!q || !out) return fail(KDA_ERR_INVALID_ARG, "latent decode: q or out is NULL");
    if (!al(q, 16) || !al(out, 16) || (lse && !al(lse, 4)) || (rows && !al(rows, 4)) ||
        (cu_tokens && !al(cu_tokens, 4)) || (tree_mask && !al(tree_mask, 8)) || (dev_status && !al(dev_status, 4)))
        return fail(KDA_ERR_INVALID_ARG, "latent decode: q and out must be 16-byte aligned, tree_mask 8-byte, the "
                                         "others 4-byte");
    const int64_t d = a.c.rank + a.c.rope;
    if (bad_stride(q_token_stride, num_tokens > 1 ? 8 : 0, num_tokens) || bad_stride(q_head_stride, H > 1 ? d : 0, H))
        return fail(KDA_ERR_INVALID_ARG, "latent decode: q strides must be multiples of 8 that hold a row");
    const size_t need = latent_decode_workspace_bytes(a.c.rank, H, n, max_tokens);
    if (!workspace || workspace_bytes < need || !al(workspace, 16))
        return fail(KDA_ERR_WORKSPACE, "latent decode: workspace NULL, misaligned or smaller than "
                                       "kda_latent_decode_workspace_bytes()");
    a.c.pages += layer * a.c.layer_stride;
    a.n = n;
    a.max_tokens = max_tokens;
    a.H = H;
    a.rows = rows;
    a.cu = cu_tokens;
    a.num_tokens = num_tokens;
    a.q = static_cast<const uint16_t *>(q);
    a.q_ts = q_token_stride;
    a.q_hs = q_head_stride;
    a.tree = tree_mask;
    a.scale = scale;
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    a.ws = workspace;
    a.status = dev_status;
    return launch_latent_decode(a, reinterpret_cast<cudaStream_t>(stream));
}

int kda_latent_prefill(int32_t dtype, int32_t H, int32_t nope, int32_t rope, int32_t dv, int32_t nseq,
                       const int32_t *cu_q, const int32_t *cu_k, int64_t num_q, int64_t num_k, int32_t max_q,
                       int32_t causal, const void *q, int64_t q_token_stride, int64_t q_head_stride,
                       const void *k_nope, int64_t k_token_stride, int64_t k_head_stride, const void *k_rope,
                       int64_t rope_token_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
                       float scale, void *out, float *lse, int32_t *dev_status, kda_stream_t stream) {
    clear_error();
    if (dtype != KDA_ELEM_BF16 && dtype != KDA_ELEM_FP16)
        return fail(KDA_ERR_INVALID_ARG, "latent prefill: dtype is neither KDA_ELEM_BF16 nor KDA_ELEM_FP16");
    if ((nope != 64 && nope != 128) || (dv != 64 && dv != 128) || rope < 16 || rope > 64 || rope % 16)
        return fail(KDA_ERR_UNSUPPORTED_SHAPE, "latent prefill: nope and dv must be 64 or 128 and rope a multiple of 16 "
                                               "up to 64");
    if (H < 1 || H > KDA_LATENT_MAX_HEADS || nseq < 0 || nseq > 65535 || num_q < 0 || num_q >= kMaxCount || num_k < 0 ||
        num_k > kMaxCount - 256 || max_q < 0 || max_q > KDA_LATENT_MAX_QUERIES)
        return fail(KDA_ERR_INVALID_ARG, "latent prefill: H, nseq, num_q, num_k or max_q out of range");
    if (!good_scale(scale)) return fail(KDA_ERR_INVALID_ARG, "latent prefill: scale must be from 1e-30 to 1e30");
    // a CTA for each tile of queries that a sequence may have, most of them ended at once where max_q is far above the
    // others' lengths: 250 a microsecond, so a quarter of a second for these
    if ((int64_t)H * nseq * ((std::min<int64_t>(max_q, num_q) + 255) / 256) > (int64_t)1 << 26)
        return fail(KDA_ERR_INVALID_ARG, "latent prefill: H * nseq * ceil(max_q / 256) must be at most 2^26");
    if (nseq == 0 || num_q == 0 || max_q == 0) return KDA_OK;
    if (!cu_q || !cu_k || !q || !out || (num_k > 0 && (!k_nope || !k_rope || !v)))
        return fail(KDA_ERR_INVALID_ARG, "latent prefill: a required pointer is NULL");
    if (!al(q, 16) || !al(k_nope, 16) || !al(k_rope, 16) || !al(v, 16) || !al(out, 16))
        return fail(KDA_ERR_INVALID_ARG, "latent prefill: q, k_nope, k_rope, v and out must be 16-byte aligned");
    if (!al(cu_q, 4) || !al(cu_k, 4) || (lse && !al(lse, 4)) || (dev_status && !al(dev_status, 4)))
        return fail(KDA_ERR_INVALID_ARG, "latent prefill: tables, lse or status misaligned");
    if (bad_stride(q_token_stride, 8, num_q) || bad_stride(q_head_stride, 8, H) || bad_stride(k_token_stride, 8, num_k) ||
        bad_stride(k_head_stride, 8, H) || bad_stride(rope_token_stride, 8, num_k) ||
        bad_stride(v_token_stride, 8, num_k) || bad_stride(v_head_stride, 8, H))
        return fail(KDA_ERR_INVALID_ARG, "latent prefill: strides must be positive multiples of 8 in range");
    LatentPrefillArgs a;
    a.fp16 = dtype == KDA_ELEM_FP16;
    a.H = H;
    a.nope = nope;
    a.rope = rope;
    a.dv = dv;
    a.nseq = nseq;
    a.max_q = max_q;
    a.causal = causal != 0;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.num_q = num_q;
    a.num_k = num_k;
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint16_t *>(k_nope);
    a.r = static_cast<const uint16_t *>(k_rope);
    a.v = static_cast<const uint16_t *>(v);
    a.q_ts = q_token_stride;
    a.q_hs = q_head_stride;
    a.k_ts = k_token_stride;
    a.k_hs = k_head_stride;
    a.r_ts = rope_token_stride;
    a.v_ts = v_token_stride;
    a.v_hs = v_head_stride;
    a.scale = scale;
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    a.status = dev_status;
    return launch_latent_prefill(a, reinterpret_cast<cudaStream_t>(stream));
}

size_t kda_pages_workspace_bytes(const kda_page_table *pt, int32_t n) {
    clear_error();
    if (!pt || n < 0 || n > kMaxItems || pt->max_seqs < 1 || pt->max_seqs > kMaxItems || pt->num_pages < 1 ||
        pt->num_pages >= kMaxCount)
        return 0;
    return pages_workspace_bytes(pt->max_seqs, pt->num_pages, n);
}

static int pages_call(PageOp op, const kda_page_table *pt, const kda_latent_cache *cache, int32_t n, const int32_t *x,
                      const int32_t *y, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                      kda_stream_t stream) {
    clear_error();
    PagesArgs a;
    int rc = check_table(pt, true, &a.t);
    if (rc != KDA_OK) return rc;
    if (op != PAGES_TRUNCATE) {
        rc = check_cache(cache, &a.c, true);
        if (rc == KDA_OK) rc = check_same(a.c, a.t);
        if (rc != KDA_OK) return rc;
    } else {
        a.c = LatentCacheArgs{};
    }
    if (n < 0 || n > kMaxItems) return fail(KDA_ERR_INVALID_ARG, "pages: n out of range");
    if (op != PAGES_COMPACT) {
        if (n == 0) return KDA_OK;
        if (!x || !y || !al(x, 4) || !al(y, 4))
            return fail(KDA_ERR_INVALID_ARG, "pages: rows or lengths NULL or misaligned");
    }
    if (dev_status && !al(dev_status, 4)) return fail(KDA_ERR_INVALID_ARG, "pages: status misaligned");
    if (!workspace || !al(workspace, 16) ||
        workspace_bytes < pages_workspace_bytes(a.t.max_seqs, a.t.num_pages, n))
        return fail(KDA_ERR_WORKSPACE, "pages: workspace NULL, misaligned or smaller than kda_pages_workspace_bytes()");
    a.n = n;
    a.x = x;
    a.y = y;
    a.ws = static_cast<int32_t *>(workspace);
    a.status = dev_status;
    return launch_pages(op, a, reinterpret_cast<cudaStream_t>(stream));
}

int kda_pages_reserve(const kda_page_table *pt, const kda_latent_cache *cache, int32_t n, const int32_t *rows,
                      const int32_t *new_lens, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                      kda_stream_t stream) {
    return pages_call(PAGES_RESERVE, pt, cache, n, rows, new_lens, workspace, workspace_bytes, dev_status, stream);
}

int kda_pages_truncate(const kda_page_table *pt, int32_t n, const int32_t *rows, const int32_t *keep_lens,
                       void *workspace, size_t workspace_bytes, int32_t *dev_status, kda_stream_t stream) {
    return pages_call(PAGES_TRUNCATE, pt, nullptr, n, rows, keep_lens, workspace, workspace_bytes, dev_status, stream);
}

int kda_pages_fork(const kda_page_table *pt, const kda_latent_cache *cache, int32_t n, const int32_t *parents,
                   const int32_t *children, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                   kda_stream_t stream) {
    return pages_call(PAGES_FORK, pt, cache, n, parents, children, workspace, workspace_bytes, dev_status, stream);
}

int kda_pages_compact(const kda_page_table *pt, const kda_latent_cache *cache, void *workspace,
                      size_t workspace_bytes, int32_t *dev_status, kda_stream_t stream) {
    return pages_call(PAGES_COMPACT, pt, cache, 0, nullptr, nullptr, workspace, workspace_bytes, dev_status, stream);
}

int kda_pages_copy(const kda_latent_cache *cache, int32_t n, const int32_t *src, const int32_t *dst,
                   int32_t *dev_status, kda_stream_t stream) {
    clear_error();
    LatentCacheArgs c;
    const int rc = check_cache(cache, &c, true);
    if (rc != KDA_OK) return rc;
    if (n < 0 || n > kMaxItems) return fail(KDA_ERR_INVALID_ARG, "pages copy: n out of range");
    if (n == 0) return KDA_OK;
    if (!src || !dst || !al(src, 4) || !al(dst, 4) || (dev_status && !al(dev_status, 4)))
        return fail(KDA_ERR_INVALID_ARG, "pages copy: src, dst or status NULL or misaligned");
    return launch_pages_copy(c, n, src, dst, dev_status, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
