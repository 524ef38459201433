// kda_latent_api.cu -- the C ABI of the latent attention and page pool calls (include/kda.h): argument
// validation and dispatch.  No allocation, no host synchronisation, no CUDA call before the checks pass.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/kda.h"
#include "kda_internal.h"

using namespace kda;

namespace {

bool al(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Tokens, pages, strides and the elements from a tensor's first index to its last beyond these are refused, so that no
// product here or in the kernels overflows 64 bits; sequences, table rows and items beyond kMaxItems, so that 32-bit
// indices that step past the last one by a grid or a block do not wrap around.
constexpr int64_t kMaxCount = (int64_t)1 << 31;
constexpr int64_t kMaxStride = (int64_t)1 << 36;
constexpr int64_t kMaxExtent = (int64_t)1 << 44;
constexpr int32_t kMaxItems = 1 << 30;

// Whether `count` indices at that stride reach past kMaxExtent (both checked before: not negative).
bool too_far(int64_t count, int64_t stride) { return count > 1 && stride > kMaxExtent / (count - 1); }

int check_cache(const kda_latent_cache *c, LatentCacheArgs *o) {
    if (!c || !c->pages) return fail(KDA_ERR_INVALID_ARG, "latent cache: cache or pages is NULL");
    if (c->dtype != KDA_ELEM_BF16 && c->dtype != KDA_ELEM_FP16)
        return fail(KDA_ERR_INVALID_ARG, "latent cache: dtype is neither KDA_ELEM_BF16 nor KDA_ELEM_FP16");
    if (c->rank < 128 || c->rank > 512 || c->rank % 128 || c->rope < 0 || c->rope > 64 || c->rope % 16)
        return fail(KDA_ERR_UNSUPPORTED_SHAPE, "latent cache: rank must be 128, 256, 384 or 512 and rope a multiple "
                                               "of 16 up to 64");
    if (!(c->page_size == 16 || c->page_size == 32 ||
          (c->page_size >= 64 && c->page_size <= 1024 && c->page_size % 64 == 0)))
        return fail(KDA_ERR_UNSUPPORTED_SHAPE, "latent cache: page_size must be 16, 32 or a multiple of 64 up to 1024");
    if (c->layers < 1 || c->layers > 4096 || c->num_pages < 1 || c->num_pages >= kMaxCount)
        return fail(KDA_ERR_INVALID_ARG, "latent cache: layers or num_pages out of range");
    if (!al(c->pages, 16) || c->layer_stride % 8 || c->page_stride % 8)
        return fail(KDA_ERR_INVALID_ARG, "latent cache: pages and strides must be 16-byte aligned");
    const int64_t page = (int64_t)c->page_size * (c->rank + c->rope);
    if (c->layer_stride < 0 || c->page_stride < 0 || c->layer_stride > kMaxStride || c->page_stride > kMaxStride ||
        too_far(c->layers, c->layer_stride) || too_far(c->num_pages, c->page_stride))
        return fail(KDA_ERR_INVALID_ARG, "latent cache: stride out of range");
    const bool pages_inside = c->num_pages == 1 || c->page_stride >= page;
    const bool layers_inside = c->layers == 1 || c->layer_stride >= page;
    // either all pages of a layer lie before the next layer's, or all layers of a page before the next page's
    const bool nested = c->layers == 1 || c->num_pages == 1 ||
                        c->layer_stride >= (c->num_pages - 1) * c->page_stride + page ||
                        c->page_stride >= (c->layers - 1) * c->layer_stride + page;
    if (!pages_inside || !layers_inside || !nested)
        return fail(KDA_ERR_INVALID_ARG, "latent cache: strides make pages overlap");
    o->rank = c->rank;
    o->rope = c->rope;
    o->page_size = c->page_size;
    o->layers = c->layers;
    o->fp16 = c->dtype == KDA_ELEM_FP16;
    o->num_pages = c->num_pages;
    // the stride of a single page or layer means nothing; a whole page keeps later arithmetic uniform
    o->page_stride = c->num_pages == 1 ? page : c->page_stride;
    o->layer_stride = c->layers == 1 ? 0 : c->layer_stride;
    o->pages = static_cast<uint16_t *>(c->pages);
    return KDA_OK;
}

int check_table(const kda_page_table *p, bool counts, PageTableArgs *o) {
    if (!p || !p->table || !p->lens || (counts && !p->refcount))
        return fail(KDA_ERR_INVALID_ARG, "page table: table, lens or refcount is NULL");
    if (!al(p->table, 4) || !al(p->lens, 4) || (p->refcount && !al(p->refcount, 4)))
        return fail(KDA_ERR_INVALID_ARG, "page table: table, lens or refcount misaligned");
    if (p->max_seqs < 1 || p->max_seqs > kMaxItems || p->max_pages < 1 || p->page_size < 1 || p->page_size > 1024 || p->num_pages < 1 ||
        p->num_pages >= kMaxCount)
        return fail(KDA_ERR_INVALID_ARG, "page table: sizes out of range");
    if ((int64_t)p->max_pages * p->page_size > kMaxCount - 64)  // whole tiles of 64 tokens stay below 2^31
        return fail(KDA_ERR_INVALID_ARG, "page table: max_pages * page_size must be at most 2^31 - 64 tokens");
    o->max_seqs = p->max_seqs;
    o->max_pages = p->max_pages;
    o->page_size = p->page_size;
    o->num_pages = p->num_pages;
    o->table = p->table;
    o->lens = p->lens;
    o->refcount = p->refcount;
    return KDA_OK;
}

int check_same(const LatentCacheArgs &c, const PageTableArgs &t) {
    if (c.page_size != t.page_size || c.num_pages != t.num_pages)
        return fail(KDA_ERR_INVALID_ARG, "the cache's page_size and num_pages differ from the page table's");
    return KDA_OK;
}

// The kernels work with scale * log2(e) and 6 or 8 / that, which have to be normal numbers; a NaN fails both comparisons.
bool good_scale(float s) { return s >= 1e-30f && s <= 1e30f; }

// A stride of `count` indices.
bool bad_stride(int64_t s, int64_t least, int64_t count) {
    return s < least || s > kMaxStride || s % 8 || too_far(count, s);
}

}  // namespace

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
        rc = check_cache(cache, &a.c);
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
    const int rc = check_cache(cache, &c);
    if (rc != KDA_OK) return rc;
    if (n < 0 || n > kMaxItems) return fail(KDA_ERR_INVALID_ARG, "pages copy: n out of range");
    if (n == 0) return KDA_OK;
    if (!src || !dst || !al(src, 4) || !al(dst, 4) || (dev_status && !al(dev_status, 4)))
        return fail(KDA_ERR_INVALID_ARG, "pages copy: src, dst or status NULL or misaligned");
    return launch_pages_copy(c, n, src, dst, dev_status, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
