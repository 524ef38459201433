// kda_checks.h -- argument checks that the latent attention, key-value attention and page pool calls share.
#pragma once

#include <stdint.h>

#include "../../include/kda.h"
#include "kda_internal.h"

namespace kda {

inline bool al(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Tokens, pages, strides and the elements from a tensor's first index to its last beyond these are refused, so that no
// product here or in the kernels overflows 64 bits; sequences, table rows and items beyond kMaxItems, so that 32-bit
// indices that step past the last one by a grid or a block do not wrap around.
constexpr int64_t kMaxCount = (int64_t)1 << 31;
constexpr int64_t kMaxStride = (int64_t)1 << 36;
constexpr int64_t kMaxExtent = (int64_t)1 << 44;
constexpr int32_t kMaxItems = 1 << 30;

// kda_latent_cache.reserved of what kda_kv_cache_pages() fills in, and the most words of a token there (128 heads of 256
// channels, and stats).
constexpr int32_t kPagesOfKv = 0x6b765f70;
constexpr int32_t kMaxKvRow = 128 * (2 * 256 + 4);

// Whether `count` indices at that stride reach past kMaxExtent (both checked before: not negative).
inline bool too_far(int64_t count, int64_t stride) { return count > 1 && stride > kMaxExtent / (count - 1); }

inline bool good_page_size(int32_t n) { return n == 16 || n == 32 || (n >= 64 && n <= 1024 && n % 64 == 0); }

// Pages and layers at these strides (16-bit words): KDA_OK when all lie apart and within what 64 bits hold, else
// refused with the text that fits.
inline int check_strides(int64_t layers, int64_t num_pages, int64_t page, int64_t layer_stride, int64_t page_stride,
                         const char *far, const char *overlap) {
    if (layer_stride < 0 || page_stride < 0 || layer_stride > kMaxStride || page_stride > kMaxStride ||
        too_far(layers, layer_stride) || too_far(num_pages, page_stride))
        return fail(KDA_ERR_INVALID_ARG, far);
    const bool pages_inside = num_pages == 1 || page_stride >= page;
    const bool layers_inside = layers == 1 || layer_stride >= page;
    // either all pages of a layer lie before the next layer's, or all layers of a page before the next page's
    const bool nested = layers == 1 || num_pages == 1 || layer_stride >= (num_pages - 1) * page_stride + page ||
                        page_stride >= (layers - 1) * layer_stride + page;
    if (!pages_inside || !layers_inside || !nested)
        return fail(KDA_ERR_INVALID_ARG, overlap);
    return KDA_OK;
}

// rows_only: for the calls that only copy pages, which take those of a kda_kv_cache as well.
inline int check_cache(const kda_latent_cache *c, LatentCacheArgs *o, bool rows_only = false) {
    if (!c || !c->pages) return fail(KDA_ERR_INVALID_ARG, "latent cache: cache or pages is NULL");
    if (c->dtype != KDA_ELEM_BF16 && c->dtype != KDA_ELEM_FP16)
        return fail(KDA_ERR_INVALID_ARG, "latent cache: dtype is neither KDA_ELEM_BF16 nor KDA_ELEM_FP16");
    const bool of_kv = c->reserved == kPagesOfKv;
    if (of_kv && !rows_only) return fail(KDA_ERR_INVALID_ARG, "latent cache: these are the pages of a kda_kv_cache");
    if (of_kv) {
        if (c->rank < 32 || c->rank > kMaxKvRow || c->rank % 4 || c->rope)
            return fail(KDA_ERR_INVALID_ARG, "pages of a kda_kv_cache: not as kda_kv_cache_pages() describes them");
    } else if (c->rank < 128 || c->rank > 512 || c->rank % 128 || c->rope < 0 || c->rope > 64 || c->rope % 16)
        return fail(KDA_ERR_UNSUPPORTED_SHAPE, "latent cache: rank must be 128, 256, 384 or 512 and rope a multiple "
                                               "of 16 up to 64");
    if (!good_page_size(c->page_size))
        return fail(KDA_ERR_UNSUPPORTED_SHAPE, "latent cache: page_size must be 16, 32 or a multiple of 64 up to 1024");
    if (c->layers < 1 || c->layers > 4096 || c->num_pages < 1 || c->num_pages >= kMaxCount)
        return fail(KDA_ERR_INVALID_ARG, "latent cache: layers or num_pages out of range");
    if (!al(c->pages, 16) || c->layer_stride % 8 || c->page_stride % 8)
        return fail(KDA_ERR_INVALID_ARG, "latent cache: pages and strides must be 16-byte aligned");
    const int64_t page = (int64_t)c->page_size * (c->rank + c->rope);
    const int rc = check_strides(c->layers, c->num_pages, page, c->layer_stride, c->page_stride,
                                 "latent cache: stride out of range", "latent cache: strides make pages overlap");
    if (rc != KDA_OK) return rc;
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

inline int check_table(const kda_page_table *p, bool counts, PageTableArgs *o) {
    if (!p || !p->table || !p->lens || (counts && !p->refcount))
        return fail(KDA_ERR_INVALID_ARG, "page table: table, lens or refcount is NULL");
    if (!al(p->table, 4) || !al(p->lens, 4) || (p->refcount && !al(p->refcount, 4)))
        return fail(KDA_ERR_INVALID_ARG, "page table: table, lens or refcount misaligned");
    if (p->max_seqs < 1 || p->max_seqs > kMaxItems || p->max_pages < 1 || p->page_size < 1 || p->page_size > 1024 ||
        p->num_pages < 1 || p->num_pages >= kMaxCount)
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

inline int check_same(const LatentCacheArgs &c, const PageTableArgs &t) {
    if (c.page_size != t.page_size || c.num_pages != t.num_pages)
        return fail(KDA_ERR_INVALID_ARG, "the cache's page_size and num_pages differ from the page table's");
    return KDA_OK;
}

// The kernels work with scale * log2(e) and 6 or 8 / that, which have to be normal numbers; a NaN fails both comparisons.
inline bool good_scale(float s) { return s >= 1e-30f && s <= 1e30f; }

// A stride of `count` indices.
inline bool bad_stride(int64_t s, int64_t least, int64_t count) {
    return s < least || s > kMaxStride || s % 8 || too_far(count, s);
}

}  // namespace kda
