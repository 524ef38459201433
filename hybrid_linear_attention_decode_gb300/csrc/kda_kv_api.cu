// kda_kv_api.cu -- the C ABI of the key-value attention, eviction and rotary calls (include/kda.h): argument validation
// and dispatch.  No allocation, no host synchronisation, no CUDA call before the checks pass.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_checks.h"

using namespace kda;

namespace {

int64_t page_words(int64_t page_size, int64_t heads, int64_t d, bool stats) {
    return page_size * heads * (2 * d + (stats ? 4 : 0));
}

int check_kv(const kda_kv_cache *c, KvCacheArgs *o) {
    if (!c || !c->pages) return fail(KDA_ERR_INVALID_ARG, "kv cache: cache or pages is NULL");
    if (c->dtype != KDA_ELEM_BF16 && c->dtype != KDA_ELEM_FP16)
        return fail(KDA_ERR_INVALID_ARG, "kv cache: dtype is neither KDA_ELEM_BF16 nor KDA_ELEM_FP16");
    if (c->stats != 0 && c->stats != 1) return fail(KDA_ERR_INVALID_ARG, "kv cache: stats is neither 0 nor 1");
    if (c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 8 || c->heads < 1 || c->heads > 128)
        return fail(KDA_ERR_UNSUPPORTED_SHAPE, "kv cache: head_dim must be a multiple of 8 from 16 to 256, heads 1 to 128");
    if (!good_page_size(c->page_size))
        return fail(KDA_ERR_UNSUPPORTED_SHAPE, "kv cache: page_size must be 16, 32 or a multiple of 64 up to 1024");
    if (c->layers < 1 || c->layers > 4096 || c->num_pages < 1 || c->num_pages >= kMaxCount)
        return fail(KDA_ERR_INVALID_ARG, "kv cache: layers or num_pages out of range");
    if (!al(c->pages, 16) || c->layer_stride % 8 || c->page_stride % 8)
        return fail(KDA_ERR_INVALID_ARG, "kv cache: pages and strides must be 16-byte aligned");
    const int64_t page = page_words(c->page_size, c->heads, c->head_dim, c->stats);
    const int rc = check_strides(c->layers, c->num_pages, page, c->layer_stride, c->page_stride,
                                 "kv cache: stride out of range", "kv cache: strides make pages overlap");
    if (rc != KDA_OK) return rc;
    o->heads = c->heads;
    o->d = c->head_dim;
    o->page_size = c->page_size;
    o->layers = c->layers;
    o->fp16 = c->dtype == KDA_ELEM_FP16;
    o->stats = c->stats;
    o->num_pages = c->num_pages;
    o->page_stride = c->num_pages == 1 ? page : c->page_stride;
    o->layer_stride = c->layers == 1 ? 0 : c->layer_stride;
    o->pages = static_cast<uint16_t *>(c->pages);
    return KDA_OK;
}

int check_both(const kda_kv_cache *cache, const kda_page_table *pt, bool counts, KvCacheArgs *c, PageTableArgs *t) {
    int rc = check_kv(cache, c);
    if (rc == KDA_OK) rc = check_table(pt, counts, t);
    if (rc != KDA_OK) return rc;
    if (c->page_size != t->page_size || c->num_pages != t->num_pages)
        return fail(KDA_ERR_INVALID_ARG, "the cache's page_size and num_pages differ from the page table's");
    return KDA_OK;
}

int check_rope(const kda_rope *r, int32_t D, RopeArgs *o) {
    if (!r || !r->turns || !al(r->turns, 8)) return fail(KDA_ERR_INVALID_ARG, "rope: turns NULL or misaligned");
    if (r->dim < 2 || r->dim > 256 || r->dim % 2 || r->offset < 0 || r->offset > D - r->dim)
        return fail(KDA_ERR_INVALID_ARG, "rope: dim must be even, 2 to 256, and offset + dim lie within the head");
    if (r->interleaved != 0 && r->interleaved != 1)
        return fail(KDA_ERR_INVALID_ARG, "rope: interleaved is neither 0 nor 1");
    if (!(fabsf(r->scale) >= 1e-30f && fabsf(r->scale) <= 1e30f))
        return fail(KDA_ERR_INVALID_ARG, "rope: scale must be from 1e-30 to 1e30 in size");
    o->dim = r->dim;
    o->offset = r->offset;
    o->interleaved = r->interleaved;
    o->scale = r->scale;
    o->turns = r->turns;
    return KDA_OK;
}

// theta / 2 pi as a fraction of a turn times 2^64, whole turns left out, rounded to a whole number.  The quotient's 53 bits reach
// below 2^-64 of a turn only where it is below 2^-11; there rounding (and not cutting off) halves the error.  Above, y is a whole
// number already, so that it never becomes 2^64.
uint64_t turns_of(double theta) {
    double x = theta / 6.283185307179586476925286766559;
    x -= floor(x);                     // whole turns a position do nothing
    const double y = ldexp(x, 64);     // below 2^64: x is below 1
    return (uint64_t)round(y);
}

}  // namespace

extern "C" {

int kda_kv_cache_pages(const kda_kv_cache *cache, kda_latent_cache *out) {
    clear_error();
    KvCacheArgs c;
    const int rc = check_kv(cache, &c);
    if (rc != KDA_OK) return rc;
    if (!out) return fail(KDA_ERR_INVALID_ARG, "kv cache: out is NULL");
    out->rank = c.heads * (2 * c.d + (c.stats ? 4 : 0));
    out->rope = 0;
    out->page_size = c.page_size;
    out->layers = c.layers;
    out->dtype = cache->dtype;
    out->reserved = kPagesOfKv;
    out->num_pages = c.num_pages;
    out->layer_stride = cache->layer_stride;
    out->page_stride = cache->page_stride;
    out->pages = cache->pages;
    return KDA_OK;
}

int kda_rope_turns_of(int32_t count, const double *theta, uint64_t *turns) {
    clear_error();
    if (count < 0 || (count > 0 && (!theta || !turns))) return fail(KDA_ERR_INVALID_ARG, "rope turns: bad count or NULL");
    for (int32_t i = 0; i < count; ++i)
        if (!(theta[i] >= 0 && theta[i] < 1048576.0))
            return fail(KDA_ERR_INVALID_ARG, "rope turns: frequencies must be from 0 to below 2^20");
    for (int32_t i = 0; i < count; ++i) turns[i] = turns_of(theta[i]);
    return KDA_OK;
}

int kda_rope_turns(int32_t dim, double base, int32_t scaling, double factor, double original, double low, double high,
                   uint64_t *turns) {
    clear_error();
    if (dim < 2 || dim > 256 || dim % 2 || !turns)
        return fail(KDA_ERR_INVALID_ARG, "rope turns: dim must be even, 2 to 256, and turns not NULL");
    if (!(base >= 1.0 && base <= 1e30)) return fail(KDA_ERR_INVALID_ARG, "rope turns: base must be from 1 to 1e30");
    if (scaling < KDA_ROPE_PLAIN || scaling > KDA_ROPE_PARTS)
        return fail(KDA_ERR_INVALID_ARG, "rope turns: unknown scaling");
    if (scaling != KDA_ROPE_PLAIN && !(factor >= 1.0 && factor <= 1e9))
        return fail(KDA_ERR_INVALID_ARG, "rope turns: factor must be from 1 to 1e9");
    if (scaling == KDA_ROPE_NTK && dim < 4) return fail(KDA_ERR_INVALID_ARG, "rope turns: this scaling needs dim 4 or more");
    if (scaling == KDA_ROPE_PARTS &&
        !(original > 0 && original <= 1e12 && low >= 0 && high > low && high <= 1e12))
        return fail(KDA_ERR_INVALID_ARG, "rope turns: original must be positive and 0 <= low < high");
    if (scaling == KDA_ROPE_NTK) base *= pow(factor, (double)dim / (dim - 2));
    for (int32_t i = 0; i < dim / 2; ++i) {
        double theta = pow(base, -2.0 * i / dim);
        if (scaling == KDA_ROPE_LINEAR) theta /= factor;
        if (scaling == KDA_ROPE_PARTS) {
            double g = (original * theta / 6.283185307179586476925286766559 - low) / (high - low);
            g = g < 0 ? 0 : g > 1 ? 1 : g;
            theta = theta / factor * (1 - g) + theta * g;
        }
        turns[i] = turns_of(theta);
    }
    return KDA_OK;
}

int kda_rope_apply(const kda_rope *rope, int32_t dtype, int64_t num_tokens, int32_t H, int32_t D,
                   const int32_t *positions, int32_t inverse, const void *x, int64_t x_token_stride,
                   int64_t x_head_stride, void *out, int64_t out_token_stride, int64_t out_head_stride,
                   kda_stream_t stream) {
    clear_error();
    RotateArgs a;
    if (dtype != KDA_ELEM_BF16 && dtype != KDA_ELEM_FP16)
        return fail(KDA_ERR_INVALID_ARG, "rope: dtype is neither KDA_ELEM_BF16 nor KDA_ELEM_FP16");
    if (D < 8 || D > 1024 || D % 8 || H < 1 || H > 1024)
        return fail(KDA_ERR_UNSUPPORTED_SHAPE, "rope: D must be a multiple of 8 up to 1024 and H 1 to 1024");
    const int rc = check_rope(rope, D, &a.r);
    if (rc != KDA_OK) return rc;
    if (num_tokens < 0 || num_tokens >= kMaxCount) return fail(KDA_ERR_INVALID_ARG, "rope: num_tokens out of range");
    if (num_tokens == 0) return KDA_OK;
    if (!positions || !x || !out) return fail(KDA_ERR_INVALID_ARG, "rope: a required pointer is NULL");
    if (!al(x, 16) || !al(out, 16) || !al(positions, 4))
        return fail(KDA_ERR_INVALID_ARG, "rope: x and out must be 16-byte aligned, positions 4-byte");
    if (bad_stride(x_token_stride, num_tokens > 1 ? D : 0, num_tokens) || bad_stride(x_head_stride, H > 1 ? D : 0, H) ||
        bad_stride(out_token_stride, num_tokens > 1 ? D : 0, num_tokens) || bad_stride(out_head_stride, H > 1 ? D : 0, H))
        return fail(KDA_ERR_INVALID_ARG, "rope: strides must be multiples of 8 that hold a row");
    a.fp16 = dtype == KDA_ELEM_FP16;
    a.H = H;
    a.D = D;
    a.inverse = inverse != 0;
    a.in_place = x == out && (num_tokens == 1 || x_token_stride == out_token_stride) &&
                 (H == 1 || x_head_stride == out_head_stride);
    if (x == out && !a.in_place) return fail(KDA_ERR_INVALID_ARG, "rope: out is x with other strides");
    a.num_tokens = num_tokens;
    a.positions = positions;
    a.x = static_cast<const uint16_t *>(x);
    a.out = static_cast<uint16_t *>(out);
    a.x_ts = x_token_stride;
    a.x_hs = x_head_stride;
    a.o_ts = out_token_stride;
    a.o_hs = out_head_stride;
    return launch_rotate(a, reinterpret_cast<cudaStream_t>(stream));
}

int kda_kv_append(const kda_kv_cache *cache, int32_t layer, const kda_page_table *pt, int32_t n, const int32_t *rows,
                  const int32_t *cu_tokens, int64_t num_tokens, const void *k, int64_t k_token_stride,
                  int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
                  const int32_t *positions, const kda_rope *rope, int32_t H, const void *q, int64_t q_token_stride,
                  int64_t q_head_stride, void *q_out, int32_t *dev_status, kda_stream_t stream) {
    clear_error();
    KvAppendArgs a;
    int rc = check_both(cache, pt, false, &a.c, &a.t);
    if (rc != KDA_OK) return rc;
    a.r = RopeArgs{0, 0, 0, 1.f, nullptr};
    if (rope) rc = check_rope(rope, a.c.d, &a.r);
    if (rc != KDA_OK) return rc;
    if (layer < 0 || layer >= a.c.layers) return fail(KDA_ERR_INVALID_ARG, "kv append: layer out of range");
    if (n < 0 || n > kMaxItems || num_tokens < 0 || num_tokens >= kMaxCount)
        return fail(KDA_ERR_INVALID_ARG, "kv append: n or num_tokens out of range");
    if (q && (!rope || !q_out || H < 1 || H > 1024))
        return fail(KDA_ERR_INVALID_ARG, "kv append: q needs rope, q_out and H from 1 to 1024");
    if (n == 0 || num_tokens == 0) return KDA_OK;
    if (!cu_tokens || !k || !v || (!positions && (rope || a.c.stats)))
        return fail(KDA_ERR_INVALID_ARG, "kv append: a required pointer is NULL");
    if (!al(k, 16) || !al(v, 16) || !al(cu_tokens, 4) || (rows && !al(rows, 4)) || (positions && !al(positions, 4)) ||
        (q && (!al(q, 16) || !al(q_out, 16))) || (dev_status && !al(dev_status, 4)))
        return fail(KDA_ERR_INVALID_ARG, "kv append: k, v, q and q_out must be 16-byte aligned, the others 4-byte");
    const int64_t d = a.c.d, least = num_tokens > 1 ? d : 0;
    const int32_t kv = a.c.heads;
    if (bad_stride(k_token_stride, least, num_tokens) || bad_stride(k_head_stride, kv > 1 ? d : 0, kv) ||
        bad_stride(v_token_stride, least, num_tokens) || bad_stride(v_head_stride, kv > 1 ? d : 0, kv) ||
        (q && (bad_stride(q_token_stride, least, num_tokens) || bad_stride(q_head_stride, H > 1 ? d : 0, H))))
        return fail(KDA_ERR_INVALID_ARG, "kv append: strides must be multiples of 8 that hold a row");
    if (q && q == q_out && ((num_tokens > 1 && q_token_stride != H * d) || (H > 1 && q_head_stride != d)))
        return fail(KDA_ERR_INVALID_ARG, "kv append: q_out is q, which is not contiguous");
    a.c.pages += layer * a.c.layer_stride;
    a.n = n;
    a.H = q ? H : 0;
    a.rows = rows;
    a.cu = cu_tokens;
    a.positions = positions;
    a.num_tokens = num_tokens;
    a.k = static_cast<const uint16_t *>(k);
    a.v = static_cast<const uint16_t *>(v);
    a.q = static_cast<const uint16_t *>(q);
    a.q_out = static_cast<uint16_t *>(q_out);
    a.k_ts = k_token_stride;
    a.k_hs = k_head_stride;
    a.v_ts = v_token_stride;
    a.v_hs = v_head_stride;
    a.q_ts = q_token_stride;
    a.q_hs = q_head_stride;
    a.status = dev_status;
    return launch_kv_append(a, reinterpret_cast<cudaStream_t>(stream));
}

static bool decode_sizes(const KvCacheArgs &c, int32_t H, int32_t n, int32_t max_tokens, int64_t max_slots) {
    return H >= 1 && H <= KDA_KV_MAX_HEADS && H % c.heads == 0 && n >= 0 && n <= 65535 && max_tokens >= 1 &&
           max_tokens <= KDA_KV_MAX_TOKENS && max_slots >= 0 && max_slots <= (int64_t)1 << 40;
}

size_t kda_kv_decode_workspace_bytes(const kda_kv_cache *cache, int32_t H, int32_t n, int32_t max_tokens,
                                     int64_t max_slots) {
    clear_error();
    KvCacheArgs c;
    if (check_kv(cache, &c) != KDA_OK || !decode_sizes(c, H, n, max_tokens, max_slots)) return 0;
    return kv_decode_workspace_bytes(c, H, n, max_tokens, max_slots);
}

int kda_kv_decode(const kda_kv_cache *cache, int32_t layer, const kda_page_table *pt, int32_t n, const int32_t *rows,
                  const int32_t *cu_tokens, int64_t num_tokens, int32_t max_tokens, int32_t H, const void *q,
                  int64_t q_token_stride, int64_t q_head_stride, const uint64_t *tree_mask, float scale, void *out,
                  float *lse, int32_t add_weights, float weight_decay, int64_t max_slots, void *workspace,
                  size_t workspace_bytes, int32_t *dev_status, kda_stream_t stream) {
    clear_error();
    KvDecodeArgs a;
    const int rc = check_both(cache, pt, add_weights != 0, &a.c, &a.t);
    if (rc != KDA_OK) return rc;
    if (layer < 0 || layer >= a.c.layers) return fail(KDA_ERR_INVALID_ARG, "kv decode: layer out of range");
    if (!decode_sizes(a.c, H, n, max_tokens, max_slots) || num_tokens < 0 || num_tokens >= kMaxCount)
        return fail(KDA_ERR_INVALID_ARG, "kv decode: n, num_tokens, max_tokens, max_slots or H out of range, or H not a "
                                         "multiple of the cache's heads");
    if (!cu_tokens && num_tokens != (int64_t)n * max_tokens)
        return fail(KDA_ERR_INVALID_ARG, "kv decode: num_tokens differs from n * max_tokens without cu_tokens");
    if (!good_scale(scale)) return fail(KDA_ERR_INVALID_ARG, "kv decode: scale must be from 1e-30 to 1e30");
    if (add_weights && (!a.c.stats || !(weight_decay >= 0.f && weight_decay <= 1.f)))
        return fail(KDA_ERR_INVALID_ARG, "kv decode: add_weights needs a cache with stats and weight_decay from 0 to 1");
    if (n == 0 || num_tokens == 0) return KDA_OK;
    if (add_weights && max_slots < 1)  // a workspace for a bound of 0 has no places for sums and scores
        return fail(KDA_ERR_INVALID_ARG, "kv decode: add_weights needs max_slots of 1 or more, as the workspace was asked for");
    if (!q || !out) return fail(KDA_ERR_INVALID_ARG, "kv decode: q or out is NULL");
    if (!al(q, 16) || !al(out, 16) || (lse && !al(lse, 4)) || (rows && !al(rows, 4)) ||
        (cu_tokens && !al(cu_tokens, 4)) || (tree_mask && !al(tree_mask, 8)) || (dev_status && !al(dev_status, 4)))
        return fail(KDA_ERR_INVALID_ARG, "kv decode: q and out must be 16-byte aligned, tree_mask 8-byte, the others "
                                         "4-byte");
    const int64_t d = a.c.d;
    if (bad_stride(q_token_stride, num_tokens > 1 ? 8 : 0, num_tokens) || bad_stride(q_head_stride, H > 1 ? d : 0, H))
        return fail(KDA_ERR_INVALID_ARG, "kv decode: q strides must be multiples of 8 that hold a row");
    const size_t need = kv_decode_workspace_bytes(a.c, H, n, max_tokens, add_weights ? max_slots : 0);
    if (!workspace || workspace_bytes < need || !al(workspace, 16))
        return fail(KDA_ERR_WORKSPACE, "kv decode: workspace NULL, misaligned or smaller than "
                                       "kda_kv_decode_workspace_bytes()");
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
    a.add_weights = add_weights != 0;
    a.decay = weight_decay;
    a.max_slots = add_weights ? max_slots : 0;
    a.ws = workspace;
    a.status = dev_status;
    return launch_kv_decode(a, reinterpret_cast<cudaStream_t>(stream));
}

int kda_kv_evict(const kda_kv_cache *cache, const kda_page_table *pt, int32_t n, const int32_t *rows, const int32_t *keep,
                 int32_t first, const int32_t *since, int32_t max_len, int32_t *new_lens, int32_t *dev_status,
                 kda_stream_t stream) {
    clear_error();
    KvEvictArgs a;
    const int rc = check_both(cache, pt, true, &a.c, &a.t);
    if (rc != KDA_OK) return rc;
    if (!a.c.stats) return fail(KDA_ERR_INVALID_ARG, "kv evict: the cache has no stats");
    if (n < 0 || n > 65535 || (int64_t)n * a.c.layers * a.c.heads > (int64_t)1 << 26)
        return fail(KDA_ERR_INVALID_ARG, "kv evict: n must be at most 65535 and n * layers * heads 2^26");
    if (first < 0) return fail(KDA_ERR_INVALID_ARG, "kv evict: first must not be negative");
    if (max_len < 0 || max_len > KDA_KV_EVICT_MAX_LEN)
        return fail(KDA_ERR_INVALID_ARG, "kv evict: max_len must be from 0 to KDA_KV_EVICT_MAX_LEN");
    if (n == 0) return KDA_OK;
    if (!keep || !new_lens) return fail(KDA_ERR_INVALID_ARG, "kv evict: keep or new_lens is NULL");
    if (!al(keep, 4) || !al(new_lens, 4) || (rows && !al(rows, 4)) || (since && !al(since, 4)) ||
        (dev_status && !al(dev_status, 4)))
        return fail(KDA_ERR_INVALID_ARG, "kv evict: tables or status misaligned");
    a.n = n;
    a.first = first;
    a.max_len = KDA_KV_EVICT_MAX_LEN;
    const int64_t room = (int64_t)a.t.max_pages * a.t.page_size;
    if (room < a.max_len) a.max_len = (int32_t)room;
    if (max_len > 0 && max_len < a.max_len) a.max_len = max_len;
    a.rows = rows;
    a.keep = keep;
    a.since = since;
    a.new_lens = new_lens;
    a.status = dev_status;
    return launch_kv_evict(a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
