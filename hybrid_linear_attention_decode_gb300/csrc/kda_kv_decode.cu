// kda_kv_decode.cu -- kda_kv_decode's workspace and launches, and the launch that adds weights to the pages' sums.
#include "kda_kv_decode.cuh"

namespace kda {
namespace kv {

constexpr int WW = 8;  // warps of a CTA of the third launch

// sum = decay * sum + sum over rows of 2^(x - lse2): a warp for 64 tokens of one key-value head, two tokens a lane.
__global__ void __launch_bounds__(WW * 32) kda_kv_weights_kernel(const DecodeP p) {
    wait_for_previous();
    allow_dependent_launch();
    const KvDecodeArgs &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, kv = a.c.heads, ps = a.c.page_size;
    // tiles of the sequences that take part: the last entry that is not left out
    int n = 0;
    {
        int lo = 0, hi = a.n + 1;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.base[mid] != INT64_MAX)
                lo = mid;
            else
                hi = mid;
        }
        n = lo;
    }
    const int64_t items = p.base[n] * kv;
    for (int64_t i = (int64_t)blockIdx.x * WW + warp; i < items; i += (int64_t)gridDim.x * WW) {
        const int64_t tile = i / kv;
        const int hk = (int)(i - tile * kv);
        int lo = 0, hi = n;  // base[lo] <= tile < base[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.base[mid] <= tile)
                lo = mid;
            else
                hi = mid;
        }
        const Seq s = seq_of(a, lo);
        const int key = (int)(tile - p.base[lo]) * 64 + 2 * lane;
        if (key >= s.len) continue;
        const int rows = s.nq * p.G;
        const float *x = p.scores + score_at(p, s, tile, hk) + 2 * lane;
        const float *lse = p.lse2 + (int64_t)lo * a.max_tokens * a.H + hk * p.G;
        float2 add = make_float2(0.f, 0.f);
        for (int t = 0; t < s.nq; ++t)
#pragma unroll 4
            for (int g = 0; g < p.G; ++g) {
                const float l2 = lse[t * a.H + g];
                const float2 v = *reinterpret_cast<const float2 *>(x + (t * p.G + g) * 64);
                const bool none = isnan(l2) || l2 == -INFINITY;
                add.x += none ? 0.f : exp2_(v.x - l2);
                add.y += none ? 0.f : exp2_(v.y - l2);
            }
        const int32_t page = a.t.table[(int64_t)s.row * a.t.max_pages + key / ps];
        if (!page_ok(a.t, page) || a.t.refcount[page] > 1) continue;
        float *w = reinterpret_cast<float *>(a.c.pages + page * a.c.page_stride + stats_at(a.c, hk)) + key % ps;
        w[0] = a.decay * w[0] + add.x;
        if (key + 1 < s.len) w[1] = a.decay * w[1] + add.y;
    }
}

// Rows of a unit: as few as hold all rows of a sequence, up to 64.
inline int block_rows(int G, int max_tokens) {
    const int rows = G * max_tokens;
    return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

struct Layout {
    size_t cut, part, part_l, lse2, base, scores, bytes;
};
inline Layout layout(const KvCacheArgs &c, int groups, int H, int n, int max_tokens, int64_t max_slots) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    Layout L;
    // for the widest block of rows, so that what is enough for some max_tokens is enough for fewer
    const size_t rows = (size_t)groups * 2 * 64;
    L.cut = 0;
    L.part = up(sizeof(Cut) * groups);
    L.part_l = L.part + up(rows * padded(c.d) * 4);
    L.lse2 = L.part_l + up(rows * 4);
    L.base = L.lse2 + (max_slots ? up((size_t)n * max_tokens * H * 4) : 0);
    L.scores = L.base + (max_slots ? up(((size_t)n + 1) * 8) : 0);
    L.bytes = L.scores + (max_slots ? up(((size_t)max_slots / 64 + n) * 64 * max_tokens * H * 4) : 0);
    return L;
}

// Keys' and then values' rows of a page, [pages][heads, keys then values, x tokens / 8][chunks of 64 channels][8 tokens][64], in
// boxes of `rows` tokens with all their channels, so that the copy reads 8 whole rows of the cache at a time and 64 channels of 8
// tokens are one swizzled block of shared memory.  Where head_dim is no multiple of 64, [pages][...x tokens][head_dim] in boxes of
// `rows` tokens x 64 channels, of which those behind the last read as zeros.
static bool cache_map(const KvCacheArgs &c, int rows, bool whole, CUtensorMap *map) {
    const latent::EncodeTiledFn enc = latent::encoder();
    if (!enc) return false;
    const int64_t tokens = (int64_t)2 * c.heads * c.page_size, d = c.d;
    if (whole) {
        const int64_t dims[5] = {64, 8, d / 64, tokens / 8, c.num_pages}, strides[4] = {d, 64, 8 * d, c.page_stride};
        const int box[5] = {64, 8, padded(c.d) / 64, rows / 8, 1};
        return latent::tensor_map(enc, map, c.fp16, c.pages, 5, dims, strides, box);
    }
    const int64_t dims[3] = {d, tokens, c.num_pages}, strides[2] = {d, c.page_stride};
    const int box[3] = {64, rows, 1};
    return latent::tensor_map(enc, map, c.fp16, c.pages, 3, dims, strides, box);
}

}  // namespace kv

size_t kv_decode_workspace_bytes(const KvCacheArgs &c, int H, int n, int max_tokens, int64_t max_slots) {
    return kv::layout(c, current_device_sms(), H, n, max_tokens, max_slots).bytes;
}

int launch_kv_decode(const KvDecodeArgs &a, cudaStream_t st) {
    using namespace kv;
    DecodeP p;
    p.a = a;
    p.groups = current_device_sms();
    p.G = a.H / a.c.heads;
    p.block = block_rows(p.G, a.max_tokens);
    p.box_rows = std::min(a.c.page_size, STAGE / (padded(a.c.d) * 4));
    p.whole = a.c.d % 64 == 0;
    const Layout L = layout(a.c, p.groups, a.H, a.n, a.max_tokens, a.max_slots);
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    p.cut = reinterpret_cast<Cut *>(ws + L.cut);
    p.part = reinterpret_cast<float *>(ws + L.part);
    p.part_l = reinterpret_cast<float *>(ws + L.part_l);
    p.lse2 = reinterpret_cast<float *>(ws + L.lse2);
    p.base = reinterpret_cast<int64_t *>(ws + L.base);
    p.scores = reinterpret_cast<float *>(ws + L.scores);
    CUtensorMap map;
    if (!cache_map(a.c, p.box_rows, p.whole, &map)) return fail(KDA_ERR_CUDA, "kv decode: the cache's tensor map was refused");
    int rc = a.c.fp16 ? launch_decode_fp16(p, map, st) : launch_decode_bf16(p, map, st);
    if (rc == KDA_OK && a.add_weights) {
        dependent_launch(kda_kv_weights_kernel, dim3((unsigned)p.groups * 8), WW * 32, 0, st, p);
        rc = launch_result("kda_kv_weights_kernel launch");
    }
    return rc;
}

}  // namespace kda
