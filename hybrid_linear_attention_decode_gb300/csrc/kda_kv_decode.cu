// kda_kv_decode.cu -- kda_kv_decode's workspace and launches, and the launch that adds weights to the pages' sums.
#include "kda_kv_decode.cuh"

namespace kda {
namespace kv {

constexpr int WW = 8;  // warps of a CTA of the third launch

// sum = decay * sum + sum over rows of 2^(x - lse2): a warp for 64 tokens of one key-value head (an item), two tokens a lane, or
// (MANY rows) several that divide the rows where there are few items.  A CTA has a contiguous part of the items, so that it
// looks for a sequence once; all CTAs are on the GPU at once.
template <bool MANY>
constexpr int kWeightCtas = MANY ? 5 : 8;  // on a multiprocessor
template <bool MANY>
__global__ void __launch_bounds__(WW * 32, kWeightCtas<MANY>) kda_kv_weights_kernel(const DecodeP p) {
    __shared__ float2 sums[MANY ? WW : 1][32];
    wait_for_previous();
    allow_dependent_launch();
    const KvDecodeArgs &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, kv = a.c.heads, ps = a.c.page_size;
    const int64_t tiles = p.base[a.n + 1], items = tiles * kv;
    const int64_t per = items >> 31 ? (items + gridDim.x - 1) / gridDim.x : ((uint32_t)items + gridDim.x - 1) / gridDim.x;
    const int64_t i0 = min(items, blockIdx.x * per), tile0 = i0 >> 31 ? i0 / kv : (uint32_t)i0 / kv;
    const int head0 = (int)(i0 - tile0 * kv), count = (int)(min(items, i0 + per) - i0);
    int split = 1;  // warps of an item, with eight rows each or more
    while (MANY && split < WW && split * 16 <= p.G * a.max_tokens && items * split * 2 <= gridDim.x * WW) split *= 2;
    const int at_once = WW / split, mine = warp / split, slice = warp % split;
    if (count == 0) return;
    int b = 0, hi = a.n + 1;  // the last sequence that does not begin behind the tile, 32 ways a step
    while (hi - b > 1) {
        const int step = (hi - b + 31) / 32, at = b + lane * step;
        const uint32_t m = __ballot_sync(FULL, at < hi && p.base[at] <= tile0);
        b += (31 - __clz(m)) * step;
        hi = min(hi, b + step);
    }
    int64_t begin = p.base[b], end = p.base[b + 1];
    int4 s = p.seqs[b];  // row, tokens, queries
    for (int j = 0; j < count; j += at_once) {
        const int i = j + mine;
        float2 add = make_float2(0.f, 0.f), sum = add;
        float *w = nullptr;
        int key = 0;
        bool stays = true;
        if (i < count) {
            const int t0 = (head0 + i) / kv, hk = head0 + i - t0 * kv;
            const int64_t tile = tile0 + t0;
            while (end <= tile) {
                begin = end;
                end = p.base[++b + 1];
                s = p.seqs[b];
            }
            key = (int)(tile - begin) * 64 + 2 * lane;
            const int rows = s.z * p.G;
            if (key < s.y) {
                // read without waiting for one another: a bad page's place is page 0
                const int32_t page = a.t.table[(int64_t)s.x * a.t.max_pages + key / ps];
                const bool good = page_ok(a.t, page);
                const int32_t place = good ? page : 0;
                w = reinterpret_cast<float *>(a.c.pages + place * a.c.page_stride + stats_at(a.c, hk)) + key % ps;
                sum = *reinterpret_cast<const float2 *>(w);
                stays = !good || slice != 0 || a.t.refcount[place] > 1;
                const float *x = p.scores + (tile * a.max_tokens * a.H + (int64_t)hk * rows) * 64 + 2 * lane;  // see score_at()
                const float *lse = p.lse2 + (int64_t)b * a.max_tokens * a.H + hk * p.G;
                auto row = [&](const float *l, const float *y) {
                    const float l2 = *l;
                    const float2 v = __ldcs(reinterpret_cast<const float2 *>(y));
                    const bool some = l2 > -INFINITY;  // (not NaN)
                    add.x += some ? exp2_(v.x - l2) : 0.f;
                    add.y += some ? exp2_(v.y - l2) : 0.f;
                };
                if (!MANY || split == 1) {
                    for (int t = 0; t < s.z; ++t, lse += a.H)
#pragma unroll 8
                        for (int g = 0; g < p.G; ++g, x += 64) row(lse + g, x);
                } else {
#pragma unroll 8
                    for (int r = slice; r < rows; r += split) row(lse + r + over_g(p, r) * (a.H - p.G), x + r * 64);
                }
            }
        }
        if (MANY && split > 1) {
            sums[warp][lane] = add;
            __syncthreads();
            if (slice == 0)
                for (int k = 1; k < split; ++k) {
                    add.x += sums[warp + k][lane].x;
                    add.y += sums[warp + k][lane].y;
                }
            __syncthreads();
        }
        if (!stays) {
            w[0] = a.decay * sum.x + add.x;
            if (key + 1 < s.y) w[1] = a.decay * sum.y + add.y;
        }
    }
}

// Rows of a unit: as few as hold all rows of a sequence, up to 64.
inline int block_rows(int G, int max_tokens) {
    const int rows = G * max_tokens;
    return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

struct Layout {
    size_t cut, part, part_l, lse2, base, seqs, scores, bytes;
};
inline Layout layout(const KvCacheArgs &c, int sms, int H, int n, int max_tokens, int64_t max_slots) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    Layout L;
    // rows of two parts for each CTA, 64 on one CTA a multiprocessor or 32 on two: whatever max_tokens is, so that what is enough
    // for some is enough for fewer
    const size_t rows = (size_t)sms * 2 * 64;
    L.cut = 0;
    L.part = up(sizeof(Cut) * sms * 2);
    L.part_l = L.part + up(rows * padded(c.d) * 4);
    L.lse2 = L.part_l + up(rows * 4);
    L.base = L.lse2 + (max_slots ? up((size_t)n * max_tokens * H * 4) : 0);
    L.seqs = L.base + (max_slots ? up(((size_t)n + 2) * 8) : 0);
    L.scores = L.seqs + (max_slots ? up((size_t)n * 16) : 0);
    L.bytes = L.scores + (max_slots ? up(((size_t)max_slots / 64 + n) * 64 * max_tokens * H * 4) : 0);
    return L;
}

}  // namespace kv

size_t kv_decode_workspace_bytes(const KvCacheArgs &c, int H, int n, int max_tokens, int64_t max_slots) {
    return kv::layout(c, current_device_sms(), H, n, max_tokens, max_slots).bytes;
}

int launch_kv_decode(const KvDecodeArgs &a, cudaStream_t st) {
    using namespace kv;
    DecodeP p;
    p.a = a;
    p.G = a.H / a.c.heads;
    p.inverse_g = p.G == 1 ? 0 : (uint32_t)(((uint64_t)1 << 32) / p.G + 1);
    p.block = block_rows(p.G, a.max_tokens);
    const int sms = current_device_sms();
    const Layout L = layout(a.c, sms, a.H, a.n, a.max_tokens, a.max_slots);
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    p.cut = reinterpret_cast<Cut *>(ws + L.cut);
    p.part = reinterpret_cast<float *>(ws + L.part);
    p.part_l = reinterpret_cast<float *>(ws + L.part_l);
    p.lse2 = reinterpret_cast<float *>(ws + L.lse2);
    p.base = reinterpret_cast<int64_t *>(ws + L.base);
    p.seqs = reinterpret_cast<int4 *>(ws + L.seqs);
    p.scores = reinterpret_cast<float *>(ws + L.scores);
    int rc = a.c.d % 64 == 0 ? (a.c.fp16 ? launch_decode_fp16(p, st) : launch_decode_bf16(p, st))
                             : (a.c.fp16 ? launch_decode_fp16_odd(p, st) : launch_decode_bf16_odd(p, st));
    if (rc == KDA_OK && a.add_weights) {
        if (p.G * a.max_tokens < 16)
            dependent_launch(kda_kv_weights_kernel<false>, dim3((unsigned)sms * kWeightCtas<false>), WW * 32, 0, st, p);
        else
            dependent_launch(kda_kv_weights_kernel<true>, dim3((unsigned)sms * kWeightCtas<true>), WW * 32, 0, st, p);
        rc = launch_result("kda_kv_weights_kernel launch");
    }
    return rc;
}

}  // namespace kda
