// kda_kv_decode.cu -- grouped-query attention over the paged cache (include/kda.h: kda_kv_decode).
//
//   s_j = scale q . k_j,   o = sum_j softmax(s)_j v_j
//
// A CTA for each query row (token, head): its warps go over the slots in turn with a running maximum and sum each, and are
// joined at the end.  A second launch adds the weights, exp(s_j - lse), to the pages' sums.
#include "kda_kv.cuh"

namespace kda {
namespace kv {

constexpr int DW = 8;  // warps

// The words of slot j's page; -1 for a bad page (flagged).
__device__ __forceinline__ int64_t page_of(const KvDecodeArgs &a, const Seq &s, int j) {
    const int32_t p = a.t.table[(int64_t)s.row * a.t.max_pages + j / a.c.page_size];
    if (page_ok(a.t, p)) return p * a.c.page_stride;
    set_status(a.status, KDA_DEV_BAD_PAGE);
    return -1;
}

template <bool FP16>
__global__ void __launch_bounds__(DW * 32) kda_kv_decode_simple(const KvDecodeArgs a) {
    __shared__ float so[DW][256], sm[DW], sl[DW];
    wait_for_previous();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = a.c.d;
    const int b = blockIdx.x / a.max_tokens, t = blockIdx.x % a.max_tokens, h = blockIdx.y;
    const Seq s = seq_of(a, b);
    if (s.bits && threadIdx.x == 0) set_status(a.status, s.bits);
    if (t >= s.nq) return;
    const int hk = h / (a.H / a.c.heads), nd = (d + 31) / 32;
    const uint16_t *q = a.q + (s.c0 + t) * a.q_ts + h * a.q_hs;
    const uint64_t seen = drafts_seen(a, s, t);
    float qv[8], o[8];
    for (int k = 0; k < nd; ++k) {
        qv[k] = lane + 32 * k < d ? to_f<FP16>(q[lane + 32 * k]) : 0.f;
        o[k] = 0;
    }
    float m = -INFINITY, l = 0;
    for (int j = warp; j < s.len; j += DW) {
        const int i = j - (s.len - s.nq);
        if (i >= 0 && !((seen >> i) & 1)) continue;
        const int64_t at = page_of(a, s, j);
        const uint16_t *kr = a.c.pages + at + key_at(a.c, hk) + (int64_t)(j % a.c.page_size) * d;
        const uint16_t *vr = a.c.pages + at + value_at(a.c, hk) + (int64_t)(j % a.c.page_size) * d;
        float x = 0;
        for (int k = 0; k < nd; ++k)
            if (lane + 32 * k < d && at >= 0) x += qv[k] * to_f<FP16>(kr[lane + 32 * k]);
        x = warp_sum(x) * a.scale;
        if (i >= 0 && (s.nq > 1 || a.tree) && at >= 0) {  // a drafted value row that is not finite
            bool bad = false;
            for (int k = 0; k < nd; ++k) bad |= lane + 32 * k < d && !isfinite(to_f<FP16>(vr[lane + 32 * k]));
            if (__any_sync(FULL, bad)) x = NAN;
        }
        const float m2 = fmaxf(m, x), mm = m2 == -INFINITY ? 0.f : m2;
        const float f = __expf(m - mm), p = isnan(x) ? x : __expf(x - mm);
        l = l * f + p;
        for (int k = 0; k < nd; ++k)
            o[k] = o[k] * f + (lane + 32 * k < d && at >= 0 ? p * to_f<FP16>(vr[lane + 32 * k]) : 0.f);
        m = m2;
    }
    for (int k = 0; k < nd; ++k) so[warp][lane + 32 * k] = o[k];
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    __syncthreads();
    float M = -INFINITY, L = 0;
    for (int w = 0; w < DW; ++w) M = fmaxf(M, sm[w]);
    const float mm = M == -INFINITY ? 0.f : M;
    for (int w = 0; w < DW; ++w) L += sl[w] * __expf(sm[w] - mm);
    for (int e = threadIdx.x; e < d; e += DW * 32) {
        float x = 0;
        for (int w = 0; w < DW; ++w) x += so[w][e] * __expf(sm[w] - mm);
        a.out[((s.c0 + t) * a.H + h) * d + e] = from_f<FP16>(L == 0.f ? 0.f : x / L);
    }
    if (threadIdx.x == 0) {
        const float lse = L == 0.f ? -INFINITY : mm + logf(L);
        if (a.lse) a.lse[(s.c0 + t) * a.H + h] = lse;
        if (a.add_weights) reinterpret_cast<float *>(a.ws)[((int64_t)b * a.max_tokens + t) * a.H + h] = lse;
    }
}

// Sums of the slots of one (sequence, key-value head): a warp a slot.
template <bool FP16>
__global__ void __launch_bounds__(DW * 32) kda_kv_weights_simple(const KvDecodeArgs a) {
    wait_for_previous();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = a.c.d;
    const int b = blockIdx.x, hk = blockIdx.y, G = a.H / a.c.heads, nd = (d + 31) / 32;
    const Seq s = seq_of(a, b);
    if (s.nq == 0 || s.len == 0) return;
    int64_t slots = 0;
    for (int i = 0; i <= b; ++i) slots += seq_of(a, i).nq > 0 ? seq_of(a, i).len : 0;
    if (slots > a.max_slots) {
        if (threadIdx.x == 0) set_status(a.status, KDA_DEV_BAD_SEQLENS);
        return;
    }
    for (int j = warp; j < s.len; j += DW) {
        const int i = j - (s.len - s.nq);
        const int64_t at = page_of(a, s, j);
        if (at < 0 || a.t.refcount[at / a.c.page_stride] > 1) continue;
        const uint16_t *kr = a.c.pages + at + key_at(a.c, hk) + (int64_t)(j % a.c.page_size) * d;
        float add = 0;
        for (int r = 0; r < s.nq * G; ++r) {
            const int t = r / G, h = hk * G + r % G;
            const float lse = reinterpret_cast<float *>(a.ws)[((int64_t)b * a.max_tokens + t) * a.H + h];
            if ((i >= 0 && !((drafts_seen(a, s, t) >> i) & 1)) || isnan(lse) || lse == -INFINITY) continue;
            const uint16_t *q = a.q + (s.c0 + t) * a.q_ts + h * a.q_hs;
            float x = 0;
            for (int k = 0; k < nd; ++k)
                if (lane + 32 * k < d) x += to_f<FP16>(q[lane + 32 * k]) * to_f<FP16>(kr[lane + 32 * k]);
            add += __expf(warp_sum(x) * a.scale - lse);
        }
        float *w = reinterpret_cast<float *>(a.c.pages + at + stats_at(a.c, hk)) + j % a.c.page_size;
        if (lane == 0) *w = a.decay * *w + add;
    }
}

}  // namespace kv

size_t kv_decode_workspace_bytes(const KvCacheArgs &, int H, int n, int max_tokens, int64_t) {
    return ((size_t)n * max_tokens * H + 4) * 4 / 16 * 16;
}

int launch_kv_decode(const KvDecodeArgs &a, cudaStream_t st) {
    using namespace kv;
    auto k = a.c.fp16 ? kda_kv_decode_simple<true> : kda_kv_decode_simple<false>;
    dependent_launch(k, dim3((unsigned)a.n * a.max_tokens, (unsigned)a.H), DW * 32, 0, st, a);
    if (a.add_weights) {
        auto w = a.c.fp16 ? kda_kv_weights_simple<true> : kda_kv_weights_simple<false>;
        dependent_launch(w, dim3((unsigned)a.n, (unsigned)a.c.heads), DW * 32, 0, st, a);
    }
    return launch_result("kda_kv_decode launch");
}

}  // namespace kda
