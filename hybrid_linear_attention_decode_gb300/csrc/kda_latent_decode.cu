// kda_latent_decode.cu -- absorbed latent attention over the paged cache (include/kda.h: kda_latent_decode).
//
// One warp per (query token, head): the query stays in registers, the keys stream past it, and the softmax runs
// online (maximum m, sum l of exp(s - m), weighted sum o; all fp32).
#include <cuda_fp16.h>

#include "kda_device.cuh"
#include "kda_internal.h"

namespace kda {
namespace latent {

__device__ __forceinline__ float elem(uint16_t x, bool fp16) {
    return fp16 ? __half2float(__ushort_as_half(x)) : bf2f(x);
}
__device__ __forceinline__ uint16_t to_elem(float x, bool fp16) {
    return fp16 ? __half_as_ushort(__float2half_rn(x)) : f2bf(x);
}

__global__ void __launch_bounds__(32) kda_latent_decode_kernel(const LatentDecodeArgs a) {
    const int lane = threadIdx.x;
    const int b = blockIdx.y, t = blockIdx.x / a.H, h = blockIdx.x - t * a.H;
    const int64_t c0 = a.cu ? a.cu[b] : (int64_t)b * a.max_tokens;
    const int64_t c1 = a.cu ? a.cu[b + 1] : c0 + a.max_tokens;
    const int64_t nq = c1 - c0;
    if (c0 < 0 || nq < 0 || nq > a.max_tokens || c1 > a.num_tokens) {
        if (blockIdx.x == 0 && lane == 0) set_status(a.status, KDA_DEV_BAD_SEQLENS);
        return;
    }
    if (t >= nq) return;
    const int32_t row = a.rows ? a.rows[b] : b;
    int64_t len = 0;
    if (row < -1 || row >= a.t.max_seqs) {
        if (lane == 0) set_status(a.status, KDA_DEV_BAD_SLOT);
    } else if (row >= 0) {
        len = a.t.lens[row];
        if (len < 0 || len > (int64_t)a.t.max_pages * a.t.page_size) {
            len = 0;
            if (lane == 0) set_status(a.status, KDA_DEV_BAD_SEQLENS);
        }
    }
    const int d = a.c.rank + a.c.rope;
    const uint64_t seen = a.tree ? a.tree[c0 + t] : (t >= 63 ? ~0ull : (2ull << t) - 1);
    const uint16_t *qp = a.q + (c0 + t) * a.q_ts + h * a.q_hs;
    float q[18], o[16];
#pragma unroll
    for (int k = 0; k < 18; ++k) q[k] = lane + 32 * k < d ? elem(qp[lane + 32 * k], a.c.fp16) * a.scale : 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = 0.f;
    float m = -INFINITY, l = 0.f;
    for (int64_t j = 0; j < len; ++j) {
        const int64_t drafted = j - (len - nq);
        if (drafted >= 0 && !(seen >> drafted & 1)) continue;
        const int32_t page = a.t.table[(int64_t)row * a.t.max_pages + j / a.t.page_size];
        const bool ok = page >= 0 && page < a.t.num_pages;
        if (!ok && lane == 0) set_status(a.status, KDA_DEV_BAD_PAGE);
        const uint16_t *x = a.c.pages + (ok ? page : 0) * a.c.page_stride + (j % a.t.page_size) * d;
        float v[18], s = 0.f;
#pragma unroll
        for (int k = 0; k < 18; ++k) {
            v[k] = ok && lane + 32 * k < d ? elem(x[lane + 32 * k], a.c.fp16) : 0.f;
            s = fmaf(q[k], v[k], s);
        }
        s = warp_sum(s);
        bool fin = true;  // a key that is not finite makes its queries NaN, also where the score would hide it
#pragma unroll
        for (int k = 0; k < 18; ++k) fin &= isfinite(v[k]);
        if (!__all_sync(0xffffffffu, fin)) s = NAN;
        const float mn = fmaxf(m, s), f = m == -INFINITY ? 0.f : expf(m - mn), p = expf(s - mn);
        l = l * f + p;
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = o[k] * f + p * v[k];
        m = mn;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t *out = a.out + ((c0 + t) * a.H + h) * a.c.rank;
#pragma unroll
    for (int k = 0; k < 16; ++k)
        if (lane + 32 * k < a.c.rank) out[lane + 32 * k] = to_elem(o[k] * inv, a.c.fp16);
    if (a.lse && lane == 0) a.lse[(c0 + t) * a.H + h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace latent

size_t latent_decode_workspace_bytes(int, int, int, int) { return 16; }

int launch_latent_decode(const LatentDecodeArgs &a, cudaStream_t st) {
    latent::kda_latent_decode_kernel<<<dim3(a.max_tokens * a.H, a.n), 32, 0, st>>>(a);
    return launch_result("kda_latent_decode_kernel launch");
}

}  // namespace kda
