// kda_latent_prefill.cu -- expanded latent attention for prompts (include/kda.h: kda_latent_prefill).
//
// One warp per (query, head): the query stays in registers, the keys stream past it, and the softmax runs
// online (maximum m, sum l of exp(s - m), weighted sum o; all fp32).
#include <cuda_fp16.h>

#include "kda_device.cuh"
#include "kda_internal.h"

namespace kda {
namespace latent {

__device__ __forceinline__ float elem2(uint16_t x, bool fp16) {
    return fp16 ? __half2float(__ushort_as_half(x)) : bf2f(x);
}
__device__ __forceinline__ uint16_t to_elem2(float x, bool fp16) {
    return fp16 ? __half_as_ushort(__float2half_rn(x)) : f2bf(x);
}

__global__ void __launch_bounds__(128) kda_latent_prefill_kernel(const LatentPrefillArgs a) {
    const int lane = threadIdx.x & 31, h = blockIdx.y, b = blockIdx.z;
    const int64_t q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
    if (q0 < 0 || q1 < q0 || q1 > a.num_q || k0 < 0 || k1 < k0 || k1 > a.num_k || q1 - q0 > a.max_q) {
        if (blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, KDA_DEV_BAD_SEQLENS);
        return;
    }
    const int64_t nq = q1 - q0, nk = k1 - k0, i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (i >= nq) return;
    const int64_t end = a.causal ? max((int64_t)0, min(nk, i + nk - nq + 1)) : nk;
    const int dq = a.nope + a.rope;
    const uint16_t *qp = a.q + (q0 + i) * a.q_ts + h * a.q_hs;
    float q[6], o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 6; ++k) q[k] = lane + 32 * k < dq ? elem2(qp[lane + 32 * k], a.fp16) * a.scale : 0.f;
    float m = -INFINITY, l = 0.f;
    for (int64_t j = k0; j < k0 + end; ++j) {
        const uint16_t *kp = a.k + j * a.k_ts + h * a.k_hs, *rp = a.r + j * a.r_ts, *vp = a.v + j * a.v_ts + h * a.v_hs;
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < 6; ++k) {
            const int e = lane + 32 * k;
            if (e < dq) s = fmaf(q[k], elem2(e < a.nope ? kp[e] : rp[e - a.nope], a.fp16), s);
        }
        s = warp_sum(s);
        const float mn = fmaxf(m, s), f = m == -INFINITY ? 0.f : expf(m - mn), p = expf(s - mn);
        l = l * f + p;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (lane + 32 * k < a.dv) o[k] = o[k] * f + p * elem2(vp[lane + 32 * k], a.fp16);
        m = mn;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t *out = a.out + ((q0 + i) * a.H + h) * a.dv;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (lane + 32 * k < a.dv) out[lane + 32 * k] = to_elem2(o[k] * inv, a.fp16);
    if (a.lse && lane == 0) a.lse[(q0 + i) * a.H + h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace latent

int launch_latent_prefill(const LatentPrefillArgs &a, cudaStream_t st) {
    latent::kda_latent_prefill_kernel<<<dim3((a.max_q + 3) / 4, a.H, a.nseq), 128, 0, st>>>(a);
    return launch_result("kda_latent_prefill_kernel launch");
}

}  // namespace kda
