// kda_latent.cuh -- what the two latent attention kernels share: element types, MN-major operand tiles and
// operands in tensor memory, 3-D tensor-map loads and the encoder of those maps.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include <atomic>

#include "kda_device.cuh"
#include "kda_internal.h"
#include "kda_umma.cuh"

namespace kda {
namespace latent {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Weights are 2^(kBias + (score - m) scale log2 e), m the row's running maximum.  m is raised (and what was summed so far
// rescaled) only when a score exceeds it by more than kRaise in units of log2, so that after the first tiles almost no
// rescaling is left; weights stay below 2^(kBias + kRaise).
// bf16 has the exponents of fp32 and needs no bias.  fp16 ends at 2^16 and is a multiple of 2^-24 below 2^-14, so its weights
// are moved up: with 9 + 6 they are rounded relative to themselves down to 2^-23 of the largest, and by at most 2^-34 of the
// largest below.  (Without a bias, weights below 2^-25 became 0 but stayed in the sum: many such keys behind one large
// weight whose values are near zero are most of the output.)  Why not more: 16 trees of 8 drafts over 2000 to 16384 tokens, 32
// heads, took 87.3 us with kRaise 8 (bias 7), 87.4 with 6 (9), 89.0 with 5 (10), 94.8 with 4 (11).
template <bool FP16>
constexpr float kRaise = FP16 ? 6.f : 8.f;
template <bool FP16>
constexpr float kBias = FP16 ? 9.f : 0.f;

__device__ __forceinline__ float exp2_(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 operations in one instruction, on register pairs.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// two floats rounded to the element type (nearest even), lo in the low half
template <bool FP16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if constexpr (FP16)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// two weights; in fp16 what is past its largest number becomes that (where one fp32 step of a score is several units of log2,
// a score may exceed m + kRaise by such a step)
template <bool FP16>
__device__ __forceinline__ uint32_t pack_weights(float lo, float hi) {
    if constexpr (FP16) {
        uint32_t r;
        asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    } else {
        return pack2<false>(lo, hi);
    }
}
// Looks for infinities and NaN, two elements an instruction: acc + x * 0 stays finite as long as every x was.
template <bool FP16>
__device__ __forceinline__ uint32_t times_zero(uint32_t x, uint32_t acc) {
    uint32_t r;
    if constexpr (FP16)
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
    else
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
    return r;
}
template <bool FP16>
__device__ __forceinline__ void times_zero4(uint4 x, uint32_t (&acc)[4]) {
    acc[0] = times_zero<FP16>(x.x, acc[0]);
    acc[1] = times_zero<FP16>(x.y, acc[1]);
    acc[2] = times_zero<FP16>(x.z, acc[2]);
    acc[3] = times_zero<FP16>(x.w, acc[3]);
}
// Whether any of the sums is not finite (then it is NaN: all exponent bits set).
template <bool FP16>
__device__ __forceinline__ bool nonfinite(const uint32_t (&acc)[4]) {
    constexpr uint32_t e = FP16 ? 0x7c00u : 0x7f80u;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) bad |= (acc[k] & e) == e || ((acc[k] >> 16) & e) == e;
    return bad;
}

// Instruction descriptor fields on top of umma::idesc(): 16-bit operand format, MN-major ("transposed") B.
template <bool FP16>
constexpr int kFmt = FP16 ? 0 : umma::kBF16;
constexpr uint32_t kBMajorMN = 1u << 16;

// Descriptor of an operand in the 128-byte swizzle, whose atoms are 8 rows of 128 bytes.  K-major (rows = M or N, k
// along the row): `sbo` bytes from one group of 8 rows to the next, lbo unused.  MN-major (rows = k, 64 elements of M or N
// along the row): `lbo` bytes from one group of 64 of M or N to the next, `sbo` from one group of 8 k to the next.  So rows
// of tokens are a K-major operand of one product (k = channel) and an MN-major one of another (k = token).
__device__ __forceinline__ uint64_t sdesc_at(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFF);
    d |= (uint64_t)((lbo >> 4) & 0x3FFF) << 16;
    d |= (uint64_t)((sbo >> 4) & 0x3FFF) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// One lane of a converged warp, the same each time.  MMAs are issued inside `if (elect_one())`: the compiler then knows
// that a single thread is active and keeps their descriptors in uniform registers.  With `if (lane == 0)`, or with a
// per-lane predicate on each instruction, one M 128, N 64 instruction took 85-90 cycles to issue (32 to execute).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r != 0;
}
// D += A B with A in tensor memory: lane = row, two consecutive 16-bit k in each column.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t id, bool acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(
            d_tmem),
        "r"(a_tmem), "l"(b), "r"(id), "r"((uint32_t)acc));
}

// Whether the phase is complete, without the suspended wait of mbar_try_wait(): for a warp that watches two barriers.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

// mbar_wait() by a whole warp, with one answer for all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t i = 1;; ++i) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if ((i & 255u) == 0 && __any_sync(0xffffffffu, global_timer_ns() - t0 > kWaitLimitNs)) return false;
    }
}

// Warp-wide, asynchronous: lanes 0..15 of this warp's quarter x 64 consecutive columns.  Register 4n + i of
// thread t holds lane t/4 + 8*(i/2), column 8n + 2*(t%4) + i%2.  Valid after umma::wait_ld(r).
__device__ __forceinline__ void ld16x64_issue(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%"
        "19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// The store of the same shape.
__device__ __forceinline__ void st16x64_issue(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%"
        "19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// Warp-wide, asynchronous: store r[16] into 32 lanes x 16 consecutive columns.
__device__ __forceinline__ void st16_issue(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int c0, int c1, int c2, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, int c0, int c1, int c2, int c3,
                                            uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// A dependent launch (launched with dependent_launch()) may be set up while the kernel before it still runs, from where all
// of that one's CTAs have called allow_dependent_launch().  Every thread of it calls wait_for_previous() before anything else
// that other work could see or have written; that returns when the kernel before is done and its writes are visible.  All
// latent attention and pool kernels are launched so: one call after another takes 0.2 to 1.4 us less (append 2.7 -> 2.35 us,
// decode over one sequence 11.9 -> 11.65, trees 88.2 -> 86.8).
// These kernels read global memory with ordinary loads (or streaming ones, or by TMA): a non-coherent load is for memory that
// nothing writes while the kernel is on the GPU, and here that begins before the kernel ahead has written the last of it.
// An ordinary load as an instruction of its own, behind the waits ahead of it; many of them stay in flight together (the
// decode kernel's queries as C++ loads: one sequence 11.9 us instead of 11.5).
__device__ __forceinline__ uint2 load_ordinary(const uint2 *p) {
    uint2 r;
    asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ void allow_dependent_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class... P, class... A>
inline cudaError_t dependent_launch(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t st,
                                    A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encoder() {
    static std::atomic<EncodeTiledFn> cached{nullptr};
    EncodeTiledFn f = cached.load(std::memory_order_acquire);
    if (f) return f;
    void *fp = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fp, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fp)
        return nullptr;
    f = reinterpret_cast<EncodeTiledFn>(fp);
    cached.store(f, std::memory_order_release);
    return f;
}

// A 16-bit tensor of rank n (outermost last) with strides[k] elements from one index of axis k + 1 to the next and
// axis 0 contiguous, read in boxes in the 128-byte swizzle; what lies outside reads as zero.
inline bool tensor_map(EncodeTiledFn enc, CUtensorMap *m, bool fp16, const void *base, int n, const int64_t *dims,
                       const int64_t *strides, const int *box) {
    cuuint64_t d[5], s[4];
    cuuint32_t b[5], one[5];
    for (int k = 0; k < n; ++k) {
        d[k] = (cuuint64_t)dims[k];
        b[k] = (cuuint32_t)box[k];
        one[k] = 1;
        if (k) s[k - 1] = (cuuint64_t)strides[k - 1] * 2;
    }
    return enc(m, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)n,
               const_cast<void *>(base), d, s, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [d2][d1][d0] in boxes of 64 x b1 x b2.
inline bool map_3d(EncodeTiledFn enc, CUtensorMap *m, bool fp16, const void *base, int64_t d0, int64_t d1, int64_t d2,
                   int64_t s1, int64_t s2, int b1, int b2) {
    const int64_t dims[3] = {d0, d1, d2}, strides[2] = {s1, s2};
    const int box[3] = {64, b1, b2};
    return tensor_map(enc, m, fp16, base, 3, dims, strides, box);
}

}  // namespace latent
}  // namespace kda
