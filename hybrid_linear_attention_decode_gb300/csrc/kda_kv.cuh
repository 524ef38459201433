// kda_kv.cuh -- what the key-value attention kernels share: where a token's rows are, 16-bit elements, and the sequence of
// a token.
#pragma once

#include "kda_latent.cuh"

namespace kda {
namespace kv {

using latent::allow_dependent_launch;
using latent::dependent_launch;
using latent::wait_for_previous;

constexpr uint32_t FULL = 0xffffffffu;

constexpr int kSmemMax = 227 * 1024;

// Lets a kernel take all shared memory, once for each device (a bit of `done`; devices past 64 each time).
template <class K>
inline cudaError_t allow_smem(K kernel, std::atomic<uint64_t> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (e != cudaSuccess || (done.load(std::memory_order_acquire) & bit)) return e;
    cudaFuncAttributes f;
    e = cudaFuncGetAttributes(&f, kernel);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax - (int)f.sharedSizeBytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

template <bool FP16>
__device__ __forceinline__ float to_f(uint16_t h) {
    if constexpr (FP16)
        return __half2float(__ushort_as_half(h));
    else
        return bf2f(h);
}
template <bool FP16>
__device__ __forceinline__ uint16_t from_f(float f) {
    if constexpr (FP16)
        return __half_as_ushort(__float2half_rn(f));
    else
        return f2bf(f);
}
template <bool FP16>
__device__ __forceinline__ float2 to_f2(uint32_t w) {
    return make_float2(to_f<FP16>((uint16_t)w), to_f<FP16>((uint16_t)(w >> 16)));
}

__device__ __forceinline__ bool page_ok(const PageTableArgs &t, int32_t p) { return p >= 0 && p < t.num_pages; }

// Words of a page before its keys of head h, its values of head h, and its sums of head h (positions follow them).
__device__ __forceinline__ int64_t key_at(const KvCacheArgs &c, int h) { return (int64_t)h * c.page_size * c.d; }
__device__ __forceinline__ int64_t value_at(const KvCacheArgs &c, int h) { return (int64_t)(c.heads + h) * c.page_size * c.d; }
__device__ __forceinline__ int64_t stats_at(const KvCacheArgs &c, int h) {
    return (int64_t)2 * c.heads * c.page_size * c.d + (int64_t)h * 4 * c.page_size;
}

// The sequence of token `tok`: the last b with cu[b] <= tok, by a 32-way search of one warp; -1 before the first, n behind
// the last.
__device__ __forceinline__ int sequence_of(const int32_t *cu, int n, int64_t tok, int lane) {
    int lo = 0, hi = n + 1;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const bool le = at < hi && cu[at] <= tok;
        const uint32_t m = __ballot_sync(FULL, le);
        if (!m) return -1;  // cu[lo] > tok
        lo += (31 - __clz(m)) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// One sequence of a decode call: its queries' first row, their number, its tokens and table row, and what is wrong with it.
struct Seq {
    int64_t c0;
    int32_t nq, len, row, bits;
};

__device__ __forceinline__ Seq seq_of(const KvDecodeArgs &a, int b) {
    Seq s;
    const int64_t c0 = a.cu ? (int64_t)a.cu[b] : (int64_t)b * a.max_tokens;
    const int64_t c1 = a.cu ? (int64_t)a.cu[b + 1] : c0 + a.max_tokens;
    s.row = a.rows ? a.rows[b] : b;
    s.c0 = c0;
    s.nq = (int32_t)(c1 - c0);
    s.bits = 0;
    s.len = 0;
    if (c0 < 0 || c1 < c0 || c1 - c0 > a.max_tokens || c1 > a.num_tokens) {
        s.bits = KDA_DEV_BAD_SEQLENS;
        s.nq = 0;
    } else if (s.row < -1 || s.row >= a.t.max_seqs) {
        s.bits = KDA_DEV_BAD_SLOT;
    } else if (s.row >= 0) {
        s.len = a.t.lens[s.row];
        if (s.len < 0 || s.len > (int64_t)a.t.max_pages * a.t.page_size) {
            s.bits = KDA_DEV_BAD_SEQLENS;
            s.len = 0;
        }
    }
    return s;
}

// Bits of the drafted tokens that the query token t of a sequence sees.
__device__ __forceinline__ uint64_t drafts_seen(const KvDecodeArgs &a, const Seq &s, int t) {
    const uint64_t chain = t >= 63 ? ~0ull : (2ull << t) - 1, all = s.nq >= 64 ? ~0ull : (1ull << s.nq) - 1;
    return (a.tree ? a.tree[s.c0 + t] : chain) & all;
}

}  // namespace kv
}  // namespace kda
