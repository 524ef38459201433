// kda_latent_prefill.cu -- expanded latent attention for prompts (include/kda.h: kda_latent_prefill).
//
//   s_ij = scale (q_i . [k_j | r_j]),   o_i = sum_j softmax(s_i)_j v_j   per head, r shared by the heads
//
// 2 (nope + rope + dv) operations a pair against a few bytes: the tensor cores bound it.  One CTA takes 256 queries
// (two tiles of 128; or one tile in small calls) of one head and walks the keys in tiles of 128; the scores of one
// query tile are turned into weights while the tensor core works for the other.  12 warps, one CTA per SM:
//   warps 0-3, 4-7  softmax of query tile 0, 1: a thread per row (tensor-memory lane), so maxima and sums need no
//                   exchange; the weights go back to tensor memory over the scores they came from
//   warp 8   TMA: keys, rotary keys and values as units of 128 rows x 64 channels (16 KiB), one ring
//   warp 9   MMA: S = Q [K | R]^T (M 128, N 128), then O += P V with P in tensor memory and V as it lies (MN-major).
//            Order O0(j), S0(j+1), O1(j), S1(j+1): one tile's softmax runs beside the other's two products.
//            With one query tile a CTA (ONE) the two are the same queries over the even and the odd key tiles, and the
//            first one's warps join the results at the end.
//   warp 10  value rows that a query of the CTA does not see: those behind the sequence become zeros, and
//            those that are not finite too (0 x NaN is NaN), with a mark that makes the sums of the queries
//            that see them NaN.  Only tiles that some query sees in part need it.
// Tensor memory: S0 S1 O0 O1, 128 columns each.  The running maximum is raised only by more than kRaise, by the
// row's own thread in place.  Weights are rounded to the element type for the second product (its operands are
// 16-bit), in fp16 moved up by 2^kBias; their sum is kept in fp32 from the unrounded weights.
// Query tiles are dealt out from the last (under a causal mask the longest) to the first.
#include <algorithm>

#include "kda_latent.cuh"

namespace kda {
namespace latent {

constexpr int PQ = 128, PK = 128;        // queries of a tile, keys of a tile
constexpr int PNT = 384;                 // threads: 12 warps, the last of them idle (registers come in warpgroups)
// Registers: launched with 168 a thread (64,512 of 65,536).  The two softmax warpgroups take 184 and the other gives down to
// 136 (one query tile: 216 and 72): 2 * 128 * 184 + 128 * 136 = 2 * 128 * 216 + 128 * 72 = 64,512, what the launch holds.
constexpr uint32_t UNIT = PK * 128;      // bytes of 128 rows x 64 channels
constexpr int MAX_UNITS = 11;            // less than four tiles of the fewest units (3)
constexpr uint32_t PSMEM_MAX = 227 * 1024;
constexpr uint32_t PMISC = 1024;         // barriers and marks

struct PrefillP {
    LatentPrefillArgs a;
    int32_t units;  // of the ring
};

template <bool FP16, bool ONE>
__global__ void __launch_bounds__(PNT, 1)
    kda_latent_prefill_kernel(const PrefillP p, const __grid_constant__ CUtensorMap mq,
                              const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mr,
                              const __grid_constant__ CUtensorMap mv) {
    wait_for_previous();
    const LatentPrefillArgs &a = p.a;
    const int h = blockIdx.x, b = blockIdx.y;
    const int64_t q_lo = a.cu_q[b], q_hi = a.cu_q[b + 1], k_lo = a.cu_k[b], k_hi = a.cu_k[b + 1];
    if (q_lo < 0 || q_hi < q_lo || q_hi > a.num_q || k_lo < 0 || k_hi < k_lo || k_hi > a.num_k || q_hi - q_lo > a.max_q) {
        if (h == 0 && blockIdx.z == 0 && threadIdx.x == 0) set_status(a.status, KDA_DEV_BAD_SEQLENS);
        return;
    }
    const int nq = (int)(q_hi - q_lo), nk = (int)(k_hi - k_lo);
    const int qt = (int)(gridDim.z - 1 - blockIdx.z) * (ONE ? PQ : 2 * PQ);  // first query of the CTA
    if (qt >= nq) return;
    // keys that query i sees: [0, limit(i))
    const int shift = nk - nq + 1;
    auto limit = [&](int i) { return a.causal ? max(0, min(nk, i + shift)) : nk; };
    int nt[2];  // key tiles of the two query tiles
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int last = min(nq, qt + (t + 1) * PQ) - 1;
        nt[t] = (ONE && t == 1) || last < qt + t * PQ ? 0 : (limit(last) + PK - 1) / PK;
    }
    const int ntile = max(nt[0], nt[1]);
    if constexpr (ONE) {  // even and odd key tiles
        nt[0] = (ntile + 1) / 2;
        nt[1] = ntile / 2;
    }
    constexpr int lead = ONE ? 2 : 1;  // the ring holds K_0 .. K_lead-1, then V_0 K_lead V_1 K_lead+1 ...
    const int jf = limit(qt) / PK;  // from this tile on some query sees a part only
    const int kc = a.nope / 64 + 1, vc = a.dv / 64;  // units of a key tile, of a value tile
    const int NU = p.units;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *Q = sm;                                  // [2][kc] units
    uint8_t *R = Q + (uint32_t)(2 * kc) * UNIT;       // the ring
    uint64_t *bars = reinterpret_cast<uint64_t *>(R + (uint32_t)NU * UNIT);
    uint64_t *k_full = bars, *k_empty = bars + 4;    // [4] key tiles, by tile number (fewer than 4 fit the ring)
    uint64_t *v_full = bars + 8, *v_empty = bars + 12;  // [4] value tiles
    uint64_t *v_raw = bars + 16, *fixed = bars + 20;  // [4] value tiles for warp 10: as loaded, and looked over
    uint64_t *s_full = bars + 24;   // [2] scores of a query tile
    uint64_t *p_ready = bars + 26;  // [2] its weights
    uint64_t *o_done = bars + 28;   // [2] its output
    uint64_t *q_full = bars + 30;
    uint64_t *drain = bars + 31;
    uint64_t *half_done = bars + 32;  // ONE: the odd key tiles' maxima and sums are written
    float *half_ml = reinterpret_cast<float *>(R);  // [2][PQ], over the ring when it is no longer used
    uint32_t *any = reinterpret_cast<uint32_t *>(bars + 33);  // [4] whether a value tile has marks
    uint32_t *tmem_s = any + 4;
    uint8_t *mark = reinterpret_cast<uint8_t *>(tmem_s + 1);  // [4][PK]
    uint8_t *tag = mark + 4 * PK;  // [MAX_UNITS] producer's note of what a unit holds: barrier slot, value or key, parity

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp == 9) umma::alloc(tmem_s, 512);
    if (tid == 0) {
        for (int i = 0; i < 33; ++i) mbar_init(bars + i, i == 26 || i == 27 || i == 32 ? 4 : 1);  // p_ready, half_done: four warps
        fence_mbar_init();
    }
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    const uint32_t tmem = *tmem_s;
    allow_dependent_launch();  // with its tensor memory in hand: a CTA that waits may hold some itself
    constexpr uint32_t T_O = 2 * PK;
    bool ok = true;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(ONE ? 72 : 136));
        if (warp == 8) {
            // ================================ producer ================================
            int ki = 0, vi = 0;  // key and value tiles sent for
            if (lane == 0 && ntile > 0) {
                const int qtiles = ONE || nt[1] == 0 ? 1 : 2;
                mbar_arrive_expect_tx(q_full, (uint32_t)(qtiles * kc) * UNIT);
                for (int t = 0; t < qtiles; ++t)
                    for (int c = 0; c < kc; ++c)
                        tma_load_3d(Q + (uint32_t)(t * kc + c) * UNIT, &mq, c * 64, h, (int)q_lo + qt + t * PQ, q_full);
                int u = 0, used = 0;  // ring position, units in use up to the whole ring
                auto next = [&](bool value, int i) {  // the unit at u, for a part of K_i or V_i, once it is free
                    if (used < NU) {
                        ++used;
                    } else {
                        const int g = tag[u];
                        ok = ok && mbar_wait((g & 4 ? v_empty : k_empty) + (g & 3), (uint32_t)g >> 3);
                    }
                    tag[u] = (uint8_t)((i & 3) | (value ? 4 : 0) | ((i >> 2) & 1) << 3);
                    const int r = u;
                    if (++u == NU) u = 0;
                    return r;
                };
                auto load_k = [&](int i) {
                    uint64_t *bar = k_full + (i & 3);
                    for (int c = 0; c < kc; ++c) {
                        uint8_t *dst = R + (uint32_t)next(false, i) * UNIT;
                        if (!ok) return;
                        if (c == 0) {
                            mbar_arrive_expect_tx(bar, (uint32_t)kc * UNIT);
                            ++ki;
                        }
                        if (c < kc - 1)
                            tma_load_3d(dst, &mk, c * 64, h, (int)k_lo + i * PK, bar);
                        else
                            tma_load_3d(dst, &mr, 0, 0, (int)k_lo + i * PK, bar);
                    }
                };
                for (int i = 0; i < min(lead, ntile) && ok; ++i) load_k(i);
                for (; vi < ntile && ok; ++vi) {
                    uint64_t *bar = vi < jf ? v_full + (vi & 3) : v_raw + ((vi - jf) & 3);
                    const int u0 = next(true, vi), u1 = vc == 2 ? next(true, vi) : u0, row = (int)k_lo + vi * PK;
                    if (!ok) break;
                    mbar_arrive_expect_tx(bar, (uint32_t)vc * UNIT);
                    tma_load_3d(R + (uint32_t)min(u0, u1) * UNIT, &mv, 0, h, row, bar);
                    if (vc == 2) tma_load_3d(R + (uint32_t)max(u0, u1) * UNIT, &mv, 64, h, row, bar);
                    if (vi + lead < ntile) load_k(vi + lead);
                }
            }
            if (__syncthreads_or(!ok) && lane == 0 && ntile > 0) {  // copies still in flight land before the CTA ends
                constexpr uint64_t kDrainNs = 10000000ull;
                mbar_wait(q_full, 0, kDrainNs);
                for (int i = max(0, ki - 4); i < ki; ++i) mbar_wait(k_full + (i & 3), (uint32_t)(i >> 2) & 1u, kDrainNs);
                for (int i = max(0, vi - 4); i < vi; ++i)
                    if (i < jf)
                        mbar_wait(v_full + (i & 3), (uint32_t)(i >> 2) & 1u, kDrainNs);
                    else
                        mbar_wait(v_raw + ((i - jf) & 3), (uint32_t)((i - jf) >> 2) & 1u, kDrainNs);
            }
        } else if (warp == 9) {
            // ================================ MMA issuer ================================
            const uint32_t id_s = umma::idesc(kFmt<FP16>, PQ, PK);
            const uint32_t id_o = umma::idesc(kFmt<FP16>, PQ, a.dv) | kBMajorMN;
            const uint64_t dq0 = umma::sdesc(smem_addr(Q)), dr0 = umma::sdesc(smem_addr(R));
            const int kr = a.rope / 16;
            constexpr uint32_t UW = UNIT >> 4;  // a unit in descriptor words
            int u = 0;
            auto after = [&](int v, int n) { return v + n < NU ? v + n : v + n - NU; };
            auto scores = [&](int t, int v) {  // one thread: S_t = Q_t [K | R]^T of the key tile at ring position v
                const uint32_t ts = tmem + t * PK;
                uint64_t dq = dq0 + (uint64_t)(ONE ? 0 : t * kc * UW);
                for (int c = 0; c < kc - 1; ++c) {
                    const uint64_t dk = dr0 + (uint64_t)(v * UW);
#pragma unroll
                    for (int k = 0; k < 4; ++k) umma::mma_bf16(ts, dq + 2 * k, dk + 2 * k, id_s, c > 0 || k > 0);
                    dq += UW;
                    v = after(v, 1);
                }
                const uint64_t dk = dr0 + (uint64_t)(v * UW);
                if (kr == 4) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) umma::mma_bf16(ts, dq + 2 * k, dk + 2 * k, id_s, true);
                } else {
                    for (int k = 0; k < kr; ++k) umma::mma_bf16(ts, dq + 2 * k, dk + 2 * k, id_s, true);
                }
                umma::commit(s_full + t);
            };
            auto weigh = [&](int t, uint64_t dv, bool first, bool last) {  // one thread: O_t += P_t V
                const uint32_t to = tmem + T_O + t * 128, tp = tmem + t * PK;
#pragma unroll
                for (int k = 0; k < PK / 16; ++k)
                    mma_ts(to, tp + k * 8, dv + (uint64_t)(k * 2048 >> 4), id_o, !first || k > 0);
                if (last) umma::commit(o_done + t);
            };
            auto wait_k = [&](int i) {
                ok = ok && warp_wait(k_full + (i & 3), (uint32_t)(i >> 2) & 1u);
                umma::fence_after();
            };
            auto wait_v = [&](int i) {
                ok = ok && (i < jf ? warp_wait(v_full + (i & 3), (uint32_t)(i >> 2) & 1u)
                                   : warp_wait(fixed + ((i - jf) & 3), (uint32_t)((i - jf) >> 2) & 1u));
            };
            // u: ring position of what is used next; the order of use is the ring's
            auto take_v = [&]() {
                const int v0 = u, v1 = vc == 2 ? after(v0, 1) : v0;
                u = after(u, vc);
                return sdesc_at(smem_addr(R + (uint32_t)min(v0, v1) * UNIT), (uint32_t)abs(v1 - v0) * UNIT, 1024);
            };
            if (ntile > 0) {
                ok = warp_wait(q_full, 0);
                wait_k(0);
                if (ok && elect_one()) {
                    scores(0, u);
                    if (!ONE && nt[1] > 0) scores(1, u);
                    umma::commit(k_empty);
                }
                __syncwarp();
                u = after(u, kc);
                if (ONE && ntile > 1) {
                    wait_k(1);
                    if (ok && elect_one()) {
                        scores(1, u);
                        umma::commit(k_empty + 1);
                    }
                    __syncwarp();
                    u = after(u, kc);
                }
            }
            if constexpr (ONE) {
                for (int i = 0; i < ntile && ok; ++i) {
                    const int t = i & 1;
                    const uint64_t dv = take_v();
                    wait_v(i);
                    ok = ok && warp_wait(p_ready + t, (uint32_t)(i >> 1) & 1u);
                    if (!ok) break;
                    umma::fence_after();
                    if (elect_one()) {
                        weigh(t, dv, i < 2, i + 2 >= ntile);
                        umma::commit(v_empty + (i & 3));
                    }
                    __syncwarp();
                    if (i + 2 < ntile) {
                        wait_k(i + 2);
                        if (!ok) break;
                        if (elect_one()) {
                            scores(t, u);
                            umma::commit(k_empty + ((i + 2) & 3));
                        }
                        __syncwarp();
                        u = after(u, kc);
                    }
                }
            } else {
                for (int j = 0; j < ntile && ok; ++j) {
                    const uint64_t dv = take_v();
                    wait_v(j);
                    bool k_in = false;
                    for (int t = 0; t < 2 && ok; ++t) {
                        if (j >= nt[t]) continue;
                        ok = warp_wait(p_ready + t, (uint32_t)j & 1u);
                        if (!ok) break;
                        umma::fence_after();
                        if (elect_one()) {
                            weigh(t, dv, j == 0, j + 1 == nt[t]);
                            if (t == 1 || j >= nt[1]) umma::commit(v_empty + (j & 3));
                        }
                        __syncwarp();
                        if (j + 1 < nt[t]) {
                            if (!k_in) {
                                wait_k(j + 1);
                                if (!ok) break;
                                k_in = true;
                            }
                            if (elect_one()) {
                                scores(t, u);
                                if (t == 1 || j + 1 >= nt[1]) umma::commit(k_empty + ((j + 1) & 3));
                            }
                            __syncwarp();
                        }
                    }
                    u = after(u, kc);
                }
            }
            if (__syncthreads_or(!ok)) {
                if (elect_one()) umma::commit(drain);
                mbar_wait(drain, 0, 10000000ull);
            }
        } else if (warp == 10) {
            // ================================ value rows that not every query sees ================================
            for (int j = jf; j < ntile && ok; ++j) {
                // V_j comes behind the first keys, V_0 .. V_j-1, and the keys between those
                const int u = (int)(((int64_t)min(lead, ntile) * kc + (int64_t)j * vc + (int64_t)max(0, min(j, ntile - lead)) * kc) %
                                    NU);
                const int f = j - jf, valid = min(PK, nk - j * PK);
                ok = __all_sync(0xffffffffu, mbar_wait(v_raw + (f & 3), (uint32_t)(f >> 2) & 1u));
                if (!ok) break;
                uint8_t *mk4 = mark + (f & 3) * PK;
                bool found = false;
                for (int r0 = 0; r0 < PK; r0 += 32) {  // a lane per row of 8 or 16 words
                    const int r = r0 + lane;
                    uint32_t acc[4] = {0, 0, 0, 0};
                    for (int c = 0; c < vc; ++c) {
                        const uint8_t *row = R + (uint32_t)((u + c) % NU) * UNIT + r * 128;
#pragma unroll
                        for (int w = 0; w < 8; ++w)
                            times_zero4<FP16>(*reinterpret_cast<const uint4 *>(row + (((w ^ lane) & 7) << 4)), acc);
                    }
                    const bool bad = nonfinite<FP16>(acc);
                    const bool mine = bad && r < valid;
                    if (bad || r >= valid)
                        for (int c = 0; c < vc; ++c) {
                            uint8_t *row = R + (uint32_t)((u + c) % NU) * UNIT + r * 128;
#pragma unroll
                            for (int w = 0; w < 8; ++w)
                                *reinterpret_cast<uint4 *>(row + (((w ^ lane) & 7) << 4)) = make_uint4(0, 0, 0, 0);
                        }
                    mk4[r] = mine;
                    found |= mine;
                }
                found = __any_sync(0xffffffffu, found);
                if (lane == 0) any[f & 3] = found;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(fixed + (f & 3));
            }
            __syncthreads_or(!ok);
        } else {
            __syncthreads_or(false);
        }
    } else {
        // ================================ softmax ================================
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(ONE ? 216 : 184));
        const int t = warp >> 2;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + lanes + t * PK, to = tmem + lanes + T_O + t * 128;
        const int i = qt + (ONE ? 0 : t * PQ) + 32 * (warp & 3) + lane;  // this thread's query
        const int lim = i < nq ? limit(i) : 0;
        const float c = a.scale * kLog2e, raise = kRaise<FP16> / c;
        float m = -INFINITY, l = 0.f;
        for (int j = 0; j < nt[t] && ok; ++j) {
            ok = warp_wait(s_full + t, (uint32_t)j & 1u);
            if (!ok) break;
            umma::fence_after();
            uint32_t s[4][32];
#pragma unroll
            for (int g = 0; g < 4; ++g) umma::ld32_issue(ts + 32 * g, s[g]);
#pragma unroll
            for (int g = 0; g < 4; ++g) umma::wait_ld(s[g]);
            const int kt = ONE ? 2 * j + t : j;  // the key tile
            const int left = lim - kt * PK;        // its keys that this query sees
            if (kt >= jf && __any_sync(0xffffffffu, left < PK)) {
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (32 * g + e >= left) s[g][e] = 0xff800000u;  // -inf
            }
            float mx[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                mx[g] = fmaxf(__uint_as_float(s[g][0]), __uint_as_float(s[g][1]));
#pragma unroll
                for (int e = 2; e < 32; e += 2)
                    mx[g] = fmaxf(mx[g], fmaxf(__uint_as_float(s[g][e]), __uint_as_float(s[g][e + 1])));
            }
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            float f = 1.f;
            if (j == 0) {
                m = top;
            } else if (top > m + raise) {
                f = exp2_((m - top) * c);  // 0 from -inf
                m = top;
                l *= f;
            }
            // the scores' commit covers the products before it: O of this query tile is complete up to tile j - 1
            if (__any_sync(0xffffffffu, f != 1.f)) {
                for (int k = 0; k < a.dv; k += 16) {
                    uint32_t o[16];
                    umma::ld16_issue(to + k, o);
                    umma::wait_ld16(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                    st16_issue(to + k, o);
                }
                umma::wait_st();
            }
            if (kt >= jf) {
                const int f4 = (kt - jf) & 3;
                ok = warp_wait(fixed + f4, (uint32_t)((kt - jf) >> 2) & 1u);
                if (!ok) break;
                if (any[f4]) {  // a marked row that this query sees makes its sum, and so its whole output, NaN
                    const uint8_t *mk4 = mark + f4 * PK;
                    for (int e = 0; e < min(left, PK); ++e)
                        if (mk4[e]) l = NAN;
                }
            }
            const float up = m == -INFINITY ? 0.f : fmaf(-m, c, kBias<FP16>);
            const uint64_t c2 = pair(c, c), up2 = pair(up, up);
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    float x0, x1;
                    unpair(fma2(pair(__uint_as_float(s[g][e]), __uint_as_float(s[g][e + 1])), c2, up2), x0, x1);
                    x0 = exp2_(x0);
                    x1 = exp2_(x1);
                    sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pair(x0, x1));
                    w[e >> 1] = pack_weights<FP16>(x0, x1);
                }
                st16_issue(ts + 16 * g, w);
            }
            float l0, l1;
            unpair(add2(sum[0], sum[1]), l0, l1);
            l += l0 + l1;
            umma::wait_st();
            umma::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_ready + t);
        }
        if (nt[t] > 0) ok = ok && warp_wait(o_done + t, 0);
        umma::fence_after();
        float share = 1.f;  // ONE: what the even and the odd key tiles' results count for in the whole
        float other = 0.f;
        if (ONE && nt[1] > 0 && ok) {
            // every product is done once both o_done are, and so is every read of the ring
            ok = warp_wait(o_done + (t ^ 1), 0);
            umma::fence_after();
            if (t == 1) {
                half_ml[i - qt] = m;
                half_ml[PQ + i - qt] = l;
                __syncwarp();
                if (lane == 0) mbar_arrive(half_done);
            } else if (ok) {
                ok = warp_wait(half_done, 0);
                const float m1 = half_ml[i - qt], l1 = half_ml[PQ + i - qt], top = fmaxf(m, m1);
                share = m == -INFINITY ? 0.f : exp2_((m - top) * c);
                other = m1 == -INFINITY ? 0.f : exp2_((m1 - top) * c);
                l = l * share + l1 * other;
                m = top;
            }
        }
        if (ok && !(ONE && t == 1) && i - lane < nq) {
            const float inv = l == 0.f ? 0.f : 1.f / l, w0 = share * inv, w1 = other * inv;
            const int64_t row = (q_lo + i) * a.H + h;
            for (int k = 0; k < a.dv; k += 16) {
                float v[16];
                uint32_t o[16];
                if (nt[t] > 0) {
                    umma::ld16_issue(to + k, o);
                    umma::wait_ld16(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(o[e]) * w0;
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = 0.f;
                }
                if (ONE && nt[1] > 0) {
                    umma::ld16_issue(to + 128 + k, o);
                    umma::wait_ld16(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] += __uint_as_float(o[e]) * w1;
                }
                if (i < nq) {
                    uint32_t pk[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) pk[e] = pack2<FP16>(v[2 * e], v[2 * e + 1]);
                    uint4 *dst = reinterpret_cast<uint4 *>(a.out + row * a.dv + k);
                    dst[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    dst[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
                }
            }
            if (a.lse && i < nq) a.lse[row] = l == 0.f ? -INFINITY : (m * c + (__log2f(l) - kBias<FP16>)) * kLn2;
        }
        __syncthreads_or(!ok);
    }
    if (!ok && lane == 0) set_status(a.status, KDA_DEV_TIMEOUT);
    umma::fence_before();
    __syncthreads();
    if (warp == 9) umma::dealloc(tmem, 512);
}

template <bool FP16, bool ONE>
static int launch(const LatentPrefillArgs &a, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return launch_result("latent prefill: cudaGetDevice");
    if (!(done.load() >> dev & 1)) {
        if (cudaFuncSetAttribute(kda_latent_prefill_kernel<FP16, ONE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 PSMEM_MAX) != cudaSuccess)
            return launch_result("latent prefill: cudaFuncSetAttribute");
        done.fetch_or(1ull << dev);
    }
    const EncodeTiledFn enc = encoder();
    if (!enc) return fail(KDA_ERR_CUDA, "latent prefill: cuTensorMapEncodeTiled is not available");
    CUtensorMap mq, mk, mr, mv;
    const int64_t nk = std::max<int64_t>(1, a.num_k);
    // without any key the key maps are never read; the queries stand in for their memory
    const void *k = a.num_k ? (const void *)a.k : a.q, *r = a.num_k ? (const void *)a.r : a.q,
               *v = a.num_k ? (const void *)a.v : a.q;
    if (!map_3d(enc, &mq, FP16, a.q, a.nope + a.rope, a.H, a.num_q, a.q_hs, a.q_ts, 1, PQ) ||
        !map_3d(enc, &mk, FP16, k, a.nope, a.H, nk, a.k_hs, a.k_ts, 1, PK) ||
        !map_3d(enc, &mr, FP16, r, a.rope, 1, nk, a.r_ts, a.r_ts, 1, PK) ||
        !map_3d(enc, &mv, FP16, v, a.dv, a.H, nk, a.v_hs, a.v_ts, 1, PK))
        return fail(KDA_ERR_CUDA, "latent prefill: tensor map encoding failed");
    PrefillP p;
    p.a = a;
    const uint32_t kc = a.nope / 64 + 1, fixed = 1024 + 2 * kc * UNIT + PMISC;
    p.units = std::min<int>(MAX_UNITS, (PSMEM_MAX - fixed) / UNIT);
    const int rows = ONE ? PQ : 2 * PQ;
    const int most = (int)std::min<int64_t>(a.max_q, a.num_q);  // no sequence has more
    const dim3 grid(a.H, a.nseq, (most + rows - 1) / rows);
    dependent_launch(kda_latent_prefill_kernel<FP16, ONE>, grid, PNT, fixed + p.units * UNIT, st, p, mq, mk, mr, mv);
    return launch_result("kda_latent_prefill_kernel launch");
}

}  // namespace latent

int launch_latent_prefill(const LatentPrefillArgs &a, cudaStream_t st) {
    using namespace latent;
    // One query tile a CTA where there is no second one, or where all such CTAs run at once: a key tile then takes the
    // CTA 1.35 us instead of 1.95 for two query tiles (four prompts of 2048 to 8192 tokens, 32 heads: 1.70 ms against 1.22;
    // three of up to 200: 10.8 us against 12.2; eight of 64 tokens over 4,000 to 8,000 earlier ones: 158 against 176).
    const int64_t ctas = (int64_t)a.H * a.nseq * ((a.max_q + PQ - 1) / PQ);
    const bool one = a.max_q <= PQ || ctas <= current_device_sms();
    if (a.fp16) return one ? launch<true, true>(a, st) : launch<true, false>(a, st);
    return one ? launch<false, true>(a, st) : launch<false, false>(a, st);
}

}  // namespace kda
