// kda_kv_decode.cu -- grouped-query attention over the paged cache (include/kda.h: kda_kv_decode).
//
//   s_j = scale q . k_j,   o = sum_j softmax(s)_j v_j
//
// for the nq H / heads rows (query token, head of the group) that share a key-value head.  Keys and values are read once,
// 4 head_dim bytes a token and head against 4 head_dim operations for each row: with up to 64 rows bound by the bytes.
//
// Split: a unit is one (sequence, key-value head, block of 16 MT rows); its tiles of 64 tokens (32 where head_dim is above
// 128) stand in one list with those of all other units, and each CTA takes an equal, contiguous part of the list, found on
// the device from lens, so that a captured launch follows its lengths.  A unit that one CTA holds whole is written at once; one
// that is cut leaves normalised fp32 parts and the log2 of their sums in the workspace, which a second launch joins.
//
// A CTA (one on each multiprocessor) has a ring of tiles in shared memory:
//   warp 8     TMA: boxes of one head's rows of a page (or 64 of them) and 64 channels, 128-byte swizzled
//   warps 0-7  groups of warps take tiles in turn; within a group each warp has one tile of 16 rows and a slice of the tokens.
//              S = Q K^T and O += P V by m16n8k16 products from registers: with 4 to 16 rows the tensor work is a small part of
//              the time the bytes take (a tile's 32 KB come in 1400 cycles), a wide tcgen05 tile would be 48 to 60 of 64 rows
//              empty, and here S becomes P without leaving the registers of its warp.
// Each warp keeps its own running maximum and sum; they meet when the unit's part ends, in shared memory.
//
// With add_weights the scores (fp32, in units of log2) also go to the workspace, and a third launch, when the rows' sums are
// known, adds exp(s - lse) to the pages: 4 bytes written and read for each row and token, mostly in L2, where reading the keys
// again would be 2 head_dim.
#include <algorithm>

#include "kda_kv.cuh"

namespace kda {
namespace kv {

constexpr int CW = 8;                  // consuming warps
constexpr int NT = (CW + 1) * 32;      // and the producer
constexpr int PAD = 40;                // floats of a row of 32 channels where warps' outputs meet: no bank conflicts
constexpr int MAX_STAGES = 12;
constexpr uint32_t MERGE = CW * 16 * PAD * 4;
// A unit counts for this many tiles more where the list is split: beginning and ending one costs about as much.
constexpr int START = 2;

// Weights are 2^(kBias + x - m), x a score in units of log2 and m its row's maximum so far.  bf16 has the exponents of fp32;
// fp16 ends at 2^16, so its weights are moved up as far as they go: rounded relative to themselves down to 2^-28 of the
// largest, by at most 2^-39 of the largest below.
template <bool FP16>
constexpr float kBias = FP16 ? 14.f : 0.f;

template <int DP>
constexpr int kTile = DP > 128 ? 32 : 64;
template <int DP>
constexpr int kStage = kTile<DP> * DP * 4;  // bytes: keys and values
// Tokens of a warp's slice of a tile, and groups of warps that take tiles in turn.
template <int DP, int MT>
constexpr int kSlice = MT * kTile<DP> / 4 < 16 ? 16 : MT * kTile<DP> / 4;
template <int DP, int MT>
constexpr int kGroups = CW * kSlice<DP, MT> / (MT * kTile<DP>);
// Stages of the ring: a multiple of the groups, so that a stage's tiles are always the same group's.  (A group that skipped
// a use of a stage could take the phase before the skipped one for its own: their parities are equal.)
template <int DP, int MT>
constexpr int kStages = DP == 64 ? 12 : DP == 128 ? 6 : kGroups<DP, MT> == 4 ? 4 : 6;

struct Cut {  // where a CTA's part of the list begins: place `off` of unit u of sequence b; places of a whole part
    int32_t b, u, off, pad;
    int64_t per;
};

struct DecodeP {
    KvDecodeArgs a;
    int32_t groups, G, mt;
    Cut *cut;         // [groups]
    float *part;      // [groups * 2][16 mt][DP] normalised parts: those that begin a unit second
    float *part_l;    // [groups * 2][16 mt] log2 of their sums
    float *lse2;      // [n max_tokens][H] log2 of the rows' sums (add_weights)
    int64_t *base;    // [n + 1] tiles of 64 tokens before each sequence (add_weights); of one left out, its last place's - 1
    float *scores;    // [tiles][H / heads rows ...], see score_at()
};

struct Range {  // a CTA's part of the list
    int32_t b, u, off;
    int64_t lo, hi, per;
    int64_t tiles, slots;  // of the sequences before b (add_weights)
};

struct Scratch {
    int64_t scan[3][CW + 1];
    int64_t b, u, off, tiles, slots;
};

__device__ __forceinline__ int units_of(const DecodeP &p, const Seq &s) {
    return p.a.c.heads * ((s.nq * p.G + 16 * p.mt - 1) / (16 * p.mt));
}
template <int TILE>
__device__ __forceinline__ int tiles_of(const Seq &s) {
    return s.nq > 0 ? (s.len + TILE - 1) / TILE : 0;
}
__device__ __forceinline__ int64_t tiles64(const Seq &s) { return s.nq > 0 ? (s.len + 63) / 64 : 0; }

// Scores of 64 tokens of one key-value head and all rows of a sequence: [row][64], from tile `t` of those in the call.
__device__ __forceinline__ int64_t score_at(const DecodeP &p, const Seq &s, int64_t t, int hk) {
    return (t * p.a.max_tokens * p.a.H + (int64_t)hk * s.nq * p.G) * 64;
}

// f(b, s, u, first tile, tiles) for each unit's part within the CTA's part of the list.
template <int TILE, class F>
__device__ __forceinline__ void walk(const DecodeP &p, const Range &R, F f) {
    int64_t at = R.lo;
    int off = R.off, u = R.u;
    for (int b = R.b; at < R.hi && b < p.a.n; ++b, u = 0) {
        const Seq s = seq_of(p.a, b);
        const int tiles = tiles_of<TILE>(s);
        if (tiles == 0) continue;
        for (const int units = units_of(p, s); u < units && at < R.hi; ++u, off = 0) {
            const int take = (int)min((int64_t)(tiles + START - off), R.hi - at);
            const int first = max(off - START, 0), nt = max(off + take - START, 0) - first;
            if (nt > 0) f(b, s, u, first, nt, tiles);
            at += take;
        }
    }
}

// Prefix sums of the sequences' places, each thread a run of sequences.  Called by all NT threads; also writes zeros for the
// queries of empty (or bad) sequences.
template <int TILE>
__device__ __forceinline__ Range range_of(const DecodeP &p, Scratch *sh) {
    const KvDecodeArgs &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = blockIdx.x;
    const int run = (a.n + NT - 1) / NT;
    const int r0 = min(a.n, tid * run), r1 = min(a.n, r0 + run);
    int64_t mine[3] = {0, 0, 0};
    for (int b = r0; b < r1; ++b) {
        const Seq s = seq_of(a, b);
        const int t = tiles_of<TILE>(s);
        if (t) mine[0] += (int64_t)units_of(p, s) * (t + START);
        if (a.add_weights && t) {
            mine[1] += tiles64(s);
            mine[2] += s.len;
        }
    }
    int64_t before[3], total = 0;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        int64_t incl = mine[k];
        if (k == 0 || a.add_weights) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t t = __shfl_up_sync(FULL, incl, o);
                if (lane >= o) incl += t;
            }
            if (lane == 31) sh->scan[k][warp] = incl;
        }
        before[k] = incl - mine[k];
    }
    if (tid == 0) {
        sh->b = a.n;
        sh->u = sh->off = sh->tiles = sh->slots = 0;
    }
    __syncthreads();
    for (int w = 0; w <= CW; ++w) {
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (w < warp && (k == 0 || a.add_weights)) before[k] += sh->scan[k][w];
        total += sh->scan[0][w];
    }
    Range R;
    R.per = max((int64_t)1, (total + p.groups - 1) / p.groups);
    R.lo = min(total, g * R.per);
    R.hi = min(total, R.lo + R.per);
    if ((mine[0] > 0 && R.lo >= before[0] && R.lo < before[0] + mine[0]) || (a.add_weights && g == 0)) {
        int64_t at = before[0], tiles = before[1], slots = before[2];
        for (int b = r0; b < r1; ++b) {
            const Seq s = seq_of(a, b);
            const int t = tiles_of<TILE>(s);
            const int64_t places = t ? (int64_t)units_of(p, s) * (t + START) : 0;
            if (R.lo >= at && R.lo < at + places) {
                sh->b = b;
                sh->u = (R.lo - at) / (t + START);
                sh->off = (R.lo - at) % (t + START);
                sh->tiles = tiles;
                sh->slots = slots;
                if (!(a.add_weights && g == 0)) break;
            }
            at += places;
            if (t) {
                tiles += tiles64(s);
                slots += s.len;
            }
            if (a.add_weights && g == 0) {
                // sequences that pass the bound come last in what the third launch goes over, and are left out of it
                p.base[b + 1] = slots <= a.max_slots ? tiles : INT64_MAX;
                if (t && slots > a.max_slots) set_status(a.status, KDA_DEV_BAD_SEQLENS);
            }
        }
    }
    if (g == 0 && tid == 0 && a.add_weights) p.base[0] = 0;
    for (int b = blockIdx.x; b < a.n; b += gridDim.x) {
        const Seq s = seq_of(a, b);
        if (s.bits && tid == 0) set_status(a.status, s.bits);
        if (s.nq == 0 || s.len > 0) continue;
        uint4 *o = reinterpret_cast<uint4 *>(a.out + s.c0 * a.H * a.c.d);
        for (int64_t i = tid; i < (int64_t)s.nq * a.H * a.c.d / 8; i += NT) o[i] = make_uint4(0, 0, 0, 0);
        if (a.lse)
            for (int i = tid; i < s.nq * a.H; i += NT) a.lse[s.c0 * a.H + i] = -INFINITY;
    }
    __syncthreads();
    R.b = (int32_t)sh->b;
    R.u = (int32_t)sh->u;
    R.off = (int32_t)sh->off;
    R.tiles = sh->tiles;
    R.slots = sh->slots;
    if (tid == 0) p.cut[g] = Cut{R.b, R.u, R.off, 0, R.per};
    return R;
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// D += A B: A 16 x 16 (row), B 16 x 8 (column), fp32.
template <bool FP16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (FP16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
            "%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
            "%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void sync_threads(int id, int n) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// The address of 16 bytes (word w of 8) of row r of 128 swizzled bytes.
__device__ __forceinline__ uint32_t swizzled(uint32_t base, int r, int w) { return base + r * 128 + ((w ^ (r & 7)) << 4); }

using latent::exp2_;

template <bool FP16, int DP, int MT>
__global__ void __launch_bounds__(NT, 1)
    kda_kv_decode_kernel(const DecodeP p, const __grid_constant__ CUtensorMap map) {
    constexpr int TILE = kTile<DP>, STAGE = kStage<DP>, STAGES = kStages<DP, MT>;
    constexpr int CH = DP / 64;                       // chunks of 64 channels
    constexpr int CHUNK = TILE * 128;                 // bytes of one
    constexpr int KS = kSlice<DP, MT>, NG = kGroups<DP, MT>;
    constexpr int WG = CW / NG;                       // warps of a group
    static_assert(WG * KS == MT * TILE && KS % 16 == 0 && KS <= TILE && STAGES % NG == 0 && STAGES <= MAX_STAGES, "");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *merge = reinterpret_cast<float *>(sm + STAGES * STAGE);  // [CW][16][PAD]
    __shared__ uint64_t full[MAX_STAGES], empty[MAX_STAGES];
    __shared__ Scratch scratch;
    __shared__ float sm_m[CW][16], sm_l[CW][16];
    const KvDecodeArgs &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int kv = a.c.heads, G = p.G, d = a.c.d;

    if (tid == CW * 32) {
        latent::prefetch_map(&map);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, WG);
        }
        fence_mbar_init();
    }
    wait_for_previous();
    const Range R = range_of<TILE>(p, &scratch);  // its barriers show the initialised ones to all
    allow_dependent_launch();
    bool ok = true;
    int it = 0;

    if (warp == CW) {
        // ---------------------------------------------------------------- producer
        const int ps = a.c.page_size, rows = min(ps, TILE);  // tokens of a box
        const int boxes = TILE / rows;                       // of a tile, for each of keys and values and each chunk
        const int box = lane % boxes, which = lane / boxes;  // lanes of a box: chunk, keys or values
        const int chunk = which % CH, value = which / CH;
        walk<TILE>(p, R, [&](int, const Seq &s, int u, int first, int nt, int) {
            const int nrb = units_of(p, s) / kv, hk = u / nrb;
            const int32_t *trow = a.t.table + (int64_t)s.row * a.t.max_pages;
            for (int j = 0; j < nt; ++j, ++it) {
                const int st = it % STAGES;
                const int key = (first + j) * TILE + box * rows;
                int page = (int)a.c.num_pages;  // outside of the tensor: reads as zeros
                if (value < 2 && key < s.len) {
                    const int e = trow[key / ps];
                    if (e >= 0 && e < a.c.num_pages)
                        page = e;
                    else
                        set_status(a.status, KDA_DEV_BAD_PAGE);
                }
                if (ok && it >= STAGES) ok = latent::warp_wait(empty + st, (it / STAGES - 1) & 1);
                if (!ok) return;
                if (lane == 0) mbar_arrive_expect_tx(full + st, STAGE);
                __syncwarp();
                if (value < 2)
                    latent::tma_load_4d(sm + st * STAGE + (value * CH + chunk) * CHUNK + box * rows * 128, &map, chunk * 64,
                                        key % ps, value * kv + hk, page, full + st);
            }
        });
        // no copy is in flight when the CTA ends, whatever the consumers saw
        for (int i = max(0, it - STAGES); i < it; ++i)
            if (!latent::warp_wait(full + i % STAGES, (i / STAGES) & 1)) ok = false;
    } else {
        // ---------------------------------------------------------------- consumers
        const int grp = warp / WG, rt = warp % MT, slice = warp % WG / MT;
        const int quad = lane & 3, top = lane >> 2;
        const float sl = a.scale * latent::kLog2e;
        int64_t tiles_before = R.tiles, slots_before = R.slots;
        int last_b = R.b;
        walk<TILE>(p, R, [&](int b, const Seq &s, int u, int first, int nt, int tiles) {
            const int nrb = units_of(p, s) / kv, hk = u / nrb, r0 = (u - hk * nrb) * 16 * MT;
            const int rows = s.nq * G;
            bool keep_scores = a.add_weights;
            if (a.add_weights) {
                for (; last_b < b; ++last_b) {  // the sequences passed over
                    const Seq q = seq_of(a, last_b);
                    if (q.nq > 0) {
                        tiles_before += tiles64(q);
                        slots_before += q.len;
                    }
                }
                keep_scores = slots_before + s.len <= a.max_slots;
            }
            // queries, as the products' A operand
            uint32_t q[DP / 16][4];
            const uint16_t *qp[2];
            uint64_t seen[2] = {~0ull, ~0ull};
            const bool drafts = s.nq > 1 || a.tree;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = r0 + rt * 16 + top + 8 * k;
                const int t = r < rows ? r / G : 0;
                qp[k] = r < rows ? a.q + (s.c0 + t) * a.q_ts + (int64_t)(hk * G + r - t * G) * a.q_hs : nullptr;
                if (drafts) seen[k] = drafts_seen(a, s, t);
            }
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = k * 16 + 2 * quad + (e >> 1) * 8;
                    q[k][e] = qp[e & 1] && c < d ? *reinterpret_cast<const uint32_t *>(qp[e & 1] + c) : 0u;
                }
            float o[DP / 8][4];
#pragma unroll
            for (int k = 0; k < DP / 8; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[k][e] = 0.f;
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
            const int draft0 = drafts ? s.len - s.nq : s.len;  // first token that not all rows see

            for (int j = 0; j < nt; ++j, ++it) {
                if (it % NG != grp) continue;
                const int st = it % STAGES;
                if (ok) ok = latent::warp_wait(full + st, (it / STAGES) & 1);
                const int key0 = (first + j) * TILE;
                const uint32_t kb = smem_addr(sm + st * STAGE), vb = kb + CH * CHUNK;
                const bool edge = key0 + TILE > draft0;
                uint64_t poison = 0;  // drafted value rows of this warp's slice that are not finite
                if (edge) {
                    const int lo = max(draft0, key0 + slice * KS), hi = min(s.len, key0 + slice * KS + KS);
                    for (int k = lo; k < hi; ++k) {
                        const int r = k - key0;
                        uint32_t acc[4] = {0, 0, 0, 0};
                        if (lane < DP / 8)
                            latent::times_zero4<FP16>(*reinterpret_cast<const uint4 *>(sm + st * STAGE + (CH + lane / 8) * CHUNK +
                                                                                       r * 128 + (((lane & 7) ^ (r & 7)) << 4)),
                                                      acc);
                        if (__any_sync(FULL, latent::nonfinite<FP16>(acc))) poison |= 1ull << (r - slice * KS);
                    }
                    sync_threads(2 + grp, WG * 32);  // every warp has looked
                    for (int r = slice * KS; r < (slice + 1) * KS; ++r)
                        if ((key0 + r >= s.len || ((poison >> (r - slice * KS)) & 1)) && lane < DP / 8)
                            *reinterpret_cast<uint4 *>(sm + st * STAGE + (CH + lane / 8) * CHUNK + r * 128 + ((lane & 7) << 4)) =
                                make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
#pragma unroll 1
                for (int ks = 0; ks < KS; ks += 16) {
                    const int row = slice * KS + ks;  // of the tile
                    if (key0 + row >= s.len) break;
                    float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k) {
                        uint32_t w[4];
                        ldmatrix4(w, swizzled(kb + k / 4 * CHUNK, row + (lane >> 4) * 8 + (lane & 7), k % 4 * 2 + ((lane >> 3) & 1)));
                        mma<FP16>(c[0], q[k], w[0], w[1]);
                        mma<FP16>(c[1], q[k], w[2], w[3]);
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) c[n][e] *= sl;
                    if (edge) {
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int at = row + n * 8 + 2 * quad + (e & 1), key = key0 + at;
                                const int i = key - draft0;
                                if (key >= s.len || (i >= 0 && !((seen[e >> 1] >> i) & 1)))
                                    c[n][e] = -INFINITY;
                                else if ((poison >> (at - slice * KS)) & 1)
                                    c[n][e] = NAN;
                            }
                    }
                    if (keep_scores) {
                        const int64_t t64 = (key0 + row) / 64;
                        float *out = p.scores + score_at(p, s, tiles_before + t64, hk) + (key0 + row) % 64 + 2 * quad;
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int r = r0 + rt * 16 + top + 8 * e;
                                if (r < rows)
                                    *reinterpret_cast<float2 *>(out + r * 64 + n * 8) = make_float2(c[n][2 * e], c[n][2 * e + 1]);
                            }
                    }
                    float mm[2], f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = fmaxf(fmaxf(c[0][2 * e], c[0][2 * e + 1]), fmaxf(c[1][2 * e], c[1][2 * e + 1]));
                        x = fmaxf(x, __shfl_xor_sync(FULL, x, 1));
                        x = fmaxf(x, __shfl_xor_sync(FULL, x, 2));
                        x = fmaxf(x, m[e]);
                        mm[e] = x == -INFINITY ? 0.f : x;
                        f[e] = exp2_(m[e] - mm[e]);
                        m[e] = x;
                    }
                    if (__any_sync(FULL, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
                        for (int k = 0; k < DP / 8; ++k) {
                            o[k][0] *= f[0];
                            o[k][1] *= f[0];
                            o[k][2] *= f[1];
                            o[k][3] *= f[1];
                        }
                        l[0] *= f[0];
                        l[1] *= f[1];
                    }
                    uint32_t w[4];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            c[n][e] = exp2_(c[n][e] - mm[e >> 1] + kBias<FP16>);
                            l[e >> 1] += c[n][e];
                        }
                        w[2 * n] = latent::pack_weights<FP16>(c[n][0], c[n][1]);
                        w[2 * n + 1] = latent::pack_weights<FP16>(c[n][2], c[n][3]);
                    }
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k) {
                        uint32_t v[4];
                        ldmatrix4_trans(v, swizzled(vb + k / 4 * CHUNK, row + (lane & 15), k % 4 * 2 + (lane >> 4)));
                        mma<FP16>(o[2 * k], w, v[0], v[1]);
                        mma<FP16>(o[2 * k + 1], w, v[2], v[3]);
                    }
                }
                __syncwarp();
                if (lane == 0) latent::mbar_arrive(empty + st);
            }

            // the warps of each row tile meet
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[e] += __shfl_xor_sync(FULL, l[e], 1);
                l[e] += __shfl_xor_sync(FULL, l[e], 2);
                if (quad == 0) {
                    sm_m[warp][top + 8 * e] = m[e];
                    sm_l[warp][top + 8 * e] = l[e];
                }
            }
            sync_threads(1, CW * 32);
            const bool whole = nt == tiles;
            const int64_t slot = (int64_t)blockIdx.x * 2 + (first == 0);
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float M = -INFINITY, L = 0.f;
#pragma unroll
                for (int w = rt; w < CW; w += MT) M = fmaxf(M, sm_m[w][top + 8 * e]);
                const float mm = M == -INFINITY ? 0.f : M;
#pragma unroll
                for (int w = rt; w < CW; w += MT) L += sm_l[w][top + 8 * e] * exp2_(sm_m[w][top + 8 * e] - mm);
                f[e] = L == 0.f ? 0.f : exp2_(m[e] - mm) / L;
                const int r = r0 + rt * 16 + top + 8 * e;
                if (warp < MT && quad == 0 && r < rows) {
                    const float l2 = L == 0.f ? -INFINITY : mm + log2f(L) - kBias<FP16>;
                    const int t = r / G, h = hk * G + r - t * G;
                    if (!whole) {
                        p.part_l[slot * 16 * MT + rt * 16 + top + 8 * e] = l2;
                    } else {
                        if (a.lse) a.lse[(s.c0 + t) * a.H + h] = l2 * latent::kLn2;
                        if (a.add_weights) p.lse2[((int64_t)b * a.max_tokens + t) * a.H + h] = l2;
                    }
                }
            }
#pragma unroll
            for (int ch = 0; ch < DP / 32; ++ch) {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    float *w = merge + (warp * 16 + top) * PAD + n * 8 + 2 * quad;
                    *reinterpret_cast<float2 *>(w) = make_float2(o[ch * 4 + n][0] * f[0], o[ch * 4 + n][1] * f[0]);
                    *reinterpret_cast<float2 *>(w + 8 * PAD) = make_float2(o[ch * 4 + n][2] * f[1], o[ch * 4 + n][3] * f[1]);
                }
                sync_threads(1, CW * 32);
#pragma unroll
                for (int i = tid; i < MT * 128; i += CW * 32) {
                    const int row = i >> 3, c = ch * 32 + (i & 7) * 4, r = r0 + row;
                    if (r < rows && c < d) {
                        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int w = row >> 4; w < CW; w += MT) {
                            const float4 y = *reinterpret_cast<const float4 *>(merge + (w * 16 + (row & 15)) * PAD + (i & 7) * 4);
                            x.x += y.x;
                            x.y += y.y;
                            x.z += y.z;
                            x.w += y.w;
                        }
                        if (whole) {
                            const int t = r / G, h = hk * G + r - t * G;
                            *reinterpret_cast<uint2 *>(a.out + ((s.c0 + t) * a.H + h) * d + c) =
                                make_uint2(latent::pack2<FP16>(x.x, x.y), latent::pack2<FP16>(x.z, x.w));
                        } else {
                            *reinterpret_cast<float4 *>(p.part + (slot * 16 * MT + row) * DP + c) = x;
                        }
                    }
                }
                sync_threads(1, CW * 32);
            }
        });
    }
    if (!ok && lane == 0) set_status(a.status, KDA_DEV_TIMEOUT);
}

constexpr int JW = 16;  // warps of a joining CTA

// Joins the parts of the unit that the beginning of part blockIdx.x + 1 of the list cuts, if no earlier beginning does.  A
// row's parts are divided among as many warps as there are for it, a lane has channels 4 lane .. 4 lane + 3 and those 128
// further on.
template <bool FP16, int DP>
__global__ void __launch_bounds__(JW * 32) kda_kv_join_kernel(const DecodeP p) {
    constexpr int TILE = kTile<DP>, V = (DP + 127) / 128;
    __shared__ float4 sm_o[JW][V][32];
    __shared__ float sm_m[JW], sm_w[JW];
    wait_for_previous();
    allow_dependent_launch();
    const KvDecodeArgs &a = p.a;
    const int g = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Cut c = p.cut[g];
    if (c.b >= a.n || c.off <= START || c.off - c.per > START) return;
    const Seq s = seq_of(a, c.b);
    const int rem = tiles_of<TILE>(s) + START - c.off;
    const int parts = 1 + (int)((rem + c.per - 1) / c.per);
    const int nrb = units_of(p, s) / a.c.heads, hk = c.u / nrb, block = 16 * p.mt, r0 = (c.u - hk * nrb) * block;
    const int rows = min(block, s.nq * p.G - r0);
    int per_row = 1;  // warps of a row
    while (per_row * 2 * rows <= JW && per_row * 2 <= parts) per_row *= 2;
    for (int first = 0; first < rows; first += JW / per_row) {
        const int row = first + warp / per_row, k = warp % per_row;
        const bool mine = row < rows;
        auto at = [&](int i) { return ((int64_t)(g - 1 + i) * 2 + (i == 0)) * block + row; };
        float m = -INFINITY, sum = 0.f;
        float4 o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (mine) {
            for (int i = k + lane * per_row; i < parts; i += 32 * per_row) {
                const float x = p.part_l[at(i)];
                m = fmaxf(m, x);
            }
#pragma unroll
            for (int w = 16; w > 0; w >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, w));
            const float mm = m == -INFINITY ? 0.f : m;
#pragma unroll 4
            for (int i = k; i < parts; i += per_row) {
                const float w = exp2_(p.part_l[at(i)] - mm);
                sum += w;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int ch = v * 128 + 4 * lane;
                    if (ch < a.c.d) {
                        const float4 x = *reinterpret_cast<const float4 *>(p.part + at(i) * DP + ch);
                        o[v].x = fmaf(w, x.x, o[v].x);
                        o[v].y = fmaf(w, x.y, o[v].y);
                        o[v].z = fmaf(w, x.z, o[v].z);
                        o[v].w = fmaf(w, x.w, o[v].w);
                    }
                }
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) sm_o[warp][v][lane] = o[v];
        if (lane == 0) {
            sm_m[warp] = m;
            sm_w[warp] = sum;
        }
        __syncthreads();
        if (mine && k == 0) {
            float M = m;
            for (int w = 1; w < per_row; ++w) M = fmaxf(M, sm_m[warp + w]);
            const float mm = M == -INFINITY ? 0.f : M;
            float4 x[V];
#pragma unroll
            for (int v = 0; v < V; ++v) x[v] = make_float4(0.f, 0.f, 0.f, 0.f);
            float L = 0.f;
            for (int w = 0; w < per_row; ++w) {
                const float f = exp2_(sm_m[warp + w] == -INFINITY ? -INFINITY : sm_m[warp + w] - mm);
                L += f * sm_w[warp + w];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float4 y = sm_o[warp + w][v][lane];
                    x[v].x = fmaf(f, y.x, x[v].x);
                    x[v].y = fmaf(f, y.y, x[v].y);
                    x[v].z = fmaf(f, y.z, x[v].z);
                    x[v].w = fmaf(f, y.w, x[v].w);
                }
            }
            const float inv = L == 0.f ? 0.f : 1.f / L;
            const int r = r0 + row, t = r / p.G, h = hk * p.G + r - t * p.G;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int ch = v * 128 + 4 * lane;
                if (ch < a.c.d)
                    *reinterpret_cast<uint2 *>(a.out + ((s.c0 + t) * a.H + h) * a.c.d + ch) =
                        make_uint2(latent::pack2<FP16>(x[v].x * inv, x[v].y * inv), latent::pack2<FP16>(x[v].z * inv, x[v].w * inv));
            }
            if (lane == 0) {
                const float l2 = L == 0.f ? -INFINITY : mm + log2f(L);
                if (a.lse) a.lse[(s.c0 + t) * a.H + h] = l2 * latent::kLn2;
                if (a.add_weights) p.lse2[((int64_t)c.b * a.max_tokens + t) * a.H + h] = l2;
            }
        }
        __syncthreads();
    }
}

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

// Row tiles of a CTA: as many as hold all rows of a sequence, up to 4.
inline int row_tiles(int G, int max_tokens) { return G * max_tokens <= 16 ? 1 : G * max_tokens <= 32 ? 2 : 4; }
inline int padded(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

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

template <bool FP16, int DP, int MT>
int launch_as(const DecodeP &p, const CUtensorMap &map, cudaStream_t st) {
    static std::atomic<uint64_t> prepared{0};
    auto k = kda_kv_decode_kernel<FP16, DP, MT>;
    if (allow_smem(k, prepared) == cudaSuccess)
        dependent_launch(k, dim3((unsigned)p.groups), NT, kStages<DP, MT> * kStage<DP> + MERGE + 1024, st, p, map);
    int rc = launch_result("kda_kv_decode_kernel launch");
    if (rc != KDA_OK) return rc;
    if (p.groups > 1) {
        dependent_launch(kda_kv_join_kernel<FP16, DP>, dim3((unsigned)p.groups - 1), JW * 32, 0, st, p);
        rc = launch_result("kda_kv_join_kernel launch");
        if (rc != KDA_OK) return rc;
    }
    if (p.a.add_weights) {
        dependent_launch(kda_kv_weights_kernel, dim3((unsigned)p.groups * 8), WW * 32, 0, st, p);
        rc = launch_result("kda_kv_weights_kernel launch");
    }
    return rc;
}

template <bool FP16, int DP>
int launch_rows(const DecodeP &p, const CUtensorMap &map, cudaStream_t st) {
    switch (p.mt) {
        case 1: return launch_as<FP16, DP, 1>(p, map, st);
        case 2: return launch_as<FP16, DP, 2>(p, map, st);
        default: return launch_as<FP16, DP, 4>(p, map, st);
    }
}
template <bool FP16>
int launch_dims(const DecodeP &p, const CUtensorMap &map, cudaStream_t st) {
    switch (padded(p.a.c.d)) {
        case 64: return launch_rows<FP16, 64>(p, map, st);
        case 128: return launch_rows<FP16, 128>(p, map, st);
        default: return launch_rows<FP16, 256>(p, map, st);
    }
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
    p.mt = row_tiles(p.G, a.max_tokens);
    const Layout L = layout(a.c, p.groups, a.H, a.n, a.max_tokens, a.max_slots);
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    p.cut = reinterpret_cast<Cut *>(ws + L.cut);
    p.part = reinterpret_cast<float *>(ws + L.part);
    p.part_l = reinterpret_cast<float *>(ws + L.part_l);
    p.lse2 = reinterpret_cast<float *>(ws + L.lse2);
    p.base = reinterpret_cast<int64_t *>(ws + L.base);
    p.scores = reinterpret_cast<float *>(ws + L.scores);
    const latent::EncodeTiledFn enc = latent::encoder();
    if (!enc) return fail(KDA_ERR_CUDA, "kv decode: the driver has no tensor-map encoder");
    // [pages][keys and values of each head][tokens][channels] in boxes of 64 channels and a page's tokens
    const int64_t ps = a.c.page_size;
    const int64_t dims[4] = {a.c.d, ps, 2 * a.c.heads, a.c.num_pages};
    const int64_t strides[3] = {a.c.d, ps * a.c.d, a.c.page_stride};
    const int tile = padded(a.c.d) > 128 ? 32 : 64;
    const int box[4] = {64, (int)std::min<int64_t>(ps, tile), 1, 1};
    CUtensorMap map;
    if (!latent::tensor_map(enc, &map, a.c.fp16, a.c.pages, 4, dims, strides, box))
        return fail(KDA_ERR_CUDA, "kv decode: the cache's tensor map was refused");
    return a.c.fp16 ? launch_dims<true>(p, map, st) : launch_dims<false>(p, map, st);
}

}  // namespace kda
