// kda_kv_decode.cuh -- grouped-query attention over the paged cache (include/kda.h: kda_kv_decode): the kernels, which
// the files kda_kv_decode_*.cu make for each type and kind of head_dim and kda_kv_decode.cu launches.
//
//   s_j = scale q . k_j,   o = sum_j softmax(s)_j v_j
//
// for the nq H / heads rows (query token, head of the group) that share a key-value head.  Keys and values are read once,
// 4 head_dim bytes a token and head against 4 head_dim operations for each row: with up to 32 rows bound by the bytes.
//
// Split: a unit is one (sequence, key-value head, block of rows); its tiles of 16 or 24 KB (64, 32 or 16 tokens) stand in one list
// with those of all other units, and each CTA takes an equal, contiguous part of the list, found on the device from lens,
// so that a captured launch follows its lengths.  A unit that one CTA holds whole is written at once; one that is cut leaves
// normalised fp32 parts and the log2 of their sums in the workspace, which a second launch joins.
//
// A CTA has a producing and four consuming warps, two CTAs a multiprocessor; with 64 rows or more than 128 channels eight consuming warps, one
// CTA.  With heads of 128, 64 sequences of 500 to 8192 and 1000 of 10 to 200 tokens on 8 key-value heads, two CTAs against one of
// eight: 8 rows 191 and 108 us against 189 and 187; 16 rows 194 and 202 against 202 and 327; 32 rows 207 and 253 against 227
// and 371 (heads of 64: 100 and 95 against 102 and 165; 103 and 175 against 111 and 251; 110 and 195 against 126 and 278).
// It has a ring of tiles in shared memory:
//   producer   walks the list: what a unit is and its queries into a ring of two, its tiles by TMA.  A box is one head's
//              keys or values of a page (or of a tile's tokens), all channels.  (With boxes of 16 tokens x 64 channels heads of
//              128 were read at 4.4 TB/s of 6.7.)
//   consumers  take tiles in turn, each the whole tile and 8 or 16 rows of queries (two or four warps share a tile where there
//              are more).  S^T = K Q^T and O^T += V^T P^T by m16n8k16 products: tokens and channels fill the 16 rows of
//              the operand that comes from shared memory, query rows the 8 columns, so that groups of 4 to 8 heads waste
//              little; S^T becomes P^T by a register transposition.  The tensor work is a small part of the time that
//              the bytes take (16 KB in 715 cycles; 64 products of 2 cycles), and a tcgen05 tile has 64 rows at least.  Units
//              of 64 rows are bound by it: 64 % of the copy's rate, where units of up to 32 rows reach 98 (64 sequences of 9000).
// Each warp keeps its own maximum and sums; they meet when the unit's part ends, in shared memory.  The maximum is raised only by
// more than kRaise, by a vote; until then nothing is exchanged or rescaled.
//
// Weights are rounded to the cache's type for the second product, as both operands of a product have one type.  Each is off by
// half a step at most, with either sign, so that an output is off by about as much as by its own rounding: 0.0023 of the outputs' size
// in bf16 where rounding the outputs alone gives 0.0017 (fp16 0.00029, 0.00021).  Weights in two parts (a second product with what
// the first rounding left) give 0.0017, at the same time where long sequences are bound by bytes, but 1000 sequences of 10 to 200
// tokens take 117 instead of 108 us (230 instead of 203 with 16 rows), trees of 20 rows 131 instead of 122, 64 rows 205 instead of 157.
// The sums of weights are of the fp32 scores.
//
// With add_weights the scores (fp32, in units of log2) also go to the workspace, and a third launch, when the rows' sums are
// known, adds exp(s - lse) to the pages: 4 bytes written and read for each row and token, mostly in L2, where reading the keys
// again would be 2 head_dim.
#pragma once

#include <algorithm>

#include "kda_kv.cuh"

namespace kda {
namespace kv {

// Barriers of the ring, more than it has stages: a multiple of the groups of warps that take tiles in turn, so that a barrier
// is always the same group's.  (A group that skipped uses of a barrier could take an earlier phase for its own: phases are
// told apart by their parity alone.)
constexpr int BARS = 16;
// A unit counts for this many tiles more where the list is split: beginning and ending one costs about as much.
constexpr int START = 8;

using latent::exp2_;
using latent::kBias;
using latent::kRaise;

// Tokens of a tile: 16 KB (24 for 192 channels: one in 12 KB cost the producer as much as one in 16, 343 us instead of 276 for 64
// sequences of 500 to 8192 tokens and 8 key-value heads; taken as 256 channels with 64 zeros 349).
template <int DP>
constexpr int kTile = DP == 192 ? 32 : 4096 / DP;

struct Cut {  // where a CTA's part of the list begins: place `off` of unit u of sequence b, which has nq queries from c0 on and
              // units of `tiles` tiles; places of a whole part
    int64_t c0, per;
    int32_t b, u, off, nq, tiles, pad;
};

struct DecodeP {
    KvDecodeArgs a;
    int32_t groups, G, block;  // CTAs, heads of a group, rows of a unit: 8, 16, 32 or 64
    uint32_t inverse_g;        // 2^32 / G rounded up: row / G is the upper half of row * inverse_g (rows are below 2^15); 0: G is 1
    int32_t box_rows;          // tokens of a box
    Cut *cut;         // [groups]
    float *part;      // [groups * 2][block][DP] normalised parts: those that begin a unit second
    float *part_l;    // [groups * 2][block] log2 of their sums
    float *lse2;      // [n max_tokens][H] log2 of the rows' sums (add_weights)
    int64_t *base;    // [n + 1] tiles of 64 tokens before each sequence (add_weights), INT64_MAX behind those that take part;
                      // then the number of tiles
    int4 *seqs;       // [n] table row, tokens and queries (add_weights)
    float *scores;    // see score_at()
};

struct Range {  // a CTA's part of the list
    int32_t b, u, off;
    int64_t lo, hi, per;
    int64_t tiles, slots;  // of the sequences before b (add_weights)
};

struct Scratch {
    int64_t scan[3][12];
    int64_t b, u, off, tiles, slots, c0;
    int32_t nq, unit_tiles;
};

__device__ __forceinline__ int units_of(const DecodeP &p, const Seq &s) {
    return p.a.c.heads * ((s.nq * p.G + p.block - 1) / p.block);
}
__device__ __forceinline__ int over_g(const DecodeP &p, int row) {
    return p.inverse_g ? (int)__umulhi((uint32_t)row, p.inverse_g) : row;
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

// Prefix sums of the sequences' places, each thread a run of sequences.  Called by all NT threads; also writes zeros for the
// queries of empty (or bad) sequences.
template <int TILE, int NT>
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
        sh->u = sh->off = sh->tiles = sh->slots = sh->c0 = 0;
        sh->nq = sh->unit_tiles = 0;
    }
    __syncthreads();
    for (int w = 0; w < NT / 32; ++w) {
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
                sh->c0 = s.c0;
                sh->nq = s.nq;
                sh->unit_tiles = t;
                if (!(a.add_weights && g == 0)) break;
            }
            at += places;
            if (t) {
                tiles += tiles64(s);
                slots += s.len;
            }
            if (a.add_weights && g == 0) {
                // sequences that pass the bound are the last ones with tokens, and the third launch ends before them
                p.base[b + 1] = slots <= a.max_slots ? tiles : INT64_MAX;
                p.seqs[b] = make_int4(s.row, s.len, s.nq, 0);
                if (slots > a.max_slots) {
                    if (t) set_status(a.status, KDA_DEV_BAD_SEQLENS);
                    if (t && slots - s.len <= a.max_slots) p.base[a.n + 1] = tiles - tiles64(s);
                } else if (b == a.n - 1) {
                    p.base[a.n + 1] = tiles;
                }
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
    if (tid == 0) p.cut[g] = Cut{sh->c0, R.per, R.b, R.u, R.off, sh->nq, sh->unit_tiles, 0};
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
__device__ __forceinline__ void ldmatrix2(uint32_t (&r)[2], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
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

// The 8 x 8 matrix that the warp holds, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ void sync_threads(int id, int n) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
// The same, with one answer for all: whether any of them says so.
__device__ __forceinline__ bool sync_threads_or(int id, int n, bool x) {
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %3, 0;\n bar.red.or.pred q, %1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
                 : "=r"(r)
                 : "r"(id), "r"(n), "r"((uint32_t)x)
                 : "memory");
    return r != 0;
}
// Loads that are the first to leave L2 again: what they read is read once, and scores and parts should stay.
__device__ __forceinline__ uint64_t evict_first() {
    uint64_t r;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(r));
    return r;
}
__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *map, int c0, int c1, int c2, int c3, int c4,
                                            uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4, "
        "%5, %6}], [%7], %8;" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int c0, int c1, int c2, uint64_t *bar,
                                            uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, "
        "%4}], [%5], %6;" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}

// What a CTA does of one unit: tiles [first, first + nt) of `tiles`.
struct Part {
    Seq s;
    int32_t b, hk, r0, first, nt, tiles;
    int64_t tile64;       // tiles of 64 tokens of the sequences before (add_weights)
    int32_t keep_scores;
};

// CW: consuming warps of a CTA, 8 / CW CTAs on a multiprocessor.
template <int DP, int RW, int RG, int CW>
struct Config {
    static constexpr int TILE = kTile<DP>, CH = DP / 64, MT = TILE / 16;
    static constexpr int STAGE = TILE * DP * 4;            // bytes of a tile: keys and values
    static constexpr int MERGE = CW * 64 * 8 * 4;          // bytes where warps' outputs meet, one of two: 64 channels of 8 rows
    // Threads: the consumers, the producer, and with eight consumers three idle warps that make the producer's warpgroup whole
    // (registers come in warpgroups): launched with 168 registers a thread (64,512 of 65,536), of which the consumers
    // take 216 and the others give down to 72: 256 * 216 + 128 * 72 = 64,512, what the launch holds.
    static constexpr int NT = CW == 8 ? 384 : (CW + 1) * 32;
    static constexpr int ROOM = (CW == 8 ? kSmemMax : kSmemMax / (8 / CW) - 1024) - 4096;  // (1 KB of each CTA is the system's)
    static constexpr int ROWS = 8 * RW * RG;               // rows of a unit
    static constexpr int QROW = DP * 2 + 16;               // bytes of a query in shared memory: no bank conflicts
    static constexpr int QBYTES = ROWS * QROW;
    static constexpr int TURNS = CW == 4 && RG == 2 ? 1 : 2;  // buffers for outputs (one where a fifth stage needs the room)
    static constexpr int FIT = (ROOM - TURNS * MERGE - 2 * QBYTES) / STAGE, STAGES = FIT < 12 ? FIT : 12;
    static constexpr int SMEM = 1024 + STAGES * STAGE + TURNS * MERGE + 2 * QBYTES;
    static constexpr int GROUPS = CW / RG;
    static_assert(RG <= CW && BARS % GROUPS == 0 && STAGES <= BARS && STAGES >= 4, "");
    static constexpr bool Q_REGS = DP * RW <= 256;         // queries stay in registers
};

// RW: 8 rows each of a warp (1 or 2); RG: warps that share a tile, with rows of their own.  WHOLE: a box has all channels
// (head_dim a multiple of 64), else there is a box for each 64.  With it known here, a tile's rows lie at constant distances and
// loads from shared memory need no arithmetic: 16 trees of 20 rows 130 -> 121 us, 16 rows of 256 channels 193 -> 184.5.
template <bool FP16, int DP, int RW, int RG, int CW, bool WHOLE>
__global__ void __launch_bounds__(Config<DP, RW, RG, CW>::NT, 8 / CW)
    kda_kv_decode_kernel(const DecodeP p, const __grid_constant__ CUtensorMap map) {
    using C = Config<DP, RW, RG, CW>;
    constexpr int TILE = C::TILE, CH = C::CH, MT = C::MT, ROWS = C::ROWS, QROW = C::QROW, STAGES = C::STAGES, NT = C::NT;
    constexpr int STAGE = C::STAGE, MERGE = C::MERGE;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *merge = reinterpret_cast<float *>(sm + STAGES * STAGE);  // [2][CW][64 channels][8 rows]
    uint8_t *qs = sm + STAGES * STAGE + C::TURNS * MERGE;                   // [2][ROWS][QROW]
    __shared__ uint64_t full[BARS], empty[BARS], q_full[2], q_empty[2];
    __shared__ Scratch scratch;
    __shared__ Part parts[2];
    __shared__ float sm_m[CW][8 * RW], sm_l[CW][8 * RW];
    __shared__ float row_m[ROWS], row_inv[ROWS];  // of the unit's rows: maximum, 1 / sum
    __shared__ int32_t row_out[ROWS];             // and words from the sequence's outputs to theirs
    const KvDecodeArgs &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int kv = a.c.heads, G = p.G, d = a.c.d;

    if (tid == CW * 32) {
        latent::prefetch_map(&map);
        for (int s = 0; s < BARS; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, RG);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(q_full + s, 1);
            mbar_init(q_empty + s, CW);
        }
        fence_mbar_init();
    }
    // channels behind the last are 0 in the queries, as they are in keys and values
    for (int i = tid; i < 2 * C::QBYTES / 16; i += NT) reinterpret_cast<uint4 *>(qs)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    wait_for_previous();
    const Range R = range_of<TILE, NT>(p, &scratch);  // its barriers show the initialised ones to all
    allow_dependent_launch();
    bool ok = true;

    if (warp >= CW) {
        if constexpr (CW == 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp > CW) return;
        // ---------------------------------------------------------------- producer
        // lanes of a box, which begins with token `box` of a tile: keys and values
        const int ps = a.c.page_size, rows = p.box_rows, box = (lane >> 1) * rows, value = lane & 1;
        const int small = ps < TILE ? TILE / ps : 0, box_page = ps < TILE ? box / ps : 0;
        const uint32_t num_pages = (uint32_t)a.c.num_pages;
        const uint64_t policy = evict_first();
        int it = 0, st = 0, n = 0;
        int64_t at = R.lo, tiles64_before = R.tiles, slots_before = R.slots;
        int off = R.off, u = R.u, b0 = R.b, left = 0;
        Seq mine = {};
        for (int b = R.b; ok && at < R.hi && b < a.n; ++b, u = 0) {
            if (left == 0) {  // the next 32 sequences, one a lane
                b0 = b;
                left = 32;
                mine = b + lane < a.n ? seq_of(a, b + lane) : Seq{};
            }
            --left;
            Seq s;
            s.c0 = __shfl_sync(FULL, mine.c0, b - b0);
            s.nq = __shfl_sync(FULL, mine.nq, b - b0);
            s.len = __shfl_sync(FULL, mine.len, b - b0);
            s.row = __shfl_sync(FULL, mine.row, b - b0);
            s.bits = 0;
            const int tiles = tiles_of<TILE>(s);
            if (tiles == 0) continue;
            const int nrb = units_of(p, s) / kv, total = s.nq * G;
            const int32_t *trow = a.t.table + (int64_t)s.row * a.t.max_pages;
            for (const int units = nrb * kv; ok && u < units && at < R.hi; ++u, off = 0) {
                const int take = (int)min((int64_t)(tiles + START - off), R.hi - at);
                const int first = max(off - START, 0), nt = max(off + take - START, 0) - first;
                at += take;
                if (nt == 0) continue;
                // the table's entries by 32 at a time, the next ones on their way while these are used
                int page0 = first * TILE / ps, in_page = first * TILE - page0 * ps;
                const int pages = (s.len - 1) / ps + 1;
                auto entries = [&](int from) { return from + lane < pages ? trow[from + lane] : (int32_t)num_pages; };
                int32_t now = entries(page0), next = entries(page0 + 32);
                int in_now = 0;  // the tile's first page among these
                const int hk = u / nrb, r0 = (u - hk * nrb) * ROWS, live = min(ROWS, total - r0);
                const int slot = n & 1;
                if (n >= 2) ok = latent::warp_wait(q_empty + slot, (n / 2 - 1) & 1);
                if (!ok) break;
                if (lane == 0) {
                    parts[slot] = Part{s, b, hk, r0, first, nt, tiles, tiles64_before,
                                       a.add_weights && slots_before + s.len <= a.max_slots};
                    mbar_arrive_expect_tx(q_full + slot, live * d * 2);
                }
                __syncwarp();
                for (int r = lane; r < live; r += 32) {
                    const int t = over_g(p, r0 + r);
                    bulk_g2s(qs + slot * C::QBYTES + r * QROW,
                             a.q + (s.c0 + t) * a.q_ts + (int64_t)(hk * G + r0 + r - t * G) * a.q_hs, d * 2, q_full + slot);
                }
                ++n;
                const int at_row = (value * kv + hk) * ps;
                for (int j = 0, rest = s.len - first * TILE - box; j < nt; ++j, ++it, rest -= TILE) {
                    uint32_t page = (uint32_t)__shfl_sync(FULL, now, (in_now + box_page) & 31);
                    const bool there = box < TILE && rest > 0;
                    if (there && page >= num_pages) set_status(a.status, KDA_DEV_BAD_PAGE);
                    if (!there || page >= num_pages) page = num_pages;  // outside of the tensor: reads as zeros
                    const int in_box = in_page;
                    in_now += small;  // pages of a tile
                    in_page += small ? 0 : TILE;
                    if (in_page == ps) in_page = 0, ++in_now;
                    if (in_now == 32) {
                        page0 += 32;
                        in_now = 0;
                        now = next;
                        next = entries(page0 + 32);
                    }
                    if (it >= STAGES) ok = latent::warp_wait(empty + ((it - STAGES) & (BARS - 1)), ((it - STAGES) / BARS) & 1);
                    if (!ok) break;
                    uint64_t *bar = full + (it & (BARS - 1));
                    if (lane == 0) mbar_arrive_expect_tx(bar, STAGE);
                    __syncwarp();
                    if (box < TILE) {
                        uint8_t *to = sm + st * STAGE + value * (STAGE / 2) + box * (DP * 2);
                        if (WHOLE)
                            tma_load_5d(to, &map, 0, 0, 0, (at_row + in_box) / 8, (int)page, bar, policy);
                        else
                            for (int ch = 0; ch < CH; ++ch)
                                tma_load_3d(to + ch * rows * 128, &map, ch * 64, at_row + in_box, (int)page, bar, policy);
                    }
                    if (++st == STAGES) st = 0;
                }
            }
            if (a.add_weights) {
                tiles64_before += tiles64(s);
                slots_before += s.len;
            }
        }
        if (n >= 2 && ok) ok = latent::warp_wait(q_empty + (n & 1), (n / 2 - 1) & 1);
        if (lane == 0) {
            parts[n & 1].nt = 0;  // the end
            mbar_arrive_expect_tx(q_full + (n & 1), 0);
        }
        // no copy is in flight when the CTA ends, whatever the consumers saw
        for (int i = max(0, it - STAGES); i < it; ++i)
            if (!latent::warp_wait(full + i % BARS, (i / BARS) & 1)) ok = false;
    } else {
        if constexpr (CW == 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        // ---------------------------------------------------------------- consumers
        const int grp = warp / RG, rg = warp % RG;  // rows rg * 8 RW of the unit's
        const int quad = lane & 3, top = lane >> 2;
        const int lane7 = lane & 7;
        // bytes from 64 channels of a token to the next 64, and from 8 tokens to the next 8; of a box: [8 tokens][chunk][token]
        // [64], or [chunk][token][64] (see cache_map)
        const int rows = p.box_rows;
        const uint32_t chunk = WHOLE ? 1024 : rows * 128, eight = WHOLE ? CH * 1024 : 1024;
        auto token_at = [&](int r) {  // a token's first 64 channels within a tile's keys or values, r a multiple of 8
            return WHOLE ? r * (DP * 2) : (r & ~(rows - 1)) * (DP * 2) + (r & (rows - 1)) * 128;
        };
        // scores stay as the products are until the exponential, whose argument is one operation then
        const float sl = a.scale * latent::kLog2e, raise_by = kRaise<FP16> / sl;
        const uint64_t sl2 = latent::pair(sl, sl);
        int it = 0;
        for (int n = 0;; ++n) {
            const int slot = n & 1;
            if (ok) ok = latent::warp_wait(q_full + slot, (n / 2) & 1);
            // a warp whose wait gave up goes on to here, so that all leave together
            if (sync_threads_or(1, CW * 32, !ok) || parts[slot].nt == 0) break;
            const Part w = parts[slot];
            const Seq &s = w.s;
            const int total = s.nq * G;
            const uint32_t qb = smem_addr(qs + slot * C::QBYTES + rg * 8 * RW * QROW);
            // queries as the products' B operand: of 8 rows two words a step of 16 channels
            uint32_t q[C::Q_REGS ? DP / 16 : 1][RW][2];
            auto load_q = [&](uint32_t (&x)[RW][2], int k) {
                if constexpr (RW == 2) {
                    uint32_t r[4];
                    ldmatrix4(r, qb + ((lane >> 4) * 8 + lane7) * QROW + k * 32 + ((lane >> 3) & 1) * 16);
                    x[0][0] = r[0], x[0][1] = r[1], x[1][0] = r[2], x[1][1] = r[3];
                } else {
                    ldmatrix2(x[0], qb + lane7 * QROW + k * 32 + ((lane >> 3) & 1) * 16);
                }
            };
            if constexpr (C::Q_REGS) {
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) load_q(q[k], k);
                __syncwarp();
                if (lane == 0) latent::mbar_arrive(q_empty + slot);
            }
            float o[DP / 16][RW][4];
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                for (int h = 0; h < RW; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[k][h][e] = 0.f;
            // Rows behind the unit's last hold queries of a unit before, perhaps another sequence's.  Nothing is above their
            // maximum, so that they never have the others' raised; what they come to (0 or NaN) stays in their column of the products
            // and is not written.
            float m[RW][2], l[RW][2];
#pragma unroll
            for (int h = 0; h < RW; ++h)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    m[h][f] = w.r0 + rg * 8 * RW + h * 8 + 2 * quad + f < total ? -INFINITY : INFINITY;
                    l[h][f] = 0.f;
                }
            const bool drafts = s.nq > 1 || a.tree;
            const int draft0 = drafts ? s.len - s.nq : s.len;  // first token that not all rows see

            const int it0 = it;
            it += w.nt;
            for (int j = (grp - it0) & (C::GROUPS - 1); j < w.nt; j += C::GROUPS) {
                const int i = it0 + j;
                if (ok) ok = latent::warp_wait(full + (i & (BARS - 1)), (i / BARS) & 1);
                uint8_t *tile = sm + i % STAGES * STAGE;
                const int key0 = (w.first + j) * TILE;
                const bool edge = key0 + TILE > draft0;
                // 16 bytes `c` (8 channels each) of the value row of token r
                auto value_word = [&](int r, int c) {
                    return reinterpret_cast<uint4 *>(tile + STAGE / 2 + token_at(r & ~7) + (c >> 3) * chunk + (r & 7) * 128 +
                                                     (((c ^ r) & 7) << 4));
                };
                uint64_t poison = 0;  // drafted value rows that are not finite
                if (edge) {
                    for (int k = max(draft0, key0); k < min(s.len, key0 + TILE); ++k) {
                        uint32_t acc[4] = {0, 0, 0, 0};
                        if (lane < DP / 8) latent::times_zero4<FP16>(*value_word(k - key0, lane), acc);
                        if (__any_sync(FULL, latent::nonfinite<FP16>(acc))) poison |= 1ull << (k - key0);
                    }
                    if (RG > 1) sync_threads(2 + grp, RG * 32);  // every warp has looked
                    __syncwarp();
                    for (int k = max(0, s.len - key0) * (DP / 8) + lane; k < TILE * (DP / 8); k += 32)
                        *value_word(k / (DP / 8), k % (DP / 8)) = make_uint4(0, 0, 0, 0);
                    for (uint64_t x = poison; x; x &= x - 1)
                        if (lane < DP / 8) *value_word(__ffsll(x) - 1, lane) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                // S^T: tokens 16 t + top (+ 8), rows 8 h + 2 quad (+ 1)
                float c[MT][RW][4];
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int h = 0; h < RW; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) c[t][h][e] = 0.f;
                const uint32_t tb = smem_addr(tile);
                uint32_t at[MT];  // this lane's token
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    at[t] = tb + token_at(t * 16) + ((lane >> 3) & 1) * eight + lane7 * 128;
                }
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    if constexpr (!C::Q_REGS) load_q(q[0], k);
                    uint32_t(&qk)[RW][2] = q[C::Q_REGS ? k : 0];
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        uint32_t x[4];
                        ldmatrix4(x, at[t] + k / 4 * chunk + (((k % 4 * 2 + (lane >> 4)) ^ lane7) << 4));
#pragma unroll
                        for (int h = 0; h < RW; ++h) mma<FP16>(c[t][h], x, qk[h][0], qk[h][1]);
                    }
                }
                if (edge) {
#pragma unroll
                    for (int h = 0; h < RW; ++h)
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            const int r = w.r0 + rg * 8 * RW + h * 8 + 2 * quad + f;
                            const uint64_t seen = drafts && r < total ? drafts_seen(a, s, over_g(p, r)) : ~0ull;
#pragma unroll
                            for (int t = 0; t < MT; ++t)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const int row = t * 16 + top + 8 * e, draft = key0 + row - draft0;
                                    if (key0 + row >= s.len || (draft >= 0 && !((seen >> draft) & 1)))
                                        c[t][h][2 * e + f] = -INFINITY;
                                    else if ((poison >> row) & 1)
                                        c[t][h][2 * e + f] = NAN;
                                }
                        }
                }
                if (w.keep_scores) {
#pragma unroll
                    for (int h = 0; h < RW; ++h)
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            const int r = w.r0 + rg * 8 * RW + h * 8 + 2 * quad + f;
                            float *out = p.scores + score_at(p, s, w.tile64 + key0 / 64, w.hk) + r * 64 + key0 % 64 + top;
                            if (r < total) {
#pragma unroll
                                for (int t = 0; t < MT; ++t) {
                                    out[t * 16] = c[t][h][f] * sl;
                                    out[t * 16 + 8] = c[t][h][2 + f] * sl;
                                }
                            }
                        }
                }
                float x[RW][2];
                bool raise = false;
#pragma unroll
                for (int h = 0; h < RW; ++h)
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        x[h][f] = fmaxf(c[0][h][f], c[0][h][2 + f]);
#pragma unroll
                        for (int t = 1; t < MT; ++t) x[h][f] = fmaxf(x[h][f], fmaxf(c[t][h][f], c[t][h][2 + f]));
                        raise |= x[h][f] > m[h][f] + raise_by;
                    }
                if (__any_sync(FULL, raise)) {
#pragma unroll
                    for (int h = 0; h < RW; ++h)
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            float y = x[h][f];
                            y = fmaxf(y, __shfl_xor_sync(FULL, y, 4));
                            y = fmaxf(y, __shfl_xor_sync(FULL, y, 8));
                            y = fmaxf(y, __shfl_xor_sync(FULL, y, 16));
                            y = fmaxf(y, m[h][f]);
                            // a score past what fp32 holds: all weights NaN, or none yet
                            if (fabsf(y * sl) == INFINITY) y = y > 0.f ? NAN : -INFINITY;
                            const float z = y == -INFINITY ? 1.f : exp2_((m[h][f] - y) * sl);
                            m[h][f] = y;
                            l[h][f] *= z;
#pragma unroll
                            for (int k = 0; k < DP / 16; ++k) {
                                o[k][h][f] *= z;
                                o[k][h][2 + f] *= z;
                            }
                        }
                }
                // P^T, as the second product's B operand
                uint32_t b[MT][RW][2];
#pragma unroll
                for (int h = 0; h < RW; ++h) {
                    float up[2];
#pragma unroll
                    for (int f = 0; f < 2; ++f) up[f] = m[h][f] == -INFINITY ? kBias<FP16> : fmaf(-m[h][f], sl, kBias<FP16>);
                    const uint64_t up2 = latent::pair(up[0], up[1]);
                    uint64_t sum = latent::pair(l[h][0], l[h][1]);
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            latent::unpair(latent::fma2(latent::pair(c[t][h][e], c[t][h][e + 1]), sl2, up2), c[t][h][e], c[t][h][e + 1]);
                            c[t][h][e] = exp2_(c[t][h][e]);
                            c[t][h][e + 1] = exp2_(c[t][h][e + 1]);
                            sum = latent::add2(sum, latent::pair(c[t][h][e], c[t][h][e + 1]));
                        }
                        b[t][h][0] = transposed(latent::pack_weights<FP16>(c[t][h][0], c[t][h][1]));
                        b[t][h][1] = transposed(latent::pack_weights<FP16>(c[t][h][2], c[t][h][3]));
                    }
                    latent::unpair(sum, l[h][0], l[h][1]);
                }
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        // V^T: 16 channels of 16 tokens
                        uint32_t v[4], y[4];
                        ldmatrix4_trans(v, at[t] + k / 4 * chunk + STAGE / 2 + (((k % 4 * 2 + (lane >> 4)) ^ lane7) << 4));
                        y[0] = v[0], y[1] = v[2], y[2] = v[1], y[3] = v[3];
#pragma unroll
                        for (int h = 0; h < RW; ++h) mma<FP16>(o[k][h], y, b[t][h][0], b[t][h][1]);
                    }
                __syncwarp();
                if (lane == 0) latent::mbar_arrive(empty + (i & (BARS - 1)));
            }
            if constexpr (!C::Q_REGS) {
                __syncwarp();
                if (lane == 0) latent::mbar_arrive(q_empty + slot);
            }

            // the warps of each group of rows meet
#pragma unroll
            for (int h = 0; h < RW; ++h)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    m[h][f] *= sl;  // in units of log2 from here on
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) l[h][f] += __shfl_xor_sync(FULL, l[h][f], x);
                    if (top == 0) {
                        sm_m[warp][h * 8 + 2 * quad + f] = m[h][f];
                        sm_l[warp][h * 8 + 2 * quad + f] = l[h][f];
                    }
                }
            sync_threads(1, CW * 32);
            const bool whole = w.nt == w.tiles;
            const int64_t part = (int64_t)blockIdx.x * 2 + (w.first == 0);
            if (tid < ROWS) {  // a row a thread (with 64 rows there are four warps at least)
                const int g = tid / (8 * RW), i = tid % (8 * RW), r = w.r0 + tid;
                float M = -INFINITY, L = 0.f;
#pragma unroll
                for (int v = 0; v < CW / RG; ++v) M = fmaxf(M, sm_m[v * RG + g][i]);
                const float mm = M == -INFINITY ? 0.f : M;
#pragma unroll
                for (int v = 0; v < CW / RG; ++v) L += sm_l[v * RG + g][i] * exp2_(sm_m[v * RG + g][i] - mm);
                row_m[tid] = mm;
                row_inv[tid] = L == 0.f ? 0.f : 1.f / L;
                if (r < total) {
                    const float l2 = L == 0.f ? -INFINITY : mm + log2f(L) - kBias<FP16>;
                    const int t = over_g(p, r), head = w.hk * G + r - t * G;
                    row_out[tid] = (t * a.H + head) * d;
                    if (!whole) {
                        p.part_l[part * ROWS + tid] = l2;
                    } else {
                        if (a.lse) a.lse[(s.c0 + t) * a.H + head] = l2 * latent::kLn2;
                        if (a.add_weights) p.lse2[((int64_t)w.b * a.max_tokens + t) * a.H + head] = l2;
                    }
                }
            }
            sync_threads(1, CW * 32);
            uint16_t *out = a.out + s.c0 * a.H * d;
            int turn = 0;
#pragma unroll
            for (int h = 0; h < RW; ++h) {
                float scale[2];
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const int row = rg * 8 * RW + h * 8 + 2 * quad + f;
                    scale[f] = exp2_(m[h][f] - row_m[row]) * row_inv[row];
                }
#pragma unroll
                for (int ch = 0; ch < CH; ++ch)
                    if (ch * 64 < d) {
                        float *half = merge + turn * (MERGE / 4);
                        if (C::TURNS == 2)
                            turn ^= 1;
                        else if (h + ch > 0)
                            sync_threads(1, CW * 32);  // all have read what is there
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float *to = half + ((warp * 64 + k * 16 + top) * 8 + 2 * quad);
                            const float(&y)[4] = o[ch * 4 + k][h];
                            *reinterpret_cast<float2 *>(to) = make_float2(y[0] * scale[0], y[1] * scale[1]);
                            *reinterpret_cast<float2 *>(to + 64) = make_float2(y[2] * scale[0], y[3] * scale[1]);
                        }
                        sync_threads(1, CW * 32);
#pragma unroll
                        for (int k = tid; k < RG * 256; k += CW * 32) {  // a thread has two channels of a row
                            const int g = k >> 8, pair = (k >> 3) & 31, row = g * 8 * RW + h * 8 + (k & 7), chn = ch * 64 + pair * 2;
                            if (w.r0 + row < total && chn < d) {
                                float x = 0.f, y = 0.f;
#pragma unroll
                                for (int v = 0; v < CW / RG; ++v) {
                                    const float *from = half + ((v * RG + g) * 64 + pair * 2) * 8 + (k & 7);
                                    x += from[0];
                                    y += from[8];
                                }
                                if (whole)
                                    *reinterpret_cast<uint32_t *>(out + row_out[row] + chn) = latent::pack2<FP16>(x, y);
                                else
                                    *reinterpret_cast<float2 *>(p.part + (part * ROWS + row) * DP + chn) = make_float2(x, y);
                            }
                        }
                    }
            }
        }
    }
    if (!ok && lane == 0) set_status(a.status, KDA_DEV_TIMEOUT);
}

constexpr int JW = 16;  // warps of a joining CTA

// Joins the parts of a cut unit: the CTAs of all beginnings of parts that lie within it share its rows; a unit of 64 rows with few of
// them has up to four CTAs for each, 16 rows a CTA (16 sequences of 64 tokens: this launch 13 -> 7 us; with up to 32 rows the CTAs
// without work cost as much as it gives).  A row's parts are divided among as many warps as there are
// for it; a lane has channels 4 lane .. 4 lane + 3 and those 128 further on.
template <bool FP16, int DP>
__global__ void __launch_bounds__(JW * 32) kda_kv_join_kernel(const DecodeP p) {
    constexpr int V = (DP + 127) / 128;
    __shared__ float4 sm_o[JW][V][32];
    __shared__ float sm_m[JW], sm_w[JW];
    wait_for_previous();
    allow_dependent_launch();
    const KvDecodeArgs &a = p.a;
    const int g = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Cut c = p.cut[g];
    if (c.b >= a.n || c.off <= START) return;  // nothing of the unit lies before
    const int nth = (int)((c.off - START - 1) / c.per);  // this is the unit's nth beginning, from 0, with tiles before it
    const int64_t rem = c.tiles + START - (c.off - nth * c.per);
    const int parts = 1 + (int)((rem + c.per - 1) / c.per), g0 = g - nth - 1;  // the first part is CTA g0's
    const int total = c.nq * p.G, nrb = (total + p.block - 1) / p.block, hk = c.u / nrb, r0 = (c.u - hk * nrb) * p.block;
    const int rows = min(p.block, total - r0);
    const int ways = min((int)gridDim.y, (rows + JW * (parts - 1) - 1) / (JW * (parts - 1)));  // CTAs for each beginning
    if (blockIdx.y >= ways) return;
    const int share = (parts - 1) * ways, turn = nth * ways + blockIdx.y;
    const int mine = rows > turn ? (rows - turn + share - 1) / share : 0;  // rows turn, turn + share, ... are this CTA's
    int per_row = 1;  // warps of a row
    while (per_row * 2 * mine <= JW && per_row * 2 <= parts) per_row *= 2;
    for (int first = 0; first < mine; first += JW / per_row) {
        const int row = turn + (first + warp / per_row) * share, k = warp % per_row;
        const bool here = row < rows;
        auto at = [&](int i) { return ((int64_t)(g0 + i) * 2 + (i == 0)) * p.block + row; };
        float m = -INFINITY, sum = 0.f;
        float4 o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (here) {
            for (int i = k + lane * per_row; i < parts; i += 32 * per_row) m = fmaxf(m, p.part_l[at(i)]);
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
        if (here && k == 0) {
            float M = m;
            for (int w = 1; w < per_row; ++w) M = fmaxf(M, sm_m[warp + w]);
            const float mm = M == -INFINITY ? 0.f : M;
            float4 x[V];
#pragma unroll
            for (int v = 0; v < V; ++v) x[v] = make_float4(0.f, 0.f, 0.f, 0.f);
            float L = 0.f;
            for (int w = 0; w < per_row; ++w) {
                const float f = exp2_(sm_m[warp + w] - mm);  // (of warps whose parts have no weight: 0)
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
            const int r = r0 + row, t = over_g(p, r), h = hk * p.G + r - t * p.G;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int ch = v * 128 + 4 * lane;
                if (ch < a.c.d)
                    *reinterpret_cast<uint2 *>(a.out + ((c.c0 + t) * a.H + h) * a.c.d + ch) =
                        make_uint2(latent::pack2<FP16>(x[v].x * inv, x[v].y * inv), latent::pack2<FP16>(x[v].z * inv, x[v].w * inv));
            }
            if (lane == 0) {
                const float l2 = L == 0.f ? -INFINITY : mm + log2f(L);
                if (a.lse) a.lse[(c.c0 + t) * a.H + h] = l2 * latent::kLn2;
                if (a.add_weights) p.lse2[((int64_t)c.b * a.max_tokens + t) * a.H + h] = l2;
            }
        }
        __syncthreads();
    }
}

// Keys' and then values' rows of a page, [pages][heads, keys then values, x tokens / 8][chunks of 64 channels][8 tokens][64], in
// boxes of `rows` tokens with all their channels, so that the copy reads 8 whole rows of the cache at a time and 64 channels of 8
// tokens are one swizzled block of shared memory.  Where head_dim is no multiple of 64, [pages][...x tokens][head_dim] in boxes of
// `rows` tokens x 64 channels, of which those behind the last read as zeros.
inline bool cache_map(const KvCacheArgs &c, int rows, bool whole, int padded, CUtensorMap *map) {
    const latent::EncodeTiledFn enc = latent::encoder();
    if (!enc) return false;
    const int64_t tokens = (int64_t)2 * c.heads * c.page_size, d = c.d;
    if (whole) {
        const int64_t dims[5] = {64, 8, d / 64, tokens / 8, c.num_pages}, strides[4] = {d, 64, 8 * d, c.page_stride};
        const int box[5] = {64, 8, padded / 64, rows / 8, 1};
        return latent::tensor_map(enc, map, c.fp16, c.pages, 5, dims, strides, box);
    }
    const int64_t dims[3] = {d, tokens, c.num_pages}, strides[2] = {d, c.page_stride};
    const int box[3] = {64, rows, 1};
    return latent::tensor_map(enc, map, c.fp16, c.pages, 3, dims, strides, box);
}

template <bool FP16, int DP, int RW, int RG, int CW, bool WHOLE>
int launch_as(DecodeP p, cudaStream_t st) {
    using C = Config<DP, RW, RG, CW>;
    p.groups = current_device_sms() * (8 / CW);
    p.box_rows = std::min(p.a.c.page_size, C::TILE);
    CUtensorMap map;
    if (!cache_map(p.a.c, p.box_rows, WHOLE, DP, &map))
        return fail(KDA_ERR_CUDA, "kv decode: the cache's tensor map was refused");
    static std::atomic<uint64_t> prepared{0};
    auto k = kda_kv_decode_kernel<FP16, DP, RW, RG, CW, WHOLE>;
    if (allow_smem(k, prepared) == cudaSuccess) dependent_launch(k, dim3((unsigned)p.groups), C::NT, C::SMEM, st, p, map);
    int rc = launch_result("kda_kv_decode_kernel launch");
    if (rc == KDA_OK && p.groups > 1) {
        dependent_launch(kda_kv_join_kernel<FP16, DP>, dim3((unsigned)p.groups - 1, p.block > 32 ? p.block / JW : 1), JW * 32, 0, st, p);
        rc = launch_result("kda_kv_join_kernel launch");
    }
    return rc;
}

template <bool FP16, int DP, int CW, bool WHOLE>
int launch_rows(const DecodeP &p, cudaStream_t st) {
    switch (p.block) {
        case 8: return launch_as<FP16, DP, 1, 1, CW, WHOLE>(p, st);
        case 16: return launch_as<FP16, DP, 2, 1, CW, WHOLE>(p, st);
        case 32: return launch_as<FP16, DP, 2, 2, CW, WHOLE>(p, st);
        default: return launch_as<FP16, DP, 2, 4, 8, WHOLE>(p, st);
    }
}

inline int padded(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : d <= 192 ? 192 : 256; }

template <bool FP16, bool WHOLE>
int launch_decode_of(const DecodeP &p, cudaStream_t st) {
    switch (padded(p.a.c.d)) {
        case 64: return launch_rows<FP16, 64, 4, WHOLE>(p, st);
        case 128: return launch_rows<FP16, 128, 4, WHOLE>(p, st);
        case 192: return launch_rows<FP16, 192, 8, WHOLE>(p, st);
        default: return launch_rows<FP16, 256, 8, WHOLE>(p, st);
    }
}

// Each in a file of its own, so that they compile side by side; head_dim a multiple of 64, or not.
int launch_decode_bf16(const DecodeP &p, cudaStream_t st);
int launch_decode_fp16(const DecodeP &p, cudaStream_t st);
int launch_decode_bf16_odd(const DecodeP &p, cudaStream_t st);
int launch_decode_fp16_odd(const DecodeP &p, cudaStream_t st);

}  // namespace kv
}  // namespace kda
