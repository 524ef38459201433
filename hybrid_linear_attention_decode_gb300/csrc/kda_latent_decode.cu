// kda_latent_decode.cu -- absorbed latent attention over the paged cache (include/kda.h: kda_latent_decode).
//
//   s_rj = scale q_r . x_j,   o_r = sum_j softmax(s_r)_j c_j,   x_j = [c_j | r_j]
//
// for the R = queries x heads rows of a sequence, all over the same cache rows x_j.  The cache is read once, so
// with few rows the bytes bound the call: 2 (rank + rope) a token, against 2 R (2 rank + rope) operations.
//
// Split: the 64-token tiles of all sequences form one list, and each group of CTAs takes an equal, contiguous
// part of it (found on the device from lens, so a captured launch follows its lengths).  A group has one CTA for
// each 64 of H max_tokens rows, side by side in the grid, so that they read the same tiles at the same time and all but
// one of them from L2; where a sequence has fewer rows, the CTAs of the others idle (64 sequences of one query, 32 heads:
// 67 us with max_tokens 1, 171 with 8).  A sequence that a group holds whole is written at once; one that is cut
// leaves normalised fp32 parts and the log2 of their sums in the workspace, which a second launch joins.
//
// A tile, by one CTA of 12 warps (one CTA per SM, ring of tiles in shared memory):
//   warp 4   TMA: boxes of 8 tokens with all their channels, into K-major 128-byte-swizzled rows
//   warp 5   S = Q X^T (M 64 rows, N 64 tokens, k = channel) and O += P C (M 64 rows, N 256 or 128 channels,
//            k = token; C is the same shared memory, read MN-major).  With M 64 an accumulator has half of the
//            tensor-memory lanes: O, rank columns wide, takes lanes 16-31 of each warp's quarter, Q and S lanes 0-15.
//            (The transposed product O^T += C^T P^T would leave no row of M unused, but an MN-major A operand
//            of M 128, N 32 took 187 cycles an instruction; as B of M 64, N 256 it takes 156.)
//   warps 6-9  the queries of the next sequence into tensor memory, as soon as the last S of this one is done
//   warps 0-3  softmax of S (8 or 16 rows a warp, a quad of threads a row), P to shared memory, and at the end O out.
// S of a tile is issued before P V of the one before, so the softmax overlaps the products.
// The running maximum is raised only by more than kRaise; then its warp rescales the rows of O in place.
// Weights P are rounded to the element type for the second product (its operands are 16-bit), in fp16 moved up by
// 2^kBias; their sum is kept in fp32 from the unrounded weights.
#include <algorithm>

#include "kda_latent.cuh"

namespace kda {
namespace latent {

constexpr int TILE = 64;             // tokens per tile
constexpr int NR = 64;               // rows (query, head) per CTA
// Threads of the main kernel: 12 warps, the last two idle (registers come in warpgroups).  Launched with 168 registers a
// thread (64,512 of 65,536); the softmax warpgroup takes 184, the others give down to 160: 128 * 184 + 256 * 160 = 64,512, what
// the launch holds.  (With the roles unsplit the softmax spilled: 64 sequences 73.7 us instead of 71.0.)
constexpr int NT = 384;
constexpr int SW = 4;                // softmax warps
// A sequence counts for this many tiles more where the list is split: ending one and beginning the next on a CTA costs
// about as much time.  us with 0 / 2 / 5 / 8: 64 sequences of 500 to 8192 tokens, 32 heads, rank 512: 73.3 / 71.5 / 70.8 / 72.4, rank
// 256: 47.2 / 46.2 / 44.0 / 45.1, rank 128: 40.5 / 38.9 / 36.9 / 38.3; 16 of these with 128 heads, rank 512: 53.5 / 45.8 / 42.8 /
// 43.5; 200 of up to 3000, 16 heads, rank 128: 49.7 / 46.4 / 45.4 / 46.6; 300 of 100 to 900, 32 heads, rank 128: 38.5 / 34.7 / 33.4 /
// 34.3, rank 512: 57.5 / 51.0 / 52.6 / 56.4 (the one where 2 would do better).
constexpr int START = 5;
constexpr int QW = 4;                // query warps, one for each quarter of the lanes
constexpr uint32_t ATOM = 1024;      // bytes of 8 tokens x 64 channels
constexpr int MAX_STAGES = 8;
constexpr uint32_t SMEM_MAX = 227 * 1024;
constexpr uint32_t MISC = 1536;      // barriers and small arrays
constexpr int CW = 8;                // warps of a combine CTA

struct Meta {  // a cut sequence: its parts, the first group, whether its part there is the group's second, its output rows
    int32_t pieces, group, second, rows;
    int64_t row0;
};

struct DecodeP {
    LatentDecodeArgs a;
    int32_t groups, nrt, nst, nch, by_seq, split_rope;
    Meta *meta;    // [n] when by_seq, else [groups]
    float *part;   // [groups * 2][nrt][NR][rank] normalised parts
    float *part_l; // [groups * 2][nrt][NR] log2 of their sums
};

struct Seq {
    int64_t c0;
    int32_t nq, len, row, tiles, bits;
};

__device__ __forceinline__ Seq seq_of(const LatentDecodeArgs &a, int b) {
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
    s.tiles = s.nq > 0 ? (s.len + TILE - 1) / TILE : 0;
    return s;
}

// Rows of a row tile go to the four softmax warps by 8 where that holds them all, else by 16.
__device__ __forceinline__ int rows_per_warp(int rows) { return rows <= 32 ? 8 : 16; }

__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, %0;" ::"n"(SW * 32) : "memory"); }
// The group's part [at, end) of the list, which begins `off` places into sequence b: `f(b, s, first tile, tiles, n, v)`
// for each sequence that has tiles in it, the n-th of the group, with v its place in the list; `get(b)` reads the sequence.
template <class G, class F>
__device__ __forceinline__ void walk(const DecodeP &p, int b, int32_t off, int64_t at, int64_t end, int64_t row0, G get,
                                     F f) {
    int piece = 0;
    for (; at < end && b < p.a.n; ++b, off = 0) {
        const Seq s = get(b);
        if (s.tiles == 0) continue;
        const int32_t take = (int32_t)min((int64_t)(s.tiles + START - off), end - at);
        const int32_t first = max(off - START, 0), nt = max(off + take - START, 0) - first;
        if (nt > 0) {
            if (row0 < s.nq * p.a.H && !f(b, s, first, nt, piece, at - off)) return;
            ++piece;
        }
        at += take;
    }
}

// A group's part of the list: places [lo, hi), beginning `off` places into sequence b; per: places of a whole part.
struct Range {
    int32_t b, off;
    int64_t lo, hi, per;
};

struct Scratch {  // shared memory of group_range()
    int64_t scan[NT / 32];
    int64_t b, off;
};

// Prefix sums of the sequences' places, each thread a run of sequences.  Called by all NT threads; also writes zeros for the
// queries of empty (or bad) sequences.  `leader`: the CTA of the group that keeps its meta record.
__device__ __forceinline__ Range group_range(const DecodeP &p, int g, bool leader, Scratch *sh) {
    const LatentDecodeArgs &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = a.c.rank, H = a.H;
    const int run = (a.n + NT - 1) / NT;
    const int r0 = min(a.n, tid * run), r1 = min(a.n, r0 + run);
    int64_t mine = 0;
    for (int b = r0; b < r1; ++b) {
        const int32_t t = seq_of(a, b).tiles;
        mine += t ? t + START : 0;
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == 31) sh->scan[warp] = incl;
    if (tid == 0) {
        sh->b = a.n;
        sh->off = 0;
    }
    __syncthreads();
    int64_t before = incl - mine, total = 0;
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += sh->scan[w];
        total += sh->scan[w];
    }
    Range R;
    R.per = (total + p.groups - 1) / p.groups;
    R.lo = min(total, g * R.per);
    R.hi = min(total, R.lo + R.per);
    if (mine > 0 && R.lo >= before && R.lo < before + mine) {
        int64_t at = before;
        for (int b = r0; b < r1; ++b) {
            int32_t t = seq_of(a, b).tiles;
            t += t ? START : 0;
            if (R.lo < at + t) {
                sh->b = b;
                sh->off = R.lo - at;
                break;
            }
            at += t;
        }
    }
    if (!p.by_seq && leader && tid == 0) p.meta[g].pieces = 0;
    for (int b = blockIdx.x; b < a.n; b += gridDim.x) {
        const Seq s = seq_of(a, b);
        if (s.bits && tid == 0) set_status(a.status, s.bits);
        if (s.tiles > 0) continue;
        if (p.by_seq && tid == 0) p.meta[b].pieces = 0;
        uint4 *o = reinterpret_cast<uint4 *>(a.out + s.c0 * H * rank);
        for (int64_t i = tid; i < (int64_t)s.nq * H * rank / 8; i += NT) o[i] = make_uint4(0, 0, 0, 0);
        if (a.lse)
            for (int i = tid; i < s.nq * H; i += NT) a.lse[s.c0 * H + i] = -INFINITY;
    }
    __syncthreads();
    R.b = (int32_t)sh->b;
    R.off = (int32_t)sh->off;
    return R;
}

// The record of a cut sequence, by the leader of the group in which it begins (places v .. v + START + tiles of the list).
__device__ __forceinline__ void record(const DecodeP &p, const Range &R, int g, int b, const Seq &s, int piece, int64_t v) {
    Meta m;
    m.pieces = (int32_t)((v + START + s.tiles - 1) / R.per - g) + 1;
    m.group = g;
    m.second = piece > 0;
    m.rows = s.nq * p.a.H;
    m.row0 = s.c0 * p.a.H;
    if (p.by_seq)
        p.meta[b] = m;
    else if (m.pieces > 1)
        p.meta[g] = m;
}

// Bits of the drafted tokens that the query token t of a sequence sees.
__device__ __forceinline__ uint64_t drafts_seen(const LatentDecodeArgs &a, const Seq &s, int t) {
    const uint64_t chain = t >= 63 ? ~0ull : (2ull << t) - 1, all = s.nq >= 64 ? ~0ull : (1ull << s.nq) - 1;
    return (a.tree ? a.tree[s.c0 + t] : chain) & all;
}

// Rows [lo, hi) of a tile made ready for the second product by the four warps of a warpgroup (warp index w4): a row
// behind the sequence becomes zeros (a zero weight times NaN is NaN), and so does a drafted row that is not finite, which
// `poison` marks.  valid: rows of the sequence; drafts: first drafted row that is looked over (valid: none).  nl, nw: 16-byte
// words of a row's latents and of all its channels here.
template <bool FP16>
__device__ __forceinline__ void fix_tile(uint8_t *x, uint32_t group, int w4, int lane, int valid, int drafts, int nl, int nw,
                                         uint32_t *poison) {
    for (int r = valid + w4; r < TILE; r += 4)
        for (int w = lane; w < nl; w += 32)
            *reinterpret_cast<uint4 *>(x + (r >> 3) * group + (w >> 3) * ATOM + (r & 7) * 128 + ((w & 7) << 4)) =
                make_uint4(0, 0, 0, 0);
    for (int r = drafts + w4; r < valid; r += 4) {
        uint32_t acc[4] = {0, 0, 0, 0};
        for (int w = lane; w < nw; w += 32)
            times_zero4<FP16>(*reinterpret_cast<const uint4 *>(x + (r >> 3) * group + (w >> 3) * ATOM + (r & 7) * 128 +
                                                               (((w ^ r) & 7) << 4)),
                              acc);
        const bool bad = __any_sync(0xffffffffu, nonfinite<FP16>(acc));
        if (bad)
            for (int w = lane; w < nl; w += 32)
                *reinterpret_cast<uint4 *>(x + (r >> 3) * group + (w >> 3) * ATOM + (r & 7) * 128 + ((w & 7) << 4)) =
                    make_uint4(0, 0, 0, 0);
        if (lane == 0) poison[r] = bad;
    }
    fence_proxy_async_smem();
}

template <bool FP16>
__global__ void __launch_bounds__(NT, 1)
    kda_latent_decode_kernel(const DecodeP p, const __grid_constant__ CUtensorMap map_c,
                             const __grid_constant__ CUtensorMap map_r) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const LatentDecodeArgs &a = p.a;
    const int nch = p.nch, nst = p.nst, rank = a.c.rank, d = rank + a.c.rope, H = a.H;
    uint8_t *P = sm;             // [NR][128 bytes]
    uint8_t *KV = P + NR * 128;  // [nst][TILE / 8][nch][8][128 bytes]: 8 tokens' rows, then the next 8
    const uint32_t GROUP = (uint32_t)nch * ATOM, STAGE = TILE / 8 * GROUP;
    uint64_t *full = reinterpret_cast<uint64_t *>(KV + (uint32_t)nst * STAGE);
    uint64_t *empty = full + MAX_STAGES;
    uint64_t *s_full = empty + MAX_STAGES;  // [2]
    uint64_t *p_ready = s_full + 2;
    uint64_t *q_ready = p_ready + 1;
    uint64_t *q_free = q_ready + 1;
    uint64_t *q_sent = q_free + 1;
    uint64_t *drain = q_sent + 1;
    Scratch *scratch = reinterpret_cast<Scratch *>(drain + 1);
    uint32_t *poison = reinterpret_cast<uint32_t *>(scratch + 1);  // [2][TILE] rows that are not finite, by tile parity
    Seq *seq_s = reinterpret_cast<Seq *>(poison + 2 * TILE);
    uint32_t *tmem_s = reinterpret_cast<uint32_t *>(seq_s + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rt = blockIdx.x % p.nrt, g = blockIdx.x / p.nrt;
    // tensor memory: Q (288 columns) and two S buffers of 64 in lanes 0-15 of each quarter, O in lanes 16-31
    constexpr uint32_t T_S = 384, T_O = 16u << 16;

    if (tid == 32 * 4) {
        prefetch_map(&map_c);
        if (p.split_rope) prefetch_map(&map_r);
    }
    if (warp == 5) umma::alloc(tmem_s, 512);
    if (tid == 0) {
        for (int s = 0; s < MAX_STAGES; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        mbar_init(s_full, 1);
        mbar_init(s_full + 1, 1);
        mbar_init(p_ready, SW);
        mbar_init(q_ready, QW);
        mbar_init(q_free, 1);
        mbar_init(q_sent, QW);
        mbar_init(drain, 1);
        fence_mbar_init();
    }

    umma::fence_before();
    wait_for_previous();
    const Range R = group_range(p, g, rt == 0, scratch);
    umma::fence_after();
    const uint32_t tmem = *tmem_s;
    allow_dependent_launch();
    bool ok = true;
    auto read = [&](int b) { return seq_of(a, b); };

    if (warp >= SW) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 160;");
        if (warp == 4) {
            // ================================ producer ================================
            // A box is 8 tokens with all their channels: 8 (rank + rope) 2 bytes in a row in the cache, whatever the page
            // size.  (Boxes of 64 tokens x 64 channels, which read 128 bytes of each row at a time, reached 4.0 TB/s of DRAM.)
            const int ps = a.c.page_size;
            int it = 0, st = 0;
            uint32_t ph = 1;  // a fresh ring is empty
            walk(p, R.b, R.off, R.lo, R.hi, rt * NR, read, [&](int, const Seq &s, int32_t off, int32_t nt, int, int64_t) {
                const int32_t *trow = a.t.table + (int64_t)s.row * a.t.max_pages;
                for (int j = 0; j < nt; ++j, ++it) {
                    const int key = (off + j) * TILE + (lane & 7) * 8;  // below 2^31: len is
                    int page = (int)a.c.num_pages;                      // a box outside the tensor reads as zeros
                    if (lane < 8 && key < s.len) {
                        const int e = trow[key / ps];
                        if (e >= 0 && e < a.c.num_pages)
                            page = e;
                        else
                            set_status(a.status, KDA_DEV_BAD_PAGE);
                    }
                    ok = it == 0 ? warp_wait(q_sent, 0) : it < nst || warp_wait(empty + st, ph);
                    if (!ok) return false;
                    if (lane == 0) mbar_arrive_expect_tx(full + st, STAGE);
                    __syncwarp();
                    if (lane < 8) {
                        uint8_t *dst = KV + (uint32_t)st * STAGE + lane * GROUP;
                        tma_load_4d(dst, &map_c, 0, key % ps, 0, page, full + st);
                        if (p.split_rope) tma_load_3d(dst + rank / 64 * ATOM, &map_r, 0, key % ps, page, full + st);
                    }
                    if (++st == nst) st = 0, ph ^= 1;
                }
                return true;
            });
            if (__syncthreads_or(!ok)) {  // copies still in flight land before the CTA ends (short bounded waits)
                for (int k = 0; k < min(it, nst); ++k) {
                    st = st ? st - 1 : nst - 1;
                    mbar_wait(full + st, (uint32_t)((it - 1 - k) / nst) & 1u, 10000000ull);
                }
            }
        } else if (warp == 5) {
            // ================================ MMA issuer ================================
            const uint32_t id_s = umma::idesc(kFmt<FP16>, 64, TILE);
            const uint32_t id_o = umma::idesc(kFmt<FP16>, 64, min(rank, 256)) | kBMajorMN;
            const uint32_t id_o2 = umma::idesc(kFmt<FP16>, 64, max(rank - 256, 128)) | kBMajorMN;  // the rest of rank > 256
            const uint64_t dp = umma::sdesc(smem_addr(P));
            const uint64_t dx0 = sdesc_at(smem_addr(KV), 0, GROUP), dc0 = sdesc_at(smem_addr(KV), ATOM, GROUP);
            const int ncr = rank / 64, kr = a.c.rope / 16;  // full chunks; instructions of the rotary chunk
            const uint32_t stage_words = STAGE >> 4, k_words = 2 * GROUP >> 4;  // of a stage, of 16 tokens
            uint32_t pieces = 0;
            int it = 0, st = 0;  // tile whose P V comes next, and its stage
            uint32_t ph = 0;     // parity of the stage's full barrier
            walk(p, R.b, R.off, R.lo, R.hi, rt * NR, read, [&](int, const Seq &, int32_t, int32_t nt, int, int64_t) {
                ok = warp_wait(q_ready, pieces++ & 1u);
                if (!ok) return false;
                umma::fence_after();
                auto issue_s = [&](int buf, int stage, bool last) {
                    if (!elect_one()) return;
                    const uint32_t ts = tmem + T_S + buf * TILE;
                    uint32_t tq = tmem;
                    uint64_t dx = dx0 + (uint64_t)(stage * stage_words);
                    for (int c = 0; c < ncr; ++c) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) mma_ts(ts, tq + 8 * k, dx + 2 * k, id_s, k > 0 || c > 0);
                        tq += 32;
                        dx += ATOM >> 4;
                    }
                    if (kr == 4) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) mma_ts(ts, tq + 8 * k, dx + 2 * k, id_s, true);
                    } else {
                        for (int k = 0; k < kr; ++k) mma_ts(ts, tq + 8 * k, dx + 2 * k, id_s, true);
                    }
                    umma::commit(s_full + buf);
                    if (last) umma::commit(q_free);  // this sequence's queries are read
                };
                bool issued = false;  // S of tile `it`
                for (int j = 0; j < nt; ++j, ++it) {
                    if (!issued) {
                        ok = warp_wait(full + st, ph);
                        if (!ok) return false;
                        umma::fence_after();
                        issue_s(it & 1, st, j + 1 == nt);
                    }
                    const int st1 = st + 1 == nst ? 0 : st + 1;
                    const uint32_t ph1 = st1 ? ph : ph ^ 1u;
                    // whichever comes first: the weights of this tile, or the rows of the next
                    issued = false;
                    uint64_t t0 = 0;
                    for (uint32_t spin = 1; !__all_sync(0xffffffffu, mbar_test(p_ready, it & 1u)); ++spin) {
                        if (!issued && j + 1 < nt && __all_sync(0xffffffffu, mbar_test(full + st1, ph1))) {
                            umma::fence_after();
                            issue_s((it + 1) & 1, st1, j + 2 == nt);
                            issued = true;
                        }
                        if ((spin & 255u) == 0) {
                            const uint64_t t = global_timer_ns();
                            if (!t0) t0 = t;
                            if (__any_sync(0xffffffffu, t - t0 > kWaitLimitNs)) {
                                ok = false;
                                return false;
                            }
                        }
                    }
                    umma::fence_after();
                    if (elect_one()) {
                        const uint64_t dc = dc0 + (uint64_t)(st * stage_words);
#pragma unroll
                        for (int k = 0; k < TILE / 16; ++k)
                            umma::mma_bf16(tmem + T_O, dp + 2 * k, dc + (uint64_t)(k * k_words), id_o, j > 0 || k > 0);
                        if (rank > 256) {
#pragma unroll
                            for (int k = 0; k < TILE / 16; ++k)
                                umma::mma_bf16(tmem + T_O + 256, dp + 2 * k, dc + (uint64_t)(k * k_words + (4 * ATOM >> 4)), id_o2,
                                               j > 0 || k > 0);
                        }
                        umma::commit(empty + st);  // O holds this tile, and its stage is free
                    }
                    __syncwarp();
                    st = st1;
                    ph = ph1;
                }
                return true;
            });
            if (__syncthreads_or(!ok)) {
                if (elect_one()) umma::commit(drain);
                mbar_wait(drain, 0, 10000000ull);
            }
        } else if (warp >= 10) {
            __syncthreads_or(false);
        } else if (warp >= 6) {
            // ================================ queries ================================
            const int w4 = warp & 3;                                 // quarter of the lanes
            const uint32_t tq = tmem + ((uint32_t)(32 * w4) << 16);
            uint32_t pieces = 0;
            walk(p, R.b, R.off, R.lo, R.hi, rt * NR, read, [&](int, const Seq &s, int32_t, int32_t, int, int64_t) {
                const int rows = min(NR, s.nq * H - rt * NR);
                const int rw = rows_per_warp(rows), i0 = rw * w4 + (lane >> 2);  // this thread's rows: i0 and, if rw 16, i0 + 8
                const uint2 *src[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int r = rt * NR + i0 + 8 * k, t = r / H, h = r - t * H;
                    src[k] = reinterpret_cast<const uint2 *>(a.q + (s.c0 + t) * a.q_ts + h * a.q_hs) + (lane & 3);
                }
                // Rounds of 128 channels (64 columns; this thread's 8-byte words 4n + lane % 4 of them), three rounds of loads in
                // flight.  The first of them are sent before the first tile's copies: those fill the memory system's queues for
                // microseconds, and no product can begin without the queries.
                constexpr int RB = 3;
                for (int ch0 = 0; ch0 < d; ch0 += 128 * RB) {
                    uint32_t v[RB][32];
#pragma unroll
                    for (int u = 0; u < RB; ++u)
#pragma unroll
                        for (int n = 0; n < 8; ++n)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int ch = ch0 + 128 * u;
                                uint2 x = make_uint2(0, 0);
                                if (8 * k < rw && i0 + 8 * k < rows && ch + 16 * n < d) x = load_ordinary(src[k] + ch / 4 + 4 * n);
                                v[u][4 * n + 2 * k] = x.x;
                                v[u][4 * n + 2 * k + 1] = x.y;
                            }
                    if (ch0 == 0) {
                        if (pieces == 0) {
                            for (int ch = 128 * RB; ch < d; ch += 64)  // a line of each row in 16 lanes
#pragma unroll
                                for (int k = 0; k < 2; ++k)
                                    if ((lane & 3) == 0 && 8 * k < rw && i0 + 8 * k < rows)
                                        asm volatile("prefetch.global.L2 [%0];" ::"l"(src[k] + ch / 4));
                            __syncwarp();
                            if (lane == 0) mbar_arrive(q_sent);
                        } else {
                            ok = warp_wait(q_free, (pieces - 1) & 1u);
                            if (!ok) return false;
                            umma::fence_after();
                        }
                    }
#pragma unroll
                    for (int u = 0; u < RB; ++u)
                        if (ch0 + 128 * u < d) st16x64_issue(tq + (ch0 + 128 * u) / 2, v[u]);
                }
                ++pieces;
                umma::wait_st();
                umma::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_ready);
                return true;
            });
            __syncthreads_or(!ok);
        }
    } else {
        // ================================ softmax ================================
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        // These warps meet at named barriers, so they take every decision alike: one thread reads each sequence
        // for all, and a wait that gives up leads on through the same barriers (without further waits) to the end.
        auto read_once = [&](int b) {
            softmax_sync();
            if (tid == 0) *seq_s = seq_of(a, b);
            softmax_sync();
            return *seq_s;
        };
        auto wait = [&](uint64_t *bar, uint32_t parity) { ok = __all_sync(0xffffffffu, ok && mbar_wait(bar, parity)); };
        const uint32_t quad = tmem + ((uint32_t)(32 * warp) << 16);
        const float c = a.scale * kLog2e, raise = kRaise<FP16> / c;
        const int nw = d / 8;
        int it = 0;
        int st_prev = 0;          // stage and parity of the empty barrier of tile it - 1
        uint32_t ph_prev = 0;
        int st = 0;
        uint32_t ph = 0;
        walk(p, R.b, R.off, R.lo, R.hi, rt * NR, read_once, [&](int b, const Seq &s, int32_t off, int32_t nt, int piece, int64_t v) {
            const int rows = min(NR, s.nq * H - rt * NR);
            // this thread's rows of the row tile, i0 and (where a warp has 16) i0 + 8, are rows i0p, i0p + 8 of the products
            const int rw = rows_per_warp(rows), i0 = rw * warp + (lane >> 2), i0p = 16 * warp + (lane >> 2);
            const int nk = rw / 8;
            const bool act = rw * warp < rows;
            const int64_t orow = s.c0 * H + rt * NR;  // output row of the row tile's first row
            if (rt == 0 && tid == 0 && off == 0) record(p, R, g, b, s, piece, v);
            // what the thread's two rows see among the drafted tokens
            const int base = s.len - s.nq;
            uint64_t see[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int i = i0 + 8 * k;
                see[k] = drafts_seen(a, s, i < rows ? (rt * NR + i) / H : 0);
            }
            const bool scan_drafts = s.nq > 1 || a.tree;
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
            for (int j = 0; j < nt; ++j, ++it) {
                const int key0 = (off + j) * TILE;
                wait(s_full + (it & 1), (uint32_t)(it >> 1) & 1u);
                umma::fence_after();
                const bool tail = key0 + TILE > base;
                if (tail) {
                    // marks of two tiles: a warp may be here while another still reads those of the tile before, but not
                    // two tiles ahead, because P needs the products of the tile before, which need all warps' weights
                    wait(full + st, ph);
                    const int valid = min(TILE, s.len - key0);
                    fix_tile<FP16>(KV + (uint32_t)st * STAGE, GROUP, warp, lane, valid,
                                   scan_drafts ? max(0, base - key0) : valid, rank / 8, nw, poison + (it & 1) * TILE);
                    softmax_sync();
                }
                uint32_t sr[32];  // 4n + i: row i0 + 8*(i/2), token 8n + 2*(lane%4) + i%2
                bool raised = false;
                float f[2] = {1.f, 1.f};
                if (act) {
                    ld16x64_issue(quad + T_S + (it & 1) * TILE, sr);
                    umma::wait_ld(sr);
                    if (tail) {
#pragma unroll
                        for (int e = 0; e < TILE / 2; ++e) {
                            const int col = 8 * (e >> 2) + 2 * (lane & 3) + (e & 1), dr = key0 + col - base;
                            if (dr >= 0 && (dr >= 64 || !(see[(e >> 1) & 1] >> dr & 1))) sr[e] = 0xff800000u;  // -inf
                        }
                        // a marked row that a query sees makes its sum, and so its whole output, NaN
                        if (scan_drafts)
                            for (int r = max(0, base - key0); r < min(TILE, s.len - key0); ++r)
                                if (poison[(it & 1) * TILE + r])
#pragma unroll
                                    for (int k = 0; k < 2; ++k)
                                        if (see[k] >> (key0 + r - base) & 1) l[k] = NAN;
                    }
                    float mx[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (k >= nk) break;
                        float y[2];
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            constexpr int HALF = TILE / 16;  // registers 4n + .. of half the columns
                            y[u] = -INFINITY;
#pragma unroll
                            for (int n = u * HALF; n < (u + 1) * HALF; ++n)
                                y[u] = fmaxf(y[u], fmaxf(__uint_as_float(sr[4 * n + 2 * k]),
                                                         __uint_as_float(sr[4 * n + 2 * k + 1])));
                        }
                        mx[k] = fmaxf(y[0], y[1]);
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (k >= nk) break;
                        mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 1));
                        mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 2));
                        if (j == 0) {
                            m[k] = mx[k];
                        } else if (mx[k] > m[k] + raise) {
                            f[k] = exp2_((m[k] - mx[k]) * c);  // 0 from -inf
                            m[k] = mx[k];
                            l[k] *= f[k];
                            raised = true;
                        }
                    }
                }
                if (it > 0) {  // O and P are this warp's again
                    wait(empty + st_prev, ph_prev);
                    umma::fence_after();
                }
                if (__any_sync(0xffffffffu, raised)) {
                    for (int ch = 0; ch < rank; ch += 64) {
                        uint32_t o[32];
                        ld16x64_issue(quad + T_O + ch, o);
                        umma::wait_ld(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f[(e >> 1) & 1]);
                        st16x64_issue(quad + T_O + ch, o);
                    }
                    umma::wait_st();
                }
                if (act) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (k >= nk) break;
                        const float up = m[k] == -INFINITY ? 0.f : fmaf(-m[k], c, kBias<FP16>);
                        const uint64_t c2 = pair(c, c), up2 = pair(up, up);
                        const int i = i0p + 8 * k;
                        uint8_t *prow = P + i * 128 + 4 * (lane & 3);
                        uint64_t sum = 0;
#pragma unroll
                        for (int n = 0; n < TILE / 8; ++n) {
                            float p0, p1;
                            unpair(fma2(pair(__uint_as_float(sr[4 * n + 2 * k]), __uint_as_float(sr[4 * n + 2 * k + 1])), c2,
                                        up2),
                                   p0, p1);
                            p0 = exp2_(p0);
                            p1 = exp2_(p1);
                            sum = add2(sum, pair(p0, p1));
                            *reinterpret_cast<uint32_t *>(prow + (((n ^ i) & 7) << 4)) = pack_weights<FP16>(p0, p1);
                        }
                        float s0, s1;
                        unpair(sum, s0, s1);
                        l[k] += s0 + s1;
                    }
                }
                fence_proxy_async_smem();
                umma::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready);
                st_prev = st;
                ph_prev = ph;
                if (++st == nst) st = 0, ph ^= 1;
            }
            // ---- the piece is done: O / l out ----
            const bool whole = off == 0 && nt == s.tiles;
            const int64_t slot = ((int64_t)g * 2 + (piece > 0)) * p.nrt + rt;
            wait(empty + st_prev, ph_prev);
            umma::fence_after();
            if (act) {
                float inv[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    inv[k] = 0.f;
                    l[k] += __shfl_xor_sync(0xffffffffu, l[k], 1);
                    l[k] += __shfl_xor_sync(0xffffffffu, l[k], 2);
                    const int i = i0 + 8 * k;
                    if (k >= nk) break;
                    inv[k] = l[k] == 0.f ? 0.f : 1.f / l[k];
                    if ((lane & 3) == 0) {
                        const float l2 = l[k] == 0.f ? -INFINITY : m[k] * c + (__log2f(l[k]) - kBias<FP16>);
                        if (!whole)
                            p.part_l[slot * NR + i] = l2;
                        else if (a.lse && i < rows)
                            a.lse[orow + i] = l2 * kLn2;
                    }
                }
                uint16_t *out = a.out + (orow + i0) * rank + 2 * (lane & 3);
                float *part = p.part + (slot * NR + i0) * rank + 2 * (lane & 3);
                auto put = [&](const uint32_t *o, int ch) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (k >= nk || i0 + 8 * k >= rows) break;
#pragma unroll
                        for (int n = 0; n < 8; ++n) {
                            const float v0 = __uint_as_float(o[4 * n + 2 * k]) * inv[k];
                            const float v1 = __uint_as_float(o[4 * n + 2 * k + 1]) * inv[k];
                            const int at8 = 8 * k * rank + ch + 8 * n;
                            if (whole)
                                *reinterpret_cast<uint32_t *>(out + at8) = pack2<FP16>(v0, v1);
                            else
                                *reinterpret_cast<float2 *>(part + at8) = make_float2(v0, v1);
                        }
                    }
                };
                for (int ch = 0; ch < rank; ch += 128) {  // two loads in flight
                    uint32_t o0[32], o1[32];
                    ld16x64_issue(quad + T_O + ch, o0);
                    ld16x64_issue(quad + T_O + ch + 64, o1);
                    umma::wait_ld(o0);
                    umma::wait_ld(o1);
                    put(o0, ch);
                    put(o1, ch + 64);
                }
            }
            umma::fence_before();
            return true;
        });
        __syncthreads_or(!ok);
    }
    if (!ok && lane == 0) set_status(a.status, KDA_DEV_TIMEOUT);
    umma::fence_before();
    __syncthreads();
    if (warp == 5) umma::dealloc(tmem, 512);
}

// Joins the parts of cut sequences.  WIDE: a CTA per row, its warps take parts in turn and meet in shared memory; for
// sequences cut into more parts than a CTA has warps.  Otherwise a warp per row.
template <bool FP16, bool WIDE>
__global__ void __launch_bounds__(CW * 32) kda_latent_combine_kernel(const DecodeP p) {
    const LatentDecodeArgs &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = a.c.rank, nv = rank / 128;
    const int r = WIDE ? blockIdx.x : blockIdx.x * CW + warp, rt = r / NR, i = r - rt * NR;
    wait_for_previous();
    allow_dependent_launch();
    const Meta mt = p.meta[blockIdx.y];
    // A call whose waits gave up may leave records unwritten: nothing outside the workspace and the output is touched then.
    if (mt.pieces < 2 || mt.group < 0 || mt.pieces > p.groups - mt.group || (mt.second | 1) != 1 || r >= mt.rows ||
        mt.rows > p.nrt * NR || mt.row0 < 0 || mt.row0 > a.num_tokens * a.H - mt.rows)
        return;
    float m = -INFINITY, l = 0.f;
    float4 acc[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int k = WIDE ? warp : 0; k < mt.pieces; k += WIDE ? CW : 1) {
        const int64_t slot = ((int64_t)(mt.group + k) * 2 + (k == 0 ? mt.second : 0)) * p.nrt + rt;
        const float lk = p.part_l[slot * NR + i];
        const float4 *o = reinterpret_cast<const float4 *>(p.part + (slot * NR + i) * rank);
        float4 x[4];
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (v < nv) x[v] = __ldcs(o + v * 32 + lane);
        if (lk == -INFINITY) continue;  // nothing seen in this part
        const float mn = fmaxf(m, lk), f = m == -INFINITY ? 0.f : exp2_(m - mn), w = exp2_(lk - mn);
        l = l * f + w;
        m = mn;
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (v < nv) {
                acc[v].x = acc[v].x * f + w * x[v].x;
                acc[v].y = acc[v].y * f + w * x[v].y;
                acc[v].z = acc[v].z * f + w * x[v].z;
                acc[v].w = acc[v].w * f + w * x[v].w;
            }
    }
    const int64_t orow = mt.row0 + r;
    if constexpr (WIDE) {
        __shared__ float acc_s[CW][512];
        __shared__ float ml[CW][2];
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (v < nv) *reinterpret_cast<float4 *>(&acc_s[warp][(v * 32 + lane) * 4]) = acc[v];
        if (lane == 0) {
            ml[warp][0] = m;
            ml[warp][1] = l;
        }
        __syncthreads();
        float mm = -INFINITY, ll = 0.f, f[CW];
#pragma unroll
        for (int w = 0; w < CW; ++w) mm = fmaxf(mm, ml[w][0]);
#pragma unroll
        for (int w = 0; w < CW; ++w) {
            f[w] = ml[w][0] == -INFINITY ? 0.f : exp2_(ml[w][0] - mm);
            ll += f[w] * ml[w][1];
        }
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        for (int ch = threadIdx.x * 2; ch < rank; ch += CW * 64) {
            float o0 = 0.f, o1 = 0.f;
#pragma unroll
            for (int w = 0; w < CW; ++w) {
                o0 += f[w] * acc_s[w][ch];
                o1 += f[w] * acc_s[w][ch + 1];
            }
            *reinterpret_cast<uint32_t *>(a.out + orow * rank + ch) = pack2<FP16>(o0 * inv, o1 * inv);
        }
        if (a.lse && threadIdx.x == 0) a.lse[orow] = ll == 0.f ? -INFINITY : (mm + __log2f(ll)) * kLn2;
    } else {
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (v < nv)
                *reinterpret_cast<uint2 *>(a.out + orow * rank + (v * 32 + lane) * 4) =
                    make_uint2(pack2<FP16>(acc[v].x * inv, acc[v].y * inv), pack2<FP16>(acc[v].z * inv, acc[v].w * inv));
        if (a.lse && lane == 0) a.lse[orow] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
    }
}

struct Plan {
    int nrt, groups, slots_meta;
    size_t off_part, off_l, bytes;
};

static Plan plan(int rank, int H, int n, int max_tokens) {
    Plan q;
    const int rows = H * max_tokens, sms = current_device_sms();
    q.nrt = (rows + NR - 1) / NR;
    q.groups = std::max(1, sms / q.nrt);
    q.slots_meta = std::min(n, q.groups);
    const size_t parts = (size_t)std::max(sms, q.nrt) * 2 * NR;  // whatever the row tiles: groups * nrt is no more
    q.off_part = ((size_t)sms * sizeof(Meta) + 255) / 256 * 256;
    q.off_l = q.off_part + parts * rank * 4;
    q.bytes = q.off_l + parts * 4;
    return q;
}

template <bool FP16>
static int launch(const LatentDecodeArgs &a, const Plan &q, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return launch_result("latent decode: cudaGetDevice");
    if (!(done.load() >> dev & 1)) {
        if (cudaFuncSetAttribute(kda_latent_decode_kernel<FP16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 SMEM_MAX) != cudaSuccess)
            return launch_result("latent decode: cudaFuncSetAttribute");
        done.fetch_or(1ull << dev);
    }
    const EncodeTiledFn enc = encoder();
    if (!enc) return fail(KDA_ERR_CUDA, "latent decode: cuTensorMapEncodeTiled is not available");
    CUtensorMap map_c, map_r;
    const int d = a.c.rank + a.c.rope;
    const bool split = a.c.rope % 64 != 0;  // one box takes the rotary channels too where they are a whole chunk
    const int64_t chunks = split ? a.c.rank / 64 : d / 64;
    const int64_t dims[4] = {64, a.c.page_size, chunks, a.c.num_pages}, strides[3] = {d, 64, a.c.page_stride};
    const int box[4] = {64, 8, (int)chunks, 1};
    if (!tensor_map(enc, &map_c, FP16, a.c.pages, 4, dims, strides, box) ||
        (split && !map_3d(enc, &map_r, FP16, a.c.pages + a.c.rank, a.c.rope, a.c.page_size, a.c.num_pages, d,
                          a.c.page_stride, 8, 1)))
        return fail(KDA_ERR_CUDA, "latent decode: tensor map encoding failed");
    if (!split) map_r = map_c;  // not read
    DecodeP p;
    p.a = a;
    p.groups = q.groups;
    p.nrt = q.nrt;
    p.nch = (d + 63) / 64;
    p.split_rope = split;
    p.by_seq = a.n <= q.groups;
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    p.meta = reinterpret_cast<Meta *>(ws);
    p.part = reinterpret_cast<float *>(ws + q.off_part);
    p.part_l = reinterpret_cast<float *>(ws + q.off_l);
    const uint32_t stage = p.nch * ATOM * (TILE / 8);
    const uint32_t fixed = 1024 + NR * 128 + MISC;
    p.nst = std::min<int>(MAX_STAGES, (SMEM_MAX - fixed) / stage);
    const uint32_t smem = fixed + p.nst * stage;
    dependent_launch(kda_latent_decode_kernel<FP16>, dim3(q.groups * q.nrt), NT, smem, st, p, map_c, map_r);
    const int rc = launch_result("kda_latent_decode_kernel launch");
    if (rc != KDA_OK) return rc;
    const int rows = a.H * a.max_tokens;
    if (q.groups > CW * a.n)  // a sequence is cut into about groups / n parts
        dependent_launch(kda_latent_combine_kernel<FP16, true>, dim3(rows, q.slots_meta), CW * 32, 0, st, p);
    else
        dependent_launch(kda_latent_combine_kernel<FP16, false>, dim3((rows + CW - 1) / CW, q.slots_meta), CW * 32, 0,
                         st, p);
    return launch_result("kda_latent_combine_kernel launch");
}

}  // namespace latent

size_t latent_decode_workspace_bytes(int rank, int H, int n, int max_tokens) {
    return latent::plan(rank, H, std::max(n, 1), max_tokens).bytes;
}

int launch_latent_decode(const LatentDecodeArgs &a, cudaStream_t st) {
    using namespace latent;
    const Plan q = plan(a.c.rank, a.H, a.n, a.max_tokens);
    return a.c.fp16 ? launch<true>(a, q, st) : launch<false>(a, q, st);
}

}  // namespace kda
