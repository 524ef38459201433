// kda_kv_evict.cu -- eviction from the paged key-value cache by accumulated attention weight (include/kda.h: kda_kv_evict).
//
// A unit is one (sequence, layer, key-value head): of its len tokens the `keep` with the largest keys stay, where a token's
// key is all ones if it is protected and else its sum, as 32 bits in the order of the numbers.  Units share nothing, so each
// is one CTA, or one cluster of CTAs that divide its slots where there are few units.
//
//   select  the keep-th largest key by its digits, 11 + 11 + 10 bits: a histogram in shared memory for each (atomics on
//           counts: their order does not matter), summed over the cluster; ties go to the lowest slots
//   mark    one bit a slot, kept or not, in every CTA of the cluster; prefix sums over blocks of 256 slots of the holes (dropped,
//           below keep) and of the sources (kept, at or behind keep), of which there are as many
//   move    a warp finds 32 holes and 32 sources at a time by their ranks, and copies the rows, 8 loads a lane in flight
//
// Filling holes instead of closing them up moves the fewest rows there are (bringing 2,112 tokens back to 2,048 moves 64 at
// most; closing up would move nearly all), and no row that is read is written, so nothing has to wait for anything.
// Bound by bytes: 8 a slot to select, twice 4 head_dim + 8 for each row that moves.
#include <cooperative_groups.h>

#include <algorithm>

#include "kda_kv.cuh"

namespace kda {
namespace kv {

namespace cg = cooperative_groups;

constexpr int ET = 512;             // threads
constexpr int EW = ET / 32;
constexpr int BINS = 2048;
constexpr int BLOCK = 256;          // slots of a prefix sum's block
constexpr int KEYS = 12288;         // keys of a CTA that stay in shared memory; more are made again from the pages
constexpr int MAX_CLUSTER = 8;
constexpr uint32_t PROTECTED = 0xffffffffu;

// Blocks that `words` words of marks have, rounded up to a multiple of 4.
__host__ __device__ constexpr int blocks_of(int words) { return (words / (BLOCK / 32) + 3) / 4 * 4; }

struct Unit {
    const int32_t *trow;
    int32_t len, keep, since;
    uint16_t *base;  // the layer's pages
    int32_t head;
};

// Larger for a larger sum; 0 for NaN.
__device__ __forceinline__ uint32_t order_of(float w) {
    if (isnan(w)) return 0;
    const uint32_t b = __float_as_uint(w + 0.f);  // -0 is 0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Keys of slots j .. j + 3 (j a multiple of 4: one page has them, as pages are multiples of 16); 0 behind the end.
__device__ __forceinline__ uint4 keys_at(const KvEvictArgs &a, const Unit &u, int j) {
    const int32_t p = u.trow[j / a.c.page_size];
    const bool shared = a.t.refcount[p] > 1;
    const uint16_t *st = u.base + p * a.c.page_stride + stats_at(a.c, u.head) + 2 * (j % a.c.page_size);
    const float4 w = *reinterpret_cast<const float4 *>(st);
    const int4 pos = *reinterpret_cast<const int4 *>(st + 2 * a.c.page_size);
    auto key = [&](int k, float x, int32_t at) {
        if (j + k >= u.len) return 0u;
        return shared || at < a.first || at >= u.since ? PROTECTED : order_of(x);
    };
    return make_uint4(key(0, w.x, pos.x), key(1, w.y, pos.y), key(2, w.z, pos.z), key(3, w.w, pos.w));
}

// The k-th (from 0) set bit of x.
__device__ __forceinline__ int nth_bit(uint32_t x, int k) {
    int at = 0;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) {
        const int c = __popc(x & ((1u << w) - 1));
        if (k >= c) {
            k -= c;
            x >>= w;
            at += w;
        }
    }
    return at;
}

// The slot with rank r among the marked ones, by prefix sums of blocks and the words f(w) of marks.
template <class F>
__device__ __forceinline__ int slot_of(const int32_t *before, int blocks, int r, F f) {
    int lo = 0, hi = blocks;  // before[lo] <= r < before[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before[mid] <= r)
            lo = mid;
        else
            hi = mid;
    }
    r -= before[lo];
    int w = lo * (BLOCK / 32);
    uint32_t x = f(w);
    for (int c = __popc(x); r >= c; c = __popc(x)) {
        r -= c;
        x = f(++w);
    }
    return w * 32 + nth_bit(x, r);
}

// Exclusive prefix sum over the CTA; total gets the sum.  part: EW + 1 ints that nothing else uses meanwhile.
__device__ __forceinline__ int cta_scan(int v, int *part, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(FULL, s, o);
        if (lane >= o) s += t;
    }
    if (lane == 31) part[warp] = s;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < EW; ++w) {
        if (w < warp) before += part[w];
        total += part[w];
    }
    __syncthreads();
    return before + s - v;
}

__global__ void __launch_bounds__(ET) kda_kv_evict_kernel(const KvEvictArgs a, int words_max) {
    // [words_max] marks, holes and sources before each block of them, histogram, keys; each a multiple of 16 bytes
    extern __shared__ __align__(16) uint32_t smem[];
    __shared__ int part[EW];
    __shared__ int found[4];   // bin, count above it, its own count
    __shared__ int ties;       // this CTA's tokens whose key is the last one taken
    const cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int blocks_max = blocks_of(words_max);
    uint32_t *marks = smem;
    int32_t *holes = reinterpret_cast<int32_t *>(marks + words_max), *sources = holes + blocks_max;
    int32_t *hist = sources + blocks_max;
    uint32_t *kept = reinterpret_cast<uint32_t *>(hist + BINS);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    wait_for_previous();
    allow_dependent_launch();
    int64_t unit = blockIdx.x / C;
    Unit u;
    u.head = (int)(unit % a.c.heads);
    unit /= a.c.heads;
    const int layer = (int)(unit % a.c.layers), i = (int)(unit / a.c.layers);
    const bool tells = layer == 0 && u.head == 0 && rank == 0 && tid == 0;
    u.base = a.c.pages + layer * a.c.layer_stride;
    const int32_t row = a.rows ? a.rows[i] : i;
    if (row < 0 || row >= a.t.max_seqs) {
        if (tells) {
            a.new_lens[i] = 0;
            if (row != -1) set_status(a.status, KDA_DEV_BAD_SLOT);
        }
        return;
    }
    u.len = a.t.lens[row];
    u.keep = a.keep[i];
    u.since = a.since ? a.since[i] : INT32_MAX;
    u.trow = a.t.table + (int64_t)row * a.t.max_pages;
    const bool bad_len = u.len < 0 || u.len > (int64_t)a.t.max_pages * a.c.page_size;
    if (bad_len || u.keep < 0 || u.len <= u.keep || u.len > KDA_KV_EVICT_MAX_LEN) {
        if (tells) {
            a.new_lens[i] = bad_len ? 0 : u.len;
            if (bad_len || u.keep < 0 || u.len > u.keep) set_status(a.status, KDA_DEV_BAD_SEQLENS);
        }
        return;
    }
    // a bad page anywhere leaves the whole row as it is, in every layer and head alike
    const int pages = (u.len + a.c.page_size - 1) / a.c.page_size;
    bool bad = false;
    for (int p = tid; p < pages; p += ET) bad |= !page_ok(a.t, u.trow[p]);
    if (__syncthreads_or(bad)) {
        if (tells) {
            a.new_lens[i] = u.len;
            set_status(a.status, KDA_DEV_BAD_PAGE);
        }
        return;
    }
    if (tells) a.new_lens[i] = u.keep;
    if (u.keep == 0) return;

    // this CTA's slots [s0, s1), whole words of marks
    const int per = ((u.len + C - 1) / C + BLOCK - 1) / BLOCK * BLOCK;
    const int s0 = min(u.len, rank * per), s1 = min(u.len, s0 + per);
    const bool stay = s1 - s0 <= KEYS;
    for (int j = s0 + 4 * tid; j < s1; j += 4 * ET)
        if (stay) *reinterpret_cast<uint4 *>(kept + j - s0) = keys_at(a, u, j);
    auto keys = [&](int j) { return stay ? *reinterpret_cast<const uint4 *>(kept + j - s0) : keys_at(a, u, j); };

    // the keep-th largest key, digit by digit: `need` of the keys that begin with `prefix` are among them
    uint32_t prefix = 0, mask = 0;
    int need = u.keep, equal = 0;
    for (int digit = 0; digit < 3; ++digit) {
        const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0, bins = digit == 2 ? 1024 : 2048;
        for (int b = tid; b < BINS; b += ET) hist[b] = 0;
        __syncthreads();
        for (int j = s0 + 4 * tid; j < s1; j += 4 * ET) {
            const uint4 k = keys(j);
            const uint32_t x[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j + e < s1 && (x[e] & mask) == prefix) atomicAdd(hist + ((x[e] >> shift) & (bins - 1)), 1);
        }
        cluster.sync();
        // bins from the top: thread t has bins [4t, 4t + 4) counted from the largest
        int c[BINS / ET], mine = 0;
#pragma unroll
        for (int e = 0; e < BINS / ET; ++e) {
            const int b = BINS - 1 - (tid * (BINS / ET) + e);
            c[e] = 0;
            for (int r = 0; r < C; ++r) c[e] += *cluster.map_shared_rank(hist + b, r);
            mine += c[e];
        }
        int total, above = cta_scan(mine, part, total);
#pragma unroll
        for (int e = 0; e < BINS / ET; ++e) {
            if (above < need && need <= above + c[e]) {
                found[0] = BINS - 1 - (tid * (BINS / ET) + e);
                found[1] = above;
                found[2] = c[e];
            }
            above += c[e];
        }
        cluster.sync();  // all have read the histograms
        prefix |= (uint32_t)found[0] << shift;
        mask |= (uint32_t)(bins - 1) << shift;
        need -= found[1];
        equal = found[2];
        __syncthreads();
    }

    // marks of this CTA's slots: larger keys, and the first `need` of the equal ones
    const bool some = need < equal;  // not all of the equal ones: their order counts
    int mine = 0, before = 0;
    if (some) {
        for (int j = s0 + 4 * tid; j < s1; j += 4 * ET) {
            const uint4 k = keys(j);
            mine += (k.x == prefix) + (j + 1 < s1 && k.y == prefix) + (j + 2 < s1 && k.z == prefix) +
                    (j + 3 < s1 && k.w == prefix);
        }
        int total;
        cta_scan(mine, part, total);
        if (tid == 0) ties = total;
        cluster.sync();
        for (int r = 0; r < rank; ++r) before += *cluster.map_shared_rank(&ties, r);
    }
    for (int j0 = s0; j0 < s1; j0 += 4 * ET) {
        const int j = j0 + 4 * tid;
        uint32_t bits = 0, same = 0;
        if (j < s1) {
            const uint4 k = keys(j);
            const uint32_t x[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j + e < s1) {
                    bits |= (uint32_t)(x[e] > prefix) << e;
                    same |= (uint32_t)(x[e] == prefix) << e;
                }
        }
        if (some) {
            int total;
            int at = before + cta_scan(__popc(same), part, total);
            before += total;
            for (int e = 0; e < 4; ++e)
                if ((same >> e) & 1) bits |= (uint32_t)(at++ < need) << e;
        } else {
            bits |= same;
        }
        // eight threads' bits are a word, which every CTA of the cluster gets
        uint32_t word = bits << (4 * (lane & 7));
        word |= __shfl_xor_sync(FULL, word, 1);
        word |= __shfl_xor_sync(FULL, word, 2);
        word |= __shfl_xor_sync(FULL, word, 4);
        if ((j & ~31) < s1)
            for (int r = lane & 7; r < C; r += 8) *cluster.map_shared_rank(marks + j / 32, r) = word;
    }
    cluster.sync();  // all marks are there, all sums have been read

    const int nb = (u.len + BLOCK - 1) / BLOCK, nw = (u.len + 31) / 32;
    const int kw = u.keep / 32;
    const uint32_t low = (1u << (u.keep % 32)) - 1;  // slots of word kw that lie below keep
    auto hole = [&](int w) { return w < kw ? ~marks[w] : w == kw ? ~marks[w] & low : 0u; };
    auto source = [&](int w) { return w < kw || w >= nw ? 0u : w == kw ? marks[w] & ~low : marks[w]; };
    int moves = 0, unused = 0;
    for (int b0 = 0; b0 < nb; b0 += ET) {
        const int b = b0 + tid;
        int nh = 0, ns = 0;
        if (b < nb)
#pragma unroll
            for (int w = b * (BLOCK / 32); w < (b + 1) * (BLOCK / 32); ++w) {
                if (w < nw) {
                    nh += __popc(hole(w));
                    ns += __popc(source(w));
                }
            }
        int th, ts;
        const int h = cta_scan(nh, part, th), s = cta_scan(ns, part, ts);
        if (b < nb) {
            holes[b] = moves + h;
            sources[b] = unused + s;
        }
        moves += th;
        unused += ts;
    }
    __syncthreads();

    // moves [m0, m1) are this warp's
    const int nwarps = C * EW, w = rank * EW + warp;
    const int share = (moves + nwarps - 1) / nwarps, m0 = min(moves, w * share), m1 = min(moves, m0 + share);
    const int nv = a.c.d / 8, both = 2 * nv, ps = a.c.page_size;
    uint16_t *keys0 = u.base + key_at(a.c, u.head);
    const int64_t values = value_at(a.c, u.head) - key_at(a.c, u.head);
    for (int m = m0; m < m1; m += 32) {
        const int cnt = min(32, m1 - m);
        int64_t from = 0, to = 0;  // words before the rows' pages
        int fs = 0, ts = 0;        // and the slots within these
        if (lane < cnt) {
            const int src = slot_of(sources, nb, m + lane, source), dst = slot_of(holes, nb, m + lane, hole);
            from = u.trow[src / ps] * a.c.page_stride;
            to = u.trow[dst / ps] * a.c.page_stride;
            fs = src % ps;
            ts = dst % ps;
            const int32_t *f = reinterpret_cast<const int32_t *>(u.base + from + stats_at(a.c, u.head)) + fs;
            int32_t *t = reinterpret_cast<int32_t *>(u.base + to + stats_at(a.c, u.head)) + ts;
            const int32_t x = f[0], y = f[ps];
            t[0] = x;
            t[ps] = y;
            from += (int64_t)fs * a.c.d;
            to += (int64_t)ts * a.c.d;
        }
        constexpr int UNROLL = 8;
        for (int v0 = 0; v0 < cnt * both; v0 += 32 * UNROLL) {
            uint4 r[UNROLL];
            int64_t at[UNROLL];
#pragma unroll
            for (int e = 0; e < UNROLL; ++e) {
                const int v = v0 + e * 32 + lane;
                const int row_ = min(v / both, 31), k = v - row_ * both;
                const int64_t f = __shfl_sync(FULL, from, row_), t = __shfl_sync(FULL, to, row_);
                const int64_t in = (k < nv ? 0 : values) + (k < nv ? k : k - nv) * 8;
                at[e] = v < cnt * both ? t + in : -1;
                if (at[e] >= 0) r[e] = __ldcs(reinterpret_cast<const uint4 *>(keys0 + f + in));
            }
#pragma unroll
            for (int e = 0; e < UNROLL; ++e)
                if (at[e] >= 0) *reinterpret_cast<uint4 *>(keys0 + at[e]) = r[e];
        }
    }
}

}  // namespace kv

int launch_kv_evict(const KvEvictArgs &a, cudaStream_t st) {
    using namespace kv;
    const int64_t units = (int64_t)a.n * a.c.layers * a.c.heads;
    const int64_t cap = std::min<int64_t>((int64_t)a.t.max_pages * a.t.page_size, KDA_KV_EVICT_MAX_LEN);
    const int words = (int)((cap + BLOCK - 1) / BLOCK * (BLOCK / 32));
    // CTAs of a unit: as many as there is room for, and as many as have 1,024 slots each
    int C = 1;
    while (C < MAX_CLUSTER && units * C * 2 <= (int64_t)current_device_sms() * 2 && cap > (int64_t)C * 1024) C *= 2;
    const size_t smem = 4 * ((size_t)words + 2 * blocks_of(words) + BINS + KEYS);
    auto k = kda_kv_evict_kernel;
    static std::atomic<uint64_t> prepared{0};
    if (allow_smem(k, prepared) == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(units * C));
        cfg.blockDim = dim3(ET);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim = {(unsigned)C, 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        cudaLaunchKernelEx(&cfg, k, a, words);
    }
    return launch_result("kda_kv_evict_kernel launch");
}

}  // namespace kda
