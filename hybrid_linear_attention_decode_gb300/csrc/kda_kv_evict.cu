// kda_kv_evict.cu -- eviction from the paged key-value cache by accumulated attention weight (include/kda.h: kda_kv_evict).
//
// A unit is one (sequence, layer, key-value head): of its len tokens the `keep` with the largest keys stay, where a token's
// key is all ones if it is protected and else its sum, as 32 bits in the order of the numbers.  Units share nothing, so each
// is one CTA, or one cluster of CTAs that divide its slots where there are few units.
//
//   select  the keep-th largest pair of key and slot (lower slots count as larger) byte by byte: a histogram of 256 bins in
//           shared memory (four copies, so that lanes with equal bytes meet less; atomics on counts: their order does not
//           matter), summed over the cluster.  It ends when a bin is taken whole, or when a bin has so few pairs that
//           votes of one warp find the last one
//   mark    one bit a slot, kept or not, in every CTA of the cluster; prefix sums over blocks of 256 slots of the holes (dropped,
//           below keep) and of the sources (kept, at or behind keep), of which there are as many; both listed in order, where
//           the keys were
//   move    a warp copies the rows of up to 32 pairs from the lists, several loads a lane in flight
//
// Filling holes instead of closing them up moves the fewest rows there are (bringing 2,112 tokens back to 2,048 moves 64 at
// most; closing up would move nearly all), and no row that is read is written, so nothing has to wait for anything.
// Bound by bytes: 8 a slot to select, twice 4 head_dim + 8 for each row that moves; with short rows by the latency of a unit's
// steps, which is why CTAs are small enough for several on a multiprocessor.
#include <cooperative_groups.h>

#include <algorithm>

#include "kda_kv.cuh"

namespace kda {
namespace kv {

namespace cg = cooperative_groups;

constexpr int BINS = 256, COPIES = 4;
constexpr int SHORT = 4096;         // slots of a row for which a CTA has 128 threads
constexpr int FEW = 128;            // pairs among which one warp finds the last
constexpr int BLOCK = 256;          // slots of a prefix sum's block
constexpr int KEYS = 16384;         // most keys of a CTA that stay in shared memory; more are made again from the pages
constexpr int MAX_CLUSTER = 8;
constexpr uint32_t PROTECTED = 0xffffffffu;

// Blocks that `words` words of marks have, rounded up to a multiple of 4.
__host__ __device__ constexpr int blocks_of(int words) { return (words / (BLOCK / 32) + 3) / 4 * 4; }

struct Unit {
    const int32_t *trow;
    int32_t len, keep, head;
    uint32_t open;    // positions first .. first + open - 1 are not protected
    uint16_t *base;   // the layer's pages
};

// Slots divided by the page size, by a multiplication: exact below 2^22 for the sizes there are (up to 1024).
struct PageSize {
    uint32_t size, inverse;  // inverse: 2^32 / size rounded up
    __device__ __forceinline__ int page(int slot) const { return (int)__umulhi((uint32_t)slot, inverse); }
    __device__ __forceinline__ int within(int slot) const { return slot - page(slot) * (int)size; }
};

// Larger for a larger sum; 0 for NaN.
__device__ __forceinline__ uint32_t order_of(float w) {
    const uint32_t b = __float_as_uint(w + 0.f);  // -0 is 0
    return isnan(w) ? 0 : b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// Keys of slots j .. j + 3 (j a multiple of 4: one page has them, as pages are multiples of 16) of page p; 0 behind the end.
struct Four {
    float4 w;
    int4 pos;
    int32_t shared;
};
__device__ __forceinline__ Four read_four(const KvEvictArgs &a, const Unit &u, PageSize ps, int j, int32_t p) {
    const uint16_t *st = u.base + p * a.c.page_stride + stats_at(a.c, u.head) + 2 * ps.within(j);
    Four f;
    f.w = *reinterpret_cast<const float4 *>(st);
    f.pos = *reinterpret_cast<const int4 *>(st + 2 * a.c.page_size);
    f.shared = a.t.refcount[p];
    return f;
}
__device__ __forceinline__ uint4 keys_of(const KvEvictArgs &a, const Unit &u, int j, const Four &f) {
    // (below `first` the difference wraps around to 2^31 - first and more, which no `open` is above)
    const uint32_t open = f.shared > 1 ? 0u : u.open;
    auto key = [&](float x, int32_t at) { return (uint32_t)at - (uint32_t)a.first >= open ? PROTECTED : order_of(x); };
    uint4 k = make_uint4(key(f.w.x, f.pos.x), key(f.w.y, f.pos.y), key(f.w.z, f.pos.z), key(f.w.w, f.pos.w));
    if (j + 3 >= u.len) {  // as a pair with its slot less than all that exist, and so never kept
        k.w = 0;
        if (j + 2 >= u.len) k.z = 0;
        if (j + 1 >= u.len) k.y = 0;
    }
    return k;
}

// The same again, for rows whose keys shared memory does not hold: out of line, so that it is in the program once.
__device__ __noinline__ uint4 keys_again(const KvEvictArgs &a, const Unit &u, PageSize ps, int j) {
    return keys_of(a, u, j, read_four(a, u, ps, j, u.trow[ps.page(j)]));
}

// The last of the keep-th largest: pairs of key and inverted slot whose bytes under the masks are as large stay.
struct Border {
    uint32_t key, key_mask, slot, slot_mask;
};

// keys_max: keys of a CTA that there is room for.
template <int ET, bool CLUSTER>
__global__ void __launch_bounds__(ET, 1024 / ET)
    kda_kv_evict_kernel(const KvEvictArgs a, const PageSize ps, int words_max, int keys_max) {
    constexpr int EW = ET / 32;
    constexpr int UNROLL = 4;  // 16-byte words of a lane in flight while rows move
    constexpr int AHEAD = 2;   // groups of four slots of a thread in flight while keys are read
    // [words_max] marks, holes and sources before each block of them, keys; each a multiple of 16 bytes
    extern __shared__ __align__(16) uint32_t smem[];
    __shared__ __align__(16) int32_t hist[CLUSTER ? 2 : 1][BINS * COPIES];  // of passes in turn
    __shared__ int32_t sums[CLUSTER ? BINS : 1];
    __shared__ uint64_t few[FEW];
    __shared__ int found[3];   // bin, count above it, its own count
    __shared__ int listed;     // pairs in few (of the cluster's first CTA)
    __shared__ int spoiled;    // this CTA's slots have a bad page
    __shared__ uint64_t part[EW];
    const cg::cluster_group cluster = cg::this_cluster();
    const int C = CLUSTER ? (int)cluster.num_blocks() : 1, rank = CLUSTER ? (int)cluster.block_rank() : 0;
    const int blocks_max = blocks_of(words_max);
    uint32_t *marks = smem;
    int32_t *holes = reinterpret_cast<int32_t *>(marks + words_max), *sources = holes + blocks_max;
    uint32_t *kept = reinterpret_cast<uint32_t *>(sources + blocks_max);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto sync_all = [&] {
        if constexpr (CLUSTER)
            cluster.sync();
        else
            __syncthreads();
    };
    auto of_rank = [&](auto *p, int r) {
        if constexpr (CLUSTER)
            return cluster.map_shared_rank(p, r);
        else
            return p;
    };
    if (tid == 0) listed = spoiled = 0;

    wait_for_previous();
    allow_dependent_launch();
    const uint32_t unit = blockIdx.x / C, above_head = unit / a.c.heads;
    Unit u;
    u.head = (int)(unit - above_head * a.c.heads);
    const int i = (int)(above_head / a.c.layers), layer = (int)(above_head - i * a.c.layers);
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
    u.open = a.since ? (uint32_t)max(a.since[i], a.first) - a.first : 0x80000000u - a.first;
    u.trow = a.t.table + (int64_t)row * a.t.max_pages;
    const bool bad_len = u.len < 0 || u.len > (int64_t)a.t.max_pages * a.c.page_size;
    if (bad_len || u.keep < 0 || u.len <= u.keep || u.len > a.max_len) {
        if (tells) {
            a.new_lens[i] = bad_len ? 0 : u.len;
            if (bad_len || u.keep < 0 || u.len > u.keep) set_status(a.status, KDA_DEV_BAD_SEQLENS);
        }
        return;
    }

    // this CTA's slots [s0, s1), whole blocks of marks
    const int per = ((u.len + C - 1) / C + BLOCK - 1) / BLOCK * BLOCK;
    const int s0 = min(u.len, rank * per), s1 = min(u.len, s0 + per);
    const bool stay = s1 - s0 <= keys_max;
    bool bad = false;
    // f(j, keys of slots j .. j + 3) for this thread's slots; again from the pages where shared memory does not hold them
    auto each = [&](auto f) {
        for (int j = s0 + 4 * tid; j < s1; j += 4 * ET)
            f(j, stay ? *reinterpret_cast<const uint4 *>(kept + j - s0) : keys_again(a, u, ps, j));
    };

    // `need` of the pairs that begin as the bytes found so far are among those that stay
    Border t = {0, 0, 0, 0};
    int need = max(u.keep, 1);  // (a row that keeps nothing has its pages looked at, too)
    for (int pass = 0; pass < 7; ++pass) {
        int32_t *h = hist[CLUSTER ? pass & 1 : 0];
        for (int b = tid; b < BINS; b += ET) reinterpret_cast<int4 *>(h)[b] = make_int4(0, 0, 0, 0);
        __syncthreads();
        const int shift = pass < 4 ? 24 - 8 * pass : 16 - 8 * (pass - 4);
        int32_t *h_lane = h + (lane & (COPIES - 1));
        auto count = [&](int, uint4 k) {
            const uint32_t x[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if ((x[e] & t.key_mask) == t.key) atomicAdd(h_lane + ((x[e] >> shift) & 255) * COPIES, 1);
        };
        auto count_slots = [&](int j, uint4 k) {
            const uint32_t x[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t slot = 0xffffffu - (j + e);
                if (x[e] == t.key && (slot & t.slot_mask) == t.slot) atomicAdd(h_lane + ((slot >> shift) & 255) * COPIES, 1);
            }
        };
        if (pass == 0) {
            for (int j0 = s0 + 4 * tid; j0 < s1; j0 += 4 * ET * AHEAD) {
                int32_t p[AHEAD];
                Four x[AHEAD];
#pragma unroll
                for (int e = 0; e < AHEAD; ++e) {
                    const int j = j0 + e * 4 * ET;
                    p[e] = j < s1 ? u.trow[ps.page(j)] : 0;
                }
#pragma unroll
                for (int e = 0; e < AHEAD; ++e) {
                    const int j = j0 + e * 4 * ET;
                    if (!page_ok(a.t, p[e])) {
                        bad = true;
                        p[e] = 0;
                    }
                    if (j < s1) x[e] = read_four(a, u, ps, j, p[e]);
                }
#pragma unroll
                for (int e = 0; e < AHEAD; ++e) {
                    const int j = j0 + e * 4 * ET;
                    if (j < s1) {
                        const uint4 k = keys_of(a, u, j, x[e]);
                        if (stay) *reinterpret_cast<uint4 *>(kept + j - s0) = k;
                        count(j, k);
                    }
                }
            }
            if (bad) spoiled = 1;
        } else if (pass < 4) {
            each(count);
        } else {
            each(count_slots);
        }
        sync_all();
        if constexpr (CLUSTER) {
            for (int b = tid; b < BINS; b += ET) {
                int c = 0;
#pragma unroll
                for (int r = 0; r < MAX_CLUSTER; ++r)
                    if (r < C) {
                        const int4 x = *reinterpret_cast<const int4 *>(of_rank(h + b * COPIES, r));
                        c += x.x + x.y + x.z + x.w;
                    }
                sums[b] = c;
            }
            __syncthreads();
        }
        if (warp == 0) {
            // a lane has eight bins, counted from the largest
            int c[BINS / 32], mine = 0;
#pragma unroll
            for (int e = 0; e < BINS / 32; ++e) {
                const int bin = BINS - 1 - (lane * (BINS / 32) + e);
                if constexpr (CLUSTER) {
                    c[e] = sums[bin];
                } else {
                    const int4 x = reinterpret_cast<const int4 *>(h)[bin];
                    c[e] = x.x + x.y + x.z + x.w;
                }
                mine += c[e];
            }
            int above = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(FULL, above, o);
                if (lane >= o) above += x;
            }
            above -= mine;
#pragma unroll
            for (int e = 0; e < BINS / 32; ++e) {
                if (above < need && need <= above + c[e]) {
                    found[0] = BINS - 1 - (lane * (BINS / 32) + e);
                    found[1] = above;
                    found[2] = c[e];
                }
                above += c[e];
            }
        }
        __syncthreads();
        if (pass == 0) {
            const bool wrong = lane < C && *of_rank(&spoiled, lane);
            if (__any_sync(FULL, wrong)) {  // the same in all CTAs of the row: it stays as it is, in every layer and head
                sync_all();
                if (tells) {
                    a.new_lens[i] = u.len;
                    set_status(a.status, KDA_DEV_BAD_PAGE);
                }
                return;
            }
        }
        if (pass < 4) {
            t.key |= (uint32_t)found[0] << shift;
            t.key_mask |= 255u << shift;
        } else {
            t.slot |= (uint32_t)found[0] << shift;
            t.slot_mask |= 255u << shift;
        }
        need -= found[1];
        const int size = found[2];
        if (need == size) break;  // all that begin so stay
        if (size <= FEW) {
            each([&](int j, uint4 k) {
                const uint32_t x[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t slot = 0xffffffu - (j + e);
                    if ((x[e] & t.key_mask) == t.key && (slot & t.slot_mask) == t.slot) {
                        const int at = atomicAdd(of_rank(&listed, 0), 1);
                        for (int r = 0; r < C; ++r) of_rank(few, r)[at] = (uint64_t)x[e] << 32 | slot;
                    }
                }
            });
            sync_all();
            if (warp == 0) {
                // bit by bit from the highest in which they differ, by votes of one warp, FEW / 32 pairs a lane
                constexpr int N = FEW / 32;
                uint32_t hi[N], lo[N], in = 0, all[2] = {~0u, ~0u}, any[2] = {0, 0};
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const uint64_t x = lane + 32 * n < size ? few[lane + 32 * n] : few[0];
                    in |= (uint32_t)(lane + 32 * n < size) << n;
                    hi[n] = (uint32_t)(x >> 32);
                    lo[n] = (uint32_t)x;
                    all[0] &= hi[n], any[0] |= hi[n];
                    all[1] &= lo[n], any[1] |= lo[n];
                }
                int left = size;  // pairs that may still be it
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t differ = __reduce_or_sync(FULL, any[half]) & ~__reduce_and_sync(FULL, all[half]);
                    for (; differ && left > 1; differ &= ~(0x80000000u >> __clz(differ))) {
                        const int bit = 31 - __clz(differ);
                        uint32_t set = 0;
                        int above = 0;
#pragma unroll
                        for (int n = 0; n < N; ++n) {
                            set |= ((half ? lo[n] : hi[n]) >> bit & 1) << n;
                            above += __popc(__ballot_sync(FULL, (set & in) >> n & 1));
                        }
                        if (above >= need) {
                            in &= set;
                            left = above;
                        } else {
                            need -= above;
                            left -= above;
                            in &= ~set;
                        }
                    }
                }
#pragma unroll
                for (int n = 0; n < N; ++n)
                    if (in >> n & 1) {
                        found[0] = (int)hi[n];
                        found[1] = (int)lo[n];
                    }
            }
            __syncthreads();
            t = Border{(uint32_t)found[0], 0xffffffffu, (uint32_t)found[1], 0xffffffu};
            break;
        }
    }
    if (tells) a.new_lens[i] = u.keep;
    if (u.keep == 0) {
        sync_all();
        return;
    }

    // marks: pairs as large as the border's, whose bytes that were not looked at are 0
    for (int j0 = s0; j0 < s1; j0 += 4 * ET) {
        const int j = j0 + 4 * tid;
        uint32_t word = 0;
        if (j < s1) {
            const uint4 k = stay ? *reinterpret_cast<const uint4 *>(kept + j - s0) : keys_again(a, u, ps, j);
            const uint32_t x[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                word |= (uint32_t)(x[e] > t.key || (x[e] == t.key && 0xffffffu - (j + e) >= t.slot)) << e;
        }
        // eight threads' bits are a word, which every CTA of the cluster gets
        word <<= 4 * (lane & 7);
        word |= __shfl_xor_sync(FULL, word, 1);
        word |= __shfl_xor_sync(FULL, word, 2);
        word |= __shfl_xor_sync(FULL, word, 4);
        if ((j & ~31) < s1)
            for (int r = lane & 7; r < C; r += 8) *of_rank(marks + j / 32, r) = word;
    }
    sync_all();  // all marks are there, all sums have been read, nobody reads another CTA's memory any more

    const int nb = (u.len + BLOCK - 1) / BLOCK, nw = (u.len + 31) / 32;
    const int kw = u.keep / 32;
    const uint32_t low = (1u << (u.keep % 32)) - 1;  // slots of word kw that lie below keep
    auto hole = [&](int w) { return w < kw ? ~marks[w] : w == kw ? ~marks[w] & low : 0u; };
    auto source = [&](int w) { return w < kw || w >= nw ? 0u : w == kw ? marks[w] & ~low : marks[w]; };
    // marks of block b: holes in the low 32 bits, sources in the high ones
    auto marked = [&](int b) {
        uint32_t nh = 0, ns = 0;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int w = b * (BLOCK / 32) + 4 * q;
            const uint4 m = *reinterpret_cast<const uint4 *>(marks + w);
            const uint32_t x[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t is = w + e < nw ? x[e] : 0u;
                nh += w + e < kw ? 32 - __popc(is) : w + e == kw ? __popc(~is & low) : 0;
                ns += w + e < kw ? 0 : w + e == kw ? __popc(is & ~low) : __popc(is);
            }
        }
        return (uint64_t)ns << 32 | nh;
    };
    uint64_t carry = 0;
    for (int b0 = 0; b0 < nb; b0 += ET) {  // in warps that have no blocks nothing is added
        const int b = b0 + tid;
        const uint64_t mine = b < nb ? marked(b) : 0;
        uint64_t incl = mine;
        if (b0 + warp * 32 < nb) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t x = __shfl_up_sync(FULL, incl, o);
                if (lane >= o) incl += x;
            }
        }
        if (lane == 31) part[warp] = incl;
        __syncthreads();
        uint64_t before = carry;
        for (int v = 0; v < EW && b0 + v * 32 < nb; ++v) {
            if (v < warp) before += part[v];
            carry += part[v];
        }
        before += incl - mine;
        if (b < nb) {
            holes[b] = (int32_t)(uint32_t)before;
            sources[b] = (int32_t)(before >> 32);
        }
        __syncthreads();
    }

    // the pairs with ranks [q0, q1) are this CTA's, in rounds of as many as the lists hold
    const int moves = (int)(uint32_t)carry, quota = (moves + C - 1) / C, q0 = min(moves, rank * quota), q1 = min(moves, q0 + quota);
    const int room = keys_max / 2;
    int32_t *list = reinterpret_cast<int32_t *>(kept);  // [room] sources, [room] holes
    // A row's key and value are `both` words of 16 bytes: to 32 lanes in turn, or several rows at once where they are 16 or less
    const int nv = a.c.d / 8, both = 2 * nv;
    const int width = both > 16 ? 32 : both > 8 ? 16 : both > 4 ? 8 : 4, at_once = 32 / width, sub = lane / width;
    uint16_t *keys0 = u.base + key_at(a.c, u.head);
    const int64_t values = value_at(a.c, u.head) - key_at(a.c, u.head);
    for (int r0 = q0; r0 < q1; r0 += room) {
        const int r1 = min(q1, r0 + room);
        // a warp has a block, a lane eight slots of it
        for (int b = warp; b < nb; b += EW) {
            const int w = b * (BLOCK / 32) + lane / 4, at = 8 * (lane & 3);
            const uint32_t before = (1u << at) - 1, here = 255u << at;
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                const int32_t *base = side ? holes : sources;
                const int first = base[b], next = b + 1 < nb ? base[b + 1] : moves;
                if (first >= r1 || next <= r0 || first == next) continue;
                const uint32_t x = side ? hole(w) : source(w);
                int k = __popc(x);  // marks of the words before, from the lanes that have these
                k = (lane & 3) == 0 ? k : 0;
                int incl = k;
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(FULL, incl, o);
                    if (lane >= o) incl += y;
                }
                k = __shfl_sync(FULL, incl - k, lane & ~3) + first + __popc(x & before);
                for (uint32_t mine = x & here; mine; mine &= mine - 1, ++k)
                    if (k >= r0 && k < r1) list[side * room + k - r0] = w * 32 + __ffs(mine) - 1;
            }
        }
        __syncthreads();
        const int share = min(32, (r1 - r0 + EW - 1) / EW);
        for (int m = r0 + warp * share; m < r1; m += EW * share) {
            const int cnt = min(share, r1 - m);
            int64_t from = 0, to = 0;  // words before the rows
            if (lane < cnt) {
                const int src = list[m - r0 + lane], dst = list[room + m - r0 + lane];
                from = u.trow[ps.page(src)] * a.c.page_stride;
                to = u.trow[ps.page(dst)] * a.c.page_stride;
                const int32_t *f = reinterpret_cast<const int32_t *>(u.base + from + stats_at(a.c, u.head)) + ps.within(src);
                int32_t *g = reinterpret_cast<int32_t *>(u.base + to + stats_at(a.c, u.head)) + ps.within(dst);
                const int32_t x = f[0], y = f[ps.size];
                g[0] = x;
                g[ps.size] = y;
                from += ps.within(src) * a.c.d;
                to += ps.within(dst) * a.c.d;
            }
            for (int k = lane & (width - 1); k - (lane & (width - 1)) < both; k += 32) {
                const int64_t in = k < nv ? k * 8 : values + (k - nv) * 8;
                for (int n = sub; n - sub < cnt; n += UNROLL * at_once) {
                    uint4 r[UNROLL];
#pragma unroll
                    for (int e = 0; e < UNROLL; ++e) {
                        const int x = n + e * at_once;
                        const uint16_t *f = keys0 + __shfl_sync(FULL, from, min(x, 31)) + in;
                        if (x < cnt && k < both) r[e] = __ldcs(reinterpret_cast<const uint4 *>(f));
                    }
#pragma unroll
                    for (int e = 0; e < UNROLL; ++e) {
                        const int x = n + e * at_once;
                        uint16_t *f = keys0 + __shfl_sync(FULL, to, min(x, 31)) + in;
                        if (x < cnt && k < both) *reinterpret_cast<uint4 *>(f) = r[e];
                    }
                }
            }
        }
        __syncthreads();
    }
}

struct Variant {
    void (*kernel)(KvEvictArgs, PageSize, int, int);
    int index;
    unsigned threads;
};
// Clusters: 1,024 threads a CTA where a multiprocessor has one CTA at most.  Single CTAs: the steps of a unit are bound by
// barriers and latencies, so that more and smaller CTAs are better where rows are short: 64 rows of 2,112 tokens in 4 layers
// and 8 heads took 39 us with 128 threads, 48 with 256 (and 57 with one warp); 6 of 2,000 to 8,192 in 8 layers 76 us with 256
// and 99 with 128.  On both sides of SHORT: 64 rows of 3,900 to 4,050 tokens 115 us with 128 threads, 122 with 256; 64 of 4,300 to
// 4,500 138 and 133; 32 of 6,000 to 8,000 cut to 512 164 and 122.  Against the rule: 12 rows of 2,000 to 4,000 cut to 1,024, 90 and
// 67, where there are too few units for the smaller CTAs to fill the GPU.
inline Variant variant(int64_t units, int C, int64_t cap) {
    if (C > 1 && units * C <= current_device_sms()) return {kda_kv_evict_kernel<1024, true>, 0, 1024};
    if (C > 1) return {kda_kv_evict_kernel<256, true>, 1, 256};
    if (cap <= SHORT) return {kda_kv_evict_kernel<128, false>, 2, 128};
    return {kda_kv_evict_kernel<256, false>, 3, 256};
}

}  // namespace kv

int launch_kv_evict(const KvEvictArgs &a, cudaStream_t st) {
    using namespace kv;
    const int64_t units = (int64_t)a.n * a.c.layers * a.c.heads;
    const int64_t cap = a.max_len;
    const int words = (int)((cap + BLOCK - 1) / BLOCK * (BLOCK / 32));
    // CTAs of a unit: more where there are few units, while each has 1,024 slots or more (384 units of 2,000 to 8,192 tokens, of
    // which 1,024 stay: 76 us with one CTA each, 87 with two)
    int C = 1;
    while (C < MAX_CLUSTER && units * C < (int64_t)current_device_sms() * 2 && cap > (int64_t)C * 1024) C *= 2;
    const int other = 4 * (words + 2 * blocks_of(words)), room = (kSmemMax - 12288 - other) / 4 / BLOCK * BLOCK;
    const int keys = (int)std::min<int64_t>({KEYS, room, ((cap + C - 1) / C + BLOCK - 1) / BLOCK * BLOCK});
    const size_t smem = (size_t)other + 4 * keys;
    const Variant v = variant(units, C, cap);
    static std::atomic<uint64_t> prepared[4];
    if (allow_smem(v.kernel, prepared[v.index]) == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(units * C));
        cfg.blockDim = dim3(v.threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim = {(unsigned)C, 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = C > 1 ? 2 : 1;
        const PageSize ps{(uint32_t)a.t.page_size, (uint32_t)(((uint64_t)1 << 32) / a.t.page_size + 1)};
        cudaLaunchKernelEx(&cfg, v.kernel, a, ps, words, keys);
    }
    return launch_result("kda_kv_evict_kernel launch");
}

}  // namespace kda
