// kda_pages.cu -- the paged cache's row writer and the page pool's operations (include/kda.h: kda_latent_append
// and kda_pages_*).  Integer bookkeeping and copies: nothing here computes on the cached values.
//
// A pool operation is two launches:
//   plan   one CTA: the free list (ascending page indices with refcount <= 0), the claim of each table row by
//          the first item that names it, each item's checks and, by an exclusive prefix sum of the items'
//          demands, the pages it takes.  One CTA, because for pools of some thousand pages a single launch with
//          barriers costs less than several launches of a wide scan.  Its time grows with the pool, whose counts reserve
//          and fork read twice and compact three times: reserve of 256 rows 6.8 us with 2,000 pages, 10.3 with 20,000, 55
//          with 100,000; compact (nothing to move) 5.6, 18.9, 126; truncate, which needs no free pages, 4.6 to 4.8.
//   apply  many CTAs: table rows and refcounts (integer atomics: their result does not depend on order), then
//          the page copies of all layers in 16-KiB pieces, four 16-byte loads of a thread in flight.  Items without a copy
//          are passed over piece by piece: 24 layers add 9 us to a reserve of 256 rows that copies nothing.
// The plan reads the pool as it was before the call and the apply launch writes it, so no item sees another's
// effect.  Copies are bandwidth-bound.
#include "kda_latent.cuh"

namespace kda {
namespace pages {

constexpr int PT = 1024;           // threads of the plan CTA
constexpr int AT = 256;            // threads of an apply CTA
constexpr int UNROLL = 4;          // 16-byte words per thread and copy piece
constexpr int PIECE = AT * UNROLL; // words of a copy piece (16 KiB)

// Workspace (int32): header, row claims, per-item records, free list or page map, copy lists.
struct Ws {
    int32_t *hdr;    // [0] entries of the copy lists
    int32_t *claim;  // [max_seqs] first item, padding aside, that names the row
    int32_t *start;  // [n] first entry of the free list the item takes
    int32_t *flag;   // [n] 0: left out; 1: served; 3: served, with a copied page
    int32_t *len;    // [n] tokens of the row (fork: of the parent) before the call
    int32_t *list;   // [num_pages] free pages; compact: new index of each page
    int32_t *src, *dst;  // [max(n, num_pages)] page copies; src -1: none
};

__host__ __device__ inline Ws layout(int32_t *ws, int64_t max_seqs, int64_t num_pages, int64_t n) {
    Ws w;
    w.hdr = ws;
    w.claim = ws + 16;
    w.start = w.claim + max_seqs;
    w.flag = w.start + n;
    w.len = w.flag + n;
    w.list = w.len + n;
    w.src = w.list + num_pages;
    w.dst = w.src + (n > num_pages ? n : num_pages);
    return w;
}

// Exclusive prefix sum over the CTA; total gets the sum.  Every thread calls it.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *part, int64_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += t;
    }
    if (lane == 31) part[warp] = s;
    __syncthreads();
    if (warp == 0) {
        int64_t t = part[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += u;
        }
        part[lane] = t;
    }
    __syncthreads();
    const int64_t before = warp ? part[warp - 1] : 0;
    total = part[PT / 32 - 1];
    __syncthreads();  // part is reused by the next call
    return before + s - v;
}

// f(p) for each page of a thread's run: the pages are dealt out in runs, so that one prefix sum over the threads places
// them all in order.
template <class F>
__device__ __forceinline__ void each_page(int64_t num_pages, F f) {
    const int64_t run = (num_pages + PT - 1) / PT, p0 = (int64_t)threadIdx.x * run, p1 = min(num_pages, p0 + run);
#pragma unroll 4
    for (int64_t p = p0; p < p1; ++p) f(p);
}

// The free pages, ascending, into list; returns how many.
__device__ int64_t free_pages(const PageTableArgs &t, int32_t *list, int64_t *part) {
    int64_t mine = 0, total;
    each_page(t.num_pages, [&](int64_t p) { mine += t.refcount[p] <= 0; });
    int64_t at = block_scan(mine, part, total);
    each_page(t.num_pages, [&](int64_t p) {
        if (t.refcount[p] <= 0) list[at++] = (int32_t)p;
    });
    return total;
}

__device__ __forceinline__ bool page_ok(const PageTableArgs &t, int32_t p) { return p >= 0 && p < t.num_pages; }

template <int OP>
__global__ void __launch_bounds__(PT) kda_pages_plan_kernel(const PagesArgs a) {
    __shared__ int64_t part[PT / 32];
    const PageTableArgs &t = a.t;
    const Ws w = layout(a.ws, t.max_seqs, t.num_pages, a.n);
    const int tid = threadIdx.x;
    latent::wait_for_previous();
    latent::allow_dependent_launch();

    if constexpr (OP == PAGES_COMPACT) {
        int64_t mine = 0, used, moves;
        each_page(t.num_pages, [&](int64_t p) { mine += t.refcount[p] > 0; });
        block_scan(mine, part, used);
        // used pages behind the first `used` places, and free ones among these: as many
        mine = 0;
        each_page(t.num_pages, [&](int64_t p) {
            if (p >= used && t.refcount[p] > 0) ++mine;
            if (p < used && t.refcount[p] <= 0) mine += (int64_t)1 << 32;
        });
        const int64_t at = block_scan(mine, part, moves);
        moves &= 0xffffffff;
        int64_t from = at & 0xffffffff, to = at >> 32;
        each_page(t.num_pages, [&](int64_t p) {
            w.list[p] = (int32_t)p;
            if (p >= used && t.refcount[p] > 0) w.src[from++] = (int32_t)p;
            if (p < used && t.refcount[p] <= 0) w.dst[to++] = (int32_t)p;
        });
        __syncthreads();
        for (int64_t j = tid; j < moves; j += PT) {
            const int32_t s = __ldcg(w.src + j), d = __ldcg(w.dst + j);
            w.list[s] = d;
            t.refcount[d] = t.refcount[s];
            t.refcount[s] = 0;
        }
        if (tid == 0) w.hdr[0] = (int32_t)moves;
        return;
    }

    const int64_t cap = (int64_t)t.max_pages * t.page_size;
    const int32_t *named = OP == PAGES_FORK ? a.y : a.x;  // the rows that the items change
    for (int s = tid; s < t.max_seqs; s += PT) w.claim[s] = INT32_MAX;
    __syncthreads();
    for (int i = tid; i < a.n; i += PT) {
        const int32_t r = named[i];
        if (OP == PAGES_FORK && a.x[i] == -1) continue;  // a padding item, whatever its child
        if (r >= 0 && r < t.max_seqs) atomicMin(w.claim + r, i);
    }
    const int64_t nfree = OP == PAGES_TRUNCATE ? 0 : free_pages(t, w.list, part);
    __syncthreads();
    int64_t taken = 0;
    for (int base = 0; base < a.n; base += PT) {
        const int i = base + tid;
        int64_t need = 0;
        int32_t flag = 0, bits = 0, len = 0, last = -1;
        if (i < a.n) {
            const int32_t r = named[i];
            const int32_t p = OP == PAGES_FORK ? a.x[i] : r;  // the row whose pages count
            if (r == -1 || p == -1) {
                // a padding item
            } else if (r < 0 || r >= t.max_seqs || p < 0 || p >= t.max_seqs || __ldcg(w.claim + r) != i) {
                bits = KDA_DEV_BAD_SLOT;
            } else {
                len = t.lens[p];
                const int32_t goal = OP == PAGES_FORK ? len : a.y[i];
                if (len < 0 || len > cap || goal < 0 || goal > cap || (OP == PAGES_RESERVE && goal < len) ||
                    (OP == PAGES_TRUNCATE && goal > len) || (OP == PAGES_FORK && t.lens[r] != 0)) {
                    bits = KDA_DEV_BAD_SEQLENS;
                } else {
                    flag = 1;
                    if constexpr (OP != PAGES_TRUNCATE) {
                        const int ps = t.page_size;
                        const int64_t have = ((int64_t)len + ps - 1) / ps;
                        bool copy = len % ps != 0 && (OP == PAGES_FORK || goal > len);
                        if (copy) {
                            last = t.table[(int64_t)p * t.max_pages + have - 1];
                            if (!page_ok(t, last)) {
                                bits = KDA_DEV_BAD_PAGE;
                                flag = 0;
                            } else if (OP == PAGES_RESERVE && t.refcount[last] <= 1) {
                                copy = false;  // private already
                            }
                        }
                        if (flag) {
                            need = (OP == PAGES_FORK ? 0 : ((int64_t)goal + ps - 1) / ps - have) + copy;
                            if (copy) flag = 3;
                        }
                    }
                }
            }
        }
        int64_t total;
        const int64_t at = taken + block_scan(need, part, total);
        taken += total;
        if (i < a.n) {
            if (flag && need > 0 && at + need > nfree) {
                bits |= KDA_DEV_NO_PAGES;
                flag = 0;
            }
            w.start[i] = (int32_t)(flag && need > 0 ? at : 0);
            w.flag[i] = flag;
            w.len[i] = len;
            if constexpr (OP != PAGES_TRUNCATE) {
                w.src[i] = flag == 3 ? last : -1;
                w.dst[i] = flag == 3 ? __ldcg(w.list + at) : -1;
            }
            if (bits) set_status(a.status, bits);
        }
    }
    if (tid == 0) w.hdr[0] = OP == PAGES_TRUNCATE ? 0 : a.n;
}

// Page copies of all layers, pieces of PIECE words dealt out over the grid.  Entries that are -1 are skipped.
__device__ __forceinline__ void copy_pages(const LatentCacheArgs &c, int64_t n, const int32_t *src, const int32_t *dst,
                                           int32_t *status) {
    const int64_t words = (int64_t)c.page_size * (c.rank + c.rope) / 8;
    const int64_t pieces = (words + PIECE - 1) / PIECE;
    for (int64_t u = blockIdx.x; u < n * c.layers * pieces; u += gridDim.x) {
        const int64_t j = u / (c.layers * pieces), rest = u - j * (c.layers * pieces);
        const int64_t layer = rest / pieces, piece = rest - layer * pieces;
        const int32_t s = src[j], d = dst[j];
        if (s == -1 || d == -1) continue;
        if (s < 0 || s >= c.num_pages || d < 0 || d >= c.num_pages) {
            if (threadIdx.x == 0 && rest == 0) set_status(status, KDA_DEV_BAD_PAGE);
            continue;
        }
        const uint16_t *base = c.pages + layer * c.layer_stride;
        const uint4 *from = reinterpret_cast<const uint4 *>(base + s * c.page_stride);
        uint4 *to = reinterpret_cast<uint4 *>(const_cast<uint16_t *>(base) + d * c.page_stride);
        const int64_t w0 = piece * PIECE + threadIdx.x;
        uint4 r[UNROLL];
#pragma unroll
        for (int k = 0; k < UNROLL; ++k)
            if (w0 + k * AT < words) r[k] = __ldcs(from + w0 + k * AT);
#pragma unroll
        for (int k = 0; k < UNROLL; ++k)
            if (w0 + k * AT < words) to[w0 + k * AT] = r[k];
    }
}

template <int OP>
__global__ void __launch_bounds__(AT) kda_pages_apply_kernel(const PagesArgs a) {
    const PageTableArgs &t = a.t;
    const Ws w = layout(a.ws, t.max_seqs, t.num_pages, a.n);
    const int ps = t.page_size;
    const int tid = threadIdx.x;
    latent::wait_for_previous();  // for the plan
    latent::allow_dependent_launch();
    if constexpr (OP == PAGES_COMPACT) {
        for (int s = blockIdx.x; s < t.max_seqs; s += gridDim.x) {
            const int64_t len = t.lens[s], have = (len + ps - 1) / ps;
            if (len < 0 || have > t.max_pages) {
                if (tid == 0) set_status(a.status, KDA_DEV_BAD_SEQLENS);
                continue;
            }
            int32_t *row = t.table + (int64_t)s * t.max_pages;
            for (int64_t j = tid; j < have; j += AT) {
                const int32_t p = row[j];
                if (page_ok(t, p))
                    row[j] = w.list[p];
                else
                    set_status(a.status, KDA_DEV_BAD_PAGE);
            }
        }
    } else {
        for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
            const int32_t flag = w.flag[i];
            if (!flag) continue;
            const int32_t r = OP == PAGES_FORK ? a.y[i] : a.x[i];
            int32_t *row = t.table + (int64_t)r * t.max_pages;
            const int64_t len = w.len[i], have = (len + ps - 1) / ps;
            const bool copy = flag == 3;
            const int32_t *fresh = w.list + w.start[i];
            if constexpr (OP == PAGES_FORK) {
                const int32_t *from = t.table + (int64_t)a.x[i] * t.max_pages;
                for (int64_t j = tid; j < len / ps; j += AT) {
                    const int32_t p = from[j];
                    row[j] = p;
                    if (page_ok(t, p))
                        atomicAdd(t.refcount + p, 1);
                    else
                        set_status(a.status, KDA_DEV_BAD_PAGE);
                }
            } else if constexpr (OP == PAGES_RESERVE) {
                const int64_t want = ((int64_t)a.y[i] + ps - 1) / ps;
                for (int64_t j = have + tid; j < want; j += AT) {
                    const int32_t p = fresh[j - have + copy];
                    row[j] = p;
                    t.refcount[p] = 1;
                }
            } else {
                for (int64_t j = ((int64_t)a.y[i] + ps - 1) / ps + tid; j < have; j += AT) {
                    const int32_t p = row[j];
                    row[j] = -1;
                    if (page_ok(t, p))
                        atomicSub(t.refcount + p, 1);
                    else
                        set_status(a.status, KDA_DEV_BAD_PAGE);
                }
            }
            if (tid == 0) {
                if (copy) {
                    row[have - 1] = fresh[0];
                    t.refcount[fresh[0]] = 1;
                    if (OP == PAGES_RESERVE) atomicSub(t.refcount + w.src[i], 1);
                }
                t.lens[r] = OP == PAGES_FORK ? (int32_t)len : a.y[i];
            }
        }
    }
    if constexpr (OP != PAGES_TRUNCATE) copy_pages(a.c, w.hdr[0], w.src, w.dst, a.status);
}

__global__ void __launch_bounds__(AT) kda_pages_copy_kernel(const LatentCacheArgs c, int32_t n, const int32_t *src,
                                                            const int32_t *dst, int32_t *status) {
    latent::wait_for_previous();
    latent::allow_dependent_launch();
    copy_pages(c, n, src, dst, status);
}

// One warp a token: its sequence by a 32-way search of cu_tokens, then 16-byte copies of its row.
__global__ void __launch_bounds__(AT) kda_latent_append_kernel(const AppendArgs a) {
    latent::wait_for_previous();
    latent::allow_dependent_launch();
    const int lane = threadIdx.x & 31;
    const int64_t tok = (int64_t)blockIdx.x * (AT / 32) + (threadIdx.x >> 5);
    if (tok >= a.num_tokens) return;
    // the row itself first: it does not depend on where it goes
    const int rw = a.c.rank / 8, w = rw + a.c.rope / 8;  // 16-byte words
    const uint4 *l = reinterpret_cast<const uint4 *>(a.latent + tok * a.latent_stride);
    const uint4 *r = reinterpret_cast<const uint4 *>(a.rope + tok * a.rope_stride);
    uint4 v[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const int j = lane + 32 * k;
        if (j < w) v[k] = j < rw ? __ldcs(l + j) : __ldcs(r + j - rw);
    }
    // the last b with cu[b] <= tok: [lo, hi) narrows to one entry, 32 ways a step
    int lo = 0, hi = a.n + 1;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const bool le = at < hi && a.cu[at] <= tok;
        const uint32_t m = __ballot_sync(0xffffffffu, le);
        const int k = m ? 31 - __clz(m) : 0;
        if (!m) {  // cu[lo] > tok: before the first sequence
            lo = -1;
            break;
        }
        lo += k * step;
        hi = min(hi, lo + step);
    }
    if (lo < 0 || lo >= a.n) return;  // behind the last sequence
    const int64_t c0 = a.cu[lo], c1 = a.cu[lo + 1];
    const int32_t row = a.rows ? a.rows[lo] : lo;
    if (row == -1) return;
    int32_t bits = 0;
    int64_t pos = 0;
    int32_t page = 0;
    if (row < 0 || row >= a.t.max_seqs) {
        bits = KDA_DEV_BAD_SLOT;
    } else {
        const int64_t len = a.t.lens[row];
        pos = len - (c1 - tok);
        if (c0 < 0 || c1 > a.num_tokens || tok >= c1 || pos < 0 || len > (int64_t)a.t.max_pages * a.t.page_size) {
            bits = KDA_DEV_BAD_SEQLENS;
        } else {
            page = a.t.table[(int64_t)row * a.t.max_pages + pos / a.t.page_size];
            if (!page_ok(a.t, page)) bits = KDA_DEV_BAD_PAGE;
        }
    }
    if (bits) {
        if (lane == 0) set_status(a.status, bits);
        return;
    }
    uint4 *to = reinterpret_cast<uint4 *>(a.c.pages + page * a.c.page_stride +
                                          (pos % a.t.page_size) * (a.c.rank + a.c.rope));
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (lane + 32 * k < w) to[lane + 32 * k] = v[k];
}

}  // namespace pages

size_t pages_workspace_bytes(int32_t max_seqs, int64_t num_pages, int32_t n) {
    const int64_t copies = n > num_pages ? n : num_pages;
    const int64_t ints = 16 + (int64_t)max_seqs + 3 * (int64_t)n + num_pages + 2 * copies;
    return (size_t)((ints * 4 + 15) / 16 * 16);
}

template <int OP>
static int launch_pages_op(const PagesArgs &a, cudaStream_t st) {
    using namespace pages;
    latent::dependent_launch(kda_pages_plan_kernel<OP>, dim3(1), PT, 0, st, a);
    const int rc = launch_result("kda_pages_plan_kernel launch");
    if (rc != KDA_OK) return rc;
    // eight CTAs a multiprocessor are resident; how much there is to copy is known on the device alone
    latent::dependent_launch(kda_pages_apply_kernel<OP>, dim3((unsigned)current_device_sms() * 8), AT, 0, st, a);
    return launch_result("kda_pages_apply_kernel launch");
}

int launch_pages(PageOp op, const PagesArgs &a, cudaStream_t st) {
    switch (op) {
        case PAGES_RESERVE: return launch_pages_op<PAGES_RESERVE>(a, st);
        case PAGES_TRUNCATE: return launch_pages_op<PAGES_TRUNCATE>(a, st);
        case PAGES_FORK: return launch_pages_op<PAGES_FORK>(a, st);
        default: return launch_pages_op<PAGES_COMPACT>(a, st);
    }
}

int launch_pages_copy(const LatentCacheArgs &c, int32_t n, const int32_t *src, const int32_t *dst, int32_t *status,
                      cudaStream_t st) {
    using namespace pages;
    latent::dependent_launch(kda_pages_copy_kernel, dim3((unsigned)current_device_sms() * 8), AT, 0, st, c, n, src, dst,
                             status);
    return launch_result("kda_pages_copy_kernel launch");
}

int launch_latent_append(const AppendArgs &a, cudaStream_t st) {
    using namespace pages;
    const int64_t blocks = (a.num_tokens + AT / 32 - 1) / (AT / 32);
    latent::dependent_launch(kda_latent_append_kernel, dim3((unsigned)blocks), AT, 0, st, a);
    return launch_result("kda_latent_append_kernel launch");
}

}  // namespace kda
