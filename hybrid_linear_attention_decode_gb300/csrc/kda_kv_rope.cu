// kda_kv_rope.cu -- rotary positions (include/kda.h: kda_rope_apply) and the key-value cache's row writer
// (kda_kv_append), which rotates on the way.
//
//   y1 = s (x1 cos a - x2 sin a),  y2 = s (x2 cos a + x1 sin a),  a = position * theta_i
//
// Every value is read once and written once: bound by bytes, and in a decode step by the latency of one launch.
// The angle in turns is the product of the position and a 64-bit fraction of a turn, modulo 2^64: whole turns fall out of
// the top exactly, so no 64-bit floating point and no long argument reduction is needed at far positions.  Its upper 32 bits
// go to sincospif as a number from -1 to 1.
//
// A thread has one chunk of 8 pairs (two 16-byte words: x1 and x2, or 8 neighbouring pairs) of HPT heads of a token, so that
// sines and cosines are computed once for these and HPT * 2 loads are in flight.  Chunks behind the rotated part are copied.
#include "kda_kv.cuh"

namespace kda {
namespace kv {

constexpr int NT = 128;

// 16 bytes, or one element where offset or dim let pairs begin inside a 16-byte word.
template <int VEC>
struct Word;
template <>
struct Word<8> {
    using T = uint4;
};
template <>
struct Word<1> {
    using T = uint16_t;
};

template <bool FP16>
__device__ __forceinline__ void unpack(uint4 w, float (&f)[8]) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 t = to_f2<FP16>(x[k]);
        f[2 * k] = t.x;
        f[2 * k + 1] = t.y;
    }
}
template <bool FP16>
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    using latent::pack2;
    return make_uint4(pack2<FP16>(f[0], f[1]), pack2<FP16>(f[2], f[3]), pack2<FP16>(f[4], f[5]), pack2<FP16>(f[6], f[7]));
}

// Where the items of a head of D elements are: the first `rot` are chunks of VEC pairs, the others copy two words each.
template <int VEC>
struct Items {
    int32_t rot, pass, words;  // chunks of pairs; copying items; words that are copied
    __host__ __device__ Items(const RopeArgs &r, int D, bool in_place) {
        rot = r.dim / (2 * VEC);
        words = in_place ? 0 : (D - r.dim) / VEC;
        pass = (words + 1) / 2;
    }
    __host__ __device__ int count() const { return rot + pass; }
    // The elements at which item i's two words begin; the second may be missing (-1).
    __device__ __forceinline__ void at(const RopeArgs &r, int i, int &e0, int &e1) const {
        if (i < rot) {
            e0 = r.offset + (r.interleaved ? 2 : 1) * VEC * i;
            e1 = r.interleaved ? e0 + VEC : e0 + r.dim / 2;
        } else {
            const int p = 2 * (i - rot);
            e0 = p * VEC < r.offset ? p * VEC : p * VEC + r.dim;
            e1 = p + 1 >= words ? -1 : (p + 1) * VEC < r.offset ? (p + 1) * VEC : (p + 1) * VEC + r.dim;
        }
    }
};

template <int VEC>
struct Turn {
    float c[VEC], s[VEC];
};

// Sines and cosines of the VEC pairs of item i, times the scale.
template <int VEC>
__device__ __forceinline__ Turn<VEC> turn_of(const RopeArgs &r, int i, int32_t position, bool inverse) {
    Turn<VEC> t;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const uint64_t turns = (uint64_t)(int64_t)position * r.turns[VEC * i + j];
        const float half = (float)(int32_t)(turns >> 32) * 0x1p-31f;  // half turns, from -1 to 1
        float sn, cs;
        sincospif(half, &sn, &cs);
        t.c[j] = cs * r.scale;
        t.s[j] = (inverse ? -sn : sn) * r.scale;
    }
    return t;
}

template <bool FP16>
__device__ __forceinline__ void rotate(uint4 &a, uint4 &b, const Turn<8> &t, bool interleaved) {
    float x[8], y[8], u[8], v[8];
    unpack<FP16>(a, x);
    unpack<FP16>(b, y);
    if (interleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u[2 * j] = fmaf(x[2 * j], t.c[j], -x[2 * j + 1] * t.s[j]);
            u[2 * j + 1] = fmaf(x[2 * j + 1], t.c[j], x[2 * j] * t.s[j]);
            v[2 * j] = fmaf(y[2 * j], t.c[4 + j], -y[2 * j + 1] * t.s[4 + j]);
            v[2 * j + 1] = fmaf(y[2 * j + 1], t.c[4 + j], y[2 * j] * t.s[4 + j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            u[j] = fmaf(x[j], t.c[j], -y[j] * t.s[j]);
            v[j] = fmaf(y[j], t.c[j], x[j] * t.s[j]);
        }
    }
    a = pack<FP16>(u);
    b = pack<FP16>(v);
}
template <bool FP16>
__device__ __forceinline__ void rotate(uint16_t &a, uint16_t &b, const Turn<1> &t, bool) {
    const float x = to_f<FP16>(a), y = to_f<FP16>(b);
    a = from_f<FP16>(fmaf(x, t.c[0], -y * t.s[0]));
    b = from_f<FP16>(fmaf(y, t.c[0], x * t.s[0]));
}

__device__ __forceinline__ uint4 load(const uint4 *p) { return __ldcs(p); }
__device__ __forceinline__ uint16_t load(const uint16_t *p) { return __ldcs(p); }

// Two words of up to HPT heads, and back.
template <int VEC, int HPT, class T = typename Word<VEC>::T>
__device__ __forceinline__ void get(T (&r)[HPT][2], const uint16_t *x, int64_t hs, int h0, int H, int e0, int e1) {
#pragma unroll
    for (int k = 0; k < HPT; ++k)
        if (h0 + k < H) {
            const uint16_t *p = x + (h0 + k) * hs;
            r[k][0] = load(reinterpret_cast<const T *>(p + e0));
            if (e1 >= 0) r[k][1] = load(reinterpret_cast<const T *>(p + e1));
        }
}
template <int VEC, int HPT, class T = typename Word<VEC>::T>
__device__ __forceinline__ void put(const T (&r)[HPT][2], uint16_t *x, int64_t hs, int h0, int H, int e0, int e1) {
#pragma unroll
    for (int k = 0; k < HPT; ++k)
        if (h0 + k < H) {
            uint16_t *p = x + (h0 + k) * hs;
            *reinterpret_cast<T *>(p + e0) = r[k][0];
            if (e1 >= 0) *reinterpret_cast<T *>(p + e1) = r[k][1];
        }
}

// Threads of a token: `groups` of HPT heads times the items.  Tokens whose threads fill less than a CTA share one; the
// threads of larger ones lie along the grid's second axis.
template <bool FP16, int VEC, int HPT>
__global__ void __launch_bounds__(NT) kda_rope_kernel(const RotateArgs a, int units, int per_cta) {
    wait_for_previous();
    allow_dependent_launch();
    const Items<VEC> items(a.r, a.D, a.in_place);
    const int in_cta = threadIdx.x / units;
    const int u = units > NT ? blockIdx.y * NT + threadIdx.x : threadIdx.x - in_cta * units;
    const int64_t tok = units > NT ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * per_cta + in_cta;
    if (u >= units || (units <= NT && in_cta >= per_cta) || tok >= a.num_tokens) return;
    const int group = u / items.count(), i = u - group * items.count();
    int e0, e1;
    items.at(a.r, i, e0, e1);
    typename Word<VEC>::T r[HPT][2];
    get<VEC, HPT>(r, a.x + tok * a.x_ts, a.x_hs, group * HPT, a.H, e0, e1);
    if (i < items.rot) {
        const Turn<VEC> t = turn_of<VEC>(a.r, i, a.positions[tok], a.inverse);
#pragma unroll
        for (int k = 0; k < HPT; ++k) rotate<FP16>(r[k][0], r[k][1], t, a.r.interleaved);
    }
    put<VEC, HPT>(r, a.out + tok * a.o_ts, a.o_hs, group * HPT, a.H, e0, e1);
}

// Where a token goes.
struct Place {
    int64_t page;  // words before its page; -1: nowhere
    int32_t slot;  // within the page
    int32_t live;  // a token of some sequence, whose queries are rotated
};

template <bool FP16, int VEC, int HPT>
__global__ void __launch_bounds__(NT) kda_kv_append_kernel(const KvAppendArgs a, int units, int per_cta) {
    __shared__ Place place[NT];
    wait_for_previous();
    allow_dependent_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const KvCacheArgs &c = a.c;
    const int d = c.d, kv = c.heads;
    const Items<VEC> items(a.r, d, false);
    const int in_cta = units > NT ? 0 : threadIdx.x / units;
    int u = units > NT ? blockIdx.y * NT + threadIdx.x : threadIdx.x - in_cta * units;
    const int64_t tok0 = (int64_t)blockIdx.x * per_cta, tok = tok0 + in_cta;
    const bool mine = u < units && in_cta < per_cta && tok < a.num_tokens;

    // the rows first: they do not depend on where they go
    const int n = items.count(), nv = (d / 8 + 1) / 2, gq = (a.H + HPT - 1) / HPT, gk = (kv + HPT - 1) / HPT;
    typename Word<VEC>::T r[HPT][2];
    uint4 single[VEC == 8 ? 1 : HPT][2];  // values are copied in 16-byte words in either case
    auto &w = [&]() -> uint4(&)[HPT][2] {
        if constexpr (VEC == 8)
            return r;
        else
            return single;
    }();
    int kind = 3, h0 = 0, i = 0, e0 = 0, e1 = -1;  // 0: queries, 1: keys, 2: values, 3: stats
    if (mine) {
        if (u < (gq + gk) * n) {
            const int group = u / n;
            i = u - group * n;
            items.at(a.r, i, e0, e1);
            kind = group >= gq;
            h0 = (kind ? group - gq : group) * HPT;
            if (kind)
                get<VEC, HPT>(r, a.k + tok * a.k_ts, a.k_hs, h0, kv, e0, e1);
            else
                get<VEC, HPT>(r, a.q + tok * a.q_ts, a.q_hs, h0, a.H, e0, e1);
        } else if ((u -= (gq + gk) * n) < gk * nv) {
            kind = 2;
            h0 = u / nv * HPT;
            e0 = (u % nv) * 16;
            e1 = e0 + 8 < d ? e0 + 8 : -1;
            get<8, HPT>(w, a.v + tok * a.v_ts, a.v_hs, h0, kv, e0, e1);
        } else {
            h0 = u - gk * nv;
        }
    }

    if (kind < 2 && i < items.rot) {  // (those of threads without a token are not used)
        const Turn<VEC> t = turn_of<VEC>(a.r, i, a.positions[tok], false);
#pragma unroll
        for (int k = 0; k < HPT; ++k) rotate<FP16>(r[k][0], r[k][1], t, a.r.interleaved);
    }

    for (int j = warp; j < per_cta && tok0 + j < a.num_tokens; j += blockDim.x / 32) {
        const int64_t t = tok0 + j;
        // in a decode step sequence t has token t: looked at first, as a search is two loads more that wait for one another
        const int g = (int)min(t, (int64_t)a.n - 1);
        const int b = a.cu[g] == t && a.cu[g + 1] == t + 1 ? g : sequence_of(a.cu, a.n, t, lane);
        Place p = {-1, 0, 0};
        if (b >= 0 && b < a.n) {
            const int64_t c0 = a.cu[b], c1 = a.cu[b + 1];
            const int32_t row = a.rows ? a.rows[b] : b;
            int32_t bits = 0;
            if (c0 < 0 || c1 > a.num_tokens || t >= c1) {
                bits = KDA_DEV_BAD_SEQLENS;
            } else {
                p.live = 1;
                if (row < -1 || row >= a.t.max_seqs) {
                    bits = KDA_DEV_BAD_SLOT;
                } else if (row >= 0) {
                    const int64_t len = a.t.lens[row], slot = len - (c1 - t);
                    if (slot < 0 || len > (int64_t)a.t.max_pages * a.t.page_size) {
                        bits = KDA_DEV_BAD_SEQLENS;
                    } else {
                        const int32_t page = a.t.table[(int64_t)row * a.t.max_pages + slot / c.page_size];
                        if (page_ok(a.t, page)) {
                            p.page = page * c.page_stride;
                            p.slot = (int32_t)(slot % c.page_size);
                        } else {
                            bits = KDA_DEV_BAD_PAGE;
                        }
                    }
                }
            }
            if (bits && lane == 0) set_status(a.status, bits);
        }
        if (lane == 0) place[j] = p;
    }
    __syncthreads();
    if (!mine) return;
    const Place p = place[in_cta];
    if (kind == 0 ? !p.live : p.page < 0) return;
    uint16_t *page = c.pages + p.page;
    if (kind < 2) {
        if (kind)
            put<VEC, HPT>(r, page + (int64_t)p.slot * d, (int64_t)c.page_size * d, h0, kv, e0, e1);
        else
            put<VEC, HPT>(r, a.q_out + tok * a.H * d, d, h0, a.H, e0, e1);
    } else if (kind == 2) {
        put<8, HPT>(w, page + value_at(c, 0) + (int64_t)p.slot * d, (int64_t)c.page_size * d, h0, kv, e0, e1);
    } else {
        int32_t *st = reinterpret_cast<int32_t *>(page + stats_at(c, h0)) + p.slot;
        st[0] = 0;
        st[c.page_size] = a.positions[tok];
    }
}

// 16-byte words where pairs of a chunk begin and end at such words, as at offset 0 (or a multiple of 8) and dim a multiple
// of 16; else single elements.
inline bool wide(const RopeArgs &r) { return r.offset % 8 == 0 && r.dim % 16 == 0; }

struct Grid {
    dim3 grid;
    unsigned threads;
    int per_cta;
};
inline Grid grid_of(int64_t tokens, int64_t units) {
    Grid g;
    g.per_cta = units > NT ? 1 : (int)(NT / units);
    g.threads = units > NT ? NT : (unsigned)(g.per_cta * units + 31) / 32 * 32;
    g.grid = dim3((unsigned)((tokens + g.per_cta - 1) / g.per_cta), (unsigned)(units > NT ? (units + NT - 1) / NT : 1));
    return g;
}

template <int VEC, int HPT>
int launch_rotate_as(const RotateArgs &a, cudaStream_t st) {
    const Items<VEC> items(a.r, a.D, a.in_place);
    const int64_t units = (int64_t)((a.H + HPT - 1) / HPT) * items.count();
    const Grid g = grid_of(a.num_tokens, units);
    auto k = a.fp16 ? kda_rope_kernel<true, VEC, HPT> : kda_rope_kernel<false, VEC, HPT>;
    dependent_launch(k, g.grid, g.threads, 0, st, a, (int)units, g.per_cta);
    return launch_result("kda_rope_kernel launch");
}

template <int VEC, int HPT>
int launch_append_as(const KvAppendArgs &a, cudaStream_t st) {
    const Items<VEC> items(a.r, a.c.d, false);
    const int64_t gq = (a.H + HPT - 1) / HPT, gk = (a.c.heads + HPT - 1) / HPT;
    const int64_t units = (gq + gk) * items.count() + gk * ((a.c.d / 8 + 1) / 2) + (a.c.stats ? a.c.heads : 0);
    const Grid g = grid_of(a.num_tokens, units);
    auto k = a.c.fp16 ? kda_kv_append_kernel<true, VEC, HPT> : kda_kv_append_kernel<false, VEC, HPT>;
    dependent_launch(k, g.grid, g.threads, 0, st, a, (int)units, g.per_cta);
    return launch_result("kda_kv_append_kernel launch");
}

}  // namespace kv

int launch_rotate(const RotateArgs &a, cudaStream_t st) {
    using namespace kv;
    const bool many = a.num_tokens * a.H >= (int64_t)current_device_sms() * 256;
    if (!wide(a.r)) return launch_rotate_as<1, 1>(a, st);
    return many ? launch_rotate_as<8, 4>(a, st) : launch_rotate_as<8, 1>(a, st);
}

int launch_kv_append(const KvAppendArgs &a, cudaStream_t st) {
    using namespace kv;
    const bool many = a.num_tokens * (a.H + a.c.heads) >= (int64_t)current_device_sms() * 256;
    if (!wide(a.r)) return launch_append_as<1, 1>(a, st);
    return many ? launch_append_as<8, 4>(a, st) : launch_append_as<8, 1>(a, st);
}

}  // namespace kda
