// kvcache.cu -- dflash2_rope_append and dflash2_kv_evict: what writes to the
// paged cache.
#include "common.cuh"
#include "host.hpp"

namespace dfl {

bool kv_cache_ok(const dflash2_kv_cache *c, const int32_t *table, int32_t max_pages, int64_t B);

// ------------------------------------------------------------------ append --
struct AppendArgs {
    char *ck, *cv;
    float *weight;
    int32_t *pos;
    int64_t num_pages, page_stride, head_stride, slot_stride;
    int Hkv, page_size, d;
    const int32_t *table;
    int max_pages;
    const int32_t *kv_len, *q_len, *seq_pos;
    const char *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    int64_t tokens;  // B * T
    int T, Hq;
    const float *cos_sin;
    int64_t n_pos;
    int rot;
    const int32_t *pos_ids;
    int axes;
    const uint8_t *pair_axis;
    const void *q_norm, *k_norm;
    float eps;
    void *q_out;
    int32_t *kv_len_out;
    const unsigned int *hold;  // test hook: NULL, or a word that the streaming kernel's filling warps wait on
    long long hold_cycles;
};

// Where a new token goes.
struct AppendToken {
    bool live;      // t < q_len
    int page, off;  // page -1: nowhere
    int seq;        // position in the sequence
};

// What the call's arrays say of a token's request.
struct AppendRaw {
    int64_t b;
    int t, n, nq, sp;
};
__device__ __forceinline__ AppendRaw append_raw(const AppendArgs &a, int64_t tok) {
    AppendRaw x;
    const uint32_t tk = static_cast<uint32_t>(tok), b = tk / static_cast<uint32_t>(a.T);  // B * T < 2^31
    x.b = b;
    x.t = static_cast<int>(tk - b * static_cast<uint32_t>(a.T));
    x.n = a.kv_len[x.b];
    x.nq = a.q_len ? a.q_len[x.b] : a.T;
    x.sp = a.seq_pos ? a.seq_pos[x.b] : x.n;
    return x;
}
__device__ __forceinline__ AppendToken append_token(const AppendArgs &a, const AppendRaw &x, bool lead) {
    AppendToken r;
    const int nq = x.nq < 0 ? 0 : (x.nq > a.T ? a.T : x.nq);
    r.live = x.t < nq;
    r.page = -1;
    r.off = 0;
    if (x.n >= 0) {
        const uint32_t slot = static_cast<uint32_t>(x.n) + static_cast<uint32_t>(x.t);
        const uint32_t pi = slot / static_cast<uint32_t>(a.page_size);
        if (pi < static_cast<uint32_t>(a.max_pages)) {
            const int page = a.table[x.b * a.max_pages + pi];
            if (page >= 0 && page < a.num_pages) r.page = page;
            r.off = static_cast<int>(slot - pi * static_cast<uint32_t>(a.page_size));
        }
    }
    r.seq = x.sp + x.t;
    if (lead && x.t == 0 && a.kv_len_out) a.kv_len_out[x.b] = x.n + nq;
    return r;
}

template <typename E>
__device__ __forceinline__ float ld1(const void *p, int64_t i);
template <>
__device__ __forceinline__ float ld1<float>(const void *p, int64_t i) {
    return static_cast<const float *>(p)[i];
}
template <>
__device__ __forceinline__ float ld1<unsigned short>(const void *p, int64_t i) {
    return __uint_as_float(static_cast<uint32_t>(static_cast<const unsigned short *>(p)[i]) << 16);
}
__device__ __forceinline__ void st1(float *p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void st1(unsigned short *p, int64_t i, float v) {
    unsigned short o;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(o) : "f"(v));
    p[i] = o;
}

// Any d and rot: one warp per (token, head), a pair of entries per step.
// Bound: one entry per load and store, and the table's row read by every head.
// 28 heads of 96, rot 24: 3.6 us a token; 512 tokens of 56 such heads 15.7 us
// (11 MB), 16384 of 32 236 us (201 MB, 0.9 TB/s); 4096 tokens of 12 heads of 1024
// 93 us (201 MB, 2.2 TB/s).
template <typename E, bool INTER>
__global__ void __launch_bounds__(256) k_append_any(AppendArgs a) {
    pdl_wait();
    const int heads = a.Hq + 2 * a.Hkv, lane = threadIdx.x & 31, half = a.rot / 2;
    const int64_t units = a.tokens * heads, step = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); u < units; u += step) {
        const int64_t tok = u / heads;
        const int head = static_cast<int>(u - tok * heads);
        const AppendToken at = append_token(a, append_raw(a, tok), head == 0 && lane == 0);
        const bool is_q = head < a.Hq, is_v = head >= a.Hq + a.Hkv;
        const int kh = is_q ? 0 : (is_v ? head - a.Hq - a.Hkv : head - a.Hq);
        const E *src;
        E *dst;
        if (is_q) {
            src = reinterpret_cast<const E *>(a.q) + tok * a.q_stride + static_cast<int64_t>(head) * a.d;
            dst = static_cast<E *>(a.q_out) + (tok * a.Hq + head) * a.d;
            if (!at.live || at.page < 0) {
                for (int i = lane; i < a.d; i += 32) st1(dst, i, at.live ? NAN : 0.f);
                continue;
            }
        } else {
            if (!at.live || at.page < 0) continue;
            src = is_v ? reinterpret_cast<const E *>(a.v) + tok * a.v_stride + static_cast<int64_t>(kh) * a.d
                       : reinterpret_cast<const E *>(a.k) + tok * a.k_stride + static_cast<int64_t>(kh) * a.d;
            dst = reinterpret_cast<E *>(is_v ? a.cv : a.ck) + at.page * a.page_stride + kh * a.head_stride +
                  at.off * a.slot_stride;
        }
        if (is_v) {
            for (int i = lane; i < a.d; i += 32) dst[i] = src[i];
            continue;
        }
        if (!is_q && lane == 0) {
            const int64_t si = (static_cast<int64_t>(at.page) * a.Hkv + kh) * a.page_size + at.off;
            if (a.weight) a.weight[si] = 0.f;
            if (a.pos) a.pos[si] = at.seq;
        }
        const void *nw = is_q ? a.q_norm : a.k_norm;
        float f = 1.f;
        if (nw) {
            float ss = 0.f;
            for (int i = lane; i < a.d; i += 32) {
                const float x = ld1<E>(src, i);
                ss = fmaf(x, x, ss);
            }
            f = 1.0f / sqrtf(warp_sum(ss) / a.d + a.eps);
        }
        for (int p = lane; p < half; p += 32) {
            const int i = INTER ? 2 * p : p, j = INTER ? 2 * p + 1 : p + half;
            int ax = a.pair_axis ? a.pair_axis[p] : 0;
            ax = ax < a.axes ? ax : a.axes - 1;
            const int id = a.pos_ids[ax * a.tokens + tok];
            float cs = NAN, sn = NAN;
            if (id >= 0 && id < a.n_pos) {
                cs = a.cos_sin[static_cast<int64_t>(id) * a.rot + p];
                sn = a.cos_sin[static_cast<int64_t>(id) * a.rot + half + p];
            }
            float x = ld1<E>(src, i), y = ld1<E>(src, j);
            if (nw) {
                x = x * f * ld1<E>(nw, i);
                y = y * f * ld1<E>(nw, j);
            }
            st1(dst, i, fmaf(x, cs, -y * sn));
            st1(dst, j, fmaf(y, cs, x * sn));
        }
        for (int i = a.rot + lane; i < a.d; i += 32) {
            float x = ld1<E>(src, i);
            if (nw) x = x * f * ld1<E>(nw, i);
            st1(dst, i, x);
        }
    }
}

// 16-byte vectors: a lane takes two vectors of a head, rotated together (x of
// the pairs and y; interleaved pairs lie within a vector), so its cosines and
// sines serve the heads it walks through, which are all queries, all keys or
// all values.  A head is `lanes` neighbouring lanes, which share the norm's
// sum.  Arithmetic in packed pairs.
//
// Bound: the heads' bytes, read and written once; the table's rows are shared
// by a token's heads and stay in L1 and L2.  16384 tokens of 32 heads of 256,
// three axes, normalised (537 MB): 155 us, 3.5 TB/s, where the issue slots of
// two CTAs per SM are half used and the rest waits for dependent reads (such
// blocks stream through shared memory instead, below); more CTAs in fewer
// registers (158 to 188 us), eight heads per thread (206 us) and two (190 us)
// were slower.  One token of 28 heads: 2.4 us.
constexpr int APPEND_BATCH = 4;  // heads whose loads a thread has in flight

template <typename E>
struct Vec {
    static constexpr int N = 16 / sizeof(E);
};
// A vector's entries as packed pairs of floats.
template <typename E>
__device__ __forceinline__ void unpack(const uint4 &v, uint64_t *x);
template <>
__device__ __forceinline__ void unpack<float>(const uint4 &v, uint64_t *x) {
    x[0] = pack2(v.x, v.y);
    x[1] = pack2(v.z, v.w);
}
template <>
__device__ __forceinline__ void unpack<unsigned short>(const uint4 &v, uint64_t *x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = pack2(w[i] << 16, w[i] & 0xffff0000u);
}
template <typename E>
__device__ __forceinline__ uint4 pack(const uint64_t *x);
template <>
__device__ __forceinline__ uint4 pack<float>(const uint64_t *x) {
    return make_uint4(lo32(x[0]), hi32(x[0]), lo32(x[1]), hi32(x[1]));
}
template <>
__device__ __forceinline__ uint4 pack<unsigned short>(const uint64_t *x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
            : "=r"(w[i])
            : "f"(__uint_as_float(hi32(x[i]))), "f"(__uint_as_float(lo32(x[i]))));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
    return pack2(__float_as_uint(lo), __float_as_uint(hi));
}

template <int W>
__device__ __forceinline__ void cos_load(const float *p, float *x) {
    if (W == 4) {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        x[0] = v.x;
        x[1] = v.y;
        x[W > 2 ? 2 : 0] = v.z;
        x[W > 3 ? 3 : 0] = v.w;
    } else {
        const float2 v = *reinterpret_cast<const float2 *>(p);
        x[0] = v.x;
        x[1] = v.y;
    }
}

template <typename E>
__device__ __forceinline__ float sum_squares(const uint4 &x, const uint4 &y) {
    constexpr int H = Vec<E>::N / 2;
    uint64_t u[H], v[H];
    unpack<E>(x, u);
    unpack<E>(y, v);
    uint64_t s2 = mul2(u[0], u[0]);
#pragma unroll
    for (int k = 1; k < H; ++k) s2 = fma2(u[k], u[k], s2);
#pragma unroll
    for (int k = 0; k < H; ++k) s2 = fma2(v[k], v[k], s2);
    return __uint_as_float(lo32(s2)) + __uint_as_float(hi32(s2));
}

// A vector pair's rotation: (x, y) -> (x c - y s, y c + x s).
template <bool INTER, int H>
__device__ __forceinline__ void append_turn(uint64_t *u, uint64_t *v, const float *cs, const float *sn) {
#pragma unroll
    for (int k = 0; k < H; ++k) {
        if (INTER) {  // within the packed pair
            const uint64_t us = pack2(hi32(u[k]), lo32(u[k])), vs = pack2(hi32(v[k]), lo32(v[k]));
            u[k] = fma2(u[k], pair_of(cs[k], cs[k]), mul2(us, pair_of(-sn[k], sn[k])));
            v[k] = fma2(v[k], pair_of(cs[H + k], cs[H + k]), mul2(vs, pair_of(-sn[H + k], sn[H + k])));
        } else {
            const uint64_t c2 = pair_of(cs[2 * k], cs[2 * k + 1]), s2 = pair_of(sn[2 * k], sn[2 * k + 1]);
            const uint64_t t = fma2(v[k], c2, mul2(u[k], s2));
            u[k] = fma2(u[k], c2, mul2(v[k], pair_of(-sn[2 * k], -sn[2 * k + 1])));
            v[k] = t;
        }
    }
}

template <typename E, bool INTER, bool NORM>
__global__ void __launch_bounds__(256) k_append_vec(AppendArgs a, int lanes_log2, int per) {
    constexpr int N = Vec<E>::N, H = N / 2;  // entries and pairs of a vector
    pdl_wait();
    const int half = a.rot / 2;
    // a token's units: those of its queries, of its keys, of its values; a unit has heads first, first + step, ..
    const int nq = (a.Hq + per - 1) / per, nk = (a.Hkv + per - 1) / per;
    const uint32_t unit = blockIdx.x * (256u >> lanes_log2) + (threadIdx.x >> lanes_log2);  // below 2^32
    const int c = threadIdx.x & ((1 << lanes_log2) - 1);  // the lane's pair of vectors
    const uint32_t units = static_cast<uint32_t>(nq + 2 * nk), tk = unit / units;
    const bool inside = tk < a.tokens, mine = inside && c * 2 * N < a.d;
    const int64_t tok = inside ? tk : 0;
    int first = inside ? static_cast<int>(unit - tk * units) : 0;
    const bool is_q = first < nq, is_v = first >= nq + nk, lead = inside && first == 0 && c == 0;
    first -= is_q ? 0 : is_v ? nq + nk : nq;
    const int step = is_q ? nq : nk, heads = is_q ? a.Hq : a.Hkv;
    const bool turned = mine && c * 2 * N < a.rot;
    // The vectors' first entries: one in each half of what is rotated, or of the rest, so that neighbouring lanes'
    // vectors lie side by side.
    const int e0 = turned ? c * N : a.rot + (c - half / N) * N;
    const int e1 = e0 + (turned ? half : (a.d - a.rot) / 2);
    // The reads in the order of their dependence: what the arrays say of the token, its heads, then its row of the
    // table and its page.
    const AppendRaw raw = append_raw(a, tok);
    const int id0 = a.pos_ids[tok];
    const E *src = is_q   ? reinterpret_cast<const E *>(a.q) + tok * a.q_stride
                   : is_v ? reinterpret_cast<const E *>(a.v) + tok * a.v_stride
                          : reinterpret_cast<const E *>(a.k) + tok * a.k_stride;
    uint4 x[APPEND_BATCH], y[APPEND_BATCH];
#pragma unroll
    for (int i = 0; i < APPEND_BATCH; ++i) {
        const int h = first + i * step;
        x[i] = y[i] = make_uint4(0, 0, 0, 0);
        if (i < per && h < heads && mine) {
            x[i] = *reinterpret_cast<const uint4 *>(src + h * a.d + e0);
            y[i] = *reinterpret_cast<const uint4 *>(src + h * a.d + e1);
        }
    }
    // cosine i of the lane is pair pair(i)'s: entries e0 + i and e1 + i, or, interleaved, first the pairs within the
    // vector at e0, then those within the one at e1
    constexpr int W = INTER ? N / 2 : 4;
    auto pair = [&](int i) { return !INTER ? c * N + i : i < N / 2 ? c * N / 2 + i : (half + c * N) / 2 + i - N / 2; };
    float cs[N], sn[N];
    if (turned && !is_v) {
        if (a.axes == 1) {
            const bool ok = id0 >= 0 && id0 < a.n_pos;
            const float *row = a.cos_sin + static_cast<int64_t>(ok ? id0 : 0) * a.rot;
#pragma unroll
            for (int i = 0; i < N; i += W) {
                cos_load<W>(row + pair(i), cs + i);
                cos_load<W>(row + half + pair(i), sn + i);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) cs[i] = ok ? cs[i] : NAN;
        } else {
            int id[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                int ax = a.pair_axis ? a.pair_axis[pair(i)] : 0;
                ax = ax < a.axes ? ax : a.axes - 1;
                id[i] = a.pos_ids[ax * a.tokens + tok];
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const bool ok = id[i] >= 0 && id[i] < a.n_pos;
                const float *row = a.cos_sin + static_cast<int64_t>(ok ? id[i] : 0) * a.rot + pair(i);
                cs[i] = ok ? row[0] : NAN;
                sn[i] = row[half];
            }
        }
    }
    const void *nw = is_q ? a.q_norm : a.k_norm;
    const bool norm = NORM && !is_v && nw;
    uint64_t wx[H], wy[H];
    if (norm && mine) {
        unpack<E>(*reinterpret_cast<const uint4 *>(static_cast<const E *>(nw) + e0), wx);
        unpack<E>(*reinterpret_cast<const uint4 *>(static_cast<const E *>(nw) + e1), wy);
    }
    const AppendToken at = append_token(a, raw, lead);
    const bool stored = at.live && at.page >= 0;
    E *dst = is_q ? static_cast<E *>(a.q_out) + tok * a.Hq * a.d
                  : reinterpret_cast<E *>(is_v ? a.cv : a.ck) + (at.page * a.page_stride + at.off * a.slot_stride);
    const int64_t dst_step = is_q ? a.d : a.head_stride;
    const float inv_d = 1.0f / a.d;
    float ss[APPEND_BATCH];
    if (NORM) {  // the heads' sums go through the lanes side by side
#pragma unroll
        for (int i = 0; i < APPEND_BATCH; ++i) ss[i] = norm ? sum_squares<E>(x[i], y[i]) : 0.f;
        for (int d = 1 << lanes_log2 >> 1; d >= 1; d >>= 1)
#pragma unroll
            for (int i = 0; i < APPEND_BATCH; ++i) ss[i] += __shfl_xor_sync(FULL, ss[i], d);
    }
#pragma unroll
    for (int i = 0; i < APPEND_BATCH; ++i) {
        if (i >= per) break;
        const int h = first + i * step;
        uint64_t u[H], v[H];
        if (!is_v) {
            unpack<E>(x[i], u);
            unpack<E>(y[i], v);
        }
        if (NORM && norm) {
            const float f = rsqrtf(ss[i] * inv_d + a.eps);
            const uint64_t ff = pair_of(f, f);
#pragma unroll
            for (int k = 0; k < H; ++k) {
                u[k] = mul2(mul2(u[k], ff), wx[k]);
                v[k] = mul2(mul2(v[k], ff), wy[k]);
            }
        }
        if (turned && !is_v) append_turn<INTER, H>(u, v, cs, sn);
        if (!mine || h >= heads || (!is_q && !stored)) continue;
        uint4 ox = x[i], oy = y[i];
        if (!is_v) {
            ox = pack<E>(u);
            oy = pack<E>(v);
        }
        if (is_q && !stored) {
            const uint32_t w = !at.live ? 0u : sizeof(E) == 2 ? 0x7fc07fc0u : 0x7fc00000u;  // 0 or NaN
            ox = oy = make_uint4(w, w, w, w);
        }
        *reinterpret_cast<uint4 *>(dst + h * dst_step + e0) = ox;
        *reinterpret_cast<uint4 *>(dst + h * dst_step + e1) = oy;
        if (!is_q && !is_v && c == 0) {
            const int64_t si = (static_cast<int64_t>(at.page) * a.Hkv + h) * a.page_size + at.off;
            if (a.weight) a.weight[si] = 0.f;
            if (a.pos) a.pos[si] = at.seq;
        }
    }
}

// Long blocks: tokens stream through shared memory by bulk copies, one CTA per
// SM.  A slot of the ring holds a token's queries, keys and values and has a
// warp that fills it (three copies, the token's cosines, sines and place in the
// cache) and that, when the heads have been turned in place, stores it (its
// queries in one copy, each cached row in one; values are never touched) and
// waits until the copies have read it.  Teams of warps turn the heads, each
// every n-th token; the number of slots is a multiple of theirs, so that a slot
// is always the same team's and neither side of a barrier is ever more than a
// round ahead.
//
// Bound: the heads' bytes, once the turning keeps up: with 16 KB tokens its
// chain of shared-memory reads, sums over lanes and stores takes a warp 1000
// cycles a round, so several tokens are turned at once.  16384 tokens of 32
// heads of 256, three axes, normalised (537 MB): 95.6 us, 5.6 TB/s, against
// 155 us in k_append_vec; four teams of two warps 108 us, two of four 136, a
// team for each slot 118 to 129.  float32 (1.07 GB): 169 us, 6.4 TB/s, against
// 222; its six slots do better with two teams of four than of six (182 us).
constexpr int AS_SLOTS = 12, AS_TURN = 12;  // slots and turning warps at most
constexpr int64_t STREAM_SMEM = 224 * 1024;
constexpr long long AS_WAIT = 4000000000ll, AS_DRAIN = 400000000ll;  // cycles after which a wait gives up
// Which calls: tokens of 7 KB and more, 24 and more of them per SM, else a
// token's fixed costs and the ring's start weigh more than the smoother stream.
// Measured, this against k_append_vec: 3040 tokens of 7 KB 10.2 against 9.1 us,
// 4864 14.7 against 15.2, 16384 44.8 against 52.3; 1824 of 16 KB 16.2 against
// 15.9, 3648 26.2 against 37.0; 16384 of 4 KB 31.9 against 32.4 but 4864 of them
// 11.3 against 7.8; 512 of 14 KB 7.5 against 5.3.
// float32 without a norm has little to compute and stays with k_append_vec:
// 16384 tokens of 28 KB 156 against 139 us.
constexpr int STREAM_TOKENS = 24, STREAM_LEAST = 7 * 1024;

struct StreamShared {
    uint64_t full[AS_SLOTS], done[AS_SLOTS];
    int live[AS_SLOTS], stored[AS_SLOTS];
    int abort;
};
static __device__ unsigned int g_err_append;
unsigned int read_error_append(bool clear) {
    unsigned int v = 0;
    cudaMemcpyFromSymbol(&v, g_err_append, sizeof v);
    if (clear && v) {
        const unsigned int z = 0;
        cudaMemcpyToSymbol(g_err_append, &z, sizeof z);
    }
    return v;
}

static __device__ __noinline__ bool stream_wait_long(StreamShared &sm, uint64_t *bar, uint32_t parity) {
    const long long t0 = clock64();
    while (*reinterpret_cast<volatile int *>(&sm.abort) == 0) {
        if (mbar_try_wait(bar, parity)) return true;
        if (clock64() - t0 > AS_WAIT) {
            atomicOr(&g_err_append, ERR_WAIT_TIMEOUT);
            *reinterpret_cast<volatile int *>(&sm.abort) = 1;
        }
    }
    return false;
}
// A whole warp's wait, with one answer for its lanes.
__device__ __forceinline__ bool stream_wait(StreamShared &sm, uint64_t *bar, uint32_t parity) {
    return __all_sync(FULL, mbar_try_wait(bar, parity) || stream_wait_long(sm, bar, parity));
}
// Test hook: a warp waits for the hook's word; if that runs out it gives up as after any time-out.
__device__ __forceinline__ bool stream_hold(StreamShared &sm, const AppendArgs &a) {
    if (a.hold == nullptr) return true;
    int seen = 1;
    if ((threadIdx.x & 31) == 0 && !hold_wait(a.hold, a.hold_cycles)) {
        atomicOr(&g_err_append, ERR_WAIT_TIMEOUT);
        *reinterpret_cast<volatile int *>(&sm.abort) = 1;
        seen = 0;
    }
    return __shfl_sync(FULL, seen, 0) != 0;
}
// A token that a time-out kept from being turned: NaN in its queries, and in its keys and values if it has a place.
template <typename E>
__device__ __forceinline__ void append_lost(const AppendArgs &a, int64_t tok, int lane) {
    const AppendToken at = append_token(a, append_raw(a, tok), lane == 0);
    const uint32_t w = !at.live ? 0u : sizeof(E) == 2 ? 0x7fc07fc0u : 0x7fc00000u;
    const uint4 x = make_uint4(w, w, w, w);
    const int vecs = a.d * static_cast<int>(sizeof(E)) / 16;
    uint4 *const q = reinterpret_cast<uint4 *>(static_cast<E *>(a.q_out) + tok * a.Hq * a.d);
    for (int i = lane; i < a.Hq * vecs; i += 32) q[i] = x;
    if (!at.live || at.page < 0) return;
    for (int h = 0; h < a.Hkv; ++h) {
        const int64_t row = at.page * a.page_stride + h * a.head_stride + at.off * a.slot_stride;
        for (int i = lane; i < vecs; i += 32) {
            reinterpret_cast<uint4 *>(reinterpret_cast<E *>(a.ck) + row)[i] = x;
            reinterpret_cast<uint4 *>(reinterpret_cast<E *>(a.cv) + row)[i] = x;
        }
        const int64_t si = (static_cast<int64_t>(at.page) * a.Hkv + h) * a.page_size + at.off;
        if (lane == 0 && a.weight) a.weight[si] = 0.f;
        if (lane == 0 && a.pos) a.pos[si] = at.seq;
    }
}
__device__ __forceinline__ void bulk_s2g(void *gdst, const void *ssrc, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(gdst), "r"(smem_addr(ssrc)),
                 "r"(bytes)
                 : "memory");
}

// The heads of one kind in a slot, norm and rotation in place.
template <typename E, bool INTER, bool NORM>
__device__ __forceinline__ void stream_turn(const AppendArgs &a, E *base, int heads, const E *nw, bool norm, bool mine,
                                            bool turned, int e0, int e1, int gt, int step, int lanes_log2,
                                            const float *cs, const float *sn) {
    constexpr int N = Vec<E>::N, H = N / 2;
    const float inv_d = 1.0f / a.d;
    const int rounds = (heads + step - 1) / step;
    E *p = base + (gt >> lanes_log2) * a.d;
    int h = gt >> lanes_log2;
#pragma unroll 2
    for (int r = 0; r < rounds; ++r, h += step, p += step * a.d) {
        const bool in = mine && h < heads;
        uint4 x = make_uint4(0, 0, 0, 0), y = x;
        if (in) {
            x = *reinterpret_cast<const uint4 *>(p + e0);
            y = *reinterpret_cast<const uint4 *>(p + e1);
        }
        uint64_t u[H], v[H];
        unpack<E>(x, u);
        unpack<E>(y, v);
        if (NORM && norm) {
            uint64_t s2 = mul2(u[0], u[0]);
#pragma unroll
            for (int k = 1; k < H; ++k) s2 = fma2(u[k], u[k], s2);
#pragma unroll
            for (int k = 0; k < H; ++k) s2 = fma2(v[k], v[k], s2);
            float ss = __uint_as_float(lo32(s2)) + __uint_as_float(hi32(s2));
            for (int d = 1 << lanes_log2 >> 1; d >= 1; d >>= 1) ss += __shfl_xor_sync(FULL, ss, d);
            const float f = rsqrtf(ss * inv_d + a.eps);
            const uint64_t ff = pair_of(f, f);
            uint64_t wx[H], wy[H];
            unpack<E>(*reinterpret_cast<const uint4 *>(nw + (mine ? e0 : 0)), wx);
            unpack<E>(*reinterpret_cast<const uint4 *>(nw + (mine ? e1 : 0)), wy);
#pragma unroll
            for (int k = 0; k < H; ++k) {
                u[k] = mul2(mul2(u[k], ff), wx[k]);
                v[k] = mul2(mul2(v[k], ff), wy[k]);
            }
        }
        if (turned) append_turn<INTER, H>(u, v, cs, sn);
        if (in && (turned || (NORM && norm))) {
            *reinterpret_cast<uint4 *>(p + e0) = pack<E>(u);
            *reinterpret_cast<uint4 *>(p + e1) = pack<E>(v);
        }
    }
}

template <typename E, bool INTER, bool NORM>
__global__ void __launch_bounds__((AS_SLOTS + AS_TURN) * 32, 1)
    k_append_stream(AppendArgs a, int lanes_log2, int slots, int teams, int team, int slot_bytes) {
    constexpr int N = Vec<E>::N;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ StreamShared sm;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = a.rot / 2, row = a.d * static_cast<int>(sizeof(E));
    const int q_bytes = a.Hq * row, kv_bytes = a.Hkv * row, data = q_bytes + 2 * kv_bytes;
    if (threadIdx.x == 0) {
        for (int i = 0; i < slots; ++i) {
            mbar_init(&sm.full[i], 2);
            mbar_init(&sm.done[i], team);
        }
        sm.abort = 0;
        fence_barrier_init();
    }
    pdl_wait();
    E *const norms = reinterpret_cast<E *>(ring + static_cast<size_t>(slots) * slot_bytes);  // the queries', the keys'
    if (NORM)
        for (int i = threadIdx.x; i < a.d; i += blockDim.x) {
            if (a.q_norm) norms[i] = static_cast<const E *>(a.q_norm)[i];
            if (a.k_norm) norms[a.d + i] = static_cast<const E *>(a.k_norm)[i];
        }
    __syncthreads();
    const int64_t G = gridDim.x;
    if (warp >= teams * team) {
        const int s = warp - teams * team;
        unsigned char *const slot = ring + static_cast<size_t>(s) * slot_bytes;
        float *const trig = reinterpret_cast<float *>(slot + data);
        uint64_t *const full = &sm.full[s], *const done = &sm.done[s];
        const uint64_t pol = l2_policy_evict_first();
        AppendToken was = {};
        int64_t was_tok = 0;
        uint32_t k = 0;
        auto store = [&]() {
            if (lane == 0) bulk_s2g(static_cast<char *>(a.q_out) + was_tok * q_bytes, slot, q_bytes);
            if (was.live && was.page >= 0)
                for (int r = lane; r < 2 * a.Hkv; r += 32) {
                    const bool v = r >= a.Hkv;
                    const int h = v ? r - a.Hkv : r;
                    bulk_s2g((v ? a.cv : a.ck) + (was.page * a.page_stride + h * a.head_stride +
                                                  was.off * a.slot_stride) * static_cast<int64_t>(sizeof(E)),
                             slot + q_bytes + r * row, row);
                }
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        };
        int64_t tok = blockIdx.x + s * G;
        bool ok = stream_hold(sm, a);
        for (; ok && tok < a.tokens; tok += slots * G, ++k) {
            const AppendToken at = append_token(a, append_raw(a, tok), lane == 0);
            if (k > 0) {
                ok = stream_wait(sm, done, (k - 1) & 1);
                if (!ok) break;
                store();
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
            }
            if (lane == 0) mbar_arrive_expect_tx(full, data);
            __syncwarp();
            if (lane < 3) {
                const char *src = lane == 0 ? a.q + tok * a.q_stride * static_cast<int64_t>(sizeof(E))
                                  : lane == 1 ? a.k + tok * a.k_stride * static_cast<int64_t>(sizeof(E))
                                              : a.v + tok * a.v_stride * static_cast<int64_t>(sizeof(E));
                bulk_g2s_hint(slot + (lane == 0 ? 0 : lane == 1 ? q_bytes : q_bytes + kv_bytes), src,
                              lane == 0 ? q_bytes : kv_bytes, full, pol);
            }
            for (int p = lane; p < half; p += 32) {
                int ax = a.pair_axis ? a.pair_axis[p] : 0;
                ax = ax < a.axes ? ax : a.axes - 1;
                const int id = a.pos_ids[ax * a.tokens + tok];
                const bool ok = id >= 0 && id < a.n_pos;
                const float *t = a.cos_sin + static_cast<int64_t>(ok ? id : 0) * a.rot + p;
                const float c = t[0], sn = t[half];
                trig[p] = ok ? c : NAN;
                trig[half + p] = sn;
            }
            const bool stored = at.live && at.page >= 0;
            if (lane == 0) {
                sm.live[s] = at.live;
                sm.stored[s] = stored;
            }
            if (stored)
                for (int h = lane; h < a.Hkv; h += 32) {
                    const int64_t si = (static_cast<int64_t>(at.page) * a.Hkv + h) * a.page_size + at.off;
                    if (a.weight) a.weight[si] = 0.f;
                    if (a.pos) a.pos[si] = at.seq;
                }
            __syncwarp();
            if (lane == 0) mbar_arrive(full);
            was = at;
            was_tok = tok;
        }
        if (k > 0) {
            ok = ok && stream_wait(sm, done, (k - 1) & 1);
            if (ok)
                store();
            else
                mbar_wait(full, (k - 1) & 1, AS_DRAIN);
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
            if (!ok) tok -= slots * G;  // the slot's token was not stored
        }
        for (; tok < a.tokens; tok += slots * G) append_lost<E>(a, tok, lane);  // only after a time-out
        return;
    }
    int s = warp / team;
    const int first = s, gt = (warp - s * team) * 32 + lane, step = (team * 32) >> lanes_log2;
    const int c = lane & ((1 << lanes_log2) - 1);
    const bool mine = c * 2 * N < a.d, turned = mine && c * 2 * N < a.rot;
    const int e0 = turned ? c * N : a.rot + (c - half / N) * N;
    const int e1 = e0 + (turned ? half : (a.d - a.rot) / 2);
    uint32_t parity = 0;
    for (int64_t tok = blockIdx.x + first * G; tok < a.tokens; tok += teams * G) {
        if (!stream_wait(sm, &sm.full[s], parity)) return;
        unsigned char *const slot = ring + static_cast<size_t>(s) * slot_bytes;
        E *const base = reinterpret_cast<E *>(slot);
        if (sm.stored[s]) {
            constexpr int W = INTER ? N / 2 : 4;
            auto pair = [&](int i) {
                return !INTER ? c * N + i : i < N / 2 ? c * N / 2 + i : (half + c * N) / 2 + i - N / 2;
            };
            const float *trig = reinterpret_cast<const float *>(slot + data);
            float cs[N], sn[N];
            if (turned) {
#pragma unroll
                for (int i = 0; i < N; i += W) {
                    cos_load<W>(trig + pair(i), cs + i);
                    cos_load<W>(trig + half + pair(i), sn + i);
                }
            }
            stream_turn<E, INTER, NORM>(a, base, a.Hq, norms, a.q_norm != nullptr, mine, turned, e0, e1, gt, step,
                                        lanes_log2, cs, sn);
            stream_turn<E, INTER, NORM>(a, base + a.Hq * a.d, a.Hkv, norms + a.d, a.k_norm != nullptr, mine, turned,
                                        e0, e1, gt, step, lanes_log2, cs, sn);
        } else {  // zeros past q_len, NaN for a token that has no place
            const uint32_t w = !sm.live[s] ? 0u : sizeof(E) == 2 ? 0x7fc07fc0u : 0x7fc00000u;
            for (int i = gt; i < q_bytes / 16; i += team * 32)
                reinterpret_cast<uint4 *>(slot)[i] = make_uint4(w, w, w, w);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.done[s]);
        s += teams;
        if (s >= slots) {
            s = first;
            parity ^= 1;
        }
    }
}

// ------------------------------------------------------------------- evict --
struct EvictArgs {
    char *ck, *cv;
    float *weight;
    int32_t *pos;
    int64_t num_pages, page_bytes, head_bytes, slot_bytes;  // strides in bytes
    int Hkv, page_size, row_bytes;
    const int32_t *table;
    int max_pages;
    const int32_t *kv_len, *seq_len;
    int budget, recent, sink;
    int32_t *kv_len_out;
    int *count;     // [B * Hkv]
    int2 *moves;    // [B * Hkv][max_moves]: (from, to) slots
    int64_t max_moves;
};

constexpr int EV_THREADS = 512;  // two CTAs per SM
constexpr int EV_WARPS = EV_THREADS / 32;

__device__ __forceinline__ int evict_page(const EvictArgs &a, int64_t b, int slot) {
    const int page = a.table[b * a.max_pages + slot / a.page_size];
    return page >= 0 && page < a.num_pages ? page : -1;
}

// The rank of a slot among its head's: larger stays.  Protected slots above
// every weight, NaN below, a slot without a page last.
__device__ __forceinline__ uint32_t evict_key(const EvictArgs &a, int64_t b, int h, int slot, int64_t newest) {
    const int page = evict_page(a, b, slot);
    if (page < 0) return 0u;
    const int64_t i = (static_cast<int64_t>(page) * a.Hkv + h) * a.page_size + slot % a.page_size;
    const int p = a.pos[i];
    if (p >= newest - a.recent || p < a.sink) return 0xffffffffu;
    const float w = a.weight[i];
    if (w != w) return 1u;
    return f2ord(w == 0.f ? 0.f : w);
}

__device__ __forceinline__ void evict_length(const EvictArgs &a, int64_t b) {
    const int64_t cap = static_cast<int64_t>(a.max_pages) * a.page_size;
    const int64_t n = a.kv_len[b] < cap ? a.kv_len[b] : cap;
    a.kv_len_out[b] = static_cast<int>(n < 0 ? 0 : (n < a.budget ? n : a.budget));
}

// Moves of a (request, head): a warp takes eight at a time (the first warp of
// `stride` warps has moves 8 first .. 8 first + 7), one lane per move for its
// places, and 16 bytes per lane of all of them in flight.
constexpr int EV_BATCH = 8;
__device__ __forceinline__ void evict_moves(const EvictArgs &a, int64_t b, int h, const int2 *m, int count, int first,
                                            int stride, int lane) {
    const int vecs = a.row_bytes / 16;
    for (int i = first * EV_BATCH; i < count; i += stride * EV_BATCH) {
        int64_t from = -1, to = 0;  // of lane's move, if it has one
        if (lane < EV_BATCH && i + lane < count) {
            const int2 mv = m[i + lane];
            const int ps = evict_page(a, b, mv.x), pd = evict_page(a, b, mv.y);
            if (ps >= 0 && pd >= 0) {
                const int os = mv.x % a.page_size, od = mv.y % a.page_size;
                from = ps * a.page_bytes + h * a.head_bytes + os * a.slot_bytes;
                to = pd * a.page_bytes + h * a.head_bytes + od * a.slot_bytes;
                const int64_t is = (static_cast<int64_t>(ps) * a.Hkv + h) * a.page_size + os;
                const int64_t id = (static_cast<int64_t>(pd) * a.Hkv + h) * a.page_size + od;
                a.weight[id] = a.weight[is];
                a.pos[id] = a.pos[is];
            }
        }
        int64_t f[EV_BATCH], t[EV_BATCH];
#pragma unroll
        for (int k = 0; k < EV_BATCH; ++k) {
            f[k] = __shfl_sync(FULL, from, k);
            t[k] = __shfl_sync(FULL, to, k);
        }
        for (int j = lane; j < 2 * vecs; j += 32) {
            char *base = j < vecs ? a.ck : a.cv;
            const int64_t o = static_cast<int64_t>(j < vecs ? j : j - vecs) * 16;
            uint4 x[EV_BATCH];
#pragma unroll
            for (int k = 0; k < EV_BATCH; ++k)
                if (f[k] >= 0) x[k] = *reinterpret_cast<const uint4 *>(base + f[k] + o);
#pragma unroll
            for (int k = 0; k < EV_BATCH; ++k)
                if (f[k] >= 0) *reinterpret_cast<uint4 *>(base + t[k] + o) = x[k];
        }
    }
}

// One CTA per (request, head): the budget-th largest key by four passes of a
// radix select (8 bits each), then the kept slots in slot order by ballots.
// The keys are made once and stay in shared memory (KEYS: the table's slots
// fit it, 50000 of them), so weights and positions are read once; otherwise
// every pass makes them again.  Bound: the latency of the passes and their
// barriers (8 heads of 32 requests with up to 8192 slots: 35 us for 16 MB;
// 2112 slots: 15 us).  Longer tables read weights, positions and pages in all
// seven passes: 4 requests of 8 heads from 65536 to 32768 slots 615 us with the
// moves (554 MB, 83 us).  Adding once per digit and warp (match) was slower, 43 us.
constexpr int EV_KEYS = 50000;
// Moves per head up to which the selecting CTA makes them itself.  GPU time of one launch and of two, in us: 64 moves,
// 128 heads 14.9 and 15.5, 16 heads 14.4 and 15.3; 256 moves 19.7 and 19.9, 18.9 and 16.5; 1024 moves 48.5 and 38.8,
// 34.5 and 18.2.  A launch less also saves the caller 3 us.
constexpr int EVICT_FEW = 128;
constexpr int EV_HISTS = 8;  // histograms, to spread the equal digits that weights have
// MOVE: the CTA carries its head's moves out itself, in one launch.
template <bool KEYS, bool MOVE>
__global__ void __launch_bounds__(EV_THREADS, 2) k_evict_select(EvictArgs a) {
    extern __shared__ uint32_t keys[];
    __shared__ int hists[EV_HISTS][256];
    __shared__ int s_warp[3][EV_WARPS];
    __shared__ uint32_t s_prefix;
    __shared__ int s_left;
    pdl_wait();
    const int64_t b = blockIdx.x / a.Hkv;
    const int h = static_cast<int>(blockIdx.x % a.Hkv);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t cap = static_cast<int64_t>(a.max_pages) * a.page_size;
    const int64_t n64 = a.kv_len[b] < cap ? a.kv_len[b] : cap;
    const int n = static_cast<int>(n64);
    if (MOVE && h == 0 && tid == 0) evict_length(a, b);
    if (n <= a.budget) {
        if (!MOVE && tid == 0) a.count[blockIdx.x] = 0;
        return;
    }
    const int64_t newest = a.seq_len ? a.seq_len[b] : n64;
    if (tid == 0) {
        s_prefix = 0;
        s_left = a.budget;
    }
    if (KEYS) {
#pragma unroll 8
        for (int s = tid; s < n; s += EV_THREADS) keys[s] = evict_key(a, b, h, s, newest);
    }
    auto key_of = [&](int s) { return KEYS ? keys[s] : evict_key(a, b, h, s, newest); };
    int *hist = hists[warp % EV_HISTS];
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < EV_HISTS * 256; i += EV_THREADS) (&hists[0][0])[i] = 0;
        __syncthreads();
        const uint32_t prefix = s_prefix;
        const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        for (int s = tid; s < n; s += EV_THREADS) {
            const uint32_t k = key_of(s);
            if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid < 256) {
            int sum = 0;
#pragma unroll
            for (int i = 0; i < EV_HISTS; ++i) sum += hists[i][tid];
            hists[0][tid] = sum;
        }
        __syncthreads();
        if (warp == 0) {
            // from the largest digit down: the one in which the s_left-th key lies
            int mine[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                mine[i] = hists[0][255 - (lane * 8 + i)];
                sum += mine[i];
            }
            int inc = sum;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(FULL, inc, d);
                if (lane >= d) inc += o;
            }
            int before = inc - sum;
            const int left = s_left;
            __syncwarp();
            if (before < left && left <= inc) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (before < left && left <= before + mine[i]) {
                        s_prefix = prefix | (static_cast<uint32_t>(255 - (lane * 8 + i)) << shift);
                        s_left = left - before;
                    }
                    before += mine[i];
                }
            }
        }
        __syncthreads();
    }
    const uint32_t T = s_prefix;
    const int ties = s_left;  // of the keys equal to T, the first `ties` slots stay
    // each warp takes a stretch of slots
    const int per = ((n + EV_WARPS - 1) / EV_WARPS + 31) / 32 * 32, s0 = warp * per, s1 = s0 + per < n ? s0 + per : n;
    int eq = 0;
    for (int s = s0; s < s1; s += 32) {
        const bool in = s + lane < n;
        eq += __popc(__ballot_sync(FULL, in && key_of(in ? s + lane : 0) == T));
    }
    if (lane == 0) s_warp[0][warp] = eq;
    __syncthreads();
    int eq_before = 0;
    for (int w = 0; w < warp; ++w) eq_before += s_warp[0][w];
    for (int pass = 0; pass < 2; ++pass) {
        int holes = 0, movers = 0, seen = eq_before;
        if (pass == 1)
            for (int w = 0; w < warp; ++w) {
                holes += s_warp[1][w];
                movers += s_warp[2][w];
            }
        for (int s = s0; s < s1; s += 32) {
            const int slot = s + lane;
            const bool in = slot < n;
            const uint32_t k = key_of(in ? slot : 0);
            const unsigned tie = __ballot_sync(FULL, in && k == T);
            const unsigned below = (1u << lane) - 1u;
            const bool kept = in && (k > T || (k == T && seen + __popc(tie & below) < ties));
            seen += __popc(tie);
            const bool hole = in && !kept && slot < a.budget, mover = kept && slot >= a.budget;
            const unsigned bh = __ballot_sync(FULL, hole), bm = __ballot_sync(FULL, mover);
            if (pass == 1) {
                int2 *m = a.moves + static_cast<int64_t>(blockIdx.x) * a.max_moves;
                if (hole) m[holes + __popc(bh & below)].y = slot;
                if (mover) m[movers + __popc(bm & below)].x = slot;
            }
            holes += __popc(bh);
            movers += __popc(bm);
        }
        if (pass == 0) {
            if (lane == 0) {
                s_warp[1][warp] = holes;
                s_warp[2][warp] = movers;
            }
            __syncthreads();
        } else if (warp == EV_WARPS - 1 && lane == 0) {
            if (MOVE)
                s_left = holes;
            else
                a.count[blockIdx.x] = holes;
        }
    }
    if (MOVE) {
        __syncthreads();
        evict_moves(a, b, h, a.moves + static_cast<int64_t>(blockIdx.x) * a.max_moves, s_left, warp, EV_WARPS, lane);
    }
}

// The moves as a kernel of their own.  32 requests cut from 8192 to 4096 keys
// (144 MB moved): 57 us, 4.6 TB/s read and written; three CTAs per SM instead
// of two took it from 64.
__global__ void __launch_bounds__(256, 3) k_evict_move(EvictArgs a) {
    pdl_wait();
    const int64_t b = blockIdx.x / a.Hkv;
    const int h = static_cast<int>(blockIdx.x % a.Hkv);
    if (blockIdx.y == 0 && h == 0 && threadIdx.x == 0) evict_length(a, b);
    evict_moves(a, b, h, a.moves + static_cast<int64_t>(blockIdx.x) * a.max_moves, a.count[blockIdx.x],
                blockIdx.y * 8 + (threadIdx.x >> 5), gridDim.y * 8, threadIdx.x & 31);
}

template <typename A>
static dflash2_status launch_pdl(void (*fn)(A), const A &a, dim3 grid, int threads, size_t smem, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, fn, a) != cudaSuccess) return DFLASH2_ERR_CUDA;
    return after_launch();
}

static dflash2_status launch_append_vec(AppendArgs &a, dflash2_dtype dt, bool inter, bool norm, int lanes_log2, int per,
                                        dim3 grid, cudaStream_t s) {
    using Fn = void (*)(AppendArgs, int, int);
    using H = unsigned short;
    static const Fn table[8] = {k_append_vec<H, false, false>,     k_append_vec<H, false, true>,
                                k_append_vec<H, true, false>,      k_append_vec<H, true, true>,
                                k_append_vec<float, false, false>, k_append_vec<float, false, true>,
                                k_append_vec<float, true, false>,  k_append_vec<float, true, true>};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const Fn fn = table[(dt == DFLASH2_F32 ? 4 : 0) + (inter ? 2 : 0) + (norm ? 1 : 0)];
    if (cudaLaunchKernelEx(&cfg, fn, a, lanes_log2, per) != cudaSuccess) return DFLASH2_ERR_CUDA;
    return after_launch();
}

static dflash2_status launch_append_stream(AppendArgs &a, dflash2_dtype dt, bool inter, bool norm, int lanes_log2,
                                           cudaStream_t s) {
    using Fn = void (*)(AppendArgs, int, int, int, int, int);
    using H = unsigned short;
    static const Fn table[8] = {k_append_stream<H, false, false>,     k_append_stream<H, false, true>,
                                k_append_stream<H, true, false>,      k_append_stream<H, true, true>,
                                nullptr,                              k_append_stream<float, false, true>,
                                nullptr,                              k_append_stream<float, true, true>};
    const Fn fn = table[(dt == DFLASH2_F32 ? 4 : 0) + (inter ? 2 : 0) + (norm ? 1 : 0)];
    scan_hold(&a.hold, &a.hold_cycles);
    // raises the shared-memory limit, once
    blocks_per_sm(reinterpret_cast<const void *>(fn), (AS_SLOTS + AS_TURN) * 32, STREAM_SMEM);
    const int row = a.d * esize(dt), slot_bytes = (a.Hq + 2 * a.Hkv) * row + (a.rot * 4 + 15) / 16 * 16;
    const int most = static_cast<int>((STREAM_SMEM - 2 * row) / slot_bytes), teams = most >= AS_SLOTS ? 6 : 2,
              team = most >= AS_SLOTS ? 2 : 4, slots = (most < AS_SLOTS ? most : AS_SLOTS) / teams * teams;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sm_count());
    cfg.blockDim = dim3((teams * team + slots) * 32, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(slots) * slot_bytes + 2 * row;
    cfg.stream = s;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, fn, a, lanes_log2, slots, teams, team, slot_bytes) != cudaSuccess)
        return DFLASH2_ERR_CUDA;
    return after_launch();
}

static int64_t evict_max_moves(int64_t capacity, int32_t budget) {
    const int64_t over = capacity > budget ? capacity - budget : 0;
    return over < budget ? over : budget;
}
static size_t evict_count_bytes(int64_t B, int32_t Hkv) {
    return (static_cast<size_t>(B) * Hkv * sizeof(int) + 255) / 256 * 256;
}

}  // namespace dfl

using namespace dfl;

static bool al4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// Memory that a device copy can reach.
static bool registered(const void *p) {
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
        cudaGetLastError();  // no device: nothing is the device's
        return false;
    }
    return at.type != cudaMemoryTypeUnregistered;
}

// A block of no tokens: the lengths stay what they were.  Lengths that are not the device's (the arguments' checks
// tried alone, on a machine without a GPU too) are not touched.
static dflash2_status append_no_tokens(const int32_t *kv_len, int64_t B, int32_t *kv_len_out, cudaStream_t s) {
    if (!kv_len_out) return DFLASH2_OK;
    if (!kv_len || !al4(kv_len) || !al4(kv_len_out)) return DFLASH2_ERR_INVALID_ARG;
    if (!registered(kv_len) || !registered(kv_len_out)) return DFLASH2_OK;
    const cudaError_t e = cudaMemcpyAsync(kv_len_out, kv_len, static_cast<size_t>(B) * sizeof(int32_t),
                                          cudaMemcpyDeviceToDevice, s);
    return e == cudaSuccess ? DFLASH2_OK : DFLASH2_ERR_CUDA;
}

extern "C" dflash2_status dflash2_rope_append(const dflash2_kv_cache *cache, const int32_t *page_table,
                                              int32_t max_pages, const int32_t *kv_len, const int32_t *q_len,
                                              const int32_t *seq_pos, const void *q, const void *k, const void *v,
                                              int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t B,
                                              int32_t T, int32_t Hq, const float *cos_sin, int64_t n_pos, int32_t rot,
                                              const int32_t *pos_ids, int32_t axes, const uint8_t *pair_axis,
                                              int32_t interleaved, const void *q_norm, const void *k_norm, float eps,
                                              void *q_out, int32_t *kv_len_out, dflash2_stream stream) {
    if (!kv_cache_ok(cache, page_table, max_pages, B) || B < 0 || T < 0 || Hq < 1 || rot < 2 || rot % 2 != 0 ||
        rot > cache->d || axes < 1 || n_pos < 1)
        return DFLASH2_ERR_INVALID_ARG;
    if (B == 0) return DFLASH2_OK;
    // tokens read what one of them would write
    if (kv_len_out && (kv_len_out == kv_len || kv_len_out == q_len || kv_len_out == seq_pos))
        return DFLASH2_ERR_INVALID_ARG;
    if (T == 0) return append_no_tokens(kv_len, B, kv_len_out, reinterpret_cast<cudaStream_t>(stream));
    const int e = esize(cache->dt);
    const int64_t d = cache->d;
    if (!q || !k || !v || !q_out || !kv_len || !cos_sin || !pos_ids || !aligned16(q) || !aligned16(k) ||
        !aligned16(v) || !aligned16(q_out) || !aligned16(q_norm) || !aligned16(k_norm) || !aligned16(cos_sin) ||
        !al4(kv_len) || !al4(q_len) || !al4(seq_pos) || !al4(pos_ids) || !al4(kv_len_out) || q_stride < Hq * d ||
        k_stride < cache->Hkv * d || v_stride < cache->Hkv * d || q_stride * e % 16 || k_stride * e % 16 ||
        v_stride * e % 16)
        return DFLASH2_ERR_INVALID_ARG;
    const int64_t heads = static_cast<int64_t>(Hq) + 2 * static_cast<int64_t>(cache->Hkv);
    if (d > 1024 || B * T >= (int64_t(1) << 31) || heads >= (int64_t(1) << 31)) return DFLASH2_ERR_UNSUPPORTED;
    // a token's queries would go where another's queries, or a key or value, are still to be read
    if ((q_out == q && q_stride != Hq * d && B * T > 1) || q_out == k || q_out == v) return DFLASH2_ERR_INVALID_ARG;
    AppendArgs a = {};
    a.ck = static_cast<char *>(cache->k);
    a.cv = static_cast<char *>(cache->v);
    a.weight = cache->weight;
    a.pos = cache->pos;
    a.num_pages = cache->num_pages;
    a.page_stride = cache->page_stride;
    a.head_stride = cache->head_stride;
    a.slot_stride = cache->slot_stride;
    a.Hkv = cache->Hkv;
    a.page_size = cache->page_size;
    a.d = cache->d;
    a.table = page_table;
    a.max_pages = max_pages;
    a.kv_len = kv_len;
    a.q_len = q_len;
    a.seq_pos = seq_pos;
    a.q = static_cast<const char *>(q);
    a.k = static_cast<const char *>(k);
    a.v = static_cast<const char *>(v);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.tokens = B * T;
    a.T = T;
    a.Hq = Hq;
    a.cos_sin = cos_sin;
    a.n_pos = n_pos;
    a.rot = rot;
    a.pos_ids = pos_ids;
    a.axes = axes;
    a.pair_axis = axes > 1 ? pair_axis : nullptr;
    a.q_norm = q_norm;
    a.k_norm = k_norm;
    a.eps = eps;
    a.q_out = q_out;
    a.kv_len_out = kv_len_out;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int two = 32 / e;  // entries of two vectors
    // in vectors: places within a token are counted in 31 bits
    if (rot % two == 0 && d % two == 0 && d / two <= 32 && heads * d < (int64_t(1) << 31)) {
        int lanes_log2 = 0;
        while ((1 << lanes_log2) * two < d) ++lanes_log2;
        const bool norm = q_norm || k_norm;
        const int64_t token_bytes = heads * d * e;
        if ((norm || cache->dt == DFLASH2_BF16) && a.tokens >= static_cast<int64_t>(sm_count()) * STREAM_TOKENS &&
            token_bytes >= STREAM_LEAST && token_bytes <= STREAM_SMEM / 4 - 4096)
            return launch_append_stream(a, cache->dt, interleaved != 0, norm, lanes_log2, s);
        // Many tokens: a thread takes four heads, so that a token's cosines are read by a quarter of the threads;
        // few: one, so that there are enough threads (192 per SM).
        auto units = [&](int64_t per) { return (Hq + per - 1) / per + 2 * ((cache->Hkv + per - 1) / per); };
        const int per = (a.tokens * units(APPEND_BATCH) << lanes_log2) >= static_cast<int64_t>(sm_count()) * 192
                            ? APPEND_BATCH : 1;
        const int64_t threads = a.tokens * units(per) << lanes_log2;
        if (a.tokens * units(per) < (int64_t(1) << 32) - 256 && (threads + 255) / 256 < (int64_t(1) << 31)) {
            const dim3 vgrid(static_cast<unsigned>((threads + 255) / 256));
            return launch_append_vec(a, cache->dt, interleaved != 0, norm, lanes_log2, per, vgrid, s);
        }
    }
    const int64_t units = a.tokens * heads;
    const int64_t blocks = (units + 7) / 8, most = static_cast<int64_t>(sm_count()) * 64;
    const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most));
    if (cache->dt == DFLASH2_BF16)
        return interleaved ? launch_pdl(k_append_any<unsigned short, true>, a, grid, 256, 0, s)
                           : launch_pdl(k_append_any<unsigned short, false>, a, grid, 256, 0, s);
    return interleaved ? launch_pdl(k_append_any<float, true>, a, grid, 256, 0, s)
                       : launch_pdl(k_append_any<float, false>, a, grid, 256, 0, s);
}

extern "C" size_t dflash2_kv_evict_workspace_bytes(int64_t B, int32_t Hkv, int64_t capacity, int32_t budget) {
    if (B < 0 || Hkv < 1 || capacity < 0 || budget < 1) return 0;
    return WS_ZERO_BYTES + evict_count_bytes(B, Hkv) +
           static_cast<size_t>(B) * Hkv * evict_max_moves(capacity, budget) * sizeof(int2);
}

extern "C" dflash2_status dflash2_kv_evict(const dflash2_kv_cache *cache, const int32_t *page_table,
                                           int32_t max_pages, const int32_t *kv_len, const int32_t *seq_len, int64_t B,
                                           int32_t budget, int32_t recent, int32_t sink, int32_t *kv_len_out, void *ws,
                                           size_t ws_bytes, dflash2_stream stream) {
    if (!kv_cache_ok(cache, page_table, max_pages, B) || !cache->weight || !cache->pos || B < 0 || budget < 1 ||
        recent < 0 || sink < 0)
        return DFLASH2_ERR_INVALID_ARG;
    if (B == 0) return DFLASH2_OK;
    if (!kv_len || !kv_len_out || !ws || !aligned16(ws) || !al4(kv_len) || !al4(kv_len_out) || !al4(seq_len))
        return DFLASH2_ERR_INVALID_ARG;
    const int64_t cap = static_cast<int64_t>(max_pages) * cache->page_size;
    if (cap >= (int64_t(1) << 31) - 2048 || B * cache->Hkv >= (int64_t(1) << 31)) return DFLASH2_ERR_UNSUPPORTED;
    if (ws_bytes < dflash2_kv_evict_workspace_bytes(B, cache->Hkv, cap, budget)) return DFLASH2_ERR_WORKSPACE;
    const int e = esize(cache->dt);
    EvictArgs a = {};
    a.ck = static_cast<char *>(cache->k);
    a.cv = static_cast<char *>(cache->v);
    a.weight = cache->weight;
    a.pos = cache->pos;
    a.num_pages = cache->num_pages;
    a.page_bytes = cache->page_stride * e;
    a.head_bytes = cache->head_stride * e;
    a.slot_bytes = cache->slot_stride * e;
    a.Hkv = cache->Hkv;
    a.page_size = cache->page_size;
    a.row_bytes = cache->d * e;
    a.table = page_table;
    a.max_pages = max_pages;
    a.kv_len = kv_len;
    a.seq_len = seq_len;
    a.budget = budget;
    a.recent = recent;
    a.sink = sink;
    a.kv_len_out = kv_len_out;
    char *const scratch = static_cast<char *>(ws) + WS_ZERO_BYTES;
    a.count = reinterpret_cast<int *>(scratch);
    a.moves = reinterpret_cast<int2 *>(scratch + evict_count_bytes(B, cache->Hkv));
    a.max_moves = evict_max_moves(cap, budget);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int64_t heads = B * cache->Hkv;
    const dim3 sgrid(static_cast<unsigned>(heads));
    // One launch where a head has few moves to make; a launch of its own spreads many over the GPU.  Lengths in one
    // array need the second launch: heads read what one would write.
    const bool one = a.max_moves <= EVICT_FEW && kv_len_out != kv_len && kv_len_out != seq_len;
    auto select = [&](auto *fn, size_t most, size_t bytes) {
        blocks_per_sm(reinterpret_cast<const void *>(fn), EV_THREADS, most);  // raises the shared-memory limit, once
        return launch_pdl(fn, a, sgrid, EV_THREADS, bytes, s);
    };
    const size_t keys = cap <= EV_KEYS ? static_cast<size_t>(cap) * 4 : 0;
    const dflash2_status st = keys ? (one ? select(&k_evict_select<true, true>, EV_KEYS * 4, keys)
                                          : select(&k_evict_select<true, false>, EV_KEYS * 4, keys))
                                   : (one ? select(&k_evict_select<false, true>, 0, 0)
                                          : select(&k_evict_select<false, false>, 0, 0));
    if (st != DFLASH2_OK || one) return st;
    int64_t x = (a.max_moves + 8 * EV_BATCH - 1) / (8 * EV_BATCH);
    const int64_t want = (static_cast<int64_t>(sm_count()) * 16 + heads - 1) / heads;
    if (x > want) x = want;
    if (x < 1) x = 1;
    return launch_pdl(k_evict_move, a, dim3(static_cast<unsigned>(heads), static_cast<unsigned>(x)), 256, 0, s);
}
