// sample.cu -- dflash2_sample: one token per row of logits from a given uniform.
//
// temperature -> top_k -> top_p -> min_p, then the inverse of the cumulative
// distribution over the kept tokens, best first (larger logit, then lower id).
// FreeToken PR 857 "Speed" gives the filters' values (temperature 1.0, top_p
// 0.95, top_k 20).
//
// Every filter keeps a prefix of one ranking, so a filter is a mass: the mass Z
// of the shortest of the prefixes is what u is multiplied with, and the token
// is where the running mass passes u Z.  Three questions of one kind remain, up
// to which rank (top_k) or to which mass (top_p, the draw) the ranking runs, and
// each is answered by a histogram and one bin's elements:
//
//   A cluster of CTAs holds a row in shared memory, read once.  One pass adds
//   each token's mass to one of 2048 bins, linear in log2 of the mass from the
//   best token down to 2^-45 of it (lighter ones are no whole unit).  The first
//   CTA adds the cluster's bins and finds the bin in question; its elements are
//   collected there, sorted and summed.  A bin with more than S_LIST elements is
//   split by the bits of its keys until few are left or all are one value.
//
// A bf16 row has few values: there a bin is one value, its mass the tokens times
// the value's, and the questions are answered without a list (by_values).  The
// 6144 bins reach down from the largest value past some 47 binades; the values
// between -2^-8 and 2^-8, of which there are 30000 and hardly ever many tokens,
// and those past the bins have a sum each, and a question that ends among them
// goes the general way.
//
// Masses are whole numbers of 2^-shift of the best token's, exp in two floats
// (relative error about 2^-37, below), so sums do not depend on their order:
// a row's token is the same alone, in a batch and over any cluster.  In f32 they
// would be off by 2^-24, and one draw in a few hundred of a flat row of 150000
// tokens would be another token than in 64 bits.
//
// Up to some 40 to 80 rows: bound by latency, a chain of passes, cluster barriers and
// one thread's 64-bit arithmetic.  One row of 151936 takes 7 us greedy, 13 with top_k
// 20, 23 with top_p in bf16 and 40 in f32; 64 rows in bf16 with top_p 38 us (bins and
// lists took 65).  More rows than fit the SMs' shared memory go in waves, each of which
// waits through the chain while little is read: 512 rows of 262144 with top_k and min_p
// 261 us, 1.0 TB/s.  At 64 registers a thread (two CTAs to an SM) 168 bytes spill in
// f32 and 60 in bf16.
#include "common.cuh"
#include "host.hpp"
#include "tc.cuh"

namespace dfl {

typedef unsigned long long u64;

constexpr int S_THREADS = 512;
constexpr int S_WARPS = S_THREADS / 32;
constexpr int S_BINS = 2048;
constexpr int S_PER = S_BINS / S_THREADS;  // bins of a thread in a scan
constexpr int S_LIST = 1024;
constexpr int S_CLUSTER = 8;
constexpr float S_MAGIC = 12582912.0f;  // 1.5 * 2^23: adding it rounds to a whole number

struct SampleArgs {
    const void *logits;
    int64_t V, ld;
    const dflash2_sampling *params;
    const float *min_p;
    int64_t rows_per_param;
    const float *u;
    int32_t *token;
    float *prob;
    int shift;
    int slice;     // entries of a CTA, a multiple of 8
    int resident;  // whether they fit its shared memory
};

struct alignas(128) SampleSmem {
    uint32_t cnt[S_BINS], lo[S_BINS], hi[S_BINS];  // the first CTA's, once added: what lies above the bin
    u64 list[S_LIST];
    float2 root[32];  // 2^(-j/32), and what the float lacks
    double inv_t, t_log;
    float ch, cl;
    u64 sum[S_WARPS + 1], sum2[S_WARPS + 1];
    // written by the cluster's CTAs, each in its own place
    float in_max[S_CLUSTER], in_min[S_CLUSTER];
    int in_bad[S_CLUSTER];
    u64 in_word[S_CLUSTER], in_far[S_CLUSTER], in_near[S_CLUSTER];
    // written by the first CTA in all of them
    u64 go_a, go_b;
    uint32_t go_key, go_n;
    // the first CTA's alone
    uint32_t list_n[4];  // one for a call of find in turn: a CTA may still read the last call's; and the short list's
    uint32_t floor_bin[2];
    int go_i[3];
    u64 hit_above_n, hit_above_m;
    uint32_t hit_bin;
};

template <class T>
__device__ __forceinline__ T *peer(T *local, int rank) {
    u64 out;
    asm("mapa.u64 %0, %1, %2;" : "=l"(out) : "l"(local), "r"(rank));
    return reinterpret_cast<T *>(out);
}

// exp(-(m - z) / T) in units of 2^-shift.
//
// t = (m - z) log2(e) / T in two floats; t = n/32 + r with |r| <= 1/64; 2^-r - 1
// by its series in y = -r ln 2 (|y| < 0.011, five terms), the first term in two
// floats; times a stored root.  Errors: t 2^-42 (two floats of up to 47), the
// series 2^-38 where its square term is rounded, the last sum 2^-45.
struct Mass {
    float m, ch, cl;
    int shift;
    const float2 *root;

    template <bool BF16>
    __device__ __forceinline__ float t_of(float z) const { return __fmul_rn(m - z, ch); }

    template <bool BF16>
    __device__ __forceinline__ u64 of(float z) const {
        const float d = m - z;
        const float th = __fmul_rn(d, ch);  // the compiler must not fuse what the next lines take apart
        if (!(th < 47.0f)) return 0;
        float tl = fmaf(d, ch, -th);
        tl = fmaf(d, cl, tl);
        // what d lacks of m - z (of bf16 too, where z's last bit is below 2^-24 of m)
        const float b = d - m;
        tl = fmaf((m - (d - b)) + (-z - b), ch, tl);
        const float f = fmaf(th, 32.0f, S_MAGIC);
        const int n = __float_as_int(f) - __float_as_int(S_MAGIC);
        const float r = fmaf(f - S_MAGIC, -1.0f / 32.0f, th);
        const float s = r + tl, se = (r - s) + tl;
        constexpr float L = 0.693147180559945f, LL = static_cast<float>(0.693147180559945309 - static_cast<double>(L));
        const float y = __fmul_rn(s, -L);
        float e = fmaf(s, -L, -y);
        e = fmaf(s, -LL, e);
        e = fmaf(se, -L, e);
        float q = fmaf(y, 1.0f / 120.0f, 1.0f / 24.0f);
        q = fmaf(q, y, 1.0f / 6.0f);
        q = fmaf(q, y, 0.5f);
        e = fmaf(q, y * y, e);  // 2^-r - 1 = y + e
        const float2 w = root[n & 31];
        const float a = __fmul_rn(w.x, y);
        float ae = fmaf(w.x, y, -a);
        ae = fmaf(w.x, e, ae);
        ae += fmaf(w.y, y, w.y);
        const float s1 = __fadd_rn(w.x, a);
        ae += __fadd_rn(__fadd_rn(w.x, -s1), a);  // up to 2^-14: the series' square
        const float S = __fadd_rn(s1, ae), Se = __fadd_rn(ae, -__fadd_rn(S, -s1));
        const float up = __int_as_float((127 + 22 - (n >> 5)) << 23);
        const float f1 = fmaf(S, up, S_MAGIC), n1 = f1 - S_MAGIC;
        const float rest = fmaf(S, up, -n1);
        const float f2 = fmaf(fmaf(Se, up, rest), __int_as_float((127 + shift - 22) << 23), S_MAGIC);
        const int hi = __float_as_int(f1) - __float_as_int(S_MAGIC), lo = __float_as_int(f2) - __float_as_int(S_MAGIC);
        return static_cast<u64>(static_cast<long long>(hi) * (1 << (shift - 22)) + lo);
    }
    // Its value, rounded once.
    template <bool BF16>
    __device__ double exactly(float z, double inv_t) const { return exp((static_cast<double>(z) - m) * inv_t); }
};

template <class T>
__device__ __forceinline__ T warp_scan(T v, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T o = __shfl_up_sync(FULL, v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// Where a running mass has to come to: share of Z, rounded up (at least 1), or just past it (at most Z).
__device__ __forceinline__ u64 goal_reach(float share, u64 Z) {
    const u64 g = __double2ull_ru(static_cast<double>(share) * __ull2double_rn(Z));
    return g < 1 ? 1 : g;
}
__device__ __forceinline__ u64 goal_pass(float u, u64 Z) {
    const u64 g = __double2ull_rd(static_cast<double>(fminf(fmaxf(u, 0.0f), 1.0f)) * __ull2double_rn(Z)) + 1;
    return g < Z ? g : Z;
}

template <bool BF16>
struct Sampler {
    static constexpr int VEC = BF16 ? 8 : 4;
    SampleSmem *sm;
    const void *data;  // the slice, in shared memory or where it lies
    int n;             // its entries
    int64_t id0;
    int rank, C, lane, warp;
    Mass mass;
    float t_cap, t_scale;  // tokens of the ranking's part in question: t < t_cap; their bins
    float z_floor;         // and z >= z_floor
    int calls;             // of find
    bool dirty;            // the bins no longer hold the whole ranking

    __device__ __forceinline__ float entry(int i) const {
        return BF16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(data)[i]) << 16)
                    : static_cast<const float *>(data)[i];
    }

    __device__ __forceinline__ uint4 vector(int i) const {
        return *reinterpret_cast<const uint4 *>(static_cast<const char *>(data) + static_cast<size_t>(i) * (16 / VEC));
    }
    __device__ __forceinline__ static void split(const uint4 &v, float (&z)[VEC]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (BF16) z[2 * j] = bf16lo(w[j]), z[(2 * j + 1) % VEC] = bf16hi(w[j]);
            else z[j] = __uint_as_float(w[j]);
        }
    }
    __device__ __forceinline__ void rest(int i, float (&z)[VEC]) const {  // the last, cut vector
#pragma unroll
        for (int j = 0; j < VEC; ++j) z[j] = i + j < n ? entry(i + j) : NEG_INF;
    }

    // f(z, place) for every entry of the slice, by vectors dealt to the threads in turn.
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        for (int i = threadIdx.x * VEC; i < n; i += S_THREADS * VEC) {
            float z[VEC];
            if (i + VEC <= n) split(vector(i), z);
            else rest(i, z);
#pragma unroll
            for (int j = 0; j < VEC; ++j) f(z[j], i + j);
        }
    }
    // The same for those with lo <= z <= hi: few.
    template <class F>
    __device__ __forceinline__ void each_within(float lo, float hi, F f) const {
        for (int i = threadIdx.x * VEC; i < n; i += S_THREADS * VEC) {
            float z[VEC];
            if (i + VEC <= n) split(vector(i), z);
            else rest(i, z);
            bool any = false;
#pragma unroll
            for (int j = 0; j < VEC; ++j) any |= z[j] >= lo && z[j] <= hi;
            if (any)
#pragma unroll 1
                for (int j = 0; j < VEC; ++j) {
                    float x = z[0];
#pragma unroll
                    for (int k = 1; k < VEC; ++k) x = k == j ? z[k] : x;
                    if (x >= lo && x <= hi) f(x, i + j);
                }
        }
    }
    // This thread's largest entry; NaN if it has one.  least: of f32 rows, the smallest above -infinity.
    __device__ __forceinline__ float largest(float &least) const {
        float m = NEG_INF;
        least = __builtin_huge_valf();
        if (BF16) {
            uint32_t m2 = 0xff80ff80u;  // two -infinities
            for (int i = threadIdx.x * VEC; i < n; i += S_THREADS * VEC) {
                if (i + VEC <= n) {
                    const uint4 v = vector(i);
                    m2 = bmax2_nan(m2, bmax2_nan(bmax2_nan(v.x, v.y), bmax2_nan(v.z, v.w)));
                } else {
                    for (int j = i; j < n; ++j) m = fmax_nan(m, entry(j));
                }
            }
            m = fmax_nan(m, fmax_nan(bf16lo(m2), bf16hi(m2)));
        } else {
            each([&](float z, int) {
                m = fmax_nan(m, z);
                least = fminf(least, z == NEG_INF ? least : z);
            });
        }
        return m;
    }
    // Bounds of z where t lies in [lo, hi], a little further out than rounding goes.
    __device__ __forceinline__ float z_below(float t) const { return __fsub_rd(mass.m, t * 1.00001f / mass.ch); }
    __device__ __forceinline__ float z_above(float t) const { return __fsub_ru(mass.m, t * 0.99999f / mass.ch); }

    __device__ __forceinline__ int bin_of(float t) const { return min(static_cast<int>(t * t_scale), S_BINS - 1); }
    __device__ __forceinline__ bool inside(float z, float t) const { return t < t_cap && z >= z_floor; }
    __device__ __forceinline__ static uint32_t key_of(float z) { return f2ord(z + 0.0f); }  // one zero

    __device__ __forceinline__ void add(int b, u64 q, bool count) {
        if (count) atomicAdd(&sm->cnt[b], 1u);
        const uint32_t ql = static_cast<uint32_t>(q);
        uint32_t up = static_cast<uint32_t>(q >> 32);
        const uint32_t old = atomicAdd(&sm->lo[b], ql);
        up += old + ql < old;
        if (up) atomicAdd(&sm->hi[b], up);
    }

    __device__ void clear(bool counts) {
        for (int i = threadIdx.x; i < S_BINS; i += S_THREADS) {
            sm->lo[i] = sm->hi[i] = 0;
            if (counts) sm->cnt[i] = 0;
        }
        __syncthreads();
    }

    // A value of each thread added up over the CTA.
    __device__ u64 block_sum(u64 v) {
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(FULL, v, d);
        __syncthreads();
        if (lane == 0) sm->sum[warp] = v;
        __syncthreads();
        u64 s = 0;
#pragma unroll
        for (int i = 0; i < S_WARPS; ++i) s += sm->sum[i];
        return s;
    }

    // First CTA, all threads, behind a cluster barrier: bin by bin, what the cluster's CTAs counted becomes what lies
    // above the bin.  Returns the totals.
    __device__ void gather_bins(u64 *total_n, u64 *total_m) {
        uint32_t c[S_PER];
        u64 w[S_PER];
#pragma unroll
        for (int j = 0; j < S_PER; ++j) c[j] = 0, w[j] = 0;
        const int b0 = threadIdx.x * S_PER;
        for (int q = 0; q < C; ++q) {
            const uint4 vc = *reinterpret_cast<const uint4 *>(peer(sm->cnt, q) + b0);
            const uint4 vl = *reinterpret_cast<const uint4 *>(peer(sm->lo, q) + b0);
            const uint4 vh = *reinterpret_cast<const uint4 *>(peer(sm->hi, q) + b0);
            c[0] += vc.x, c[1] += vc.y, c[2] += vc.z, c[3] += vc.w;
            w[0] += (static_cast<u64>(vh.x) << 32) + vl.x, w[1] += (static_cast<u64>(vh.y) << 32) + vl.y;
            w[2] += (static_cast<u64>(vh.z) << 32) + vl.z, w[3] += (static_cast<u64>(vh.w) << 32) + vl.w;
        }
        u64 tn = 0, tm = 0;
#pragma unroll
        for (int j = 0; j < S_PER; ++j) tn += c[j], tm += w[j];
        const u64 in = warp_scan(tn, lane), im = warp_scan(tm, lane);
        if (lane == 31) sm->sum[warp] = in, sm->sum2[warp] = im;
        __syncthreads();
        u64 an = in - tn, am = im - tm, N = 0, M = 0;
#pragma unroll
        for (int i = 0; i < S_WARPS; ++i) {
            const u64 x = sm->sum[i], y = sm->sum2[i];
            if (i < warp) an += x, am += y;
            N += x, M += y;
        }
#pragma unroll
        for (int j = 0; j < S_PER; ++j) {
            sm->cnt[b0 + j] = static_cast<uint32_t>(an);
            sm->lo[b0 + j] = static_cast<uint32_t>(am);
            sm->hi[b0 + j] = static_cast<uint32_t>(am >> 32);
            an += c[j], am += w[j];
        }
        *total_n = N, *total_m = M;
        __syncthreads();
    }

    // First CTA: the bin where the count or the mass reaches `target`, given the totals.  base_*: what lies above all
    // bins.
    __device__ void find_bin(bool by_mass, u64 target, u64 base_n, u64 base_m, u64 total_n, u64 total_m) {
        const int b0 = threadIdx.x * S_PER;
#pragma unroll
        for (int j = 0; j < S_PER; ++j) {
            const int b = b0 + j;
            const u64 n0 = sm->cnt[b], m0 = (static_cast<u64>(sm->hi[b]) << 32) | sm->lo[b];
            const u64 n1 = b + 1 < S_BINS ? sm->cnt[b + 1] : total_n;
            const u64 m1 = b + 1 < S_BINS ? (static_cast<u64>(sm->hi[b + 1]) << 32) | sm->lo[b + 1] : total_m;
            if (by_mass ? base_m + m0 < target && base_m + m1 >= target : base_n + n0 < target && base_n + n1 >= target) {
                sm->hit_bin = b;
                sm->hit_above_n = base_n + n0;
                sm->hit_above_m = base_m + m0;
            }
        }
        __syncthreads();
    }

    // First CTA: the first cnt of the list, descending (bitonic), behind a barrier.
    __device__ void sort_list(int cnt) {
        if (cnt <= 256) {  // keys are distinct: a key's place is the number of larger ones
            const u64 mine = threadIdx.x < cnt ? sm->list[threadIdx.x] : 0;
            int place = 0;
            if (threadIdx.x < ((cnt + 31) & ~31))
#pragma unroll 8
                for (int i = 0; i < cnt; ++i) place += sm->list[i] > mine;
            __syncthreads();
            if (threadIdx.x < cnt) sm->list[place] = mine;
            __syncthreads();
            return;
        }
        int pow = 512;
        while (pow < cnt) pow *= 2;
        for (int i = threadIdx.x; i < pow; i += S_THREADS)
            if (i >= cnt) sm->list[i] = 0;
        __syncthreads();
        for (int k = 2; k <= pow; k *= 2)
            for (int j = k / 2; j > 0; j /= 2) {
                for (int i = threadIdx.x; i < pow / 2; i += S_THREADS) {
                    const int a = 2 * j * (i / j) + i % j, b = a + j;
                    const u64 x = sm->list[a], y = sm->list[b];
                    if ((x < y) == ((a & k) == 0)) sm->list[a] = y, sm->list[b] = x;
                }
                __syncthreads();
            }
    }

    // Where the ranking's running count or mass reaches `target` (known to the first CTA; within the totals).  In the
    // first CTA: the running mass there (with the token), its key, and its id or, for a key with many ties, -1 and
    // which of them it is.
    struct Found {
        u64 through;
        uint32_t key;
        int64_t id;
        u64 tie;
    };

    // All CTAs.  want_id: the id is asked for.
    __device__ Found find(bool by_mass, u64 target, u64 total_n, u64 total_m, bool want_id) {
        Found r = {0, 0, -1, 0};
        int bin = 0;
        if (rank == 0) {
            find_bin(by_mass, target, 0, 0, total_n, total_m);
            if (threadIdx.x == 0) sm->list_n[(calls + 1) % 3] = 0;
            if (threadIdx.x < C) peer(&sm->go_n, threadIdx.x)[0] = sm->hit_bin;
        }
        cluster_sync();
        bin = static_cast<int>(sm->go_n);
        // the bin's elements, into the first CTA's list
        uint32_t *my_n = &sm->list_n[calls % 3], *list_n = peer(my_n, 0);
        ++calls;
        u64 *list = peer(sm->list, 0);
        uint32_t k_min = 0xffffffffu, k_max = 0;
        const float z_lo = z_below(static_cast<float>(bin + 1) / t_scale), z_hi = bin == 0 ? mass.m : z_above(static_cast<float>(bin) / t_scale);
        each_within(bin == S_BINS - 1 ? fminf(z_lo, z_below(t_cap)) : z_lo, z_hi, [&](float z, int i) {
            const float t = mass.template t_of<BF16>(z);
            if (inside(z, t) && bin_of(t) == bin) {
                const uint32_t k = key_of(z);
                k_min = min(k_min, k), k_max = max(k_max, k);
                const uint32_t at = atomicAdd(list_n, 1u);
                if (at < S_LIST) list[at] = (static_cast<u64>(k) << 32) | static_cast<uint32_t>(~static_cast<uint32_t>(id0 + i));
            }
        });
        cluster_sync();
        const uint32_t many = *list_n;
        u64 above_n = 0, above_m = 0;
        if (rank == 0) above_n = sm->hit_above_n, above_m = sm->hit_above_m;
        if (many > S_LIST) {
            // a wide bin: split it by its keys
            dirty = true;
            k_min = __reduce_min_sync(FULL, k_min), k_max = __reduce_max_sync(FULL, k_max);
            if (lane == 0) sm->sum[warp] = (static_cast<u64>(k_max) << 32) | k_min;
            __syncthreads();
            for (int i = 0; i < S_WARPS; ++i)
                k_min = min(k_min, static_cast<uint32_t>(sm->sum[i])), k_max = max(k_max, static_cast<uint32_t>(sm->sum[i] >> 32));
            if (threadIdx.x < C) peer(&sm->in_word[rank], threadIdx.x)[0] = (static_cast<u64>(k_max) << 32) | k_min;
            cluster_sync();
            for (int q = 0; q < C; ++q)
                k_min = min(k_min, static_cast<uint32_t>(sm->in_word[q])),
                k_max = max(k_max, static_cast<uint32_t>(sm->in_word[q] >> 32));
            for (;;) {
                int s = 0;
                while (((k_max - k_min) >> s) >= S_BINS) ++s;
                clear(true);
                each([&](float z, int) {
                    const float t = mass.template t_of<BF16>(z);
                    const uint32_t k = key_of(z);
                    if (inside(z, t) && bin_of(t) == bin && k >= k_min && k <= k_max)
                        add((k_max - k) >> s, mass.template of<BF16>(z), true);
                });
                cluster_sync();
                if (rank == 0) {
                    u64 tn, tm;
                    gather_bins(&tn, &tm);
                    find_bin(by_mass, target, above_n, above_m, tn, tm);
                    above_n = sm->hit_above_n, above_m = sm->hit_above_m;
                    const uint32_t b = sm->hit_bin;
                    const u64 next = b + 1 < S_BINS ? sm->cnt[b + 1] : tn;
                    if (threadIdx.x == 0) *my_n = 0;
                    if (threadIdx.x < C) {
                        peer(&sm->go_key, threadIdx.x)[0] = b;
                        peer(&sm->go_n, threadIdx.x)[0] = static_cast<uint32_t>(next - sm->cnt[b]);
                    }
                }
                cluster_sync();
                const uint32_t top = k_max - (sm->go_key << s), low = top - ((1u << s) - 1);
                k_min = max(k_min, low > top ? 0u : low), k_max = top;
                if (sm->go_n <= S_LIST || k_min == k_max) break;
            }
            const uint32_t left = sm->go_n;
            if (left > S_LIST) {  // one value
                if (rank == 0) {
                    const u64 q = mass.template of<BF16>(ord2f(k_min));
                    r.key = k_min;
                    r.tie = by_mass ? (target - above_m + q - 1) / q : target - above_n;
                    r.through = above_m + r.tie * q;
                }
                if (want_id) r.id = place_of(k_min, r.tie);
                cluster_sync();
                return r;
            }
            each([&](float z, int i) {
                const float t = mass.template t_of<BF16>(z);
                const uint32_t k = key_of(z);
                if (inside(z, t) && bin_of(t) == bin && k >= k_min && k <= k_max)
                    list[atomicAdd(list_n, 1u)] = (static_cast<u64>(k) << 32) | static_cast<uint32_t>(~static_cast<uint32_t>(id0 + i));
            });
            cluster_sync();
        }
        if (rank == 0) {
            const int cnt = static_cast<int>(*my_n);
            sort_list(cnt);
            // running masses, two elements to a thread
            const int i0 = threadIdx.x * 2;
            u64 q[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                q[j] = i0 + j < cnt ? mass.template of<BF16>(ord2f(static_cast<uint32_t>(sm->list[i0 + j] >> 32))) : 0;
            const u64 inc = warp_scan(q[0] + q[1], lane);
            if (lane == 31) sm->sum[warp] = inc;
            __syncthreads();
            u64 run = above_m + inc - q[0] - q[1];
            for (int i = 0; i < warp; ++i) run += sm->sum[i];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const u64 next = run + q[j];
                if (i0 + j < cnt && (by_mass ? run < target && next >= target : above_n + i0 + j + 1 == target)) {
                    sm->hit_above_m = next;
                    sm->hit_bin = i0 + j;
                }
                run = next;
            }
            __syncthreads();
            const u64 k = sm->list[sm->hit_bin];
            r.through = sm->hit_above_m;
            r.key = static_cast<uint32_t>(k >> 32);
            r.id = key_idx(k);
            __syncthreads();
        }
        return r;
    }

    // ---- bf16 rows by the values themselves: see the head of this file.
    static constexpr int KEYS = 3 * S_BINS, K_PER = KEYS / S_THREADS;  // bins, and a thread's in a scan
    static constexpr uint32_t K_POS = 0xbb80u, K_NEG = 0x447fu;        // the keys of 2^-8 and -2^-8

    // What the first CTA finds: the key of the drawn token, which of its ties it is, and Z.  All CTAs; false where a
    // question ends among values that have no bin of their own.
    __device__ bool by_values(int top_k, bool by_k, float top_p, float z_min, float u, uint32_t *key,
                              u64 *tie, u64 *Z_out) {
        uint32_t *bins = sm->cnt;  // and lo, hi behind it
        for (int i = threadIdx.x * 4; i < KEYS; i += S_THREADS * 4) *reinterpret_cast<uint4 *>(bins + i) = make_uint4(0, 0, 0, 0);
        __syncthreads();
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // the first CTA's bins may be added to
        const uint32_t k_max = key_of(mass.m) >> 16;
        // place of a value: its key below the largest, the keys between -2^-8 and 2^-8 counting as one
        const int np = k_max >= K_POS ? static_cast<int>(k_max - K_POS) + 1 : 0;
        const int gap = k_max >= K_POS ? static_cast<int>(K_POS - K_NEG) - 2 : k_max > K_NEG ? static_cast<int>(k_max - K_NEG) - 1 : -1;
        // ... for a value's upper 16 bits h: above - h, or below + (h less its sign)
        const int above = static_cast<int>(k_max) - 0x8000, below = static_cast<int>(k_max) - 0x7fff - gap;
        u64 near = 0, far = 0;  // masses between -2^-8 and 2^-8, and past the bins
        uint32_t near_n = 0;
        for (int i = threadIdx.x * VEC; i < n; i += S_THREADS * VEC) {
            float z[VEC];
            if (i + VEC <= n) split(vector(i), z);
            else rest(i, z);
            uint32_t others = 0;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                // the bits of a positive value below the largest one's, of a negative one above its own sign's first
                const int h = __float_as_int(z[j]) >> 16, at = (h < 0 ? (h & 0x7fff) + below : above - h);
                if ((h & 0x7fff) >= 0x3b80 && at < KEYS) atomicAdd(bins + at, 1u);
                else if (z[j] != NEG_INF) others |= 1u << j;
            }
            while (others) {
                const int j = __ffs(others) - 1;
                others &= others - 1;
                float x = z[0];
#pragma unroll
                for (int k = 1; k < VEC; ++k) x = k == j ? z[k] : x;
                const u64 q = mass.template of<BF16>(x);
                if (x < 0.00390625f && x > -0.00390625f) near += q, ++near_n;
                else far += q;
            }
        }
        __syncwarp();
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) near += __shfl_xor_sync(FULL, near, d), far += __shfl_xor_sync(FULL, far, d);
        near_n = __reduce_add_sync(FULL, near_n);
        if (lane == 0) sm->list[warp] = near, sm->list[32 + warp] = far, sm->list[64 + warp] = near_n;
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        __syncthreads();
        if (threadIdx.x < 3) {
            u64 all = 0;
            for (int i = 0; i < S_WARPS; ++i) all += sm->list[32 * threadIdx.x + i];
            peer(threadIdx.x == 0 ? &sm->in_word[rank] : threadIdx.x == 1 ? &sm->in_far[rank] : &sm->in_near[rank], 0)[0] = all;
        }
        if (rank != 0) {
            uint32_t *first = peer(bins, 0);
            for (int i = threadIdx.x; i < KEYS; i += S_THREADS)
                if (const uint32_t c = bins[i]) atomicAdd(first + i, c);
        }
        cluster_sync();
        if (rank == 0) {
            near = far = 0, near_n = 0;
            for (int q = 0; q < C; ++q) near += sm->in_word[q], far += sm->in_far[q], near_n += static_cast<uint32_t>(sm->in_near[q]);
            // below a largest value of about 2^40 and more the place between -2^-8 and 2^-8 is past the bins like what lies below it
            if (np >= KEYS) far += near, near = 0, near_n = 0;
            // Runs of K_PER bins, neighbouring ones to different warps: most tokens lie in a few hundred bins.  The counts
            // stay in this CTA's bins, what lies above a run in the list's place.
            const int g = lane * S_WARPS + warp, b0 = g * K_PER;
            u64 tn = 0, tm = 0, kept = 0;
            bool open = false;  // min_p ends where values have no bin
#pragma unroll 1
            for (int j = 0; j < K_PER; j += 4) {
                uint4 c4 = *reinterpret_cast<const uint4 *>(bins + b0 + j);
                if (np >= b0 + j && np < b0 + j + 4) {
                    uint32_t *c = np == b0 + j ? &c4.x : np == b0 + j + 1 ? &c4.y : np == b0 + j + 2 ? &c4.z : &c4.w;
                    if (near_n) {
                        *c = near_n;
                        open = z_min > -0.00390625f && z_min <= 0.00390625f;
                        tm += near, kept += z_min <= -0.00390625f ? near : 0;
                    }
                }
                *reinterpret_cast<uint4 *>(bins + b0 + j) = c4;
                tn += static_cast<u64>(c4.x) + c4.y + c4.z + c4.w;
                if ((c4.x | c4.y | c4.z | c4.w) == 0) continue;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t n1 = i == 0 ? c4.x : i == 1 ? c4.y : i == 2 ? c4.z : c4.w;
                    const float z = value_at(b0 + j + i, k_max, np, gap);
                    const u64 all = b0 + j + i == np && near_n ? 0 : n1 * mass.template of<BF16>(z);
                    tm += all, kept += z >= z_min ? all : 0;
                }
            }
            u64 *run_m = sm->list, *run_n = sm->list + S_THREADS;
            run_m[g] = tm, run_n[g] = tn;
            __syncthreads();
            const u64 my_n = run_n[threadIdx.x], my_m = run_m[threadIdx.x];
            const u64 in = warp_scan(my_n, lane), im = warp_scan(my_m, lane);
            if (lane == 31) sm->sum[warp] = in, sm->sum2[warp] = im;
            __syncthreads();
            u64 an = in - my_n, am = im - my_m, N = 0, M = 0;
#pragma unroll
            for (int i = 0; i < S_WARPS; ++i) {
                const u64 x = sm->sum[i], y = sm->sum2[i];
                if (i < warp) an += x, am += y;
                N += x, M += y;
            }
            run_m[threadIdx.x] = am, run_n[threadIdx.x] = an;
            u64 Z = M + far;
            kept = block_sum(kept);
            if (far && z_min <= value_at(KEYS - 1, k_max, np, gap)) kept = z_min == NEG_INF ? Z : 0, open |= z_min != NEG_INF;
            bool fine = !__syncthreads_or(open);
            // where count or mass comes to the goal: key, tie, mass through it; false among values without a bin
            auto settle = [&](bool by_mass, u64 goal) {
                if (threadIdx.x == 0) sm->go_n = 0, sm->go_i[0] = -1;
                __syncthreads();
                if (by_mass ? am < goal && am + my_m >= goal : an < goal && an + my_n >= goal) sm->go_i[0] = threadIdx.x;
                __syncthreads();
                const int run = sm->go_i[0];
                if (warp == 0 && run >= 0) {  // a lane to a bin of the run
                    const int b = run * K_PER + lane;
                    u64 n1 = 0, w = 0, all = 0;
                    if (lane < K_PER) {
                        n1 = bins[b];
                        const bool is_near = b == np && near_n;
                        w = n1 == 0 || is_near ? 0 : mass.template of<BF16>(value_at(b, k_max, np, gap));
                        all = is_near ? near : n1 * w;
                    }
                    const u64 nn1 = run_n[run] + warp_scan(n1, lane), mm = run_m[run] + warp_scan(all, lane);
                    if (lane < K_PER && w && (by_mass ? mm - all < goal && mm >= goal : nn1 - n1 < goal && nn1 >= goal)) {
                        const u64 t = by_mass ? (goal - (mm - all) + w - 1) / w : goal - (nn1 - n1);
                        sm->go_n = 1;
                        sm->go_key = key_of(value_at(b, k_max, np, gap));
                        sm->go_a = t;
                        sm->hit_above_m = mm - all + t * w;
                    }
                }
                __syncthreads();
                return sm->go_n != 0;
            };
            if (fine && by_k && static_cast<u64>(top_k) < N) {
                fine = settle(false, top_k);
                Z = sm->hit_above_m;
            } else if (by_k && far) {
                fine = false;
            }
            if (fine && top_p < 1.0f) {
                if (threadIdx.x == 0) sm->hit_above_n = goal_reach(top_p, Z);
                __syncthreads();
                fine = settle(true, sm->hit_above_n);
                Z = sm->hit_above_m;
            }
            if (fine) {
                Z = kept < Z ? kept : Z;
                if (threadIdx.x == 0) sm->hit_above_n = goal_pass(u, Z);
                __syncthreads();
                fine = settle(true, sm->hit_above_n);
            }
            const uint32_t k = sm->go_key;
            *key = k, *tie = sm->go_a, *Z_out = Z;
            __syncthreads();
            if (threadIdx.x < C) peer(&sm->go_n, threadIdx.x)[0] = fine, peer(&sm->go_key, threadIdx.x)[0] = k;
        }
        cluster_sync();
        *key = sm->go_key;
        return sm->go_n != 0;
    }
    // The value whose place is b.
    __device__ __forceinline__ static float value_at(int b, uint32_t k_max, int np, int gap) {
        const int k = static_cast<int>(k_max) - b - (b < np ? 0 : gap);
        const uint32_t o = static_cast<uint32_t>(k < 0 ? 0 : k) << 16;
        return ord2f((o & 0x80000000u) ? o : o | 0xffffu);
    }

    // The id of the tie-th (known to the first CTA) entry with a key.  All CTAs; the answer is the first CTA's.
    __device__ int64_t place_of(uint32_t key, u64 tie) {
        if (rank == 0 && threadIdx.x < C) peer(&sm->go_a, threadIdx.x)[0] = tie;
        const int per = (n + S_THREADS * VEC - 1) / (S_THREADS * VEC) * VEC, a = per * threadIdx.x, b = min(a + per, n);
        const float value = ord2f(key);
        uint32_t mine = 0;
        for (int i = a; i < b; i += VEC) {
            float z[VEC];
            if (i + VEC <= n) split(vector(i), z);
            else rest(i, z);
#pragma unroll
            for (int j = 0; j < VEC; ++j) mine += z[j] == value;
        }
        const uint32_t inc = warp_scan(mine, lane);
        __syncthreads();
        if (lane == 31) sm->sum[warp] = inc;
        __syncthreads();
        u64 before = inc - mine, all = 0;
        for (int i = 0; i < S_WARPS; ++i) {
            if (i < warp) before += sm->sum[i];
            all += sm->sum[i];
        }
        if (threadIdx.x < C) peer(&sm->in_word[rank], threadIdx.x)[0] = all;
        cluster_sync();
        for (int q = 0; q < rank; ++q) before += sm->in_word[q];
        const u64 want = sm->go_a;
        if (want > before && want <= before + mine) {
            u64 left = want - before;
            for (int i = a; i < b; i += VEC) {
                float z[VEC];
                if (i + VEC <= n) split(vector(i), z);
                else rest(i, z);
                uint32_t hits = 0;
#pragma unroll
                for (int j = 0; j < VEC; ++j) hits |= z[j] == value ? 1u << j : 0u;
                const uint32_t c = __popc(hits);
                if (left <= c) {
                    while (--left) hits &= hits - 1;
                    peer(&sm->go_b, 0)[0] = static_cast<u64>(id0 + i + __ffs(hits) - 1);
                    break;
                }
                left -= c;
            }
        }
        cluster_sync();
        return static_cast<int64_t>(sm->go_b);
    }
};

template <bool BF16>
__global__ void __launch_bounds__(S_THREADS, 2) k_sample(const SampleArgs a, int C) {
    extern __shared__ __align__(128) unsigned char raw[];
    SampleSmem *sm = reinterpret_cast<SampleSmem *>(raw);
    constexpr int E = BF16 ? 2 : 4;
    const int64_t r = blockIdx.x / C;
    Sampler<BF16> s;
    s.sm = sm;
    s.C = C;
    s.rank = C > 1 ? static_cast<int>(cluster_rank()) : 0;
    s.lane = threadIdx.x & 31, s.warp = threadIdx.x >> 5;
    s.id0 = static_cast<int64_t>(a.slice) * s.rank;
    const int64_t left = a.V - s.id0;
    s.n = left <= 0 ? 0 : static_cast<int>(left < a.slice ? left : a.slice);
    const char *src = static_cast<const char *>(a.logits) + (r * a.ld + s.id0) * E;
    // a thread copies the vectors that it reads itself
    if (a.resident) {
        char *dst = reinterpret_cast<char *>(raw) + sizeof(SampleSmem);
        for (int i = threadIdx.x * s.VEC; i < s.n; i += S_THREADS * s.VEC) {
            if (i + s.VEC <= s.n)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst + i * E)), "l"(src + i * E) : "memory");
            else
                for (int j = i; j < s.n; ++j) {
                    if (BF16) reinterpret_cast<uint16_t *>(dst)[j] = reinterpret_cast<const uint16_t *>(src)[j];
                    else reinterpret_cast<float *>(dst)[j] = reinterpret_cast<const float *>(src)[j];
                }
        }
        s.data = dst;
    } else {
        s.data = src;
    }
    // the other CTAs have started when this is waited for
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    float T = 0.0f, top_p = 1.0f, min_p = 0.0f;
    int top_k = 0;
    if (a.params) {
        const dflash2_sampling p = a.params[r / a.rows_per_param];
        T = p.temperature, top_k = p.top_k, top_p = p.top_p;
    }
    if (a.min_p) min_p = a.min_p[r / a.rows_per_param];
    const float u = a.u[r];
    if (threadIdx.x < 4) sm->list_n[threadIdx.x] = 0;
    // 64-bit arithmetic is slow here: one thread's, for all
    if (threadIdx.x == 0) {
        const double t = T == 0.0f ? 1.0 : fmax(static_cast<double>(T), 0x1p-127);  // so that c is a float
        const double inv_t = 1.0 / t, c = 1.4426950408889634074 * inv_t;
        sm->inv_t = inv_t;
        sm->ch = static_cast<float>(c), sm->cl = static_cast<float>(c - static_cast<double>(sm->ch));
        sm->t_log = min_p > 0.0f ? t * log(static_cast<double>(min_p)) : 0.0;
    }
    if (threadIdx.x >= 32 && threadIdx.x < 64) {
        const double v = exp2(-static_cast<double>(threadIdx.x - 32) / 32);
        const float h = static_cast<float>(v);
        sm->root[threadIdx.x - 32] = make_float2(h, static_cast<float>(v - h));
    }
    asm volatile("cp.async.wait_all;" ::: "memory");

    // ---- the largest logit
    float least;
    const float mine = s.largest(least);
    bool bad = __any_sync(FULL, !(mine < __builtin_huge_valf()));
    float m = warp_max_f(mine);
    least = -warp_max_f(-least);
    if (s.lane == 0) sm->sum[s.warp] = (static_cast<u64>(bad) << 32) | __float_as_uint(m), sm->sum2[s.warp] = __float_as_uint(least);
    __syncthreads();
    for (int i = 0; i < S_WARPS; ++i) {
        m = fmaxf(m, __uint_as_float(static_cast<uint32_t>(sm->sum[i])));
        bad |= (sm->sum[i] >> 32) != 0;
        least = fminf(least, __uint_as_float(static_cast<uint32_t>(sm->sum2[i])));
    }
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (threadIdx.x < C) {
        peer(&sm->in_max[s.rank], threadIdx.x)[0] = m;
        peer(&sm->in_bad[s.rank], threadIdx.x)[0] = bad;
        peer(&sm->in_min[s.rank], threadIdx.x)[0] = least;
    }
    cluster_sync();
    for (int q = 0; q < C; ++q) m = fmaxf(m, sm->in_max[q]), bad |= sm->in_bad[q] != 0, least = fminf(least, sm->in_min[q]);
    if (bad || m == NEG_INF || !(T >= 0.0f) || isinf(T) || top_k < 0 || !(top_p > 0.0f && top_p <= 1.0f) ||
        !(min_p >= 0.0f && min_p <= 1.0f) || isnan(u)) {
        if (s.rank == 0 && threadIdx.x == 0) a.token[r] = -1, a.prob[r] = __uint_as_float(0x7fc00000u);
        return;
    }
    if (T == 0.0f || top_k == 1) {
        uint32_t at = 0xffffffffu;
        s.each([&](float z, int i) {
            if (z == m) at = min(at, static_cast<uint32_t>(s.id0 + i));
        });
        at = __reduce_min_sync(FULL, at);
        __syncthreads();
        if (s.lane == 0) sm->sum[s.warp] = at;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 0; i < S_WARPS; ++i) at = min(at, static_cast<uint32_t>(sm->sum[i]));
            peer(&sm->in_word[s.rank], 0)[0] = at;
        }
        cluster_sync();
        if (s.rank == 0 && threadIdx.x == 0) {
            for (int q = 0; q < C; ++q) at = min(at, static_cast<uint32_t>(sm->in_word[q]));
            a.token[r] = static_cast<int32_t>(at), a.prob[r] = 1.0f;
        }
        return;
    }
    s.mass.m = m;
    s.mass.ch = sm->ch, s.mass.cl = sm->cl;
    s.mass.shift = a.shift;
    s.mass.root = sm->root;
    s.t_cap = static_cast<float>(a.shift + 1);
    s.z_floor = NEG_INF;
    float z_min = NEG_INF;  // min_p's tokens: z >= z_min
    if (min_p > 0.0f) {
        z_min = __double2float_ru(static_cast<double>(m) + sm->t_log);
        if (top_p == 1.0f) {
            s.z_floor = z_min;
            s.t_cap = fminf(s.t_cap, fmaf(m - z_min, s.mass.ch, 1.0f));
        }
    }
    // no further than the row goes, so that the bins are as fine as they can be
    if (!BF16) s.t_cap = fminf(s.t_cap, fmaf(m - least, s.mass.ch * 1.00001f, 1e-30f));
    s.t_scale = S_BINS / s.t_cap;
    const bool by_k = top_k > 0 && top_k < a.V;
    u64 total_n = 0, total_m = 0;
    if (by_k && top_k <= C * S_THREADS) {
        // A floor that at least top_k tokens reach: the best CTA's top_k-th largest of its threads' maxima, or the worst
        // CTA's (top_k / C)-th, whichever is higher.
        s.clear(true);
        const float t = s.mass.template t_of<BF16>(mine);
        if (s.inside(mine, t)) atomicAdd(&sm->cnt[s.bin_of(t)], 1u);
        __syncthreads();
        const uint4 c4 = *reinterpret_cast<const uint4 *>(sm->cnt + threadIdx.x * S_PER);
        uint32_t c[S_PER] = {c4.x, c4.y, c4.z, c4.w}, run = c4.x + c4.y + c4.z + c4.w;
        run = warp_scan(run, s.lane) - run;
        if (s.lane == 31) sm->sum[s.warp] = run + c4.x + c4.y + c4.z + c4.w;
        if (threadIdx.x < 2) sm->floor_bin[threadIdx.x] = S_BINS - 1;
        __syncthreads();
        for (int i = 0; i < s.warp; ++i) run += static_cast<uint32_t>(sm->sum[i]);
        const uint32_t part = (top_k + C - 1) / C;
#pragma unroll
        for (int j = 0; j < S_PER; ++j) {
            const uint32_t next = run + c[j];
            if (run < static_cast<uint32_t>(top_k) && next >= static_cast<uint32_t>(top_k)) sm->floor_bin[0] = threadIdx.x * S_PER + j;
            if (run < part && next >= part) sm->floor_bin[1] = threadIdx.x * S_PER + j;
            run = next;
        }
        __syncthreads();
        if (threadIdx.x < C) peer(&sm->in_word[s.rank], threadIdx.x)[0] = (static_cast<u64>(sm->floor_bin[0]) << 32) | sm->floor_bin[1];
        cluster_sync();
        uint32_t best = S_BINS - 1, worst = 0;
        for (int q = 0; q < C; ++q)
            best = min(best, static_cast<uint32_t>(sm->in_word[q] >> 32)), worst = max(worst, static_cast<uint32_t>(sm->in_word[q]));
        // up to the bin's far end, and a little more for the rounding of the bins
        s.t_cap = fminf(s.t_cap, (static_cast<float>(min(best, worst) + 1) / s.t_scale) * 1.00001f);
        s.t_scale = S_BINS / s.t_cap;
    }
    if ((by_k && top_k <= S_LIST / 2) || s.z_floor > NEG_INF) {
        // few tokens, perhaps: all of them into the first CTA's list, which then answers everything
        uint32_t *list_n = peer(&sm->list_n[3], 0);
        u64 *list = peer(sm->list, 0);
        s.each_within(fmaxf(s.z_floor, s.z_below(s.t_cap)), m, [&](float z, int i) {
            if (s.inside(z, s.mass.template t_of<BF16>(z))) {
                const uint32_t at = atomicAdd(list_n, 1u);
                if (at < S_LIST) list[at] = (static_cast<u64>(s.key_of(z)) << 32) | static_cast<uint32_t>(~static_cast<uint32_t>(s.id0 + i));
            }
        });
        cluster_sync();
        const uint32_t many = *list_n;
        if (many <= S_LIST) {
            if (s.rank != 0) {
                __syncwarp();
                asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // the count has been read
                return;
            }
            s.sort_list(static_cast<int>(many));
            u64 *mass = reinterpret_cast<u64 *>(sm->cnt);  // running masses of the ranking
            const int i0 = threadIdx.x * 2;
            u64 q[2];
            uint32_t kept = 0;  // of this thread's, by min_p
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float z = ord2f(static_cast<uint32_t>(sm->list[i0 + j] >> 32));
                const bool in = i0 + j < static_cast<int>(many);
                q[j] = in ? s.mass.template of<BF16>(z) : 0;
                kept += in && z >= z_min;
            }
            const u64 inc = warp_scan(q[0] + q[1], s.lane);
            if (s.lane == 31) sm->sum[s.warp] = inc;
            kept = __reduce_add_sync(FULL, kept);
            if (s.lane == 0) sm->sum2[s.warp] = kept;
            if (threadIdx.x < 3) sm->go_i[threadIdx.x] = S_LIST;
            __syncthreads();
            u64 run = inc - q[0] - q[1];
            uint32_t keep = by_k ? min(many, static_cast<uint32_t>(top_k)) : many, floor_n = 0;
            for (int i = 0; i < S_WARPS; ++i) {
                if (i < s.warp) run += sm->sum[i];
                floor_n += static_cast<uint32_t>(sm->sum2[i]);
            }
            mass[i0] = run + q[0], mass[i0 + 1] = run + q[0] + q[1];
            __syncthreads();
            // the first place whose running mass reaches the goal, which one thread works out
            auto place = [&](int slot) {
                const u64 goal = sm->go_a;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const u64 before = i0 + j ? mass[i0 + j - 1] : 0;
                    if (before < goal && mass[i0 + j] >= goal) sm->go_i[slot] = i0 + j;
                }
                __syncthreads();
                return sm->go_i[slot];
            };
            if (top_p < 1.0f) {
                if (threadIdx.x == 0) sm->go_a = goal_reach(top_p, mass[keep - 1]);
                __syncthreads();
                keep = min(keep, static_cast<uint32_t>(place(0)) + 1);
            }
            if (min_p > 0.0f) keep = min(keep, max(floor_n, 1u));
            const u64 Z = mass[keep - 1];
            if (threadIdx.x == 0) sm->go_a = goal_pass(u, Z);
            __syncthreads();
            const int at = place(1);
            if (threadIdx.x == 0) {
                const u64 k = sm->list[at];
                a.token[r] = key_idx(k);
                a.prob[r] = static_cast<float>(s.mass.template exactly<BF16>(key_val(k), sm->inv_t) / ldexp(__ull2double_rn(Z), -a.shift));
            }
            cluster_sync();  // the others' reads of the count
            return;
        }
    }
    if constexpr (BF16) {
        uint32_t key;
        u64 tie = 0, Z = 0;
        if (s.by_values(top_k, by_k, top_p, z_min, u, &key, &tie, &Z)) {
            const int64_t id = s.place_of(key, tie);
            if (s.rank == 0 && threadIdx.x == 0) {
                a.token[r] = static_cast<int32_t>(id);
                a.prob[r] = static_cast<float>(s.mass.template exactly<BF16>(ord2f(key), sm->inv_t) / ldexp(__ull2double_rn(Z), -a.shift));
            }
            return;
        }
    }
    // ---- masses into bins.  Asked again where a wide bin's splitting has overwritten them.
    u64 kept_min = 0;
    auto fill = [&]() {
        s.clear(true);
        u64 own = 0;
        s.each([&](float z, int) {
            const float t = s.mass.template t_of<BF16>(z);
            if (s.inside(z, t)) {
                const u64 q = s.mass.template of<BF16>(z);
                if (z >= z_min) own += q;
                s.add(s.bin_of(t), q, by_k);
            }
        });
        own = s.block_sum(own);
        // (not in in_word: the first CTA may still be reading its floors there)
        if (threadIdx.x == 0) peer(&sm->in_far[s.rank], 0)[0] = own;
        cluster_sync();
        if (s.rank == 0) {
            kept_min = 0;
            for (int q = 0; q < C; ++q) kept_min += sm->in_far[q];
            s.gather_bins(&total_n, &total_m);
        }
    };
    // ---- top_k, top_p, the draw: where the ranking reaches a count or a mass
    s.calls = 0;
    s.dirty = true;
    u64 Z = 0;
    typename Sampler<BF16>::Found f = {};
#pragma unroll 1
    for (int stage = 0; stage < 3; ++stage) {
        if ((stage == 0 && !by_k) || (stage == 1 && !(top_p < 1.0f))) continue;
        if (s.dirty) {
            fill();
            if (s.calls == 0) Z = total_m;
            s.dirty = false;
        }
        u64 goal = 0;
        if (stage == 0) {
            // tokens of no whole unit are not in the bins: a top_k that reaches past the others keeps them all
            if (s.rank == 0 && threadIdx.x < C) peer(&sm->go_a, threadIdx.x)[0] = static_cast<u64>(top_k) < total_n;
            cluster_sync();
            if (!sm->go_a) continue;
            goal = top_k;
        } else if (stage == 1) {
            if (threadIdx.x == 0) goal = goal_reach(top_p, Z);
        } else {
            Z = kept_min < Z ? kept_min : Z;
            if (threadIdx.x == 0) goal = goal_pass(u, Z);
        }
        if (s.rank == 0 && threadIdx.x == 0) sm->hit_above_m = goal;
        __syncthreads();
        goal = sm->hit_above_m;
        __syncthreads();
        f = s.find(stage != 0, goal, total_n, total_m, stage == 2);
        if (stage != 2) Z = f.through;
    }
    if (s.rank == 0 && threadIdx.x == 0) {
        a.token[r] = static_cast<int32_t>(f.id);
        a.prob[r] = static_cast<float>(s.mass.template exactly<BF16>(ord2f(f.key), sm->inv_t) / ldexp(__ull2double_rn(Z), -a.shift));
    }
    cluster_sync();  // the first CTA's list is read until here
}

template <bool BF16>
static dflash2_status launch_sample(const SampleArgs &a, unsigned grid, int C, size_t smem, cudaStream_t s) {
    auto fn = &k_sample<BF16>;
    {
        static int opted[64] = {0};
        static std::mutex mu;
        const int dev = current_device();
        std::lock_guard<std::mutex> lock(mu);
        if (dev < 0 || dev >= 64 || !opted[dev]) {
            if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 226 * 1024) != cudaSuccess)
                return DFLASH2_ERR_CUDA;
            if (dev >= 0 && dev < 64) opted[dev] = 1;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(S_THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(C);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, fn, a, C) != cudaSuccess) return DFLASH2_ERR_CUDA;
    return after_launch();
}

}  // namespace dfl

using namespace dfl;

extern "C" dflash2_status dflash2_sample(const void *logits, dflash2_dtype dt, int64_t rows, int64_t V, int64_t ld,
                                         const dflash2_sampling *params, const float *min_p, int64_t rows_per_param,
                                         const float *u, int32_t *token, float *prob, dflash2_stream stream) {
    if (!dtype_ok(dt) || rows < 0 || V < 1 || V > 0x7fffffff || ld < V || ld * esize(dt) % 16 != 0 || rows_per_param < 1)
        return DFLASH2_ERR_INVALID_ARG;
    if (rows == 0) return DFLASH2_OK;
    if (rows > 0x7fffffff / S_CLUSTER) return DFLASH2_ERR_UNSUPPORTED;
    if (!logits || !u || !token || !prob || !aligned16(logits)) return DFLASH2_ERR_INVALID_ARG;
    for (const void *p : {static_cast<const void *>(params), static_cast<const void *>(min_p),
                          static_cast<const void *>(u), static_cast<const void *>(token),
                          static_cast<const void *>(prob)})
        if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return DFLASH2_ERR_INVALID_ARG;
    SampleArgs a = {};
    a.logits = logits, a.V = V, a.ld = ld, a.params = params, a.min_p = min_p, a.rows_per_param = rows_per_param;
    a.u = u, a.token = token, a.prob = prob;
    a.shift = 44;  // (2^-22 and 2^-22: what two roundings to whole floats give)
    while ((V >> (63 - a.shift)) != 0) --a.shift;
    // CTAs of a row: until a slice lets two CTAs share an SM, and while CTA slots are left over and slices long
    const size_t fixed = sizeof(SampleSmem), e = esize(dt);
    const auto slice_of = [&](int C) { return (V + 8 * C - 1) / (8 * C) * 8; };
    int C = 1;
    while (C < S_CLUSTER && (fixed + slice_of(C) * e > 112 * 1024 || (rows * C < sm_count() && slice_of(C) > 4096))) C *= 2;
    a.slice = static_cast<int>(slice_of(C));
    const bool resident = slice_of(C) * static_cast<int64_t>(e) <= static_cast<int64_t>(226 * 1024 - fixed);
    a.resident = resident;
    const size_t smem = fixed + (resident ? slice_of(C) * e : 0);
    const unsigned grid = static_cast<unsigned>(rows * C);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dt == DFLASH2_BF16 ? launch_sample<true>(a, grid, C, smem, s) : launch_sample<false>(a, grid, C, smem, s);
}
