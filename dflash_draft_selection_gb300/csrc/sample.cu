// sample.cu -- dflash2_sample: one token per row of logits from a given uniform.
//
// temperature -> top_k -> top_p -> min_p, then the inverse of the cumulative
// distribution over the kept tokens, best first (larger logit, then lower id).
#include "common.cuh"
#include "host.hpp"

namespace dfl {

constexpr int SAMPLE_THREADS = 1024;
typedef unsigned long long u64;

template <bool BF16>
__device__ __forceinline__ float logit(const void *row, int64_t i) {
    const float v = BF16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(row)[i]) << 16)
                         : static_cast<const float *>(row)[i];
    return v == 0.0f ? 0.0f : v;
}

struct SampleSmem {
    uint32_t count[256], lo[256], hi[256];
    uint32_t warp[32];
    float fmax[32];
    u64 above_n, above_m;
    uint32_t digit;
    int bad;
};

template <bool BF16>
struct RowSampler {
    const void *row;
    int64_t V;
    float m;
    double inv_t;
    int shift;  // masses are in units of 2^-shift
    SampleSmem *sm;

    __device__ u64 mass(float z) const { return __double2ull_rn(ldexp(exp((static_cast<double>(z) - m) * inv_t), shift)); }

    // The key at which the running measure (count or mass) from the largest key down reaches `target` >= 1, among
    // keys >= floor.  above_n and above_m: count and mass of the larger keys.  False if it never does.
    __device__ bool descend(bool by_mass, u64 target, uint32_t floor, uint32_t *key, u64 *above_n, u64 *above_m) {
        uint32_t prefix = 0, mask = 0;
        u64 an = 0, am = 0;
        for (int level = 3; level >= 0; --level) {
            const int s = level * 8;
            for (int i = threadIdx.x; i < 256; i += SAMPLE_THREADS) sm->count[i] = sm->lo[i] = sm->hi[i] = 0;
            __syncthreads();
            for (int64_t i = threadIdx.x; i < V; i += SAMPLE_THREADS) {
                const float z = logit<BF16>(row, i);
                const uint32_t k = f2ord(z);
                if ((k & mask) != prefix || k < floor) continue;
                const uint32_t d = (k >> s) & 255;
                atomicAdd(&sm->count[d], 1u);
                const u64 q = mass(z);
                const uint32_t ql = static_cast<uint32_t>(q), old = atomicAdd(&sm->lo[d], ql);
                const uint32_t up = static_cast<uint32_t>(q >> 32) + (old + ql < old ? 1u : 0u);
                if (up) atomicAdd(&sm->hi[d], up);
            }
            __syncthreads();
            if (threadIdx.x == 0) {
                u64 n = an, w = am;
                int d = 255;
                for (; d >= 0; --d) {
                    const u64 cn = sm->count[d], cm = (static_cast<u64>(sm->hi[d]) << 32) | sm->lo[d];
                    if ((by_mass ? w + cm : n + cn) >= target) break;
                    n += cn;
                    w += cm;
                }
                sm->digit = d < 0 ? 256 : d;
                sm->above_n = n;
                sm->above_m = w;
            }
            __syncthreads();
            const uint32_t d = sm->digit;
            an = sm->above_n;
            am = sm->above_m;
            __syncthreads();
            if (d == 256) {
                *above_n = an;
                *above_m = am;
                return false;
            }
            prefix |= d << s;
            mask |= 255u << s;
        }
        *key = prefix;
        *above_n = an;
        *above_m = am;
        return true;
    }
};

template <bool BF16>
__global__ void __launch_bounds__(SAMPLE_THREADS) k_sample(const void *logits, int64_t V, int64_t ld,
                                                           const dflash2_sampling *params, const float *min_ps,
                                                           int64_t rows_per_param, const float *us, int32_t *token,
                                                           float *prob, int shift) {
    __shared__ SampleSmem smem;
    SampleSmem *sm = &smem;
    const int64_t r = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float T = 0.0f, top_p = 1.0f, min_p = 0.0f;
    int top_k = 0;
    if (params) {
        const dflash2_sampling p = params[r / rows_per_param];
        T = p.temperature, top_k = p.top_k, top_p = p.top_p;
    }
    if (min_ps) min_p = min_ps[r / rows_per_param];
    const float u = us[r];
    const void *row = static_cast<const char *>(logits) + r * ld * (BF16 ? 2 : 4);
    if (threadIdx.x == 0) sm->bad = 0;
    __syncthreads();
    float m = NEG_INF;
    bool bad = false;
    for (int64_t i = threadIdx.x; i < V; i += SAMPLE_THREADS) {
        const float z = logit<BF16>(row, i);
        bad |= !(z < __builtin_huge_valf());
        m = fmaxf(m, z);
    }
    if (bad) sm->bad = 1;
    m = warp_max_f(m);
    if (lane == 0) sm->fmax[warp] = m;
    __syncthreads();
    m = warp_max_f(sm->fmax[lane]);
    bad = sm->bad || m == NEG_INF || !(T >= 0.0f) || isinf(T) || top_k < 0 || !(top_p > 0.0f && top_p <= 1.0f) ||
          !(min_p >= 0.0f && min_p <= 1.0f) || isnan(u);
    if (bad) {
        if (threadIdx.x == 0) token[r] = -1, prob[r] = __uint_as_float(0x7fc00000u);
        return;
    }
    if (T == 0.0f) T = 1.0f, top_k = 1;
    RowSampler<BF16> rs{row, V, m, 1.0 / static_cast<double>(T), shift, sm};
    // the kept tokens: keys above `cut`, and the first `ties` (by id) at it
    uint32_t cut = f2ord(NEG_INF), key;
    u64 ties = V, an, am, Z;
    if (top_k > 0 && top_k < V) {
        rs.descend(false, top_k, 0, &key, &an, &am);
        cut = key;
        ties = top_k - an;
        Z = am + ties * rs.mass(ord2f(key));
    } else {
        rs.descend(true, ~0ull, 0, &key, &an, &Z);
    }
    if (top_p < 1.0f) {
        u64 target = __double2ull_ru(static_cast<double>(top_p) * __ull2double_rn(Z));
        if (target < 1) target = 1;
        rs.descend(true, target, cut, &key, &an, &am);
        const u64 q = rs.mass(ord2f(key)), t = (target - am + q - 1) / q;
        cut = key;
        ties = t;
        Z = am + t * q;
    }
    if (min_p > 0.0f) {
        const double thr = static_cast<double>(m) + static_cast<double>(T) * log(static_cast<double>(min_p));
        float f = __double2float_ru(thr);
        f = f == 0.0f ? 0.0f : f;
        if (f2ord(f) > cut) {
            cut = f2ord(f);
            ties = V;
            rs.descend(true, ~0ull, cut, &key, &an, &Z);
        }
    }
    u64 target = __double2ull_rd(static_cast<double>(fminf(fmaxf(u, 0.0f), 1.0f)) * __ull2double_rn(Z)) + 1;
    if (target > Z) target = Z;
    rs.descend(true, target, cut, &key, &an, &am);
    const u64 q = rs.mass(ord2f(key));
    u64 want = (target - am + q - 1) / q;  // the want-th occurrence of the key, by id
    if (key == cut && want > ties) want = ties;
    // contiguous stretches per thread, so that ids ascend with threads
    const int64_t per = (V + SAMPLE_THREADS - 1) / SAMPLE_THREADS, a = per * threadIdx.x;
    uint32_t mine = 0;
    for (int64_t i = a; i < a + per && i < V; ++i) mine += f2ord(logit<BF16>(row, i)) == key;
    uint32_t inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t t = __shfl_up_sync(FULL, inc, d);
        if (lane >= d) inc += t;
    }
    if (lane == 31) sm->warp[warp] = inc;
    __syncthreads();
    uint32_t base = 0;
    for (int i = 0; i < warp; ++i) base += sm->warp[i];
    const u64 before = base + inc - mine;
    if (want > before && want <= before + mine) {
        u64 left = want - before;
        for (int64_t i = a; i < a + per && i < V; ++i)
            if (f2ord(logit<BF16>(row, i)) == key && --left == 0) {
                token[r] = static_cast<int32_t>(i);
                prob[r] = static_cast<float>(exp((static_cast<double>(ord2f(key)) - m) * rs.inv_t) /
                                             ldexp(__ull2double_rn(Z), -shift));
                break;
            }
    }
}

}  // namespace dfl

using namespace dfl;

extern "C" dflash2_status dflash2_sample(const void *logits, dflash2_dtype dt, int64_t rows, int64_t V, int64_t ld,
                                         const dflash2_sampling *params, const float *min_p, int64_t rows_per_param,
                                         const float *u, int32_t *token, float *prob, dflash2_stream stream) {
    if (!dtype_ok(dt) || rows < 0 || V < 1 || V > 0x7fffffff || ld < V || ld * esize(dt) % 16 != 0 || rows_per_param < 1)
        return DFLASH2_ERR_INVALID_ARG;
    if (rows == 0) return DFLASH2_OK;
    if (!logits || !u || !token || !prob || !aligned16(logits)) return DFLASH2_ERR_INVALID_ARG;
    for (const void *p : {static_cast<const void *>(params), static_cast<const void *>(min_p),
                          static_cast<const void *>(u), static_cast<const void *>(token),
                          static_cast<const void *>(prob)})
        if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return DFLASH2_ERR_INVALID_ARG;
    if (rows > 0x7fffffff) return DFLASH2_ERR_UNSUPPORTED;
    int shift = 45;
    while (shift > 0 && (V >> (63 - shift)) != 0) --shift;
    const unsigned grid = static_cast<unsigned>(rows);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dt == DFLASH2_BF16)
        k_sample<true><<<grid, SAMPLE_THREADS, 0, s>>>(logits, V, ld, params, min_p, rows_per_param, u, token, prob, shift);
    else
        k_sample<false><<<grid, SAMPLE_THREADS, 0, s>>>(logits, V, ld, params, min_p, rows_per_param, u, token, prob, shift);
    return after_launch();
}
