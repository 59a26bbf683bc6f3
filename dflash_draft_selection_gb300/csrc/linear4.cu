// linear4.cu -- dflash2_quant4, dflash2_dequant4 and dflash2_linear4: weights in
// 4 bits with a scale (and a zero point) per group, and products with them.
//
// TensorRT-LLM issue 18085 and FreeToken PR 857 run this path for targets and
// drafters whose weights are held in 4 bits; the pages name the formats and give
// no kernel.
#include "weight4.cuh"

namespace dfl {

__device__ __forceinline__ float load_f(const void *p, dflash2_dtype dt, int64_t i) { return side_at(p, dt, i); }

// One warp per group: scale, zero point, codes.
__global__ void __launch_bounds__(256) k_quant4(const void *W, dflash2_dtype dt, int64_t ld, dflash2_weight4 w, int64_t G) {
    const int lane = threadIdx.x & 31;
    const int64_t item = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    if (item >= w.N * G) return;
    const int64_t n = item / G, gi = item % G;
    const int64_t k0 = gi * w.group;
    const int per = w.group / 32;
    float v[4];
    float lo = 0.0f, hi = 0.0f;
    bool bad = false;
    for (int i = 0; i < per; ++i) {
        const int64_t k = k0 + lane * per + i;
        v[i] = k < w.K ? load_f(W, dt, n * ld + k) : 0.0f;
        bad |= !isfinite(v[i]);
        lo = fminf(lo, v[i]);
        hi = fmaxf(hi, v[i]);
    }
    bad = __any_sync(FULL, bad);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(FULL, lo, d));
        hi = fmaxf(hi, __shfl_xor_sync(FULL, hi, d));
    }
    float scale = w.zero ? __fsub_rn(__fdiv_rn(hi, 15.0f), __fdiv_rn(lo, 15.0f)) : __fdiv_rn(fmaxf(hi, -lo), 7.0f);
    if (w.side_dt == DFLASH2_BF16) scale = __uint_as_float(static_cast<uint32_t>(bf16_bits(scale)) << 16);
    const float step = scale == 0.0f ? 1.0f : scale;
    const float zero = w.zero ? fminf(fmaxf(rintf(__fdiv_rn(-lo, step)), 0.0f), 15.0f) : 8.0f;
    for (int i = 0; i < per; ++i) {
        const int64_t k = k0 + lane * per + i;
        const int c = bad ? 8 : static_cast<int>(fminf(fmaxf(rintf(__fdiv_rn(v[i], step)) + zero, 0.0f), 15.0f));
        v[i] = static_cast<float>(k < w.K ? c : 8);
    }
    uint8_t *row = static_cast<uint8_t *>(w.codes) + n * w.code_stride;
    const int64_t end = (w.K + 31) / 32 * 32;
    for (int i = 0; i < per; ++i) {
        const int64_t k = k0 + lane * per + i;
        const float next = per == 1 ? __shfl_down_sync(FULL, v[0], 1) : v[i | 1];
        if ((k & 1) == 0 && k < end) row[k / 2] = static_cast<uint8_t>(static_cast<int>(v[i]) | (static_cast<int>(next) << 4));
    }
    if (lane == 0) {
        if (bad) scale = __uint_as_float(0x7fc00000u);
        const int64_t at = n * w.side_stride + gi;
        if (w.side_dt == DFLASH2_F32) {
            static_cast<float *>(w.scale)[at] = scale;
            if (w.zero) static_cast<float *>(w.zero)[at] = bad ? 8.0f : zero;
        } else {
            static_cast<uint16_t *>(w.scale)[at] = bf16_bits(scale);
            if (w.zero) static_cast<uint16_t *>(w.zero)[at] = bf16_bits(bad ? 8.0f : zero);
        }
    }
}

__device__ __forceinline__ float weight_at(const dflash2_weight4 &w, int64_t n, int64_t k) {
    const uint8_t b = static_cast<const uint8_t *>(w.codes)[n * w.code_stride + k / 2];
    const float code = static_cast<float>((k & 1) ? b >> 4 : b & 15);
    const int64_t at = n * w.side_stride + k / w.group;
    return (code - (w.zero ? side_at(w.zero, w.side_dt, at) : 8.0f)) * side_at(w.scale, w.side_dt, at);
}

__global__ void __launch_bounds__(256) k_dequant4(dflash2_weight4 w, void *out, dflash2_dtype dt, int64_t ld) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= w.N * w.K) return;
    const int64_t n = i / w.K, k = i % w.K;
    const float v = weight_at(w, n, k);
    if (dt == DFLASH2_F32) static_cast<float *>(out)[n * ld + k] = v;
    else static_cast<uint16_t *>(out)[n * ld + k] = bf16_bits(v);
}

// One warp per weight row and 8 rows of x.
__global__ void __launch_bounds__(256) k_linear4(const void *x, dflash2_dtype dt, int64_t rows, int64_t x_stride,
                                                 dflash2_weight4 w, void *y, dflash2_dtype y_dt, int64_t y_stride) {
    const int lane = threadIdx.x & 31;
    const int64_t n = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    if (n >= w.N) return;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 8;
    float acc[8] = {};
    for (int64_t k = lane; k < w.K; k += 32) {
        const float v = weight_at(w, n, k);
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (r0 + r < rows) {
                const float a = load_f(x, dt, (r0 + r) * x_stride + k);
                acc[r] = fmaf(isfinite(a) ? a : NAN, v, acc[r]);
            }
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const float v = warp_sum(acc[r]);
        if (lane == 0 && r0 + r < rows) {
            if (y_dt == DFLASH2_F32) static_cast<float *>(y)[(r0 + r) * y_stride + n] = v;
            else static_cast<uint16_t *>(y)[(r0 + r) * y_stride + n] = bf16_bits(v);
        }
    }
}

}  // namespace dfl

using namespace dfl;

extern "C" dflash2_status dflash2_quant4(const void *W, dflash2_dtype dt, int64_t ld, const dflash2_weight4 *w,
                                         dflash2_stream stream) {
    if (!dtype_ok(dt) || !weight4_ok(w) || ld < w->K) return DFLASH2_ERR_INVALID_ARG;
    if (w->N == 0) return DFLASH2_OK;
    if (!W || !aligned_to(W, dt)) return DFLASH2_ERR_INVALID_ARG;
    const int64_t G = groups_of(w), blocks = (w->N * G + 7) / 8;
    if (w->K > (int64_t(1) << 36) / w->N) return DFLASH2_ERR_UNSUPPORTED;
    k_quant4<<<static_cast<unsigned>(blocks), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(W, dt, ld, *w, G);
    return after_launch();
}

extern "C" dflash2_status dflash2_dequant4(const dflash2_weight4 *w, void *out, dflash2_dtype dt, int64_t ld,
                                           dflash2_stream stream) {
    if (!dtype_ok(dt) || !weight4_ok(w) || ld < w->K) return DFLASH2_ERR_INVALID_ARG;
    if (w->N == 0) return DFLASH2_OK;
    if (!out || !aligned_to(out, dt)) return DFLASH2_ERR_INVALID_ARG;
    const int64_t blocks = (w->N * w->K + 255) / 256;
    if (w->K > (int64_t(1) << 36) / w->N) return DFLASH2_ERR_UNSUPPORTED;
    k_dequant4<<<static_cast<unsigned>(blocks), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(*w, out, dt, ld);
    return after_launch();
}

extern "C" dflash2_status dflash2_linear4(const void *x, dflash2_dtype dt, int64_t rows, int64_t x_stride,
                                          const dflash2_weight4 *w, void *y, dflash2_dtype y_dt, int64_t y_stride,
                                          dflash2_stream stream) {
    if (!dtype_ok(dt) || !dtype_ok(y_dt) || (dt == DFLASH2_F32 && y_dt != DFLASH2_F32) || !weight4_ok(w) || rows < 0 ||
        x_stride < w->K || y_stride < w->N)
        return DFLASH2_ERR_INVALID_ARG;
    if (rows == 0 || w->N == 0) return DFLASH2_OK;
    if (!x || !y || !aligned_to(x, dt) || !aligned_to(y, y_dt)) return DFLASH2_ERR_INVALID_ARG;
    const int64_t by = (rows + 7) / 8;
    if (by > 65535) return DFLASH2_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>((w->N + 7) / 8), static_cast<unsigned>(by));
    k_linear4<<<grid, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(x, dt, rows, x_stride, *w, y, y_dt, y_stride);
    return after_launch();
}
