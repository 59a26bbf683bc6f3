// linear4.cuh -- what the two kernels of dflash2_linear4 share (linear4.cu: few
// rows; linear4_tc.cu: many).
//
// Codes are operands as they lie.  A bf16 whose exponent field is 0 or 1 is its
// low 8 bits times 2^-133 (subnormal, then the first normal binade), so
// w & 0x000f000f is a pair of codes times 2^-133 and w & 0x00f000f0 another pair
// times 2^-129: five instructions turn a word into four operand registers.  The
// rows of x are scaled by a power of two (largest entry near 2^126) and, at the
// second pairs' columns, by 2^-4; both are exact.  A word's eight columns stand
// in x in the order of its pairs, 0 4 1 5 2 6 3 7.
#pragma once

#include "weight4.cuh"

namespace dfl {

constexpr int L4_BLOCK = 128;  // columns of a block: 64 bytes of a row of codes

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }  // -126..127
// v * 2^e for e in -252..254
__device__ __forceinline__ float scale2(float v, int e) { return v * pow2f(e / 2) * pow2f(e - e / 2); }

// The exponent a row of x is scaled by, from the bits of its largest |x|: that ends up below 2^127.  133 - e is even, so
// that the product's power of two has a root.  133 where there is nothing to scale.
__device__ __forceinline__ int x_exponent(uint32_t top) {
    if (top >= 0x7f800000u || top == 0) return 133;
    const int e = (252 - static_cast<int>(top >> 23)) | 1;
    return e < 251 ? e : 251;
}
// The root of what a product with such a row is multiplied by; NaN for a row that is not finite.
__device__ __forceinline__ float x_root(uint32_t top, int e) { return top >= 0x7f800000u ? NAN : pow2f((133 - e) / 2); }

// Eight neighbours of a row of x, zeros from `left` on.
template <bool F32X>
__device__ __forceinline__ void load8(const void *x, int64_t at, int left, bool vec, float (&v)[8]) {
    if (left >= 8 && vec) {
        if (F32X) {
            const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(x) + at);
            const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(x) + at + 4);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + at);
            const uint32_t q[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) v[2 * i] = bf16lo(q[i]), v[2 * i + 1] = bf16hi(q[i]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? side_at(x, F32X ? DFLASH2_F32 : DFLASH2_BF16, at + i) : 0.0f;
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Packed bf16 arithmetic, each half rounded once; subnormals are kept.
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// A number of bf16, twice.
__device__ __forceinline__ uint32_t pair_of(float v) {
    const uint32_t h = __float_as_uint(v) >> 16;
    return h | h << 16;
}

// Eight columns of a row scaled for the operand (exponent e, odd; no infinities); returns their sum in the product's units.
__device__ __forceinline__ float scale8(float (&v)[8], int e) {
    const float f1 = pow2f(e >> 1), f2 = pow2f(e - (e >> 1)), f3 = pow2f(e - (e >> 1) - 4);
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] *= f1;  // below 2^64, so that sums of a group do not overflow
        sum += v[j];
        v[j] *= (j & 1) ? f3 : f2;
    }
    return sum * pow2f((e - 133) / 2 - (e >> 1) / 2) * pow2f(e - 133 - (e >> 1) - ((e - 133) / 2 - (e >> 1) / 2));
}

// Many rows (linear4_tc.cu).
size_t linear4_tc_bytes(bool f32x, int64_t rows, int64_t K);
dflash2_status linear4_tc(const void *x, bool f32x, int64_t rows, int64_t x_stride, const dflash2_weight4 *w, void *y,
                          dflash2_dtype y_dt, int64_t y_stride, bool exact, void *ws, cudaStream_t s);

}  // namespace dfl
