// weight4.cuh -- weights held in 4 bits: what a dflash2_weight4 stands for, and
// its checks.
//
// A row of N x K weights is cut into groups of 32, 64 or 128 neighbours (the
// last one may be short).  Weight (n, k) is (code - zero) * scale with the
// group's scale and zero point (8 where the record has none); the code of an
// even k is the low half of its byte.  Rows of codes start on 16-byte
// boundaries and are padded to 16 bytes (32 codes).
#pragma once

#include "common.cuh"
#include "host.hpp"

namespace dfl {

__device__ __forceinline__ float side_at(const void *p, dflash2_dtype dt, int64_t i) {
    if (dt == DFLASH2_F32) return static_cast<const float *>(p)[i];
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(p)[i]) << 16);
}

// The same in two steps: bits now, the number where it is needed (a conversion would wait for the load).
__device__ __forceinline__ uint32_t side_bits(const void *p, dflash2_dtype dt, int64_t i) {
    return dt == DFLASH2_F32 ? static_cast<const uint32_t *>(p)[i] : static_cast<const uint16_t *>(p)[i];
}
__device__ __forceinline__ float side_of(uint32_t bits, dflash2_dtype dt) {
    return __uint_as_float(dt == DFLASH2_F32 ? bits : bits << 16);
}

// f32 to bf16, nearest, ties to even; NaN to a quiet NaN.
__device__ __forceinline__ uint16_t bf16_bits(float v) {
    uint16_t h;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
    return h;
}

inline bool aligned_to(const void *p, dflash2_dtype dt) { return reinterpret_cast<uintptr_t>(p) % esize(dt) == 0; }

inline int64_t groups_of(const dflash2_weight4 *w) { return (w->K + w->group - 1) / w->group; }

// A record's sizes and pointers.  Whatever is not read or written is not looked at.
inline bool weight4_ok(const dflash2_weight4 *w) {
    return w && w->N >= 0 && w->K >= 1 && w->N <= 0x7fffffff && w->K <= 0x7fffffff - 128 &&
           (w->group == 32 || w->group == 64 || w->group == 128) && dtype_ok(w->side_dt) &&
           w->code_stride % 16 == 0 && w->code_stride >= (w->K + 31) / 32 * 16 && w->side_stride >= groups_of(w) &&
           (w->N == 0 || (w->codes && w->scale && aligned16(w->codes) && aligned_to(w->scale, w->side_dt) &&
                           aligned_to(w->zero, w->side_dt)));
}

}  // namespace dfl
