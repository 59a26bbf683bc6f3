// linear4.cu -- dflash2_quant4, dflash2_dequant4 and dflash2_linear4: weights in
// 4 bits with a scale (and a zero point) per group, and products with them.
//
// TensorRT-LLM issue 18085 and FreeToken PR 857 run this path for targets and
// drafters whose weights are held in 4 bits; the pages name the formats and give
// no kernel.
#include "linear4.cuh"
#include "tc.cuh"

namespace dfl {

// ----------------------------------------------------- to codes and back ----
constexpr float Q4_MAGIC = 12582912.0f;  // 1.5 * 2^23: adding it rounds to a whole number

struct Quant4 {
    const void *W;
    dflash2_weight4 w;
    int64_t ld;
    uint32_t pieces;  // of 32 columns in a row, whole groups
    uint32_t all;     // of them in all rows
    int codes;        // vectors of 8 columns that have a place in a row
    int span_log2;    // log2 of the lanes to a row (back)
    int part;         // vectors of a row to a warp (back), a multiple of what it reads at once
    bool vec;
};

// 32 columns to a thread, so that what a group costs (a scale and two or three divisions) is shared by as many; a group is
// 4, 2 or 1 neighbouring lanes.  A quotient's whole number comes from the product with the reciprocal; where that (off by
// at most 2^-18) is next to a half, the entry is read again and divided.
// 151936 x 2560 bf16: 264 us (3.7 TB/s), with zero points 299 us.  Bound by instruction issue (2.6 a cycle, about 15 to an
// entry).  One entry to a thread with a division each, the two directions of a head took 3.9 ms, now 0.46.
template <bool F32W, int LG, bool ZERO>
__global__ void __launch_bounds__(256) k_quant4(const Quant4 p) {
    constexpr int LANES = 4 >> LG;
    const uint32_t item = blockIdx.x * 256u + threadIdx.x;
    const bool row = item < p.all;
    const uint32_t n32 = row ? item / p.pieces : 0, c = item - n32 * p.pieces;
    const int64_t n = n32, k0 = static_cast<int64_t>(c) * 32, base = n * p.ld + k0;
    const int left = !row || k0 >= p.w.K ? 0 : p.w.K - k0 < 32 ? static_cast<int>(p.w.K - k0) : 32;
    float v[32];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float(&o)[8] = *reinterpret_cast<float(*)[8]>(v + q * 8);
        if (left > q * 8) load8<F32W>(p.W, base + q * 8, left - q * 8, p.vec, o);
        else
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = 0.0f;
    }
    // NaN propagates through the maxima, infinities are the largest
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        hi = fmax_nan(hi, ZERO ? v[j] : fabsf(v[j]));
        if (ZERO) lo = -fmax_nan(-lo, -v[j]);
    }
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) {
        hi = fmax_nan(hi, __shfl_xor_sync(FULL, hi, d));
        if (ZERO) lo = -fmax_nan(-lo, -__shfl_xor_sync(FULL, lo, d));
    }
    if (!row) return;
    const bool bad = !(fmax_nan(hi, -lo) < __builtin_huge_valf());
    float scale = ZERO ? __fsub_rn(__fdiv_rn(hi, 15.0f), __fdiv_rn(lo, 15.0f)) : __fdiv_rn(hi, 7.0f);
    if (p.w.side_dt == DFLASH2_BF16) scale = __uint_as_float(static_cast<uint32_t>(bf16_bits(scale)) << 16);
    const float step = scale == 0.0f ? 1.0f : scale, inv = __frcp_rn(step);
    const float zero = ZERO ? fminf(fmaxf(rintf(__fdiv_rn(-lo, step)), 0.0f), 15.0f) : 8.0f;
    // Past 2^-123, where a scale has its full bits, quotients without zero points stay within 7.1: nothing to clamp.  Four
    // codes are added up as one float below 2^24.
    uint32_t word[4], open = step > 1e-37f ? 0u : FULL;
    const float most = 15.0f - zero;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float four[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            four[h] = 8388608.0f + zero * 4369.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = v[q * 8 + h * 4 + j], r = __fadd_rn(fmaf(x, inv, Q4_MAGIC), -Q4_MAGIC);
                if (!(fabsf(fmaf(x, inv, -r)) < 0.49999f)) open |= 1u << (q * 8 + h * 4 + j);
                const float held = ZERO ? fminf(fmaxf(r, -zero), most) : r;
                four[h] = fmaf(held, static_cast<float>(1 << (4 * j)), four[h]);
            }
        }
        word[q] = (__float_as_uint(four[0]) & 0xffffu) | (__float_as_uint(four[1]) << 16);
    }
    if (left < 32) open &= (1u << left) - 1;
    if (bad) open = 0;
    while (open) {
        const int j = __ffs(open) - 1;
        open &= open - 1;
        const float q = rintf(__fdiv_rn(side_at(p.W, F32W ? DFLASH2_F32 : DFLASH2_BF16, base + j), step));
        const uint32_t code = static_cast<uint32_t>(fminf(fmaxf(q + zero, 0.0f), 15.0f)) << (4 * (j & 7)), keep = ~(15u << (4 * (j & 7)));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (j >> 3 == i) word[i] = (word[i] & keep) | code;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int have = left - q * 8;  // the codes behind the row are 8
        if (bad || have <= 0) word[q] = 0x88888888u;
        else if (have < 8) word[q] = (word[q] & ((1u << (4 * have)) - 1)) | (0x88888888u << (4 * have));
    }
    if (left > 0)
        *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.w.codes) + n * p.w.code_stride + k0 / 2) =
            make_uint4(word[0], word[1], word[2], word[3]);
    if (c % LANES == 0) {
        const float s = bad ? __uint_as_float(0x7fc00000u) : scale, z = bad ? 8.0f : zero;
        const int64_t at = n * p.w.side_stride + c / LANES;
        if (p.w.side_dt == DFLASH2_F32) {
            static_cast<float *>(p.w.scale)[at] = s;
            if (p.w.zero) static_cast<float *>(p.w.zero)[at] = z;
        } else {
            static_cast<uint16_t *>(p.w.scale)[at] = bf16_bits(s);
            if (p.w.zero) static_cast<uint16_t *>(p.w.zero)[at] = bf16_bits(z);
        }
    }
}

// Eight columns to a thread (4 bytes of codes, 16 of bf16); a warp takes a row, or several short ones, or a part of a long
// one where rows are few, and reads Q4_AHEAD vectors before it works on them.  151936 x 2560 to bf16: 146 us (6.7 TB/s),
// HBM-bound; in f32 arithmetic throughout it took 30 us more.
//
// VEC: the rows start on 16-byte boundaries.  Where they do not, a warp's 256 values take their places in shared memory and
// are written as neighbours by neighbouring lanes (152001 x 2561: 456 us, by the lanes that have them 949).
constexpr int Q4_AHEAD = 4;
template <bool F32W, int LG, bool VEC>
__global__ void __launch_bounds__(256) k_dequant4(const Quant4 p, void *out) {
    constexpr int LANES = 16 >> LG;
    const int lane = threadIdx.x & 31, span = 1 << p.span_log2;
    const int64_t n = (((static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5) << (5 - p.span_log2)) + (lane >> p.span_log2);
    const int first = static_cast<int>(blockIdx.y) * p.part, end = min(first + p.part, p.codes);
    if constexpr (!VEC) {
        __shared__ float4 place[8][64];
        const int64_t n0 = n - (lane >> p.span_log2);
        float4 *mine = place[threadIdx.x >> 5];
        for (int c0 = first; c0 < end; c0 += span) {
            const int c = c0 + (lane & (span - 1));
            float v[8] = {};
            if (n < p.w.N && static_cast<int64_t>(c) * 8 < p.w.K) {
                const uint32_t word = *reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(p.w.codes) +
                                                                          n * p.w.code_stride + static_cast<int64_t>(c) * 4);
                const int64_t at = n * p.w.side_stride + c / LANES;
                const float s = side_at(p.w.scale, p.w.side_dt, at), z = p.w.zero ? side_at(p.w.zero, p.w.side_dt, at) : 8.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = (static_cast<float>((word >> (4 * j)) & 15u) - z) * s;
            }
            __syncwarp();  // the last values have been read
            mine[lane * 2] = make_float4(v[0], v[1], v[2], v[3]), mine[lane * 2 + 1] = make_float4(v[4], v[5], v[6], v[7]);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int e = j * 32 + lane, from = e >> 3;
                const int64_t row = n0 + (from >> p.span_log2), k = static_cast<int64_t>(c0 + (from & (span - 1))) * 8 + (e & 7);
                const float o = reinterpret_cast<const float *>(mine)[e];
                if (row < p.w.N && k < p.w.K) {
                    if (F32W) static_cast<float *>(out)[row * p.ld + k] = o;
                    else static_cast<uint16_t *>(out)[row * p.ld + k] = bf16_bits(o);
                }
            }
        }
        return;
    }
    if (n >= p.w.N) return;
    const uint8_t *codes = static_cast<const uint8_t *>(p.w.codes) + n * p.w.code_stride;
    for (int c0 = first + (lane & (span - 1)); c0 < end; c0 += span * Q4_AHEAD) {
        uint32_t word[Q4_AHEAD], sb[Q4_AHEAD], zb[Q4_AHEAD];
#pragma unroll
        for (int i = 0; i < Q4_AHEAD; ++i) {
            const int c = c0 + i * span;
            const int64_t at = n * p.w.side_stride + c / LANES;
            word[i] = sb[i] = zb[i] = 0;
            if (static_cast<int64_t>(c) * 8 < p.w.K) {
                word[i] = *reinterpret_cast<const uint32_t *>(codes + c * 4);
                sb[i] = side_bits(p.w.scale, p.w.side_dt, at);
                if (p.w.zero) zb[i] = side_bits(p.w.zero, p.w.side_dt, at);
            }
        }
#pragma unroll
        for (int i = 0; i < Q4_AHEAD; ++i) {
            const int c = c0 + i * span;
            const int64_t left = p.w.K - static_cast<int64_t>(c) * 8, at = n * p.ld + static_cast<int64_t>(c) * 8;
            if (left <= 0) break;
            const float s = side_of(sb[i], p.w.side_dt), z = p.w.zero ? side_of(zb[i], p.w.side_dt) : 8.0f;
            if (!F32W && left >= 8 && p.w.side_dt == DFLASH2_BF16 && fabsf(s) < 1e30f &&
                (!p.w.zero || (fabsf(z) <= 128.0f && z == rintf(z)))) {
                // In packed bf16: 128 + code is a number whose low bits are the code, code - zero is exact for whole zero
                // points up to 128, and one rounding is left.
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t c2 = sub_bf16x2(((word[i] >> (4 * j)) & 0x000f000fu) | 0x43004300u, 0x43004300u);
                    o[j] = mul_bf16x2(sub_bf16x2(c2, pair_of(z)), pair_of(s));
                }
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at) =
                    make_uint4(__byte_perm(o[0], o[1], 0x5410), __byte_perm(o[2], o[3], 0x5410), __byte_perm(o[0], o[1], 0x7632),
                               __byte_perm(o[2], o[3], 0x7632));
                continue;
            }
            float v[8];
            // 2^23 + code is a float whose low bits are the code
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(((word[i] >> (4 * j)) & 15u) | 0x4b000000u);
            if (p.w.zero) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = ((v[j] - 8388608.0f) - z) * s;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = (v[j] - 8388616.0f) * s;
            }
            if (left >= 8) {
                if (F32W) {
                    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(out) + at);
                    o[0] = make_float4(v[0], v[1], v[2], v[3]), o[1] = make_float4(v[4], v[5], v[6], v[7]);
                } else {
                    uint4 o;
                    o.x = bf16_pair(v[0], v[1]), o.y = bf16_pair(v[2], v[3]), o.z = bf16_pair(v[4], v[5]), o.w = bf16_pair(v[6], v[7]);
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at) = o;
                }
            } else {
                for (int j = 0; j < 8 && j < left; ++j) {
                    if (F32W) static_cast<float *>(out)[at + j] = v[j];
                    else static_cast<uint16_t *>(out)[at + j] = bf16_bits(v[j]);
                }
            }
        }
    }
}

// ---------------------------------------------------------- few rows: mma ----
// y = x . W^T for a few rows of x, bound by reading the codes once.
//
// A warp takes tiles of 16 weight rows in blocks of 128 columns (1 KB of codes
// by cp.async, L4_STAGES blocks ahead) and multiplies them with up to 32 rows
// of x by mma.sync m16n8k16 (x on the n side, 8 rows a tile): the codes go from
// shared memory into the operand's registers with no second trip.
//
//   Codes are operands as they lie (linear4.cuh).
//   A group of columns is summed from zero, so that
//     acc += scale * (sum of code * x - zero * sum of x)
//   in f32: products of a code and a bf16 are exact.  f32 rows are split into
//   three bf16 parts, which is exact too.
//
// The CTA's range of x stays in shared memory for all its tiles.  Few tiles are
// cut along K: over the warps of a CTA (kw), then over a cluster (ks CTAs, read
// back through distributed shared memory); parts are added in order.
//
// 151936 x 5120, one row: 77 us (5.2 TB/s).  Bound by instruction issue: about
// 150 for a block of 1 KB, most of them masks and shifts that share one pipe;
// three CTAs to an SM leave too few registers for the copies (112 us).  Eight
// rows 99 us: the same and the MMAs' operands of x.  Few tiles are bound by
// their latency (2560 x 2560, one row: 6.2 us).  25 to 32 rows at a time spill 20 to 32
// bytes at 128 registers.
constexpr int L4_THREADS = 256;
constexpr int L4_WARPS = L4_THREADS / 32;
constexpr int L4_STAGES = 4;
constexpr int64_t L4_MAX_K = 1 << 17, L4_MAX_ROWS = 1 << 19;
constexpr int64_t L4_MANY_ROWS = 9;
constexpr int64_t L4_LONG_ROWS = 1 << 15, L4_LONG_K = 1 << 13;
constexpr int L4_SMEM_MAX = 226 * 1024;

struct Lin4 {
    const void *x;
    int64_t rows, x_stride;
    dflash2_weight4 w;
    void *y;
    int64_t y_stride;
    dflash2_dtype y_dt;
    int G;          // groups in a row
    int gpb_log2;   // log2 of the groups in a block (the kernels' LG)
    int rb;         // rows of x to a CTA
    int kblocks;    // blocks in a row
    int kper;       // blocks of the largest range of a CTA
    int kw_log2;    // log2 of the warps that share a tile
    int ks;         // CTAs that share a tile
    int64_t tiles;
};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void lds32(uint32_t at, uint32_t (&v)[1]) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[0]) : "r"(at));
}
__device__ __forceinline__ void lds64(uint32_t at, uint32_t (&v)[2]) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(at));
}
__device__ __forceinline__ void lds128(uint32_t at, uint32_t (&v)[4]) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at));
}

// Floats of the cross-warp sums: [row of x][16 + 1] per warp.
__host__ __device__ constexpr int l4_red(int nt) { return nt * 8 * 17; }

// LG: log2 of the groups in a block.
template <int NT, int LG, bool F32X>
__global__ void __launch_bounds__(L4_THREADS, 2) k_linear4_mma(const Lin4 p) {
    constexpr int PARTS = F32X ? 3 : 1, GPB = 1 << LG, WPG = 4 >> LG;  // words of a thread in a group's row
    extern __shared__ __align__(128) unsigned char raw[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int rank = p.ks > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * p.rb;
    const int nr = static_cast<int>(p.rows - r0 < p.rb ? p.rows - r0 : p.rb);
    const int kb_lo = p.kblocks * rank / p.ks, nkb = p.kblocks * (rank + 1) / p.ks - kb_lo;
    const uint32_t pitch = static_cast<uint32_t>(p.kper) * (L4_BLOCK * 2) + 64;  // 64 past 128: rows take turns in the banks
    const int sums_ld = NT * 8 + 2;
    unsigned char *ring = raw;
    float *red = reinterpret_cast<float *>(ring + L4_WARPS * L4_STAGES * 1024);
    float *xsum = red + ((p.kw_log2 || p.ks > 1) ? L4_WARPS * l4_red(NT) : 0);  // [group][sums_ld]
    float *half = xsum + p.kper * GPB * sums_ld;                                // [NT * 8]: root of the power of two
    uint32_t *top = reinterpret_cast<uint32_t *>(half + NT * 8);                // [NT * 8]: bits of the largest |x|
    unsigned char *xs = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(top + NT * 8) + 127) & ~static_cast<uintptr_t>(127));

    // ---- this warp's tiles and blocks
    const int kw = 1 << p.kw_log2, sub = warp & (kw - 1);
    const int kb0 = nkb * sub / kw, count = nkb * (sub + 1) / kw - kb0;  // within the CTA's range
    const int64_t step = static_cast<int64_t>(gridDim.x / p.ks) * (L4_WARPS >> p.kw_log2);
    const int64_t first = static_cast<int64_t>(blockIdx.x / p.ks) * (L4_WARPS >> p.kw_log2) + (warp >> p.kw_log2);
    const int row_bytes = static_cast<int>((p.w.K + 31) / 32 * 16);
    const int at0 = (kb_lo + kb0) * (L4_BLOCK / 2);
    // row of the tile that this lane copies (and r + 8), and where the copy lands; the swizzle spreads the reads below
    const uint32_t copy_to = smem_addr(ring) + warp * (L4_STAGES * 1024) + g * 64 +
                             ((t ^ (LG == 0 ? 0 : LG == 1 ? g & 2 : (g >> 1) & 3)) << 4);
    int64_t c_tile = first;  // the block to copy next
    int c_left = 0;
    const unsigned char *c0 = nullptr, *c1 = nullptr;
    int c_at = 0;
    auto copy = [&](uint32_t stage) {
        if (c_left == 0 && c_tile < p.tiles && count) {
            int64_t n0 = c_tile * 16 + g, n1 = n0 + 8;
            n0 = n0 < p.w.N ? n0 : p.w.N - 1, n1 = n1 < p.w.N ? n1 : p.w.N - 1;
            c0 = static_cast<const unsigned char *>(p.w.codes) + n0 * p.w.code_stride + at0 + t * 16;
            c1 = static_cast<const unsigned char *>(p.w.codes) + n1 * p.w.code_stride + at0 + t * 16;
            c_at = at0 + t * 16;
            c_left = count;
            c_tile += step;
        }
        if (c_left) {
            const bool take = c_at < row_bytes;
            const void *q = p.w.codes;
            cp_async16(copy_to + stage, take ? c0 : q, take);
            cp_async16(copy_to + stage + 512, take ? c1 : q, take);
            c0 += 64, c1 += 64, c_at += 64, --c_left;
        }
        cp_async_commit();
    };
    // scales and zero points, four groups (a quad's lane each) at a time, one step ahead
    int64_t s_tile = first;
    int s_left = 0, s_gi = 0;
    int64_t s_at0 = 0, s_at1 = 0;
    uint32_t sn0 = 0, sn1 = 0, zn0 = 0, zn1 = 0;
    auto sides = [&]() {
        if (s_left == 0 && s_tile < p.tiles && count) {
            int64_t n0 = s_tile * 16 + g, n1 = n0 + 8;
            n0 = n0 < p.w.N ? n0 : p.w.N - 1, n1 = n1 < p.w.N ? n1 : p.w.N - 1;
            s_gi = (kb_lo + kb0) * GPB + t;
            s_at0 = n0 * p.w.side_stride + s_gi, s_at1 = n1 * p.w.side_stride + s_gi;
            s_left = (count * GPB + 3) / 4;
            s_tile += step;
        }
        if (s_left) {
            sn0 = sn1 = zn0 = zn1 = 0;
            if (s_gi < p.G) {
                sn0 = side_bits(p.w.scale, p.w.side_dt, s_at0), sn1 = side_bits(p.w.scale, p.w.side_dt, s_at1);
                if (p.w.zero) zn0 = side_bits(p.w.zero, p.w.side_dt, s_at0), zn1 = side_bits(p.w.zero, p.w.side_dt, s_at1);
            }
            s_gi += 4, s_at0 += 4, s_at1 += 4, --s_left;
        }
    };
    const int chunks = nkb * (L4_BLOCK / 8);
    const bool vec = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.x_stride * (F32X ? 4 : 2) % 16 == 0;
    const bool staged = !F32X && vec;  // the range of x comes to its place as it is, and is worked on there
    if (staged) {
        for (int i = threadIdx.x; i < nr * chunks; i += L4_THREADS) {
            const int r = i / chunks, c = i - r * chunks, k = c * 8 + kb_lo * L4_BLOCK;
            const int left = static_cast<int>(p.w.K) - k, bytes = left <= 0 ? 0 : left < 8 ? left * 2 : 16;
            const void *src = static_cast<const uint16_t *>(p.x) + (r0 + r) * p.x_stride + (bytes ? k : 0);
            asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(xs) + r * pitch + c * 16), "l"(src),
                         "r"(bytes)
                         : "memory");
        }
        cp_async_commit();
    }
#pragma unroll
    for (int s = 0; s < L4_STAGES - 1; ++s) copy(s * 1024);
    sides();

    // ---- x: largest entry of each row, then scaled, split, reordered, and its group sums
    if (threadIdx.x < NT * 8) top[threadIdx.x] = 0;
    if (staged) cp_async_wait<L4_STAGES - 1>();  // x was asked for first
    __syncthreads();
    auto take8 = [&](int r, int c, float (&v)[8]) {
        if (staged) {
            uint32_t q[4];
            lds128(smem_addr(xs) + r * pitch + c * 16, q);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[2 * i] = bf16lo(q[i]), v[2 * i + 1] = bf16hi(q[i]);
        } else {
            const int k = c * 8 + kb_lo * L4_BLOCK;
            load8<F32X>(p.x, (r0 + r) * p.x_stride + k, static_cast<int>(p.w.K) - k, vec, v);
        }
    };
    // rows are dealt to the warps, or the warps to the rows
    int wpr = L4_WARPS;
    while (wpr > 1 && wpr / 2 >= (L4_WARPS + nr - 1) / nr) wpr /= 2;
    const int x_first = (warp & (wpr - 1)) * 32 + lane, x_step = wpr * 32, x_rows = L4_WARPS / wpr;
    for (int r = warp / wpr; r < nr; r += x_rows) {
        uint32_t m = 0;
#pragma unroll 2
        for (int c = x_first; c < chunks; c += x_step) {
            float v[8];
            take8(r, c, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
        }
        m = __reduce_max_sync(FULL, m);
        if (lane == 0) atomicMax(&top[r], m);
    }
    __syncthreads();
    if (threadIdx.x < nr) {
        const uint32_t m = top[threadIdx.x];
        const int e = x_exponent(m);
        half[threadIdx.x] = x_root(m, e);
        top[threadIdx.x] = static_cast<uint32_t>(e);
    }
    __syncthreads();
    for (int r = warp / wpr; r < nr; r += x_rows)
#pragma unroll 2
    for (int c = x_first; c < chunks; c += x_step) {  // a range has a multiple of 16 chunks: half-warps stay whole
        float v[8];
        take8(r, c, v);
        if (isnan(half[r])) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        }
        float sum = scale8(v, static_cast<int>(top[r]));
        constexpr int LANES = 16 >> LG;  // chunks of a group
#pragma unroll
        for (int d = LANES >> 1; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffu << (lane & 16), sum, d);
        if ((c & (LANES - 1)) == 0) xsum[c / LANES * sums_ld + r] = sum;
        // where thread t finds its j-th word's columns: the words of a group lie WPG to a thread.  A block is written over
        // by the half-warp that has just read it.
        const int cc = c & 15, cg = cc / LANES, ci = cc % LANES;
        unsigned char *dst = xs + r * pitch + ((c & ~15) + (cg * WPG + ci % WPG) * 4 + ci / WPG) * 16;
        __syncwarp(0xffffu << (lane & 16));
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
            uint4 o;
            uint32_t *ow = &o.x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                ow[j] = bf16_pair(v[j], v[j + 4]);
                if (PARTS > 1) v[j] -= bf16lo(ow[j]), v[j + 4] -= bf16hi(ow[j]);
            }
            *reinterpret_cast<uint4 *>(dst + static_cast<size_t>(q) * p.rb * pitch) = o;
        }
    }
    __syncthreads();

    // ---- tiles
    uint32_t xb[NT];
    float hf[NT][2];
#pragma unroll
    for (int q = 0; q < NT; ++q) {
        const int r = q * 8 + g;
        xb[q] = smem_addr(xs) + (r < nr ? r : nr - 1) * pitch + t * 16 + kb0 * (L4_BLOCK * 2);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = q * 8 + 2 * t + j;
            hf[q][j] = half[c < nr ? c : nr - 1];
        }
    }
    uint32_t words[WPG == 4 ? 1 : GPB];  // where this lane's words of a group lie in a block
#pragma unroll
    for (int j = 0; j < (WPG == 4 ? 1 : GPB); ++j)
        words[j] = smem_addr(ring) + warp * (L4_STAGES * 1024) + g * 64 +
                   (LG == 0   ? t * 16
                    : LG == 1 ? ((((2 * j + (t >> 1)) ^ (g & 2)) << 4) + (t & 1) * 8)
                              : (((j ^ ((g >> 1) & 3)) << 4) + t * 4));
    const float *sums0 = xsum + kb0 * GPB * sums_ld + 2 * t;
    uint32_t s = 0, s_next = (L4_STAGES - 1) * 1024;  // stage of the next block, and of the next copy
    for (int64_t tile0 = first - (warp >> p.kw_log2); tile0 < p.tiles; tile0 += step) {
        const int64_t tile = tile0 + (warp >> p.kw_log2);
        float acc[NT][4];
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[q][j] = 0.0f;
        if (tile < p.tiles) {
            float sd0 = 0.0f, sd1 = 0.0f, zr0 = 8.0f, zr1 = 8.0f;
            const float *sums = sums0;
            uint32_t xo = 0;
            for (int i = 0; i < count; ++i, xo += L4_BLOCK * 2) {
                copy(s_next);
                if (LG == 2 || (i & (WPG - 1)) == 0) {
                    sd0 = side_of(sn0, p.w.side_dt), sd1 = side_of(sn1, p.w.side_dt);
                    if (p.w.zero) zr0 = side_of(zn0, p.w.side_dt), zr1 = side_of(zn1, p.w.side_dt);
                    sides();
                }
                cp_async_wait<L4_STAGES - 1>();
                __syncwarp();
#pragma unroll
                for (int j = 0; j < GPB; ++j, sums += sums_ld) {
                    uint32_t wl[WPG], wh[WPG];
                    if constexpr (LG == 0) {
                        lds128(words[0] + s, wl), lds128(words[0] + s + 512, wh);
                    } else if constexpr (LG == 1) {
                        lds64(words[j] + s, wl), lds64(words[j] + s + 512, wh);
                    } else {
                        lds32(words[j] + s, wl), lds32(words[j] + s + 512, wh);
                    }
                    const int from = (lane & ~3) | (LG == 2 ? j : ((i << LG) + j) & 3);
                    const float s0 = __shfl_sync(FULL, sd0, from), s1 = __shfl_sync(FULL, sd1, from);
                    float z0 = 8.0f, z1 = 8.0f;
                    if (p.w.zero) z0 = __shfl_sync(FULL, zr0, from), z1 = __shfl_sync(FULL, zr1, from);
                    // the sum starts at - zero * sum of x
                    float part[NT][4];
#pragma unroll
                    for (int q = 0; q < NT; ++q) {
                        const float2 xg = *reinterpret_cast<const float2 *>(sums + q * 8);
                        part[q][0] = -z0 * xg.x, part[q][1] = -z0 * xg.y;
                        part[q][2] = -z1 * xg.x, part[q][3] = -z1 * xg.y;
                    }
#pragma unroll
                    for (int v = 0; v < WPG; ++v) {
                        const uint32_t ul = wl[v] >> 8, uh = wh[v] >> 8;
#pragma unroll
                        for (int q = 0; q < NT; ++q)
#pragma unroll
                            for (int h = 0; h < PARTS; ++h) {
                                uint32_t b[4];
                                lds128(xb[q] + h * p.rb * pitch + xo + (j * WPG + v) * 64, b);
                                mma_16816(part[q], wl[v] & 0x000f000fu, wh[v] & 0x000f000fu, wl[v] & 0x00f000f0u,
                                          wh[v] & 0x00f000f0u, b[0], b[1]);
                                mma_16816(part[q], ul & 0x000f000fu, uh & 0x000f000fu, ul & 0x00f000f0u,
                                          uh & 0x00f000f0u, b[2], b[3]);
                            }
                    }
#pragma unroll
                    for (int q = 0; q < NT; ++q) {
                        acc[q][0] = fmaf(s0, part[q][0], acc[q][0]), acc[q][1] = fmaf(s0, part[q][1], acc[q][1]);
                        acc[q][2] = fmaf(s1, part[q][2], acc[q][2]), acc[q][3] = fmaf(s1, part[q][3], acc[q][3]);
                    }
                }
                __syncwarp();
                s_next = s;
                s = s == (L4_STAGES - 1) * 1024 ? 0 : s + 1024;
            }
#pragma unroll
            for (int q = 0; q < NT; ++q)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[q][j] = acc[q][j] * hf[q][j & 1] * hf[q][j & 1];
        }
        if (kw == 1 && p.ks == 1) {
            if (tile < p.tiles)
#pragma unroll
                for (int q = 0; q < NT; ++q)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int c = q * 8 + 2 * t + (j & 1);
                        const int64_t n = tile * 16 + g + (j >> 1) * 8;
                        if (c < nr && n < p.w.N) {
                            const int64_t at = (r0 + c) * p.y_stride + n;
                            if (p.y_dt == DFLASH2_F32) static_cast<float *>(p.y)[at] = acc[q][j];
                            else static_cast<uint16_t *>(p.y)[at] = bf16_bits(acc[q][j]);
                        }
                    }
            continue;
        }
        // parts of a tile: the warps of a CTA in order, then the CTAs of the cluster in order
        float *mine = red + warp * l4_red(NT);
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int j = 0; j < 4; ++j) mine[(q * 8 + 2 * t + (j & 1)) * 17 + g + (j >> 1) * 8] = acc[q][j];
        if (p.ks > 1) cluster_sync();
        else __syncthreads();
        const int per_tile = nr * 16, here = (L4_WARPS >> p.kw_log2) * per_tile;
        for (int i = threadIdx.x + rank * L4_THREADS; i < here; i += L4_THREADS * p.ks) {
            const int slot = i / per_tile, c = (i - slot * per_tile) >> 4, n16 = i & 15;
            const int64_t n = (tile0 + slot) * 16 + n16;
            float v = 0.0f;
            for (int q = 0; q < p.ks; ++q)
                for (int w = 0; w < kw; ++w) {
                    const float *src = red + ((slot << p.kw_log2) + w) * l4_red(NT) + c * 17 + n16;
                    if (p.ks > 1) {
                        uint32_t remote;
                        float f;
                        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr(src)), "r"(q));
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(remote));
                        v += f;
                    } else {
                        v += *src;
                    }
                }
            if (n < p.w.N) {
                const int64_t at = (r0 + c) * p.y_stride + n;
                if (p.y_dt == DFLASH2_F32) static_cast<float *>(p.y)[at] = v;
                else static_cast<uint16_t *>(p.y)[at] = bf16_bits(v);
            }
        }
        if (p.ks > 1) cluster_sync();
        else __syncthreads();
    }
    cp_async_wait<0>();
}

// ------------------------------------------------------------------ host ----
// Shared memory of a CTA.
static size_t l4_smem(const Lin4 &p, int nt, int parts) {
    size_t b = static_cast<size_t>(L4_WARPS) * L4_STAGES * 1024;
    if (p.kw_log2 || p.ks > 1) b += static_cast<size_t>(L4_WARPS) * l4_red(nt) * 4;
    b += (static_cast<size_t>(p.kper << p.gpb_log2) * (nt * 8 + 2) + 2 * nt * 8) * 4 + 128;
    return b + (static_cast<size_t>(p.kper) * (L4_BLOCK * 2) + 64) * p.rb * parts;
}

template <int NT, int LG, bool F32X>
static dflash2_status launch_l4(const Lin4 &p, size_t smem, unsigned gx, unsigned gy, cudaStream_t s) {
    auto fn = &k_linear4_mma<NT, LG, F32X>;
    {
        static int opted[64] = {0};
        static std::mutex mu;
        const int dev = current_device();
        std::lock_guard<std::mutex> lock(mu);
        if (dev < 0 || dev >= 64 || !opted[dev]) {
            if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, L4_SMEM_MAX) != cudaSuccess)
                return DFLASH2_ERR_CUDA;
            if (dev >= 0 && dev < 64) opted[dev] = 1;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(gx, gy, 1);
    cfg.blockDim = dim3(L4_THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(p.ks);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.ks > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, fn, p) != cudaSuccess) return DFLASH2_ERR_CUDA;
    return after_launch();
}

template <int NT, bool F32X>
static dflash2_status launch_l4_groups(const Lin4 &p, size_t smem, unsigned gx, unsigned gy, cudaStream_t s) {
    if (p.gpb_log2 == 0) return launch_l4<NT, 0, F32X>(p, smem, gx, gy, s);
    if (p.gpb_log2 == 1) return launch_l4<NT, 1, F32X>(p, smem, gx, gy, s);
    return launch_l4<NT, 2, F32X>(p, smem, gx, gy, s);
}

static dflash2_status linear4_mma(Lin4 p, bool f32x, cudaStream_t s) {
    const int parts = f32x ? 3 : 1;
    const int most_rows = f32x ? 16 : 32;
    p.rb = static_cast<int>(p.rows < most_rows ? p.rows : most_rows);
    if (p.rows > most_rows) {  // even blocks of rows
        const int64_t nb = (p.rows + most_rows - 1) / most_rows;
        p.rb = static_cast<int>((p.rows + nb - 1) / nb);
    }
    p.tiles = (p.w.N + 15) / 16;
    p.kblocks = static_cast<int>((p.w.K + L4_BLOCK - 1) / L4_BLOCK);
    const int64_t sms = sm_count();
    // The split with the least estimated time (in ns; the constants were measured): a block takes an SM 31 ns and a warp
    // 300 ns at least, more with more tiles of x rows; a row's block of x takes its CTA 17 ns; warps that share a tile meet
    // in 300 ns, CTAs that share one in 1200 ns.  Against every split of 11 shapes (1 to 8 rows, 4096 x 256 to 151936 x
    // 5120) the choice is within 15 % of the best; without clusters 8 rows of 7168 x 5120 take 17.2 us instead of 13.9.
    int64_t ctas = 0;
    for (;; p.rb = (p.rb + 1) / 2) {
        const int nt = (p.rb + 7) / 8 * parts;
        const int64_t gy = (p.rows + p.rb - 1) / p.rb;
        int64_t best = -1;
        Lin4 q = p;
        for (q.ks = 1; q.ks <= 8 && q.ks <= p.kblocks; q.ks *= 2) {
            q.kper = (p.kblocks + q.ks - 1) / q.ks;
            for (q.kw_log2 = 0; q.kw_log2 <= 3 && (q.kw_log2 == 0 || (1 << q.kw_log2) <= p.kblocks / q.ks); ++q.kw_log2) {
                const int64_t smem = static_cast<int64_t>(l4_smem(q, (p.rb + 7) / 8, parts));
                if (smem > L4_SMEM_MAX) continue;
                const int64_t per_sm = 2 * (smem + 1024) <= 227 * 1024 ? 2 : 1;
                const int64_t sets = (p.tiles + (L4_WARPS >> q.kw_log2) - 1) / (L4_WARPS >> q.kw_log2);
                int64_t slots = sms * per_sm / (q.ks * gy);
                slots = slots < 1 ? 1 : slots < sets ? slots : sets;
                const int64_t rounds = (sets + slots - 1) / slots, blocks = (q.kper + (1 << q.kw_log2) - 1) >> q.kw_log2;
                const int64_t warps = (slots * q.ks * gy * L4_WARPS + sms - 1) / sms, full = warps < per_sm * L4_WARPS ? warps : per_sm * L4_WARPS;
                const int64_t block = full * (23 + 8 * nt) > 270 + 30 * nt ? full * (23 + 8 * nt) : 270 + 30 * nt;
                const int64_t waves = (slots * q.ks * gy + sms * per_sm - 1) / (sms * per_sm);
                const int64_t time = waves * (p.rb * parts * q.kper * 17 +
                                              rounds * (blocks * block + (q.kw_log2 ? 300 : 0) + (q.ks > 1 ? 1200 : 0)));
                if (best < 0 || time < best) best = time, p.kper = q.kper, p.ks = q.ks, p.kw_log2 = q.kw_log2, ctas = slots;
            }
        }
        if (best >= 0) break;  // one row of L4_MAX_K columns fits
    }
    const int nt = (p.rb + 7) / 8;
    const size_t smem = l4_smem(p, nt, parts);
    const unsigned gx = static_cast<unsigned>(ctas * p.ks), gy = static_cast<unsigned>((p.rows + p.rb - 1) / p.rb);
    if (f32x) return nt == 1 ? launch_l4_groups<1, true>(p, smem, gx, gy, s) : launch_l4_groups<2, true>(p, smem, gx, gy, s);
    if (nt == 1) return launch_l4_groups<1, false>(p, smem, gx, gy, s);
    if (nt == 2) return launch_l4_groups<2, false>(p, smem, gx, gy, s);
    if (nt == 3) return launch_l4_groups<3, false>(p, smem, gx, gy, s);
    return launch_l4_groups<4, false>(p, smem, gx, gy, s);
}

}  // namespace dfl

using namespace dfl;

// The sizes that the two kernels share, and their grid.
static Quant4 quant4_of(const void *W, dflash2_dtype dt, int64_t ld, const dflash2_weight4 *w, bool back, dim3 *grid) {
    Quant4 p = {};
    p.W = W, p.w = *w, p.ld = ld;
    p.pieces = static_cast<uint32_t>(groups_of(w) * (w->group / 32));
    p.all = static_cast<uint32_t>(w->N * p.pieces);
    p.codes = static_cast<int>((w->K + 31) / 32) * 4;
    for (p.span_log2 = 2; p.span_log2 < 5 && (1 << p.span_log2) < p.codes;) ++p.span_log2;
    p.vec = aligned16(W) && ld * esize(dt) % 16 == 0;
    const int64_t warps = (w->N + (32 >> p.span_log2) - 1) / (32 >> p.span_log2);
    // rows are cut while warps are fewer than the GPU holds: 16 x 20480 2.6 us (a warp to a row 15), of 20481 columns 4.2 (49)
    const int64_t room = sm_count() * int64_t(64), parts = warps < room ? room / warps : 1, once = Q4_AHEAD << p.span_log2;
    p.part = static_cast<int>(((p.codes + parts - 1) / parts + once - 1) / once * once);
    *grid = back ? dim3(static_cast<unsigned>((warps + 7) / 8), static_cast<unsigned>((p.codes + p.part - 1) / p.part))
                 : dim3((p.all + 255) / 256);
    return p;
}

// Matrices whose pieces of 32 columns, whole groups, are counted in 32 bits.
static bool quant4_fits(const dflash2_weight4 *w) {
    return groups_of(w) * (w->group / 32) <= ((int64_t(1) << 31) - 1) / w->N;
}

template <bool F32W, int LG>
static void launch_quant4(const Quant4 &p, dim3 grid, cudaStream_t s) {
    if (p.w.zero) k_quant4<F32W, LG, true><<<grid, 256, 0, s>>>(p);
    else k_quant4<F32W, LG, false><<<grid, 256, 0, s>>>(p);
}
template <bool F32W>
static void launch_quant4_groups(const Quant4 &p, dim3 grid, cudaStream_t s) {
    if (p.w.group == 128) launch_quant4<F32W, 0>(p, grid, s);
    else if (p.w.group == 64) launch_quant4<F32W, 1>(p, grid, s);
    else launch_quant4<F32W, 2>(p, grid, s);
}
template <bool F32W, int LG>
static void launch_dequant4_rows(const Quant4 &p, void *out, dim3 grid, cudaStream_t s) {
    if (p.vec) k_dequant4<F32W, LG, true><<<grid, 256, 0, s>>>(p, out);
    else k_dequant4<F32W, LG, false><<<grid, 256, 0, s>>>(p, out);
}
template <bool F32W>
static void launch_dequant4(const Quant4 &p, void *out, dim3 grid, cudaStream_t s) {
    if (p.w.group == 128) launch_dequant4_rows<F32W, 0>(p, out, grid, s);
    else if (p.w.group == 64) launch_dequant4_rows<F32W, 1>(p, out, grid, s);
    else launch_dequant4_rows<F32W, 2>(p, out, grid, s);
}

extern "C" dflash2_status dflash2_quant4(const void *W, dflash2_dtype dt, int64_t ld, const dflash2_weight4 *w,
                                         dflash2_stream stream) {
    if (!dtype_ok(dt) || !weight4_ok(w) || ld < w->K) return DFLASH2_ERR_INVALID_ARG;
    if (w->N == 0) return DFLASH2_OK;
    if (!W || !aligned_to(W, dt)) return DFLASH2_ERR_INVALID_ARG;
    if (!quant4_fits(w)) return DFLASH2_ERR_UNSUPPORTED;
    dim3 grid;
    const Quant4 p = quant4_of(W, dt, ld, w, false, &grid);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dt == DFLASH2_F32) launch_quant4_groups<true>(p, grid, s);
    else launch_quant4_groups<false>(p, grid, s);
    return after_launch();
}

extern "C" dflash2_status dflash2_dequant4(const dflash2_weight4 *w, void *out, dflash2_dtype dt, int64_t ld,
                                           dflash2_stream stream) {
    if (!dtype_ok(dt) || !weight4_ok(w) || ld < w->K) return DFLASH2_ERR_INVALID_ARG;
    if (w->N == 0) return DFLASH2_OK;
    if (!out || !aligned_to(out, dt)) return DFLASH2_ERR_INVALID_ARG;
    if (!quant4_fits(w)) return DFLASH2_ERR_UNSUPPORTED;
    dim3 grid;
    const Quant4 p = quant4_of(out, dt, ld, w, true, &grid);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dt == DFLASH2_F32) launch_dequant4<true>(p, out, grid, s);
    else launch_dequant4<false>(p, out, grid, s);
    return after_launch();
}

// Whether the tensor cores' kernel is the faster one.  Its time follows K while its items are no more than the SMs (5120
// columns: 20 to 35 us, on rounded weights 18 to 24; 1024: 8 to 14 and 8 to 11), that of the kernel for few rows N x rows
// (5120 columns, 32 rows of 1024, 4096, 8192: 16, 20, 36 us).  At 396 sizes (9 to 512 rows, N 128 to 8192, K 256 to 17408;
// groups of 128) the choice takes 1.5 % more than the faster one on average and 27 % at most, but for 128 exact rows of
// 4096 x 256 (10 us for 7).  In groups of 32 the tensor cores' kernel takes up to twice as long on exact weights, and the
// other one 1.1 times: there the choice (180 sizes) takes 1.4 % more on average and 41 % at most; that of the other groups
// took 9 and 81 %.  `group`: 0 for rounded weights.
// f32 rows (three times the products either way) at 300 sizes up to 32768 x 17408: 1.2 % more, at most 47 % (9 rows of 8192 x
// 17408, 111 us for 76); 64 rows of 32768 x 5120 take 267 and 87 us.
static bool l4_many(dflash2_dtype dt, int64_t rows, int64_t N, int64_t K, int group) {
    if (rows < L4_MANY_ROWS) return false;
    if (dt == DFLASH2_F32) return rows * N >= 3 << 15;
    if (group == 32) {
        const int64_t at = (1 << 18) - (1 << 24) / K;
        return rows * N >= (rows > 64 ? at + at / 2 : 2 * at);
    }
    const int64_t at = (1 << 17) - (3 << 26) / K;
    return rows * N >= (group == 0 ? at : rows > 64 ? 2 * at : at + at / 2);
}

extern "C" size_t dflash2_linear4_workspace_bytes(dflash2_dtype dt, int64_t rows, int64_t N, int64_t K) {
    if (!dtype_ok(dt) || rows < 1 || N < 1 || K < 1 || K > L4_MAX_K || rows > L4_MAX_ROWS || !l4_many(dt, rows, N, K, 0)) return 0;
    return linear4_tc_bytes(dt == DFLASH2_F32, rows, K);
}

// rounded: bf16 results of bf16 scales may be taken on weights in bf16.
static dflash2_status linear4(const void *x, dflash2_dtype dt, int64_t rows, int64_t x_stride, const dflash2_weight4 *w,
                              void *y, dflash2_dtype y_dt, int64_t y_stride, bool rounded, void *ws, size_t ws_bytes,
                              dflash2_stream stream) {
    if (!dtype_ok(dt) || !dtype_ok(y_dt) || (dt == DFLASH2_F32 && y_dt != DFLASH2_F32) || !weight4_ok(w) || rows < 0 ||
        x_stride < w->K || y_stride < w->N)
        return DFLASH2_ERR_INVALID_ARG;
    if (rows == 0 || w->N == 0) return DFLASH2_OK;
    if (!x || !y || !aligned_to(x, dt) || !aligned_to(y, y_dt)) return DFLASH2_ERR_INVALID_ARG;
    if (w->K > L4_MAX_K || rows > L4_MAX_ROWS) return DFLASH2_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (l4_many(dt, rows, w->N, w->K, 0)) {
        if (!ws || !aligned16(ws)) return DFLASH2_ERR_INVALID_ARG;
        if (ws_bytes < linear4_tc_bytes(dt == DFLASH2_F32, rows, w->K)) return DFLASH2_ERR_WORKSPACE;
        const bool exact = !rounded || y_dt == DFLASH2_F32 || w->side_dt == DFLASH2_F32;
        // (also where the kernel for few rows does not count as many blocks, as below)
        if (l4_many(dt, rows, w->N, w->K, exact ? w->group : 0) || (rows > L4_LONG_ROWS && w->K > L4_LONG_K))
            return linear4_tc(x, dt == DFLASH2_F32, rows, x_stride, w, y, y_dt, y_stride, exact, ws, s);
    }
    // blocks of rows are counted in 16 bits: of up to L4_LONG_K columns they have 16 rows, of more one at least
    if (rows > L4_LONG_ROWS && w->K > L4_LONG_K) return DFLASH2_ERR_UNSUPPORTED;
    Lin4 p = {};
    p.x = x, p.rows = rows, p.x_stride = x_stride, p.w = *w, p.y = y, p.y_stride = y_stride, p.y_dt = y_dt;
    p.G = static_cast<int>(groups_of(w));
    p.gpb_log2 = w->group == 128 ? 0 : w->group == 64 ? 1 : 2;
    return linear4_mma(p, dt == DFLASH2_F32, s);
}

extern "C" dflash2_status dflash2_linear4(const void *x, dflash2_dtype dt, int64_t rows, int64_t x_stride,
                                          const dflash2_weight4 *w, void *y, dflash2_dtype y_dt, int64_t y_stride,
                                          void *ws, size_t ws_bytes, dflash2_stream stream) {
    return linear4(x, dt, rows, x_stride, w, y, y_dt, y_stride, false, ws, ws_bytes, stream);
}

extern "C" dflash2_status dflash2_linear4_rounded(const void *x, dflash2_dtype dt, int64_t rows, int64_t x_stride,
                                                  const dflash2_weight4 *w, void *y, dflash2_dtype y_dt, int64_t y_stride,
                                                  void *ws, size_t ws_bytes, dflash2_stream stream) {
    return linear4(x, dt, rows, x_stride, w, y, y_dt, y_stride, true, ws, ws_bytes, stream);
}
