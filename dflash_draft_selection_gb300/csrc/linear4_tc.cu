// linear4_tc.cu -- dflash2_linear4 for many rows, on the 5th-generation tensor
// cores.
//
// Weights on the M side (128 rows), x on the N side (up to 128 rows):
//   part[128 x R] = codes[128 x group] . x'[R x group]^T     per group of columns
//   acc += scale * (part - zero * sum of x)                  in registers, f32
// so products are exact whatever the scales, and a result is rounded once.  f32
// rows are three bf16 parts, which is exact too: three products into the same
// accumulator, blocks of up to 32 rows.
//
// The codes go by TMA into a warp's own ring in shared memory and through its
// registers into tensor memory, where the MMA takes its A operand: with A in
// shared memory its 4 KB per step of 16 columns bound the MMA to 56 cycles at R
// = 64, from tensor memory it takes 32.  x' (scaled and reordered once by a
// kernel of its own into the workspace) comes by TMA, 128-byte swizzle, with its
// groups' sums beside it.
//
// One CTA per SM walks its items: a tile of 128 weight rows and a block of x
// rows.  A tile's items go to neighbouring CTAs at one time, so its codes come
// from HBM once.
//   warps 0-7    epilogue: a weight row per lane, half of the R columns each
//   4 or 8 warps operand and scales: 32 weight rows each; of 8, 4 take the odd pairs of
//                blocks of 128 columns
//   2 warps      copies of x', MMAs
// Tensor memory: 4 accumulators of R columns (2 of 128), 4 blocks of A of 64 columns.
//
// Results in bf16 on weights in bf16 (dflash2_linear4_rounded): one accumulator over all columns.  512 rows
// of 151936 x 5120: 538 us, 1480 TFLOP/s; bound by the operand's conversion (two
// instructions a pair of codes, three with zero points) and a barrier's 150 cycles.
// 64 rows: 122 us, all of it the operand.  Results on codes: 512 rows of the same
// in groups of 128 854 us, of 64 1898, of 32 (zero points) 3983; 64 rows of
// 151936 x 2560 in groups of 128 94 us, of 32 228 us; bound by the chain MMA -
// barrier - tensor memory load - barrier per group; loads of a second group ahead
// gained nothing, and spilled at 128 rows.  512 rounded rows of 7168 x 5120 by items
// 40 us, by whole tiles 73.  64 f32 rows of 32768 x 5120 87 us (k_linear4_mma: 267).
//
// Waits are bounded: after a time-out every role stops waiting, the error word
// is set and the CTA's remaining outputs are NaN.
#include "host.hpp"
#include "linear4.cuh"
#include "tc.cuh"

namespace dfl {

static __device__ unsigned int g_err_linear4;

// Warps: 8 for the epilogue, the operand's 4 (where the exact epilogue needs 128 registers a thread) or 8, copies of x',
// MMAs.
constexpr int t4_sets(int rh, bool exact) { return exact && rh > 32 ? 1 : 2; }
constexpr int t4_threads(int rh, bool exact) { return (8 + 4 * t4_sets(rh, exact) + 2) * 32; }
constexpr int T4_XS = 4;                                     // stages of x'
// Blocks of 128 columns in a stage: a barrier costs its waiter 150 cycles.  The parts of f32 rows leave room for one.
constexpr int t4_blocks(int rh, int parts) { return rh > 32 || parts > 1 ? 1 : 2; }
constexpr int t4_ring(int rh, bool exact) { return exact && rh > 32 ? 4 : 2; }  // pairs of blocks of codes that an operand warp has room for
constexpr int T4_AS = 4;      // blocks of A in tensor memory
// Blocks whose scales are kept.  A block's are overwritten when the operand is this many further on: it is at most 4
// blocks ahead of the last MMA that completed, and that at most T4_DS accumulators (4, 2 or 1 blocks) ahead of the
// epilogue.
constexpr int t4_sides(int lg) { return lg == 0 ? 8 : 6; }
constexpr int T4_DS = 4;      // accumulators, at most: 2 of 128 columns
constexpr int T4_M = 128;
// Weights in bf16 are held times 2^-40, and their rows of x have their largest entry near 2^80: with scales from 2^-80 to
// 2^30 and entries from 2^-80 of a row's largest nothing vanishes or overflows.
constexpr int T4_DOWN = 40, T4_TOP = 207;  // (and the field of that entry's exponent)
constexpr uint32_t T4_SCALE_LO = (127u - 80u) << 7, T4_SCALE_HI = (127u + 30u) << 7, T4_ZERO_HI = (127u + 39u) << 7;
// Bits of a scale as the weights in bf16 take it: NaN where it, or its zero point, leaves that range.
__device__ __forceinline__ uint32_t t4_scale(uint32_t scale, uint32_t zero) {
    const uint32_t m = scale & 0x7fffu;
    return (m == 0 || m - T4_SCALE_LO <= T4_SCALE_HI - T4_SCALE_LO) && (zero & 0x7fffu) <= T4_ZERO_HI ? scale : 0x7fc0u;
}
constexpr long long T4_WAIT = 4000000000ll, T4_DRAIN = 200000000ll;

struct Tc4Shared {
    uint64_t x_full[T4_XS], x_empty[T4_XS];
    uint64_t a_empty[T4_AS];
    uint64_t c_full[8][4];  // an operand warp's codes
    uint64_t d_full[T4_DS], d_empty[T4_DS];
    uint64_t done;
    uint32_t tmem;
    int abort;
};

struct Tc4 {
    dflash2_weight4 w;
    void *y;
    int64_t rows, y_stride;
    dflash2_dtype y_dt;
    int lg, G, kpairs, rblocks;  // lg: log2 of the groups in a block
    int tiles;
    int step_tile, step_rb;  // from an item to the CTA's next
    const float *sums;  // [row block][2 * kpairs << lg][R]
    const float *root;  // [rows_pad]
    const unsigned int *hold;
    long long hold_cycles;
};

// ---------------------------------------------------------------- x' ----
// One CTA per row: x' [rows_pad, kblocks * 128] (f32: three matrices of bf16 parts, exact), scaled for the codes as operands or for weights in bf16 (then without
// the groups' sums), and the root of the power of two.  Rows past the last are zeros.
template <bool F32X>
__global__ void __launch_bounds__(256) k_linear4_rows(const void *x, int64_t rows, int64_t x_stride, int K, int lg,
                                                      int kblocks, int R, bool scaled, uint16_t *out, float *sums,
                                                      float *root) {
    __shared__ uint32_t top;
    const int64_t r = blockIdx.x;
    const int chunks = kblocks * (L4_BLOCK / 8), lanes = 16 >> lg;
    const bool vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && x_stride * (F32X ? 4 : 2) % 16 == 0;
    pdl_trigger();  // the product may start; it waits before it reads what is written here
    if (threadIdx.x == 0) top = 0;
    __syncthreads();
    uint32_t m = 0;
    if (r < rows)
        for (int c = threadIdx.x; c < chunks; c += 256) {
            float v[8];
            load8<F32X>(x, r * x_stride + c * 8, K - c * 8, vec, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
        }
    m = __reduce_max_sync(FULL, m);
    if ((threadIdx.x & 31) == 0) atomicMax(&top, m);
    __syncthreads();
    m = top;
    const int e = scaled ? x_exponent(m) : (T4_TOP - static_cast<int>(m >> 23)) & ~1;  // even: the result's power has a root
    const bool bad = m >= 0x7f800000u;
    if (threadIdx.x == 0) root[r] = scaled || bad ? x_root(m, e) : pow2f((T4_DOWN - e) / 2);
    for (int c = threadIdx.x; c < chunks; c += 256) {  // chunks is a multiple of 16: half-warps stay whole
        float v[8] = {};
        if (r < rows) load8<F32X>(x, r * x_stride + c * 8, K - c * 8, vec, v);
        if (bad) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        }
        if (scaled) {
            float sum = scale8(v, e);
            for (int d = lanes >> 1; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffu << (threadIdx.x & 16), sum, d);
            if ((c & (lanes - 1)) == 0) sums[(r / R * (chunks / lanes) + c / lanes) * R + r % R] = sum;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = scale2(v[j], e);
        }
#pragma unroll
        for (int q = 0; q < (F32X ? 3 : 1); ++q) {
            uint4 o;
            uint32_t *ow = &o.x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                ow[j] = bf16_pair(v[j], v[j + 4]);
                if (F32X) v[j] -= bf16lo(ow[j]), v[j + 4] -= bf16hi(ow[j]);
            }
            *reinterpret_cast<uint4 *>(out + ((q * static_cast<int64_t>(gridDim.x) + r) * kblocks * L4_BLOCK + c * 8)) = o;
        }
    }
}

// ------------------------------------------------------------- product ----
__device__ __forceinline__ bool t4_aborted(Tc4Shared &sm) { return *reinterpret_cast<volatile int *>(&sm.abort) != 0; }
__device__ __forceinline__ void t4_abort(Tc4Shared &sm) {
    atomicOr(&g_err_linear4, ERR_WAIT_TIMEOUT);
    *reinterpret_cast<volatile int *>(&sm.abort) = 1;
}
// False after a time-out, this one or another role's.
__device__ __forceinline__ bool t4_wait(Tc4Shared &sm, uint64_t *bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!t4_aborted(sm)) {
        if (mbar_try_wait(bar, parity)) return true;
        if (clock64() - t0 > T4_WAIT) t4_abort(sm);
    }
    return false;
}

__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void bulk_g2s(void *sdst, const void *gsrc, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_addr(sdst)),
                 "l"(gsrc), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}

// Walks a CTA's blocks: item by item, their blocks of columns.
struct Walk4 {
    int tile, rb, kb;
    __device__ __forceinline__ explicit Walk4(const Tc4 &p)
        : tile(static_cast<int>(blockIdx.x) / p.rblocks), rb(static_cast<int>(blockIdx.x) % p.rblocks), kb(0) {}
    __device__ __forceinline__ void next(const Tc4 &p, int blocks) {  // 1 or 2: an item has pairs
        kb += blocks;
        if (kb < 2 * p.kpairs) return;
        kb = 0, tile += p.step_tile, rb += p.step_rb;
        if (rb >= p.rblocks) rb -= p.rblocks, ++tile;
    }
};

// 128 columns of a weight row, 16 words of codes, into tensor memory.  KIND 0: the codes as they are; 1 and 2: the weights
// times 2^-T4_DOWN in bf16, without and with zero points, from the groups' bits in bf16.  The masked codes are operands of
// the fused step as they lie (times 2^-133 or, the second pairs, 2^-129), so that
//   weight 2^-40 = code * (scale 2^-40) - 8 * (scale 2^-40)           one rounding
//   with zero points: (code - zero) 2^-40, exact for whole zero points, times the scale.
template <int LG, int KIND>
__device__ __forceinline__ void operand(const uint32_t *v, uint32_t to, const uint32_t *sr, const uint32_t *zr) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {  // 32 columns
        uint32_t first = 0, second = 0, less = 0, scale = 0;
        if constexpr (KIND != 0) {
            const uint32_t sb = t4_scale(sr[q * 32 >> (7 - LG)], KIND == 2 ? zr[q * 32 >> (7 - LG)] : 0);
            const float sc = __uint_as_float(sb << 16);
            const float f = KIND == 1 ? sc : 1.0f, z = KIND == 1 ? 8.0f * sc : __uint_as_float(zr[q * 32 >> (7 - LG)] << 16);
            first = pair_of(f * pow2f(133 - T4_DOWN)), second = pair_of(f * pow2f(129 - T4_DOWN));
            less = pair_of(-z * pow2f(-T4_DOWN)), scale = sb * 0x10001u;
        }
        uint32_t a[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t w = v[q * 4 + j], u = w >> 8;
            uint32_t *o = a + j * 4;
            o[0] = w & 0x000f000fu, o[1] = w & 0x00f000f0u, o[2] = u & 0x000f000fu, o[3] = u & 0x00f000f0u;
            if constexpr (KIND != 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    o[k] = fma_bf16x2(o[k], k & 1 ? second : first, less);
                    if (KIND == 2) o[k] = mul_bf16x2(o[k], scale);
                }
            }
        }
        tmem_st16(to + q * 16, a);
    }
}

// RH: half of the block's rows of x, the columns of an epilogue warp.  LG: log2 of the groups in a block.  EXACT: the
// operand is the codes; otherwise it is the weights in bf16.  PARTS: matrices of x', 3 for f32 rows.
template <int RH, int LG, bool EXACT, int PARTS>
__global__ void __launch_bounds__(t4_threads(RH, EXACT), 1) k_linear4_tc(const __grid_constant__ CUtensorMap tm_x,
                                                              const __grid_constant__ CUtensorMap tm_c, const Tc4 p) {
    constexpr int R = RH * 2, XB = R * L4_BLOCK * 2;  // bytes of a block of a part of x'
    constexpr int gpb = 1 << LG, STEPS = 8 >> LG;      // groups of a block, steps of 16 columns in a group
    constexpr int T4_SIDES = t4_sides(LG);
    constexpr int XS = T4_XS, SB = t4_blocks(RH, PARTS), RING = t4_ring(RH, EXACT), SETS = t4_sets(RH, EXACT), T4_COPY = 8 + 4 * SETS, T4_MMA = T4_COPY + 1;
    extern __shared__ unsigned char raw[];
    __shared__ Tc4Shared sm;
    unsigned char *xs = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *rings = xs + XS * SB * PARTS * XB;                              // 4 KB each: 32 rows of 256 codes
    float *sums = reinterpret_cast<float *>(rings + 4 * SETS * RING * 4096);  // [stage][group of the stage][R]
    float2 *sides = reinterpret_cast<float2 *>(sums + XS * SB * gpb * R);  // [block][group][weight row]: scale, -scale * zero
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        // A stage is there when x' has landed and the operand's four warps have left its blocks in tensor memory and
        // their scales; it is free after its MMAs and the epilogue's warps.  Accumulators are there when their MMAs are
        // done and the warp that issued them, which has seen the stage's rest, says so.
        for (int i = 0; i < XS; ++i) mbar_init(&sm.x_full[i], 5), mbar_init(&sm.x_empty[i], EXACT ? 9 : 1);
        for (int i = 0; i < T4_AS; ++i) mbar_init(&sm.a_empty[i], 1);
        for (int i = 0; i < 4 * SETS; ++i)
            for (int j = 0; j < RING; ++j) mbar_init(&sm.c_full[i][j], 1);
        for (int i = 0; i < T4_DS; ++i) mbar_init(&sm.d_full[i], 2), mbar_init(&sm.d_empty[i], 8);
        mbar_init(&sm.done, 1);
        sm.abort = 0;
        fence_barrier_init();
    }
    __syncwarp();
    if (warp == T4_MMA) tmem_alloc(&sm.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // accumulators, and how many of them the epilogue is given at a time
    constexpr uint32_t DS = R > 64 || !EXACT ? 2 : 4, U = R > 64 || !EXACT ? 1 : 2;
    const uint32_t tmem = sm.tmem, tmem_a = tmem + DS * R;
    const int mine = static_cast<int>((static_cast<int64_t>(p.tiles) * p.rblocks - blockIdx.x - 1) / gridDim.x) + 1;  // items of this CTA
    const int total = mine * p.kpairs * 2;                                                      // and their blocks

    if (warp == T4_COPY) {
        if (lane == 0) {
            int i = 0;
            bool ok = true;
            if (p.hold != nullptr && !hold_wait(p.hold, p.hold_cycles)) t4_abort(sm), ok = false;
            Walk4 at(p);
            pdl_wait();  // x' and its sums
            for (; ok && i < total / SB; ++i) {
                const int s = i % XS;
                if (i >= XS && !t4_wait(sm, &sm.x_empty[s], static_cast<uint32_t>(i / XS - 1) & 1)) break;
                mbar_arrive_expect_tx(&sm.x_full[s], SB * (PARTS * XB + (EXACT ? gpb * R * 4 : 0)));
#pragma unroll
                for (int q = 0; q < PARTS; ++q)
#pragma unroll
                    for (int h = 0; h < 2 * SB; ++h)
                        tma_load_2d(xs + ((s * PARTS + q) * 2 * SB + h) * (XB / 2), &tm_x, at.kb * L4_BLOCK + h * 64,
                                    (q * p.rblocks + at.rb) * R, &sm.x_full[s]);
                // sums [row block][group][R]: a stage's lie together
                if (EXACT)
                    bulk_g2s(sums + s * SB * gpb * R, p.sums + (static_cast<int64_t>(at.rb) * 2 * p.kpairs + at.kb) * gpb * R,
                             SB * gpb * R * 4, &sm.x_full[s]);
                at.next(p, SB);
            }
            // Leave no copy in flight into this CTA's shared memory.  A block is waited for with its scales; after a
            // time-out those may not come, and the copies have the whole limit to land.
            for (int j = i > XS ? i - XS : 0; j < i; ++j)
                mbar_wait(&sm.x_full[j % XS], static_cast<uint32_t>(j / XS) & 1, T4_DRAIN);
        }
    } else if (warp == T4_MMA) {
        // The whole warp walks, so that addresses stay in uniform registers; one thread issues.
        constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(R >> 3) << 17) |
                                   (static_cast<uint32_t>(T4_M >> 4) << 24);
        const uint64_t x0 = sw128_desc(xs);
        const bool leader = elect_one();
        uint32_t d = 0;
        int kb = 0;
        bool ok = true;
        for (int i = 0; ok && i < total; ++i) {
            const int s = i / SB % XS, sa = i % T4_AS;
            if (i % SB == 0) ok = __all_sync(FULL, t4_wait(sm, &sm.x_full[s], static_cast<uint32_t>(i / SB / XS) & 1));
            if (!ok) break;
            const uint64_t b0 = x0 + ((s * SB * PARTS + i % SB) * XB >> 4);
            const uint32_t a0 = tmem_a + sa * 64;
            if constexpr (EXACT) {
#pragma unroll
                for (int j = 0; j < gpb; ++j, ++d) {
                    // U accumulators at a time
                    const uint32_t u = d / U;
                    if (d % U == 0 && u >= DS / U) ok = __all_sync(FULL, t4_wait(sm, &sm.d_empty[u % (DS / U)], (u / (DS / U) - 1) & 1));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t to = tmem + (d % DS) * R;
                    if (leader) {
#pragma unroll
                        for (int q = PARTS - 1; q >= 0; --q)  // the small parts first
#pragma unroll
                            for (int k = 0; k < STEPS; ++k) {
                                const int at = j * STEPS + k;  // 16 columns: 32 bytes of x', 8 columns of tensor memory
                                mma_bf16_ts(to, a0 + at * 8, b0 + (q * XB >> 4) + (at & 4 ? (XB / 2 >> 4) : 0) + 2 * (at & 3), idesc,
                                            q < PARTS - 1 || k > 0);
                            }
                        if (d % U == U - 1) mma_commit(&sm.d_full[u % (DS / U)]), mbar_arrive(&sm.d_full[u % (DS / U)]);
                    }
                    __syncwarp();
                }
                if (!ok) break;
            } else {
                if (kb == 0 && d >= DS) ok = __all_sync(FULL, t4_wait(sm, &sm.d_empty[d % DS], (d / DS - 1) & 1));
                if (!ok) break;
                tc_fence_after();
                const uint32_t to = tmem + (d % DS) * R;
                if (leader) {
#pragma unroll
                    for (int at = 0; at < 8; ++at)
                        mma_bf16_ts(to, a0 + at * 8, b0 + (at & 4 ? (XB / 2 >> 4) : 0) + 2 * (at & 3), idesc, at > 0 || kb > 0);
                    if (kb == 2 * p.kpairs - 1) mma_commit(&sm.d_full[d % DS]), mbar_arrive(&sm.d_full[d % DS]);
                }
                __syncwarp();
                if (++kb == 2 * p.kpairs) kb = 0, ++d;
            }
            if (leader) {
                mma_commit(&sm.a_empty[sa]);
                if (i % SB == SB - 1) mma_commit(&sm.x_empty[s]);
            }
            __syncwarp();
        }
        // every MMA issued has completed once this commit arrives
        if (leader) mma_commit(&sm.done);
        __syncwarp();
        mbar_wait(&sm.done, 0, T4_DRAIN);
    } else if (warp >= 8) {
        // The operand: 32 weight rows of every (second) pair of blocks.  A warp's codes come by TMA, 128 bytes of its rows
        // (zeros past the last row and column), 128-byte swizzle.
        const int quad = warp & 3, odd = (warp - 8) >> 2, me = warp - 8;
        unsigned char *ring = rings + me * (RING * 4096);
        const uint32_t ring_row = smem_addr(ring) + lane * 128;
        const int pairs = total / 2;
        Walk4 cw(p);  // pair to copy next, and how far it is
        int c = odd;
        auto copy = [&](int stage) {
            if (lane == 0) {
                mbar_arrive_expect_tx(&sm.c_full[me][stage], 4096);
                tma_load_2d(ring + stage * 4096, &tm_c, cw.kb * (L4_BLOCK / 2), cw.tile * T4_M + quad * 32,
                            &sm.c_full[me][stage]);
            }
#pragma unroll
            for (int j = 0; j < SETS; ++j) cw.next(p, 2);
            c += SETS;
        };
        if (odd) cw.next(p, 2);
        int issued = 0;
#pragma unroll
        for (int j = 0; j < RING; ++j)
            if (c < pairs) copy(j), ++issued;
        // scales and zero points of the lane's own row, one of the warp's pairs ahead
        Walk4 sw(p);
        int64_t side0 = 0;
        uint32_t sr[2 * gpb], zr[2 * gpb];
        auto side_row = [&]() {
            const int64_t n = static_cast<int64_t>(sw.tile) * T4_M + quad * 32 + lane;
            side0 = (n < p.w.N ? n : p.w.N - 1) * p.w.side_stride;
        };
        auto load_sides = [&]() {
            if (sw.tile >= p.tiles) return;
            const int was = sw.tile;
#pragma unroll
            for (int j = 0; j < 2 * gpb; ++j) {
                const int gi = sw.kb * gpb + j;
                sr[j] = zr[j] = 0;
                if (gi < p.G) {
                    sr[j] = side_bits(p.w.scale, p.w.side_dt, side0 + gi);
                    if (p.w.zero) zr[j] = side_bits(p.w.zero, p.w.side_dt, side0 + gi);
                }
            }
#pragma unroll
            for (int j = 0; j < SETS; ++j) sw.next(p, 2);
            if (sw.tile != was) side_row();
        };
        if (odd) sw.next(p, 2);
        side_row();
        load_sides();
        int st = 0;
        uint32_t round = 0;
        for (int i = odd, ok = 1; ok && i < pairs; i += SETS) {
            ok = __all_sync(FULL, t4_wait(sm, &sm.c_full[me][st], round & 1));
            if (!ok) break;
            uint32_t v[32];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(v[q * 4]), "=r"(v[q * 4 + 1]), "=r"(v[q * 4 + 2]), "=r"(v[q * 4 + 3])
                             : "r"(ring_row + st * 4096 + ((q ^ (lane & 7)) << 4)));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int b = 2 * i + h, sa = b % T4_AS;
                if (b >= T4_AS) ok = __all_sync(FULL, t4_wait(sm, &sm.a_empty[sa], static_cast<uint32_t>(b / T4_AS - 1) & 1));
                if (!ok) break;
                tc_fence_after();
                const uint32_t to = tmem_a + (static_cast<uint32_t>(quad * 32) << 16) + sa * 64;
                if (EXACT) operand<LG, 0>(v + h * 16, to, sr + h * gpb, zr + h * gpb);
                else if (p.w.zero) operand<LG, 2>(v + h * 16, to, sr + h * gpb, zr + h * gpb);
                else operand<LG, 1>(v + h * 16, to, sr + h * gpb, zr + h * gpb);
                if (h == 0) {
                    __syncwarp();  // every lane has its codes
                    if (c < pairs) copy(st), ++issued;
                }
                if constexpr (EXACT) {
#pragma unroll
                    for (int j = 0; j < gpb; ++j) {
                        const float sc = side_of(sr[h * gpb + j], p.w.side_dt);
                        sides[((b % T4_SIDES) * gpb + j) * T4_M + quad * 32 + lane] =
                            make_float2(sc, -sc * (p.w.zero ? side_of(zr[h * gpb + j], p.w.side_dt) : 8.0f));
                    }
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && b % SB == SB - 1) mbar_arrive(&sm.x_full[b / SB % XS]);
            }
            if (!ok) break;
            load_sides();
            if (++st == RING) st = 0, ++round;
        }
        // leave no copy in flight
        if (lane == 0)
            for (int j = issued > RING ? issued - RING : 0; j < issued; ++j)
                mbar_wait(&sm.c_full[me][j % RING], static_cast<uint32_t>(j / RING) & 1, T4_DRAIN);
        __syncwarp();
    } else {
        // epilogue
        const int quad = warp & 3, half = warp >> 2;
        const uint32_t tm = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * RH;
        int i = 0;
        uint32_t d = 0;
        bool ok = true;
        pdl_wait();  // the roots
        for (int item = 0; item < mine; ++item) {
            uint64_t acc[RH / 2];
#pragma unroll
            for (int j = 0; j < RH / 2; ++j) acc[j] = 0;
            if constexpr (EXACT) {
                for (int kb = 0; ok && kb < 2 * p.kpairs; ++kb, ++i) {
                    const int s = i / SB % XS;
#pragma unroll
                    for (int j = 0; j < gpb; ++j, ++d) {
                        const uint32_t u = d / U;
                        if (d % U == 0) ok = ok && __all_sync(FULL, t4_wait(sm, &sm.d_full[u % (DS / U)], (u / (DS / U)) & 1));
                        if (!ok) break;
                        tc_fence_after();
                        const float2 side = sides[((i % T4_SIDES) * gpb + j) * T4_M + quad * 32 + lane];
                        const uint64_t s2 = pack2(__float_as_uint(side.x), __float_as_uint(side.x));
                        const uint64_t z2 = pack2(__float_as_uint(side.y), __float_as_uint(side.y));
                        const float *xg = sums + ((s * SB + i % SB) * gpb + j) * R + half * RH;
                        constexpr int CH = RH < 16 ? RH : RH < 32 ? 16 : 32;
#pragma unroll
                        for (int c = 0; c < RH; c += CH) {
                            uint32_t v[CH];
                            if constexpr (CH == 8) {
                                tmem_ld8(tm + (d % DS) * R, v);
                            } else {
#pragma unroll
                                for (int k = 0; k < CH; k += 16) tmem_ld16_nowait(tm + (d % DS) * R + c + k, v + k);
                            }
                            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                            for (int k = 0; k < CH; k += 4) {
                                const ulonglong2 x2 = *reinterpret_cast<const ulonglong2 *>(xg + c + k);
                                const int at = (c + k) / 2;
                                acc[at] = fma2(z2, x2.x, fma2(s2, pack2(v[k], v[k + 1]), acc[at]));
                                acc[at + 1] = fma2(z2, x2.y, fma2(s2, pack2(v[k + 2], v[k + 3]), acc[at + 1]));
                            }
                        }
                        if (d % U == U - 1) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&sm.d_empty[u % (DS / U)]);
                        }
                    }
                    __syncwarp();
                    if (i % SB == SB - 1 && ok && lane == 0) mbar_arrive(&sm.x_empty[s]);
                }
            } else {
                ok = ok && __all_sync(FULL, t4_wait(sm, &sm.d_full[d % DS], (d / DS) & 1));
                if (ok) {
                    tc_fence_after();
                    uint32_t v[RH];
                    if constexpr (RH == 8) {
                        tmem_ld8(tm + (d % DS) * R, v);
                    } else {
#pragma unroll
                        for (int c = 0; c < RH; c += 16) tmem_ld16_nowait(tm + (d % DS) * R + c, v + c);
                    }
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                    for (int c = 0; c < RH; c += 2) acc[c / 2] = pack2(v[c], v[c + 1]);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.d_empty[d % DS]);
                    ++d;
                }
            }
            const uint32_t nth = blockIdx.x + item * gridDim.x, tile = nth / p.rblocks;
            const int64_t n = static_cast<int64_t>(tile) * T4_M + quad * 32 + lane;
            // the roots of columns l and 32 + l
            const int64_t r0 = static_cast<int64_t>(nth - tile * p.rblocks) * R + half * RH;
            const float f0 = lane < RH ? p.root[r0 + lane] : 0.0f, f1 = RH > 32 ? p.root[r0 + 32 + lane] : 0.0f;
#pragma unroll
            for (int j = 0; j < RH; ++j) {
                const float f = __shfl_sync(FULL, j < 32 ? f0 : f1, j & 31);
                if (r0 + j < p.rows && n < p.w.N) {
                    const float v = ok ? __uint_as_float((j & 1) ? hi32(acc[j / 2]) : lo32(acc[j / 2])) * f * f : NAN;
                    if (p.y_dt == DFLASH2_F32) static_cast<float *>(p.y)[(r0 + j) * p.y_stride + n] = v;
                    else static_cast<uint16_t *>(p.y)[(r0 + j) * p.y_stride + n] = bf16_bits(v);
                }
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == T4_MMA) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ host ----
// Rows of x to a block, 32, 64 or 128 at most.
static int t4_rows(int64_t rows, int most) { return rows <= 16 ? 16 : rows <= 32 || most == 32 ? 32 : rows <= 64 || most == 64 ? 64 : 128; }
static int64_t t4_pad(int64_t rows, int most) { return (rows + t4_rows(rows, most) - 1) / t4_rows(rows, most) * t4_rows(rows, most); }
static int64_t t4_kpad(int64_t K) { return (K + 2 * L4_BLOCK - 1) / (2 * L4_BLOCK) * (2 * L4_BLOCK); }

// Workspace: x', the sums (of the smallest groups), the roots.
size_t linear4_tc_bytes(bool f32x, int64_t rows, int64_t K) {
    return static_cast<size_t>(t4_pad(rows, f32x ? 32 : 128)) * (t4_kpad(K) * (f32x ? 6 : 2) + t4_kpad(K) / 32 * 4 + 4);
}

template <int RH, int LG, bool EXACT, int PARTS>
static dflash2_status launch_tc4(const CUtensorMap &tm, const CUtensorMap &tc, Tc4 p, cudaStream_t s) {
    auto fn = &k_linear4_tc<RH, LG, EXACT, PARTS>;
    constexpr int R = RH * 2, threads = t4_threads(RH, EXACT);
    constexpr size_t smem = 1024 + T4_XS * t4_blocks(RH, PARTS) * (PARTS * R * L4_BLOCK * 2 + (EXACT ? R * 4 << LG : 0)) +
                            4 * t4_sets(RH, EXACT) * t4_ring(RH, EXACT) * 4096 + (EXACT ? t4_sides(LG) * T4_M * 8 << LG : 0);
    static_assert(smem + sizeof(Tc4Shared) <= 227 * 1024, "shared memory of a CTA");
    blocks_per_sm(reinterpret_cast<const void *>(fn), threads, smem);  // raises the shared-memory limit once per device
    const int64_t sms = sm_count();
    cudaLaunchConfig_t cfg = {};
    const int64_t items = static_cast<int64_t>(p.tiles) * p.rblocks, grid = items < sms ? items : sms;
    p.step_tile = static_cast<int>(grid / p.rblocks), p.step_rb = static_cast<int>(grid % p.rblocks);
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};  // beside the kernel that prepares x: the codes' first copies
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, fn, tm, tc, p) != cudaSuccess) return DFLASH2_ERR_CUDA;
    return after_launch();
}

template <int RH, bool EXACT, int PARTS>
static dflash2_status launch_tc4_groups(const CUtensorMap &tm, const CUtensorMap &tc, const Tc4 &p, cudaStream_t s) {
    if (p.lg == 0) return launch_tc4<RH, 0, EXACT, PARTS>(tm, tc, p, s);
    if (p.lg == 1) return launch_tc4<RH, 1, EXACT, PARTS>(tm, tc, p, s);
    return launch_tc4<RH, 2, EXACT, PARTS>(tm, tc, p, s);
}
template <int RH>
static dflash2_status launch_tc4_kind(const CUtensorMap &tm, const CUtensorMap &tc, const Tc4 &p, bool exact, cudaStream_t s) {
    return exact ? launch_tc4_groups<RH, true, 1>(tm, tc, p, s) : launch_tc4_groups<RH, false, 1>(tm, tc, p, s);
}

// Codes [N, bytes of a row], boxes of 32 rows of 128 bytes; zeros past the edges.
static bool codes_map(CUtensorMap *m, const dflash2_weight4 *w) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>((w->K + 31) / 32 * 16), static_cast<cuuint64_t>(w->N)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(w->code_stride)};
    const cuuint32_t box[2] = {128u, 32u};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, w->codes, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

dflash2_status linear4_tc(const void *x, bool f32x, int64_t rows, int64_t x_stride, const dflash2_weight4 *w, void *y,
                          dflash2_dtype y_dt, int64_t y_stride, bool exact, void *ws, cudaStream_t s) {
    // items, and a CTA's blocks, are counted in 31 bits
    // several groups to a block of columns take the epilogue of 128 rows more registers than it has (512 rows of 151936 x
    // 5120 in groups of 32: 4125 us, with 64 rows 3373; of 64: 2075 and 1896)
    const int most = f32x ? 32 : exact && w->group < 128 ? 64 : 128, R = t4_rows(rows, most);
    const int64_t rows_pad = t4_pad(rows, most), items = (w->N + T4_M - 1) / T4_M * (rows_pad / R);
    if (items > 0x7fffffff || (items / sm_count() + 1) * (t4_kpad(w->K) / L4_BLOCK) > (1 << 30))
        return DFLASH2_ERR_UNSUPPORTED;
    Tc4 p = {};
    const int64_t kp = t4_kpad(w->K);
    p.w = *w, p.y = y, p.rows = rows, p.y_stride = y_stride, p.y_dt = y_dt;
    p.lg = w->group == 128 ? 0 : w->group == 64 ? 1 : 2;
    p.G = static_cast<int>(groups_of(w));
    p.kpairs = static_cast<int>(kp / (2 * L4_BLOCK));
    p.rblocks = static_cast<int>(rows_pad / R);
    p.tiles = static_cast<int>((w->N + T4_M - 1) / T4_M);
    uint16_t *xp = static_cast<uint16_t *>(ws);
    const int parts = f32x ? 3 : 1;
    float *sums = reinterpret_cast<float *>(xp + parts * rows_pad * kp);
    float *root = sums + rows_pad * (kp / 32);
    p.sums = sums, p.root = root;
    scan_hold(&p.hold, &p.hold_cycles);
    CUtensorMap tm;
    if (!make_map_k64(&tm, xp, static_cast<uint64_t>(kp), static_cast<uint64_t>(parts * rows_pad), static_cast<uint32_t>(R)))
        return DFLASH2_ERR_CUDA;
    CUtensorMap tc;
    if (!codes_map(&tc, w)) return DFLASH2_ERR_CUDA;
    auto prepare = f32x ? &k_linear4_rows<true> : &k_linear4_rows<false>;
    prepare<<<static_cast<unsigned>(rows_pad), 256, 0, s>>>(x, rows, x_stride, static_cast<int>(w->K), p.lg, 2 * p.kpairs, R,
                                                            exact, xp, sums, root);
    const dflash2_status st = after_launch();
    if (st != DFLASH2_OK) return st;
    if (f32x) return R == 16 ? launch_tc4_groups<8, true, 3>(tm, tc, p, s) : launch_tc4_groups<16, true, 3>(tm, tc, p, s);
    if (R == 16) return launch_tc4_kind<8>(tm, tc, p, exact, s);
    if (R == 32) return launch_tc4_kind<16>(tm, tc, p, exact, s);
    if (R == 64) return launch_tc4_kind<32>(tm, tc, p, exact, s);
    return exact ? launch_tc4<64, 0, true, 1>(tm, tc, p, s) : launch_tc4_groups<64, false, 1>(tm, tc, p, s);
}

unsigned int read_error_linear4(bool clear) {
    unsigned int v = 0;
    cudaMemcpyFromSymbol(&v, g_err_linear4, sizeof v);
    if (clear) {
        const unsigned int z = 0;
        cudaMemcpyToSymbol(g_err_linear4, &z, sizeof z);
    }
    return v;
}

}  // namespace dfl
