// attn_tc.cuh -- dflash2_paged_attn on the tensor cores (bf16 caches, head
// dimensions 64, 128 and 256).
//
// The rows of a block (tokens x query heads that share a cached head) are the
// narrow side of both products, so they go on the N side of the MMA and the
// keys and the head dimension on its 128-wide M side:
//   S^T [128 keys x N rows]  = K [128 x d] . Q^T       per tile of 128 keys
//   O^T [d x N rows]        += V^T [d x 128] . P^T      (d in blocks of 128)
// N is 16 to 128, so the softmax works on the rows there are; padded to the M
// side, a single token's few rows would cost it 128.  (The products take the
// same time either way: 56 cycles for 16 steps of the contraction at N up to
// 64, 64 cycles at 128, whatever the operands' layouts.)  K and V tiles go
// from the pages to shared memory by TMA exactly as they lie there (V^T is
// the M-major reading of the same rows), and each is read once.
//
// One CTA per SM takes an equal stretch of the call's line of tiles
// (attn.cuh).  Warps 9 and 10 copy the keys and the values, page by page,
// each through a ring of its own; warp 11 copies the queries.
// Warp 8 issues the MMAs, the next tile's scores before this tile's output
// product.  Warps 0-3 take the first half of the rows and warps 4-7 the
// second, each thread one key: it reads the key's scores from tensor memory,
// takes p = 2^(x - m) with the row's reference m, adds p to its own share of
// the row sums (reduced over the threads only at the end of an item) and
// writes P^T for the second product.  The halves share no row, so within a tile
// they wait for each other only where some rows see a key and some do not: there
// they vote on whether its values are finite.
// The reference m of a row is the maximum of the item's first tile and moves
// only when a score exceeds it by more than 8 (p <= 256, so nothing
// overflows, and the result is the same up to rounding): then the sums and
// O^T are multiplied by 2^(m - m'), which is rare.
//
// Bound: HBM.  A tile is d * 512 bytes, 2800 cycles of an SM's share of the
// bandwidth for d = 128, and 900 to 1000 cycles of the tensor cores.
// Measured (d 128 unless said, bytes of keys and values over the time):
//   one token, 5 rows, 131071 slots x 8 heads         89 us, 6.0 TB/s
//   32 requests of 1 to 16384 slots, 40 rows         182 us, 6.1 TB/s
//   16 requests of 500 to 16384 slots, d 256, 96 rows 116 us, 4.9 TB/s
//   64 requests, window 2048, 40 rows                 63 us, 4.0 TB/s
//   32 requests of 8 to 8192 slots, 64 rows          102 us, 4.7 TB/s
// What is left is the change from item to item, 10000 to 16000 cycles: the eight
// softmax warps take the last product's drain, the outputs and the join of cut
// items one after the other, and the next item's copies and first scores, which
// run ahead, wait for them.  (Warps of their own for it would need registers:
// 384 threads have 168 each.)  With wide heads and 96 rows the ring holds one
// tile, so copies also wait for products.
// Long blocks (prompts) are right but slow: every row block walks all slots that
// some token of the block's request sees.  8192 tokens, 40 heads on 8: 5300 us for
// 687 GFLOP of visible pairs.
// Tried and slower: one ring for keys and values (256 us for the second case
// with four times the copies per tile), a lane looping over a tile's copies
// (340 us), cp.async (3 TB/s at best).
//
// Rounding: scores, sums and O^T are fp32; P is rounded to bf16 because the
// MMA takes bf16 beside bf16 values; the sums are of the unrounded p.
//
// Waits are bounded: after a time-out every role stops waiting, the error
// word is set and the CTA's outputs are NaN.
#pragma once

#include "attn.cuh"
#include "tc.cuh"

namespace dfl {

constexpr int TK = 128;            // keys per tile
constexpr int SLOT_BYTES = 16384;  // 128 keys x 64 dims: the swizzle's width
constexpr int TC_THREADS = 384;    // warps 0-3 and 4-7 softmax (half of the rows each), 8 MMA, 9-11 copies
constexpr int MMA_WARP = 8, K_WARP = 9, V_WARP = 10, Q_WARP = 11;
constexpr int HOLES = 16;          // tiles whose flags are kept: more than the ring holds
constexpr int MAX_UNITS = 12;
constexpr float M_STEP = 8.f;      // a row's reference moves when a score exceeds it by more (in log2)
// The reference of a row that has seen nothing: below every finite score, so that the first one replaces it or, if it is
// no larger, is taken from it.
constexpr float M_NONE = -3.402823466e38f;
// x = s c2 - m in one fused step leaves what the reference's own product was rounded by, up to ulp(m) / 2: nothing to
// speak of, but past this reference 2 and more, and past 2^31 more than an exponent holds.
constexpr float M_HUGE = 16777216.f;
constexpr long long TC_WAIT = 4000000000ll;  // ~2 s
constexpr long long TC_DRAIN = 200000000ll;  // ~0.1 s
constexpr int SM_BYTES = 232448;   // shared memory of a CTA

struct TcShared {
    uint64_t full[MAX_UNITS], empty[MAX_UNITS];
    uint64_t s_full[2];   // scores of tile n in buffer n & 1
    uint64_t p_full[2];   // P of tile n written (weights pass: its scores read)
    uint64_t pv_done[2];  // output product of tile n complete
    uint64_t q_full, q_empty, done;
    int row_at[128];  // index of the row in lse (times d: in out) from the item's first row's
    int scratch[TC_THREADS / 32 + 2];
    alignas(16) float neg_m[128];
    alignas(16) float fac[128];
    float part[4][128];
    float inv[128];
    int hole[HOLES];        // tile n has slots without a page
    int filled[MAX_UNITS];  // rounds of the ring in which a unit was filled
    alignas(16) unsigned short side[256];
    uint32_t bad[4];
    uint32_t tmem;
    int abort, acc_first, flag, q_filled;
};

// A head dimension's slots and units, and a call's ring.
template <int DS>  // 64-dim slots of a row
struct TcDims {
    static constexpr int US = DS > 1 ? 2 : 1;  // slots of a unit: what a copy, its barriers and a block of V^T cover
    static constexpr int UPT = DS / US;        // units of a tile's keys, and of its values; blocks of O^T
    static constexpr int UNIT = US * SLOT_BYTES;
};
static __host__ __device__ constexpr int q_bytes(int n, int ds) { return n * ds * 128; }
static __host__ __device__ constexpr int p_bytes(int n) { return n * TK * 2; }
// Two P buffers where they are small.
static __host__ __device__ constexpr int p_bufs(int n) { return n > 64 ? 1 : 2; }
static __host__ __device__ constexpr int ring_units(int n, int ds) {
    const int rest = SM_BYTES - 1024 - static_cast<int>(sizeof(TcShared)) - 256 - q_bytes(n, ds) - p_bufs(n) * p_bytes(n);
    const int units = rest / ((ds > 1 ? 2 : 1) * SLOT_BYTES);
    return units < MAX_UNITS ? units : MAX_UNITS;
}
// The ring's units for values: half, and at least a tile's (the softmax warps may wait for all of a tile's values
// before its product starts); the rest are for keys, which are consumed unit by unit.
static __host__ __device__ constexpr int v_units(int n, int ds) {
    const int half = ring_units(n, ds) / 2, upt = ds > 2 ? 2 : 1;
    return half > upt ? half : upt;
}
static __host__ __device__ constexpr int tc_smem(int n, int ds) {
    return 1024 + ring_units(n, ds) * (ds > 1 ? 2 : 1) * SLOT_BYTES + q_bytes(n, ds) + p_bufs(n) * p_bytes(n);
}
static __host__ __device__ constexpr int tmem_cols(int need) {
    return need <= 64 ? 64 : need <= 128 ? 128 : need <= 256 ? 256 : 512;
}

__device__ __forceinline__ uint32_t tc_idesc(int n, bool major_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10)           // D fp32, A and B bf16
           | (major_mn ? (1u << 15) | (1u << 16) : 0u)  // both operands M- / N-major
           | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(TK >> 4) << 24);
}
// V^T: M-major, 128-byte swizzle; 8-key groups 1024 bytes apart, the second 64 dims one slot further (0: the
// same 64 dims again).
__device__ __forceinline__ uint64_t v_desc(const void *smem, uint32_t second) {
    return ((static_cast<uint64_t>(smem_addr(smem)) & 0x3ffffull) >> 4) | (static_cast<uint64_t>(second >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// P^T: N-major, no swizzle: 8 rows of one key are 16 bytes, 8 keys 128 bytes, the next 8 rows TK * 16 bytes further.
__device__ __forceinline__ uint64_t p_desc(const void *smem) {
    return ((static_cast<uint64_t>(smem_addr(smem)) & 0x3ffffull) >> 4) | (static_cast<uint64_t>(128 >> 4) << 16) |
           (static_cast<uint64_t>(TK * 16 >> 4) << 32) | (1ull << 46);
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld8_nowait(uint32_t taddr, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
                 : "memory");
}
// C columns (a multiple of 8) of the warp's lanes.
template <int C>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t *r) {
#pragma unroll
    for (int i = 0; i + 16 <= C; i += 16) tmem_ld16_nowait(taddr + i, r + i);
    if (C % 16) tmem_ld8_nowait(taddr + C - 8, r + C - 8);
    tmem_wait_ld();
}

__device__ __forceinline__ void tma_load_4d(void *sdst, const CUtensorMap *tmap, int x, int y, int z, int w,
                                            uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, "
        "%6}], [%2];" ::"r"(smem_addr(sdst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// Barriers of one softmax group (half) or of both (each warp reconverges first).
__device__ __forceinline__ void soft_sync(int half) {
    __syncwarp();
    asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
}
__device__ __forceinline__ void both_sync() {
    __syncwarp();
    asm volatile("bar.sync 3, 256;" ::: "memory");
}
__device__ __forceinline__ bool soft_any(int half, bool p) {
    __syncwarp();
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(p ? 1u : 0u), "r"(1 + half)
        : "memory");
    return r != 0;
}
// ... over both groups.
__device__ __forceinline__ bool both_any(bool p) {
    __syncwarp();
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 3, 256, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(p ? 1u : 0u)
        : "memory");
    return r != 0;
}

// ... with an L2 policy for the lines it reads.
__device__ __forceinline__ void tma_load_4d_hint(void *sdst, const CUtensorMap *tmap, int x, int y, int z, int w,
                                                 uint64_t *bar, uint64_t pol) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, "
        "{%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_addr(sdst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z), "r"(w), "l"(pol)
        : "memory");
}

__device__ __forceinline__ bool tc_aborted(TcShared &sm) { return *reinterpret_cast<volatile int *>(&sm.abort) != 0; }
// A bounded wait that gives up at once when another role has.
static __device__ __noinline__ bool tc_wait_long(TcShared &sm, uint64_t *bar, uint32_t parity, unsigned int *err) {
    const long long t0 = clock64();
    while (!tc_aborted(sm)) {
        if (mbar_try_wait(bar, parity)) return true;
        if (clock64() - t0 > TC_WAIT) {
            atomicOr(err, ERR_WAIT_TIMEOUT);
            *reinterpret_cast<volatile int *>(&sm.abort) = 1;
        }
    }
    return false;
}
__device__ __forceinline__ bool tc_wait(TcShared &sm, uint64_t *bar, uint32_t parity, unsigned int *err) {
    return mbar_try_wait(bar, parity) || tc_wait_long(sm, bar, parity, err);
}

// Test hook: warp `warp` waits for the hook's word; if that runs out it takes
// no part in the work, as after any time-out.  (Asked before the roles begin:
// within the copying warps' loops the question alone cost 1 to 2 us a call.)
__device__ __forceinline__ bool tc_hold(TcShared &sm, const AttnArgs &a, int warp) {
    if (a.hold == nullptr || static_cast<int>(threadIdx.x >> 5) != warp) return true;
    int seen = 1;
    if ((threadIdx.x & 31) == 0 && !hold_wait(a.hold, a.hold_cycles)) {
        atomicOr(a.err, ERR_WAIT_TIMEOUT);
        *reinterpret_cast<volatile int *>(&sm.abort) = 1;
        seen = 0;
    }
    return __shfl_sync(FULL, seen, 0) != 0;
}

// A place in the ring of keys (units 0 .. K - 1) or of values (the others).
// Each has one warp that fills it and one that empties it, both in order, so
// neither is ever more than a round ahead and a phase's parity tells it apart.
template <int FIRST, int COUNT>
struct RingPos {
    int unit = FIRST;
    uint32_t round = 0;
    __device__ __forceinline__ void step() {
        if (++unit == FIRST + COUNT) {
            unit = FIRST;
            ++round;
        }
    }
};

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// A request's page table, 64 entries of it at a time in the warp's registers:
// the reads are far ahead of their use.
struct PageWindow {
    const int32_t *table;
    int used, at;    // entries the request's slots need; the window's first
    int now, next;   // entries at + lane and at + 32 + lane

    __device__ __forceinline__ int load(int i) const { return i < used ? table[i] : -1; }
    __device__ __forceinline__ void start(const AttnArgs &a, const AttnWalk &w, int lane) {
        table = a.table + static_cast<int64_t>(w.b) * a.max_pages;
        used = w.r.n == 0 ? 0 : (w.r.n - 1) / a.page_size + 1;
        at = w.t0 * TK / a.page_size;
        now = load(at + lane);
        next = load(at + 32 + lane);
    }
    // Entry i of every lane, at least the window's first and less than 64 ahead of it.
    __device__ __forceinline__ int get(int i) const {
        const int k = i - at, lo = __shfl_sync(FULL, now, k & 31), hi = __shfl_sync(FULL, next, k & 31);
        return k < 32 ? lo : hi;
    }
    // No entry before `first` is asked for any more.
    __device__ __forceinline__ void advance(int first, int lane) {
        if (first >= at + 32) {
            at += 32;
            now = next;
            next = load(at + 32 + lane);
        }
    }
};
// The lane's box of the tiles of an item: lane l holds box l % (128 / box), the
// part of a tile that one page's copy covers.
struct BoxAt {
    int pi, off, s;  // entry of the request's table, offset in the page, slot number
    int page;        // -1: no slots in use, or no page

    __device__ __forceinline__ void start(const AttnArgs &a, const AttnWalk &w, int box_log2, int lane) {
        s = w.t0 * TK + ((lane & ((TK >> box_log2) - 1)) << box_log2);
        pi = s / a.page_size;
        off = s - pi * a.page_size;
    }
    __device__ __forceinline__ void look(const AttnArgs &a, const AttnWalk &w, PageWindow &pages, int lane) {
        pages.advance(__shfl_sync(FULL, pi, 0), lane);
        page = pages.get(pi);
        if (s >= w.r.n || static_cast<unsigned>(page) >= static_cast<unsigned long long>(a.num_pages)) page = -1;
    }
    __device__ __forceinline__ void step(const AttnArgs &a, int dpi, int doff) {
        s += TK;
        pi += dpi;
        off += doff;
        if (off >= a.page_size) {
            off -= a.page_size;
            ++pi;
        }
    }
};

// Copies a tile's keys or values (UPT units).  All lanes of the copying warp:
// each its box of one of the unit's 64-dim slots (a loop of one lane over the
// boxes takes up to twice as long).
template <int DS, typename Ring>
__device__ __forceinline__ bool copy_tile(TcShared &sm, unsigned char *ring, Ring &rp, bool leader,
                                          const CUtensorMap *map, const BoxAt &box, int box_log2, int h, uint64_t pol,
                                          unsigned int *err) {
    using D = TcDims<DS>;
    const int nb = TK >> box_log2, lane = threadIdx.x & 31, slot = lane / nb;
    const int dst = slot * SLOT_BYTES + (((lane & (nb - 1)) << box_log2) * 128);
    const unsigned there = __ballot_sync(FULL, box.page >= 0) & ((1u << nb) - 1u);
#pragma unroll
    for (int u = 0; u < D::UPT; ++u) {
        bool ok = true;
        if (leader) {
            ok = rp.round == 0 || tc_wait(sm, &sm.empty[rp.unit], (rp.round - 1) & 1, err);
            if (ok) {
                sm.filled[rp.unit] = rp.round + 1;
                mbar_arrive_expect_tx(&sm.full[rp.unit], (__popc(there) << box_log2) * 128 * D::US);
            }
        }
        if (!__all_sync(FULL, ok)) return false;
        if (box.page >= 0 && slot < D::US)
            tma_load_4d_hint(ring + rp.unit * D::UNIT + dst, map, (u * D::US + slot) * 64, box.off, h, box.page,
                             &sm.full[rp.unit], pol);
        rp.step();
    }
    return true;
}

// One tile's score product from the ring's next units; kd and qd describe the
// ring's and Q's first 64 dims.
template <int DS, typename Ring>
__device__ __forceinline__ bool issue_scores(TcShared &sm, uint64_t kd, uint64_t qd, Ring &rp,
                                             uint32_t d_tmem, uint32_t idesc, int N, unsigned int *err) {
    using D = TcDims<DS>;
#pragma unroll
    for (int u = 0; u < D::UPT; ++u) {
        if (!tc_wait(sm, &sm.full[rp.unit], rp.round & 1, err)) return false;
        tc_fence_after();
        const uint64_t ud = kd + rp.unit * (D::UNIT >> 4);
#pragma unroll
        for (int s = 0; s < D::US; ++s)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                mma_bf16(d_tmem, ud + s * (SLOT_BYTES >> 4) + 2 * k, qd + (u * D::US + s) * (N * 128 >> 4) + 2 * k,
                         idesc, u > 0 || s > 0 || k > 0);
        mma_commit(&sm.empty[rp.unit]);
        rp.step();
    }
    return true;
}

__device__ __forceinline__ void st_bf16(unsigned short *p, float v) {
    unsigned short o;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(o) : "f"(v));
    *p = o;
}
__device__ __forceinline__ bool bad_bf16(uint32_t h) { return (h & 0x7f80u) == 0x7f80u; }

// Sums of v[0 .. 7] over the warp's lanes: lane l returns row l / 4's.
__device__ __forceinline__ float lane_sums8(const float *v, int lane) {
    float a[4], b[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float send = (lane & 16) ? v[i] : v[i + 4], keep = (lane & 16) ? v[i + 4] : v[i];
        a[i] = keep + __shfl_xor_sync(FULL, send, 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float send = (lane & 8) ? a[i] : a[i + 2], keep = (lane & 8) ? a[i + 2] : a[i];
        b[i] = keep + __shfl_xor_sync(FULL, send, 8);
    }
    const float send = (lane & 4) ? b[0] : b[1], keep = (lane & 4) ? b[1] : b[0];
    float c = keep + __shfl_xor_sync(FULL, send, 4);
    c += __shfl_xor_sync(FULL, c, 2);
    return c + __shfl_xor_sync(FULL, c, 1);
}

// The same for maxima.
__device__ __forceinline__ float lane_max8(const float *v, int lane) {
    float a[4], b[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float send = (lane & 16) ? v[i] : v[i + 4], keep = (lane & 16) ? v[i + 4] : v[i];
        a[i] = fmaxf(keep, __shfl_xor_sync(FULL, send, 16));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float send = (lane & 8) ? a[i] : a[i + 2], keep = (lane & 8) ? a[i + 2] : a[i];
        b[i] = fmaxf(keep, __shfl_xor_sync(FULL, send, 8));
    }
    const float send = (lane & 4) ? b[0] : b[1], keep = (lane & 4) ? b[1] : b[0];
    float c = fmaxf(keep, __shfl_xor_sync(FULL, send, 4));
    c = fmaxf(c, __shfl_xor_sync(FULL, c, 2));
    return fmaxf(c, __shfl_xor_sync(FULL, c, 1));
}

// Barriers, tensor memory, and Q's rows that no copy reaches (they stay zero).
__device__ __forceinline__ void tc_setup(TcShared &sm, unsigned char *sq, int qbytes, int units, int cols, int readers) {
    const int tid = threadIdx.x;
    if (tid == 0) {
        for (int i = 0; i < units; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
            sm.filled[i] = 0;
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_full[i], readers);
            mbar_init(&sm.pv_done[i], 1);
        }
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_empty, 1);
        mbar_init(&sm.done, 1);
        sm.abort = 0;
        sm.acc_first = 0;
        sm.q_filled = 0;
        fence_barrier_init();
    }
    if (tid / 32 == MMA_WARP) tmem_alloc(&sm.tmem, cols);
    for (int i = tid; i < qbytes / 16; i += TC_THREADS) reinterpret_cast<uint4 *>(sq)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
}

template <int N, int DS>
__global__ void __launch_bounds__(TC_THREADS, 1) k_attn_tc(const __grid_constant__ CUtensorMap mk,
                                                           const __grid_constant__ CUtensorMap mv,
                                                           const __grid_constant__ CUtensorMap mq,
                                                           const __grid_constant__ AttnArgs a, int box_log2) {
    using D = TcDims<DS>;
    constexpr int UNITS = ring_units(N, DS), VU = v_units(N, DS), KU = UNITS - VU, NP = p_bufs(N), MB = D::UPT;
    static_assert(KU >= 1, "a unit for keys is left");
    using KRing = RingPos<0, KU>;
    using VRing = RingPos<KU, VU>;
    constexpr int COLS = tmem_cols(N * (2 + MB));
    extern __shared__ unsigned char raw[];
    __shared__ TcShared sm;
    unsigned char *ring =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *sq = ring + UNITS * D::UNIT, *sp = sq + q_bytes(N, DS);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    tc_setup(sm, sq, q_bytes(N, DS), UNITS, COLS, 8);
    const uint32_t tm_s = sm.tmem, tm_o = tm_s + 2 * N;
    unsigned int *err = a.err;
    pdl_wait();
    const AttnPlan plan = attn_plan<TC_THREADS>(a, sm.scratch);
    const bool work = plan.begin < plan.end && tc_hold(sm, a, V_WARP);
    AttnWalk w;
    if (work) w.start(a, plan);

    if (work && warp == Q_WARP) {
        // ------------------------------------------------------- copies --
        if (lane == 0) {
            uint32_t seg = 0;
            while (w.next(a)) {
                const int h = w.item / a.row_blocks, tok0 = (w.item % a.row_blocks) * a.tok_block;
                if (seg > 0 && !tc_wait(sm, &sm.q_empty, (seg - 1) & 1, err)) break;
                mbar_arrive_expect_tx(&sm.q_full, a.tok_block * a.group * 128 * DS);
#pragma unroll
                for (int s = 0; s < DS; ++s)
                    tma_load_4d(sq + s * N * 128, &mq, s * 64, h * a.group, tok0, w.b, &sm.q_full);
                sm.q_filled = ++seg;
            }
        }
        __syncwarp();
    } else if (work && warp >= K_WARP) {
        const bool keys = warp == K_WARP, leader = elect_one();
        const int dpi = TK / a.page_size, doff = TK % a.page_size;
        const uint64_t pol = l2_policy_evict_first();
        KRing kr;
        VRing vr;
        uint32_t n = 0;
        bool ok = true;
        while (ok && w.next(a)) {
            const int h = w.item / a.row_blocks, nt = w.t1 - w.t0;
            BoxAt box;
            PageWindow pages;
            box.start(a, w, box_log2, lane);
            pages.start(a, w, lane);
            for (int i = 0; ok && i < nt; ++i, ++n) {
                box.look(a, w, pages, lane);
                if (keys) {  // for the softmax warps: slots in use without a page
                    const bool hole = __any_sync(FULL, box.page < 0 && box.s < w.r.n);
                    if (leader) sm.hole[n % HOLES] = hole;
                    ok = copy_tile<DS>(sm, ring, kr, leader, &mk, box, box_log2, h, pol, err);
                } else {
                    ok = copy_tile<DS>(sm, ring, vr, leader, &mv, box, box_log2, h, pol, err);
                }
                box.step(a, dpi, doff);
            }
        }
        __syncwarp();
    } else if (work && warp == MMA_WARP) {
        // ---------------------------------------------------------- MMA --
        if (lane == 0) {
            KRing kr;
            VRing vr;
            const uint32_t ids = tc_idesc(N, false), idp = tc_idesc(N, true);
            const uint64_t kd = sw128_desc(ring), qd = sw128_desc(sq), pd = p_desc(sp);
            const uint64_t vd = v_desc(ring, DS > 1 ? SLOT_BYTES : 0);
            uint32_t seg = 0, n = 0;
            bool ok = true;
            while (ok && w.next(a)) {
                const int nt = w.t1 - w.t0;
                ok = tc_wait(sm, &sm.q_full, seg & 1, err) &&
                     issue_scores<DS>(sm, kd, qd, kr, tm_s + (n & 1) * N, ids, N, err);
                ++seg;
                if (!ok) break;
                mma_commit(&sm.s_full[n & 1]);
                if (nt == 1) mma_commit(&sm.q_empty);
                for (int i = 0; i < nt; ++i, ++n) {
                    if (i + 1 < nt) {
                        ok = issue_scores<DS>(sm, kd, qd, kr, tm_s + ((n + 1) & 1) * N, ids, N, err);
                        if (!ok) break;
                        mma_commit(&sm.s_full[(n + 1) & 1]);
                        if (i + 2 == nt) mma_commit(&sm.q_empty);
                    }
                    ok = tc_wait(sm, &sm.p_full[n & 1], (n >> 1) & 1, err);
                    if (!ok) break;
                    const uint64_t bd = pd + (n % NP) * (p_bytes(N) >> 4);
                    const bool acc = i > 0 || *reinterpret_cast<volatile int *>(&sm.acc_first) != 0;
#pragma unroll
                    for (int m = 0; m < MB; ++m) {
                        ok = tc_wait(sm, &sm.full[vr.unit], vr.round & 1, err);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t ad = vd + vr.unit * (D::UNIT >> 4);
#pragma unroll
                        for (int k = 0; k < TK / 16; ++k)  // 16 keys: 2048 bytes of V, 256 of P
                            mma_bf16(tm_o + m * N, ad + 128 * k, bd + 16 * k, idp, acc || k > 0);
                        mma_commit(&sm.empty[vr.unit]);
                        vr.step();
                    }
                    if (!ok) break;
                    mma_commit(&sm.pv_done[n & 1]);
                }
            }
            // every MMA issued has completed once this commit arrives
            mma_commit(&sm.done);
            mbar_wait(&sm.done, 0, TC_DRAIN);
        }
        __syncwarp();
    } else if (work) {
        // ------------------------------------------------------ softmax --
        constexpr int NR = N / 2;  // rows of this group: row0 .. row0 + NR - 1
        const int half = warp >> 2, key = tid & 127, row0 = half * NR;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const float c2 = a.scale * LOG2E;
        float *neg_m = sm.neg_m + row0, *fac = sm.fac + row0;
        uint32_t n = 0;  // tiles so far
        int seq = 0;     // units of values before this item's
        while (w.next(a)) {
            const int h = w.item / a.row_blocks, tok0 = (w.item % a.row_blocks) * a.tok_block;
            const int toks = min(a.tok_block, a.T - tok0), rows = toks * a.group;
            const int live = max(min(w.r.nq - tok0, toks), 0), real = live * a.group;
            const int nt = w.t1 - w.t0;
            const int64_t first_row = attn_row(a, w.b, h, tok0, 0);
            float l[NR];
#pragma unroll
            for (int i = 0; i < NR; ++i) l[i] = 0.f;
            if (key < NR) {
                neg_m[key] = -M_NONE;
                if (row0 + key < rows)
                    sm.row_at[row0 + key] = (row0 + key) / a.group * a.Hq + (row0 + key) % a.group;
            }
            if (tid == 0) sm.acc_first = 0;
            soft_sync(half);
            // With an array of positions a key's view takes two dependent loads: the page one tile further ahead than
            // the position.
            auto slot_page = [&](int t) {
                const int s = t * TK + key;
                return a.pos && t < w.t1 && s < w.r.n ? attn_page(a, w.b, s) : -1;
            };
            auto slot_pos = [&](int t, int page) {
                return page < 0 ? 0
                                : a.pos[(static_cast<int64_t>(page) * a.Hkv + h) * a.page_size +
                                        (t * TK + key) % a.page_size];
            };
            // Tiles [clean0, clean1) are seen by all rows in whole (if no page is missing).
            const int64_t see0 = w.r.q0 + tok0;  // the last position that the first row sees, causally
            int clean0 = 0, clean1 = 0;
            if (!a.pos && live > 0) {
                int64_t e = w.r.n;
                if (a.causal) e = min(e, see0 + 1);
                clean1 = static_cast<int>(max(e, static_cast<int64_t>(0)) / TK);
                if (a.window > 0)
                    clean0 = static_cast<int>(
                        min((max(see0 + live - a.window, static_cast<int64_t>(0)) + TK - 1) / TK, int64_t(1) << 30));
            }
            // This thread's key's values of tile i, 64 dims at a time (once they are there).  The ring may hold no more
            // than one tile's values: only after the product before tile i's are its units' last contents used up, and
            // the phase that is waited for the next one.
            auto v_row = [&](int i, int e) {
                const int q = seq + i * D::UPT + e / D::US;
                if (n > 0) tc_wait(sm, &sm.pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1, err);
                tc_wait(sm, &sm.full[KU + q % VU], (q / VU) & 1, err);
                return reinterpret_cast<uint4 *>(ring + ((KU + q % VU) * D::US + e % D::US) * SLOT_BYTES + key * 128);
            };
            int page_now = slot_page(w.t0), page_next = slot_page(w.t0 + 1);
            int pos_now = slot_pos(w.t0, page_now);
            bool huge = false;  // a row of the group has a reference beyond M_HUGE
            for (int i = 0; i < nt; ++i, ++n) {
                const int t = w.t0 + i, ks = t * TK;
                const int page_after = slot_page(t + 2), pos_next = slot_pos(t + 1, page_next);
                tc_wait(sm, &sm.s_full[n & 1], (n >> 1) & 1, err);
                __syncwarp();
                tc_fence_after();
                const uint32_t ts = tm_s + lanes + (n & 1) * N + row0;
                float x[NR];
                tmem_ld<NR>(ts, reinterpret_cast<uint32_t *>(x));
                // which rows see this thread's key; nothing to look at if all rows see the whole tile
                int r0 = 0, r1 = NR;
                bool none = false, poison = false;
                const bool hole = *reinterpret_cast<volatile int *>(&sm.hole[n % HOLES]);
                bool masked = hole || t < clean0 || t >= clean1;
                if (masked) {
                    int lo = 0, hi = 0;
                    if (a.pos) {
                        if (page_now >= 0) attn_view(a, w.r, pos_now, lo, hi);
                    } else if (ks + key < w.r.n && (!hole || attn_page(a, w.b, ks + key) >= 0)) {
                        attn_view(a, w.r, ks + key, lo, hi);
                    }
                    lo = max(lo - tok0, 0) * a.group;
                    hi = min((hi - tok0) * a.group, real);
                    none = lo >= hi;
                    const bool part = !none && (lo > 0 || hi < real);
                    r0 = lo - row0;
                    r1 = none ? r0 : hi - row0;
                    masked = __any_sync(FULL, none || part);
                    // Of a key that only some rows see, values that are not finite are taken out of the tile and
                    // added by hand: p = 0 times NaN would be NaN.
                    if (part) {
                        for (int e = 0; e < DS; ++e) {
                            const uint4 *row = v_row(i, e);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const uint4 v = row[j];
                                poison = poison || bad_bf16(v.x) || bad_bf16(v.x >> 16) || bad_bf16(v.y) ||
                                         bad_bf16(v.y >> 16) || bad_bf16(v.z) || bad_bf16(v.z >> 16) ||
                                         bad_bf16(v.w) || bad_bf16(v.w >> 16);
                            }
                        }
                    }
                    // Values of a key that no row sees are set to zero.
                    if (none && half == 0) {
                        for (int e = 0; e < DS; ++e) {
                            uint4 *row = v_row(i, e);
#pragma unroll
                            for (int j = 0; j < 8; ++j) row[j] = make_uint4(0, 0, 0, 0);
                        }
                    }
                    __syncwarp();
                }
                // x = s f - m, in place
                auto exponents = [&](float f) {
#pragma unroll
                    for (int j = 0; j < NR; j += 4) {
                        const float4 m = *reinterpret_cast<const float4 *>(neg_m + j);
                        x[j] = fmaf(x[j], f, m.x);
                        x[j + 1] = fmaf(x[j + 1], f, m.y);
                        x[j + 2] = fmaf(x[j + 2], f, m.z);
                        x[j + 3] = fmaf(x[j + 3], f, m.w);
                    }
                    if (masked) {
#pragma unroll
                        for (int j = 0; j < NR; ++j)
                            if (j < r0 || j >= r1) x[j] = NEG_INF;
                    }
                };
                bool slow = true;
                if (i > 0) {
                    exponents(c2);
                    float xm = NEG_INF;
#pragma unroll
                    for (int j = 0; j < NR; ++j) xm = fmaxf(xm, x[j]);
                    slow = soft_any(half, xm > M_STEP || poison || huge);
                }
                if (slow) {
                    // the rows' maxima over the tile, new references, and what has been summed scaled to them
                    if (i > 0) tmem_ld<NR>(ts, reinterpret_cast<uint32_t *>(x));
#pragma unroll
                    for (int c = 0; c < NR; c += 8) {
                        float y[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            y[j] = masked && (c + j < r0 || c + j >= r1) ? NEG_INF : x[c + j] * c2;
                        const float v = lane_max8(y, lane);
                        if ((lane & 3) == 0) sm.part[warp & 3][row0 + c + lane / 4] = v;
                    }
                    soft_sync(half);
                    bool far = false;
                    if (key < NR) {
                        const int r = row0 + key;
                        const float mo = -neg_m[key];
                        float mn = fmaxf(fmaxf(sm.part[0][r], sm.part[1][r]), fmaxf(sm.part[2][r], sm.part[3][r]));
                        mn = fmaxf(mn, mo);
                        fac[key] = ex2(mo - mn);
                        neg_m[key] = -mn;
                        far = mn != M_NONE && fabsf(mn) > M_HUGE;
                    }
                    huge = soft_any(half, far);
                    if (huge) {  // the products rounded as the references are
#pragma unroll
                        for (int j = 0; j < NR; ++j) x[j] *= c2;
                    }
                    exponents(huge ? 1.f : c2);
                    if (i > 0) {
#pragma unroll
                        for (int j = 0; j < NR; ++j) l[j] *= fac[j];
                        tc_wait(sm, &sm.pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1, err);
                        __syncwarp();
                        tc_fence_after();
                        for (int m = 0; m < MB; ++m)
                            for (int j = 0; j < NR; j += 8) {
                                uint32_t o[8];
                                float f[8];
                                const uint32_t at = tm_o + lanes + m * N + row0 + j;
                                tmem_ld<8>(at, o);
#pragma unroll
                                for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(o[k]) * fac[j + k];
                                tmem_st8(at, f);
                            }
                        tmem_wait_st();
                    }
                }
                uint32_t pk[NR / 2];
#pragma unroll
                for (int j = 0; j < NR; j += 2) {
                    const float p0 = ex2(x[j]), p1 = ex2(x[j + 1]);
                    l[j] += p0;
                    l[j + 1] += p1;
                    pk[j / 2] = pack_bf16(p0, p1);
                }
                // P buffer n % np is free once the product that read it last is done
                if (n >= NP) {
                    const uint32_t k = n - NP;
                    tc_wait(sm, &sm.pv_done[k & 1], (k >> 1) & 1, err);
                    __syncwarp();
                }
                unsigned char *pb = sp + (n % NP) * p_bytes(N);
#pragma unroll
                for (int j = 0; j < NR; j += 8)
                    *reinterpret_cast<uint4 *>(pb + ((row0 + j) / 8) * (TK * 16) + key * 16) =
                        make_uint4(pk[j / 2], pk[j / 2 + 1], pk[j / 2 + 2], pk[j / 2 + 3]);
                // Keys that some rows see and some do not, with values that are not finite: their products with p go
                // straight into O^T.  Both groups vote, in every tile that can hold such keys, and go through them
                // together: whether they do hangs on nothing that a time-out leaves open to one of them alone.
                if ((a.pos || t < clean0 || t >= clean1) && both_any(poison)) {
                    const int vseq = seq + i * D::UPT;
                    const unsigned mine = __ballot_sync(FULL, poison);
                    if (half == 0 && lane == 0) sm.bad[warp] = mine;
                    if (i == 0) {
                        float z[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) z[j] = 0.f;
                        for (int m = 0; m < MB; ++m)
                            for (int j = 0; j < NR; j += 8) tmem_st8(tm_o + lanes + m * N + row0 + j, z);
                        tmem_wait_st();
                        if (tid == 0) sm.acc_first = 1;
                    }
                    both_sync();
                    for (int k = 0; k < TK; ++k) {
                        if (!(sm.bad[k >> 5] >> (k & 31) & 1)) continue;
                        if (tid == k) {
                            for (int e = 0; e < DS * 64; ++e) {
                                const int q = vseq + e / 64 / D::US, chunk = (e % 64) / 8;
                                unsigned short *v = reinterpret_cast<unsigned short *>(
                                    ring + ((KU + q % VU) * D::US + e / 64 % D::US) * SLOT_BYTES + k * 128 +
                                    ((chunk ^ (k & 7)) * 16) + (e % 8) * 2);
                                const bool b = bad_bf16(*v);
                                sm.side[e] = b ? *v : 0;
                                if (b) *v = 0;
                            }
                        }
                        both_sync();
                        for (int m = 0; m < MB; ++m) {
                            const int e = DS > 1 ? m * 128 + key : key & 63;
                            const float v = __uint_as_float(static_cast<uint32_t>(sm.side[e]) << 16);
                            for (int r = row0; r < row0 + NR; r += 8) {
                                uint32_t o[8];
                                float f[8];
                                tmem_ld<8>(tm_o + lanes + m * N + r, o);
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    const unsigned short pk = *reinterpret_cast<const unsigned short *>(
                                        pb + (r / 8) * (TK * 16) + k * 16 + j * 2);
                                    const float p = __uint_as_float(static_cast<uint32_t>(pk) << 16);
                                    f[j] = __uint_as_float(o[j]);
                                    if (p != 0.f && v != 0.f) f[j] = fmaf(p, v, f[j]);
                                }
                                tmem_st8(tm_o + lanes + m * N + r, f);
                            }
                        }
                        tmem_wait_st();
                        both_sync();
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_full[n & 1]);
                page_now = page_next;
                page_next = page_after;
                pos_now = pos_next;
            }
            seq += nt * D::UPT;
            // the rows' sums over all keys
#pragma unroll
            for (int j = 0; j < NR; j += 8) {
                const float v = lane_sums8(l + j, lane);
                if ((lane & 3) == 0) sm.part[warp & 3][row0 + j + lane / 4] = v;
            }
            soft_sync(half);
            const int mine = min(rows - row0, NR);  // rows of this group (none or negative: the group has none)
            float L = 0.f;
            const float m_row = key < NR ? -neg_m[key] : 0.f;
            if (key < mine) {
                const int r = row0 + key;
                L = r < real ? sm.part[0][r] + sm.part[1][r] + sm.part[2][r] + sm.part[3][r] : 0.f;
            }
            // An item cut in two whose other part is there is joined at once with what is still in tensor memory (the
            // next CTA takes its part first, so this is the usual case at the end of a stretch).
            const AttnParts q(a, plan, w);
            float *scratch = reinterpret_cast<float *>(sp);  // once the last product has read P
            if (!w.whole && tid == 0) {
                int there;
                asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(there) : "l"(a.tickets + q.c0) : "memory");
                sm.flag = q.n == 2 && there == 1;
            }
            tc_wait(sm, &sm.pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1, err);
            both_sync();
            tc_fence_after();
            if (tc_aborted(sm)) L = NAN;  // asked once nothing of the item is waited for any more
            const bool direct = !w.whole && sm.flag != 0;
            const int own = direct ? static_cast<int>(blockIdx.x) - q.c0 : -1;
            float *part = w.whole || direct ? nullptr : attn_part(a, blockIdx.x, w.starts);
            if (key < mine) {
                const int r = row0 + key;
                if (part) {
                    sm.inv[r] = L == 0.f ? 0.f : 1.f;
                    part[a.rows_cap * a.d + r] = m_row;
                    part[a.rows_cap * (a.d + 1) + r] = L;
                } else {
                    float lse = L == 0.f ? NEG_INF : (m_row + log2f(L)) * 0.6931471805599453f, g = L == 0.f ? 0.f : 1.0f / L;
                    if (direct) {
                        __threadfence();
                        const float *x = q.at(own ^ 1) + static_cast<int64_t>(a.rows_cap) * a.d + r;
                        float ml[4];
                        ml[own] = m_row;
                        ml[own ^ 1] = __ldcg(x);
                        ml[2 + own] = L;
                        ml[2 + (own ^ 1)] = r < real ? __ldcg(x + a.rows_cap) : 0.f;
                        g = attn_join_row(2, ml, ml + 2, &lse);
                        scratch[2 * r] = ml[0];
                        scratch[2 * r + 1] = ml[1];
                    }
                    sm.inv[r] = g;
                    if (a.lse) a.lse[first_row + sm.row_at[r]] = lse;
                }
            }
            soft_sync(half);
            if (DS > 1 || (warp & 3) < 2) {
                unsigned short *out = static_cast<unsigned short *>(a.out) + first_row * (DS * 64);
                constexpr int CR = NR % 24 == 0 ? 24 : NR % 16 == 0 ? 16 : 8;  // rows at a time
#pragma unroll 1
                for (int m = 0; m < MB; ++m) {
                    const int e = m * 128 + key;
#pragma unroll 1
                    for (int j0 = 0; j0 < mine; j0 += CR) {
                        float o[CR];
                        tmem_ld<CR>(tm_o + lanes + m * N + row0 + j0, reinterpret_cast<uint32_t *>(o));
                        if (direct) {
                            // f0 x0 + f1 x1 in the parts' order, as attn_join_sum has it
                            const int last = mine - 1 - j0;
                            const float *src = q.at(own ^ 1) + (row0 + j0) * (DS * 64) + e;
                            float x[CR];
#pragma unroll
                            for (int j = 0; j < CR; ++j) x[j] = __ldcg(src + min(j, last) * (DS * 64));
#pragma unroll
                            for (int j = 0; j < CR; ++j) {
                                const float2 f = *reinterpret_cast<const float2 *>(scratch + 2 * (row0 + j0 + min(j, last)));
                                const float x0 = own == 0 ? o[j] : x[j], x1 = own == 0 ? x[j] : o[j];
                                float sum = f.x == 0.f ? 0.f : fmaf(x0, f.x, 0.f);
                                sum = f.y == 0.f ? sum : fmaf(x1, f.y, sum);
                                o[j] = sum;
                            }
                        }
#pragma unroll
                        for (int j = 0; j < CR; ++j) {
                            const int r = row0 + j0 + j;
                            const float f = sm.inv[r];
                            const float v = f == 0.f ? 0.f : o[j] * f;
                            if (j0 + j < mine) {
                                if (part)
                                    part[r * (DS * 64) + e] = v;
                                else
                                    st_bf16(out + sm.row_at[r] * (DS * 64) + e, v);
                            }
                        }
                    }
                }
            }
            tc_fence_before();
            both_sync();
            if (direct && tid == 0) a.tickets[q.c0] = 0;
            if (part) {
                attn_join<unsigned short, DS * 64>(a, q, w, rows, tok0, 256, tid, &sm.flag, scratch, p_bytes(N) / 4,
                                                   sm.inv, first_row, sm.row_at, both_sync);
                both_sync();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tc_aborted(sm)) {  // leave no copy in flight into this CTA's shared memory
        if (tid < UNITS && sm.filled[tid] > 0) mbar_wait(&sm.full[tid], (sm.filled[tid] - 1) & 1, TC_DRAIN);
        if (tid == UNITS && sm.q_filled > 0) mbar_wait(&sm.q_full, (sm.q_filled - 1) & 1, TC_DRAIN);
        __syncthreads();
    }
    if (warp == MMA_WARP) tmem_dealloc(tm_s, COLS);
}

// weight_s += sum over the rows that see s of exp(x_s - lse): the second pass,
// over the keys alone, with the first one's lse.  Work is cut by (request,
// cached head) and a row block is a round over the stretch's tiles, so one
// CTA has all of a key's rows, one thread adds to a key's word, and its
// additions have an order.  Warps 0-3 take the even tiles and warps 4-7 the
// odd ones, each thread one key and all rows.  Bound: the keys' bytes; 16
// requests of 2048 to 4160 slots x 8 heads of 128, 4 rows: 30 us (105 MB, 3.5
// TB/s), of them 10 before the first tile and after the last.
template <int N, int DS>
__global__ void __launch_bounds__(TC_THREADS, 1) k_weights_tc(const __grid_constant__ CUtensorMap mk,
                                                              const __grid_constant__ CUtensorMap mq,
                                                              const __grid_constant__ AttnArgs a, int box_log2) {
    using D = TcDims<DS>;
    constexpr int UNITS = ring_units(N, DS), COLS = tmem_cols(2 * N);
    using KRing = RingPos<0, UNITS>;
    extern __shared__ unsigned char raw[];
    __shared__ TcShared sm;
    unsigned char *ring =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *sq = ring + UNITS * D::UNIT;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    tc_setup(sm, sq, q_bytes(N, DS), UNITS, COLS, 4);
    const uint32_t tm_s = sm.tmem;
    unsigned int *err = a.err;
    pdl_wait();
    const AttnPlan plan = attn_plan<TC_THREADS>(a, sm.scratch);
    const bool work = plan.begin < plan.end && tc_hold(sm, a, K_WARP);
    AttnWalk w;
    if (work) w.start(a, plan);

    if (work && warp == Q_WARP) {
        if (lane == 0) {
            uint32_t seg = 0;
            bool ok = true;
            while (ok && w.next(a)) {
                for (int rb = 0; ok && rb < a.row_blocks; ++rb) {
                    ok = seg == 0 || tc_wait(sm, &sm.q_empty, (seg - 1) & 1, err);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&sm.q_full, a.tok_block * a.group * 128 * DS);
#pragma unroll
                    for (int s = 0; s < DS; ++s)
                        tma_load_4d(sq + s * N * 128, &mq, s * 64, w.item * a.group, rb * a.tok_block, w.b, &sm.q_full);
                    sm.q_filled = ++seg;
                }
            }
        }
        __syncwarp();
    } else if (work && warp == K_WARP) {
        const bool leader = elect_one();
        const int dpi = TK / a.page_size, doff = TK % a.page_size;
        const uint64_t pol = l2_policy_evict_first();
        KRing kr;
        bool ok = true;
        while (ok && w.next(a)) {
            for (int rb = 0; ok && rb < a.row_blocks; ++rb) {
                BoxAt box;
                PageWindow pages;
                box.start(a, w, box_log2, lane);
                pages.start(a, w, lane);
                for (int t = w.t0; ok && t < w.t1; ++t) {
                    box.look(a, w, pages, lane);
                    ok = copy_tile<DS>(sm, ring, kr, leader, &mk, box, box_log2, w.item, pol, err);
                    box.step(a, dpi, doff);
                }
            }
        }
        __syncwarp();
    } else if (work && warp == MMA_WARP) {
        if (lane == 0) {
            KRing kr;
            const uint32_t ids = tc_idesc(N, false);
            const uint64_t kd = sw128_desc(ring), qd = sw128_desc(sq);
            uint32_t seg = 0, used[2] = {0, 0};
            bool ok = true;
            while (ok && w.next(a)) {
                const int nt = w.t1 - w.t0;
                for (int rb = 0; ok && rb < a.row_blocks; ++rb, ++seg) {
                    ok = tc_wait(sm, &sm.q_full, seg & 1, err);
                    for (int i = 0; ok && i < nt; ++i) {
                        const int buf = i & 1;
                        if (used[buf] > 0) ok = tc_wait(sm, &sm.p_full[buf], (used[buf] - 1) & 1, err);
                        if (!ok) break;
                        tc_fence_after();
                        ok = issue_scores<DS>(sm, kd, qd, kr, tm_s + buf * N, ids, N, err);
                        if (!ok) break;
                        mma_commit(&sm.s_full[buf]);
                        ++used[buf];
                        if (i + 1 == nt) mma_commit(&sm.q_empty);
                    }
                }
            }
            mma_commit(&sm.done);
            mbar_wait(&sm.done, 0, TC_DRAIN);
        }
        __syncwarp();
    } else if (work && warp < MMA_WARP) {
        constexpr int CH = N < 32 ? N : 16;  // columns at a time
        const int half = warp >> 2, key = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tm_s + lanes + half * N;
        const float c2 = a.scale * LOG2E;
        uint32_t used = 0;
        while (w.next(a)) {
            const int h = w.item, nt = w.t1 - w.t0;
            for (int rb = 0; rb < a.row_blocks; ++rb) {
                const int tok0 = rb * a.tok_block, toks = min(a.tok_block, a.T - tok0);
                const int real = max(min(w.r.nq - tok0, toks), 0) * a.group;
                both_sync();
                if (tid < N) {  // -lse in log2; a row that saw nothing adds nothing
                    float z = NEG_INF;
                    if (tid < real) z = a.lse[attn_row(a, w.b, h, tok0, tid)];
                    sm.neg_m[tid] = z == NEG_INF ? NEG_INF : -z * LOG2E;
                }
                both_sync();
                auto look = [&](int i) {
                    const int s = (w.t0 + i) * TK + key;
                    return i < nt && s < w.r.n ? attn_page(a, w.b, s) : -1;
                };
                auto place = [&](int i, int page) {
                    return (static_cast<int64_t>(page) * a.Hkv + h) * a.page_size + ((w.t0 + i) * TK + key) % a.page_size;
                };
                // pages, and positions where the cache has them, ahead of their use
                int page = look(half), page_next = look(half + 2);
                int pos = a.pos && page >= 0 ? a.pos[place(half, page)] : 0;
                for (int i = half; i < nt; i += 2, ++used) {
                    const int page_after = look(i + 4);
                    const int pos_next = a.pos && page_next >= 0 ? a.pos[place(i + 2, page_next)] : 0;
                    int r0 = 0, r1 = 0;
                    if (page >= 0) {
                        attn_view(a, w.r, a.pos ? pos : (w.t0 + i) * TK + key, r0, r1);
                        r0 = max(r0 - tok0, 0) * a.group;
                        r1 = min((r1 - tok0) * a.group, real);
                    }
                    const bool ok = tc_wait(sm, &sm.s_full[half], used & 1, err);
                    __syncwarp();
                    tc_fence_after();
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                    for (int c = 0; c < N; c += CH) {
                        if (c >= real) break;
                        float x[CH];
                        tmem_ld<CH>(ts + c, reinterpret_cast<uint32_t *>(x));
#pragma unroll
                        for (int j = 0; j < CH; j += 4) {
                            const float4 m = *reinterpret_cast<const float4 *>(sm.neg_m + c + j);
                            const float z[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int r = c + j + k;
                                const float p = ex2(fmaf(x[j + k], c2, z[k]));
                                sum[k] += r >= r0 && r < r1 && z[k] != NEG_INF ? p : 0.f;
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.p_full[half]);
                    if (r0 < r1) atomicAdd(a.weight + place(i, page), ok ? (sum[0] + sum[1]) + (sum[2] + sum[3]) : NAN);
                    page = page_next;
                    page_next = page_after;
                    pos = pos_next;
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tc_aborted(sm)) {  // leave no copy in flight into this CTA's shared memory
        if (tid < UNITS && sm.filled[tid] > 0) mbar_wait(&sm.full[tid], (sm.filled[tid] - 1) & 1, TC_DRAIN);
        if (tid == UNITS && sm.q_filled > 0) mbar_wait(&sm.q_full, (sm.q_filled - 1) & 1, TC_DRAIN);
        __syncthreads();
    }
    if (warp == MMA_WARP) tmem_dealloc(tm_s, COLS);
}

// Launches the kernel of N rows (host).
struct TcLaunch {
    CUtensorMap mk, mv, mq;
    AttnArgs a;
    int box_log2, n;
    int64_t ctas;
    bool weights;  // the second pass
    cudaStream_t stream;
};

template <int N, int DS>
static dflash2_status tc_launch_n(TcLaunch &t) {
    void *fn = t.weights ? reinterpret_cast<void *>(&k_weights_tc<N, DS>) : reinterpret_cast<void *>(&k_attn_tc<N, DS>);
    blocks_per_sm(fn, TC_THREADS, tc_smem(N, DS));  // raises the shared-memory limit, once per device
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(t.ctas), 1, 1);
    cfg.blockDim = dim3(TC_THREADS, 1, 1);
    cfg.dynamicSmemBytes = tc_smem(N, DS);
    cfg.stream = t.stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[5] = {&t.mk, &t.mv, &t.mq, &t.a, &t.box_log2}, *wargs[4] = {&t.mk, &t.mq, &t.a, &t.box_log2};
    if (cudaLaunchKernelExC(&cfg, fn, t.weights ? wargs : args) != cudaSuccess) return DFLASH2_ERR_CUDA;
    return after_launch();
}

template <int DS>
static dflash2_status tc_launch(TcLaunch &t) {
    switch (t.n) {
        case 16: return tc_launch_n<16, DS>(t);
        case 32: return tc_launch_n<32, DS>(t);
        case 48: return tc_launch_n<48, DS>(t);
        case 64: return tc_launch_n<64, DS>(t);
        case 96: return tc_launch_n<96, DS>(t);
        default: return tc_launch_n<128, DS>(t);
    }
}

}  // namespace dfl
