// attn_tc.cu -- dflash2_paged_attn on the tensor cores (bf16 caches, head
// dimensions 64, 128 and 256).
//
// The rows of a block (tokens x query heads that share a cached head) are the
// narrow side of both products, so they go on the N side of the MMA and the
// keys and the head dimension on its 128-wide M side:
//   S^T [128 keys x N rows]  = K [128 x d] . Q^T       per tile of 128 keys
//   O^T [d x N rows]        += V^T [d x 128] . P^T      (d in blocks of 128)
// N is 16 to 128: a single token's few rows cost a sixteenth of the
// tensor work that padding the rows to the M side would.  K and V tiles go
// from the pages to shared memory by TMA exactly as they lie there (V^T is
// the M-major reading of the same rows), and each is read once.
//
// One CTA per SM takes an equal stretch of the call's line of tiles
// (attn.cuh).  Warp 8 copies: 16 KB boxes of 128 keys x 64 dims through a
// ring, in the order in which they are used (K0 K1 V0 K2 V1 ..), page by page.
// Warp 9 issues the MMAs, the next tile's scores before this tile's output
// product.  Warps 0-3 take the first half of the rows and warps 4-7 the
// second, each thread one key: it reads the key's scores from tensor memory,
// takes p = 2^(x - m) with the row's reference m, adds p to its own share of
// the row sums (reduced over the threads only at the end of an item) and
// writes P^T for the second product.  The halves share no row, so they never
// wait for each other within a tile.
// The reference m of a row is the maximum of the item's first tile and moves
// only when a score exceeds it by more than 8 (p <= 256, so nothing
// overflows, and the result is the same up to rounding): then the sums and
// O^T are multiplied by 2^(m - m'), which is rare.
//
// Bound: HBM.  A tile is d * 512 bytes (3000 cycles of an SM's share of
// bandwidth for d = 128); the tensor cores need 16 k-steps of N / 2 cycles
// for it.
//
// Rounding: scores, sums and O^T are fp32; P is rounded to bf16 because the
// MMA takes bf16 beside bf16 values; the sums are of the unrounded p.
//
// Waits are bounded: after a time-out every role stops waiting, the error
// word is set and the CTA's outputs are NaN.
#include "attn.cuh"
#include "tc.cuh"

namespace dfl {

static __device__ unsigned int g_err_attn;

constexpr int TK = 128;            // keys per tile
constexpr int SLOT_BYTES = 16384;  // 128 keys x 64 dims: the swizzle's width
constexpr int TC_THREADS = 320;    // warps 0-3 and 4-7 softmax (half of the rows each), 8 copies, 9 MMA
constexpr int COPY_WARP = 8, MMA_WARP = 9;
constexpr int HOLES = 16;          // tiles whose flags are kept: more than the ring holds
constexpr int MAX_UNITS = 12;
constexpr float M_STEP = 8.f;      // a row's reference moves when a score exceeds it by more (in log2)
constexpr float M_NONE = -1e30f;   // the reference of a row that has seen nothing
constexpr long long TC_WAIT = 4000000000ll;  // ~2 s
constexpr long long TC_DRAIN = 200000000ll;  // ~0.1 s
constexpr int SM_BYTES = 232448;   // shared memory of a CTA

struct TcShared {
    uint64_t full[MAX_UNITS], empty[MAX_UNITS];
    uint64_t s_full[2];   // scores of tile n in buffer n & 1
    uint64_t p_full[2];   // P of tile n written (weights pass: scores read)
    uint64_t pv_done[2];  // output product of tile n complete
    uint64_t q_full, q_empty, done;
    int64_t scratch[TC_THREADS / 32 + 2];
    int64_t row_at[128];  // index of the row in lse (times d: in out)
    alignas(16) float neg_m[128];
    alignas(16) float fac[128];
    float part[4][128];
    float inv[128];
    int hole[HOLES];      // tile n has slots without a page
    alignas(16) unsigned short side[256];
    uint32_t bad[4];
    uint32_t tmem;
    int abort, acc_first, flag;
};

struct TcGeom {
    int ds;        // 64-dim slots of a row
    int us;        // slots of a unit: what a copy, its barriers and a block of V^T cover (at most 128 dims)
    int upt;       // units of a tile's keys, and of its values
    int nunits;    // ring
    int np;        // P buffers
    int box;       // log2 of the keys per copy: the largest power of two that divides the page size, at most 128
};

static __host__ __device__ constexpr int q_bytes(int n, int ds) { return n * ds * 128; }
static __host__ __device__ constexpr int p_bytes(int n) { return n * TK * 2; }

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

__device__ __forceinline__ bool tc_aborted(TcShared &sm) { return *reinterpret_cast<volatile int *>(&sm.abort) != 0; }
// A bounded wait that gives up at once when another role has.
__device__ __forceinline__ bool tc_wait(TcShared &sm, uint64_t *bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!tc_aborted(sm)) {
        if (mbar_try_wait(bar, parity)) return true;
        if (clock64() - t0 > TC_WAIT) {
            atomicOr(&g_err_attn, ERR_WAIT_TIMEOUT);
            *reinterpret_cast<volatile int *>(&sm.abort) = 1;
        }
    }
    return false;
}

// A place in the ring: counts units in the order in which they are filled.
struct RingPos {
    int unit = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void step(int nunits) {
        if (++unit == nunits) {
            unit = 0;
            ++round;
        }
    }
};

// The copying warp's state.  Lane = (64-dim slot of the unit, box of keys);
// page and offset of the lane's box in the tiles to come.
struct Copier {
    int lane, slot, rb;     // slot >= us: the lane copies nothing
    int dst;                // of the box in the unit
    int dpi, doff;          // a tile's step in the page table
    RingPos rp;

    __device__ __forceinline__ void init(const AttnArgs &a, const TcGeom &g, int l) {
        const int nb = TK >> g.box;
        lane = l;
        rb = l & (nb - 1);
        slot = l / nb;
        dst = slot * SLOT_BYTES + ((rb << g.box) * 128);
        dpi = TK / a.page_size;
        doff = TK % a.page_size;
    }
};
struct BoxAt {
    int pi, off, s;  // entry of the request's table, offset in the page, slot number
    int raw;         // the entry read (-1 past the request's slots)

    __device__ __forceinline__ void start(const AttnArgs &a, const AttnWalk &w, const TcGeom &g, const Copier &c) {
        s = w.t0 * TK + (c.rb << g.box);
        pi = s / a.page_size;
        off = s - pi * a.page_size;
        load(a, w);
    }
    __device__ __forceinline__ void load(const AttnArgs &a, const AttnWalk &w) {
        raw = -1;
        if (s < w.r.n) raw = a.table[w.b * a.max_pages + pi];
    }
    // this := the next tile's box after `o`
    __device__ __forceinline__ void after(const BoxAt &o, const AttnArgs &a, const AttnWalk &w, const Copier &c) {
        s = o.s + TK;
        pi = o.pi + c.dpi;
        off = o.off + c.doff;
        if (off >= a.page_size) {
            off -= a.page_size;
            ++pi;
        }
        load(a, w);
    }
};

// Copies a tile's keys or values (upt units).  All lanes of the copying warp.
__device__ __forceinline__ bool copy_tile(TcShared &sm, const TcGeom &g, unsigned char *ring, Copier &c,
                                          const CUtensorMap *map, int page, int off, int h, uint32_t bytes) {
    for (int u = 0; u < g.upt; ++u) {
        bool ok = true;
        if (c.lane == 0) {
            ok = c.rp.round == 0 || tc_wait(sm, &sm.empty[c.rp.unit], (c.rp.round - 1) & 1);
            if (ok) mbar_arrive_expect_tx(&sm.full[c.rp.unit], bytes);
        }
        if (!__all_sync(FULL, ok)) return false;
        if (page >= 0 && c.slot < g.us)
            tma_load_4d(ring + c.rp.unit * g.us * SLOT_BYTES + c.dst, map, (u * g.us + c.slot) * 64, off, h, page,
                        &sm.full[c.rp.unit]);
        c.rp.step(g.nunits);
    }
    return true;
}

// Leave no copy in flight into this CTA's shared memory: the last nunits
// units that were asked for.
__device__ __forceinline__ void drain(TcShared &sm, const TcGeom &g, RingPos rp) {
    for (int i = 0; i < g.nunits; ++i) {
        if (rp.unit == 0) {
            if (rp.round == 0) return;
            rp.unit = g.nunits;
            --rp.round;
        }
        --rp.unit;
        mbar_wait(&sm.full[rp.unit], rp.round & 1, TC_DRAIN);
    }
}

// One tile's score product from the ring's next units.
__device__ __forceinline__ bool issue_scores(TcShared &sm, const TcGeom &g, unsigned char *ring,
                                             const unsigned char *sq, RingPos &rp, uint32_t d_tmem, int N) {
    const uint32_t idesc = tc_idesc(N, false);
    for (int u = 0; u < g.upt; ++u) {
        if (!tc_wait(sm, &sm.full[rp.unit], rp.round & 1)) return false;
        tc_fence_after();
        for (int s = 0; s < g.us; ++s) {
            const uint64_t ad = sw128_desc(ring + (rp.unit * g.us + s) * SLOT_BYTES);
            const uint64_t bd = sw128_desc(sq + (u * g.us + s) * N * 128);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_bf16(d_tmem, ad + 2 * k, bd + 2 * k, idesc, u > 0 || s > 0 || k > 0);
        }
        mma_commit(&sm.empty[rp.unit]);
        rp.step(g.nunits);
    }
    return true;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
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

// Set-up that both kernels share; returns the ring's base.
__device__ __forceinline__ unsigned char *tc_setup(TcShared &sm, unsigned char *ring, const TcGeom &g, int N,
                                                   int cols) {
    const int tid = threadIdx.x;
    if (tid == 0) {
        for (int i = 0; i < g.nunits; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_full[i], 8);
            mbar_init(&sm.pv_done[i], 1);
        }
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_empty, 1);
        mbar_init(&sm.done, 1);
        sm.abort = 0;
        sm.acc_first = 0;
        fence_barrier_init();
    }
    if (tid / 32 == MMA_WARP) tmem_alloc(&sm.tmem, cols);
    // rows that the copies of Q do not reach stay zero
    uint4 *q = reinterpret_cast<uint4 *>(ring + g.nunits * g.us * SLOT_BYTES);
    for (int i = tid; i < q_bytes(N, g.ds) / 16; i += TC_THREADS) q[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    return ring;
}

template <int N>
__global__ void __launch_bounds__(TC_THREADS, 1) k_attn_tc(const __grid_constant__ CUtensorMap mk,
                                                           const __grid_constant__ CUtensorMap mv,
                                                           const __grid_constant__ CUtensorMap mq, AttnArgs a,
                                                           TcGeom g) {
    extern __shared__ unsigned char raw[];
    __shared__ TcShared sm;
    unsigned char *ring =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *sq = ring + g.nunits * g.us * SLOT_BYTES, *sp = sq + q_bytes(N, g.ds);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int mb = g.ds > 2 ? 2 : 1;  // 128-dim blocks of O^T
    const int cols = N * (2 + mb) <= 64 ? 64 : N * (2 + mb) <= 128 ? 128 : N * (2 + mb) <= 256 ? 256 : 512;
    tc_setup(sm, ring, g, N, cols);
    const uint32_t tm_s = sm.tmem, tm_o = tm_s + 2 * N;
    pdl_wait();
    const AttnPlan plan = attn_plan<TC_THREADS>(a, sm.scratch);
    const bool work = plan.begin < plan.end;
    AttnWalk w;
    if (work) w.start(a, plan);

    if (work && warp == COPY_WARP) {
        // ------------------------------------------------------- copies --
        Copier c;
        c.init(a, g, lane);
        uint32_t seg = 0, n = 0;
        bool ok = true;
        while (ok && w.next(a)) {
            const int h = w.item / a.row_blocks, tok0 = (w.item % a.row_blocks) * a.tok_block;
            const int nt = w.t1 - w.t0;
            BoxAt now, next, after;  // this tile's box, the next one's, the one after: table entries ahead of their use
            now.start(a, w, g, c);
            next.after(now, a, w, c);
            if (lane == 0) {
                ok = seg == 0 || tc_wait(sm, &sm.q_empty, (seg - 1) & 1);
                if (ok) {
                    mbar_arrive_expect_tx(&sm.q_full, a.tok_block * a.group * 128 * g.ds);
                    for (int s = 0; s < g.ds; ++s)
                        tma_load_4d(sq + s * N * 128, &mq, s * 64, h * a.group, tok0, static_cast<int>(w.b),
                                    &sm.q_full);
                }
            }
            ok = __all_sync(FULL, ok);
            if (!ok) break;
            ++seg;
            // a tile's page, its bytes, and whether slots in use have no page (for the softmax warps)
            auto page_of = [&](const BoxAt &b, uint32_t tile, uint32_t &bytes) {
                const int page = static_cast<unsigned>(b.raw) < static_cast<unsigned long long>(a.num_pages) ? b.raw : -1;
                const unsigned there = __ballot_sync(FULL, page >= 0 && c.slot == 0);
                const bool hole = __any_sync(FULL, page < 0 && b.s < w.r.n);
                if (lane == 0) sm.hole[tile % HOLES] = hole;
                bytes = (__popc(there) << g.box) * 128 * g.us;
                return page;
            };
            uint32_t bytes, bytes_next = 0;
            int page = page_of(now, n, bytes), page_next = -1;
            ok = copy_tile(sm, g, ring, c, &mk, page, now.off, h, bytes);
            for (int i = 0; ok && i < nt; ++i, ++n) {
                after.after(next, a, w, c);
                if (i + 1 < nt) {
                    page_next = page_of(next, n + 1, bytes_next);
                    ok = copy_tile(sm, g, ring, c, &mk, page_next, next.off, h, bytes_next);
                }
                ok = ok && copy_tile(sm, g, ring, c, &mv, page, now.off, h, bytes);
                now = next;
                next = after;
                page = page_next;
                bytes = bytes_next;
            }
        }
        if (lane == 0) {
            drain(sm, g, c.rp);
            if (seg > 0) mbar_wait(&sm.q_full, (seg - 1) & 1, TC_DRAIN);
        }
        __syncwarp();
    } else if (work && warp == MMA_WARP) {
        // ---------------------------------------------------------- MMA --
        if (lane == 0) {
            RingPos rp;
            const uint32_t idesc = tc_idesc(N, true);
            uint32_t seg = 0, n = 0;
            bool ok = true;
            while (ok && w.next(a)) {
                const int nt = w.t1 - w.t0;
                ok = tc_wait(sm, &sm.q_full, seg & 1);
                ++seg;
                ok = ok && issue_scores(sm, g, ring, sq, rp, tm_s + (n & 1) * N, N);
                if (!ok) break;
                mma_commit(&sm.s_full[n & 1]);
                if (nt == 1) mma_commit(&sm.q_empty);
                for (int i = 0; ok && i < nt; ++i, ++n) {
                    if (i + 1 < nt) {
                        ok = issue_scores(sm, g, ring, sq, rp, tm_s + ((n + 1) & 1) * N, N);
                        if (!ok) break;
                        mma_commit(&sm.s_full[(n + 1) & 1]);
                        if (i + 2 == nt) mma_commit(&sm.q_empty);
                    }
                    ok = tc_wait(sm, &sm.p_full[n & 1], (n >> 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t bd = p_desc(sp + (n % g.np) * p_bytes(N));
                    const bool acc = i > 0 || *reinterpret_cast<volatile int *>(&sm.acc_first) != 0;
                    for (int m = 0; m < mb; ++m) {
                        ok = tc_wait(sm, &sm.full[rp.unit], rp.round & 1);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t ad = v_desc(ring + rp.unit * g.us * SLOT_BYTES, g.us > 1 ? SLOT_BYTES : 0);
#pragma unroll
                        for (int k = 0; k < TK / 16; ++k)  // 16 keys: 2048 bytes of V, 256 of P
                            mma_bf16(tm_o + m * N, ad + 128 * k, bd + 16 * k, idesc, acc || k > 0);
                        mma_commit(&sm.empty[rp.unit]);
                        rp.step(g.nunits);
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
        int seq = 0;     // units before this item's first
        while (w.next(a)) {
            const int h = w.item / a.row_blocks, tok0 = (w.item % a.row_blocks) * a.tok_block;
            const int toks = min(a.tok_block, a.T - tok0), rows = toks * a.group;
            const int live = max(min(w.r.nq - tok0, toks), 0), real = live * a.group;
            const int nt = w.t1 - w.t0;
            float l[NR];
#pragma unroll
            for (int i = 0; i < NR; ++i) l[i] = 0.f;
            if (key < NR) {
                neg_m[key] = -M_NONE;
                if (row0 + key < rows) sm.row_at[row0 + key] = attn_row(a, w.b, h, tok0, row0 + key);
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
            int page_now = slot_page(w.t0), page_next = slot_page(w.t0 + 1);
            int pos_now = slot_pos(w.t0, page_now);
            for (int i = 0; i < nt; ++i, ++n) {
                const int t = w.t0 + i, ks = t * TK;
                const int page_after = slot_page(t + 2), pos_next = slot_pos(t + 1, page_next);
                tc_wait(sm, &sm.s_full[n & 1], (n >> 1) & 1);
                __syncwarp();
                tc_fence_after();
                const uint32_t ts = tm_s + lanes + (n & 1) * N + row0;
                float x[NR];
                tmem_ld<NR>(ts, reinterpret_cast<uint32_t *>(x));
                // which rows see this thread's key; nothing to look at if all rows see the whole tile
                int r0 = 0, r1 = NR;
                bool none = false, poison = false;
                bool masked = a.pos || ks + TK > w.r.n || (a.causal && ks + TK - 1 > w.r.q0 + tok0) ||
                              (a.window > 0 && ks <= w.r.q0 + tok0 + live - 1 - a.window) ||
                              *reinterpret_cast<volatile int *>(&sm.hole[n % HOLES]);
                if (masked) {
                    int lo = 0, hi = 0;
                    if (a.pos) {
                        if (page_now >= 0) attn_view(a, w.r, pos_now, lo, hi);
                    } else if (ks + key < w.r.n && attn_page(a, w.b, ks + key) >= 0) {
                        attn_view(a, w.r, ks + key, lo, hi);
                    }
                    lo = max(lo - tok0, 0) * a.group;
                    hi = min((hi - tok0) * a.group, real);
                    none = lo >= hi;
                    const bool part = !none && (lo > 0 || hi < real);
                    r0 = lo - row0;
                    r1 = none ? r0 : hi - row0;
                    masked = __any_sync(FULL, none || part);
                    // Values of a key that no row sees are set to zero: p = 0 times NaN would be NaN.  Of a key that
                    // only some rows see, values that are not finite are taken out and added by hand.
                    if ((none && half == 0) || part) {
                        const int vseq = seq + (i < nt - 1 ? 2 * i + 2 : 2 * nt - 1) * g.upt;
                        for (int e = 0; e < g.ds; ++e) {
                            const int q = vseq + e / g.us;
                            tc_wait(sm, &sm.full[q % g.nunits], (q / g.nunits) & 1);
                            uint4 *row = reinterpret_cast<uint4 *>(
                                ring + (q % g.nunits * g.us + e % g.us) * SLOT_BYTES + key * 128);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                if (none) {
                                    row[j] = make_uint4(0, 0, 0, 0);
                                } else {
                                    const uint4 v = row[j];
                                    poison = poison || bad_bf16(v.x) || bad_bf16(v.x >> 16) || bad_bf16(v.y) ||
                                             bad_bf16(v.y >> 16) || bad_bf16(v.z) || bad_bf16(v.z >> 16) ||
                                             bad_bf16(v.w) || bad_bf16(v.w >> 16);
                                }
                            }
                        }
                    }
                    __syncwarp();
                }
                // x = s c2 - m, in place
                auto exponents = [&]() {
#pragma unroll
                    for (int j = 0; j < NR; j += 4) {
                        const float4 m = *reinterpret_cast<const float4 *>(neg_m + j);
                        x[j] = fmaf(x[j], c2, m.x);
                        x[j + 1] = fmaf(x[j + 1], c2, m.y);
                        x[j + 2] = fmaf(x[j + 2], c2, m.z);
                        x[j + 3] = fmaf(x[j + 3], c2, m.w);
                    }
                    if (masked) {
#pragma unroll
                        for (int j = 0; j < NR; ++j)
                            if (j < r0 || j >= r1) x[j] = NEG_INF;
                    }
                };
                bool slow = true;
                if (i > 0) {
                    exponents();
                    float xm = NEG_INF;
#pragma unroll
                    for (int j = 0; j < NR; ++j) xm = fmaxf(xm, x[j]);
                    slow = soft_any(half, xm > M_STEP || poison);
                }
                bool any_poison = false;
                if (slow) {
                    // the rows' maxima over the tile, new references, and what has been summed scaled to them
                    if (i > 0) tmem_ld<NR>(ts, reinterpret_cast<uint32_t *>(x));
#pragma unroll
                    for (int c = 0; c < NR; c += 32) {
                        float mine = NEG_INF;
#pragma unroll
                        for (int j = c; j < NR && j < c + 32; ++j) {
                            const float y = warp_max_f(masked && (j < r0 || j >= r1) ? NEG_INF : x[j] * c2);
                            if (lane == j - c) mine = y;
                        }
                        if (c + lane < NR) sm.part[warp & 3][row0 + c + lane] = mine;
                    }
                    soft_sync(half);
                    if (key < NR) {
                        const int r = row0 + key;
                        const float mo = -neg_m[key];
                        float mn = fmaxf(fmaxf(sm.part[0][r], sm.part[1][r]), fmaxf(sm.part[2][r], sm.part[3][r]));
                        mn = fmaxf(mn, mo);
                        fac[key] = ex2(mo - mn);
                        neg_m[key] = -mn;
                    }
                    any_poison = soft_any(half, poison);
                    exponents();
                    if (i > 0) {
#pragma unroll
                        for (int j = 0; j < NR; ++j) l[j] *= fac[j];
                        tc_wait(sm, &sm.pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1);
                        __syncwarp();
                        tc_fence_after();
                        for (int m = 0; m < mb; ++m)
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
                if (n >= static_cast<uint32_t>(g.np)) {
                    const uint32_t k = n - g.np;
                    tc_wait(sm, &sm.pv_done[k & 1], (k >> 1) & 1);
                    __syncwarp();
                }
                unsigned char *pb = sp + (n % g.np) * p_bytes(N);
#pragma unroll
                for (int j = 0; j < NR; j += 8)
                    *reinterpret_cast<uint4 *>(pb + ((row0 + j) / 8) * (TK * 16) + key * 16) =
                        make_uint4(pk[j / 2], pk[j / 2 + 1], pk[j / 2 + 2], pk[j / 2 + 3]);
                if (any_poison) {
                    // Keys that some rows see and some do not, with values that are not finite: their products with p
                    // go straight into O^T.  Both groups find the same keys and go through them together.
                    const int vseq = seq + (i < nt - 1 ? 2 * i + 2 : 2 * nt - 1) * g.upt;
                    const unsigned mine = __ballot_sync(FULL, poison);
                    if (half == 0 && lane == 0) sm.bad[warp] = mine;
                    if (i == 0) {
                        float z[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) z[j] = 0.f;
                        for (int m = 0; m < mb; ++m)
                            for (int j = 0; j < NR; j += 8) tmem_st8(tm_o + lanes + m * N + row0 + j, z);
                        tmem_wait_st();
                        if (tid == 0) sm.acc_first = 1;
                    }
                    both_sync();
                    for (int k = 0; k < TK; ++k) {
                        if (!(sm.bad[k >> 5] >> (k & 31) & 1)) continue;
                        if (tid == k) {
                            for (int e = 0; e < g.ds * 64; ++e) {
                                const int q = vseq + e / 64 / g.us, chunk = (e % 64) / 8;
                                unsigned short *v = reinterpret_cast<unsigned short *>(
                                    ring + (q % g.nunits * g.us + e / 64 % g.us) * SLOT_BYTES + k * 128 +
                                    ((chunk ^ (k & 7)) * 16) + (e % 8) * 2);
                                const bool b = bad_bf16(*v);
                                sm.side[e] = b ? *v : 0;
                                if (b) *v = 0;
                            }
                        }
                        both_sync();
                        for (int m = 0; m < mb; ++m) {
                            const int e = g.ds > 1 ? m * 128 + key : key & 63;
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
            seq += 2 * nt * g.upt;
            // the rows' sums over all keys
#pragma unroll
            for (int j = 0; j < NR; j += 8) {
                const float v = lane_sums8(l + j, lane);
                if ((lane & 3) == 0) sm.part[warp & 3][row0 + j + lane / 4] = v;
            }
            soft_sync(half);
            float *part = w.whole ? nullptr : attn_part(a, blockIdx.x, w.starts);
            const int mine = min(rows - row0, NR);  // rows of this group (none or negative: the group has none)
            if (key < mine) {
                const int r = row0 + key;
                float L = sm.part[0][r] + sm.part[1][r] + sm.part[2][r] + sm.part[3][r];
                const float m = -neg_m[key];
                if (tc_aborted(sm)) L = NAN;
                else if (r >= real) L = 0.f;
                sm.inv[r] = L == 0.f ? 0.f : (w.whole ? 1.0f / L : 1.f);
                if (w.whole) {
                    if (a.lse) a.lse[sm.row_at[r]] = L == 0.f ? NEG_INF : (m + log2f(L)) * 0.6931471805599453f;
                } else {
                    part[a.rows_cap * a.d + r] = m;
                    part[a.rows_cap * (a.d + 1) + r] = L;
                }
            }
            tc_wait(sm, &sm.pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1);
            soft_sync(half);
            tc_fence_after();
            if (g.ds > 1 || (warp & 3) < 2) {
                for (int m = 0; m < mb; ++m) {
                    const int e = m * 128 + key;
                    for (int j0 = 0; j0 < mine; j0 += 8) {
                        uint32_t o[8];
                        tmem_ld<8>(tm_o + lanes + m * N + row0 + j0, o);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            if (j0 + j >= mine) break;
                            const int r = row0 + j0 + j;
                            const float f = sm.inv[r];
                            const float v = f == 0.f ? 0.f : __uint_as_float(o[j]) * f;
                            if (w.whole)
                                attn_store(a, sm.row_at[r] * a.d + e, v, static_cast<unsigned short *>(nullptr));
                            else
                                part[static_cast<int64_t>(r) * a.d + e] = v;
                        }
                    }
                }
            }
            tc_fence_before();
            both_sync();
            if (!w.whole) {
                attn_join<unsigned short>(a, w, rows, h, tok0, 256, tid, &sm.flag, both_sync);
                both_sync();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == MMA_WARP) tmem_dealloc(tm_s, cols);
}

unsigned int read_error_attn(bool clear) {
    unsigned int v = 0;
    cudaMemcpyFromSymbol(&v, g_err_attn, sizeof v);
    if (clear) {
        const unsigned int z = 0;
        cudaMemcpyToSymbol(g_err_attn, &z, sizeof z);
    }
    return v;
}

static bool make_map_4d(CUtensorMap *m, const void *ptr, const cuuint64_t (&dims)[4], const cuuint64_t (&strides)[3],
                        cuuint32_t box1, cuuint32_t box2) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint32_t box[4] = {64u, box1, box2, 1u}, estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether the tensor-core kernels take a bf16 call: copies of at least 8 keys
// (one swizzle pattern) and strides that a tensor map can hold.
bool attn_tc_takes(const AttnArgs &a) {
    const int64_t lim = int64_t(1) << 39;
    return (a.d == 64 || a.d == 128 || a.d == 256) && a.page_size % 8 == 0 && a.B < (int64_t(1) << 31) &&
           (a.Hkv == 1 || (a.head_stride > 0 && a.head_stride < lim)) &&
           (a.num_pages == 1 || (a.page_stride > 0 && a.page_stride < lim)) && a.slot_stride < lim &&
           static_cast<int64_t>(a.T) * a.Hq * a.d < lim;
}

dflash2_status attn_tc_launch(AttnArgs a, cudaStream_t s) {
    a.tile = TK;
    const int most = TK / a.group;                            // tokens that fit a block
    const int blocks = (a.T + most - 1) / most;
    a.tok_block = (a.T + blocks - 1) / blocks;                // blocks of like size
    a.row_blocks = (a.T + a.tok_block - 1) / a.tok_block;
    a.rows_cap = a.tok_block * a.group;
    a.items = a.Hkv * a.row_blocks;
    const int N = a.rows_cap <= 16   ? 16
                  : a.rows_cap <= 32 ? 32
                  : a.rows_cap <= 48 ? 48
                  : a.rows_cap <= 64 ? 64
                  : a.rows_cap <= 96 ? 96
                                     : 128;
    TcGeom g;
    g.ds = a.d / 64;
    g.us = g.ds > 1 ? 2 : 1;
    g.upt = g.ds / g.us;
    g.np = N > 64 ? 1 : 2;
    g.box = 3;
    while (g.box < 7 && a.page_size % (2 << g.box) == 0) ++g.box;
    const int rest = SM_BYTES - 1024 - static_cast<int>(sizeof(TcShared)) - 256 - q_bytes(N, g.ds) - g.np * p_bytes(N);
    g.nunits = rest / (g.us * SLOT_BYTES);
    if (g.nunits > MAX_UNITS) g.nunits = MAX_UNITS;
    const size_t smem =
        1024 + static_cast<size_t>(g.nunits) * g.us * SLOT_BYTES + q_bytes(N, g.ds) + g.np * p_bytes(N);

    CUtensorMap mk, mv, mq;
    const cuuint64_t cd[4] = {static_cast<cuuint64_t>(a.d), static_cast<cuuint64_t>(a.page_size),
                              static_cast<cuuint64_t>(a.Hkv), static_cast<cuuint64_t>(a.num_pages)};
    // a dimension of one element has no stride of its own
    const int64_t hs = a.Hkv == 1 ? a.slot_stride * a.page_size : a.head_stride;
    const int64_t ps = a.num_pages == 1 ? hs * a.Hkv : a.page_stride;
    const cuuint64_t cs[3] = {static_cast<cuuint64_t>(a.slot_stride) * 2, static_cast<cuuint64_t>(hs) * 2,
                              static_cast<cuuint64_t>(ps) * 2};
    const cuuint64_t qd[4] = {static_cast<cuuint64_t>(a.d), static_cast<cuuint64_t>(a.Hq),
                              static_cast<cuuint64_t>(a.T), static_cast<cuuint64_t>(a.B)};
    const cuuint64_t qs[3] = {static_cast<cuuint64_t>(a.d) * 2, static_cast<cuuint64_t>(a.Hq) * a.d * 2,
                              static_cast<cuuint64_t>(a.T) * a.Hq * a.d * 2};
    if (!make_map_4d(&mk, a.k, cd, cs, 1u << g.box, 1) || !make_map_4d(&mv, a.v, cd, cs, 1u << g.box, 1) ||
        !make_map_4d(&mq, a.q, qd, qs, a.group, a.tok_block))
        return DFLASH2_ERR_CUDA;

    const double tiles = static_cast<double>(a.B) * a.items *
                         ((static_cast<int64_t>(a.max_pages) * a.page_size + TK - 1) / TK);
    const int ctas = tiles < sm_count() ? static_cast<int>(tiles) : sm_count();
    void *fn = N == 16   ? reinterpret_cast<void *>(&k_attn_tc<16>)
               : N == 32 ? reinterpret_cast<void *>(&k_attn_tc<32>)
               : N == 48 ? reinterpret_cast<void *>(&k_attn_tc<48>)
               : N == 64 ? reinterpret_cast<void *>(&k_attn_tc<64>)
               : N == 96 ? reinterpret_cast<void *>(&k_attn_tc<96>)
                         : reinterpret_cast<void *>(&k_attn_tc<128>);
    blocks_per_sm(fn, TC_THREADS, SM_BYTES - sizeof(TcShared) - 256);  // raises the shared-memory limit, once per device
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(TC_THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[5] = {&mk, &mv, &mq, &a, &g};
    if (cudaLaunchKernelExC(&cfg, fn, args) != cudaSuccess) return DFLASH2_ERR_CUDA;
    return after_launch();
}

}  // namespace dfl
