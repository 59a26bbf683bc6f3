// attn_tc.cu -- dflash2_paged_attn on the tensor cores (bf16 caches, head
// dimensions 64, 128 and 256).
//
// The rows of a block (tokens x query heads that share a cached head) are the
// narrow side of both products, so they go on the N side of the MMA and the
// keys and the head dimension on its 128-wide M side:
//   S^T [128 keys x N rows]  = K [128 x d] . Q^T       per tile of 128 keys
//   O^T [d x N rows]        += V^T [d x 128] . P^T      (d in blocks of 128)
// N is 16, 32, 64 or 128: a single token's few rows cost a sixteenth of the
// tensor work that padding the rows to the M side would.  K and V tiles go
// from the pages to shared memory by TMA exactly as they lie there (V^T is
// the M-major reading of the same rows), and each is read once.
//
// One CTA per SM takes an equal stretch of the call's line of tiles
// (attn.cuh).  Warp 4 copies: 16 KB boxes of 128 keys x 64 dims through a
// ring, in the order in which they are used (K0 K1 V0 K2 V1 ..), page by page.
// Warp 5 issues the MMAs, the next tile's scores before this tile's output
// product.  Warps 0-3 hold one key per thread: they read the key's scores of
// all rows from tensor memory, take p = 2^(x - m) with the row's reference m,
// add p to the thread's own share of the row sums (reduced over the threads
// only at the end of an item) and write P^T for the second product.
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
constexpr int SLOT_BYTES = 16384;  // 128 keys x 64 dims
constexpr int TC_THREADS = 192;    // warps 0-3 softmax, 4 copies, 5 MMA
constexpr int MAX_SLOTS = 12;
constexpr float M_STEP = 8.f;      // a row's reference moves when a score exceeds it by more (in log2)
constexpr float M_NONE = -1e30f;   // the reference of a row that has seen nothing
constexpr long long TC_WAIT = 4000000000ll;  // ~2 s
constexpr long long TC_DRAIN = 200000000ll;  // ~0.1 s
constexpr int SM_BYTES = 232448;   // shared memory of a CTA

struct TcShared {
    uint64_t full[MAX_SLOTS], empty[MAX_SLOTS];
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
    alignas(16) unsigned short side[256];
    uint32_t bad[4];
    uint32_t tmem;
    int abort, acc_first, flag;
};

struct TcGeom {
    int ds;       // 64-dim slots of a row
    int nslots;   // ring
    int np;       // P buffers
    int box;      // keys per copy: the largest power of two that divides the page size, at most 128
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

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16};" ::"r"(taddr),
        "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]),
        "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
template <int C>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t *r) {
#pragma unroll
    for (int i = 0; i < C; i += 16) tmem_ld16_nowait(taddr + i, r + i);
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

// Barriers of the softmax warps (each warp reconverges first).
__device__ __forceinline__ void soft_sync() {
    __syncwarp();
    asm volatile("bar.sync 1, 128;" ::: "memory");
}
__device__ __forceinline__ bool soft_any(bool p) {
    __syncwarp();
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(p ? 1u : 0u)
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

// A place in the ring: counts slots in the order in which they are filled.
struct RingPos {
    int slot = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void step(int nslots) {
        if (++slot == nslots) {
            slot = 0;
            ++round;
        }
    }
};

// Copies the slots of one tile's keys or values; `page` is this lane's page of
// the tile (or -1: nothing there).  All lanes of the copying warp call it.
__device__ __forceinline__ bool copy_tile(TcShared &sm, const TcGeom &g, unsigned char *ring, RingPos &rp,
                                          const CUtensorMap *map, int lane, int page, int off, int h) {
    const int nb = TK / g.box, rb = lane & (nb - 1), first = lane / nb, per = 32 / nb;
    // every box has the same number of lanes on it
    const uint32_t bytes = static_cast<uint32_t>(__popc(__ballot_sync(FULL, page >= 0)) / per * g.box * 128);
    for (int s = 0; s < g.ds; ++s) {
        const bool ok = rp.round == 0 || tc_wait(sm, &sm.empty[rp.slot], (rp.round - 1) & 1);
        if (!__all_sync(FULL, ok)) return false;
        if (lane == 0) mbar_arrive_expect_tx(&sm.full[rp.slot], bytes);
        __syncwarp();
        if (page >= 0 && s % per == first)
            tma_load_4d(ring + rp.slot * SLOT_BYTES + rb * g.box * 128, map, s * 64, off, h, page, &sm.full[rp.slot]);
        rp.step(g.nslots);
    }
    return true;
}

// This lane's page of tile t and the key's offset in it.
__device__ __forceinline__ int lane_page(const AttnArgs &a, const AttnWalk &w, const TcGeom &g, int t, int lane,
                                         int &off) {
    const int s = t * TK + (lane & (TK / g.box - 1)) * g.box;
    off = s % a.page_size;
    return s < w.r.n ? attn_page(a, w.b, s) : -1;
}

// Leave no copy in flight into this CTA's shared memory: the last nslots
// slots that were asked for.
__device__ __forceinline__ void drain(TcShared &sm, const TcGeom &g, RingPos rp) {
    for (int i = 0; i < g.nslots; ++i) {
        if (rp.slot == 0) {
            if (rp.round == 0) return;
            rp.slot = g.nslots;
            --rp.round;
        }
        --rp.slot;
        mbar_wait(&sm.full[rp.slot], rp.round & 1, TC_DRAIN);
    }
}

// One tile's score product from the ring's next slots into S buffer n & 1.
__device__ __forceinline__ bool issue_scores(TcShared &sm, const TcGeom &g, unsigned char *ring,
                                             const unsigned char *sq, RingPos &rp, uint32_t d_tmem, int N) {
    const uint32_t idesc = tc_idesc(N, false);
    for (int s = 0; s < g.ds; ++s) {
        if (!tc_wait(sm, &sm.full[rp.slot], rp.round & 1)) return false;
        tc_fence_after();
        const uint64_t ad = sw128_desc(ring + rp.slot * SLOT_BYTES), bd = sw128_desc(sq + s * N * 128);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_bf16(d_tmem, ad + 2 * k, bd + 2 * k, idesc, s > 0 || k > 0);
        mma_commit(&sm.empty[rp.slot]);
        rp.step(g.nslots);
    }
    return true;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ bool bad_bf16(uint32_t h) { return (h & 0x7f80u) == 0x7f80u; }

// Sum of v[r] over the warp's lanes; lane l ends with rows l * N / 32 .. (N < 32: row l * N / 32) in v[0 ..].
template <int N>
__device__ __forceinline__ void lane_sums(float (&v)[N], int lane) {
    int cnt = N;
#pragma unroll
    for (int step = 16; step >= 1; step >>= 1) {
        if (cnt > 1) {
            const int half = cnt / 2;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                if (i >= half) break;
                const float send = (lane & step) ? v[i] : v[i + half];
                const float keep = (lane & step) ? v[i + half] : v[i];
                v[i] = keep + __shfl_xor_sync(FULL, send, step);
            }
            cnt = half;
        } else {
            v[0] += __shfl_xor_sync(FULL, v[0], step);
        }
    }
}

// Set-up that both kernels share; returns the ring's base.
__device__ __forceinline__ unsigned char *tc_setup(TcShared &sm, unsigned char *ring, const TcGeom &g, int N,
                                                   int cols) {
    const int tid = threadIdx.x;
    if (tid == 0) {
        for (int i = 0; i < g.nslots; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_full[i], 4);
            mbar_init(&sm.pv_done[i], 1);
        }
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_empty, 1);
        mbar_init(&sm.done, 1);
        sm.abort = 0;
        sm.acc_first = 0;
        fence_barrier_init();
    }
    if (tid / 32 == 5) tmem_alloc(&sm.tmem, cols);
    // rows that the copies of Q do not reach stay zero
    uint4 *q = reinterpret_cast<uint4 *>(ring + g.nslots * SLOT_BYTES);
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
    unsigned char *sq = ring + g.nslots * SLOT_BYTES, *sp = sq + q_bytes(N, g.ds);
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

    if (work && warp == 4) {
        // ------------------------------------------------------- copies --
        RingPos rp;
        uint32_t seg = 0;
        bool ok = true;
        while (ok && w.next(a)) {
            const int h = w.item / a.row_blocks, tok0 = (w.item % a.row_blocks) * a.tok_block;
            const int nt = w.t1 - w.t0;
            int off[2], page[2];  // by tile parity: this tile's and the next one's
            page[0] = lane_page(a, w, g, w.t0, lane, off[0]);
            page[1] = nt > 1 ? lane_page(a, w, g, w.t0 + 1, lane, off[1]) : -1;
            ok = seg == 0 || tc_wait(sm, &sm.q_empty, (seg - 1) & 1);
            ok = __all_sync(FULL, ok);
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&sm.q_full, a.tok_block * a.group * 128 * g.ds);
                for (int s = 0; s < g.ds; ++s)
                    tma_load_4d(sq + s * N * 128, &mq, s * 64, h * a.group, tok0, static_cast<int>(w.b), &sm.q_full);
            }
            __syncwarp();
            ++seg;
            ok = copy_tile(sm, g, ring, rp, &mk, lane, page[0], off[0], h);
            for (int i = 0; ok && i < nt; ++i) {
                const int c = i & 1;
                int pn = -1, on = 0;
                if (i + 2 < nt) pn = lane_page(a, w, g, w.t0 + i + 2, lane, on);
                if (i + 1 < nt) ok = copy_tile(sm, g, ring, rp, &mk, lane, page[c ^ 1], off[c ^ 1], h);
                ok = ok && copy_tile(sm, g, ring, rp, &mv, lane, page[c], off[c], h);
                page[c] = pn;
                off[c] = on;
            }
        }
        if (lane == 0) {
            drain(sm, g, rp);
            if (seg > 0) mbar_wait(&sm.q_full, (seg - 1) & 1, TC_DRAIN);
        }
        __syncwarp();
    } else if (work && warp == 5) {
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
                    for (int m = 0; ok && m < mb; ++m) {
                        const int s0 = rp.slot;
                        for (int s = 0; ok && s < (g.ds > 1 ? 2 : 1); ++s) {
                            ok = tc_wait(sm, &sm.full[rp.slot], rp.round & 1);
                            rp.step(g.nslots);
                        }
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t ad = v_desc(ring + s0 * SLOT_BYTES, g.ds > 1 ? SLOT_BYTES : 0);
#pragma unroll
                        for (int k = 0; k < TK / 16; ++k)  // 16 keys: 2048 bytes of V, 256 of P
                            mma_bf16(tm_o + m * N, ad + 128 * k, bd + 16 * k, idesc, acc || k > 0);
                        mma_commit(&sm.empty[s0]);
                        if (g.ds > 1) mma_commit(&sm.empty[s0 + 1]);
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
        constexpr int CH = N < 32 ? N : 32, NCH = N / CH;
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
        const float c2 = a.scale * LOG2E;
        uint32_t n = 0;            // tiles so far
        int seq = 0;               // slots before this item's first
        while (w.next(a)) {
            const int h = w.item / a.row_blocks, tok0 = (w.item % a.row_blocks) * a.tok_block;
            const int toks = min(a.tok_block, a.T - tok0), rows = toks * a.group;
            const int real = max(min(w.r.nq - tok0, toks), 0) * a.group;
            const int nt = w.t1 - w.t0;
            float l[N];
#pragma unroll
            for (int i = 0; i < N; ++i) l[i] = 0.f;
            if (tid < N) {
                sm.neg_m[tid] = -M_NONE;
                if (tid < rows) sm.row_at[tid] = attn_row(a, w.b, h, tok0, tid);
            }
            if (tid == 0) sm.acc_first = 0;
            soft_sync();
            for (int i = 0; i < nt; ++i, ++n) {
                int lo, hi, page;
                attn_view_slot(a, w.r, w.b, h, (w.t0 + i) * TK + tid, lo, hi, page);
                const int r0 = max(lo - tok0, 0) * a.group, r1 = min((hi - tok0) * a.group, real);
                const bool none = r0 >= r1, part = !none && (r0 > 0 || r1 < real);
                const bool masked = __any_sync(FULL, none || part);
                // Values of a key that no row sees are set to zero: p = 0 times NaN would be NaN.  Of a key that
                // only some rows see, values that are not finite are taken out and added by hand.
                bool poison = false;
                const int vseq = seq + (i < nt - 1 ? 2 * i + 2 : 2 * nt - 1) * g.ds;
                if (none || part) {
                    for (int s = 0; s < g.ds; ++s) {
                        const int q = vseq + s;
                        tc_wait(sm, &sm.full[q % g.nslots], (q / g.nslots) & 1);
                        uint4 *row = reinterpret_cast<uint4 *>(ring + (q % g.nslots) * SLOT_BYTES + tid * 128);
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
                tc_wait(sm, &sm.s_full[n & 1], (n >> 1) & 1);
                __syncwarp();
                tc_fence_after();
                const uint32_t ts = tm_s + lanes + (n & 1) * N;
                uint32_t s[CH];
                if (NCH == 1) tmem_ld<CH>(ts, s);
                bool slow = true;
                if (i > 0) {
                    float xm = NEG_INF;
#pragma unroll
                    for (int c = 0; c < NCH; ++c) {
                        if (NCH > 1) tmem_ld<CH>(ts + c * CH, s);
#pragma unroll
                        for (int j = 0; j < CH; j += 4) {
                            const float4 m4 = *reinterpret_cast<const float4 *>(sm.neg_m + c * CH + j);
                            const float m[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int r = c * CH + j + k;
                                float x = fmaf(__uint_as_float(s[j + k]), c2, m[k]);
                                if (masked && (r < r0 || r >= r1)) x = NEG_INF;
                                xm = fmaxf(xm, x);
                            }
                        }
                    }
                    slow = soft_any(xm > M_STEP || poison);
                }
                bool any_poison = false;
                if (slow) {
                    // the rows' maxima over the tile, new references, and what has been summed scaled to them
#pragma unroll
                    for (int c = 0; c < NCH; ++c) {
                        if (NCH > 1) tmem_ld<CH>(ts + c * CH, s);
                        float mine = NEG_INF;
#pragma unroll
                        for (int j = 0; j < CH; ++j) {
                            const int r = c * CH + j;
                            float y = __uint_as_float(s[j]) * c2;
                            if (masked && (r < r0 || r >= r1)) y = NEG_INF;
                            y = warp_max_f(y);
                            if (lane == j) mine = y;
                        }
                        if (lane < CH) sm.part[warp][c * CH + lane] = mine;
                    }
                    soft_sync();
                    if (tid < N) {
                        const float mo = -sm.neg_m[tid];
                        float mn = fmaxf(fmaxf(sm.part[0][tid], sm.part[1][tid]),
                                         fmaxf(sm.part[2][tid], sm.part[3][tid]));
                        mn = fmaxf(mn, mo);
                        sm.fac[tid] = ex2(mo - mn);
                        sm.neg_m[tid] = -mn;
                    }
                    any_poison = soft_any(poison);
#pragma unroll
                    for (int j = 0; j < N; ++j) l[j] *= sm.fac[j];
                    if (i > 0) {
                        tc_wait(sm, &sm.pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1);
                        __syncwarp();
                        tc_fence_after();
                        for (int m = 0; m < mb * N; m += 16) {
                            uint32_t o[16];
                            float f[16];
                            tmem_ld<16>(tm_o + lanes + m, o);
#pragma unroll
                            for (int j = 0; j < 16; ++j) f[j] = __uint_as_float(o[j]) * sm.fac[(m + j) % N];
                            tmem_st16(tm_o + lanes + m, f);
                        }
                        tmem_wait_st();
                    }
                    if (NCH == 1) tmem_ld<CH>(ts, s);
                }
                // P buffer n % np is free once the product that read it last is done
                if (n >= static_cast<uint32_t>(g.np)) {
                    const uint32_t k = n - g.np;
                    tc_wait(sm, &sm.pv_done[k & 1], (k >> 1) & 1);
                    __syncwarp();
                }
                unsigned char *pb = sp + (n % g.np) * p_bytes(N);
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
                    if (NCH > 1) tmem_ld<CH>(ts + c * CH, s);
#pragma unroll
                    for (int j = 0; j < CH; j += 8) {
                        float p[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int r = c * CH + j + k;
                            float x = fmaf(__uint_as_float(s[j + k]), c2, sm.neg_m[r]);
                            if (masked && (r < r0 || r >= r1)) x = NEG_INF;
                            p[k] = ex2(x);
                            l[r] += p[k];
                        }
                        *reinterpret_cast<uint4 *>(pb + ((c * CH + j) / 8) * (TK * 16) + tid * 16) =
                            make_uint4(pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]), pack_bf16(p[4], p[5]),
                                       pack_bf16(p[6], p[7]));
                    }
                }
                if (any_poison) {
                    // keys that some rows see and some do not, with values that are not finite: their products
                    // with p go straight into O^T
                    const unsigned mine = __ballot_sync(FULL, poison);
                    if (lane == 0) sm.bad[warp] = mine;
                    if (i == 0) {
                        float z[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) z[j] = 0.f;
                        for (int m = 0; m < mb * N; m += 16) tmem_st16(tm_o + lanes + m, z);
                        tmem_wait_st();
                        if (tid == 0) sm.acc_first = 1;
                    }
                    soft_sync();
                    for (int key = 0; key < TK; ++key) {
                        if (!(sm.bad[key >> 5] >> (key & 31) & 1)) continue;
                        if (tid == key) {
                            for (int e = 0; e < g.ds * 64; ++e) {
                                const int q = vseq + e / 64, chunk = (e % 64) / 8;
                                unsigned short *v = reinterpret_cast<unsigned short *>(
                                    ring + (q % g.nslots) * SLOT_BYTES + key * 128 + ((chunk ^ (key & 7)) * 16) +
                                    (e % 8) * 2);
                                const bool b = bad_bf16(*v);
                                sm.side[e] = b ? *v : 0;
                                if (b) *v = 0;
                            }
                        }
                        soft_sync();
                        for (int m = 0; m < mb; ++m) {
                            const int e = g.ds > 1 ? m * 128 + tid : tid & 63;
                            const float v = __uint_as_float(static_cast<uint32_t>(sm.side[e]) << 16);
                            for (int r = 0; r < N; r += 16) {
                                uint32_t o[16];
                                float f[16];
                                tmem_ld<16>(tm_o + lanes + m * N + r, o);
#pragma unroll
                                for (int j = 0; j < 16; ++j) {
                                    const unsigned short pk = *reinterpret_cast<const unsigned short *>(
                                        pb + ((r + j) / 8) * (TK * 16) + key * 16 + (j % 8) * 2);
                                    const float p = __uint_as_float(static_cast<uint32_t>(pk) << 16);
                                    f[j] = __uint_as_float(o[j]);
                                    if (p != 0.f && v != 0.f) f[j] = fmaf(p, v, f[j]);
                                }
                                tmem_st16(tm_o + lanes + m * N + r, f);
                            }
                        }
                        tmem_wait_st();
                        soft_sync();
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_full[n & 1]);
            }
            seq += 2 * nt * g.ds;
            // the rows' sums over all keys
            lane_sums<N>(l, lane);
#pragma unroll
            for (int j = 0; j < (N + 31) / 32; ++j) {
                const int r = N >= 32 ? lane * (N / 32) + j : lane / (32 / N);
                sm.part[warp][r] = l[j];
            }
            soft_sync();
            float *part = w.whole ? nullptr : attn_part(a, blockIdx.x, w.starts);
            if (tid < rows) {
                float L = sm.part[0][tid] + sm.part[1][tid] + sm.part[2][tid] + sm.part[3][tid];
                float m = -sm.neg_m[tid];
                if (tc_aborted(sm)) L = NAN;
                else if (tid >= real) L = 0.f;
                sm.inv[tid] = L == 0.f ? 0.f : (w.whole ? 1.0f / L : 1.f);
                if (w.whole) {
                    if (a.lse) a.lse[sm.row_at[tid]] = L == 0.f ? NEG_INF : (m + log2f(L)) * 0.6931471805599453f;
                } else {
                    part[a.rows_cap * a.d + tid] = m;
                    part[a.rows_cap * (a.d + 1) + tid] = L;
                }
            }
            tc_wait(sm, &sm.pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1);
            soft_sync();
            tc_fence_after();
            if (g.ds > 1 || warp < 2) {
                for (int m = 0; m < mb; ++m) {
                    const int e = m * 128 + tid;
                    for (int r = 0; r < rows; r += 16) {
                        uint32_t o[16];
                        tmem_ld<16>(tm_o + lanes + m * N + r, o);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            if (r + j >= rows) break;
                            const float f = sm.inv[r + j];
                            const float v = f == 0.f ? 0.f : __uint_as_float(o[j]) * f;
                            if (w.whole)
                                attn_store(a, sm.row_at[r + j] * a.d + e, v, static_cast<unsigned short *>(nullptr));
                            else
                                part[static_cast<int64_t>(r + j) * a.d + e] = v;
                        }
                    }
                }
            }
            tc_fence_before();
            if (!w.whole) attn_join<unsigned short>(a, w, rows, h, tok0, 128, tid, &sm.flag, soft_sync);
            soft_sync();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 5) tmem_dealloc(tm_s, cols);
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
    const int N = a.rows_cap <= 16 ? 16 : a.rows_cap <= 32 ? 32 : a.rows_cap <= 64 ? 64 : 128;
    TcGeom g;
    g.ds = a.d / 64;
    g.np = N == 128 ? 1 : 2;
    g.box = 8;
    while (g.box < TK && a.page_size % (2 * g.box) == 0) g.box *= 2;
    const int rest = SM_BYTES - 1024 - static_cast<int>(sizeof(TcShared)) - 256 - q_bytes(N, g.ds) - g.np * p_bytes(N);
    g.nslots = rest / SLOT_BYTES / 2 * 2;                     // even: the two slots of a V block are neighbours
    if (g.nslots > MAX_SLOTS) g.nslots = MAX_SLOTS;
    const size_t smem = 1024 + static_cast<size_t>(g.nslots) * SLOT_BYTES + q_bytes(N, g.ds) + g.np * p_bytes(N);

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
    if (!make_map_4d(&mk, a.k, cd, cs, g.box, 1) || !make_map_4d(&mv, a.v, cd, cs, g.box, 1) ||
        !make_map_4d(&mq, a.q, qd, qs, a.group, a.tok_block))
        return DFLASH2_ERR_CUDA;

    const double tiles = static_cast<double>(a.B) * a.items *
                         ((static_cast<int64_t>(a.max_pages) * a.page_size + TK - 1) / TK);
    const int ctas = tiles < sm_count() ? static_cast<int>(tiles) : sm_count();
    void *fn = N == 16   ? reinterpret_cast<void *>(&k_attn_tc<16>)
               : N == 32 ? reinterpret_cast<void *>(&k_attn_tc<32>)
               : N == 64 ? reinterpret_cast<void *>(&k_attn_tc<64>)
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
