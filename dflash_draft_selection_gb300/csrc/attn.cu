// attn.cu -- dflash2_paged_attn: the entry point, and the CUDA-core kernels
// that take float32 caches and the head dimensions the tensor-core kernels
// (attn_tc.cu) do not.
//
//   x_s = scale <q, k_s>,  out = sum_s exp(x_s) v_s / sum_s exp(x_s)
// in one pass over the cache: a row keeps its running maximum m and sum l,
// and what it has summed so far is multiplied by exp(m - m') when the maximum
// grows to m'.  Everything is fp32; exponentials are taken in base 2.
#include "attn.cuh"
#include "tc.cuh"

namespace dfl {

// The tensor-core kernels (attn_tc.cu).
bool attn_tc_takes(const AttnArgs &a);
dflash2_status attn_tc_launch(AttnArgs a, bool weights, cudaStream_t s);

constexpr int SIMT_THREADS = 256;
constexpr int SIMT_KEYS_LOG2 = 5, SIMT_KEYS = 32;  // keys per tile: one per lane in the score step
constexpr int SIMT_TILE_ROWS = 32;  // query rows of a block: four per warp in the score step
constexpr int SIMT_ROWS = 16;       // ... of the weights pass: two per warp

template <bool V>
struct BoolC {
    static constexpr bool value = V;
};

template <typename E>
__device__ __forceinline__ float4 ld4(const void *p, int64_t i);
template <>
__device__ __forceinline__ float4 ld4<float>(const void *p, int64_t i) {
    return *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
}
template <>
__device__ __forceinline__ float4 ld4<unsigned short>(const void *p, int64_t i) {
    const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const unsigned short *>(p) + i);
    return make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
}

// Shared memory: Q [ROWS][ld], K [KEYS][ld], V [KEYS][d] as floats (ld = d + 4:
// the lanes' float4 reads of their own key's row fall into different banks).
template <typename E>
__device__ __forceinline__ void simt_load_q(const AttnArgs &a, const AttnWalk &w, int h, int tok0, int row0, int rows,
                                            float *sq, int ld) {
    const int d4 = a.d / 4;
    for (int i = threadIdx.x; i < SIMT_ROWS * d4; i += SIMT_THREADS) {
        const int r = i / d4, c = (i % d4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row0 + r < rows) x = ld4<E>(a.q, attn_row(a, w.b, h, tok0, row0 + r) * a.d + c);
        *reinterpret_cast<float4 *>(sq + r * ld + c) = x;
    }
}

template <typename E>
__device__ __forceinline__ void simt_load_tile(const AttnArgs &a, const void *src, const int *s_page, int h, int tile,
                                               float *dst, int ld) {
    const int d4 = a.d / 4;
    for (int i = threadIdx.x; i < SIMT_KEYS * d4; i += SIMT_THREADS) {
        const int j = i / d4, c = (i % d4) * 4;
        const int page = s_page[j];
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (page >= 0) {
            const int off = (tile * SIMT_KEYS + j) % a.page_size;
            x = ld4<E>(src, page * a.page_stride + h * a.head_stride + off * a.slot_stride + c);
        }
        *reinterpret_cast<float4 *>(dst + j * ld + c) = x;
    }
}

// The two scores of this thread's lane (key) and warp (rows warp, warp + 8).
__device__ __forceinline__ void simt_scores(const float *sq, const float *sk, int ld, int d, int warp, int lane,
                                            float &x0, float &x1) {
    x0 = x1 = 0.f;
    const float *kp = sk + lane * ld, *q0 = sq + warp * ld, *q1 = sq + (warp + 8) * ld;
#pragma unroll 4
    for (int c = 0; c < d; c += 4) {
        const float4 k = *reinterpret_cast<const float4 *>(kp + c);
        const float4 u = *reinterpret_cast<const float4 *>(q0 + c);
        const float4 v = *reinterpret_cast<const float4 *>(q1 + c);
        x0 = fmaf(k.x, u.x, fmaf(k.y, u.y, fmaf(k.z, u.z, fmaf(k.w, u.w, x0))));
        x1 = fmaf(k.x, v.x, fmaf(k.y, v.y, fmaf(k.z, v.z, fmaf(k.w, v.w, x1))));
    }
}

static __device__ __forceinline__ void cta_sync() { __syncthreads(); }

static __host__ __device__ size_t attn_simt_smem(int d, int e) {
    return static_cast<size_t>(SIMT_TILE_ROWS) * (d + 4) * 4 + static_cast<size_t>(4) * SIMT_KEYS * (d + 16 / e) * e;
}

// One CTA per stretch, 32 query rows against tiles of 32 keys, which arrive by
// asynchronous copies one tile ahead.  Scores: warp w has rows 4 w .. 4 w + 3
// and lane l key l, so a row's maximum and sum are the warp's; the four rows
// share the reads of the key.  Output: a thread has RPT rows x 4 dims, so a
// value read from shared memory feeds RPT products.
// Bound: the fp32 units (rows * d * 4 operations per key) once more than a
// few rows share a key, the bytes below that; short calls are bound by the
// chain of lookups, copies and the join.  4 requests of 100 to 4096 slots, 32
// rows on 4 heads of 64 (23 MB, 0.37 GFLOP): 35 us on 304 CTAs of 3.5 tiles,
// about 20 of them the plan, the first copy and the join of 19 parts.
// bf16 caches that the tensor-core kernels do not take: 32 requests of 8 to 8192
// slots, 8 tokens, 40 heads on 8: d 80 789 us, d 96 924, d 192 1631, pages of 20
// slots 1087 (d 128), 15 to 18 TFLOP/s, 15 to 17 times their bytes' time.  The
// score step reads five vectors of shared memory for sixteen products.
template <typename E>
struct SimtTile {
    static constexpr int PAD = 16 / sizeof(E);  // elements between rows: the lanes' reads fall into different banks
};
constexpr int P_LD = SIMT_TILE_ROWS + 4;

template <typename E>
__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}

// A tile's keys: their pages and places in them, and the rows that see them.
struct SimtKeys {
    int page[SIMT_KEYS], off[SIMT_KEYS], lo[SIMT_KEYS], hi[SIMT_KEYS];
};

// Asks for a tile's keys and values; rows without a page become zero.
template <typename E>
__device__ __forceinline__ void simt_ask(const AttnArgs &a, int h, const SimtKeys &t, E *sk, E *sv, int ld) {
    constexpr int N = 16 / sizeof(E);
    const int vecs = a.d / N;
    for (int i = threadIdx.x; i < SIMT_KEYS * vecs; i += SIMT_THREADS) {
        const int j = i / vecs, c = (i - j * vecs) * N, page = t.page[j];
        E *dk = sk + j * ld + c, *dv = sv + j * ld + c;
        if (page >= 0) {
            const int64_t at = page * a.page_stride + h * a.head_stride + t.off[j] * a.slot_stride + c;
            cp_async16<E>(dk, reinterpret_cast<const E *>(a.k) + at);
            cp_async16<E>(dv, reinterpret_cast<const E *>(a.v) + at);
        } else {
            *reinterpret_cast<uint4 *>(dk) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(dv) = make_uint4(0, 0, 0, 0);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <typename E, int RPT>
__global__ void __launch_bounds__(SIMT_THREADS, 2) k_attn_simt(AttnArgs a) {
    extern __shared__ float smem[];
    __shared__ int scratch[SIMT_THREADS / 32 + 2];
    __shared__ SimtKeys s_keys[3];  // this tile's, the next one's and the one after
    __shared__ int s_flag;
    __shared__ alignas(16) float s_p[SIMT_KEYS * P_LD];
    __shared__ float s_f[SIMT_TILE_ROWS], s_m[SIMT_TILE_ROWS], s_inv[128];
    __shared__ int s_row[128];
    const int d = a.d, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, ld = d + SimtTile<E>::PAD, ldq = d + 4;
    float *sq = smem;
    E *kv = reinterpret_cast<E *>(sq + SIMT_TILE_ROWS * ldq);  // [2][keys, values][KEYS][ld]
    pdl_wait();
    const AttnPlan p = attn_plan<SIMT_THREADS>(a, scratch);
    if (p.begin >= p.end) return;
    const int d4 = d / 4, oc = (tid % d4) * 4, or0 = tid / d4 * RPT;  // output step: dims oc .., rows or0 ..
    const bool out_on = or0 < SIMT_TILE_ROWS;
    const float c2 = a.scale * LOG2E;
    AttnWalk w;
    w.start(a, p);
    while (w.next(a)) {
        const int h = w.item / a.row_blocks, tok0 = (w.item % a.row_blocks) * a.tok_block;
        const int rows = min(a.tok_block, a.T - tok0) * a.group;
        for (int row0 = 0; row0 < rows; row0 += SIMT_TILE_ROWS) {  // more than one round only where group > 32
            // one warp looks a tile's pages and positions up, two tiles ahead
            auto look = [&](int t) {
                if (tid < SIMT_KEYS) {
                    SimtKeys &k = s_keys[(t - w.t0) % 3];
                    const int slot = t * SIMT_KEYS + tid;
                    int lo = 0, hi = 0, page = -1;
                    if (t < w.t1) attn_view_slot(a, w.r, w.b, h, slot, lo, hi, page);
                    k.page[tid] = page;
                    k.off[tid] = slot % a.page_size;
                    k.lo[tid] = (lo - tok0) * a.group - row0;  // rows of this block that see the key
                    k.hi[tid] = (hi - tok0) * a.group - row0;
                }
            };
            __syncthreads();
            look(w.t0);
            look(w.t0 + 1);
            __syncthreads();
            simt_ask<E>(a, h, s_keys[0], kv, kv + SIMT_KEYS * ld, ld);
            for (int i = tid; i < SIMT_TILE_ROWS * d4; i += SIMT_THREADS) {
                const int r = i / d4, c = (i - r * d4) * 4;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (row0 + r < rows) x = ld4<E>(a.q, attn_row(a, w.b, h, tok0, row0 + r) * d + c);
                *reinterpret_cast<float4 *>(sq + r * ldq + c) = x;
            }
            float m[4], l[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                m[k] = NEG_INF;
                l[k] = 0.f;
            }
            float4 acc[RPT];
#pragma unroll
            for (int i = 0; i < RPT; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int t = w.t0; t < w.t1; ++t) {
                const int buf = (t - w.t0) & 1;
                const E *sk = kv + buf * 2 * SIMT_KEYS * ld, *sv = sk + SIMT_KEYS * ld;
                asm volatile("cp.async.wait_all;" ::: "memory");
                __syncthreads();
                if (t + 1 < w.t1) {
                    E *next = kv + (buf ^ 1) * 2 * SIMT_KEYS * ld;
                    simt_ask<E>(a, h, s_keys[(t + 1 - w.t0) % 3], next, next + SIMT_KEYS * ld, ld);
                    look(t + 2);
                }
                float x[4] = {0.f, 0.f, 0.f, 0.f};
                const E *kp = sk + lane * ld;
                const float *qp = sq + warp * 4 * ldq;
#pragma unroll 4
                for (int c = 0; c < d; c += 4) {
                    const float4 k = ld4<E>(kp, c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 q = *reinterpret_cast<const float4 *>(qp + i * ldq + c);
                        x[i] = fmaf(k.x, q.x, fmaf(k.y, q.y, fmaf(k.z, q.z, fmaf(k.w, q.w, x[i]))));
                    }
                }
                const SimtKeys &keys = s_keys[(t - w.t0) % 3];
                const int lo = keys.lo[lane], hi = keys.hi[lane];
                float f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = warp * 4 + i;
                    const bool on = r >= lo && r < hi;
                    x[i] = on ? x[i] * c2 : NEG_INF;
                    const float n = fmaxf(m[i], warp_max_one(x[i]));
                    // a row that has seen nothing yet keeps m = -inf and adds nothing; a NaN score stays NaN
                    const float e = !on || (n == NEG_INF && x[i] == NEG_INF) ? 0.f : ex2(x[i] - n);
                    f[i] = m[i] == NEG_INF ? 0.f : ex2(m[i] - n);
                    l[i] = (m[i] == NEG_INF ? l[i] : l[i] * f[i]) + e;  // the lane's keys; the warp's at the end
                    m[i] = n;
                    x[i] = e;
                }
                *reinterpret_cast<float4 *>(s_p + lane * P_LD + warp * 4) = make_float4(x[0], x[1], x[2], x[3]);
                if (lane == 0) *reinterpret_cast<float4 *>(s_f + warp * 4) = make_float4(f[0], f[1], f[2], f[3]);
                // some row does not see some key: what it does not see may be NaN
                const bool partial = __syncthreads_or(lo > 0 || hi < min(rows - row0, SIMT_TILE_ROWS));
                if (out_on) {
#pragma unroll
                    for (int i = 0; i < RPT; ++i) {
                        const float g = s_f[or0 + i];
                        acc[i] = make_float4(acc[i].x * g, acc[i].y * g, acc[i].z * g, acc[i].w * g);
                    }
                    auto add = [&](auto checked) {
#pragma unroll 4
                        for (int j = 0; j < SIMT_KEYS; ++j) {
                            const float4 v = ld4<E>(sv + j * ld, oc);
                            float q[RPT];
#pragma unroll
                            for (int i = 0; i < RPT; i += 2) {
                                const float2 y = *reinterpret_cast<const float2 *>(s_p + j * P_LD + or0 + i);
                                q[i] = y.x;
                                q[i + 1] = y.y;
                            }
#pragma unroll
                            for (int i = 0; i < RPT; ++i)
                                if (!decltype(checked)::value || q[i] != 0.f) {
                                    acc[i].x = fmaf(q[i], v.x, acc[i].x);
                                    acc[i].y = fmaf(q[i], v.y, acc[i].y);
                                    acc[i].z = fmaf(q[i], v.z, acc[i].z);
                                    acc[i].w = fmaf(q[i], v.w, acc[i].w);
                                }
                        }
                    };
                    if (partial)
                        add(BoolC<true>());
                    else
                        add(BoolC<false>());
                }
            }
            // l and m of the rows to everyone
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 4; ++k) l[k] = warp_sum(l[k]);
            if (lane == 0) {
                *reinterpret_cast<float4 *>(s_f + warp * 4) = make_float4(l[0], l[1], l[2], l[3]);
                *reinterpret_cast<float4 *>(s_m + warp * 4) = make_float4(m[0], m[1], m[2], m[3]);
            }
            __syncthreads();
            float *part = w.whole ? nullptr : attn_part(a, blockIdx.x, w.starts);
            if (out_on) {
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const int r = or0 + i;
                    if (row0 + r >= rows) break;
                    const float L = s_f[r];
                    if (w.whole) {
                        const float inv = L == 0.f ? 0.f : 1.0f / L;
                        const int64_t row = attn_row(a, w.b, h, tok0, row0 + r);
                        const bool on = L != 0.f;
                        attn_store4(a, row * d + oc, on ? acc[i].x * inv : 0.f, on ? acc[i].y * inv : 0.f,
                                    on ? acc[i].z * inv : 0.f, on ? acc[i].w * inv : 0.f, static_cast<E *>(nullptr));
                        if (oc == 0 && a.lse) a.lse[row] = on ? (s_m[r] + log2f(L)) * 0.6931471805599453f : NEG_INF;
                    } else {
                        *reinterpret_cast<float4 *>(part + static_cast<int64_t>(row0 + r) * d + oc) = acc[i];
                        if (oc == 0) {
                            part[a.rows_cap * d + row0 + r] = s_m[r];
                            part[a.rows_cap * (d + 1) + row0 + r] = L;
                        }
                    }
                }
            }
        }
        if (!w.whole) {
            if (tid < rows) s_row[tid] = tid / a.group * a.Hq + tid % a.group;
            attn_join<E, 0>(a, AttnParts(a, p, w), w, rows, tok0, SIMT_THREADS, tid, &s_flag, smem,
                            static_cast<int>(attn_simt_smem(d, sizeof(E)) / 4), s_inv, attn_row(a, w.b, h, tok0, 0), s_row, cta_sync);
        }
    }
}

// weight_s += sum over the rows that see s of exp(x_s - lse): the second pass,
// over the keys alone.  One CTA owns a (request, head)'s tile, so no two add
// to the same word, and the rows are added in a fixed order.  Bound: the loads of
// the rows, again for each tile of 32 keys, and of the tile, with no copy ahead.  4
// requests of 100 to 4096 slots, 8 tokens, 16 heads on 4 of 64, float32: 56 us
// with the attention; 16 requests of 2048 to 4028 slots, a token of 32 heads on 8
// of 96, bf16: 391 us with the attention.
template <typename E>
__global__ void __launch_bounds__(SIMT_THREADS) k_weights_simt(AttnArgs a) {
    extern __shared__ float smem[];
    __shared__ int scratch[SIMT_THREADS / 32 + 2];
    __shared__ int s_page[SIMT_KEYS], s_lo[SIMT_KEYS], s_hi[SIMT_KEYS];
    __shared__ float s_w[8][SIMT_KEYS];
    const int d = a.d, ld = d + 4, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float *sq = smem, *sk = sq + SIMT_ROWS * ld;
    pdl_wait();
    const AttnPlan p = attn_plan<SIMT_THREADS>(a, scratch);
    if (p.begin >= p.end) return;
    const float c2 = a.scale * LOG2E;
    AttnWalk w;
    w.start(a, p);
    while (w.next(a)) {
        const int h = w.item, rows = w.r.nq * a.group;
        for (int t = w.t0; t < w.t1; ++t) {
            __syncthreads();
            if (tid < SIMT_KEYS) attn_view_slot(a, w.r, w.b, h, t * SIMT_KEYS + tid, s_lo[tid], s_hi[tid], s_page[tid]);
            __syncthreads();
            simt_load_tile<E>(a, a.k, s_page, h, t, sk, ld);
            float sum = 0.f;
            for (int row0 = 0; row0 < rows; row0 += SIMT_ROWS) {
                __syncthreads();
                simt_load_q<E>(a, w, h, 0, row0, rows, sq, ld);
                __syncthreads();
                float x[2];
                simt_scores(sq, sk, ld, d, warp, lane, x[0], x[1]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = row0 + warp + 8 * i;
                    if (r >= rows || r < s_lo[lane] * a.group || r >= s_hi[lane] * a.group) continue;
                    const float z = a.lse[attn_row(a, w.b, h, 0, r)];
                    if (z != NEG_INF) sum += ex2(fmaf(x[i], c2, -z * LOG2E));
                }
            }
            s_w[warp][lane] = sum;
            __syncthreads();
            if (tid < SIMT_KEYS && s_page[tid] >= 0 && s_lo[tid] < s_hi[tid]) {
                float g = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) g += s_w[i][tid];
                const int off = (t * SIMT_KEYS + tid) % a.page_size;
                a.weight[(static_cast<int64_t>(s_page[tid]) * a.Hkv + h) * a.page_size + off] += g;
            }
        }
    }
}

static size_t simt_smem(int d) { return static_cast<size_t>((SIMT_ROWS + SIMT_KEYS) * (d + 4) + SIMT_KEYS * d) * 4; }

static dflash2_status launch_simple(void *fn, AttnArgs &a, int threads, size_t smem, int64_t ctas, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[1] = {&a};
    if (cudaLaunchKernelExC(&cfg, fn, args) != cudaSuccess) return DFLASH2_ERR_CUDA;
    return after_launch();
}

// CTAs of the CUDA-core kernels at most: two per SM (their registers).  The tensor-core kernels take one per SM.
static int attn_ctas() { return sm_count() * 2 < ATTN_MAX_CTAS ? sm_count() * 2 : ATTN_MAX_CTAS; }

// CTAs of a call: no more than there can be tiles.
static int64_t simt_grid(const AttnArgs &a) {
    const int64_t cap = (static_cast<int64_t>(a.max_pages) * a.page_size + SIMT_KEYS - 1) / SIMT_KEYS;
    const double t = static_cast<double>(a.B) * a.items * cap;
    return t < attn_ctas() ? static_cast<int64_t>(t) : attn_ctas();
}

template <typename E>
static dflash2_status launch_simt(AttnArgs a, cudaStream_t s) {
    // rows a thread has in the output step: 256 threads over d / 4 vectors and 32 rows
    void *fn = a.d <= 64 ? reinterpret_cast<void *>(&k_attn_simt<E, 2>)
               : a.d <= 128 ? reinterpret_cast<void *>(&k_attn_simt<E, 4>)
                            : reinterpret_cast<void *>(&k_attn_simt<E, 8>);
    blocks_per_sm(fn, SIMT_THREADS, attn_simt_smem(256, sizeof(E)));  // raises the shared-memory limit, once per device
    a.tile_log2 = SIMT_KEYS_LOG2;
    a.tok_block = SIMT_TILE_ROWS / a.group > 0 ? SIMT_TILE_ROWS / a.group : 1;
    if (a.tok_block > a.T) a.tok_block = a.T;
    a.row_blocks = (a.T + a.tok_block - 1) / a.tok_block;
    a.rows_cap = a.tok_block * a.group;
    a.items = a.Hkv * a.row_blocks;
    a.item_cost = 1;
    return launch_simple(fn, a, SIMT_THREADS, attn_simt_smem(a.d, sizeof(E)), simt_grid(a), s);
}

template <typename E>
static dflash2_status launch_weights_simt(AttnArgs a, cudaStream_t s) {
    void *fn = reinterpret_cast<void *>(&k_weights_simt<E>);
    a.tile_log2 = SIMT_KEYS_LOG2;
    a.items = a.Hkv;
    blocks_per_sm(fn, SIMT_THREADS, simt_smem(256));
    return launch_simple(fn, a, SIMT_THREADS, simt_smem(a.d), simt_grid(a), s);
}

// Rows of one part in the workspace, for either kind of kernel.
static int part_rows(int32_t T, int32_t group) {
    const int64_t rows = static_cast<int64_t>(T) * group;
    return rows < 128 ? static_cast<int>(rows) : 128;
}

// The cache, and the page table of B requests (an empty batch has none).
bool kv_cache_ok(const dflash2_kv_cache *c, const int32_t *table, int32_t max_pages, int64_t B) {
    if (!c || !c->k || !c->v || !dtype_ok(c->dt)) return false;
    if (B != 0 && (!table || max_pages < 1)) return false;
    const int e = esize(c->dt);
    auto al4 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; };
    return c->num_pages >= 1 && c->Hkv >= 1 && c->page_size >= 1 && c->d >= 1 && max_pages >= 0 && aligned16(c->k) &&
           aligned16(c->v) && c->page_stride * e % 16 == 0 && c->head_stride * e % 16 == 0 &&
           c->slot_stride * e % 16 == 0 && static_cast<int64_t>(c->d) * e % 16 == 0 && c->slot_stride >= c->d &&
           c->head_stride >= 0 && c->page_stride >= 0 && al4(c->weight) && al4(c->pos) && al4(table);
}

}  // namespace dfl

using namespace dfl;

extern "C" size_t dflash2_paged_attn_workspace_bytes(int64_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t d,
                                                     dflash2_dtype dt) {
    if (B < 0 || T < 0 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || d < 1 || !dtype_ok(dt)) return 0;
    return WS_ZERO_BYTES +
           static_cast<size_t>(attn_ctas()) * 2 * attn_part_floats(part_rows(T, Hq / Hkv), d) * sizeof(float);
}

extern "C" dflash2_status dflash2_paged_attn(const dflash2_kv_cache *cache, const int32_t *page_table,
                                             int32_t max_pages, const int32_t *kv_len, const int32_t *q_len,
                                             const int32_t *seq_pos, const void *q, int64_t B, int32_t T, int32_t Hq,
                                             float scale, int32_t window, uint32_t flags, void *out, float *lse,
                                             void *ws, size_t ws_bytes, dflash2_stream stream) {
    if (!kv_cache_ok(cache, page_table, max_pages, B) || B < 0 || T < 0 || Hq < 1 || Hq % cache->Hkv != 0 ||
        !(scale - scale == 0.f) || window < 0 || (flags & ~3u))
        return DFLASH2_ERR_INVALID_ARG;
    const bool weights = (flags & DFLASH2_ATTN_WEIGHTS) != 0;
    if (weights && !cache->weight) return DFLASH2_ERR_INVALID_ARG;
    if (B == 0 || T == 0) return DFLASH2_OK;  // outputs of no elements may be NULL
    if (weights && !lse) return DFLASH2_ERR_INVALID_ARG;
    auto al4 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; };
    if (!q || !out || !kv_len || !ws || !aligned16(q) || !aligned16(out) || !aligned16(ws) || !al4(kv_len) ||
        !al4(q_len) || !al4(seq_pos) || !al4(lse) || out == q)
        return DFLASH2_ERR_INVALID_ARG;
    const int group = Hq / cache->Hkv;
    // 128 rows of Hq heads are counted in 31 bits
    if (cache->d > 256 || group > 128 || Hq >= (1 << 24) || cache->num_pages >= (int64_t(1) << 31) ||
        static_cast<int64_t>(max_pages) * cache->page_size >= (int64_t(1) << 31) - 256)
        return DFLASH2_ERR_UNSUPPORTED;
    // The places of a call's line are counted in 31 bits.  There are at most B Hkv T items, each of the tiles of cap
    // slots (32 keys at the least: cap / 32 + 1) and of its cost beside them (1 or ATTN_ITEM_COST).
    if (static_cast<double>(B) * cache->Hkv * T *
            (static_cast<double>(max_pages) * cache->page_size / SIMT_KEYS + 1 + ATTN_ITEM_COST) >=
        2147483648.0)
        return DFLASH2_ERR_UNSUPPORTED;
    if (ws_bytes < dflash2_paged_attn_workspace_bytes(B, T, Hq, cache->Hkv, cache->d, cache->dt))
        return DFLASH2_ERR_WORKSPACE;
    AttnArgs a = {};
    a.k = static_cast<const char *>(cache->k);
    a.v = static_cast<const char *>(cache->v);
    a.weight = cache->weight;
    a.pos = cache->pos;
    a.num_pages = cache->num_pages;
    a.page_stride = cache->page_stride;
    a.head_stride = cache->head_stride;
    a.slot_stride = cache->slot_stride;
    a.Hkv = cache->Hkv;
    a.page_size = cache->page_size;
    a.d = cache->d;
    a.table = page_table;
    a.max_pages = max_pages;
    a.kv_len = kv_len;
    a.q_len = q_len;
    a.seq_pos = seq_pos;
    a.q = q;
    a.B = B;
    a.T = T;
    a.Hq = Hq;
    a.group = group;
    a.scale = scale;
    a.window = window;
    a.causal = (flags & DFLASH2_ATTN_CAUSAL) ? 1 : 0;
    a.out = out;
    a.lse = lse;
    a.tickets = static_cast<int *>(ws);
    a.parts = reinterpret_cast<float *>(static_cast<char *>(ws) + WS_ZERO_BYTES);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    dflash2_status st;
    if (cache->dt == DFLASH2_F32) {
        st = launch_simt<float>(a, s);
        return st == DFLASH2_OK && weights ? launch_weights_simt<float>(a, s) : st;
    }
    if (attn_tc_takes(a)) return attn_tc_launch(a, weights, s);
    st = launch_simt<unsigned short>(a, s);
    return st == DFLASH2_OK && weights ? launch_weights_simt<unsigned short>(a, s) : st;
}
