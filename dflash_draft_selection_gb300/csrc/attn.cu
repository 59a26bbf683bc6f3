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
constexpr int SIMT_ROWS = 16;  // query rows per block: two per warp in the score step

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

template <typename E>
__global__ void __launch_bounds__(SIMT_THREADS) k_attn_simt(AttnArgs a) {
    extern __shared__ float smem[];
    __shared__ int scratch[SIMT_THREADS / 32 + 2];
    __shared__ int s_page[SIMT_KEYS], s_lo[SIMT_KEYS], s_hi[SIMT_KEYS], s_flag;
    __shared__ float s_p[SIMT_ROWS][SIMT_KEYS], s_f[SIMT_ROWS], s_inv[128];
    __shared__ int64_t s_row[128];
    const int d = a.d, ld = d + 4, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float *sq = smem, *sk = sq + SIMT_ROWS * ld, *sv = sk + SIMT_KEYS * ld;
    pdl_wait();
    const AttnPlan p = attn_plan<SIMT_THREADS>(a, scratch);
    if (p.begin >= p.end) return;
    const int d4 = d / 4, groups = SIMT_THREADS / d4;  // output step: thread = (4 dims, rows og, og + groups, ..)
    const int oc = (tid % d4) * 4, og = tid / d4;
    const float c2 = a.scale * LOG2E;
    AttnWalk w;
    w.start(a, p);
    while (w.next(a)) {
        const int h = w.item / a.row_blocks, tok0 = (w.item % a.row_blocks) * a.tok_block;
        const int rows = min(a.tok_block, a.T - tok0) * a.group;
        for (int row0 = 0; row0 < rows; row0 += SIMT_ROWS) {  // more than one pass only where group > ROWS
            __syncthreads();
            simt_load_q<E>(a, w, h, tok0, row0, rows, sq, ld);
            float m0 = NEG_INF, m1 = NEG_INF, l0 = 0.f, l1 = 0.f;
            float4 acc[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int t = w.t0; t < w.t1; ++t) {
                __syncthreads();
                if (tid < SIMT_KEYS) {
                    int lo, hi, page;
                    attn_view_slot(a, w.r, w.b, h, t * SIMT_KEYS + tid, lo, hi, page);
                    s_page[tid] = page;
                    s_lo[tid] = (lo - tok0) * a.group - row0;  // rows of this block that see the key
                    s_hi[tid] = (hi - tok0) * a.group - row0;
                }
                __syncthreads();
                simt_load_tile<E>(a, a.k, s_page, h, t, sk, ld);
                simt_load_tile<E>(a, a.v, s_page, h, t, sv, d);
                __syncthreads();
                float x0, x1;
                simt_scores(sq, sk, ld, d, warp, lane, x0, x1);
                const int lo = s_lo[lane], hi = s_hi[lane];
                const bool on0 = warp >= lo && warp < hi, on1 = warp + 8 >= lo && warp + 8 < hi;
                x0 = on0 ? x0 * c2 : NEG_INF;
                x1 = on1 ? x1 * c2 : NEG_INF;
                const float n0 = fmaxf(m0, warp_max_f(x0)), n1 = fmaxf(m1, warp_max_f(x1));
                // a row that has seen nothing yet keeps m = -inf and adds nothing; a NaN score stays NaN
                const float p0 = !on0 || (n0 == NEG_INF && x0 == NEG_INF) ? 0.f : ex2(x0 - n0);
                const float p1 = !on1 || (n1 == NEG_INF && x1 == NEG_INF) ? 0.f : ex2(x1 - n1);
                const float f0 = m0 == NEG_INF ? 0.f : ex2(m0 - n0), f1 = m1 == NEG_INF ? 0.f : ex2(m1 - n1);
                l0 = (m0 == NEG_INF ? l0 : l0 * f0) + warp_sum(p0);
                l1 = (m1 == NEG_INF ? l1 : l1 * f1) + warp_sum(p1);
                m0 = n0;
                m1 = n1;
                s_p[warp][lane] = p0;
                s_p[warp + 8][lane] = p1;
                if (lane == 0) {
                    s_f[warp] = f0;
                    s_f[warp + 8] = f1;
                }
                __syncthreads();
                if (og < groups) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = og + i * groups;
                        if (r >= SIMT_ROWS) break;
                        const float f = s_f[r];
                        float4 o = acc[i];
                        if (f != 1.f) o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll 8
                        for (int j = 0; j < SIMT_KEYS; ++j) {
                            const float q = s_p[r][j];
                            const float4 v = *reinterpret_cast<const float4 *>(sv + j * d + oc);
                            if (q != 0.f) {  // what a row does not see may be NaN
                                o.x = fmaf(q, v.x, o.x);
                                o.y = fmaf(q, v.y, o.y);
                                o.z = fmaf(q, v.z, o.z);
                                o.w = fmaf(q, v.w, o.w);
                            }
                        }
                        acc[i] = o;
                    }
                }
            }
            // l and m of the rows to everyone
            __syncthreads();
            if (lane == 0) {
                s_f[warp] = l0;
                s_f[warp + 8] = l1;
                s_p[0][warp] = m0;
                s_p[0][warp + 8] = m1;
            }
            __syncthreads();
            float *part = w.whole ? nullptr : attn_part(a, blockIdx.x, w.starts);
            if (og < groups) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = og + i * groups;
                    if (r >= SIMT_ROWS || row0 + r >= rows) break;
                    const float l = s_f[r];
                    if (w.whole) {
                        const float inv = l == 0.f ? 0.f : 1.0f / l;
                        const int64_t row = attn_row(a, w.b, h, tok0, row0 + r), at = row * d + oc;
                        const float o[4] = {acc[i].x, acc[i].y, acc[i].z, acc[i].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) attn_store(a, at + k, l == 0.f ? 0.f : o[k] * inv, static_cast<E *>(nullptr));
                        if (oc == 0 && a.lse) a.lse[row] = l == 0.f ? NEG_INF : (s_p[0][r] + log2f(l)) * 0.6931471805599453f;
                    } else {
                        *reinterpret_cast<float4 *>(part + static_cast<int64_t>(row0 + r) * d + oc) = acc[i];
                        if (oc == 0) {
                            part[a.rows_cap * d + row0 + r] = s_p[0][r];
                            part[a.rows_cap * (d + 1) + row0 + r] = l;
                        }
                    }
                }
            }
        }
        if (!w.whole) {
            if (tid < rows) s_row[tid] = attn_row(a, w.b, h, tok0, tid);
            attn_join<E, 0>(a, AttnParts(a, p, w), w, rows, tok0, SIMT_THREADS, tid, &s_flag, smem, SIMT_KEYS * ld, s_inv, s_row, cta_sync);
        }
    }
}

// weight_s += sum over the rows that see s of exp(x_s - lse): the second pass,
// over the keys alone.  One CTA owns a (request, head)'s tile, so no two add
// to the same word, and the rows are added in a fixed order.
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

static int attn_ctas() { return sm_count() * 3 < ATTN_MAX_CTAS ? sm_count() * 3 : ATTN_MAX_CTAS; }

// CTAs of a call: as many as are resident, no more than there can be tiles.
static int64_t simt_grid(const AttnArgs &a, const void *fn) {
    const int64_t per = blocks_per_sm(fn, SIMT_THREADS, simt_smem(256));
    const int64_t slots = static_cast<int64_t>(sm_count()) * (per < 3 ? per : 3);
    const int64_t most = slots < ATTN_MAX_CTAS ? slots : ATTN_MAX_CTAS;
    const int64_t cap = (static_cast<int64_t>(a.max_pages) * a.page_size + SIMT_KEYS - 1) / SIMT_KEYS;
    const double t = static_cast<double>(a.B) * a.items * cap;
    return t < most ? static_cast<int64_t>(t) : most;
}

template <typename E>
static dflash2_status launch_simt(AttnArgs a, cudaStream_t s) {
    void *fn = reinterpret_cast<void *>(&k_attn_simt<E>);
    a.tile_log2 = SIMT_KEYS_LOG2;
    a.tok_block = SIMT_ROWS / a.group > 0 ? SIMT_ROWS / a.group : 1;
    if (a.tok_block > a.T) a.tok_block = a.T;
    a.row_blocks = (a.T + a.tok_block - 1) / a.tok_block;
    a.rows_cap = a.tok_block * a.group;
    a.items = a.Hkv * a.row_blocks;
    return launch_simple(fn, a, SIMT_THREADS, simt_smem(a.d), simt_grid(a, fn), s);
}

template <typename E>
static dflash2_status launch_weights_simt(AttnArgs a, cudaStream_t s) {
    void *fn = reinterpret_cast<void *>(&k_weights_simt<E>);
    a.tile_log2 = SIMT_KEYS_LOG2;
    a.items = a.Hkv;
    return launch_simple(fn, a, SIMT_THREADS, simt_smem(a.d), simt_grid(a, fn), s);
}

// Rows of one part in the workspace, for either kind of kernel.
static int part_rows(int32_t T, int32_t group) {
    const int64_t rows = static_cast<int64_t>(T) * group;
    return rows < 128 ? static_cast<int>(rows) : 128;
}

bool kv_cache_ok(const dflash2_kv_cache *c, const int32_t *table, int32_t max_pages) {
    if (!c || !c->k || !c->v || !table || !dtype_ok(c->dt)) return false;
    const int e = esize(c->dt);
    auto al4 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; };
    return c->num_pages >= 1 && c->Hkv >= 1 && c->page_size >= 1 && c->d >= 1 && max_pages >= 1 && aligned16(c->k) &&
           aligned16(c->v) && c->page_stride * e % 16 == 0 && c->head_stride * e % 16 == 0 &&
           c->slot_stride * e % 16 == 0 && static_cast<int64_t>(c->d) * e % 16 == 0 && c->slot_stride >= c->d &&
           c->head_stride >= 0 && c->page_stride >= 0 && al4(c->weight) && al4(c->pos) && al4(table);
}

}  // namespace dfl

using namespace dfl;

extern "C" size_t dflash2_paged_attn_workspace_bytes(int64_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t d,
                                                     dflash2_dtype dt) {
    if (B < 0 || T < 0 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || d < 1 || !dtype_ok(dt)) return 0;
    return ATTN_TICKET_BYTES +
           static_cast<size_t>(attn_ctas()) * 2 * attn_part_floats(part_rows(T, Hq / Hkv), d) * sizeof(float);
}

extern "C" dflash2_status dflash2_paged_attn(const dflash2_kv_cache *cache, const int32_t *page_table,
                                             int32_t max_pages, const int32_t *kv_len, const int32_t *q_len,
                                             const int32_t *seq_pos, const void *q, int64_t B, int32_t T, int32_t Hq,
                                             float scale, int32_t window, uint32_t flags, void *out, float *lse,
                                             void *ws, size_t ws_bytes, dflash2_stream stream) {
    if (!kv_cache_ok(cache, page_table, max_pages) || B < 0 || T < 0 || Hq < 1 || Hq % cache->Hkv != 0 ||
        !(scale - scale == 0.f) || window < 0 || (flags & ~3u))
        return DFLASH2_ERR_INVALID_ARG;
    const bool weights = (flags & DFLASH2_ATTN_WEIGHTS) != 0;
    if (weights && (!lse || !cache->weight)) return DFLASH2_ERR_INVALID_ARG;
    if (B == 0 || T == 0) return DFLASH2_OK;
    auto al4 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; };
    if (!q || !out || !kv_len || !ws || !aligned16(q) || !aligned16(out) || !aligned16(ws) || !al4(kv_len) ||
        !al4(q_len) || !al4(seq_pos) || !al4(lse))
        return DFLASH2_ERR_INVALID_ARG;
    const int group = Hq / cache->Hkv;
    if (cache->d > 256 || group > 128 || cache->num_pages >= (int64_t(1) << 31) ||
        static_cast<int64_t>(max_pages) * cache->page_size >= (int64_t(1) << 31) - 256)
        return DFLASH2_ERR_UNSUPPORTED;
    // the places of a call's line are counted in 31 bits (32 keys and one token at the least)
    if (static_cast<double>(B) * cache->Hkv * T * (static_cast<double>(max_pages) * cache->page_size / SIMT_KEYS + 4) >=
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
    a.parts = reinterpret_cast<float *>(static_cast<char *>(ws) + ATTN_TICKET_BYTES);
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
