// attn.cuh -- what the paged-attention kernels share: arguments, the split of
// the work over the CTAs, which rows see a key, and the join of parts.
//
// The work of a call is a line of key tiles: request by request, cached head
// by cached head, row block by row block, the tiles of the slots that some
// token of the request may see.  Lengths are known on the device only, so
// every CTA sums the requests' tile counts itself (one pass over kv_len) and
// takes an equal stretch of the line, whatever the lengths are.  A stretch
// covers whole items (request, head, row block) and at most one cut item at
// either end.  A cut item's parts (unnormalised output, running maximum, sum)
// go to the workspace; the CTA that finishes its part last adds them up in
// the order of the stretches, so the result does not depend on who is last.
// No CTA waits for another one.
#pragma once

#include "common.cuh"
#include "host.hpp"

namespace dfl {

struct AttnArgs {
    const char *k, *v;
    float *weight;
    const int32_t *pos;
    int64_t num_pages, page_stride, head_stride, slot_stride;  // strides in elements
    int Hkv, page_size, d;
    const int32_t *table;
    int max_pages;
    const int32_t *kv_len, *q_len, *seq_pos;
    const void *q;
    int64_t B;
    int T, Hq, group;
    float scale;
    int window, causal;
    void *out;
    float *lse;
    int tile_log2;   // keys per tile
    int tok_block;   // tokens of a row block (tok_block * group rows)
    int row_blocks;  // row blocks per request
    int items;       // items per request: Hkv * row_blocks (weights pass: Hkv)
    int item_cost;   // what an item costs beside its tiles, in tiles
    int rows_cap;    // rows of a part in the workspace
    int *tickets;    // [gridDim.x], zero between calls
    float *parts;    // [2 * gridDim.x][attn_part_floats(rows_cap, d)]
    unsigned int *err;  // the library's error word of these kernels
    const unsigned int *hold;  // test hook: NULL, or a word that a copying warp of the tensor-core kernels waits on
    long long hold_cycles;
};

// Floats of a part: O [rows][d], m [rows], l [rows], padded to 16 bytes.
__host__ __device__ __forceinline__ int64_t attn_part_floats(int rows, int d) {
    return (static_cast<int64_t>(rows) * (d + 2) + 3) / 4 * 4;
}

constexpr int ATTN_MAX_CTAS = 1024;
constexpr size_t ATTN_TICKET_BYTES = ATTN_MAX_CTAS * sizeof(int);
static_assert(ATTN_TICKET_BYTES <= WS_ZERO_BYTES, "the tickets lie in what other calls leave alone");

// What an item of the tensor-core kernels costs beside its tiles, in tiles:
// the drain of the pipeline, its sums and outputs, the join of a cut one, the
// first tile's maxima.  Measured with 1, 2, 3, 4, 6, 8: 64 requests in a window
// 78, 71, 70, 66, 70, 68 us; 32 ragged ones 207, 194, 188, 185, 184, 187; 16
// with wide heads 136, 139, 123, 121, 118, 116.
constexpr int ATTN_ITEM_COST = 4;

// One request as the call sees it.  (Slots, and the tiles of a call, are
// below 2^31: checked by the caller.)
struct AttnReq {
    int n;        // slots that may be seen
    int nq;       // tokens
    int64_t q0;   // position of token 0
    int first;    // first tile some token may see
    int nt;       // tiles from there (at least one: its rows are written even if nothing is seen)
};

// What the call's arrays say of a request (0 past the last one).
struct AttnRaw {
    int n, nq, sp;
};
__device__ __forceinline__ AttnRaw attn_raw(const AttnArgs &a, int b) {
    AttnRaw x = {0, 0, 0};
    if (b < a.B) {
        x.n = a.kv_len[b];
        x.nq = a.q_len ? a.q_len[b] : a.T;
        x.sp = a.seq_pos ? a.seq_pos[b] : 0;
    }
    return x;
}
__device__ __forceinline__ AttnReq attn_req(const AttnArgs &a, const AttnRaw &x) {
    AttnReq r;
    int n = x.n, nq = x.nq;
    const int sp = x.sp;
    n = min(max(n, 0), a.max_pages * a.page_size);
    nq = min(max(nq, 0), a.T);
    r.nq = nq;
    r.q0 = a.seq_pos ? sp : n - nq;
    int lo = 0;
    if (!a.pos) {  // slot = position: the slots outside every token's view are not visited
        if (a.causal) n = static_cast<int>(min(static_cast<int64_t>(n), max(r.q0 + nq, static_cast<int64_t>(0))));
        if (a.window > 0)
            lo = static_cast<int>(min(static_cast<int64_t>(n), max(r.q0 - a.window + 1, static_cast<int64_t>(0))));
    }
    if (nq == 0) n = 0;
    r.n = n;
    const int last = (n + (1 << a.tile_log2) - 1) >> a.tile_log2;
    r.first = min(lo >> a.tile_log2, max(last - 1, 0));
    r.nt = max(last - r.first, 1);
    return r;
}
__device__ __forceinline__ AttnReq attn_req(const AttnArgs &a, int b) { return attn_req(a, attn_raw(a, b)); }

// This CTA's stretch [begin, end) of the line and the request that holds its
// start (`base`: the line's places before that request).
struct AttnPlan {
    int total, begin, end, base, b;
    int ctas;   // the CTAs that have a stretch: no more than there are places, so that no stretch is empty
    int q, rem; // places of a stretch: q, and one more in the first rem
    int cost;   // an item's places beside its tiles
    __device__ __forceinline__ int at(int cta) const { return q * cta + min(cta, rem); }
    // The CTA whose stretch holds place x.
    __device__ __forceinline__ int owner(int x) const {
        const int cut = rem * (q + 1);
        return x < cut ? x / (q + 1) : rem + (x - cut) / q;
    }
};

// All threads call it.
template <int THREADS>
__device__ __forceinline__ AttnPlan attn_plan(const AttnArgs &a, int *scratch /* [THREADS / 32 + 2] */) {
    constexpr int W = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int B = static_cast<int>(a.B);
    AttnPlan p;
    int sum = 0, mine = 0;
    for (int b = tid; b < B; b += THREADS) {
        mine = attn_req(a, b).nt * a.items;
        sum += mine;
    }
    if (B == 1) {  // the only request's tiles, known to thread 0
        if (tid == 0) scratch[0] = mine;
        __syncthreads();
        p.total = scratch[0];
    } else {
        sum = __reduce_add_sync(FULL, sum);
        if (lane == 0) scratch[warp] = sum;
        __syncthreads();
        p.total = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) p.total += scratch[w];
    }
    // where every tile has a CTA of its own there is nothing to balance
    p.cost = p.total <= static_cast<int>(gridDim.x) ? 0 : a.item_cost;
    p.total += B * a.items * p.cost;
    p.ctas = min(p.total, static_cast<int>(gridDim.x));
    p.q = p.total / p.ctas;
    p.rem = p.total - p.q * p.ctas;
    p.b = 0;
    p.base = 0;
    p.begin = p.end = 0;
    if (static_cast<int>(blockIdx.x) >= p.ctas) return p;
    p.begin = p.at(blockIdx.x);
    p.end = p.at(blockIdx.x + 1);
    if (B == 1) return p;
    // find the request that holds `begin`
    __syncthreads();
    int carry = 0;
    for (int at = 0; at < B; at += THREADS) {
        const int b = at + tid;
        const int v = b < B ? (B <= THREADS ? mine : attn_req(a, b).nt * a.items) + p.cost * a.items : 0;
        int inc = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(FULL, inc, d);
            if (lane >= d) inc += o;
        }
        if (lane == 31) scratch[warp] = inc;
        __syncthreads();
        int before = carry, all = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const int x = scratch[w];
            if (w < warp) before += x;
            all += x;
        }
        const int lo = before + inc - v;
        if (v > 0 && lo <= p.begin && p.begin - lo < v) {
            scratch[W] = b;
            scratch[W + 1] = lo;
        }
        const bool here = p.begin - carry < all;
        carry += all;
        __syncthreads();
        if (here) break;
    }
    p.b = scratch[W];
    p.base = scratch[W + 1];
    return p;
}

// Walks the items of a stretch.
struct AttnWalk {
    AttnReq r;
    AttnRaw ahead;  // of request b + 1: read before it is needed
    int b, base, at, end, cost;
    int item;     // within the request
    int t0, t1;   // this stretch's tiles of the item (absolute: the first key is t0 * tile)
    bool whole;   // the stretch holds all of the item's tiles
    bool starts;  // ... or its first ones

    __device__ __forceinline__ void start(const AttnArgs &a, const AttnPlan &p) {
        b = p.b;
        base = p.base;
        at = p.begin;
        end = p.end;
        cost = p.cost;
        r = attn_req(a, b);
        ahead = attn_raw(a, b + 1);
    }
    // The next item that has tiles here; false at the end of the stretch.
    __device__ __forceinline__ bool next(const AttnArgs &a) {
        while (at < end) {
            int len = r.nt + cost;
            while (at - base >= len * a.items) {
                base += len * a.items;
                ++b;
                r = attn_req(a, ahead);
                ahead = attn_raw(a, b + 1);
                len = r.nt + cost;
            }
            item = (at - base) / len;
            const int first = base + item * len, from = at - first - cost;  // in tiles of the item
            const int last = min(len, end - first), to = last - cost;
            at = first + last;
            t0 = r.first + max(from, 0);
            t1 = r.first + to;
            starts = from <= 0;
            whole = starts && to == r.nt;
            if (t0 < t1) return true;
        }
        return false;
    }
    // The place of the item's first tile.
    __device__ __forceinline__ int item_base() const {
        return base + item * (r.nt + cost) + cost;
    }
};

// The page of a slot, or -1.
__device__ __forceinline__ int attn_page(const AttnArgs &a, int b, int slot) {
    const int page = a.table[static_cast<int64_t>(b) * a.max_pages + slot / a.page_size];
    return static_cast<unsigned>(page) < static_cast<unsigned long long>(a.num_pages) ? page : -1;
}

// The tokens [lo, hi) of 0 .. nq - 1 that see a key at position P.
__device__ __forceinline__ void attn_view(const AttnArgs &a, const AttnReq &r, int64_t P, int &lo, int &hi) {
    const int64_t rel = P - r.q0;
    int64_t l = 0, h = r.nq;
    if (a.causal && rel > l) l = rel;
    if (a.window > 0 && rel + a.window < h) h = rel + a.window;
    lo = static_cast<int>(min(l, static_cast<int64_t>(r.nq)));
    hi = static_cast<int>(max(h, static_cast<int64_t>(lo)));
}

// ... for slot s of the request in cached head h (nothing is seen of a slot
// past the request's or without a page).
__device__ __forceinline__ void attn_view_slot(const AttnArgs &a, const AttnReq &r, int b, int h, int s, int &lo,
                                               int &hi, int &page) {
    lo = hi = 0;
    page = -1;
    if (s >= r.n) return;
    page = attn_page(a, b, s);
    if (page < 0) return;
    int64_t P = s;
    if (a.pos) P = a.pos[(static_cast<int64_t>(page) * a.Hkv + h) * a.page_size + s % a.page_size];
    attn_view(a, r, P, lo, hi);
}

// Query row r of a row block: token tok0 + r / group, head h * group + r % group.
__device__ __forceinline__ int64_t attn_row(const AttnArgs &a, int b, int h, int tok0, int r) {
    return (static_cast<int64_t>(b) * a.T + tok0 + r / a.group) * a.Hq + static_cast<int64_t>(h) * a.group + r % a.group;
}


__device__ __forceinline__ void attn_store4(const AttnArgs &a, int64_t i, float x, float y, float z, float w, float *) {
    *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + i) = make_float4(x, y, z, w);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void attn_store4(const AttnArgs &a, int64_t i, float x, float y, float z, float w,
                                            unsigned short *) {
    *reinterpret_cast<uint2 *>(static_cast<unsigned short *>(a.out) + i) = make_uint2(pack_bf16(x, y), pack_bf16(z, w));
}

// The largest of the warp's values (NaN only if all are).
__device__ __forceinline__ float warp_max_one(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float *attn_part(const AttnArgs &a, int cta, bool starts) {
    return a.parts + (static_cast<int64_t>(cta) * 2 + (starts ? 1 : 0)) * attn_part_floats(a.rows_cap, a.d);
}

// The parts of a cut item: n of them, the first from CTA c0; part k's place in
// the workspace (c0's second slot, then the first slots of c0 + 1 ..).
struct AttnParts {
    int c0, n;
    int64_t step;
    const float *base;
    __device__ __forceinline__ AttnParts(const AttnArgs &a, const AttnPlan &p, const AttnWalk &w) {
        const int first = w.item_base();
        c0 = p.owner(first);
        n = p.owner(first + w.r.nt - 1) - c0 + 1;
        step = attn_part_floats(a.rows_cap, a.d);
        base = a.parts + (static_cast<int64_t>(c0) * 2 + 1) * step;
    }
    __device__ __forceinline__ const float *at(int k) const { return base + (k == 0 ? 0 : 2 * k - 1) * step; }
};

// A row's weights over n parts with (m_k, l_k): f_k = 2^(m_k - M), 0 for a part
// that saw nothing, written over m; 1 / sum l_k f_k is returned (0 for a row
// that saw nothing) and the row's lse.  Sums over parts run in their order, so
// the result is the same whoever takes them.
__device__ __forceinline__ float attn_join_row(int n, float *m, const float *l, float *lse) {
    float M = NEG_INF, L = 0.f;
    for (int k = 0; k < n; ++k) M = fmax_nan(M, m[k]);
    for (int k = 0; k < n; ++k) {
        const float lk = l[k];
        const float f = lk == 0.f ? 0.f : ex2(m[k] - M);  // a sum that is NaN is taken along
        L = fmaf(lk, f, L);
        m[k] = f;
    }
    *lse = L == 0.f ? NEG_INF : (M + log2f(L)) * 0.6931471805599453f;
    return L == 0.f ? 0.f : 1.0f / L;
}

// The join's sum over the parts: U vectors of four entries per thread and K
// parts at a time, all their loads in flight together (other CTAs keep the
// memory busy: a load's latency is what a join costs).  D: the head dimension
// (0: a.d).
template <typename E, int D, int U, int K, typename Weight>
__device__ __forceinline__ void attn_join_sum(const AttnArgs &a, const AttnParts &q, int rows, Weight weight,
                                              const float *inv, int64_t first_row, const int *row_at, int threads,
                                              int tid) {
    const int d = D ? D : a.d, d4 = d / 4, total = rows * d4;
#pragma unroll 1
    for (int i0 = tid; i0 < total; i0 += U * threads) {
        float4 o[U];
        int r[U], at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = min(i0 + u * threads, total - 1);
            r[u] = i / d4;
            at[u] = i * 4;
            o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll 1
        for (int k0 = 0; k0 < q.n; k0 += K) {
            float4 x[U * K];
#pragma unroll
            for (int v = 0; v < U * K; ++v)
                x[v] = __ldcg(reinterpret_cast<const float4 *>(q.at(min(k0 + v / U, q.n - 1)) + at[v % U]));
#pragma unroll
            for (int v = 0; v < U * K; ++v) {
                const int u = v % U, k = k0 + v / U;
                const float f = k < q.n ? weight(r[u], k) : 0.f;
                if (f == 0.f) continue;
                o[u].x = fmaf(x[v].x, f, o[u].x);
                o[u].y = fmaf(x[v].y, f, o[u].y);
                o[u].z = fmaf(x[v].z, f, o[u].z);
                o[u].w = fmaf(x[v].w, f, o[u].w);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * threads < total) {
                const float g = inv[r[u]];
                attn_store4(a, (first_row + row_at[r[u]]) * d + (at[u] - r[u] * d), g == 0.f ? 0.f : o[u].x * g,
                            g == 0.f ? 0.f : o[u].y * g, g == 0.f ? 0.f : o[u].z * g, g == 0.f ? 0.f : o[u].w * g,
                            static_cast<E *>(nullptr));
            }
    }
}

// After this CTA's part of a cut item is written: take the item's ticket, and
// if every other part is there, join them (all `threads` threads call it; E is
// the output's element type, D the head dimension or 0).  `scratch`
// (`cap` floats) holds the rows' m and l; where they do not fit (very many
// parts of many rows) the weights go over the m of the parts, which nobody
// else reads any more.  first_row + row_at: the rows' indexes in lse.
template <typename E, int D, typename Sync>
__device__ __forceinline__ void attn_join(const AttnArgs &a, const AttnParts &q, const AttnWalk &w, int rows, int tok0,
                                          int threads, int tid, int *flag /* shared */, float *scratch, int cap,
                                          float *inv /* shared, [rows] */, int64_t first_row,
                                          const int *row_at /* shared */,
                                          Sync sync) {
    __threadfence();
    sync();
    if (tid == 0) {
        const int old = atomic_add_acq_rel(&a.tickets[q.c0], 1);
        *flag = old == q.n - 1;
        if (old == q.n - 1) a.tickets[q.c0] = 0;
    }
    sync();
    if (!*flag) return;
    __threadfence();
    const int real = min(rows, max(w.r.nq - tok0, 0) * a.group), all = rows * q.n;
    const int64_t om = static_cast<int64_t>(a.rows_cap) * a.d;
    if (2 * all > cap) {
        float lse;
        if (tid < rows) {
            float M = NEG_INF, L = 0.f;
            for (int k = 0; k < q.n; ++k) M = fmax_nan(M, __ldcg(q.at(k) + om + tid));
            for (int k = 0; k < q.n; ++k) {
                const float l = tid < real ? __ldcg(q.at(k) + om + a.rows_cap + tid) : 0.f;
                float *m = const_cast<float *>(q.at(k)) + om + tid;
                const float f = l == 0.f ? 0.f : ex2(__ldcg(m) - M);
                L = fmaf(l, f, L);
                __stcg(m, f);
            }
            lse = L == 0.f ? NEG_INF : (M + log2f(L)) * 0.6931471805599453f;
            inv[tid] = L == 0.f ? 0.f : 1.0f / L;
            if (a.lse) a.lse[first_row + row_at[tid]] = lse;
        }
        __threadfence();
        sync();
        attn_join_sum<E, D, 4, 4>(
            a, q, rows, [&](int r, int k) { return __ldcg(q.at(k) + om + r); }, inv, first_row, row_at, threads, tid);
        return;
    }
    float *m = scratch, *l = scratch + all;
#pragma unroll 4
    for (int i = tid; i < all; i += threads) {
        const int r = i / q.n;
        const float *x = q.at(i - r * q.n) + om + r;
        const float mk = __ldcg(x), lk = __ldcg(x + a.rows_cap);
        m[i] = mk;
        l[i] = r < real ? lk : 0.f;
    }
    sync();
    if (tid < rows) {
        float lse;
        inv[tid] = attn_join_row(q.n, m + tid * q.n, l + tid * q.n, &lse);
        if (a.lse) a.lse[first_row + row_at[tid]] = lse;
    }
    sync();
    auto weight = [&](int r, int k) { return m[r * q.n + k]; };
    if (rows * (a.d / 4) <= threads)
        attn_join_sum<E, D, 1, 16>(a, q, rows, weight, inv, first_row, row_at, threads, tid);
    else if (q.n > 2)
        attn_join_sum<E, D, 2, 8>(a, q, rows, weight, inv, first_row, row_at, threads, tid);
    else
        attn_join_sum<E, D, 8, 2>(a, q, rows, weight, inv, first_row, row_at, threads, tid);
}

}  // namespace dfl
