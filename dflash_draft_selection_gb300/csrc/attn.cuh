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
    int tile;        // keys per tile
    int tok_block;   // tokens of a row block (tok_block * group rows)
    int row_blocks;  // row blocks per request
    int items;       // items per request: Hkv * row_blocks (weights pass: Hkv)
    int rows_cap;    // rows of a part in the workspace
    int *tickets;    // [gridDim.x], zero between calls
    float *parts;    // [2 * gridDim.x][attn_part_floats(rows_cap, d)]
};

// Floats of a part: O [rows][d], m [rows], l [rows], padded to 16 bytes.
__host__ __device__ __forceinline__ int64_t attn_part_floats(int rows, int d) {
    return (static_cast<int64_t>(rows) * (d + 2) + 3) / 4 * 4;
}

constexpr int ATTN_MAX_CTAS = 1024;
constexpr size_t ATTN_TICKET_BYTES = ATTN_MAX_CTAS * sizeof(int);

// One request as the call sees it.
struct AttnReq {
    int n;        // slots that may be seen
    int nq;       // tokens
    int64_t q0;   // position of token 0
    int first;    // first tile some token may see
    int nt;       // tiles from there (at least one: its rows are written even if nothing is seen)
};

__device__ __forceinline__ AttnReq attn_req(const AttnArgs &a, int64_t b) {
    AttnReq r;
    const int64_t cap = static_cast<int64_t>(a.max_pages) * a.page_size;
    int64_t n = a.kv_len[b];
    n = n < 0 ? 0 : (n > cap ? cap : n);
    int nq = a.q_len ? a.q_len[b] : a.T;
    nq = nq < 0 ? 0 : (nq > a.T ? a.T : nq);
    r.nq = nq;
    r.q0 = a.seq_pos ? a.seq_pos[b] : n - nq;
    int64_t lo = 0;
    if (!a.pos) {  // slot = position: the slots outside every token's view are not visited
        if (a.causal) n = min(n, max(r.q0 + nq, static_cast<int64_t>(0)));
        if (a.window > 0) lo = max(r.q0 - a.window + 1, static_cast<int64_t>(0));
    }
    if (nq == 0) n = 0;
    r.n = static_cast<int>(n);
    const int last = static_cast<int>((n + a.tile - 1) / a.tile);
    r.first = static_cast<int>(min(lo / a.tile, static_cast<int64_t>(last > 0 ? last - 1 : 0)));
    r.nt = last > r.first ? last - r.first : 1;
    return r;
}

// This CTA's stretch [begin, end) of the line and the request that holds its
// start (`base`: the line's tiles before that request).  All threads call it.
struct AttnPlan {
    int64_t total, begin, end, base, b;
    int ctas;  // the CTAs that have a stretch: no more than there are tiles, so that no stretch is empty
};

__device__ __forceinline__ int64_t attn_begin(int64_t total, int cta, int ctas) { return total * cta / ctas; }
// The CTA whose stretch holds tile x.
__device__ __forceinline__ int attn_owner(int64_t total, int64_t x, int ctas) {
    return static_cast<int>(((x + 1) * ctas - 1) / total);
}

template <int THREADS>
__device__ __forceinline__ AttnPlan attn_plan(const AttnArgs &a, int64_t *scratch /* [THREADS / 32 + 2] */) {
    constexpr int W = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    AttnPlan p;
    int64_t sum = 0, mine = 0;
    for (int64_t b = tid; b < a.B; b += THREADS) {
        mine = static_cast<int64_t>(attn_req(a, b).nt) * a.items;
        sum += mine;
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(FULL, sum, d);
    if (lane == 0) scratch[warp] = sum;
    __syncthreads();
    p.total = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) p.total += scratch[w];
    __syncthreads();
    p.ctas = static_cast<int>(min(p.total, static_cast<int64_t>(gridDim.x)));
    p.b = 0;
    p.base = 0;
    p.begin = p.end = 0;
    if (blockIdx.x >= p.ctas) return p;
    p.begin = attn_begin(p.total, blockIdx.x, p.ctas);
    p.end = attn_begin(p.total, blockIdx.x + 1, p.ctas);
    // find the request that holds `begin`
    int64_t carry = 0;
    for (int64_t at = 0; at < a.B; at += THREADS) {
        const int64_t b = at + tid;
        const int64_t v = b < a.B ? (a.B <= THREADS ? mine : static_cast<int64_t>(attn_req(a, b).nt) * a.items) : 0;
        int64_t inc = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(FULL, inc, d);
            if (lane >= d) inc += o;
        }
        if (lane == 31) scratch[warp] = inc;
        __syncthreads();
        int64_t before = carry;
        for (int w = 0; w < warp; ++w) before += scratch[w];
        int64_t all = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) all += scratch[w];
        const int64_t lo = before + inc - v;
        __syncthreads();
        if (v > 0 && lo <= p.begin && p.begin < lo + v) {
            scratch[W] = b;
            scratch[W + 1] = lo;
        }
        const bool here = p.begin < carry + all;
        carry += all;
        if (here) break;
    }
    __syncthreads();
    p.b = scratch[W];
    p.base = scratch[W + 1];
    return p;
}

// Walks the items of a stretch.
struct AttnWalk {
    AttnReq r;
    int64_t b, base, at, end, total;
    int ctas;
    int item;     // within the request
    int t0, t1;   // this stretch's tiles of the item (absolute: the first key is t0 * tile)
    bool whole;   // the stretch holds all of the item's tiles
    bool starts;  // ... or its first ones

    __device__ __forceinline__ void start(const AttnArgs &a, const AttnPlan &p) {
        b = p.b;
        base = p.base;
        at = p.begin;
        end = p.end;
        total = p.total;
        ctas = p.ctas;
        r = attn_req(a, b);
    }
    // The next item; false at the end of the stretch.
    __device__ __forceinline__ bool next(const AttnArgs &a) {
        if (at >= end) return false;
        while (at >= base + static_cast<int64_t>(r.nt) * a.items) {
            base += static_cast<int64_t>(r.nt) * a.items;
            ++b;
            r = attn_req(a, b);
        }
        item = static_cast<int>((at - base) / r.nt);
        const int64_t first = base + static_cast<int64_t>(item) * r.nt;
        const int64_t last = min(first + r.nt, end);
        t0 = r.first + static_cast<int>(at - first);
        t1 = r.first + static_cast<int>(last - first);
        starts = at == first;
        whole = starts && last == first + r.nt;
        at = last;
        return true;
    }
    __device__ __forceinline__ int64_t item_base() const { return base + static_cast<int64_t>(item) * r.nt; }
};

// The page of a slot, or -1.
__device__ __forceinline__ int attn_page(const AttnArgs &a, int64_t b, int slot) {
    const int page = a.table[b * a.max_pages + slot / a.page_size];
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
__device__ __forceinline__ void attn_view_slot(const AttnArgs &a, const AttnReq &r, int64_t b, int h, int s, int &lo,
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
__device__ __forceinline__ int64_t attn_row(const AttnArgs &a, int64_t b, int h, int tok0, int r) {
    return (b * a.T + tok0 + r / a.group) * a.Hq + static_cast<int64_t>(h) * a.group + r % a.group;
}

__device__ __forceinline__ void attn_store(const AttnArgs &a, int64_t i, float v, float *) {
    static_cast<float *>(a.out)[i] = v;
}
__device__ __forceinline__ void attn_store(const AttnArgs &a, int64_t i, float v, unsigned short *) {
    unsigned short o;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(o) : "f"(v));
    static_cast<unsigned short *>(a.out)[i] = o;
}

__device__ __forceinline__ float *attn_part(const AttnArgs &a, int cta, bool starts) {
    return a.parts + (static_cast<int64_t>(cta) * 2 + (starts ? 1 : 0)) * attn_part_floats(a.rows_cap, a.d);
}

// After this CTA's part of a cut item is written: take the item's ticket, and
// if every other part is there, join them (all threads call it; E is the
// output's element type).  Part layout: O [rows][d], m [rows], l [rows], m in
// units of log2.
constexpr int JOIN_BATCH = 8;
template <typename E, typename Sync>
__device__ __forceinline__ void attn_join(const AttnArgs &a, const AttnWalk &w, int rows, int h, int tok0, int nthreads,
                                          int tid, int *flag /* shared */, Sync sync) {
    const int64_t first = w.item_base();
    const int c0 = attn_owner(w.total, first, w.ctas);
    const int c1 = attn_owner(w.total, first + w.r.nt - 1, w.ctas);
    __threadfence();
    sync();
    if (tid == 0) {
        const int old = atomic_add_acq_rel(&a.tickets[c0], 1);
        *flag = old == c1 - c0;
        if (old == c1 - c0) a.tickets[c0] = 0;
    }
    sync();
    const bool last = *flag != 0;
    if (!last) return;
    __threadfence();
    const int64_t step = attn_part_floats(a.rows_cap, a.d);
    const int real = min(rows, max(w.r.nq - tok0, 0) * a.group);
    // the parts in order: c0's second slot, then the first slots of c0 + 1 .. c1
    auto part = [&](int c) { return a.parts + (static_cast<int64_t>(c) * 2 + (c == c0 ? 1 : 0)) * step; };
    const int d4 = a.d / 4;
    for (int i = tid; i < rows * d4; i += nthreads) {
        const int r = i / d4, c4 = i % d4;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float M = NEG_INF, L = 0.f;
        if (r < real) {
            for (int c = c0; c <= c1; c += JOIN_BATCH) {  // a batch's loads are in flight together
                float m[JOIN_BATCH], l[JOIN_BATCH];
                float4 x[JOIN_BATCH];
#pragma unroll
                for (int k = 0; k < JOIN_BATCH; ++k) {
                    const float *p = part(min(c + k, c1));
                    m[k] = __ldcg(p + a.rows_cap * a.d + r);
                    l[k] = c + k <= c1 ? __ldcg(p + a.rows_cap * (a.d + 1) + r) : 0.f;
                    x[k] = __ldcg(reinterpret_cast<const float4 *>(p + static_cast<int64_t>(r) * a.d) + c4);
                }
#pragma unroll
                for (int k = 0; k < JOIN_BATCH; ++k) {
                    if (l[k] == 0.f) continue;  // the part saw nothing (a NaN sum is taken along)
                    const float nm = fmax_nan(M, m[k]);
                    const float wo = M == NEG_INF ? 0.f : ex2(M - nm), wn = ex2(m[k] - nm);
                    o.x = o.x * wo + x[k].x * wn;
                    o.y = o.y * wo + x[k].y * wn;
                    o.z = o.z * wo + x[k].z * wn;
                    o.w = o.w * wo + x[k].w * wn;
                    L = L * wo + l[k] * wn;
                    M = nm;
                }
            }
        }
        const float inv = L == 0.f ? 0.f : 1.0f / L;
        const int64_t row = attn_row(a, w.b, h, tok0, r);
        const int64_t at = row * a.d + c4 * 4;
        attn_store(a, at, o.x * inv, static_cast<E *>(nullptr));
        attn_store(a, at + 1, o.y * inv, static_cast<E *>(nullptr));
        attn_store(a, at + 2, o.z * inv, static_cast<E *>(nullptr));
        attn_store(a, at + 3, o.w * inv, static_cast<E *>(nullptr));
        if (c4 == 0 && a.lse) a.lse[row] = L == 0.f ? NEG_INF : (M + log2f(L)) * 0.6931471805599453f;
    }
}


}  // namespace dfl
