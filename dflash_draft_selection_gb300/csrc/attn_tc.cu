// attn_tc.cu -- the host side of the tensor-core paged attention: which calls
// it takes, the cut of the rows, tensor maps, and the kernels' error word.
#include "attn_tc.cuh"

namespace dfl {

static __device__ unsigned int g_err_attn;

dflash2_status attn_tc64(TcLaunch &t);
dflash2_status attn_tc128(TcLaunch &t);
dflash2_status attn_tc256(TcLaunch &t);

unsigned int read_error_attn(bool clear) {
    unsigned int v = 0;
    cudaMemcpyFromSymbol(&v, g_err_attn, sizeof v);
    if (clear) {
        const unsigned int z = 0;
        cudaMemcpyToSymbol(g_err_attn, &z, sizeof z);
    }
    return v;
}

// The error word's address on the current device, looked up once.
static unsigned int *err_word() {
    static unsigned int *cache[64] = {nullptr};
    const int dev = current_device();
    if (dev >= 0 && dev < 64 && cache[dev]) return cache[dev];
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_err_attn) != cudaSuccess) return nullptr;
    if (dev >= 0 && dev < 64) cache[dev] = static_cast<unsigned int *>(p);
    return static_cast<unsigned int *>(p);
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
// (one swizzle pattern), strides that a tensor map can hold, and a block's
// outputs within 2^31 elements of its first row's.
bool attn_tc_takes(const AttnArgs &a) {
    const int64_t lim = int64_t(1) << 38;
    return (a.d == 64 || a.d == 128 || a.d == 256) && a.page_size % 8 == 0 &&
           (a.Hkv == 1 || (a.head_stride > 0 && a.head_stride < lim)) &&
           (a.num_pages == 1 || (a.page_stride > 0 && a.page_stride < lim)) &&
           a.slot_stride * a.page_size < lim / a.Hkv && static_cast<int64_t>(a.T) * a.Hq * a.d < lim &&
           static_cast<int64_t>(a.T < TK ? a.T : TK) * a.Hq * a.d < (int64_t(1) << 31);
}

dflash2_status attn_tc_launch(AttnArgs a, bool weights, cudaStream_t s) {
    TcLaunch t;
    a.tile_log2 = 7;
    const int most = TK / a.group;                            // tokens that fit a block
    const int blocks = (a.T + most - 1) / most;
    a.tok_block = (a.T + blocks - 1) / blocks;                // blocks of like size
    a.row_blocks = (a.T + a.tok_block - 1) / a.tok_block;
    a.rows_cap = a.tok_block * a.group;
    a.items = a.Hkv * a.row_blocks;
    a.item_cost = ATTN_ITEM_COST;
    a.err = err_word();
    if (!a.err) return DFLASH2_ERR_CUDA;
    const unsigned int *hold;
    scan_hold(&hold, &a.hold_cycles);
    t.n = a.rows_cap <= 16 ? 16 : a.rows_cap <= 32 ? 32 : a.rows_cap <= 48 ? 48 : a.rows_cap <= 64 ? 64
          : a.rows_cap <= 96 ? 96 : 128;
    t.box_log2 = 3;
    while (t.box_log2 < 7 && a.page_size % (2 << t.box_log2) == 0) ++t.box_log2;

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
    if (!make_map_4d(&t.mk, a.k, cd, cs, 1u << t.box_log2, 1) || !make_map_4d(&t.mv, a.v, cd, cs, 1u << t.box_log2, 1) ||
        !make_map_4d(&t.mq, a.q, qd, qs, a.group, a.tok_block))
        return DFLASH2_ERR_CUDA;
    const double cap = static_cast<double>((static_cast<int64_t>(a.max_pages) * a.page_size + TK - 1) / TK);
    auto launch = [&](bool second) {
        const double tiles = static_cast<double>(a.B) * a.items * cap;
        t.ctas = tiles < sm_count() ? static_cast<int64_t>(tiles) : sm_count();
        a.hold = second == weights ? hold : nullptr;  // the call's last launch
        t.a = a;
        t.weights = second;
        return a.d == 64 ? attn_tc64(t) : a.d == 128 ? attn_tc128(t) : attn_tc256(t);
    };
    t.stream = s;
    const dflash2_status st = launch(false);
    if (st != DFLASH2_OK || !weights) return st;
    a.items = a.Hkv;
    a.item_cost = 1;
    return launch(true);
}

}  // namespace dfl
