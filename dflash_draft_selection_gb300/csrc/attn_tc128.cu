// attn_tc128.cu -- the tensor-core paged attention for head dimension 128 (a
// translation unit of its own, so that the dimensions compile in parallel).
#include "attn_tc.cuh"

namespace dfl {
dflash2_status attn_tc128(TcLaunch &t) { return tc_launch<2>(t); }
}  // namespace dfl
