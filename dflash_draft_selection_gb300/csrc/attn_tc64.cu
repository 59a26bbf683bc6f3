// attn_tc64.cu -- the tensor-core paged attention for head dimension 64 (a
// translation unit of its own, so that the dimensions compile in parallel).
#include "attn_tc.cuh"

namespace dfl {
dflash2_status attn_tc64(TcLaunch &t) { return tc_launch<1>(t); }
}  // namespace dfl
