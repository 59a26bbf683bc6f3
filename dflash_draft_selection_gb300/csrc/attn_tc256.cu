// attn_tc256.cu -- the tensor-core paged attention for head dimension 256 (a
// translation unit of its own, so that the dimensions compile in parallel).
#include "attn_tc.cuh"

namespace dfl {
dflash2_status attn_tc256(TcLaunch &t) { return tc_launch<4>(t); }
}  // namespace dfl
