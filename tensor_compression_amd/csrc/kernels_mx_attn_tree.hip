// Attention over the microscaled paged cache for drafts: the kernels of
// mx_attn.h with masks.  Only tiles that reach into a draft, its last few,
// look at them; everything before is the same work.
#include "mx_attn.h"

namespace kvtc {

hipError_t launch_mx_attn_tree(const MxAttnParams* prefix, const MxAttnParams* own, int D, int bk, int bv, bool f32,
                               hipStream_t s) {
  return launch_any<true>(prefix, own, D, bk, bv, f32, s);
}

}  // namespace kvtc
