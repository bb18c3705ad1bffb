// Attention over the microscaled paged cache for drafts, heads of 128 channels:
// the kernels of mx_attn.h with masks.  Only tiles that reach into a draft, its
// last few, look at them; everything before is the same work.  (Heads of 64
// channels are compiled in a file of their own, beside this one.)
#include "mx_attn.h"

namespace kvtc {

hipError_t launch_mx_attn_tree(const MxAttnParams* prefix, const MxAttnParams* own, int D, int bk, int bv, bool f32,
                               hipStream_t s) {
  return D == 128 ? launch_any<128, true>(prefix, own, bk, bv, f32, s)
                  : launch_mx_attn_tree64(prefix, own, bk, bv, f32, s);
}

}  // namespace kvtc
