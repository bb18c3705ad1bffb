// Attention over the microscaled paged cache for drafts, heads of 64 channels.
#include "mx_attn.h"

namespace kvtc {

hipError_t launch_mx_attn_tree64(const MxAttnParams* prefix, const MxAttnParams* own, int bk, int bv, bool f32,
                                 hipStream_t s) {
  return launch_any<64, true>(prefix, own, bk, bv, f32, s);
}

}  // namespace kvtc
