// Shared declarations of the microscaled paged cache (kernels_mx.hip,
// kernels_mx_attn.hip, kvtc_api_mx.hip).
#pragma once

#include "kvtc_internal.h"

namespace kvtc {

// Record of one (page, head): key codes, value codes, key scales, value scales.
struct MxRecord {
  int32_t kc, vc, sc, bytes;
};
KVTC_HD constexpr MxRecord mx_record(int D, int bk, int bv) {
  return MxRecord{KVTC_MX_PAGE * D * bk / 8, KVTC_MX_PAGE * D * bv / 8, KVTC_MX_PAGE * D / 32,
                  KVTC_MX_PAGE * D * (bk + bv) / 8 + KVTC_MX_PAGE * D / 16};
}

// Rows of one write or read.
struct MxIoParams {
  kvtc_mx_batch b;
  int32_t H, n_units, pool_pages;
  int32_t n_layers;
  uint8_t* pool;        // record of (first layer, page 0, head 0)
  int64_t layer_bytes;  // pool bytes of a layer
  void* x[2];           // keys, values
  int64_t st[2][3];     // (layer, head, row) strides in elements
  uint32_t* status;
};

// One pass of the attention over the tokens [begin, end) of the sequences
// (or of the shared prefix): partial results per range of `chunk` tokens, or
// the outputs themselves when ws_o is null.
struct MxAttnParams {
  kvtc_mx_batch b;
  const uint8_t* pool;  // record of (layer, page 0, head 0)
  int32_t pool_pages, H, G;
  const void* q;
  int64_t q_stride;
  float c;  // scale log2(e)
  int32_t causal;
  void* out;
  float* lse;
  int32_t prefix;      // 1: rows of all sequences against the first one's pages
  int32_t begin, end;  // token range of this pass
  int32_t nt;        // 16-row tiles of a workgroup: 1 or 2 (k_mx_attn), 8 (k_mx_rows)
  int32_t waves;     // waves of a workgroup: 4, or 8 with nt 1
  int32_t fold;      // pair long tiles with short ones
  int32_t once;      // read the codes past the caches (nt 1)
  int32_t together;  // (own tokens) in one launch with the prefix
  int32_t pair;      // sequences by length, the longest `pair` in rising order, then falling; 0: as they come
  int32_t tiles, nsplit, chunk;
  int32_t slot0;   // first partial slot of this pass
  float* ws_o;     // [slot][total_rows q_heads][D]
  float2* ws_ml;   // [slot][total_rows q_heads]: running maximum (base 2), sum
  uint32_t* status;
};

// Joining the partials: slots [0, prefix_splits) cover the prefix in chunks
// of prefix_chunk tokens, the others start at `begin` in chunks of `chunk`.
struct MxJoinParams {
  kvtc_mx_batch b;
  int32_t Hq, D, causal;
  int32_t begin, prefix_splits, prefix_chunk, nsplit, chunk;
  const float* ws_o;
  const float2* ws_ml;
  void* out;
  float* lse;
  uint32_t* status;
};

hipError_t launch_mx_write(const MxIoParams& p, int D, int bk, int bv, bool f32, hipStream_t s);
hipError_t launch_mx_read(const MxIoParams& p, int D, int bk, int bv, bool f32, hipStream_t s);
// The passes of a call (either may be null), both before the join.
hipError_t launch_mx_attn(const MxAttnParams* prefix, const MxAttnParams* own, int D, int bk, int bv, bool f32,
                          hipStream_t s);
hipError_t launch_mx_join(const MxJoinParams& p, bool f32, hipStream_t s);

#if defined(__HIPCC__)

// A sequence's rows and length as the device arrays give them; a sequence
// outside the bounds has no rows and raises the status bit.
struct MxSeq {
  int row0, n, len;
};
__device__ __forceinline__ MxSeq mx_seq(const kvtc_mx_batch& b, int z, uint32_t* status) {
  MxSeq s{b.row_start[z], 0, b.kv_lens[z]};
  const int r1 = b.row_start[z + 1];
  const bool ok = s.row0 >= 0 && r1 >= s.row0 && r1 <= b.total_rows && r1 - s.row0 <= b.max_rows && s.len >= 0 &&
                  s.len <= b.max_len;
  if (ok) s.n = r1 - s.row0;
  else {
    s.len = 0;
    if (status) atomicOr(status, 1u << KVTC_ERR_INVALID_ARG);
  }
  return s;
}

#endif

}  // namespace kvtc
