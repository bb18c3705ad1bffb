// Attention over the microscaled paged cache, rows one behind the other: the
// kernels of mx_attn.h, and the join of ranges.
#include "mx_attn.h"

namespace kvtc {

namespace {

// Joins a row's partials: W waves a (row, head), sixteen lanes on its
// channels, so 4 W partials at once; W = 4 where there are many.
template <int D, bool F32, int W>
__global__ __launch_bounds__(256) void k_mx_join(const MxJoinParams p) {
  constexpr int C = D / 16;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c0 = (lane & 15) * C;
  const int g = (W == 4 ? wave * 4 : 0) + (lane >> 4);
  const int64_t at = W == 4 ? blockIdx.x : (int64_t)blockIdx.x * 4 + wave;
  const int64_t all = (int64_t)p.b.total_rows * p.Hq;
  if (at >= all) return;
  const int row = (int)(at / p.Hq);
  const MxSeq s = mx_seq(p.b, seq_of(p.b, row), p.status);
  if (row < s.row0 || row >= s.row0 + s.n) return;  // a row of no sequence
  const int lim = limit_of(s, row - s.row0, p.causal);
  // how many partials of each pass hold tokens of this row
  const int a = p.prefix_splits ? (min(lim, p.begin) + p.prefix_chunk - 1) / p.prefix_chunk : 0;
  const int b = lim > p.begin ? (lim - p.begin + p.chunk - 1) / p.chunk : 0;
  float M = kLow, L = 0.f, o[C];
#pragma unroll
  for (int j = 0; j < C; ++j) o[j] = 0.f;
  auto add = [&](float m, float l, const float (&v)[C]) {
    const float nm = fmaxf(M, m), u = __builtin_amdgcn_exp2f(M - nm), w = __builtin_amdgcn_exp2f(m - nm);
    M = nm;
    L = __fmaf_rn(L, u, l * w);
#pragma unroll
    for (int j = 0; j < C; ++j) o[j] = __fmaf_rn(o[j], u, v[j] * w);
  };
#pragma unroll 2
  for (int k = g; k < a + b; k += 4 * W) {
    const int64_t slot = (int64_t)(k < a ? k : p.prefix_splits + k - a) * all + at;
    const float2 x = p.ws_ml[slot];
    const float4* y = reinterpret_cast<const float4*>(p.ws_o + slot * D + c0);
    float v[C];
#pragma unroll
    for (int j = 0; j < C / 4; ++j) {
      const float4 t = y[j];
      v[4 * j] = t.x;
      v[4 * j + 1] = t.y;
      v[4 * j + 2] = t.z;
      v[4 * j + 3] = t.w;
    }
    add(x.x, x.y, v);
  }
#pragma unroll
  for (int d = 16; d < 64; d <<= 1) {
    const float m = __shfl_xor(M, d), l = __shfl_xor(L, d);
    float v[C];
#pragma unroll
    for (int j = 0; j < C; ++j) v[j] = __shfl_xor(o[j], d);
    add(m, l, v);
  }
  if constexpr (W == 4) {
    __shared__ float part[3][16][C + 2];
    if (wave > 0 && lane < 16) {
      part[wave - 1][lane][0] = M;
      part[wave - 1][lane][1] = L;
#pragma unroll
      for (int j = 0; j < C; ++j) part[wave - 1][lane][2 + j] = o[j];
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int w = 0; w < 3; ++w) {
      float v[C];
#pragma unroll
      for (int j = 0; j < C; ++j) v[j] = part[w][lane & 15][2 + j];
      add(part[w][lane & 15][0], part[w][lane & 15][1], v);
    }
  }
  if (lane >= 16) return;
  store_row<F32>(nullptr, p.out, at, D, c0, o, L);
  if (p.lse && c0 == 0) p.lse[at] = log_sum(M, L);
}

}  // namespace

hipError_t launch_mx_attn(const MxAttnParams* prefix, const MxAttnParams* own, int D, int bk, int bv, bool f32,
                          hipStream_t s) {
  return D == 128 ? launch_any<128, false>(prefix, own, bk, bv, f32, s) : launch_any<64, false>(prefix, own, bk, bv, f32, s);
}

template <int D, bool F32>
static void launch_join(const MxJoinParams& p, hipStream_t s) {
  const int64_t all = (int64_t)p.b.total_rows * p.Hq;
  // one wave a row is done in two rounds of loads up to 8 partials; more of
  // them are worth the barrier while there are few rows (64 rows of 32
  // partials: 6.2 -> 4.6 us, but 2048 rows of 33: 8.2 -> 9.4 us)
  if (p.prefix_splits + p.nsplit > 8 && all <= 512) k_mx_join<D, F32, 4><<<(unsigned)all, 256, 0, s>>>(p);
  else k_mx_join<D, F32, 1><<<(unsigned)((all + 3) / 4), 256, 0, s>>>(p);
}

hipError_t launch_mx_join(const MxJoinParams& p, bool f32, hipStream_t s) {
  if (p.D == 128) f32 ? launch_join<128, true>(p, s) : launch_join<128, false>(p, s);
  else f32 ? launch_join<64, true>(p, s) : launch_join<64, false>(p, s);
  return hipGetLastError();
}

}  // namespace kvtc
