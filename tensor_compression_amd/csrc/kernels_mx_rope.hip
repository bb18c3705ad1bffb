// Microscaled paged cache: rows quantised into their pages with the rotation
// of their positions on the way, queries rotated beside them.
//
// A workgroup takes the rows of one page of a sequence and some of their row
// vectors (keys and values of every head, queries).  It first turns the
// positions into (cos, sin), one angle a thread, in LDS, where all heads find
// them; then sixteen lanes take a (row, vector) at a time, as in the write
// without rotation: head_dim / 16 channels a lane, a block's maximum an
// exchange within 4 or 8 lanes, the codes consecutive words of the record.
// Rows vary fastest, so that a full page leaves in whole lines and a decode
// step's lone rows still fill the lanes with their heads.
//
// Keys are rotated in fp64 (as fast as fp32 on this card, but for the
// conversions) and rounded to fp32 so that no later rounding can tell: to
// nearest, unless that lands on what may be a border of the elements or their
// scales (19 zero bits at the end); then to the odd neighbour.
#include "mx_codes.h"

namespace kvtc {

namespace {

// cos and sin of an angle in fp64: the nearest multiple of pi / 2 taken off
// (pi / 2 as a sum of two fp64 numbers; n times the first is subtracted
// exactly), Taylor's polynomials on [-pi / 4, pi / 4] (their first terms left
// out are below 5e-17), and the quadrant.
__device__ __forceinline__ double2 turn_of(double a) {
  constexpr double kHi = 1.57079632679489661923, kLo = 6.123233995736766036e-17, kMagic = 6755399441055744.0;
  const double t = __fma_rn(a, 0.63661977236758134308, kMagic);  // the low bits of its word: n mod 4
  const double n = t - kMagic;
  const double r = __fma_rn(-n, kLo, __fma_rn(-n, kHi, a)), z = r * r;
  double s = __fma_rn(z, -1.0 / 1307674368000.0, 1.0 / 6227020800.0);
  s = __fma_rn(z, s, -1.0 / 39916800.0);
  s = __fma_rn(z, s, 1.0 / 362880.0);
  s = __fma_rn(z, s, -1.0 / 5040.0);
  s = __fma_rn(z, s, 1.0 / 120.0);
  s = __fma_rn(z, s, -1.0 / 6.0);
  s = __fma_rn(r * z, s, r);
  double c = __fma_rn(z, 1.0 / 20922789888000.0, -1.0 / 87178291200.0);
  c = __fma_rn(z, c, 1.0 / 479001600.0);
  c = __fma_rn(z, c, -1.0 / 3628800.0);
  c = __fma_rn(z, c, 1.0 / 40320.0);
  c = __fma_rn(z, c, -1.0 / 720.0);
  c = __fma_rn(z, c, 1.0 / 24.0);
  c = __fma_rn(z, c, -0.5);
  c = __fma_rn(z, c, 1.0);
  const int q = (int)__double_as_longlong(t);
  const double u = (q & 1) ? s : c, v = (q & 1) ? c : s;  // cos, sin up to their signs
  return make_double2(((q + 1) & 2) ? -u : u, (q & 2) ? -v : v);
}

// y rounded to fp32 so that rounding the result again, to 23 bits or fewer,
// is rounding y: the neighbour with an odd last bit unless y is a fp32 number;
// finite numbers stay finite.
__device__ __forceinline__ float to_odd(double y) {
  float f = (float)y;
  const double d = f;
  if (__builtin_isinf(f) && !__builtin_isinf(y)) return copysignf(3.4028234663852886e38f, f);
  const uint32_t b = __float_as_uint(f);
  if (!(d != y) || __builtin_isnan(f) || (b & 1)) return f;
  return __uint_as_float(__builtin_fabs(d) < __builtin_fabs(y) ? b + 1 : b - 1);
}

// Where (cos, sin) of pair j lie in a row's table: a lane's i-th pairs next to
// each other for all lanes.
template <int D>
__device__ __forceinline__ int turn_at(int j, int interleaved) {
  constexpr int C = D / 16;
  return interleaved ? (j % (C / 2)) * 16 + j / (C / 2) : (j % C) * 8 + j / C;
}

// A row vector on its way through a group of lanes.
struct Vec {
  int hd, t;         // which one of its token's, and which token
  const void* src;   // the lane's channels
  bool on;
};

template <int D, int BK, int BV, typename T>
__global__ __launch_bounds__(256) void k_mx_rope(const MxRopeParams p) {
  constexpr MxRecord R = mx_record(D, BK, BV);
  constexpr int C = D / 16, HP = D / 2, W = C * (int)sizeof(T) / 4;
  __shared__ __attribute__((aligned(16))) double2 turns[KVTC_MX_PAGE * HP];

  const kvtc_mx_batch& b = p.io.b;
  const int z = (int)blockIdx.x / p.io.n_units;
  const MxSeq s = mx_seq(b, z, p.io.status);
  const int first = s.len - s.n;  // position of the first row; queries may stand before the first token
  const int pg = (first >> 4) + (int)blockIdx.x % p.io.n_units;
  const int t0 = max(first, pg * KVTC_MX_PAGE), nt = min(s.len, (pg + 1) * KVTC_MX_PAGE) - t0;
  if (s.n == 0 || nt <= 0) return;
  const int kv = 2 * p.io.n_layers * p.io.H;  // key vectors, then value vectors, then queries
  const int h0 = (int)blockIdx.y * p.slice, h1 = min(h0 + p.slice, p.all);
  int page = -1;
  if (pg >= 0 && h0 < kv) {
    page = b.page_table[(int64_t)z * b.max_pages + pg];
    if ((uint32_t)page >= (uint32_t)p.io.pool_pages) {
      page = -1;
      if (p.io.status && threadIdx.x == 0) atomicOr(p.io.status, 1u << KVTC_ERR_INVALID_ARG);
    }
  }
  const int pairs = p.rot / 2, row0 = s.row0 + t0 - first;  // row of token t0
  if (h0 < kv / 2 || h1 > kv) {
    for (int i = threadIdx.x; i < nt * HP; i += 256) {
      const int t = i / HP, j = i % HP;
      if (j >= pairs) continue;
      int pos = t0 + t;
      if (p.positions) {
        const int axis = (int)(p.axis[j >> 5] >> (2 * (j & 31))) & 3;
        pos = p.positions[(int64_t)axis * b.total_rows + row0 + t];
      }
      turns[t * HP + turn_at<D>(j, p.interleaved)] = turn_of((double)pos * p.freqs[j]);
    }
    __syncthreads();
  }

  const int lane = threadIdx.x & 63, n = lane & 15, g = threadIdx.x >> 4;
  const int all = nt * (h1 - h0), inv = 65536 / nt + 1;  // c / nt for c < 4096 by the product
  auto vec_of = [&](int c) {
    Vec v;
    const int k = (c * inv) >> 16;
    v.t = c - k * nt;
    v.hd = h0 + k;
    v.on = c < all;
    if (v.hd < kv) {
      int h = v.hd, value = 0, l = 0;
      if (h >= kv / 2) {
        h -= kv / 2;
        value = 1;
      }
      if (p.io.n_layers > 1) {
        l = h / p.io.H;
        h -= l * p.io.H;
      }
      const int64_t* st = p.io.st[value];
      v.src = reinterpret_cast<const T*>(p.io.x[value]) + l * st[0] + h * st[1] + (int64_t)(row0 + v.t) * st[2] + n * C;
      v.on = v.on && page >= 0;
    } else {
      v.src = reinterpret_cast<const T*>(p.q) + (int64_t)(row0 + v.t) * p.q_stride + (v.hd - kv) * D + n * C;
    }
    return v;
  };
  auto load = [&](const Vec& v, uint32_t (&raw)[W]) {
    if constexpr (W == 2) {
      const uint2 x = v.on ? *reinterpret_cast<const uint2*>(v.src) : make_uint2(0, 0);
      raw[0] = x.x;
      raw[1] = x.y;
    } else {
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        const uint4 x = v.on ? reinterpret_cast<const uint4*>(v.src)[i] : make_uint4(0, 0, 0, 0);
        raw[4 * i] = x.x;
        raw[4 * i + 1] = x.y;
        raw[4 * i + 2] = x.z;
        raw[4 * i + 3] = x.w;
      }
    }
  };

  // the lane's place in the rotation
  const int ch = n * C;
  const bool turned = ch < p.rot, upper = turned && ch >= pairs;
  const int across = p.rot == D ? 0 : (upper ? -1 : 1) * (pairs / C);  // lanes to the other half of the pairs; 0: 8, by DPP
  const int slot = p.interleaved ? n : !turned ? 0 : (upper ? ch - pairs : ch) / C;
  auto partner = [&](const uint32_t (&raw)[W], uint32_t (&other)[W]) {
    if (across == 0) {
#pragma unroll
      for (int i = 0; i < W; ++i) other[i] = xor16_u32<8>(raw[i]);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) other[i] = (uint32_t)__shfl((int)raw[i], turned ? lane + across : lane);
    }
  };

  bool bad = false;
  auto work = [&](const Vec& v, const uint32_t (&raw)[W]) {
    float x[C];
    unpack<T, C>(raw, x);
    const double2* const tab = turns + v.t * HP + slot;
    const int pos = t0 + v.t, kg = (pos & 15) >> 2, t4 = pos & 3;
    if (v.hd < kv / 2) {
      double y[C];
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < C / 2; ++i) {
          const double2 w = tab[i * 16];
          const double a = x[2 * i], c = x[2 * i + 1];
          y[2 * i] = __fma_rn(a, w.x, -(c * w.y));
          y[2 * i + 1] = __fma_rn(a, w.y, c * w.x);
        }
      } else {
        uint32_t other[W];
        float o[C];
        partner(raw, other);
        unpack<T, C>(other, o);
#pragma unroll
        for (int i = 0; i < C; ++i) {
          const double2 w = tab[i * 8];
          const double sin = upper ? w.y : -w.y;
          y[i] = __fma_rn((double)x[i], w.x, (double)o[i] * sin);
        }
      }
      uint32_t low = 0xFFFFFFFFu;  // 0: some value may lie on a border
      float r[C];
#pragma unroll
      for (int i = 0; i < C; ++i) {
        r[i] = (float)y[i];
        low = min(low, __float_as_uint(r[i]) << 13);
      }
      if (__builtin_amdgcn_ballot_w64(low == 0)) {
#pragma unroll
        for (int i = 0; i < C; ++i) r[i] = to_odd(y[i]);
      }
#pragma unroll
      for (int i = 0; i < C; ++i) x[i] = turned ? r[i] : x[i];
    }
    if (v.hd < kv) {
      int h = v.hd, l = 0;
      const bool value = h >= kv / 2;
      if (value) h -= kv / 2;
      if (p.io.n_layers > 1) {
        l = h / p.io.H;
        h -= l * p.io.H;
      }
      uint8_t* rec = p.io.pool + l * p.io.layer_bytes + ((int64_t)page * p.io.H + h) * R.bytes;
      if (value) bad |= put_row<D, BV>(x, true, rec + R.kc, rec + R.kc + R.vc + R.sc, kg, t4, n, v.on);
      else bad |= put_row<D, BK>(x, false, rec, rec + R.kc + R.vc, kg, t4, n, v.on);
      return;
    }
    if (p.interleaved) {
#pragma unroll
      for (int i = 0; i < C / 2; ++i) {
        const double2 w = tab[i * 16];
        const float c = (float)w.x, d = (float)w.y, a = x[2 * i], e = x[2 * i + 1];
        x[2 * i] = turned ? __fmaf_rn(a, c, -(e * d)) : a;
        x[2 * i + 1] = turned ? __fmaf_rn(a, d, e * c) : e;
      }
    } else {
      uint32_t other[W];
      float o[C];
      partner(raw, other);
      unpack<T, C>(other, o);
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const double2 w = tab[i * 8];
        const float sin = upper ? (float)w.y : -(float)w.y;
        x[i] = turned ? __fmaf_rn(x[i], (float)w.x, o[i] * sin) : x[i];
      }
    }
    if (!v.on) return;
    T* dst = reinterpret_cast<T*>(p.q_out) + (int64_t)(row0 + v.t) * p.q_out_stride + (v.hd - kv) * D + n * C;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < C / 4; ++i)
        reinterpret_cast<float4*>(dst)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    } else {
      uint32_t w[C / 2];
#pragma unroll
      for (int i = 0; i < C / 2; ++i) w[i] = pack2(x[2 * i], x[2 * i + 1]);
      if constexpr (C == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
      else *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    }
  };

  // the next vector's channels on their way while one is worked on
  Vec now = vec_of(g);
  uint32_t raw[W];
  load(now, raw);
  for (int c = g; c < all; c += 16) {
    const Vec next = vec_of(c + 16);
    uint32_t ahead[W];
    load(next, ahead);
    work(now, raw);
    now = next;
#pragma unroll
    for (int i = 0; i < W; ++i) raw[i] = ahead[i];
  }
  if (bad && p.io.status) atomicOr(p.io.status, 1u << KVTC_ERR_NONFINITE);
}

template <int D, int BK, int BV>
hipError_t launch_rope(const MxRopeParams& p, bool f32, hipStream_t s) {
  const dim3 grid((unsigned)(p.io.b.n_seqs * p.io.n_units), (unsigned)((p.all + p.slice - 1) / p.slice));
  if (f32) k_mx_rope<D, BK, BV, float><<<grid, 256, 0, s>>>(p);
  else k_mx_rope<D, BK, BV, uint16_t><<<grid, 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_rope(const MxRopeParams& p, int D, int bk, int bv, bool f32, hipStream_t s) {
  if (D == 128) {
    if (bk == 4) return bv == 4 ? launch_rope<128, 4, 4>(p, f32, s) : launch_rope<128, 4, 8>(p, f32, s);
    return bv == 4 ? launch_rope<128, 8, 4>(p, f32, s) : launch_rope<128, 8, 8>(p, f32, s);
  }
  if (bk == 4) return bv == 4 ? launch_rope<64, 4, 4>(p, f32, s) : launch_rope<64, 4, 8>(p, f32, s);
  return bv == 4 ? launch_rope<64, 8, 4>(p, f32, s) : launch_rope<64, 8, 8>(p, f32, s);
}

}  // namespace kvtc
