// Microscaled paged cache: rows quantised into their pages with the rotation
// of their positions on the way, queries rotated beside them.
//
// A workgroup takes the rows of one page of a sequence and some of the row
// vectors of a layer: keys, values or queries.  It first turns the positions
// into (cos, sin), one angle a thread, in LDS, where all heads find them; then
// sixteen lanes take a (row, vector) at a time, as in the write without
// rotation: head_dim / 16 channels a lane, a block's maximum an exchange
// within 4 or 8 lanes, the codes consecutive words of the record.  Rows vary
// fastest, so that a full page leaves in whole lines, each row keeps its lanes
// (and a query its angles their registers), and a decode step's lone rows
// still fill the lanes with their heads.  All channels of a workgroup are on
// their way before the angles are worked out: with a loop over sixteen vectors
// and the next one's loads under way 32 layers x 8 heads x 4096 tokens x 128
// took 255 us, with four vectors loaded at once 148, with eight 133.
//
// Bound by memory: those (bf16, 4-bit codes, 680 MB) take 132 us (5.2 TB/s; the
// write without rotation 117, a plain copy 5.1 TB/s), 15900 rows of prompts
// with 32 query heads (385 MB) 88 us (4.4 TB/s; 92 with loads through the
// caches, 96 with the queries' stores through them too); a step of 64 rows 5
// us, the launch and five loads in a row.  Vector instructions issue in 73% and
// 36% of the clocks.  An attention right behind finds queries stored through
// the caches sooner, by more than the append loses if they are many: both, the
// prompts 367 us so and 377 as it is (the append alone 91 and 82 there), a step
// of 64 rows 38.2 and 37.7.
//
// A key's codes have to be those of its rotation in fp64, so that is what it
// is rotated in (products there are as fast as in fp32 on this card), and it
// is rounded to fp32 so that no later rounding can tell: to nearest, unless
// that lands on what may be a border of the elements or their scales (19 zero
// bits at the end); then to the odd neighbour.  (Deciding the codes in fp32
// from both ends of its error first, fp64 for what that leaves open: 8-bit keys
// leave a vector of every other workgroup open, 161 us and 116.)
#include <type_traits>

#include "mx_codes.h"

namespace kvtc {

namespace {

// An angle without its nearest multiple of pi / 2, which is q of them (pi / 2
// as a sum of two fp64 numbers; n times the first is subtracted exactly).
__device__ __forceinline__ double reduce(double a, int& q) {
  constexpr double kHi = 1.57079632679489661923, kLo = 6.123233995736766036e-17, kMagic = 6755399441055744.0;
  const double t = __fma_rn(a, 0.63661977236758134308, kMagic);  // the low bits of its word: n mod 4
  const double n = t - kMagic;
  q = (int)__double_as_longlong(t);
  return __fma_rn(-n, kLo, __fma_rn(-n, kHi, a));
}
// (cos, sin) from those of the reduced angle.
template <typename F2, typename F>
__device__ __forceinline__ F2 quadrant(F s, F c, int q) {
  const F u = (q & 1) ? s : c, v = (q & 1) ? c : s;
  return F2{((q + 1) & 2) ? -u : u, (q & 2) ? -v : v};
}
// Both by Taylor's polynomials on [-pi / 4, pi / 4], whose first terms left out
// are below 2^-29 and 5e-17.
template <typename F2>
__device__ __forceinline__ F2 turn_of(double a);
template <>
__device__ __forceinline__ float2 turn_of<float2>(double a) {
  int q;
  const float r = (float)reduce(a, q), z = r * r;
  float s = __fmaf_rn(z, 1.0f / 362880.0f, -1.0f / 5040.0f);
  s = __fmaf_rn(z, s, 1.0f / 120.0f);
  s = __fmaf_rn(z, s, -1.0f / 6.0f);
  s = __fmaf_rn(r * z, s, r);
  float c = __fmaf_rn(z, -1.0f / 3628800.0f, 1.0f / 40320.0f);
  c = __fmaf_rn(z, c, -1.0f / 720.0f);
  c = __fmaf_rn(z, c, 1.0f / 24.0f);
  c = __fmaf_rn(z, c, -0.5f);
  c = __fmaf_rn(z, c, 1.0f);
  return quadrant<float2>(s, c, q);
}
// (The coefficients are read where they are used: as literals they would take
// registers all through the kernel.)
__constant__ double kSin[] = {-1.0 / 1307674368000.0, 1.0 / 6227020800.0, -1.0 / 39916800.0, 1.0 / 362880.0, -1.0 / 5040.0, 1.0 / 120.0, -1.0 / 6.0};
__constant__ double kCos[] = {1.0 / 20922789888000.0, -1.0 / 87178291200.0, 1.0 / 479001600.0, -1.0 / 3628800.0, 1.0 / 40320.0, -1.0 / 720.0, 1.0 / 24.0, -0.5};
template <>
__device__ __forceinline__ double2 turn_of<double2>(double a) {
  typedef const __attribute__((address_space(4))) double* numbers_t;
  numbers_t ks = (numbers_t)(uintptr_t)kSin, kc = (numbers_t)(uintptr_t)kCos;
  asm volatile("" : "+s"(ks), "+s"(kc));
  int q;
  const double r = reduce(a, q), z = r * r;
  double s = ks[0], c = kc[0];
#pragma unroll
  for (int i = 1; i < 7; ++i) s = __fma_rn(z, s, ks[i]);
#pragma unroll
  for (int i = 1; i < 8; ++i) c = __fma_rn(z, c, kc[i]);
  return quadrant<double2>(__fma_rn(r * z, s, r), __fma_rn(z, c, 1.0), q);
}

// y rounded to fp32 so that rounding the result again, to 22 bits or fewer,
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
template <int D, bool INTER>
__device__ __forceinline__ int turn_at(int j) {
  constexpr int C = D / 16;
  return INTER ? (j % (C / 2)) * 16 + j / (C / 2) : (j % C) * 8 + j / C;
}

// The C channels of a lane rotated in F, by (cos, sin) of its pairs.  INTER:
// its pairs are its own channels; else o holds their other halves, negated in
// the lower one.
__device__ __forceinline__ float fma_of(float a, float b, float c) { return __fmaf_rn(a, b, c); }
__device__ __forceinline__ double fma_of(double a, double b, double c) { return __fma_rn(a, b, c); }
template <bool INTER, typename F, int C, typename F2, int N>
__device__ __forceinline__ void rotate(const float (&x)[C], const float (&o)[C], const F2 (&w)[N], F (&y)[C]) {
  if constexpr (INTER) {
#pragma unroll
    for (int i = 0; i < C / 2; ++i) {
      const F a = x[2 * i], b = x[2 * i + 1];
      y[2 * i] = fma_of(a, w[i].x, -(b * w[i].y));
      y[2 * i + 1] = fma_of(a, w[i].y, b * w[i].x);
    }
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) y[i] = fma_of((F)x[i], w[i].x, (F)o[i] * w[i].y);
  }
}

enum { kKeys, kValues, kQueries };

template <int D, int BK, int BV, typename T, bool INTER>
__global__ __launch_bounds__(256) void k_mx_rope(const MxRopeParams p) {
  constexpr MxRecord R = mx_record(D, BK, BV);
  constexpr int C = D / 16, HP = D / 2, W = C * (int)sizeof(T) / 4, PAIRS = INTER ? C / 2 : C;
  constexpr int SLICE = kMxRopeSlice, ROWS = KVTC_MX_PAGE;
  __shared__ __attribute__((aligned(16))) double2 turns[ROWS * HP];  // float2 for queries

  const kvtc_mx_batch& b = p.io.b;
  const int z = (int)blockIdx.x / p.io.n_units, H = p.io.H;
  const MxSeq s = mx_seq(b, z, p.io.status);
  const int first = s.len - s.n;  // position of the first row; queries may stand before the first token
  const int pg = (first >> 4) + (int)blockIdx.x % p.io.n_units;
  const int t0 = max(first, pg * ROWS), nt = min(s.len, (pg + 1) * ROWS) - t0;
  if (s.n == 0 || nt <= 0) return;
  const int row0 = s.row0 + t0 - first;  // row of token t0
  const int layer = (int)blockIdx.y / p.parts, part = (int)blockIdx.y % p.parts;

  const int lane = threadIdx.x & 63, n = lane & 15, g = threadIdx.x >> 4;
  const int pairs = p.rot / 2, ch = n * C;  // the lane's channels, and the first of its pairs
  const bool turned = ch < p.rot, upper = turned && ch >= pairs;
  const int pair0 = !turned ? 0 : INTER ? n * PAIRS : upper ? ch - pairs : ch;
  const int slot = INTER ? n : pair0 / C;

  // the vectors h0 .. h0 + count - 1 of a kind, row t of a vector at src + h head_stride + t row_stride
  auto run = [&](auto kind_, int h0, int count, const T* src, int64_t head_stride, int64_t row_stride) {
    constexpr int kind = decltype(kind_)::value;
    using F2 = std::conditional_t<kind == kKeys, double2, float2>;
    F2* const table = reinterpret_cast<F2*>(turns);
    uint8_t* head = nullptr;
    if constexpr (kind != kQueries) {
      if (pg < 0) return;
      const int page = __builtin_amdgcn_readfirstlane(b.page_table[(int64_t)z * b.max_pages + pg]);
      if ((uint32_t)page >= (uint32_t)p.io.pool_pages) {
        if (p.io.status && threadIdx.x == 0) atomicOr(p.io.status, 1u << KVTC_ERR_INVALID_ARG);
        return;
      }
      head = p.io.pool + layer * p.io.layer_bytes + ((int64_t)page * H + h0) * R.bytes;
    }
    src += h0 * head_stride + row0 * row_stride + ch;

    // What a thread needs for its angles, requested before all else.
    constexpr int STEP = 256 / HP;
    const int my_pair = threadIdx.x % HP, my_row = threadIdx.x / HP;
    double freq = 0.0;
    int where[ROWS / STEP] = {};
    if (kind != kValues && my_pair < pairs) {
      freq = p.freqs[my_pair];
      const int axis = (int)(p.axis[my_pair >> 5] >> (2 * (my_pair & 31))) & 3;
#pragma unroll
      for (int i = 0; i < ROWS / STEP; ++i) {
        const int t = my_row + i * STEP;
        where[i] = t0 + t;
        if (p.positions && t < nt) where[i] = p.positions[(int64_t)axis * b.total_rows + row0 + t];
      }
    }

    bool bad = false;
    auto pass = [&](auto full_) {
      // a full page: group g stays at row g, every step is one vector on for all
      constexpr bool FULL = decltype(full_)::value;
      const int all = nt * count, inv = 65536 / nt + 1;  // c / nt for c < 4096 by the product
      auto at = [&](int c, int& h, int& t) {
        if constexpr (FULL) {
          h = c;
          t = g;
          return c < count;
        }
        h = (c * 16 + g) * inv >> 16;
        t = c * 16 + g - h * nt;
        return c * 16 + g < all;
      };
      uint32_t raw[SLICE][W];
#pragma unroll
      for (int c = 0; c < SLICE; ++c) {
        int h, t;
        const bool on = at(c, h, t);
        const T* x = src + h * head_stride + t * row_stride;
        if constexpr (W == 2) {
          const uint2 u = on ? *reinterpret_cast<const uint2*>(x) : make_uint2(0, 0);
          raw[c][0] = u.x;
          raw[c][1] = u.y;
        } else {
#pragma unroll
          for (int i = 0; i < W / 4; ++i) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (on) u = __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const u32x4_out*>(x) + i));
            raw[c][4 * i] = u.x;
            raw[c][4 * i + 1] = u.y;
            raw[c][4 * i + 2] = u.z;
            raw[c][4 * i + 3] = u.w;
          }
        }
      }
      if constexpr (kind != kValues) {
        if (my_pair < pairs) {
#pragma unroll
          for (int i = 0; i < ROWS / STEP; ++i) {
            const int t = my_row + i * STEP;
            if (t < nt) table[t * HP + turn_at<D, INTER>(my_pair)] = turn_of<F2>((double)where[i] * freq);
          }
        }
        __syncthreads();
      }
      F2 w[PAIRS];
#pragma unroll
      for (int c = 0; c < SLICE; ++c) {
        if (FULL ? c >= count : c * 16 >= all) break;
        int h, t;
        const bool on = at(c, h, t);
        const int pos = t0 + t, kg = (pos & 15) >> 2, t4 = pos & 3;
        float x[C];
        unpack<T, C>(raw[c], x);
        uint8_t* const rec = head + h * (int64_t)R.bytes;
        if constexpr (kind == kValues) {
          bad |= put_row<D, BV>(x, true, rec + R.kc, rec + R.kc + R.vc + R.sc, kg, t4, n, on);
          continue;
        }
        if (c == 0 || !FULL || kind == kKeys) {  // (a key's would take 32 registers)
#pragma unroll
          for (int k = 0; k < PAIRS; ++k) w[k] = table[t * HP + slot + k * (INTER ? 16 : 8)];
        }
        float o[C];
        if constexpr (!INTER) {  // the other halves of the lane's pairs
          uint32_t other[W];
          if (p.rot == D) {
#pragma unroll
            for (int i = 0; i < W; ++i) other[i] = xor16_u32<8>(raw[c][i]);
          } else {
            const int from = !turned ? lane : lane + (upper ? -1 : 1) * (pairs / C);
#pragma unroll
            for (int i = 0; i < W; ++i) other[i] = (uint32_t)__shfl((int)raw[c][i], from);
          }
          const uint32_t flip = upper ? 0 : sizeof(T) == 4 ? 0x80000000u : 0x80008000u;
#pragma unroll
          for (int i = 0; i < W; ++i) other[i] ^= flip;
          unpack<T, C>(other, o);
        }
        if constexpr (kind == kKeys) {
          double y[C];
          float r[C];
          rotate<INTER>(x, o, w, y);
          uint32_t low = 0xFFFFFFFFu;  // 0: some value may lie on a border
#pragma unroll
          for (int i = 0; i < C; ++i) {
            r[i] = (float)y[i];
            low = min(low, __float_as_uint(r[i]) << 13);
          }
          if (__builtin_amdgcn_ballot_w64(low == 0)) {
#pragma unroll
            for (int i = 0; i < C; ++i) r[i] = to_odd(y[i]);
          }
          if (p.rot < D) {
#pragma unroll
            for (int i = 0; i < C; ++i) r[i] = turned ? r[i] : x[i];
          }
          bad |= put_row<D, BK>(r, false, rec, rec + R.kc + R.vc, kg, t4, n, on);
        } else {
          float y[C];
          rotate<INTER>(x, o, w, y);
          if (p.rot < D) {
#pragma unroll
            for (int i = 0; i < C; ++i) y[i] = turned ? y[i] : x[i];
          }
          if (!on) continue;
          T* dst = reinterpret_cast<T*>(p.q_out) + (row0 + t) * p.q_out_stride + (int64_t)(h0 + h) * D + ch;
          if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < C / 4; ++i)
              store_out16(dst + 4 * i, make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]));
          } else {
            uint32_t u[C / 2];
#pragma unroll
            for (int i = 0; i < C / 2; ++i) u[i] = pack2(y[2 * i], y[2 * i + 1]);
            if constexpr (C == 8) store_out16(dst, make_uint4(u[0], u[1], u[2], u[3]));
            else *reinterpret_cast<uint2*>(dst) = make_uint2(u[0], u[1]);
          }
        }
      }
    };
    if (nt == ROWS) pass(std::true_type{});
    else pass(std::false_type{});
    if (bad && p.io.status) atomicOr(p.io.status, 1u << KVTC_ERR_NONFINITE);
  };

  const int kv_parts = (H + SLICE - 1) / SLICE;
  if (part < 2 * kv_parts) {
    const int value = part >= kv_parts, h0 = (part - value * kv_parts) * SLICE, count = min(SLICE, H - h0);
    const int64_t* st = p.io.st[value];
    const T* src = reinterpret_cast<const T*>(p.io.x[value]) + layer * st[0];
    if (value) run(std::integral_constant<int, kValues>{}, h0, count, src, st[1], st[2]);
    else run(std::integral_constant<int, kKeys>{}, h0, count, src, st[1], st[2]);
  } else {
    const int h0 = (part - 2 * kv_parts) * SLICE;
    run(std::integral_constant<int, kQueries>{}, h0, min(SLICE, p.Hq - h0), reinterpret_cast<const T*>(p.q), (int64_t)D, p.q_stride);
  }
}

template <int D, int BK, int BV>
hipError_t launch_rope(const MxRopeParams& p, bool f32, hipStream_t s) {
  const dim3 grid((unsigned)(p.io.b.n_seqs * p.io.n_units), (unsigned)(p.io.n_layers * p.parts));
  if (p.interleaved) {
    if (f32) k_mx_rope<D, BK, BV, float, true><<<grid, 256, 0, s>>>(p);
    else k_mx_rope<D, BK, BV, uint16_t, true><<<grid, 256, 0, s>>>(p);
  } else {
    if (f32) k_mx_rope<D, BK, BV, float, false><<<grid, 256, 0, s>>>(p);
    else k_mx_rope<D, BK, BV, uint16_t, false><<<grid, 256, 0, s>>>(p);
  }
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
