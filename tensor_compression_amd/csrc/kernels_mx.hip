// Microscaled paged cache: quantising rows into pages and reading them back.
//
// Both kernels move bytes and do little else.  One wave takes one page of one
// (layer, head, keys or values): sixteen lanes a token, each with head_dim /
// 16 channels, so rows are read and written 16 bytes a lane and whole lines
// at a time, a block's maximum is an exchange within 4 (head_dim 128) or 8
// lanes, and both the key rows and the value groups of the record come out as
// consecutive words of consecutive lanes.  A page is the unit because it is
// the only stretch of a sequence that lies together, and because a lone token
// (a decode step) then costs one wave of latency (64 sequences: 3.4 us to
// write, 2.9 to read, most of it the launch).
//
// Bound by memory: 32 layers x 8 heads x 4096 tokens x 128 in bf16 against
// 4-bit codes, 680 MB, are written in 118 us (5.8 TB/s) and read back in 105
// (6.5 TB/s; a plain copy reaches 5.2).  Outputs are stored past the caches:
// through them a read of 278000 tokens takes 268 us instead of 252, and the
// write that follows a read 146 instead of 117, its codes having been pushed
// out.  Inputs are loaded through them: past them made no difference.  The
// order matters as much: consecutive workgroups on consecutive pages, each on
// the keys and values of two heads, read 278000 tokens in 252 us; four heads'
// keys a workgroup 261, four pages of a head 280, heads before pages 272, keys
// and values in one wave 270.
#include "mx_internal.h"

namespace kvtc {

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef short s16x2_t __attribute__((ext_vector_type(2)));

namespace {

// Largest value of the lanes that share a 32-channel block (32 / C lanes).
template <int C>
__device__ __forceinline__ uint32_t block_max(uint32_t a) {
  a = max(a, xor16_u32<1>(a));
  a = max(a, xor16_u32<2>(a));
  if constexpr (C == 4) a = max(a, xor16_u32<4>(a));
  return a;
}

// Scale byte of a block whose largest magnitude has the bits a: the exponent
// of a less that of the largest element, one more where the mantissa of a is
// half a step past it or further (1.75, between 6 and 8; 1.8125, between 448
// and where 480 would be).
template <int B>
__device__ __forceinline__ uint32_t scale_byte(uint32_t a) {
  const int up = (a & 0x7FFFFFu) >= (B == 4 ? 0x600000u : 0x680000u);
  const int s = (int)(a >> 23) - (B == 4 ? 2 : 8) + up;
  return (uint32_t)min(max(s, 15), B == 4 ? 252 : 246);
}

// C elements under scale 2^(s - 127): 4-bit codes in w[0], 8-bit codes four a word.
template <int B, int C>
__device__ __forceinline__ void encode(const float (&x)[C], uint32_t s, uint32_t (&w)[2]) {
  const float sc = __uint_as_float(s << 23);
  if constexpr (B == 4) {
    uint32_t o = 0;
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, x[0], x[1], sc, 0);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, x[2], x[3], sc, 1);
    if constexpr (C == 8) {
      o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, x[4], x[5], sc, 2);
      o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, x[6], x[7], sc, 3);
    }
    w[0] = o;
  } else {
    // the conversion does not saturate; only a clamped scale needs it to
    const float top = 448.0f * sc;
#pragma unroll
    for (int i = 0; i < C / 4; ++i) {
      s16x2_t o = {0, 0};
      o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, __builtin_amdgcn_fmed3f(x[4 * i], -top, top),
                                                   __builtin_amdgcn_fmed3f(x[4 * i + 1], -top, top), sc, false);
      o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, __builtin_amdgcn_fmed3f(x[4 * i + 2], -top, top),
                                                   __builtin_amdgcn_fmed3f(x[4 * i + 3], -top, top), sc, true);
      w[i] = __builtin_bit_cast(uint32_t, o);
    }
  }
}

// Bytes of a lane's C codes.
template <int B, int C>
__device__ __forceinline__ void store_codes(uint8_t* d, const uint32_t (&w)[2]) {
  if constexpr (B * C == 64) *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
  else if constexpr (B * C == 32) *reinterpret_cast<uint32_t*>(d) = w[0];
  else *reinterpret_cast<uint16_t*>(d) = (uint16_t)w[0];
}
template <int B, int C>
__device__ __forceinline__ void load_codes(const uint8_t* d, uint32_t (&w)[2]) {
  if constexpr (B * C == 64) {
    const uint2 u = *reinterpret_cast<const uint2*>(d);
    w[0] = u.x;
    w[1] = u.y;
  } else if constexpr (B * C == 32) w[0] = *reinterpret_cast<const uint32_t*>(d);
  else w[0] = *reinterpret_cast<const uint16_t*>(d);
}

// Where lane (token t = 4 kg + t4, entry n) finds its codes and scale in a record.
template <int D, int B>
__device__ __forceinline__ int code_at(bool value, int kg, int t4, int n) {
  constexpr int U = D / 16 * B / 8;  // bytes of a lane's codes
  return value ? ((kg * 16 + n) * 4 + t4) * U : ((kg * 4 + t4) * 16 + n) * U;
}
template <int D>
__device__ __forceinline__ int scale_at(bool value, int kg, int t4, int blk) {
  return value ? (kg * (D / 32) + blk) * 4 + t4 : (kg * 4 + t4) * (D / 32) + blk;
}

// What a wave works on: page `pg` of sequence z, head h, keys or values.
struct Unit {
  MxSeq s;
  int first, pg, page, h, kv, l;  // first: position of the sequence's first row, at least 0
  bool ok;
};
__device__ __forceinline__ Unit unit_of(const MxIoParams& p) {
  Unit u;
  const int z = (int)blockIdx.x / p.n_units, k = (int)blockIdx.x % p.n_units;
  const int w = __builtin_amdgcn_readfirstlane((int)(blockIdx.y * 4 + (threadIdx.x >> 6)));
  u.kv = w & 1;
  u.h = (w >> 1) % p.H;
  u.l = (w >> 1) / p.H;
  u.s = mx_seq(p.b, z, p.status);
  u.first = max(u.s.len - u.s.n, 0);
  u.pg = u.first / KVTC_MX_PAGE + k;
  u.ok = u.l < p.n_layers && u.s.n > 0 && u.pg * KVTC_MX_PAGE < u.s.len;
  u.page = 0;
  if (u.ok) {
    u.page = p.b.page_table[(int64_t)z * p.b.max_pages + u.pg];
    if ((uint32_t)u.page >= (uint32_t)p.pool_pages) {
      u.ok = false;
      if (p.status && (threadIdx.x & 63) == 0) atomicOr(p.status, 1u << KVTC_ERR_INVALID_ARG);
    }
  }
  return u;
}

template <int D, int B, typename T>
__device__ __forceinline__ void write_page(const MxIoParams& p, const Unit& u, int kc, int vc, uint8_t* rec) {
  constexpr int C = D / 16;
  const int lane = threadIdx.x & 63, t4 = lane >> 4, n = lane & 15;
  const T* src = reinterpret_cast<const T*>(p.x[u.kv]) + u.l * p.st[u.kv][0] + u.h * p.st[u.kv][1] + n * C;
  uint8_t* codes = rec + (u.kv ? kc : 0);
  uint8_t* scales = rec + kc + vc + (u.kv ? KVTC_MX_PAGE * D / 32 : 0);
  const int row_of_0 = u.s.row0 - (u.s.len - u.s.n);  // row of position 0
  uint32_t raw[4][C * (int)sizeof(T) / 4];
  bool on[4];
#pragma unroll
  for (int kg = 0; kg < 4; ++kg) {
    const int pos = u.pg * KVTC_MX_PAGE + kg * 4 + t4;
    on[kg] = pos >= u.first && pos < u.s.len;
    if (on[kg]) {
      const T* x = src + (int64_t)(row_of_0 + pos) * p.st[u.kv][2];
      if constexpr (C * sizeof(T) == 8) {
        const uint2 v = *reinterpret_cast<const uint2*>(x);
        raw[kg][0] = v.x;
        raw[kg][1] = v.y;
      } else {
#pragma unroll
        for (int i = 0; i < (int)(C * sizeof(T) / 16); ++i) {
          const uint4 v = reinterpret_cast<const uint4*>(x)[i];
          raw[kg][4 * i] = v.x;
          raw[kg][4 * i + 1] = v.y;
          raw[kg][4 * i + 2] = v.z;
          raw[kg][4 * i + 3] = v.w;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < (int)(C * sizeof(T) / 4); ++i) raw[kg][i] = 0;
    }
  }
  bool bad = false;
#pragma unroll
  for (int kg = 0; kg < 4; ++kg) {
    float x[C];
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      if constexpr (sizeof(T) == 4) x[i] = __uint_as_float(raw[kg][i]);
      else x[i] = __uint_as_float((i & 1) ? raw[kg][i / 2] & 0xFFFF0000u : raw[kg][i / 2] << 16);
      a = max(a, __float_as_uint(x[i]) & 0x7FFFFFFFu);  // magnitudes order as their bits, NaN above infinity
    }
    a = block_max<C>(a);
    const bool nan = a >= 0x7F800000u;
    uint32_t s = scale_byte<B>(a), w[2];
    encode<B, C>(x, s, w);
    if (nan) {
      s = 255;
      w[0] = w[1] = 0;
    }
    if (on[kg]) {
      store_codes<B, C>(codes + code_at<D, B>(u.kv, kg, t4, n), w);
      if (n % (32 / C) == 0) scales[scale_at<D>(u.kv, kg, t4, n / (32 / C))] = (uint8_t)s;
      bad |= nan;
    }
  }
  if (bad && p.status) atomicOr(p.status, 1u << KVTC_ERR_NONFINITE);
}

template <int D, int BK, int BV, typename T>
__global__ __launch_bounds__(256) void k_mx_write(const MxIoParams p) {
  constexpr MxRecord R = mx_record(D, BK, BV);
  const Unit u = unit_of(p);
  if (!u.ok) return;
  uint8_t* rec = p.pool + u.l * p.layer_bytes + ((int64_t)u.page * p.H + u.h) * R.bytes;
  if (u.kv) write_page<D, BV, T>(p, u, R.kc, R.vc, rec);
  else write_page<D, BK, T>(p, u, R.kc, R.vc, rec);
}

template <int D, int B, typename T>
__device__ __forceinline__ void read_page(const MxIoParams& p, const Unit& u, int kc, int vc, const uint8_t* rec) {
  constexpr int C = D / 16;
  const int lane = threadIdx.x & 63, t4 = lane >> 4, n = lane & 15;
  T* dst = reinterpret_cast<T*>(p.x[u.kv]) + u.l * p.st[u.kv][0] + u.h * p.st[u.kv][1] + n * C;
  const uint8_t* codes = rec + (u.kv ? kc : 0);
  const uint8_t* scales = rec + kc + vc + (u.kv ? KVTC_MX_PAGE * D / 32 : 0);
  const int row_of_0 = u.s.row0 - (u.s.len - u.s.n);
  uint32_t w[4][2], s[4];
#pragma unroll
  for (int kg = 0; kg < 4; ++kg) {  // the whole page is the record's own: read it without looking at the rows
    load_codes<B, C>(codes + code_at<D, B>(u.kv, kg, t4, n), w[kg]);
    s[kg] = scales[scale_at<D>(u.kv, kg, t4, n / (32 / C))];
  }
#pragma unroll
  for (int kg = 0; kg < 4; ++kg) {
    const int pos = u.pg * KVTC_MX_PAGE + kg * 4 + t4;
    if (pos < u.first || pos >= u.s.len) continue;
    const float sc = __uint_as_float(s[kg] << 23);
    T* y = dst + (int64_t)(row_of_0 + pos) * p.st[u.kv][2];
    f32x2_t f[C / 2];
#define KVTC_MX_PAIR(i, word, sel)                                                                    \
  if constexpr (B == 4) f[i] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[kg][0], sc, i);             \
  else f[i] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[kg][word], sc, sel);
    KVTC_MX_PAIR(0, 0, false)
    KVTC_MX_PAIR(1, 0, true)
    if constexpr (C == 8) {
      KVTC_MX_PAIR(2, 1, false)
      KVTC_MX_PAIR(3, 1, true)
    }
#undef KVTC_MX_PAIR
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < C / 4; ++i)
        store_out16(y + 4 * i, make_float4(f[2 * i][0], f[2 * i][1], f[2 * i + 1][0], f[2 * i + 1][1]));
    } else {  // every value is a bf16 number: its upper half
      uint32_t o[C / 2];
#pragma unroll
      for (int i = 0; i < C / 2; ++i)
        o[i] = __builtin_amdgcn_perm(__float_as_uint(f[i][1]), __float_as_uint(f[i][0]), 0x07060302u);
      if constexpr (C == 8) store_out16(y, make_uint4(o[0], o[1], o[2], o[3]));
      else *reinterpret_cast<uint2*>(y) = make_uint2(o[0], o[1]);
    }
  }
}

template <int D, int BK, int BV, typename T>
__global__ __launch_bounds__(256) void k_mx_read(const MxIoParams p) {
  constexpr MxRecord R = mx_record(D, BK, BV);
  const Unit u = unit_of(p);
  if (!u.ok) return;
  const uint8_t* rec = p.pool + u.l * p.layer_bytes + ((int64_t)u.page * p.H + u.h) * R.bytes;
  if (u.kv) read_page<D, BV, T>(p, u, R.kc, R.vc, rec);
  else read_page<D, BK, T>(p, u, R.kc, R.vc, rec);
}

template <int D, int BK, int BV>
hipError_t launch_io(const MxIoParams& p, bool write, bool f32, hipStream_t s) {
  const dim3 grid((unsigned)(p.b.n_seqs * p.n_units), (unsigned)((p.n_layers * p.H * 2 + 3) / 4));
  if (write) {
    if (f32) k_mx_write<D, BK, BV, float><<<grid, 256, 0, s>>>(p);
    else k_mx_write<D, BK, BV, uint16_t><<<grid, 256, 0, s>>>(p);
  } else {
    if (f32) k_mx_read<D, BK, BV, float><<<grid, 256, 0, s>>>(p);
    else k_mx_read<D, BK, BV, uint16_t><<<grid, 256, 0, s>>>(p);
  }
  return hipGetLastError();
}

hipError_t launch_io_any(const MxIoParams& p, int D, int bk, int bv, bool write, bool f32, hipStream_t s) {
  if (D == 128) {
    if (bk == 4) return bv == 4 ? launch_io<128, 4, 4>(p, write, f32, s) : launch_io<128, 4, 8>(p, write, f32, s);
    return bv == 4 ? launch_io<128, 8, 4>(p, write, f32, s) : launch_io<128, 8, 8>(p, write, f32, s);
  }
  if (bk == 4) return bv == 4 ? launch_io<64, 4, 4>(p, write, f32, s) : launch_io<64, 4, 8>(p, write, f32, s);
  return bv == 4 ? launch_io<64, 8, 4>(p, write, f32, s) : launch_io<64, 8, 8>(p, write, f32, s);
}

}  // namespace

hipError_t launch_mx_write(const MxIoParams& p, int D, int bk, int bv, bool f32, hipStream_t s) {
  return launch_io_any(p, D, bk, bv, true, f32, s);
}
hipError_t launch_mx_read(const MxIoParams& p, int D, int bk, int bv, bool f32, hipStream_t s) {
  return launch_io_any(p, D, bk, bv, false, f32, s);
}

}  // namespace kvtc
