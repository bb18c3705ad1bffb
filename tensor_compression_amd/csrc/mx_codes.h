// Elements, scales and their places in a record: what writing, reading and
// moving the microscaled cache share.  Device code only.
#pragma once

#include "mx_internal.h"

namespace kvtc {

typedef float f32x2_t __attribute__((ext_vector_type(2)));
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

// C channels of a row as fp32.
template <typename T, int C>
__device__ __forceinline__ void unpack(const uint32_t (&raw)[C * sizeof(T) / 4], float (&x)[C]) {
#pragma unroll
  for (int i = 0; i < C; ++i) {
    if constexpr (sizeof(T) == 4) x[i] = __uint_as_float(raw[i]);
    else x[i] = __uint_as_float((i & 1) ? raw[i / 2] & 0xFFFF0000u : raw[i / 2] << 16);
  }
}

// Two values as bf16, to nearest.
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef __bf16 pair_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, pair_t));
}

// A row's channels n C ... of the token (4 kg + t4) of a record, quantised and
// stored by the 16 lanes that hold them; true where the lane's block was not
// finite.
template <int D, int B>
__device__ __forceinline__ bool put_row(const float (&x)[D / 16], bool value, uint8_t* codes, uint8_t* scales, int kg,
                                        int t4, int n, bool on) {
  constexpr int C = D / 16;
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < C; ++i) a = max(a, __float_as_uint(x[i]) & 0x7FFFFFFFu);  // magnitudes order as their bits, NaN above infinity
  a = block_max<C>(a);
  const bool nan = a >= 0x7F800000u;
  uint32_t s = scale_byte<B>(a), w[2];
  encode<B, C>(x, s, w);
  if (nan) {
    s = 255;
    w[0] = w[1] = 0;
  }
  if (on) {
    store_codes<B, C>(codes + code_at<D, B>(value, kg, t4, n), w);
    if (n % (32 / C) == 0) scales[scale_at<D>(value, kg, t4, n / (32 / C))] = (uint8_t)s;
  }
  return nan && on;
}

}  // namespace

}  // namespace kvtc
