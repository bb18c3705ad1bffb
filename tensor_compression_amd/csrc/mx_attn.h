// Attention over the microscaled paged cache.
//
// For 16 NT query rows of one kv head (row r = token r / G, head r % G of its
// group) and a range of tokens, a workgroup computes
//   s = q k^T, running maximum m, sum l of 2^(c s - m), o = sum 2^(c s - m) v
// in one pass.  Up to 64 rows its waves take pairs of pages in turn and are
// joined through LDS at the end (k_mx_attn); more rows share the converted
// codes in LDS (k_mx_rows); ranges of tokens are joined by k_mx_join.
//
// The pool is laid out for v_mfma_f32_16x16x32_bf16, so nothing is shuffled
// or staged on its way to the matrix unit:
//  * S^T = K Q^T, one page (16 tokens) as the rows.  Lane (kg, n) = (lane /
//    16, lane % 16) holds token n and the channel quarter kg, which are
//    consecutive bytes of the record under one scale; the contraction order
//    is the same permutation for Q.
//  * The result gives the lane tokens 4 kg .. 4 kg + 3 of query row n, which
//    is exactly the slice of P^T that it has to supply as the other operand
//    of O^T = V^T P^T, two pages making the contraction of 32.  The values
//    are stored so that the lane's four tokens and head_dim / 16 channels are
//    consecutive bytes; v_perm pairs tokens after the conversion.
//  * Elements become bf16 exactly (v_cvt_scalef32_pk_bf16_*), two a
//    instruction, scale included.
// The running maximum only moves when a score exceeds it by more than 2^8:
// weights stay below 2^8, which costs no accuracy in floating point and
// saves the exchange between lanes and the rescaling of o in most steps.
#pragma once

#include <type_traits>

#include "mx_internal.h"

namespace kvtc {

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

namespace {

constexpr float kLow = -3.0e38f;  // running maximum (scaled) of a row that has seen nothing; its first score moves it
constexpr float kSlack = 8.0f;    // growth (in powers of two) that leaves the maximum as it is
constexpr float kLn2 = 0.69314718055994531f;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}
__device__ __forceinline__ bf16x8_t operand(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(bf16x8_t, make_uint4(a, b, c, d));
}
__device__ __forceinline__ f32x4_t mfma(bf16x8_t a, bf16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16_t mfma(bf16x8_t a, bf16x8_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ float max2(float a, float b) { return __builtin_elementwise_maximum(a, b); }
__device__ __forceinline__ float max3(float a, float b, float c) { return max2(max2(a, b), c); }

// Two elements of a word as bf16 under a scale: pair i of its 8 / (B / 4).
template <int B, int I>
__device__ __forceinline__ uint32_t two(uint32_t w, float sc) {
  if constexpr (B == 4) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, I));
  else return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, sc, I != 0));
}

// Eight consecutive elements (8 B bits at w) as one operand.
template <int B>
__device__ __forceinline__ bf16x8_t eight(const uint32_t* w, float sc) {
  if constexpr (B == 4) return operand(two<4, 0>(w[0], sc), two<4, 1>(w[0], sc), two<4, 2>(w[0], sc), two<4, 3>(w[0], sc));
  else return operand(two<8, 0>(w[0], sc), two<8, 1>(w[0], sc), two<8, 0>(w[1], sc), two<8, 1>(w[1], sc));
}

// The part of a bf16 split that is left after `h` (two values a word).
__device__ __forceinline__ float rest(float x, uint32_t h, int hi) {
  return x - __uint_as_float(hi ? h & 0xFFFF0000u : h << 16);
}

// Codes on their way in; ONCE: past the caches, where no other workgroup reads
// them and they are more than the memory-side cache could keep for the next
// call (64 ragged sequences, 309 MB: 72 -> 67 us; 16 of 8000 tokens, 139 MB
// and so still there when read again: 28 -> 36 us, so those are cached).
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
template <bool ONCE, typename T>
__device__ __forceinline__ T load(const uint8_t* src) {
  const T* s = reinterpret_cast<const T*>(src);
  if constexpr (ONCE) return __builtin_nontemporal_load(s);
  else return *s;
}
template <bool ONCE, int N>
__device__ __forceinline__ void load_words(const uint8_t* src, uint32_t (&w)[N]) {
  if constexpr (N == 1) w[0] = load<ONCE, uint32_t>(src);
  else if constexpr (N == 2) {
    const u32x2_t u = load<ONCE, u32x2_t>(src);
    w[0] = u[0];
    w[1] = u[1];
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4_t u = load<ONCE, u32x4_t>(src + 16 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[4 * i + j] = u[j];
    }
  }
}

// Sequence of a row: the last one that starts at or before it (decode steps
// have one row a sequence: look there first).
__device__ __forceinline__ int seq_of(const kvtc_mx_batch& b, int row) {
  int lo = 0, hi = b.n_seqs - 1;
  const int g = min(row, hi);
  if (b.row_start[g] <= row) {
    if (g == hi || b.row_start[g + 1] > row) return g;
    lo = g;
  } else hi = max(g - 1, 0);
  while (lo < hi) {
    const int m = (lo + hi + 1) >> 1;
    if (b.row_start[m] <= row) lo = m;
    else hi = m - 1;
  }
  return lo;
}

// Tokens that row i of a sequence attends to (not of a draft).
__device__ __forceinline__ int limit_of(const MxSeq& s, int i, int causal) {
  return causal ? max(s.len - s.n + i + 1, 0) : s.len;
}

// Least and greatest value of a 16-lane row.
__device__ __forceinline__ int row_min(int v) {
  v = min(v, (int)xor16_u32<1>((uint32_t)v));
  v = min(v, (int)xor16_u32<2>((uint32_t)v));
  v = min(v, (int)xor16_u32<4>((uint32_t)v));
  return min(v, (int)xor16_u32<8>((uint32_t)v));
}
__device__ __forceinline__ int row_max(int v) { return -row_min(-v); }

// The 16 NT query rows from r0 on, column n of each tile in lane n: tensor
// row (-1 for none), query head, tokens it attends to.  lo, hi: every row
// attends to the tokens below lo, none to those from hi on.  TREE, rows of
// drafts: those below lim that its mask names from `base` on, all before it.
template <int NT, bool TREE>
struct Rows {
  int at[NT], head[NT], lim[NT], lo, hi;
  int base[TREE ? NT : 0];
};
template <int NT, bool TREE>
__device__ __forceinline__ Rows<NT, TREE> rows_of(const MxAttnParams& p, const MxSeq& sq, int h, int r0, int rows, int n) {
  Rows<NT, TREE> o;
  o.lo = 0x7FFFFFFF;
  o.hi = 0;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = r0 + 16 * t + n, i = r / p.G;
    o.at[t] = -1;
    o.head[t] = h * p.G + r - i * p.G;
    o.lim[t] = 0;
    if constexpr (TREE) o.base[t] = 0;
    if (r < rows) {
      if (p.prefix) {
        const MxSeq s = mx_seq(p.b, seq_of(p.b, i), p.status);
        if (i >= s.row0 && i < s.row0 + s.n) {
          o.at[t] = i;
          o.lim[t] = TREE ? s.len : limit_of(s, i - s.row0, p.causal);
          if constexpr (TREE) o.base[t] = s.len - s.n;
        }
      } else {
        o.at[t] = sq.row0 + i;
        o.lim[t] = TREE ? sq.len : limit_of(sq, i, p.causal);
        if constexpr (TREE) o.base[t] = sq.len - sq.n;
      }
    }
    if (o.at[t] >= 0) o.lo = min(o.lo, TREE ? o.base[t] : o.lim[t]);
    o.hi = max(o.hi, o.lim[t]);
  }
  o.lo = __builtin_amdgcn_readfirstlane(row_min(o.lo));
  o.hi = __builtin_amdgcn_readfirstlane(row_max(o.hi));
  return o;
}

// Which of the tokens t .. t + 3 a draft's row has before it or in its mask,
// bits 0 to 3 (its sequence's length is the caller's to look at).  Only the
// few tiles that reach into a draft ask, so the words are read where they are
// needed: two neighbouring ones, shifted.
__device__ __forceinline__ uint32_t seen4(const MxAttnParams& p, int row, int base, int t) {
  const int j = t - base;
  if (j <= -4) return 15;
  if (row < 0) return 0;
  const uint32_t* m = p.masks + (int64_t)row * p.words;
  const int w = j >> 5;  // -1: tokens before the draft
  const uint32_t lo = w < 0 ? ~0u : w < p.words ? m[w] : 0, hi = w + 1 < p.words ? m[w + 1] : 0;
  return __builtin_amdgcn_alignbit(hi, lo, j & 31) & 15;
}

// Eight fp32 values as one bf16 operand, or as three whose sum keeps 24 bits.
// One for bf16 outputs: rounding a weight costs half a step of 2^-8 of it, and
// an average of values off by at most that is what the output is rounded to
// anyway; the sum l is of the unrounded weights, in fp32.  Against 64 bits the
// outputs are off by 0.0023 of their norm, 0.0017 from their own rounding
// alone.  A second part takes the rest away at the price of half the
// products again: 2048 rows on 4096 tokens 181 -> 232 us, 16 prompts of 1024
// 209 -> 253, 64 sequences of 511 to 8191 tokens 65.5 -> 68.1, with 5 rows
// each 79 -> 85; callers who need more than that have fp32.  Three for fp32.
template <int NP>
__device__ __forceinline__ void split8(float (&x)[8], bf16x8_t (&o)[NP]) {
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
      if (k + 1 < NP) {
        x[2 * i] = rest(x[2 * i], u[i], 0);
        x[2 * i + 1] = rest(x[2 * i + 1], u[i], 1);
      }
    }
    o[k] = operand(u[0], u[1], u[2], u[3]);
  }
}

// A query operand: 8 channels at `off` of q, zeros for no row.
template <bool F32>
__device__ __forceinline__ void load_query(const MxAttnParams& p, int64_t off, bool on, bf16x8_t (&q)[F32 ? 3 : 1]) {
  if constexpr (!F32) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (on) w = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.q) + off);
    q[0] = __builtin_bit_cast(bf16x8_t, w);
  } else {
    float4 x[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    if (on) {
      const float4* src = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.q) + off);
      x[0] = src[0];
      x[1] = src[1];
    }
    float f[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    split8<3>(f, q);
  }
}

// Where a lane finds its share of a record.
template <int D, int BK, int BV>
struct Share {
  static constexpr MxRecord R = mx_record(D, BK, BV);
  static constexpr int KW = D * BK / 128, VW = D * BV / 128;  // words of keys and values
  int k, v, ks, vs;
  __device__ __forceinline__ Share(int n, int kg)
      : k(n * (D * BK / 8) + kg * KW * 4),
        v(R.kc + (kg * 16 + n) * VW * 4),
        ks(R.kc + R.vc + n * (D / 32) + kg * (D / 32) / 4),
        vs(R.kc + R.vc + R.sc + (kg * (D / 32) + n * (D / 16) / 32) * 4) {}
};

// Value words of a lane: token i of its four without value, scale 1.
template <int VW>
__device__ __forceinline__ void drop(uint32_t (&v)[VW], uint32_t& vs, int i) {
  if constexpr (VW == 2) v[i / 2] &= (i & 1) ? 0x0000FFFFu : 0xFFFF0000u;
  else {
#pragma unroll
    for (int w = 0; w < VW / 4; ++w) v[i * (VW / 4) + w] = 0;
  }
  vs = (vs & ~(0xFFu << (8 * i))) | (0x7Fu << (8 * i));
}
__device__ __forceinline__ bool nan_scale(uint32_t vs, int i) { return ((vs >> (8 * i)) & 0xFFu) == 0xFFu; }

// Channel pair c2 of the lane's entry at its four tokens, a word per channel
// and token pair: even channel in x[0], x[1], odd channel in x[2], x[3].
template <int D, int BV, int c2, int VW>
__device__ __forceinline__ void value_words(const uint32_t (&v)[VW], uint32_t vs, uint32_t (&x)[4]) {
  constexpr int C = D / 16;
  uint32_t y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float sc = __uint_as_float(((vs >> (8 * i)) & 0xFFu) << 23);
    if constexpr (BV == 4 && C == 8) y[i] = two<4, c2>(v[i], sc);
    else if constexpr (BV == 4) y[i] = (i & 1) ? two<4, 2 + c2>(v[i / 2], sc) : two<4, c2>(v[i / 2], sc);
    else y[i] = two<8, c2 & 1>(v[i * (C / 4) + c2 / 2], sc);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[i] = __builtin_amdgcn_perm(y[2 * i + 1], y[2 * i], 0x05040100u);
    x[2 + i] = __builtin_amdgcn_perm(y[2 * i + 1], y[2 * i], 0x07060302u);
  }
}

// Rows of a score tile that attend to a NaN value: bit 4 t + b for channel
// block b.  vs: the value scales of the lane's four tokens of a page.
template <int D, int NT, bool TREE>
__device__ __forceinline__ void mark_poison(const MxAttnParams& p, const uint8_t* vs, int t0, int have, const Rows<NT, TREE>& rw,
                                            uint32_t& poison) {
  for (int i = 0; i < 4; ++i)
    if (i < have)
      for (int b = 0; b < D / 32; ++b)
        if (vs[4 * b + i] == 0xFFu) {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            bool sees = t0 + i < rw.lim[t];
            if constexpr (TREE) sees = sees && ((seen4(p, rw.at[t], rw.base[t], t0) >> i) & 1u);
            if (sees) poison |= 1u << (4 * t + b);
          }
        }
}

// Running softmax of NT tiles over a pair of pages: scores in, weights out as
// PV operands.  One vote decides whether any maximum has to move.
template <int NT, int C, int NP>
struct Softmax {
  float m[NT], l[NT], raise[NT];  // raise: the score from which on the maximum moves
  __device__ __forceinline__ Softmax() {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t] = kLow;
      raise[t] = -INFINITY;
      l[t] = 0.f;
    }
  }
  __device__ __forceinline__ void step(const f32x4_t (&s)[NT][2], float c, float inv_c, f32x4_t (&acc)[NT][C],
                                       bf16x8_t (&pf)[NT][NP]) {
    float mx[NT];
    bool up = false;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      // NaN here leaves the maximum as it is: the row's sum becomes NaN anyway
      mx[t] = max3(max3(s[t][0][0], s[t][0][1], s[t][0][2]), max3(s[t][0][3], s[t][1][0], s[t][1][1]),
                   max2(s[t][1][2], s[t][1][3]));
      up |= mx[t] > raise[t];
    }
    if (__builtin_amdgcn_ballot_w64(up)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float x = mx[t] * c;
        x = fmaxf(x, __shfl_xor(x, 16));
        x = fmaxf(x, __shfl_xor(x, 32));
        const float nm = fmaxf(m[t], x), a = __builtin_amdgcn_exp2f(m[t] - nm);
        m[t] = nm;
        raise[t] = (nm + kSlack) * inv_c;
        l[t] *= a;
#pragma unroll
        for (int j = 0; j < C; ++j) acc[t][j] *= a;
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __builtin_amdgcn_exp2f(__fmaf_rn(s[t][i / 4][i % 4], c, -m[t]));
      l[t] += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
      split8<NP>(w, pf[t]);
    }
  }
};

// Scores of tokens that a row does not attend to: `top` of the lane's four
// tokens of a page count.
__device__ __forceinline__ void mask(f32x4_t& s, int top) {
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = i < top ? s[i] : -INFINITY;
}
__device__ __forceinline__ void mask(f32x4_t& s, int top, uint32_t seen) {
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = i < top && ((seen >> i) & 1u) ? s[i] : -INFINITY;
}

// A row's result: the partial sums, or o / L and the log-sum-exp.
template <bool F32, int N>
__device__ __forceinline__ void store_row(float* ws_o, void* out, int64_t at, int D, int c0, const float (&o)[N], float L) {
  if (ws_o) {
    float4* d = reinterpret_cast<float4*>(ws_o + at * D + c0);
#pragma unroll
    for (int j = 0; j < N / 4; ++j) d[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
    return;
  }
  const float r = L == 0.f ? 0.f : 1.0f / L;
  if constexpr (F32) {
    float4* d = reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + at * D + c0);
#pragma unroll
    for (int j = 0; j < N / 4; ++j) d[j] = make_float4(o[4 * j] * r, o[4 * j + 1] * r, o[4 * j + 2] * r, o[4 * j + 3] * r);
  } else {
    uint2* d = reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(out) + at * D + c0);
#pragma unroll
    for (int j = 0; j < N / 4; ++j)
      d[j] = make_uint2(pack_bf16(o[4 * j] * r, o[4 * j + 1] * r), pack_bf16(o[4 * j + 2] * r, o[4 * j + 3] * r));
  }
}
__device__ __forceinline__ float log_sum(float M, float L) {
  return L == 0.f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * kLn2;
}

// What a workgroup works on.  Heads vary fastest, so that (with 8 of them) a
// head's tiles stay on one XCD and its pages in one L2.  The last tiles,
// longest when causal, come first; where all workgroups are on the card at
// once, two a CU, the second half goes the other way, so that a long tile
// shares its CU with a short one.
struct Work {
  int h, tile, split, z;
};
__device__ __forceinline__ Work work_of(const MxAttnParams& p, int b) {
  Work w;
  w.h = b % p.H;
  b /= p.H;
  w.tile = b % p.tiles;
  if (!p.fold || 2 * w.tile < p.tiles) w.tile = p.tiles - 1 - w.tile;
  else w.tile -= (p.tiles + 1) / 2;
  b /= p.tiles;
  w.split = b % p.nsplit;
  w.z = b / p.nsplit;
  return w;
}

// The sequence that is number `rank` (below n_seqs, at most 256 of them) when
// they are taken from the longest on, to 1/256 of max_len, equal ones in their
// order.  Every wave finds it for itself.
__device__ __forceinline__ int by_length(const kvtc_mx_batch& b, int rank) {
  const int lane = threadIdx.x & 63, shift = max(24 - __builtin_clz(b.max_len | 1), 0);
  int key[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int i = 64 * w + lane;
    key[w] = i < b.n_seqs ? min(max(b.kv_lens[i], 0), b.max_len) >> shift : -1;
  }
  auto at_least = [&](int v) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      if (64 * w < b.n_seqs) n += __builtin_popcountll(__builtin_amdgcn_ballot_w64(key[w] >= v));
    return n;
  };
  int v = 0;
#pragma unroll
  for (int bit = 128; bit; bit >>= 1)
    if (at_least(v + bit) > rank) v += bit;
  int left = rank - at_least(v + 1), z = 0;  // those of length v that come before it
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint64_t same = __builtin_amdgcn_ballot_w64(key[w] == v);
    const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0));
    const uint64_t it = __builtin_amdgcn_ballot_w64(key[w] == v && before == left);
    if (it) z = 64 * w + __builtin_ctzll(it);
    left -= __builtin_popcountll(same);
  }
  return z;
}

// Few rows: one pass over the codes with as many loads in flight as the
// registers allow.  The W waves take pairs of pages in turn, all for the same
// 16 NT rows, and are joined at the end.  Bound by memory where the card is
// full (64 sequences of 511 to 8191 tokens and 8 heads, 4 bits: 309 MB in 62 us,
// 5.0 TB/s; one of 131072, keys in 8 bits: 210 MB in 40 us, 5.2 TB/s), by vector
// issue (173 instructions a wave and 32 tokens, about 45 GB/s a CU) where a
// unit has one workgroup, and by the launch and four loads in a row (row
// bounds, page numbers, codes, values) at a few hundred tokens (500: 6.5 us).
// The smallest parts of 32 fp32 queries of 128 channels stay in LDS, for the
// registers (64 sequences of 3 rows and 3000 tokens, k8v8: 119 -> 99 us).
template <int D, int NT, bool F32>
constexpr bool few_tight = F32 && D == 128 && NT == 2;
template <int D, int NT, bool F32, int W>
struct FewShared {
  uint4 q[few_tight<D, NT, F32> ? NT : 0][D / 32][64];  // row tile, contraction step, lane
  float o[W * 16 * (D + 4)];
  float2 ml[W][16];
};
template <int D, int BK, int BV, int NT, bool F32, bool ONCE, int W, bool TREE>
__device__ __forceinline__ void few_rows(const MxAttnParams& p, int block, FewShared<D, NT, F32, W>& lds) {
  using Sh = Share<D, BK, BV>;
  constexpr MxRecord R = Sh::R;
  constexpr int C = D / 16;       // channels of an entry of the value groups
  constexpr int KS = D / 32;      // contraction steps of S
  constexpr int NP = F32 ? 3 : 1;  // bf16 parts of queries and weights
  constexpr int OS = D + 4;       // row stride of the joining buffer
  constexpr bool TIGHT = few_tight<D, NT, F32>;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int n = lane & 15, kg = lane >> 4;
  Work wk = work_of(p, block);
  const int h = wk.h;
  if constexpr (W == 4)
    if (p.pair) wk.z = by_length(p.b, wk.z < p.pair ? p.pair - 1 - wk.z : wk.z);

  const int Hq = p.H * p.G;
  MxSeq sq{0, 0, 0};
  if (!p.prefix) sq = mx_seq(p.b, wk.z, p.status);
  const int rows = (p.prefix ? p.b.total_rows : sq.n) * p.G;
  const int r0 = wk.tile * 16 * NT;
  if (r0 >= rows) return;
  const Rows<NT, TREE> rw = rows_of<NT, TREE>(p, sq, h, r0, rows, n);
  const int begin = p.begin + wk.split * p.chunk;
  const int end = min(min(p.end, begin + p.chunk), rw.hi);
  if (p.ws_o && begin >= end) return;

  const int32_t* table = p.b.page_table + (p.prefix ? 0 : (int64_t)wk.z * p.b.max_pages);
  const uint8_t* head = p.pool + (int64_t)h * R.bytes;
  const int64_t page_bytes = (int64_t)p.H * R.bytes;
  const Sh sh(n, kg);
  const int p1 = (end + KVTC_MX_PAGE - 1) / KVTC_MX_PAGE;  // end of the range's pages
  const int q0 = begin / KVTC_MX_PAGE + 2 * wave;          // this wave takes pages q0 + 2 W k and the one after
  const int steps = (p1 - q0 + 2 * W - 1) / (2 * W);       // (not positive: none)

  // Page numbers: those of 32 steps at a time, one a lane, the next 32 steps'
  // on their way; -1 past the range and, once reported, outside the pool
  // (such pages are read as page 0 and masked).
  auto load_ids = [&](int step) {
    const int pg = q0 + (step + (lane >> 1)) * 2 * W + (lane & 1);
    int id = -1;
    if (pg < p1) {
      id = table[pg];
      if ((uint32_t)id >= (uint32_t)p.pool_pages) {
        if (p.status) atomicOr(p.status, 1u << KVTC_ERR_INVALID_ARG);
        id = -1;
      }
    }
    return id;
  };
  // A lane's share of a step's two pages as it lies in their records.  The
  // keys of the next step are requested as soon as this step's have become
  // operands, its values at the end of this step (after the last step, page 0:
  // a condition would make the loop wait for the loads).
  int id[2];
  uint32_t k[2][Sh::KW], v[2][Sh::VW], ks[2], vs[2];
  int ids = load_ids(0), ids2 = load_ids(32);
  auto load_keys = [&](int step, bool later) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      id[e] = __builtin_amdgcn_readlane(later ? ids2 : ids, 2 * (step & 31) + e);
      const uint8_t* rec = head + max(id[e], 0) * page_bytes;
      load_words<ONCE>(rec + sh.k, k[e]);
      ks[e] = load<ONCE, uint8_t>(rec + sh.ks);
    }
  };
  auto load_values = [&]() {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint8_t* rec = head + max(id[e], 0) * page_bytes;
      load_words<ONCE>(rec + sh.v, v[e]);
      vs[e] = load<ONCE, uint32_t>(rec + sh.vs);
    }
  };

  bf16x8_t qf[NT][KS][NP];
  // channels (D / 4) kg + 8 s .. + 7 of the lane's rows
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int s = 0; s < KS; ++s)
      load_query<F32>(p, rw.at[t] * p.q_stride + rw.head[t] * D + (D / 4) * kg + 8 * s, rw.at[t] >= 0, qf[t][s]);
  if constexpr (TIGHT) {  // (all waves have the same rows)
    if (wave == 0)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int s = 0; s < KS; ++s) lds.q[t][s][lane] = __builtin_bit_cast(uint4, qf[t][s][2]);
    __syncthreads();
  }
  if (steps > 0) {
    load_keys(0, false);
    load_values();
  }

  f32x4_t acc[NT][C];
  Softmax<NT, C, NP> sm;
  const float inv_c = 1.0f / p.c;
  uint32_t poison = 0;  // bit 4 t + b: a value of channel block b was NaN at a token that row t attends to
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int j = 0; j < C; ++j) acc[t][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  for (int step = 0; step < steps; ++step) {
    if (step && (step & 31) == 0) {
      ids = ids2;
      ids2 = load_ids(step + 32);
    }
    const int t0 = (q0 + 2 * W * step) * KVTC_MX_PAGE;
    // tokens of page e that exist for this workgroup, 0 .. 16
    int have[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) have[e] = id[e] < 0 ? 0 : min(max(end - t0 - 16 * e, 0), 16);
    const bool whole = have[0] + have[1] == 32 && t0 + 32 <= rw.lo;

    if (!whole) {
      // Values of tokens that no row attends to may be anything: make them 0.
      // A NaN value that only some rows attend to: 0 in the product, and a
      // mark for the rows that do.
      bool nan = false;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (4 * kg + i >= have[e]) drop(v[e], vs[e], i);
          nan |= nan_scale(vs[e], i);
        }
      if (__builtin_amdgcn_ballot_w64(nan)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mark_poison<D, NT, TREE>(p, head + max(id[e], 0) * page_bytes + R.kc + R.vc + R.sc + kg * (D / 32) * 4,
                                   t0 + 16 * e + 4 * kg, have[e] - 4 * kg, rw, poison);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (nan_scale(vs[e], i)) drop(v[e], vs[e], i);
        }
      }
    }

    f32x4_t sa[NT][2];
    int ql = lane;
    if constexpr (TIGHT) asm volatile("" : "+v"(ql));  // read in every step, not kept from the first
    {
      bf16x8_t kf[2][KS];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float sc = __uint_as_float(ks[e] << 23);
#pragma unroll
        for (int s = 0; s < KS; ++s) kf[e][s] = eight<BK>(k[e] + s * (BK / 4), sc);
      }
      load_keys(step + 1, ((step + 1) ^ step) & 32);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        sa[t][0] = sa[t][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kp = NP - 1; kp >= 0; --kp)  // small parts first
#pragma unroll
          for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              bf16x8_t q = qf[t][s][kp];
              if constexpr (TIGHT)
                if (kp == 2) q = __builtin_bit_cast(bf16x8_t, lds.q[t][s][ql]);
              sa[t][e] = mfma(kf[e][s], q, sa[t][e]);
            }
      }
    }
    if (!whole) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int top = min(rw.lim[t] - t0 - 16 * e, have[e]) - 4 * kg;
          if constexpr (TREE) mask(sa[t][e], top, seen4(p, rw.at[t], rw.base[t], t0 + 16 * e + 4 * kg));
          else mask(sa[t][e], top);
        }
    }
    bf16x8_t pf[NT][NP];
    sm.step(sa, p.c, inv_c, acc, pf);

    auto channels = [&](auto ic) {
      constexpr int c2 = decltype(ic)::value;
      uint32_t a[4], b[4];
      value_words<D, BV, c2>(v[0], vs[0], a);
      value_words<D, BV, c2>(v[1], vs[1], b);
      const bf16x8_t ev = operand(a[0], a[1], b[0], b[1]), od = operand(a[2], a[3], b[2], b[3]);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int kp = NP - 1; kp >= 0; --kp) {
          acc[t][2 * c2] = mfma(ev, pf[t][kp], acc[t][2 * c2]);
          acc[t][2 * c2 + 1] = mfma(od, pf[t][kp], acc[t][2 * c2 + 1]);
        }
    };
    channels(std::integral_constant<int, 0>{});
    channels(std::integral_constant<int, 1>{});
    if constexpr (C == 8) {
      channels(std::integral_constant<int, 2>{});
      channels(std::integral_constant<int, 3>{});
    }
    load_values();
  }

  // ---- join the waves, 16 rows at a time
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float sum = sm.l[t];
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    uint32_t pz = poison >> (4 * t);
    pz |= (uint32_t)__shfl_xor((int)pz, 16);
    pz |= (uint32_t)__shfl_xor((int)pz, 32);
    const bool dead = (pz >> (kg * (D / 32) / 4)) & 1u;  // this lane's channels [kg D / 4, (kg + 1) D / 4)
    if (t) __syncthreads();                              // the buffer is free
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < C; j += 4) {
        float4 o = make_float4(acc[t][j][i], acc[t][j + 1][i], acc[t][j + 2][i], acc[t][j + 3][i]);
        if (dead) o = make_float4(NAN, NAN, NAN, NAN);
        *reinterpret_cast<float4*>(&lds.o[(wave * 16 + n) * OS + C * (4 * kg + i) + j]) = o;
      }
    if (kg == 0) lds.ml[wave][n] = make_float2(sm.m[t], sum);
    const int r = (threadIdx.x >> 4) & 15, c0 = (threadIdx.x & 15) * C;
    const int row = __shfl(rw.at[t], r), hq = __shfl(rw.head[t], r);
    __syncthreads();
    if (row < 0 || wave >= 4) continue;
    const int64_t at = (int64_t)row * Hq + hq;
    float M = kLow, L = 0.f, a[W];
#pragma unroll
    for (int w = 0; w < W; ++w) M = fmaxf(M, lds.ml[w][r].x);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      a[w] = __builtin_amdgcn_exp2f(lds.ml[w][r].x - M);
      L = __fmaf_rn(a[w], lds.ml[w][r].y, L);
    }
    float o[C];
#pragma unroll
    for (int j = 0; j < C; j += 4) {
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(&lds.o[(w * 16 + r) * OS + c0 + j]);
        s.x = __fmaf_rn(a[w], x.x, s.x);
        s.y = __fmaf_rn(a[w], x.y, s.y);
        s.z = __fmaf_rn(a[w], x.z, s.z);
        s.w = __fmaf_rn(a[w], x.w, s.w);
      }
      o[j] = s.x;
      o[j + 1] = s.y;
      o[j + 2] = s.z;
      o[j + 3] = s.w;
    }
    const int64_t slot = (int64_t)(p.slot0 + wk.split) * p.b.total_rows * Hq;
    store_row<F32>(p.ws_o ? p.ws_o + slot * D : nullptr, p.out, at, D, c0, o, L);
    if (c0 == 0) {
      if (p.ws_o) p.ws_ml[slot + at] = make_float2(M, L);
      else if (p.lse) p.lse[at] = log_sum(M, L);
    }
  }
}

template <int D, int BK, int BV, int NT, bool F32, bool ONCE, int W, bool TREE>
__global__ __launch_bounds__(W * 64, W == 4 && NT == 1 && !F32 ? 3 : 2) void k_mx_attn(const MxAttnParams p) {
  __shared__ __attribute__((aligned(16))) FewShared<D, NT, F32, W> lds;
  few_rows<D, BK, BV, NT, F32, ONCE, W, TREE>(p, blockIdx.x, lds);
}

// Many rows: bound by the issue of matrix and vector instructions (2048 rows
// of 4 heads on 4096 tokens before them: 173 GFLOP in 174 to 196 us, as the
// clock allows; the matrix unit is busy for 42% of the clocks, vector
// instructions issue in 51%, two waves a SIMD).  A workgroup takes 128 rows, 32 a wave, and walks over the tokens 32 at a
// time; each wave turns half of a page into operands in LDS, in the order in
// which all four read them back, so a code is converted once for 128 rows.
// Three buffers, so that in one stretch between barriers a wave multiplies
// the keys of tile t + 1, weighs the scores of tile t, multiplies its values
// and converts tile t + 2: matrix and vector work of the same wave overlap.
//
// v_mfma_f32_32x32x16_bf16 (half the instructions of the 16-row form): S^T
// has the two pages' tokens as rows; lane (hh, q) = (lane / 32, lane % 32)
// gets tokens 4 hh .. + 3 and 8 + 4 hh .. + 3 of each page for query row q,
// the slice of P^T that the product with 16 tokens' values takes from it.
// Value rows of a 32-channel product: row n + 16 o is channel 2 ct + o of
// entry n of the value groups.
// fp32 queries of 128 channels do not fit the registers next to the rest: the
// smallest parts of all but 16 channels go to LDS, as many as leave room for
// two workgroups a CU, and one tile's codes are on their way instead of three
// (2048 rows on 4096 tokens: k4v4 545 -> 490 us, k8v8 706 -> 455; 64 channels
// fit: 241 us, 250 this way).  k4v4 fits so, the other formats are still 1 to 5
// registers too many (8 to 24 bytes of scratch a lane; with masks up to 3, both
// passes of drafts in one launch up to 9).  An earlier form, with 9 to 12
// spilled, took the same beside it on one card: 411 (k4v4) to 425 us (k8v8).
template <int D, bool F32>
constexpr bool many_tight = F32 && D == 128;
template <int D, bool F32>
struct ManyShared {
  uint4 q[4][many_tight<D, F32> ? D / 16 - 1 : 0][64];  // wave, contraction step, lane
  struct Tile {
    uint4 k[D / 16][64];     // contraction step, operand lane
    uint4 v[2][D / 32][64];  // page, channel tile, operand lane
    int2 state[2];           // per page and half: tokens that exist, bit 8 if a NaN value was taken out
  };
  union {
    Tile tile[3];
    float o[4 * 32 * (D / 2 + 4)];  // wave, row, half of the channels
  };
  int2 bounds[4];
  int odd[4];  // per wave: it met a page outside the pool, so every tile's state is looked at
};
template <int D, int BK, int BV, bool F32, bool TREE>
__device__ __forceinline__ void many_rows(const MxAttnParams& p, int block, ManyShared<D, F32>& lds) {
  using Sh = Share<D, BK, BV>;
  constexpr MxRecord R = Sh::R;
  constexpr int C = D / 16, KS = D / 32, QS = D / 16, CT = D / 32, NP = F32 ? 3 : 1;
  constexpr bool TIGHT = many_tight<D, F32>;
  constexpr int NR = TIGHT ? 1 : 3;  // codes of so many tiles in registers

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int n = lane & 15, kg = lane >> 4, hh = lane >> 5;
  using Tile = typename ManyShared<D, F32>::Tile;
  Tile(&tile)[3] = lds.tile;
  const Work wk = work_of(p, block);
  const int h = wk.h;

  const int Hq = p.H * p.G;
  MxSeq sq{0, 0, 0};
  if (!p.prefix) sq = mx_seq(p.b, wk.z, p.status);
  const int rows = (p.prefix ? p.b.total_rows : sq.n) * p.G;
  if (wk.tile * 128 >= rows) return;
  const int begin = p.begin + wk.split * p.chunk;
  int end = min(begin + p.chunk, p.prefix ? p.end : sq.len);

  // This wave converts half `half` (of a lane's key channels and of the value
  // channel pairs) of page p0 + 2 t + own of tile t: the numbers of 64 tiles,
  // one a lane, the next 64 on their way; -1 as in few_rows.  They and the
  // first pages are asked for before the rows are looked up.
  const int32_t* table = p.b.page_table + (p.prefix ? 0 : (int64_t)wk.z * p.b.max_pages);
  const uint8_t* head = p.pool + (int64_t)h * R.bytes;
  const int64_t page_bytes = (int64_t)p.H * R.bytes;
  const Sh sh(n, kg);
  const int p0 = begin / KVTC_MX_PAGE, p1 = (end + KVTC_MX_PAGE - 1) / KVTC_MX_PAGE;
  const int own = wave & 1, half = wave >> 1;
  auto load_ids = [&](int t, bool& bad) {
    const int pg = p0 + (t + lane) * 2 + own;
    int id = -1;
    if (pg < p1) {
      id = table[pg];
      if ((uint32_t)id >= (uint32_t)p.pool_pages) {
        if (p.status) atomicOr(p.status, 1u << KVTC_ERR_INVALID_ARG);
        id = -1;
        bad = true;
      }
    }
    return id;
  };
  bool bad = false;
  int ids = load_ids(0, bad), ids2 = load_ids(64, bad);
  {
    const uint64_t any = __builtin_amdgcn_ballot_w64(bad);
    if (lane == 0) lds.odd[wave] = any != 0;
  }
  auto id_of = [&](int t) {  // called for every t in turn
    if (t && (t & 63) == 0) {
      ids = ids2;
      bool more = false;
      ids2 = load_ids(t + 64, more);
      if (more) lds.odd[wave] = 1;
    }
    return __builtin_amdgcn_readlane(ids, t & 63);
  };
  struct Raw {
    int id;
    uint32_t k[Sh::KW / 2], v[Sh::VW], ks, vs;
  };
  auto load_page = [&](Raw& g, int id) {
    g.id = id;
    const uint8_t* rec = head + max(id, 0) * page_bytes;
    load_words<false>(rec + sh.k + half * Sh::KW * 2, g.k);
    load_words<false>(rec + sh.v, g.v);
    g.ks = rec[sh.ks];
    g.vs = *reinterpret_cast<const uint32_t*>(rec + sh.vs);
  };
  // Codes of tile t in raw[t % NR]: those of tile t + 2 are converted while
  // those of t + 3 and t + 4 are on their way (2000 clocks from the request
  // on); TIGHT: then those of t + 3 are requested, a step ahead, which takes
  // as long with three times the products.
  Raw raw[NR];
#pragma unroll
  for (int t = 0; t < NR; ++t) load_page(raw[t], id_of(t));

  Rows<1, TREE> rw = rows_of<1, TREE>(p, sq, h, wk.tile * 128 + wave * 32, rows, lane & 31);
  {  // rows_of looks at the first 16 lanes
    int lo = 0x7FFFFFFF;
    if constexpr (TREE) lo = rw.at[0] >= 0 ? rw.base[0] : lo;
    else lo = rw.at[0] >= 0 ? rw.lim[0] : lo;
    rw.lo = min(rw.lo, __builtin_amdgcn_readlane(row_min(lo), 16));
    rw.hi = max(rw.hi, __builtin_amdgcn_readlane(row_max(rw.lim[0]), 16));
  }
  // queries: channels 16 s + 8 hh .. + 7 of the lane's row
  bf16x8_t qf[QS][NP];
#pragma unroll
  for (int c = 0; c < QS; ++c)
    load_query<F32>(p, rw.at[0] * p.q_stride + rw.head[0] * D + 16 * c + 8 * hh, rw.at[0] >= 0, qf[c]);
  if constexpr (TIGHT)  // (only this wave reads them)
#pragma unroll
    for (int c = 0; c < QS - 1; ++c) lds.q[wave][c][lane] = __builtin_bit_cast(uint4, qf[c][2]);
  if (lane == 0) lds.bounds[wave] = make_int2(rw.lo, rw.hi);
  __syncthreads();
  int lo = 0x7FFFFFFF, hi = 0;  // of all four waves
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    lo = min(lo, lds.bounds[w].x);
    hi = max(hi, lds.bounds[w].y);
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  end = min(end, __builtin_amdgcn_readfirstlane(hi));
  if (p.ws_o && begin >= end) return;
  const int tiles = (end - p0 * KVTC_MX_PAGE + 31) / 32;

  // what must not reach the products, as in few_rows; each wave marks its own rows
  auto clean = [&](Raw& g, int t, Tile& to) {
    const int t0 = (p0 + 2 * t + own) * KVTC_MX_PAGE;
    const int have = g.id < 0 ? 0 : min(max(end - t0, 0), 16);
    int state = have;
    if (have < 16 || t0 + 16 > lo) {
      bool nan = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (4 * kg + i >= have) drop(g.v, g.vs, i);
        if (nan_scale(g.vs, i)) {
          nan = true;
          drop(g.v, g.vs, i);
        }
      }
      if (__builtin_amdgcn_ballot_w64(nan)) state |= 256;
    }
    if (lane == 0) reinterpret_cast<int*>(&to.state[own])[half] = state;
  };
  auto convert = [&](const Raw& g, Tile& to) {
    const float sc = __uint_as_float(g.ks << 23);
#pragma unroll
    for (int i = 0; i < KS / 2; ++i) {  // channels 8 f .. + 7 of the lane's quarter: step f / 2, lane half f % 2
      const int f = half * (KS / 2) + i;
      to.k[(kg * KS + f) >> 1][(f & 1) * 32 + own * 16 + n] = __builtin_bit_cast(uint4, eight<BK>(g.k + i * (BK / 4), sc));
    }
    // the channel pairs of this half: the words move down, so that the pair is a constant
    uint32_t y[Sh::VW];
#pragma unroll
    for (int i = 0; i < Sh::VW; ++i) {
      if constexpr (BV == 8 && C == 8) y[i] = half ? g.v[i | 1] : g.v[i];
      else y[i] = g.v[i] >> (half * (BV * C / 2));
    }
    auto channels = [&](auto ic) {
      constexpr int c2 = decltype(ic)::value;
      uint32_t x[4];
      value_words<D, BV, c2>(y, g.vs, x);
      uint4* const to_v = &to.v[own][half * (C / 4) + c2][(kg & 1) * 32 + n];
      reinterpret_cast<uint2*>(to_v)[kg >> 1] = make_uint2(x[0], x[1]);
      reinterpret_cast<uint2*>(to_v + 16)[kg >> 1] = make_uint2(x[2], x[3]);
    };
    channels(std::integral_constant<int, 0>{});
    if constexpr (C == 8) channels(std::integral_constant<int, 1>{});
  };

  f32x16_t acc[CT], sa;
  float m = kLow, l = 0.f, raise = -INFINITY;
  const float inv_c = 1.0f / p.c;
  uint32_t poison = 0;  // bit b: a value of channel block b was NaN at a token that the lane's row attends to
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[c][i] = 0.f;
  auto scores = [&](const Tile& from, f32x16_t& s) {
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = 0.f;
#pragma unroll
    for (int kp = NP - 1; kp >= 0; --kp)  // small parts first
#pragma unroll
      for (int c = 0; c < QS; ++c) {
        bf16x8_t q = qf[c][kp];
        if constexpr (TIGHT)
          if (kp == 2 && c < QS - 1) q = __builtin_bit_cast(bf16x8_t, lds.q[wave][c][lane]);
        s = mfma(__builtin_bit_cast(bf16x8_t, from.k[c][lane]), q, s);
      }
  };

  if (tiles > 0) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      clean(raw[t % NR], t, tile[t]);
      convert(raw[t % NR], tile[t]);
      if (TIGHT) load_page(raw[0], id_of(t + 1));
    }
    if (!TIGHT) load_page(raw[0], id_of(3));
    __syncthreads();
    scores(tile[0], sa);
  }
  int slow = 0;
  auto step = [&](int t, auto bc) {
    constexpr int b = decltype(bc)::value;  // t % 3
    Tile &now = tile[b], &next = tile[(b + 1) % 3], &after = tile[(b + 2) % 3];
    Raw &use = raw[(b + 2) % NR], &load = raw[(b + 1) % NR];
    const int t0 = (p0 + 2 * t) * KVTC_MX_PAGE;
    // the page numbers of tile t were read at least 64 tiles, or the opening barrier, ago
    if ((t & 63) == 0) slow = __builtin_amdgcn_readfirstlane(lds.odd[0] | lds.odd[1] | lds.odd[2] | lds.odd[3]);
    // (by the bound of all four waves: `clean` may have taken a NaN out that this wave's rows attend to)
    if (slow || t0 + 32 > min(end, lo)) {
      const int2 s0 = now.state[0], s1 = now.state[1];
      const int st[2] = {__builtin_amdgcn_readfirstlane(s0.x | s0.y), __builtin_amdgcn_readfirstlane(s1.x | s1.y)};
      const int have[2] = {st[0] & 255, st[1] & 255};
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int e = i / 8, tok = 8 * ((i / 4) & 1) + 4 * hh, top = min(rw.lim[0] - t0 - 16 * e, have[e]) - tok;
        f32x4_t s = {sa[i], sa[i + 1], sa[i + 2], sa[i + 3]};
        if constexpr (TREE) mask(s, top, seen4(p, rw.at[0], rw.base[0], t0 + 16 * e + tok));
        else mask(s, top);
#pragma unroll
        for (int k = 0; k < 4; ++k) sa[i + k] = s[k];
      }
      if ((st[0] | st[1]) & 256)
        for (int e = 0; e < 2; ++e)
          if (have[e] > 0) {  // then its page is in the pool
            const uint8_t* vs = head + table[t0 / KVTC_MX_PAGE + e] * page_bytes + R.kc + R.vc + R.sc;
            for (int g = hh; g < 4; g += 2)
              mark_poison<D, 1, TREE>(p, vs + g * (D / 32) * 4, t0 + 16 * e + 4 * g, have[e] - 4 * g, rw, poison);
          }
    }
    {  // one vote on whether a maximum has to move
      const float mx = max2(max3(max3(sa[0], sa[1], sa[2]), max3(sa[3], sa[4], sa[5]), max3(sa[6], sa[7], sa[8])),
                            max3(max3(sa[9], sa[10], sa[11]), max3(sa[12], sa[13], sa[14]), sa[15]));
      if (__builtin_amdgcn_ballot_w64(mx > raise)) {
        float x = mx * p.c;
        x = fmaxf(x, __shfl_xor(x, 32));
        const float nm = fmaxf(m, x), a = __builtin_amdgcn_exp2f(m - nm);
        m = nm;
        raise = (nm + kSlack) * inv_c;
        l *= a;
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[c] *= a;
      }
    }
    if (!TIGHT) clean(use, t + 2, after);
    const int id = id_of(TIGHT ? t + 3 : t + 4);
    __syncthreads();  // tile t + 1 is in its buffer, nobody reads tile t - 1 any more
    if (!TIGHT) load_page(load, id);
    __builtin_amdgcn_sched_barrier(0);  // the loads first
    __builtin_amdgcn_s_setprio(1);
    float w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = __fmaf_rn(sa[i], p.c, -m);
    scores(next, sa);
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = __builtin_amdgcn_exp2f(w[i]);
    l += (((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]))) +
         (((w[8] + w[9]) + (w[10] + w[11])) + ((w[12] + w[13]) + (w[14] + w[15])));
    bf16x8_t pf[2][NP];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = w[8 * u + i];
      split8<NP>(x, pf[u]);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        const bf16x8_t vf = __builtin_bit_cast(bf16x8_t, now.v[u][c][lane]);
#pragma unroll
        for (int kp = NP - 1; kp >= 0; --kp) acc[c] = mfma(vf, pf[u][kp], acc[c]);
      }
    if (TIGHT) clean(use, t + 2, after);
    convert(use, after);
    if (TIGHT) load_page(use, id);
    __builtin_amdgcn_s_setprio(0);
  };
  for (int t = 0; t < tiles; t += 3) {
    step(t, std::integral_constant<int, 0>{});
    if (t + 1 < tiles) step(t + 1, std::integral_constant<int, 1>{});
    if (t + 2 < tiles) step(t + 2, std::integral_constant<int, 2>{});
  }

  // ---- a lane has channels C e .. of its row for the eight e = 8 a + 4 hh +
  // i.  bf16 outputs are stored from there, fp32 rows through LDS, half a row
  // at a time, in lines (partials of 64 rows of 4 heads on 8192 tokens: 25.6
  // -> 23.8 us; bf16 outputs of 16 prompts of 1024: 220 us, 222 that way).
  l += __shfl_xor(l, 32);
  poison |= (uint32_t)__shfl_xor((int)poison, 32);
  const int at = rw.at[0] < 0 ? -1 : rw.at[0] * Hq + rw.head[0];
  const int64_t slot = (int64_t)(p.slot0 + wk.split) * p.b.total_rows * Hq;
  const float r = p.ws_o ? 1.0f : l == 0.f ? 0.f : 1.0f / l;
  auto channels_of = [&](int a, int i, float (&o)[C]) {
    const bool dead = (poison >> ((8 * a + 4 * hh + i) * C / 32)) & 1u;
#pragma unroll
    for (int j = 0; j < C; ++j) o[j] = dead ? NAN : acc[j / 2][4 * (a + 2 * (j & 1)) + i] * r;
  };
  if (!F32 && !p.ws_o) {
    if (at < 0) return;
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float o[C];
        channels_of(a, i, o);
        uint2* const to = reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + (int64_t)at * D + C * (8 * a + 4 * hh + i));
#pragma unroll
        for (int j = 0; j < C / 4; ++j)
          to[j] = make_uint2(pack_bf16(o[4 * j], o[4 * j + 1]), pack_bf16(o[4 * j + 2], o[4 * j + 3]));
      }
  } else {
    float* const dst = p.ws_o ? p.ws_o + slot * D : reinterpret_cast<float*>(p.out);
    constexpr int OS = D / 2 + 4;  // row stride: sixteen rows in banks of their own
    constexpr int LR = D / 8;      // lanes of half a row
    float* const half_row = &lds.o[wave * 32 * OS];
    __syncthreads();  // the tiles are done with
#pragma unroll
    for (int a = 0; a < 2; ++a) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float o[C];
        channels_of(a, i, o);
#pragma unroll
        for (int j = 0; j < C; j += 4)
          *reinterpret_cast<float4*>(&half_row[(lane & 31) * OS + C * (4 * hh + i) + j]) =
              make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
      }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int k = 0; k < LR / 2; ++k) {
        const int row = k * (64 / LR) + lane / LR, c = lane % LR * 4, to = __shfl(at, row);
        const float4 o = *reinterpret_cast<const float4*>(&half_row[row * OS + c]);
        if (to >= 0) *reinterpret_cast<float4*>(dst + (int64_t)to * D + a * (D / 2) + c) = o;
      }
      __builtin_amdgcn_wave_barrier();
    }
    if (at < 0) return;
  }
  if (hh == 0) {
    if (p.ws_o) p.ws_ml[slot + at] = make_float2(m, l);
    else if (p.lse) p.lse[at] = log_sum(m, l);
  }
}
template <int D, int BK, int BV, bool F32, bool TREE>
__global__ __launch_bounds__(256, 2) void k_mx_rows(const MxAttnParams p) {
  __shared__ __attribute__((aligned(16))) ManyShared<D, F32> lds;
  many_rows<D, BK, BV, F32, TREE>(p, blockIdx.x, lds);
}

// Drafts of many rows behind a shared prefix: both passes in one launch, so
// that the short own ranges fill what the prefix's leave (32 sequences of 10
// to 25 rows and 4 heads behind 8192, a call with its join: 125 us one after
// the other, 109 so; fp32 260 and 230).
template <int D, int BK, int BV, bool F32>
__global__ __launch_bounds__(256, 2) void k_mx_rows_both(const MxAttnParams prefix, const MxAttnParams own, int prefix_blocks) {
  __shared__ __attribute__((aligned(16))) ManyShared<D, F32> lds;
  const bool first = (int)blockIdx.x < prefix_blocks;
  many_rows<D, BK, BV, F32, true>(first ? prefix : own, (int)blockIdx.x - (first ? 0 : prefix_blocks), lds);
}

// A decode step behind a shared prefix: the prefix for all rows together and
// each sequence's own tokens in one launch (one after the other they would
// leave the card half empty twice).
template <int D, int BK, int BV, bool F32, bool TREE>
__global__ __launch_bounds__(256, 2) void k_mx_both(const MxAttnParams prefix, const MxAttnParams own, int prefix_blocks) {
  __shared__ __attribute__((aligned(16))) union {
    ManyShared<D, F32> many;
    FewShared<D, 1, F32, 4> few;
  } lds;
  if ((int)blockIdx.x < prefix_blocks) many_rows<D, BK, BV, F32, TREE>(prefix, blockIdx.x, lds.many);
  else few_rows<D, BK, BV, 1, F32, false, 4, TREE>(own, (int)blockIdx.x - prefix_blocks, lds.few);
}

unsigned blocks_of(const MxAttnParams& p) {
  return (unsigned)p.H * p.tiles * p.nsplit * (p.prefix ? 1 : p.b.n_seqs);
}
template <int D, int BK, int BV, bool F32, bool TREE>
void launch_pass(const MxAttnParams& p, hipStream_t s) {
  const unsigned grid = blocks_of(p);
  if (p.nt == 1) {
    if (p.waves == 8) {
      if (p.once) k_mx_attn<D, BK, BV, 1, F32, true, 8, TREE><<<grid, 512, 0, s>>>(p);
      else k_mx_attn<D, BK, BV, 1, F32, false, 8, TREE><<<grid, 512, 0, s>>>(p);
    } else if (p.once) k_mx_attn<D, BK, BV, 1, F32, true, 4, TREE><<<grid, 256, 0, s>>>(p);
    else k_mx_attn<D, BK, BV, 1, F32, false, 4, TREE><<<grid, 256, 0, s>>>(p);
  } else if (p.nt == 2) k_mx_attn<D, BK, BV, 2, F32, false, 4, TREE><<<grid, 256, 0, s>>>(p);
  else k_mx_rows<D, BK, BV, F32, TREE><<<grid, 256, 0, s>>>(p);
}
template <int D, int BK, int BV, bool F32, bool TREE>
hipError_t launch_format(const MxAttnParams* prefix, const MxAttnParams* own, hipStream_t s) {
  if (prefix && own && own->together) {
    const unsigned n = blocks_of(*prefix);
    if constexpr (TREE)
      if (own->nt == 8) {
        k_mx_rows_both<D, BK, BV, F32><<<n + blocks_of(*own), 256, 0, s>>>(*prefix, *own, (int)n);
        return hipGetLastError();
      }
    k_mx_both<D, BK, BV, F32, TREE><<<n + blocks_of(*own), 256, 0, s>>>(*prefix, *own, (int)n);
    return hipGetLastError();
  }
  if (prefix) launch_pass<D, BK, BV, F32, TREE>(*prefix, s);
  if (own) launch_pass<D, BK, BV, F32, TREE>(*own, s);
  return hipGetLastError();
}
template <int D, int BK, int BV, bool TREE>
hipError_t launch_attn(const MxAttnParams* prefix, const MxAttnParams* own, bool f32, hipStream_t s) {
  return f32 ? launch_format<D, BK, BV, true, TREE>(prefix, own, s) : launch_format<D, BK, BV, false, TREE>(prefix, own, s);
}

template <int D, bool TREE>
hipError_t launch_any(const MxAttnParams* prefix, const MxAttnParams* own, int bk, int bv, bool f32, hipStream_t s) {
  if (bk == 4) return bv == 4 ? launch_attn<D, 4, 4, TREE>(prefix, own, f32, s) : launch_attn<D, 4, 8, TREE>(prefix, own, f32, s);
  return bv == 4 ? launch_attn<D, 8, 4, TREE>(prefix, own, f32, s) : launch_attn<D, 8, 8, TREE>(prefix, own, f32, s);
}

}  // namespace

}  // namespace kvtc
