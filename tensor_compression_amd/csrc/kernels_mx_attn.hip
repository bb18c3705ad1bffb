// Attention over the microscaled paged cache.
//
// For 16 NT query rows of one kv head (row r = token r / G, head r % G of its
// group) and a range of tokens, a workgroup of four waves computes
//   s = q k^T, running maximum m, sum l of 2^(c s - m), o = sum 2^(c s - m) v
// in one pass; its waves take pairs of pages in turn and are joined through
// LDS at the end, ranges by k_mx_join.
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
#include <type_traits>

#include "mx_internal.h"

namespace kvtc {

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

namespace {

constexpr float kLow = -3.0e38f;  // running maximum of a row that has seen nothing
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

// A lane's share of one page as it lies in the record.
template <int KW, int VW>
struct Page {
  uint32_t k[KW], v[VW], ks, vs;
};

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* src, uint32_t (&w)[N]) {
  if constexpr (N == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(src);
    w[0] = u.x;
    w[1] = u.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 u = reinterpret_cast<const uint4*>(src)[i];
      w[4 * i] = u.x;
      w[4 * i + 1] = u.y;
      w[4 * i + 2] = u.z;
      w[4 * i + 3] = u.w;
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

// Tokens that row i of a sequence attends to.
__device__ __forceinline__ int limit_of(const MxSeq& s, int i, int causal) {
  return causal ? max(s.len - s.n + i + 1, 0) : s.len;
}

__device__ __forceinline__ int wave_min(int v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v = min(v, __shfl_xor(v, o));
  return v;
}
__device__ __forceinline__ int wave_max(int v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v = max(v, __shfl_xor(v, o));
  return v;
}

template <int D, int BK, int BV, int NT, bool F32>
__global__ __launch_bounds__(256, 2) void k_mx_attn(const MxAttnParams p) {
  constexpr MxRecord R = mx_record(D, BK, BV);
  constexpr int C = D / 16;                            // channels of an entry of the value groups
  constexpr int KS = D / 32;                           // contraction steps of S
  constexpr int KW = D * BK / 128, VW = D * BV / 128;  // words of a lane's share of a page
  constexpr int NP = F32 ? 3 : 1;                      // bf16 parts of queries and weights
  constexpr bool QL = NT > 2 || F32;                   // queries in LDS
  constexpr int OS = D + 4;                            // row stride of the joining buffer

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int n = lane & 15, kg = lane >> 4;

  // heads vary fastest, so that (with 8 of them) a head's tiles stay on one
  // XCD and its pages in one L2; the last tiles, longest when causal, first
  int bid = blockIdx.x;
  const int h = bid % p.H;
  bid /= p.H;
  const int tile = p.tiles - 1 - bid % p.tiles;
  bid /= p.tiles;
  const int split = bid % p.nsplit, z = bid / p.nsplit;

  __shared__ __attribute__((aligned(16))) float lds[4 * 16 * OS];
  __shared__ float2 ml[4][16];
  __shared__ int2 rowq[NT * 16];  // row and query head, row -1 for none
  static_assert(!QL || NT * KS * NP * 1024 <= 4 * 16 * OS * 4, "the queries fit where the joining buffer is");

  const int Hq = p.H * p.G;
  MxSeq sq{0, 0, 0};
  int rows;
  if (p.prefix) rows = p.b.total_rows * p.G;
  else {
    sq = mx_seq(p.b, z, p.status);
    rows = sq.n * p.G;
  }
  const int r0 = tile * 16 * NT;
  if (r0 >= rows) return;

  // ---- the rows of this lane's query column
  int lim[NT], lo = 0x7FFFFFFF, hi = 0;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = r0 + 16 * t + n;
    lim[t] = 0;
    int at = -1;
    if (r < rows) {
      const int i = r / p.G;
      int row = i;
      bool ok = true;
      if (p.prefix) {
        const MxSeq s = mx_seq(p.b, seq_of(p.b, row), p.status);
        ok = row >= s.row0 && row < s.row0 + s.n;
        if (ok) lim[t] = limit_of(s, row - s.row0, p.causal);
      } else {
        row = sq.row0 + i;
        lim[t] = limit_of(sq, i, p.causal);
      }
      if (ok) at = row;
    }
    if (at >= 0) lo = min(lo, lim[t]);
    hi = max(hi, lim[t]);
    if (wave == 0 && kg == 0) rowq[16 * t + n] = make_int2(at, h * p.G + r % p.G);
  }
  lo = __builtin_amdgcn_readfirstlane(wave_min(lo));  // every row attends to the tokens below
  hi = __builtin_amdgcn_readfirstlane(wave_max(hi));  // and none from here on
  const int begin = p.begin + split * p.chunk;
  const int end = min(min(p.end, begin + p.chunk), hi);
  if (p.ws_o && begin >= end) return;
  __syncthreads();  // rowq

  // ---- queries: B operands, channels (D / 4) kg + 8 s .. + 7 of row n
  bf16x8_t qf[QL ? 1 : NT][QL ? 1 : KS];
  uint4* const ql = reinterpret_cast<uint4*>(lds);
  if constexpr (QL) {
    for (int f = wave; f < NT * KS; f += 4) {
      const int t = f / KS, s = f % KS;
      const int2 at = rowq[16 * t + n];
      uint4 w[NP];
#pragma unroll
      for (int k = 0; k < NP; ++k) w[k] = make_uint4(0, 0, 0, 0);
      if (at.x >= 0) {
        const int64_t off = at.x * p.q_stride + at.y * D + (D / 4) * kg + 8 * s;
        if constexpr (!F32) w[0] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.q) + off);
        else {
          float x[8];
          *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.q) + off);
          *reinterpret_cast<float4*>(x + 4) = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.q) + off + 4);
#pragma unroll
          for (int k = 0; k < NP; ++k) {
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              u[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
              x[2 * i] = rest(x[2 * i], u[i], 0);
              x[2 * i + 1] = rest(x[2 * i + 1], u[i], 1);
            }
            w[k] = make_uint4(u[0], u[1], u[2], u[3]);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < NP; ++k) ql[(f * NP + k) * 64 + lane] = w[k];
    }
    __syncthreads();
  } else {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int2 at = rowq[16 * t + n];
      const int64_t off = at.x * p.q_stride + at.y * D + (D / 4) * kg;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (at.x >= 0) w = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.q) + off + 8 * s);
        qf[t][s] = __builtin_bit_cast(bf16x8_t, w);
      }
    }
  }

  // ---- the pass over the tokens
  f32x4_t acc[NT][C];
  float m[NT], l[NT];
  uint32_t poison[NT];  // channel blocks whose value was NaN at a token that the row attends to
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t] = kLow;
    l[t] = 0.f;
    poison[t] = 0;
#pragma unroll
    for (int j = 0; j < C; ++j) acc[t][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }

  const int32_t* table = p.b.page_table + (p.prefix ? 0 : (int64_t)z * p.b.max_pages);
  const uint8_t* head = p.pool + (int64_t)h * R.bytes;
  const int64_t page_bytes = (int64_t)p.H * R.bytes;
  const int k_off = n * (D * BK / 8) + kg * KW * 4;
  const int v_off = R.kc + (kg * 16 + n) * VW * 4;
  const int ks_off = R.kc + R.vc + n * (D / 32) + kg * (D / 32) / 4;
  const int vs_off = R.kc + R.vc + R.sc + (kg * (D / 32) + n * C / 32) * 4;
  const int p0 = begin / KVTC_MX_PAGE, p1 = (end + KVTC_MX_PAGE - 1) / KVTC_MX_PAGE;  // pages of the range

  using PageT = Page<KW, VW>;
  // pages past the range and pages outside the pool are read as page 0 and masked
  auto page_id = [&](int pg) {
    int id = pg < p1 ? table[pg] : -1;
    id = __builtin_amdgcn_readfirstlane(id);
    if (pg < p1 && (uint32_t)id >= (uint32_t)p.pool_pages) {
      if (p.status && lane == 0) atomicOr(p.status, 1u << KVTC_ERR_INVALID_ARG);
      id = -1;
    }
    return id;
  };
  auto load_page = [&](int id, PageT& g) {
    const uint8_t* rec = head + (int64_t)max(id, 0) * page_bytes;
    load_words(rec + k_off, g.k);
    load_words(rec + v_off, g.v);
    g.ks = rec[ks_off];
    g.vs = *reinterpret_cast<const uint32_t*>(rec + vs_off);
  };

  int pg = p0 + 2 * wave;
  int id[2], nid[2];
  PageT g[2], ng[2];
  if (pg < p1) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      nid[e] = page_id(pg + e);
      load_page(nid[e], ng[e]);
    }
  }
  for (; pg < p1; pg += 8) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      id[e] = nid[e];
      g[e] = ng[e];
    }
    if (pg + 8 < p1) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        nid[e] = page_id(pg + 8 + e);
        load_page(nid[e], ng[e]);
      }
    }
    const int t0 = pg * KVTC_MX_PAGE;
    // tokens of page e that exist for this workgroup, 0 .. 16
    int have[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) have[e] = id[e] < 0 ? 0 : min(max(end - t0 - 16 * e, 0), 16);
    const bool whole = have[0] + have[1] == 32 && t0 + 32 <= lo;

    if (!whole) {
      // tokens that no row attends to may be anything: make their values 0
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * kg + i >= have[e]) {
#pragma unroll
            for (int w = 0; w < VW / 4 + (VW < 4); ++w) {
              if constexpr (VW >= 4) g[e].v[i * (VW / 4) + w] = 0;
              else g[e].v[i / 2] &= (i & 1) ? 0x0000FFFFu : 0xFFFF0000u;
            }
            g[e].vs = (g[e].vs & ~(0xFFu << (8 * i))) | (0x7Fu << (8 * i));
          }
      // a NaN value that only some rows attend to: 0 in the product, and a
      // mark for the rows that do
      bool nan = false;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) nan |= ((g[e].vs >> (8 * i)) & 0xFFu) == 0xFFu;
      if (__builtin_amdgcn_ballot_w64(nan)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint8_t* vs = head + (int64_t)max(id[e], 0) * page_bytes + R.kc + R.vc + R.sc + kg * (D / 32) * 4;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (4 * kg + i < have[e]) {
#pragma unroll
              for (int b = 0; b < D / 32; ++b)
                if (vs[4 * b + i] == 0xFFu) {
#pragma unroll
                  for (int t = 0; t < NT; ++t)
                    if (t0 + 16 * e + 4 * kg + i < lim[t]) poison[t] |= 1u << b;
                }
            }
            if (((g[e].vs >> (8 * i)) & 0xFFu) == 0xFFu) {
#pragma unroll
              for (int w = 0; w < VW / 4 + (VW < 4); ++w) {
                if constexpr (VW >= 4) g[e].v[i * (VW / 4) + w] = 0;
                else g[e].v[i / 2] &= (i & 1) ? 0x0000FFFFu : 0xFFFF0000u;
              }
              g[e].vs = (g[e].vs & ~(0xFFu << (8 * i))) | (0x7Fu << (8 * i));
            }
          }
        }
      }
    }

    // ---- scores, weights
    bf16x8_t pf[NT][NP];
    {
      bf16x8_t kf[2][KS];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float sc = __uint_as_float(g[e].ks << 23);
#pragma unroll
        for (int s = 0; s < KS; ++s) kf[e][s] = eight<BK>(g[e].k + s * (BK / 4), sc);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        f32x4_t sa[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int k = NP - 1; k >= 0; --k)  // small parts first
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            bf16x8_t q;
            if constexpr (QL) q = __builtin_bit_cast(bf16x8_t, ql[((t * KS + s) * NP + k) * 64 + lane]);
            else q = qf[t][s];
#pragma unroll
            for (int e = 0; e < 2; ++e) sa[e] = mfma(kf[e][s], q, sa[e]);
          }
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int top = min(lim[t] - t0 - 16 * e, have[e]) - 4 * kg;
#pragma unroll
            for (int i = 0; i < 4; ++i) sa[e][i] = i < top ? sa[e][i] : -INFINITY;
          }
        }
        float mx = fmaxf(fmaxf(fmaxf(sa[0][0], sa[0][1]), fmaxf(sa[0][2], sa[0][3])),
                         fmaxf(fmaxf(sa[1][0], sa[1][1]), fmaxf(sa[1][2], sa[1][3])));
        mx *= p.c;
        if (__builtin_amdgcn_ballot_w64(mx > m[t] + kSlack)) {
          mx = fmaxf(mx, __shfl_xor(mx, 16));
          mx = fmaxf(mx, __shfl_xor(mx, 32));
          const float nm = fmaxf(m[t], mx), a = __builtin_amdgcn_exp2f(m[t] - nm);
          m[t] = nm;
          l[t] *= a;
#pragma unroll
          for (int j = 0; j < C; ++j) acc[t][j] *= a;
        }
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          w[i] = __builtin_amdgcn_exp2f(__fmaf_rn(sa[i / 4][i % 4], p.c, -m[t]));
        }
        l[t] += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          uint32_t u[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            u[i] = pack_bf16(w[2 * i], w[2 * i + 1]);
            if (k + 1 < NP) {
              w[2 * i] = rest(w[2 * i], u[i], 0);
              w[2 * i + 1] = rest(w[2 * i + 1], u[i], 1);
            }
          }
          pf[t][k] = operand(u[0], u[1], u[2], u[3]);
        }
      }
    }

    // ---- values: channel pair (2 i, 2 i + 1) of the lane's entry at its
    // four tokens of each page, then a word per channel and token pair
    float vsc[2][4];
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i) vsc[e][i] = __uint_as_float(((g[e].vs >> (8 * i)) & 0xFFu) << 23);
    auto value_pair = [&](int e, int i, auto ic) {
      constexpr int c2 = decltype(ic)::value;  // channel pair
      if constexpr (BV == 4 && C == 8) return two<4, c2>(g[e].v[i], vsc[e][i]);
      else if constexpr (BV == 4) return (i & 1) ? two<4, 2 + c2>(g[e].v[i / 2], vsc[e][i]) : two<4, c2>(g[e].v[i / 2], vsc[e][i]);
      else return two<8, c2 & 1>(g[e].v[i * (C / 4) + c2 / 2], vsc[e][i]);
    };
    auto channels = [&](auto ic) {
      constexpr int c2 = decltype(ic)::value;
      uint32_t x[2][4], ev[4], od[4];
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[e][i] = value_pair(e, i, ic);
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ev[2 * e + i] = __builtin_amdgcn_perm(x[e][2 * i + 1], x[e][2 * i], 0x05040100u);
          od[2 * e + i] = __builtin_amdgcn_perm(x[e][2 * i + 1], x[e][2 * i], 0x07060302u);
        }
      const bf16x8_t ve = operand(ev[0], ev[1], ev[2], ev[3]), vo = operand(od[0], od[1], od[2], od[3]);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = NP - 1; k >= 0; --k) {
          acc[t][2 * c2] = mfma(ve, pf[t][k], acc[t][2 * c2]);
          acc[t][2 * c2 + 1] = mfma(vo, pf[t][k], acc[t][2 * c2 + 1]);
        }
    };
    channels(std::integral_constant<int, 0>{});
    channels(std::integral_constant<int, 1>{});
    if constexpr (C == 8) {
      channels(std::integral_constant<int, 2>{});
      channels(std::integral_constant<int, 3>{});
    }
  }

  // ---- join the waves, 16 rows at a time
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float sum = l[t];
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    uint32_t pz = poison[t];
    pz |= (uint32_t)__shfl_xor((int)pz, 16);
    pz |= (uint32_t)__shfl_xor((int)pz, 32);
    const bool dead = (pz >> (kg * (D / 32) / 4)) & 1u;  // this lane's channels [kg D / 4, (kg + 1) D / 4)
    __syncthreads();                                     // the buffer is free
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < C; j += 4) {
        float4 o = make_float4(acc[t][j][i], acc[t][j + 1][i], acc[t][j + 2][i], acc[t][j + 3][i]);
        if (dead) o = make_float4(NAN, NAN, NAN, NAN);
        *reinterpret_cast<float4*>(&lds[(wave * 16 + n) * OS + C * (4 * kg + i) + j]) = o;
      }
    if (kg == 0) ml[wave][n] = make_float2(m[t], sum);
    __syncthreads();
    const int r = threadIdx.x >> 4, c0 = (threadIdx.x & 15) * C;
    const int2 rh = rowq[16 * t + r];
    if (rh.x < 0) continue;
    const int64_t at = (int64_t)rh.x * Hq + rh.y;
    float M = kLow, L = 0.f, a[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) M = fmaxf(M, ml[w][r].x);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      a[w] = __builtin_amdgcn_exp2f(ml[w][r].x - M);
      L = __fmaf_rn(a[w], ml[w][r].y, L);
    }
    float o[C];
#pragma unroll
    for (int j = 0; j < C; j += 4) {
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(&lds[(w * 16 + r) * OS + c0 + j]);
        s.x = __fmaf_rn(a[w], x.x, s.x);
        s.y = __fmaf_rn(a[w], x.y, s.y);
        s.z = __fmaf_rn(a[w], x.z, s.z);
        s.w = __fmaf_rn(a[w], x.w, s.w);
      }
      *reinterpret_cast<float4*>(o + j) = s;
    }
    if (p.ws_o) {
      const int64_t slot = (int64_t)(p.slot0 + split) * p.b.total_rows * Hq + at;
      float4* d = reinterpret_cast<float4*>(p.ws_o + slot * D + c0);
#pragma unroll
      for (int j = 0; j < C / 4; ++j) d[j] = *reinterpret_cast<const float4*>(o + 4 * j);
      if (c0 == 0) p.ws_ml[slot] = make_float2(M, L);
    } else {
      const float r1 = L == 0.f ? 0.f : 1.0f / L;
#pragma unroll
      for (int j = 0; j < C; ++j) o[j] *= r1;
      if constexpr (F32) {
        float4* d = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + at * D + c0);
#pragma unroll
        for (int j = 0; j < C / 4; ++j) d[j] = *reinterpret_cast<const float4*>(o + 4 * j);
      } else {
        uint2* d = reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + at * D + c0);
#pragma unroll
        for (int j = 0; j < C / 4; ++j)
          d[j] = make_uint2(pack_bf16(o[4 * j], o[4 * j + 1]), pack_bf16(o[4 * j + 2], o[4 * j + 3]));
      }
      if (p.lse && c0 == 0) p.lse[at] = L == 0.f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * kLn2;
    }
  }
}

// Joins a row's partials: one wave a (row, head), sixteen lanes on its
// channels, four partials at once.
template <int D, bool F32>
__global__ __launch_bounds__(256) void k_mx_join(const MxJoinParams p) {
  constexpr int C = D / 16;
  const int lane = threadIdx.x & 63, g = lane >> 4, c0 = (lane & 15) * C;
  const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
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
  for (int k = g; k < a + b; k += 4) {
    const int64_t slot = (int64_t)(k < a ? k : p.prefix_splits + k - a) * all + at;
    const float2 x = p.ws_ml[slot];
    const float nm = fmaxf(M, x.x), u = __builtin_amdgcn_exp2f(M - nm), w = __builtin_amdgcn_exp2f(x.x - nm);
    M = nm;
    L = __fmaf_rn(L, u, x.y * w);
    const float4* y = reinterpret_cast<const float4*>(p.ws_o + slot * D + c0);
#pragma unroll
    for (int j = 0; j < C / 4; ++j) {
      const float4 v = y[j];
      o[4 * j] = __fmaf_rn(o[4 * j], u, v.x * w);
      o[4 * j + 1] = __fmaf_rn(o[4 * j + 1], u, v.y * w);
      o[4 * j + 2] = __fmaf_rn(o[4 * j + 2], u, v.z * w);
      o[4 * j + 3] = __fmaf_rn(o[4 * j + 3], u, v.w * w);
    }
  }
#pragma unroll
  for (int d = 16; d < 64; d <<= 1) {
    const float om = __shfl_xor(M, d), nm = fmaxf(M, om), u = __builtin_amdgcn_exp2f(M - nm);
    M = nm;
    L *= u;
    L += __shfl_xor(L, d);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      o[j] *= u;
      o[j] += __shfl_xor(o[j], d);
    }
  }
  if (g) return;
  const float r1 = L == 0.f ? 0.f : 1.0f / L;
#pragma unroll
  for (int j = 0; j < C; ++j) o[j] *= r1;
  if constexpr (F32) {
    float4* d = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + at * D + c0);
#pragma unroll
    for (int j = 0; j < C / 4; ++j) d[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
  } else {
    uint2* d = reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + at * D + c0);
#pragma unroll
    for (int j = 0; j < C / 4; ++j)
      d[j] = make_uint2(pack_bf16(o[4 * j], o[4 * j + 1]), pack_bf16(o[4 * j + 2], o[4 * j + 3]));
  }
  if (p.lse && c0 == 0) p.lse[at] = L == 0.f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * kLn2;
}

template <int D, int BK, int BV>
hipError_t launch_attn(const MxAttnParams& p, bool f32, int nt, hipStream_t s) {
  const unsigned grid = (unsigned)p.H * p.tiles * p.nsplit * (p.prefix ? 1 : p.b.n_seqs);
  if (f32) {
    if (nt == 1) k_mx_attn<D, BK, BV, 1, true><<<grid, 256, 0, s>>>(p);
    else k_mx_attn<D, BK, BV, 2, true><<<grid, 256, 0, s>>>(p);
  } else {
    if (nt == 1) k_mx_attn<D, BK, BV, 1, false><<<grid, 256, 0, s>>>(p);
    else if (nt == 2) k_mx_attn<D, BK, BV, 2, false><<<grid, 256, 0, s>>>(p);
    else k_mx_attn<D, BK, BV, 4, false><<<grid, 256, 0, s>>>(p);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_attn(const MxAttnParams& p, int D, int bk, int bv, bool f32, int nt, hipStream_t s) {
  if (D == 128) {
    if (bk == 4) return bv == 4 ? launch_attn<128, 4, 4>(p, f32, nt, s) : launch_attn<128, 4, 8>(p, f32, nt, s);
    return bv == 4 ? launch_attn<128, 8, 4>(p, f32, nt, s) : launch_attn<128, 8, 8>(p, f32, nt, s);
  }
  if (bk == 4) return bv == 4 ? launch_attn<64, 4, 4>(p, f32, nt, s) : launch_attn<64, 4, 8>(p, f32, nt, s);
  return bv == 4 ? launch_attn<64, 8, 4>(p, f32, nt, s) : launch_attn<64, 8, 8>(p, f32, nt, s);
}

hipError_t launch_mx_join(const MxJoinParams& p, bool f32, hipStream_t s) {
  const int64_t all = (int64_t)p.b.total_rows * p.Hq;
  const unsigned grid = (unsigned)((all + 3) / 4);
  if (p.D == 128) {
    if (f32) k_mx_join<128, true><<<grid, 256, 0, s>>>(p);
    else k_mx_join<128, false><<<grid, 256, 0, s>>>(p);
  } else {
    if (f32) k_mx_join<64, true><<<grid, 256, 0, s>>>(p);
    else k_mx_join<64, false><<<grid, 256, 0, s>>>(p);
  }
  return hipGetLastError();
}

}  // namespace kvtc
