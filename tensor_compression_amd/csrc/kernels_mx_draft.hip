// Microscaled paged cache: the trees of drafts, and moving the accepted rows
// to where the sequence goes on.
#include <type_traits>

#include "mx_codes.h"

namespace kvtc {

namespace {

// A wave takes one word of the masks of a sequence's rows, 64 rows at a time.
// Within the 64 a row points to its parent, a row whose parent lies before
// them (or nowhere) to itself; each round joins what a row has with what the
// row that it points to has, and points it there, so that six rounds see 64
// generations, fewer where the trees are shallower.  What lies before comes
// from the words already done, in LDS.  The wave of word 0 counts ancestors
// in the same rounds.
__global__ __launch_bounds__(128) void k_mx_tree(const kvtc_mx_batch b, const int32_t* parents, uint32_t* masks, int words,
                                                 int32_t* positions, uint32_t* status, int most) {
  extern __shared__ uint32_t lds[];  // [2 waves][most] words, then [most] depths
  const int z = (int)blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int word = (int)blockIdx.y * 2 + wave;
  if (word >= words) return;
  const bool first = word == 0;
  const MxSeq s = mx_seq(b, z, first ? status : nullptr);
  uint32_t* const done = lds + wave * most;
  int* const depth = reinterpret_cast<int*>(lds + 2 * most);
  bool bad = false;
  for (int i0 = 0; i0 < s.n; i0 += 64) {
    const int i = i0 + lane;
    int parent = -1;
    if (i < s.n) {
      parent = parents[s.row0 + i];
      if (parent < -1 || parent >= i) {
        parent = -1;
        bad = true;
      }
    }
    uint32_t m = (i >> 5) == word ? 1u << (i & 31) : 0;
    const bool inside = parent >= i0;
    int to = inside ? parent - i0 : lane, d = inside;
    for (int r = 0; r < 6; ++r) {
      const int next = __shfl(to, to);
      m |= (uint32_t)__shfl((int)m, to);
      if (first) d += __shfl(d, to);
      if (!__builtin_amdgcn_ballot_w64(next != to)) break;
      to = next;
    }
    const int before = __shfl(inside ? -1 : parent, to);  // the parent of the row's ancestor that is first in the 64
    if (before >= 0) m |= done[before];
    if (first && before >= 0) d += depth[before] + 1;
    if (i < s.n) {
      done[i] = m;
      masks[(int64_t)(s.row0 + i) * words + word] = m;
      if (first) {
        depth[i] = d;
        if (positions) positions[s.row0 + i] = s.len - s.n + d;
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the next 64 read other lanes' words
  }
  if (first && bad && status) atomicOr(status, 1u << KVTC_ERR_INVALID_ARG);
}

// A workgroup lists the rows that stay, then its waves move the keys or the
// values of some heads, sixteen tokens at a time: all of them are read before
// any is written, and a token only moves down, so what is overwritten has
// been read (the k-th kept row is row k or a later one).  Tokens that stay
// where they are are not touched.
template <int D, int BK, int BV>
__global__ __launch_bounds__(256) void k_mx_keep(const MxKeepParams p) {
  constexpr MxRecord R = mx_record(D, BK, BV);
  constexpr int C = D / 16;
  __shared__ uint32_t word[KVTC_MX_MAX_DRAFT / 32], below[KVTC_MX_MAX_DRAFT / 32 + 1];
  __shared__ uint16_t row[KVTC_MX_MAX_DRAFT];
  const int z = (int)blockIdx.x, tid = threadIdx.x, lane = tid & 63;
  const int t4 = lane >> 4, n = lane & 15;
  const bool tell = blockIdx.y == 0;
  const MxSeq s = mx_seq(p.b, z, tell ? p.status : nullptr);
  const int node = p.nodes[z], old = p.b.kv_lens[z];
  const bool ok = s.n > 0 && node >= -1 && node < s.n;
  if (!ok) {
    if (tell && tid == 0) {
      p.lens_out[z] = old;
      if (s.n > 0 && p.status) atomicOr(p.status, 1u << KVTC_ERR_INVALID_ARG);
    }
    return;
  }
  const int base = s.len - s.n, skip = max(-base, 0);  // rows before the first token
  const int words = (s.n + 31) / 32;
  if (tid < words) {
    uint32_t m = node < 0 ? 0 : p.masks[(int64_t)(s.row0 + node) * p.words + tid];
    if (tid * 32 + 32 > s.n) m &= ~0u >> (32 * words - s.n);
    if (tid * 32 < skip) m = tid * 32 + 32 <= skip ? 0 : m & (~0u << (skip - tid * 32));
    word[tid] = m;
  }
  __syncthreads();
  if (tid <= words) {
    int k = 0;
    for (int w = 0; w < tid; ++w) k += __builtin_popcount(word[w]);
    below[tid] = k;
    if (tid < words)
      for (uint32_t m = word[tid]; m; m &= m - 1) row[k++] = (uint16_t)(tid * 32 + __builtin_ctz(m));
  }
  __syncthreads();
  const int kept = below[words], to0 = max(base, 0);
  if (tell && tid == 0) p.lens_out[z] = to0 + kept;
  const int32_t* table = p.b.page_table + (int64_t)z * p.b.max_pages;
  const int w = __builtin_amdgcn_readfirstlane((int)(blockIdx.y * 4 + (tid >> 6)));
  const int kv = w & 1, h = (w >> 1) % p.H, l = (w >> 1) / p.H;
  if (l >= p.n_layers) return;
  uint8_t* const head = p.pool + l * p.layer_bytes + (int64_t)h * R.bytes;
  const int64_t page_bytes = (int64_t)p.H * R.bytes;
  auto page_of = [&](int pos) {
    const int id = table[pos / KVTC_MX_PAGE];
    return (uint32_t)id < (uint32_t)p.pool_pages ? id : -1;
  };
  bool bad = false;
  auto move = [&](auto bits) {
    constexpr int B = decltype(bits)::value;
    uint8_t* const codes = head + (kv ? R.kc : 0);
    uint8_t* const scales = head + R.kc + R.vc + (kv ? R.sc : 0);
    for (int k0 = 0; k0 < kept; k0 += 16) {
      uint32_t c[4][2], sc[4];
      int64_t to[4];
      int at[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = k0 + 4 * i + t4;
        at[i] = -1;
        c[i][0] = c[i][1] = sc[i] = 0;
        to[i] = 0;
        if (k >= kept || base + row[k] == to0 + k) continue;
        const int from = base + row[k], src = page_of(from), dst = page_of(to0 + k);
        if (src < 0 || dst < 0) {
          bad = true;
          continue;
        }
        at[i] = (to0 + k) % KVTC_MX_PAGE;
        to[i] = dst * page_bytes;
        const int f = from % KVTC_MX_PAGE;
        load_codes<B, C>(codes + src * page_bytes + code_at<D, B>(kv, f >> 2, f & 3, n), c[i]);
        sc[i] = scales[src * page_bytes + scale_at<D>(kv, f >> 2, f & 3, n / (32 / C))];
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // all sixteen have been read
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (at[i] < 0) continue;
        store_codes<B, C>(codes + to[i] + code_at<D, B>(kv, at[i] >> 2, at[i] & 3, n), c[i]);
        if (n % (32 / C) == 0) scales[to[i] + scale_at<D>(kv, at[i] >> 2, at[i] & 3, n / (32 / C))] = (uint8_t)sc[i];
      }
    }
  };
  if (kv) move(std::integral_constant<int, BV>{});
  else move(std::integral_constant<int, BK>{});
  if (bad && p.status) atomicOr(p.status, 1u << KVTC_ERR_INVALID_ARG);
}

template <int D, int BK, int BV>
hipError_t launch_keep(const MxKeepParams& p, hipStream_t s) {
  const dim3 grid((unsigned)p.b.n_seqs, (unsigned)((p.n_layers * p.H * 2 + 3) / 4));
  k_mx_keep<D, BK, BV><<<grid, 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_tree(const kvtc_mx_batch& b, const int32_t* parents, uint32_t* masks, int words,
                          int32_t* positions, uint32_t* status, hipStream_t s) {
  const int most = b.max_rows < b.total_rows ? b.max_rows : b.total_rows;
  const dim3 grid((unsigned)b.n_seqs, (unsigned)((words + 1) / 2));
  k_mx_tree<<<grid, 128, (size_t)most * 3 * 4, s>>>(b, parents, masks, words, positions, status, most);
  return hipGetLastError();
}

hipError_t launch_mx_keep(const MxKeepParams& p, int D, int bk, int bv, hipStream_t s) {
  if (D == 128) {
    if (bk == 4) return bv == 4 ? launch_keep<128, 4, 4>(p, s) : launch_keep<128, 4, 8>(p, s);
    return bv == 4 ? launch_keep<128, 8, 4>(p, s) : launch_keep<128, 8, 8>(p, s);
  }
  if (bk == 4) return bv == 4 ? launch_keep<64, 4, 4>(p, s) : launch_keep<64, 4, 8>(p, s);
  return bv == 4 ? launch_keep<64, 8, 4>(p, s) : launch_keep<64, 8, 8>(p, s);
}

}  // namespace kvtc
