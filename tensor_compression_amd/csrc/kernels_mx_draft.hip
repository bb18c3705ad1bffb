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
// in the same rounds.  Bound by latency, a launch and its loads for the usual
// draft (64 of 20 to 60 rows: 3.1 us) and some 0.6 us for every 64 rows of a
// long one (16 of 300 to 1000 rows: 12.7 us; four times 64 rows in the same
// rounds 13.2, eight words leaving together from LDS 15.8).
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
// values of HEADS (layer, head) pairs, 4 GROUPS tokens at a time: all of them
// are read before any is written, and a token only moves down, so what is
// overwritten has been read (the k-th kept row is row k or a later one).
// Tokens that stay where they are are not touched, but their pages are checked.
// Bound by latency: the
// lengths, the mask, the pages, the codes (64 sequences of up to 8 rows, 32
// layers x 8 heads: one pair a wave 13.4 us, four 9.9; a path of some hundred
// rows through 10 pairs: 16 tokens at a time 13.4 us, 64 9.0).
template <int D, int BK, int BV, int HEADS, int GROUPS>
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
  // this wave: keys or values of HEADS (layer, head) pairs
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), kv = wave & 1;
  const int pair0 = ((int)blockIdx.y * 2 + (wave >> 1)) * HEADS, pairs = min(p.n_layers * p.H - pair0, HEADS);
  if (pairs <= 0) return;
  const int64_t page_bytes = (int64_t)p.H * R.bytes;
  auto page_of = [&](int pos) {
    const int id = table[pos / KVTC_MX_PAGE];
    return (uint32_t)id < (uint32_t)p.pool_pages ? id : -1;
  };
  uint8_t* head[HEADS];
#pragma unroll
  for (int j = 0; j < HEADS; ++j) {
    const int pair = pair0 + min(j, pairs - 1), l = pair / p.H;
    head[j] = p.pool + l * p.layer_bytes + (int64_t)(pair - l * p.H) * R.bytes;
  }
  bool bad = false;
  auto move = [&](auto bits) {
    constexpr int B = decltype(bits)::value;
    const int codes = kv ? R.kc : 0, scales = R.kc + R.vc + (kv ? R.sc : 0);
    for (int k0 = 0; k0 < kept; k0 += 4 * GROUPS) {
      int64_t from[GROUPS], to[GROUPS];  // the lane's codes of its tokens; from -1: nothing to move
      int from_sc[GROUPS], to_sc[GROUPS];
#pragma unroll
      for (int i = 0; i < GROUPS; ++i) {
        const int k = k0 + 4 * i + t4;
        from[i] = to[i] = -1;
        from_sc[i] = to_sc[i] = 0;
        if (k >= kept) continue;
        const int a = base + row[k], b = to0 + k, src = page_of(a), dst = page_of(b);
        if (src < 0 || dst < 0) {
          bad = true;
          continue;
        }
        if (a == b) continue;
        const int ka = a % KVTC_MX_PAGE, kb = b % KVTC_MX_PAGE, ca = code_at<D, B>(kv, ka >> 2, ka & 3, n),
                  cb = code_at<D, B>(kv, kb >> 2, kb & 3, n);
        from[i] = src * page_bytes + codes + ca;
        to[i] = dst * page_bytes + codes + cb;
        from_sc[i] = scales + scale_at<D>(kv, ka >> 2, ka & 3, n / (32 / C)) - codes - ca;  // beside the codes
        to_sc[i] = scales + scale_at<D>(kv, kb >> 2, kb & 3, n / (32 / C)) - codes - cb;
      }
      uint32_t c[HEADS][GROUPS][2], sc[HEADS][GROUPS];
#pragma unroll
      for (int j = 0; j < HEADS; ++j)
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
          c[j][i][0] = c[j][i][1] = sc[j][i] = 0;
          if (from[i] >= 0 && j < pairs) {
            load_codes<B, C>(head[j] + from[i], c[j][i]);
            sc[j][i] = head[j][from[i] + from_sc[i]];
          }
        }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // all of them have been read
#pragma unroll
      for (int j = 0; j < HEADS; ++j)
#pragma unroll
        for (int i = 0; i < GROUPS; ++i)
          if (from[i] >= 0 && j < pairs) {
            store_codes<B, C>(head[j] + to[i], c[j][i]);
            if (n % (32 / C) == 0) head[j][to[i] + to_sc[i]] = (uint8_t)sc[j][i];
          }
    }
  };
  if (kv) move(std::integral_constant<int, BV>{});
  else move(std::integral_constant<int, BK>{});
  if (bad && p.status) atomicOr(p.status, 1u << KVTC_ERR_INVALID_ARG);
}

template <int D, int BK, int BV>
hipError_t launch_keep(const MxKeepParams& p, hipStream_t s) {
  const unsigned pairs = (unsigned)(p.n_layers * p.H);
  // where that leaves waves for every pair, long paths go in larger steps
  if ((int64_t)pairs * p.b.n_seqs <= 2048)
    k_mx_keep<D, BK, BV, 1, 16><<<dim3((unsigned)p.b.n_seqs, (pairs + 1) / 2), 256, 0, s>>>(p);
  else k_mx_keep<D, BK, BV, 4, 4><<<dim3((unsigned)p.b.n_seqs, (pairs + 7) / 8), 256, 0, s>>>(p);
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
