// Gradient of the row lookup, dense over the table:
//   d[v, :] = alpha * sum_{t: token[t] = v} grad[t, :]
// with rows that no token names zero (or, when adding to what is there, left
// alone), and no contribution from tokens equal to padding_idx or outside
// [0, V).  Sums are fp32 in an order that the tokens alone decide, rounded
// once to the output type.
//
// Up to kSmallT tokens, one launch (small_kernel): a CTA owns a range of table rows
// and a slice of columns, reads every token, lists those of its rows in order,
// zeroes the rows without one and sums the others' entries along links.
//
// More tokens, three launches.
//   sort: (token, position) pairs by token, stably; tokens that contribute nothing
//     sort behind every row as key V.  Up to kRankMaxT tokens each pair's place
//     is counted by comparing it with all others (rank_kernel: T^2 comparisons on
//     all SMs, no hand-over between them).  Beyond, one cluster of 8 CTAs sorts
//     by digits of up to 9 bits, the lowest first: each warp owns a run of
//     consecutive pairs and counts its digits with match_any, the CTAs exchange
//     their digit totals through distributed shared memory, and every pair's
//     place follows from counts alone.  Either way the order is the same on
//     every run.
//   rows: the sorted list in chunks of 32 pairs, whatever rows they belong to,
//     so a row that many tokens name is spread over many CTAs.  A thread owns
//     one 16-byte column piece and adds a row's pairs in list order.  Rows that
//     begin and end inside a chunk are written; a row that crosses a chunk
//     border leaves one partial sum per chunk in the workspace.  Further CTAs
//     of the launch zero the rows that no pair names.
//   join: the chunk in which a crossing row begins adds its partials in chunk
//     order.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "lowbit.h"
#include "quantize.h"
#include "sm100.cuh"

namespace bsg {

namespace {

namespace cg = cooperative_groups;

constexpr int kSortCtas = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigits = 512;
constexpr int kSortSmem = kSortWarps * kMaxDigits * 4;
constexpr int kChunk = 32;  // sorted pairs per chunk
constexpr int kThreads = 256;
constexpr int kZeroRows = 32;  // rows per zeroing CTA of rows_kernel
constexpr int kSmallT = 512;         // tokens that the single launch takes (D = 512: 200 tokens 16 us, 1000 tokens 31 us against 21)
constexpr int kRankTokens = 32, kRankWays = kThreads / kRankTokens;  // per CTA of rank_kernel; threads per token
constexpr long long kRankMaxT = 4096;  // tokens up to which it is the faster sort (whole gradient, D = 512: 26 us against 31; 6000 tokens: 32 against 31)
constexpr int kMarkRows = 16 * 8192;  // rows marked at a time: a 16 KB bitmap

// Workspace: two (key, position) buffers of T pairs, then the partial sums of
// each chunk's first and last row.
struct Layout {
  long long chunks, dp;  // chunks; floats of a partial row (D rounded up to 8)
  size_t key[2], pos[2], part, bytes;
};

Layout layout_of(long long T, long long D) {
  Layout l;
  l.chunks = (T + kChunk - 1) / kChunk;
  l.dp = (D + 7) / 8 * 8;
  const size_t list = (static_cast<size_t>(T) * 4 + 255) / 256 * 256;
  l.key[0] = 0;
  l.pos[0] = list;
  l.key[1] = 2 * list;
  l.pos[1] = 3 * list;
  l.part = 4 * list;
  l.bytes = l.part + static_cast<size_t>(l.chunks) * 2 * static_cast<size_t>(l.dp) * 4;
  return l;
}

__device__ __forceinline__ float get(const float* p) { return *p; }
__device__ __forceinline__ float get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

struct Tokens {
  const void* tokens;
  bool tokens64;
  uint32_t T;
  uint32_t V;  // also the key of tokens that contribute nothing
  long long padding_idx;

  __device__ __forceinline__ uint32_t key(uint32_t i) const {
    const long long t = tokens64 ? __ldg(static_cast<const long long*>(tokens) + i) : __ldg(static_cast<const int*>(tokens) + i);
    return t >= 0 && t < static_cast<long long>(V) && t != padding_idx ? static_cast<uint32_t>(t) : V;
  }
};

// Zeros in columns [d0, d1) of rows [v0, v1) whose bit is not set, as many
// threads side by side in a row as it has pieces (so that long rows are written
// as one run).  `vec`: rows start on 16-byte boundaries (and d0 is a whole piece).
template <typename OutT>
__device__ __forceinline__ void zero_rows(const uint32_t* named, long long v0, long long v1, OutT* out, long long ldo,
                                          long long d0, long long d1, bool vec) {
  constexpr int Z = 16 / sizeof(OutT);
  const long long n = d1 - d0, whole = vec ? n / Z : 0;
  int log2 = 5;  // threads per row
  while ((2 << log2) <= static_cast<int>(blockDim.x) && (1 << log2) < (vec ? whole : n)) ++log2;
  const int side = 1 << log2, t = threadIdx.x & (side - 1), rows = blockDim.x >> log2;
  if (static_cast<int>(threadIdx.x >> log2) >= rows) return;  // a block that is no power of two
  for (long long v = v0 + (threadIdx.x >> log2); v < v1; v += rows) {
    const uint32_t bit = static_cast<uint32_t>(v - v0);
    if (named[bit / 32] >> (bit % 32) & 1u) continue;
    OutT* p = out + v * ldo + d0;
    for (long long i = t; i < whole; i += side) reinterpret_cast<uint4*>(p)[i] = make_uint4(0, 0, 0, 0);
    for (long long i = whole * Z + t; i < n; i += side) put(p + i, 0.f);
  }
}

// ---------------------------------------------------------------------------
// sort
// ---------------------------------------------------------------------------
struct SortArgs {
  Tokens in;
  uint32_t *key[2], *pos[2];
  int passes, bits;  // pass i takes `bits` bits; reads buffer i & 1 (pass 0: the tokens) and writes the other
};

// Four rounds of 32 pairs of one warp, from i0 on.
struct Batch {
  uint32_t k[4], p[4];

  __device__ __forceinline__ void load(const SortArgs& a, int pass, uint32_t i0, uint32_t hi) {
    const uint32_t* kin = a.key[pass & 1];
    const uint32_t* pin = a.pos[pass & 1];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t i = i0 + 32 * r + (threadIdx.x & 31);
      k[r] = i >= hi ? 0u : (pass == 0 ? a.in.key(i) : kin[i]);
      p[r] = i >= hi || pass == 0 ? i : pin[i];
    }
  }
  template <typename Fn>
  __device__ __forceinline__ void each(uint32_t i0, uint32_t hi, Fn fn) const {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (i0 + 32 * r < hi) fn(i0 + 32 * r + (threadIdx.x & 31) < hi, k[r], p[r]);
  }
};

__device__ __forceinline__ void sort_pairs(const SortArgs& a, uint32_t (*hist)[kMaxDigits]) {
  __shared__ uint32_t total[kMaxDigits];  // this CTA's digit counts, read by the whole cluster
  __shared__ uint32_t base[kMaxDigits];
  __shared__ uint32_t warp_sum[kMaxDigits / 32];
  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t rank = cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // this warp's pairs [lo, hi): runs of a multiple of 32, in (CTA, warp) order
  const uint32_t runs = kSortCtas * kSortWarps, T = a.in.T;
  const uint32_t per = ((T + runs - 1) / runs + 31) / 32 * 32;
  const uint64_t lo64 = static_cast<uint64_t>(rank * kSortWarps + warp) * per;
  const uint32_t lo = lo64 < T ? static_cast<uint32_t>(lo64) : T;
  const uint32_t hi = lo64 + per < T ? static_cast<uint32_t>(lo64 + per) : T;
  const uint32_t below = (1u << lane) - 1u;
  const int digits = 1 << a.bits;
  const uint32_t mask = digits - 1;

  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = a.bits * pass;
    uint32_t* kout = a.key[(pass & 1) ^ 1];
    uint32_t* pout = a.pos[(pass & 1) ^ 1];
    for (int d = lane; d < digits; d += 32) hist[warp][d] = 0;
    __syncwarp();
    Batch first;  // kept for the second sweep: all there is up to 32768 pairs
    first.load(a, pass, lo, hi);
    for (uint32_t i0 = lo; i0 < hi; i0 += 128) {
      Batch batch = first;
      if (i0 != lo) batch.load(a, pass, i0, hi);
      batch.each(i0, hi, [&](bool in, uint32_t k, uint32_t) {
        const uint32_t d = in ? (k >> shift) & mask : kMaxDigits;  // lanes past the end match one another only
        const uint32_t same = __match_any_sync(0xffffffffu, d);
        if (in && (same & below) == 0) hist[warp][d] += __popc(same);
        __syncwarp();
      });
    }
    __syncthreads();
    if (tid < digits) {  // counts of the warps before each warp, and the CTA's total
      uint32_t sum = 0;
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = hist[w][tid];
        hist[w][tid] = sum;
        sum += c;
      }
      total[tid] = sum;
    }
    cluster.sync();  // every CTA's totals are there
    if (tid < kMaxDigits) {
      uint32_t before = 0, all = 0;
      if (tid < digits) {
#pragma unroll
        for (uint32_t r = 0; r < kSortCtas; ++r) {
          const uint32_t c = *cluster.map_shared_rank(&total[tid], r);
          before += r < rank ? c : 0u;
          all += c;
        }
      }
      uint32_t incl = all;  // scan over the digits
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) warp_sum[warp] = incl;
      base[tid] = incl - all + before;
    }
    __syncthreads();
    if (tid < digits) {
      uint32_t pre = 0;
      for (int w = 0; w < warp; ++w) pre += warp_sum[w];
      base[tid] += pre;
    }
    __syncthreads();
    for (uint32_t i0 = lo; i0 < hi; i0 += 128) {
      Batch batch = first;
      if (i0 != lo) batch.load(a, pass, i0, hi);
      batch.each(i0, hi, [&](bool in, uint32_t k, uint32_t p) {
        const uint32_t d = in ? (k >> shift) & mask : kMaxDigits;
        const uint32_t same = __match_any_sync(0xffffffffu, d);
        uint32_t at = 0;
        if (in) at = base[d] + hist[warp][d] + __popc(same & below);
        __syncwarp();
        if (in) {
          if ((same & below) == 0) hist[warp][d] += __popc(same);
          kout[at] = k;
          pout[at] = p;
        }
        __syncwarp();
      });
    }
    // the pairs written here are read by other CTAs in the next pass, and this
    // CTA's totals are no longer read by any
    cluster.sync();
  }
}

__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads) sort_kernel(const SortArgs a) {
  extern __shared__ uint32_t sort_smem[];
  grid_dependency_wait();
  grid_launch_dependents();
  sort_pairs(a, reinterpret_cast<uint32_t(*)[kMaxDigits]>(sort_smem));
}

// A CTA places kRankTokens pairs: a pair's place is the number of pairs before
// it, counted over all tokens by kRankWays threads per pair.  Keys are below
// 2^24 and compared as fp32 integers: the saturated difference bound - k is 1
// where k < bound and 0 elsewhere, so a comparison and its count are two
// full-rate operations, a difference and an addition.
__global__ void __launch_bounds__(kThreads) rank_kernel(const SortArgs a) {
  constexpr int kTile = 2048, kLoads = kTile / kThreads, kPart = kTile / kRankWays;
  __shared__ float4 tile[kTile / 4];
  __shared__ float counts[kRankWays][kRankTokens];
  grid_dependency_wait();
  grid_launch_dependents();
  float* flat = reinterpret_cast<float*>(tile);
  const uint32_t T = a.in.T, i0 = blockIdx.x * kRankTokens;
  const int slot = threadIdx.x % kRankTokens, way = threadIdx.x / kRankTokens;
  const uint32_t i = i0 + slot;
  const uint32_t key = i < T ? a.in.key(i) : a.in.V;
  const float fkey = static_cast<float>(key);
  float count = 0.f;  // at most T
  float next[kLoads];  // the next tile's keys
  auto fetch = [&](uint32_t j0) {
#pragma unroll
    for (int r = 0; r < kLoads; ++r) {
      const uint32_t j = j0 + r * kThreads + threadIdx.x;
      next[r] = j < T ? static_cast<float>(a.in.key(j)) : 3e38f;  // before no pair
    }
  };
  fetch(0);
  for (uint32_t j0 = 0; j0 < T; j0 += kTile) {
#pragma unroll
    for (int r = 0; r < kLoads; ++r) flat[r * kThreads + threadIdx.x] = next[r];
    __syncthreads();
    if (j0 + kTile < T) fetch(j0 + kTile);
    const float4* mine = tile + way * (kPart / 4);
    if (j0 + kTile <= i0 || j0 >= i0 + kRankTokens) {
      // equal keys come before where their position does
      const float bound = j0 < i0 ? fkey + 1.f : fkey;
      float c[4] = {};
#pragma unroll 8
      for (int q = 0; q < kPart / 4; ++q) {
        const float4 k = mine[q];
        c[0] += __saturatef(bound - k.x);
        c[1] += __saturatef(bound - k.y);
        c[2] += __saturatef(bound - k.z);
        c[3] += __saturatef(bound - k.w);
      }
      count += (c[0] + c[1]) + (c[2] + c[3]);
    } else {
      for (int q = 0; q < kPart; ++q) {
        const uint32_t j = j0 + way * kPart + q;
        count += __saturatef((j < i ? fkey + 1.f : fkey) - flat[way * kPart + q]);
      }
    }
    __syncthreads();
  }
  counts[way][slot] = count;
  __syncthreads();
  if (way == 0 && i < T) {
#pragma unroll
    for (int w = 1; w < kRankWays; ++w) count += counts[w][slot];
    const uint32_t at = static_cast<uint32_t>(count);
    a.key[0][at] = key;
    a.pos[0][at] = i;
  }
}

// ---------------------------------------------------------------------------
// rows and join
// ---------------------------------------------------------------------------
struct RowArgs {
  const uint32_t *key, *pos;  // sorted
  uint32_t T, V;
  const void* grad;
  long long ldg, D;
  float alpha;
  void* out;
  long long ldo;
  bool accumulate;
  float* part;  // [chunks][2][dp]: a chunk's share of the row it begins in the middle of, and of the row it ends in
  long long dp;
  uint32_t chunks, slices;  // of columns
  bool gvec, ovec;
};

// 16 bytes of a gradient row, as read.
template <typename InT>
struct Piece {
  static constexpr int E = 16 / sizeof(InT);
  uint32_t w[4];

  // `left` of its elements exist (the others are zero); `vec`: rows start on
  // 16-byte boundaries.
  __device__ __forceinline__ void load(const InT* p, long long left, bool vec) {
    if (vec && left >= E) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if (i >= left) continue;
      if constexpr (E == 4) w[i] = __float_as_uint(p[i]);
      else w[i / 2] |= static_cast<uint32_t>(__bfloat16_as_ushort(p[i])) << (16 * (i % 2));
    }
  }

  __device__ __forceinline__ void add_to(float (&sum)[E]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (E == 4) {
        sum[i] += __uint_as_float(w[i]);
      } else {
        sum[2 * i] += __uint_as_float(w[i] << 16);
        sum[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
};

// alpha * sum into E columns of a row (added to what is there when accumulating).
template <typename OutT, int E>
__device__ __forceinline__ void write_row(const RowArgs& a, uint32_t v, long long d, const float (&sum)[E]) {
  OutT* p = static_cast<OutT*>(a.out) + v * a.ldo + d;
  const long long left = a.D - d;
  float y[E];
#pragma unroll
  for (int i = 0; i < E; ++i) y[i] = __fmul_rn(a.alpha, sum[i]);
  if (a.ovec && left >= E) {
    if constexpr (sizeof(OutT) == 4) {
#pragma unroll
      for (int i = 0; i < E; i += 4) {
        float4 v = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
        if (a.accumulate) {
          const float4 old = *reinterpret_cast<const float4*>(p + i);
          v = make_float4(old.x + v.x, old.y + v.y, old.z + v.z, old.w + v.w);
        }
        *reinterpret_cast<float4*>(p + i) = v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; i += 4) {
        if (a.accumulate) {
          const uint2 old = *reinterpret_cast<const uint2*>(p + i);
          y[i] += __uint_as_float(old.x << 16);
          y[i + 1] += __uint_as_float(old.x & 0xFFFF0000u);
          y[i + 2] += __uint_as_float(old.y << 16);
          y[i + 3] += __uint_as_float(old.y & 0xFFFF0000u);
        }
        const __nv_bfloat162 h0 = __floats2bfloat162_rn(y[i], y[i + 1]), h1 = __floats2bfloat162_rn(y[i + 2], y[i + 3]);
        *reinterpret_cast<uint2*>(p + i) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (i < left) put(p + i, a.accumulate ? __fadd_rn(get(p + i), y[i]) : y[i]);
}

// gridDim.x: the chunks' slices, then CTAs that zero kZeroRows rows each (mixed
// evenly among the chunks they cost the gradient of 16640 tokens on a table of
// 131072 x 5120 504 us in place of 450).
template <typename InT, typename OutT>
__global__ void __launch_bounds__(kThreads) rows_kernel(const RowArgs a) {
  constexpr int E = 16 / sizeof(InT);
  __shared__ uint32_t key[kChunk + 2], pos[kChunk];  // key[0] and key[kChunk + 1]: the neighbours'
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t work = a.chunks * a.slices;
  if (blockIdx.x >= work) {  // zeros: the rows that no pair names
    const long long v0 = static_cast<long long>(blockIdx.x - work) * kZeroRows;
    const long long v1 = v0 + kZeroRows < a.V ? v0 + kZeroRows : a.V;
    if (threadIdx.x < 32) {
      const long long v = v0 + threadIdx.x;
      uint32_t lo = 0, hi = a.T;  // the first key >= v
      while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (a.key[mid] < v) lo = mid + 1;
        else hi = mid;
      }
      const uint32_t bits = __ballot_sync(0xffffffffu, lo < a.T && a.key[lo] == v);
      if (threadIdx.x == 0) key[0] = bits;
    }
    __syncthreads();
    zero_rows<OutT>(key, v0, v1, static_cast<OutT*>(a.out), a.ldo, 0, a.D, a.ovec);
    return;
  }
  const uint32_t c = blockIdx.x / a.slices, slice = blockIdx.x - c * a.slices;
  const uint32_t i0 = c * kChunk;
  for (int j = threadIdx.x; j < kChunk + 2; j += blockDim.x) {
    const long long i = static_cast<long long>(i0) + j - 1;
    key[j] = i >= 0 && i < a.T ? a.key[i] : a.V;  // a.V: no row
    if (j < kChunk) pos[j] = i0 + j < a.T ? a.pos[i0 + j] : 0u;
  }
  __syncthreads();
  const long long d = (static_cast<long long>(slice) * blockDim.x + threadIdx.x) * E;
  if (d >= a.D) return;
  const InT* g = static_cast<const InT*>(a.grad) + d;
  float* part = a.part + static_cast<long long>(c) * 2 * a.dp + d;
  float sum[E] = {};
  bool from_before = key[0] == key[1];
#pragma unroll 1
  for (int j0 = 0; j0 < kChunk; j0 += 8) {
    Piece<InT> v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (key[j0 + u + 1] < a.V) v[u].load(g + pos[j0 + u] * a.ldg, a.D - d, a.gvec);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int j = j0 + u;
      const uint32_t k = key[j + 1], next = key[j + 2];
      if (k >= a.V) break;
      v[u].add_to(sum);
      const bool last = j == kChunk - 1;
      if (k != next || last) {
        const bool crosses = from_before || (last && k == next);
        if (crosses) {
          float* p = part + (from_before ? 0 : a.dp);
#pragma unroll
          for (int e = 0; e < E; e += 4)
            *reinterpret_cast<float4*>(p + e) = make_float4(sum[e], sum[e + 1], sum[e + 2], sum[e + 3]);
        } else {
          write_row<OutT, E>(a, k, d, sum);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) sum[e] = 0.f;
        from_before = false;
      }
    }
  }
}

// A row that begins in chunk c and goes on in the next: its partials, chunk by
// chunk.
template <typename OutT>
__global__ void __launch_bounds__(kThreads) join_kernel(const RowArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t c = blockIdx.x / a.slices, slice = blockIdx.x - c * a.slices;
  const long long first = static_cast<long long>(c) * kChunk, next = first + kChunk;
  if (next >= a.T) return;
  const uint32_t k = a.key[next], k_last = a.key[next - 1], k_first = a.key[first];
  const uint32_t k_before = first > 0 ? a.key[first - 1] : a.V;
  if (k >= a.V || k_last != k) return;              // no row crosses this border
  if (k_first == k && k_before == k) return;        // it began in an earlier chunk
  // chunks that it goes on through: those whose first key is its own
  uint32_t more = 0;
  for (long long i = next;; i += static_cast<long long>(blockDim.x) * kChunk) {
    const long long at = i + static_cast<long long>(threadIdx.x) * kChunk;
    const uint32_t n = __syncthreads_count(at < a.T && a.key[at] == k);
    more += n;
    if (n < blockDim.x) break;
  }
  const long long d = (static_cast<long long>(slice) * blockDim.x + threadIdx.x) * 4;
  if (d >= a.D) return;
  float sum[4];
  const float4 h = *reinterpret_cast<const float4*>(a.part + (static_cast<long long>(c) * 2 + 1) * a.dp + d);
  sum[0] = h.x, sum[1] = h.y, sum[2] = h.z, sum[3] = h.w;
  const float* p = a.part + (static_cast<long long>(c) + 1) * 2 * a.dp + d;
  for (uint32_t i0 = 0; i0 < more; i0 += 8) {
    float4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i0 + u < more) v[u] = *reinterpret_cast<const float4*>(p + (static_cast<long long>(i0) + u) * 2 * a.dp);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i0 + u < more) sum[0] += v[u].x, sum[1] += v[u].y, sum[2] += v[u].z, sum[3] += v[u].w;
  }
  write_row<OutT, 4>(a, k, d, sum);
}

// ---------------------------------------------------------------------------
// up to kSmallT tokens, in one launch
// ---------------------------------------------------------------------------
struct SmallArgs {
  Tokens in;
  RowArgs r;  // out, grad and their sizes; slices, gvec, ovec
  uint32_t ranges;
};

template <typename InT, typename OutT>
__global__ void __launch_bounds__(kThreads) small_kernel(const SmallArgs a) {
  constexpr int E = 16 / sizeof(InT);
  constexpr uint32_t kNone = 0xffffu;
  __shared__ uint32_t named[kMarkRows / 32];
  __shared__ uint32_t row[kSmallT];             // the listed tokens' rows, less v0
  __shared__ uint16_t at[kSmallT], next[kSmallT];  // their positions, and the next entry of the same row
  __shared__ uint8_t later[kSmallT];            // whether an earlier entry links to this one
  __shared__ uint32_t warp_n[kThreads / 32 + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t range = blockIdx.x / a.r.slices, slice = blockIdx.x - range * a.r.slices;
  const long long V = a.in.V;
  const long long v_lo = V * range / a.ranges, v_hi = V * (range + 1) / a.ranges;
  const long long width = static_cast<long long>(blockDim.x) * E;
  const long long d0 = slice * width, d1 = d0 + width < a.r.D ? d0 + width : a.r.D;
  grid_dependency_wait();
  grid_launch_dependents();
  for (long long v0 = v_lo; v0 < v_hi; v0 += kMarkRows) {
    const uint32_t rows = static_cast<uint32_t>(v_hi - v0 < kMarkRows ? v_hi - v0 : kMarkRows);
    for (uint32_t i = tid; i < (rows + 31) / 32; i += blockDim.x) named[i] = 0;
    __syncthreads();
    uint32_t n = 0;  // entries listed so far
    for (uint32_t i0 = 0; i0 < a.in.T; i0 += blockDim.x) {
      const uint32_t i = i0 + tid;
      const uint32_t bit = i < a.in.T ? a.in.key(i) - static_cast<uint32_t>(v0) : rows;  // wraps where below v0
      const bool mine = bit < rows;
      const uint32_t vote = __ballot_sync(0xffffffffu, mine);
      if (lane == 0) warp_n[warp] = __popc(vote);
      __syncthreads();
      uint32_t before = n, all = n;
      for (int w = 0; w < static_cast<int>(blockDim.x / 32); ++w) {
        if (w < warp) before += warp_n[w];
        all += warp_n[w];
      }
      if (mine) {
        const uint32_t e = before + __popc(vote & ((1u << lane) - 1u));
        row[e] = bit;
        at[e] = static_cast<uint16_t>(i);
        next[e] = kNone;
        later[e] = 0;
        atomicOr(&named[bit / 32], 1u << (bit % 32));
      }
      n = all;
      __syncthreads();
    }
    // link each entry to the next of its row
    for (uint32_t e = tid; e < n; e += blockDim.x) {
      const uint32_t mine = row[e];
      for (uint32_t f = e + 1; f < n; ++f) {
        if (row[f] == mine) {
          next[e] = static_cast<uint16_t>(f);
          later[f] = 1;
          break;
        }
      }
    }
    if (!a.r.accumulate)
      zero_rows<OutT>(named, v0, v0 + rows, static_cast<OutT*>(a.r.out), a.r.ldo, d0, d1, a.r.ovec);
    __syncthreads();
    const long long d = d0 + static_cast<long long>(tid) * E;
    if (d < a.r.D) {
      const InT* g = static_cast<const InT*>(a.r.grad) + d;
      for (uint32_t h = 0; h < n; ++h) {
        if (later[h]) continue;
        float sum[E] = {};
        uint32_t e = h;
        while (e != kNone) {
          Piece<InT> v[8];
          int m = 0;
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            if (e != kNone) {
              v[u].load(g + at[e] * a.r.ldg, a.r.D - d, a.r.gvec);
              e = next[e];
              m = u + 1;
            }
          }
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (u < m) v[u].add_to(sum);
        }
        write_row<OutT, E>(a.r, static_cast<uint32_t>(v0) + row[h], d, sum);
      }
    }
    __syncthreads();
  }
}

bool rows16(const void* base, long long ld_bytes) {
  return (reinterpret_cast<uintptr_t>(base) & 15u) == 0 && ld_bytes % 16 == 0;
}

int threads_for(long long pieces) { return pieces >= kThreads ? kThreads : static_cast<int>((pieces + 31) / 32 * 32); }

// A launch that may begin while the previous kernel of the stream ends (every
// kernel here waits for it before its first access).
template <typename Args>
cudaError_t launch_after(void (*kernel)(Args), long long grid, int threads, size_t smem, cudaStream_t stream,
                         const Args& args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

template <typename InT, typename OutT>
cudaError_t launch_types(const Tokens& in, const LookupGradArgs& a, int sms, cudaStream_t stream) {
  constexpr int E = 16 / sizeof(InT);
  RowArgs r = {};
  r.T = in.T;
  r.V = in.V;
  r.grad = a.grad;
  r.ldg = a.ldg;
  r.D = a.D;
  r.alpha = a.alpha;
  r.out = a.out;
  r.ldo = a.ldo;
  r.accumulate = a.accumulate;
  r.gvec = rows16(a.grad, a.ldg * static_cast<long long>(sizeof(InT)));
  r.ovec = rows16(a.out, a.ldo * static_cast<long long>(sizeof(OutT)));
  const long long pieces = (a.D + E - 1) / E;
  const int threads = threads_for(pieces);
  r.slices = static_cast<uint32_t>((pieces + threads - 1) / threads);

  if (a.T <= kSmallT) {
    SmallArgs s;
    s.in = in;
    s.r = r;
    // ranges of rows for four CTAs per SM or 128 KB of zeros a CTA, whichever are
    // more (CTAs that write near one another: 61484 x 5465 fp32 329 -> 221 us)
    const long long width = static_cast<long long>(threads) * E * static_cast<long long>(sizeof(OutT));
    const long long fill = (4LL * sms + r.slices - 1) / r.slices, near = a.accumulate ? 0 : a.V / (131072 / width + 1);
    const long long want = fill > near ? fill : near;
    s.ranges = static_cast<uint32_t>(want < a.V ? want : a.V);
    return launch_after(small_kernel<InT, OutT>, static_cast<long long>(s.ranges) * r.slices, threads, 0, stream, s);
  }

  const Layout l = layout_of(a.T, a.D);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  SortArgs s;
  s.in = in;
  for (int i = 0; i < 2; ++i) {
    s.key[i] = reinterpret_cast<uint32_t*>(ws + l.key[i]);
    s.pos[i] = reinterpret_cast<uint32_t*>(ws + l.pos[i]);
  }
  cudaError_t e;
  if (a.T <= kRankMaxT && a.V < (1 << 24)) {
    s.passes = s.bits = 0;
    e = launch_after(rank_kernel, (a.T + kRankTokens - 1) / kRankTokens, kThreads, 0, stream, s);
  } else {
    int total_bits = 1;  // of the largest key, V
    while (total_bits < 32 && (static_cast<unsigned long long>(a.V) >> total_bits) != 0) ++total_bits;
    s.passes = (total_bits + 8) / 9;
    s.bits = (total_bits + s.passes - 1) / s.passes;
    int per_sm = 0;
    e = ctas_per_sm_once<sort_kernel>(kSortThreads, kSortSmem, &per_sm);
    if (e != cudaSuccess) return e;
    e = launch_after(sort_kernel, kSortCtas, kSortThreads, kSortSmem, stream, s);
  }
  if (e != cudaSuccess) return e;

  r.key = s.key[s.passes & 1];
  r.pos = s.pos[s.passes & 1];
  r.part = reinterpret_cast<float*>(ws + l.part);
  r.dp = l.dp;
  r.chunks = static_cast<uint32_t>(l.chunks);
  const long long zeros = a.accumulate ? 0 : (a.V + kZeroRows - 1) / kZeroRows;
  e = launch_after(rows_kernel<InT, OutT>, static_cast<long long>(r.chunks) * r.slices + zeros, threads, 0, stream, r);
  if (e != cudaSuccess) return e;
  const long long quads = (a.D + 3) / 4;
  const int jt = threads_for(quads);
  r.slices = static_cast<uint32_t>((quads + jt - 1) / jt);
  return launch_after(join_kernel<OutT>, (static_cast<long long>(r.chunks) - 1) * r.slices, jt, 0, stream, r);
}

}  // namespace

size_t lookup_grad_workspace(long long T, long long V, long long D) {
  (void)V;
  return T <= kSmallT ? 0 : layout_of(T, D).bytes;
}

cudaError_t launch_lookup_grad(const LookupGradArgs& a, int sms, cudaStream_t stream) {
  Tokens in;
  in.tokens = a.tokens;
  in.tokens64 = a.tokens64;
  in.T = static_cast<uint32_t>(a.T);
  in.V = static_cast<uint32_t>(a.V);
  in.padding_idx = a.padding_idx;
  if (a.T == 0 && a.accumulate) return cudaSuccess;
  if (a.grad_bf16)
    return a.out_bf16 ? launch_types<__nv_bfloat16, __nv_bfloat16>(in, a, sms, stream)
                      : launch_types<__nv_bfloat16, float>(in, a, sms, stream);
  return a.out_bf16 ? launch_types<float, __nv_bfloat16>(in, a, sms, stream) : launch_types<float, float>(in, a, sms, stream);
}

}  // namespace bsg
