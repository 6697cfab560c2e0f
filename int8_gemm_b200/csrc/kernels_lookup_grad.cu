// Gradient of the row lookup, dense over the table:
//   d[v, :] = alpha * sum_{t: token[t] = v} grad[t, :]
// with rows that no token names zero (or, when adding to what is there, left
// alone), and no contribution from tokens equal to padding_idx or outside
// [0, V).  Sums are fp32 in an order that the tokens alone decide, rounded
// once to the output type.
//
// Three launches.
//   sort: one cluster of 8 CTAs sorts (token, position) pairs by token, stably,
//     least significant 8-bit digit first (tokens that contribute nothing sort
//     behind every row as key V).  Each warp owns a run of consecutive pairs
//     and counts its digits with match_any, the CTAs exchange their digit
//     totals through distributed shared memory, and every pair's place follows
//     from counts alone, so the order is the same on every run.
//   rows: the sorted list in chunks of 32 pairs, whatever rows they belong to,
//     so a row that many tokens name is spread over many CTAs.  A thread owns
//     one 16-byte column piece and adds a row's pairs in list order.  Rows that
//     begin and end inside a chunk are written; a row that crosses a chunk
//     border leaves one partial sum per chunk in the workspace.  Further CTAs
//     of the same launch zero the rows that no pair names.
//   join: the chunk in which a crossing row begins adds its partials in chunk
//     order.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "lowbit.h"

namespace bsg {

namespace {

namespace cg = cooperative_groups;

constexpr int kSortCtas = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigits = 256;
constexpr int kChunk = 32;     // sorted pairs per chunk
constexpr int kZeroRows = 32;  // table rows per zeroing CTA
constexpr int kThreads = 256;

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

// ---------------------------------------------------------------------------
// sort
// ---------------------------------------------------------------------------
struct SortArgs {
  const void* tokens;
  bool tokens64;
  uint32_t T;
  uint32_t V;  // also the key of pairs that contribute nothing
  long long padding_idx;
  uint32_t *key[2], *pos[2];
  int passes;  // pass i reads buffer i & 1 (pass 0: the tokens) and writes the other
};

__device__ __forceinline__ uint32_t token_key(const SortArgs& a, uint32_t i) {
  const long long t = a.tokens64 ? static_cast<const long long*>(a.tokens)[i] : static_cast<const int*>(a.tokens)[i];
  return t >= 0 && t < static_cast<long long>(a.V) && t != a.padding_idx ? static_cast<uint32_t>(t) : a.V;
}

__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads) sort_kernel(const SortArgs a) {
  __shared__ uint32_t hist[kSortWarps][kDigits];
  __shared__ uint32_t total[kDigits];  // this CTA's digit counts, read by the whole cluster
  __shared__ uint32_t base[kDigits];
  __shared__ uint32_t warp_sum[kDigits / 32];
  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t rank = cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // this warp's pairs [lo, hi): runs of a multiple of 32, in (CTA, warp) order
  const uint32_t runs = kSortCtas * kSortWarps;
  const uint32_t per = ((a.T + runs - 1) / runs + 31) / 32 * 32;
  const uint64_t lo64 = static_cast<uint64_t>(rank * kSortWarps + warp) * per;
  const uint32_t lo = lo64 < a.T ? static_cast<uint32_t>(lo64) : a.T;
  const uint32_t hi = lo64 + per < a.T ? static_cast<uint32_t>(lo64 + per) : a.T;
  const uint32_t below = (1u << lane) - 1u;

  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = 8 * pass;
    const uint32_t* kin = a.key[pass & 1];
    const uint32_t* pin = a.pos[pass & 1];
    uint32_t* kout = a.key[(pass & 1) ^ 1];
    uint32_t* pout = a.pos[(pass & 1) ^ 1];
    for (int d = lane; d < kDigits; d += 32) hist[warp][d] = 0;
    __syncwarp();
    for (uint32_t i0 = lo; i0 < hi; i0 += 32) {
      const uint32_t i = i0 + lane;
      const bool in = i < hi;
      const uint32_t k = !in ? 0u : (pass == 0 ? token_key(a, i) : kin[i]);
      const uint32_t d = in ? (k >> shift) & 255u : kDigits;  // lanes past the end match one another only
      const uint32_t same = __match_any_sync(0xffffffffu, d);
      if (in && (same & below) == 0) hist[warp][d] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    if (tid < kDigits) {  // counts of the warps before each warp, and the CTA's total
      uint32_t sum = 0;
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = hist[w][tid];
        hist[w][tid] = sum;
        sum += c;
      }
      total[tid] = sum;
    }
    cluster.sync();  // every CTA's totals are there
    uint32_t before = 0, all = 0;
    if (tid < kDigits) {
      for (uint32_t r = 0; r < kSortCtas; ++r) {
        const uint32_t c = *cluster.map_shared_rank(&total[tid], r);
        before += r < rank ? c : 0u;
        all += c;
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
    if (tid < kDigits) {
      uint32_t pre = 0;
      for (int w = 0; w < warp; ++w) pre += warp_sum[w];
      base[tid] += pre;
    }
    __syncthreads();
    for (uint32_t i0 = lo; i0 < hi; i0 += 32) {
      const uint32_t i = i0 + lane;
      const bool in = i < hi;
      const uint32_t k = !in ? 0u : (pass == 0 ? token_key(a, i) : kin[i]);
      const uint32_t d = in ? (k >> shift) & 255u : kDigits;
      const uint32_t same = __match_any_sync(0xffffffffu, d);
      uint32_t at = 0;
      if (in) at = base[d] + hist[warp][d] + __popc(same & below);
      __syncwarp();
      if (in) {
        if ((same & below) == 0) hist[warp][d] += __popc(same);
        kout[at] = k;
        pout[at] = pass == 0 ? i : pin[i];
      }
      __syncwarp();
    }
    // the pairs written here are read by other CTAs in the next pass, and this
    // CTA's totals are no longer read by any
    cluster.sync();
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
  uint32_t chunks, slices;  // column slices: gridDim.x = chunks * slices + zeroing CTAs
  bool gvec, ovec;
};

template <typename InT>
__device__ __forceinline__ void load_piece(const InT* p, long long left, bool vec, float (&v)[16 / sizeof(InT)]) {
  constexpr int E = 16 / sizeof(InT);
  if (vec && left >= E) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (E == 4) {
        v[i] = __uint_as_float(w[i]);
      } else {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      v[i] = 0.f;
      if (i < left) {
        if constexpr (E == 4) v[i] = p[i];
        else v[i] = __bfloat162float(p[i]);
      }
    }
  }
}

__device__ __forceinline__ float get(const float* p) { return *p; }
__device__ __forceinline__ float get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// alpha * sum into E columns of a row (added to what is there when accumulating).
template <typename OutT, int E>
__device__ __forceinline__ void write_row(const RowArgs& a, uint32_t v, long long d, const float (&sum)[E]) {
  OutT* p = static_cast<OutT*>(a.out) + v * a.ldo + d;
  const long long left = a.D - d;
  float y[E];
#pragma unroll
  for (int i = 0; i < E; ++i) y[i] = a.alpha * sum[i];
  if (!a.accumulate && a.ovec && left >= E) {
    if constexpr (sizeof(OutT) == 4) {
#pragma unroll
      for (int i = 0; i < E; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < E; i += 4) {
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

template <typename InT, typename OutT>
__global__ void __launch_bounds__(kThreads) rows_kernel(const RowArgs a) {
  constexpr int E = 16 / sizeof(InT);
  __shared__ uint32_t key[kChunk + 2], pos[kChunk];  // key[0] and key[kChunk + 1]: the neighbours'
  const uint32_t work = a.chunks * a.slices;
  if (blockIdx.x < work) {
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
    for (int j0 = 0; j0 < kChunk; j0 += 4) {
      float v[4][E];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (key[j0 + u + 1] < a.V) {
          load_piece<InT>(g + pos[j0 + u] * a.ldg, a.D - d, a.gvec, v[u]);
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) v[u][e] = 0.f;
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = j0 + u;
        const uint32_t k = key[j + 1], next = key[j + 2];
        if (k >= a.V) break;
#pragma unroll
        for (int e = 0; e < E; ++e) sum[e] += v[u][e];
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
    return;
  }
  // zero the rows that no pair names
  __shared__ bool named[kZeroRows];
  const long long v0 = static_cast<long long>(blockIdx.x - work) * kZeroRows;
  if (threadIdx.x < kZeroRows) {
    const long long v = v0 + threadIdx.x;
    uint32_t lo = 0, hi = a.T;  // the first key >= v
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2;
      if (a.key[mid] < v) lo = mid + 1;
      else hi = mid;
    }
    named[threadIdx.x] = v >= a.V || (lo < a.T && a.key[lo] == v);
  }
  __syncthreads();
  constexpr int Z = 16 / sizeof(OutT);
  for (int r = 0; r < kZeroRows; ++r) {
    if (named[r]) continue;
    OutT* p = static_cast<OutT*>(a.out) + (v0 + r) * a.ldo;
    if (a.ovec) {
      const long long whole = a.D / Z;
      for (long long i = threadIdx.x; i < whole; i += blockDim.x) reinterpret_cast<uint4*>(p)[i] = make_uint4(0, 0, 0, 0);
      for (long long i = whole * Z + threadIdx.x; i < a.D; i += blockDim.x) put(p + i, 0.f);
    } else {
      for (long long i = threadIdx.x; i < a.D; i += blockDim.x) put(p + i, 0.f);
    }
  }
}

// A row that begins in chunk c and goes on in the next: its partials, chunk by
// chunk.
template <typename OutT>
__global__ void __launch_bounds__(kThreads) join_kernel(const RowArgs a) {
  const uint32_t c = blockIdx.x / a.slices, slice = blockIdx.x - c * a.slices;
  const long long first = static_cast<long long>(c) * kChunk, next = first + kChunk;
  if (next >= a.T) return;
  const uint32_t k = a.key[next];
  if (k >= a.V || a.key[next - 1] != k) return;                     // no row crosses this border
  if (first > 0 && a.key[first] == k && a.key[first - 1] == k) return;  // it began in an earlier chunk
  const long long d = (static_cast<long long>(slice) * blockDim.x + threadIdx.x) * 4;
  if (d >= a.D) return;
  float sum[4];
  const float4 h = *reinterpret_cast<const float4*>(a.part + (static_cast<long long>(c) * 2 + 1) * a.dp + d);
  sum[0] = h.x, sum[1] = h.y, sum[2] = h.z, sum[3] = h.w;
  for (long long i = next; i < a.T && a.key[i] == k; i += kChunk) {
    const float4 v = *reinterpret_cast<const float4*>(a.part + (i / kChunk) * 2 * a.dp + d);
    sum[0] += v.x, sum[1] += v.y, sum[2] += v.z, sum[3] += v.w;
  }
  write_row<OutT, 4>(a, k, d, sum);
}

bool rows16(const void* base, long long ld_bytes) {
  return (reinterpret_cast<uintptr_t>(base) & 15u) == 0 && ld_bytes % 16 == 0;
}

int threads_for(long long pieces) { return pieces >= kThreads ? kThreads : static_cast<int>((pieces + 31) / 32 * 32); }

template <typename InT, typename OutT>
cudaError_t launch_rows(RowArgs r, cudaStream_t stream) {
  constexpr int E = 16 / sizeof(InT);
  r.gvec = rows16(r.grad, r.ldg * static_cast<long long>(sizeof(InT)));
  r.ovec = rows16(r.out, r.ldo * static_cast<long long>(sizeof(OutT)));
  const long long pieces = (r.D + E - 1) / E;
  const int threads = threads_for(pieces);
  r.slices = static_cast<uint32_t>((pieces + threads - 1) / threads);
  const long long zero = r.accumulate ? 0 : (static_cast<long long>(r.V) + kZeroRows - 1) / kZeroRows;
  const long long grid = static_cast<long long>(r.chunks) * r.slices + zero;
  rows_kernel<InT, OutT><<<static_cast<unsigned>(grid), threads, 0, stream>>>(r);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || r.chunks < 2) return e;
  const long long quads = (r.D + 3) / 4;
  const int jt = threads_for(quads);
  r.slices = static_cast<uint32_t>((quads + jt - 1) / jt);
  join_kernel<OutT><<<static_cast<unsigned>((r.chunks - 1) * r.slices), jt, 0, stream>>>(r);
  return cudaGetLastError();
}

}  // namespace

size_t lookup_grad_workspace(long long T, long long V, long long D) {
  (void)V;
  return layout_of(T, D).bytes;
}

cudaError_t launch_lookup_grad(const LookupGradArgs& a, int sms, cudaStream_t stream) {
  (void)sms;
  const Layout l = layout_of(a.T, a.D);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  SortArgs s;
  s.tokens = a.tokens;
  s.tokens64 = a.tokens64;
  s.T = static_cast<uint32_t>(a.T);
  s.V = static_cast<uint32_t>(a.V);
  s.padding_idx = a.padding_idx;
  for (int i = 0; i < 2; ++i) {
    s.key[i] = reinterpret_cast<uint32_t*>(ws + l.key[i]);
    s.pos[i] = reinterpret_cast<uint32_t*>(ws + l.pos[i]);
  }
  s.passes = 1;
  while (s.passes < 4 && (static_cast<unsigned long long>(a.V) >> (8 * s.passes)) != 0) ++s.passes;
  if (a.T > 0) {
    sort_kernel<<<kSortCtas, kSortThreads, 0, stream>>>(s);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  RowArgs r;
  r.key = s.key[s.passes & 1];
  r.pos = s.pos[s.passes & 1];
  r.T = s.T;
  r.V = s.V;
  r.grad = a.grad;
  r.ldg = a.ldg;
  r.D = a.D;
  r.alpha = a.alpha;
  r.out = a.out;
  r.ldo = a.ldo;
  r.accumulate = a.accumulate;
  r.part = reinterpret_cast<float*>(ws + l.part);
  r.dp = l.dp;
  r.chunks = static_cast<uint32_t>(l.chunks);
  if (a.T == 0 && a.accumulate) return cudaSuccess;
  if (a.grad_bf16)
    return a.out_bf16 ? launch_rows<__nv_bfloat16, __nv_bfloat16>(r, stream) : launch_rows<__nv_bfloat16, float>(r, stream);
  return a.out_bf16 ? launch_rows<float, __nv_bfloat16>(r, stream) : launch_rows<float, float>(r, stream);
}

}  // namespace bsg
