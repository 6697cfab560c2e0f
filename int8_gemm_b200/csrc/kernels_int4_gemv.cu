// Product of a few activation rows with a 4-bit matrix (M <= 32), a weight
// stream: out[m, n] = sum_g s[n, g] * sum_{k in g} x[m, k] * (c[n, k] - z[n, g])
// + bias[n].
//
// The codes are read once and turned into bf16 integers in registers -- a
// nibble placed in the mantissa of 128 gives 128 + c, and subtracting 128 + z
// is exact -- which feed the warp-level bf16 MMA (m16n8k16, fp32 accumulate)
// as its 16-row operand; the scale multiplies the fp32 sum of its group, so
// no weight is ever rounded.  fp32 activations are split into three bf16
// parts that add up to them exactly, one MMA each.
//
// A CTA of 8 warps owns 16 matrix rows and its warps split K.  In a block of
// 128 k, a thread takes for rows g and g + 8 (g = lane / 4) the four words of
// 8 codes at k = 32 i + 8 (lane % 4): all lanes' word i lies in the same 32 k,
// so every MMA sums inside one group whatever the group size.  A word's
// nibbles j and j + 4 form the MMA's k pairs, and the activations are paired
// the same way.  The warps' sums meet in shared memory and are added in warp
// order.
#include <cuda_bf16.h>

#include "lowbit.h"
#include "sm100.cuh"

namespace bsg {

namespace {

constexpr int kRows = 16;
constexpr int kWarps = 8;

__device__ __forceinline__ void mma_bf16_16x8x16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Codes j and j + 4 of a word less `off` = (128 + z, 128 + z), as a bf16 pair.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int j, uint32_t off) {
  const uint32_t m = ((w >> (4 * j)) & 0x000F000Fu) | 0x43004300u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&m), *reinterpret_cast<const __nv_bfloat162*>(&off));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// The high 16 bits of two fp32 values as a bf16 pair.
__device__ __forceinline__ uint32_t high_pair(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}

// Activations k .. k+7 of a row as the MMA's k pairs (j, j + 4), in PARTS bf16
// parts that add up to them.  A truncated value leaves an exact remainder, so
// three parts of 8 bits hold an fp32 value whole; a value that is not finite
// is its own first part (NaN kept a NaN) and leaves no remainder.
template <typename XT, int PARTS>
__device__ __forceinline__ void load_pairs(const XT* row, long long k, long long K, bool vec, uint32_t (&b)[PARTS][4]) {
  if constexpr (sizeof(XT) == 2) {
    uint32_t r[4] = {};
    if (vec && k + 8 <= K) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(row + k));
      r[0] = u.x, r[1] = u.y, r[2] = u.z, r[3] = u.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < K) r[i / 2] |= static_cast<uint32_t>(__bfloat16_as_ushort(row[k + i])) << (16 * (i % 2));
    }
    b[0][0] = __byte_perm(r[0], r[2], 0x5410);
    b[0][1] = __byte_perm(r[0], r[2], 0x7632);
    b[0][2] = __byte_perm(r[1], r[3], 0x5410);
    b[0][3] = __byte_perm(r[1], r[3], 0x7632);
  } else {
    float v[8];
    if (vec && k + 8 <= K) {
      const float4 u0 = __ldg(reinterpret_cast<const float4*>(row + k));
      const float4 u1 = __ldg(reinterpret_cast<const float4*>(row + k) + 1);
      v[0] = u0.x, v[1] = u0.y, v[2] = u0.z, v[3] = u0.w, v[4] = u1.x, v[5] = u1.y, v[6] = u1.z, v[7] = u1.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = k + i < K ? row[k + i] : 0.f;
    }
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (p == 0 && v[i] != v[i]) v[i] = __uint_as_float(0x7FC00000u);
#pragma unroll
      for (int j = 0; j < 4; ++j) b[p][j] = high_pair(v[j], v[j + 4]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float h = __uint_as_float(__float_as_uint(v[i]) & 0xFFFF0000u);
        v[i] = fabsf(v[i]) <= 3.40282347e38f ? __fsub_rn(v[i], h) : 0.f;
      }
    }
  }
}

// Four bytes of a row at byte offset `off`; bytes at or past `end` read as 0.
__device__ __forceinline__ uint32_t load_word(const uint8_t* row, long long off, long long end) {
  if (off + 4 <= end) return __ldg(reinterpret_cast<const uint32_t*>(row + off));
  uint32_t w = 0;
  for (int i = 0; i < 4; ++i)
    if (off + i < end) w |= static_cast<uint32_t>(row[off + i]) << (8 * i);
  return w;
}

// GPB: groups per block of 128 k (1, 2 or 4); NT: tiles of 8 activation rows.
template <typename XT, typename OutT, int GPB, int NT>
__global__ void __launch_bounds__(kWarps * 32)
    gemv_int4_kernel(const Int4Product p, bool xvec) {
  constexpr int PARTS = sizeof(XT) == 2 ? 1 : 3;
  __shared__ float red[kWarps][NT][kRows][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t = lane & 3;
  const long long n0 = blockIdx.x * static_cast<long long>(kRows);
  const int KB = static_cast<int>((p.K + 127) / 128);
  const int kb_lo = static_cast<int>(static_cast<long long>(KB) * warp / kWarps);
  const int kb_hi = static_cast<int>(static_cast<long long>(KB) * (warp + 1) / kWarps);
  const long long bytes = (p.K + 1) / 2;

  grid_dependency_wait();  // every operand may come from the previous kernel in the stream
  grid_launch_dependents();

  const XT* x = static_cast<const XT*>(p.x);
  bool ok[2];
  const uint8_t* row[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const long long n = n0 + gr + 8 * h;
    ok[h] = n < p.N;
    row[h] = p.w.q + (ok[h] ? n : 0) * p.w.ldq;
  }
  float acc[NT][4] = {};
  for (int kb = kb_lo; kb < kb_hi; ++kb) {
    const long long k0 = static_cast<long long>(kb) * 128;
    uint32_t w[2][4];
    float s[2][GPB];
    uint32_t off[2][GPB];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[h][i] = ok[h] ? load_word(row[h], k0 / 2 + 16 * i + 4 * t, bytes) : 0u;
#pragma unroll
      for (int g = 0; g < GPB; ++g) {
        const long long n = n0 + gr + 8 * h, j = static_cast<long long>(kb) * GPB + g;
        s[h][g] = 0.f;
        uint32_t z = 8;
        if (ok[h] && j * p.w.group < p.K) {
          s[h][g] = p.w.scale_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.w.scale)[n * p.w.lds + j])
                                   : static_cast<const float*>(p.w.scale)[n * p.w.lds + j];
          if (p.w.zero) z = p.w.zero[n * p.w.ldz + j] & 15u;
        }
        off[h][g] = (0x4300u + z) * 0x10001u;  // 128 + z twice: one unit of the last place of 128 is 1
      }
    }
    float part[NT][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      constexpr int kWordsPerGroup = 4 / GPB;
      const int g = i / kWordsPerGroup;
      if (i % kWordsPerGroup == 0) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) part[j][e] = 0.f;
      }
      const uint32_t a0[4] = {code_pair(w[0][i], 0, off[0][g]), code_pair(w[1][i], 0, off[1][g]),
                              code_pair(w[0][i], 1, off[0][g]), code_pair(w[1][i], 1, off[1][g])};
      const uint32_t a1[4] = {code_pair(w[0][i], 2, off[0][g]), code_pair(w[1][i], 2, off[1][g]),
                              code_pair(w[0][i], 3, off[0][g]), code_pair(w[1][i], 3, off[1][g])};
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint32_t b[PARTS][4] = {};
        const int m = gr + 8 * j;
        if (m < p.M) load_pairs<XT, PARTS>(x + m * p.ldx, k0 + 32 * i + 8 * t, p.K, xvec, b);
#pragma unroll
        for (int c = PARTS - 1; c >= 0; --c) {  // the smallest parts first
          mma_bf16_16x8x16(part[j], a0, b[c][0], b[c][1]);
          mma_bf16_16x8x16(part[j], a1, b[c][2], b[c][3]);
        }
      }
      if (i % kWordsPerGroup == kWordsPerGroup - 1) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[j][e] = fmaf(s[e / 2][g], part[j][e], acc[j][e]);
      }
    }
  }

#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[warp][j][gr + 8 * (e / 2)][2 * t + e % 2] = acc[j][e];
  __syncthreads();
  for (int i = threadIdx.x; i < NT * kRows * 8; i += kWarps * 32) {
    // consecutive threads take consecutive output columns
    const int r = i % kRows, m = i / kRows;
    const long long n = n0 + r;
    if (m < p.M && n < p.N) {
      float y = red[0][m / 8][r][m % 8];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) y += red[w][m / 8][r][m % 8];
      if (p.bias) y += p.bias[n];
      OutT* dst = static_cast<OutT*>(p.out) + m * p.ldo + n;
      if constexpr (sizeof(OutT) == 2) {
        *dst = __float2bfloat16_rn(y);
      } else {
        *dst = y;
      }
    }
  }
}

template <typename XT, typename OutT, int GPB, int NT>
cudaError_t launch_one(const Int4Product& p, cudaStream_t stream) {
  const bool xvec = (reinterpret_cast<uintptr_t>(p.x) & 15u) == 0 && (p.ldx * sizeof(XT)) % 16 == 0;
  cudaLaunchAttribute attr[1];
  // programmatic dependent launch: the prologue may overlap the previous kernel
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.N + kRows - 1) / kRows), 1, 1);
  cfg.blockDim = dim3(kWarps * 32, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gemv_int4_kernel<XT, OutT, GPB, NT>, p, xvec);
}

template <typename XT, typename OutT, int GPB>
cudaError_t launch_tiles(const Int4Product& p, cudaStream_t stream) {
  if (p.M <= 8) return launch_one<XT, OutT, GPB, 1>(p, stream);
  return p.M <= 16 ? launch_one<XT, OutT, GPB, 2>(p, stream) : launch_one<XT, OutT, GPB, 4>(p, stream);
}

template <typename XT, typename OutT>
cudaError_t launch_group(const Int4Product& p, cudaStream_t stream) {
  if (p.w.group == 128) return launch_tiles<XT, OutT, 1>(p, stream);
  return p.w.group == 64 ? launch_tiles<XT, OutT, 2>(p, stream) : launch_tiles<XT, OutT, 4>(p, stream);
}

}  // namespace

cudaError_t launch_gemv_int4(const Int4Product& p, int sms, cudaStream_t stream) {
  (void)sms;
  if (p.x_bf16)
    return p.out_bf16 ? launch_group<__nv_bfloat16, __nv_bfloat16>(p, stream) : launch_group<__nv_bfloat16, float>(p, stream);
  return p.out_bf16 ? launch_group<float, __nv_bfloat16>(p, stream) : launch_group<float, float>(p, stream);
}

}  // namespace bsg
