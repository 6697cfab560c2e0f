// Rows of a table, decoded and scaled: out[t, :] = alpha * table[token[t], :]
// (HBM-bound: each named row read once, each output row written once).
//
// Tables: bf16, fp32, e4m3 codes with one fp32 or e8m0 scale per row and 128
// elements (the 1x128 quantiser's output), or 4-bit codes with group scales
// (kernels_int4_quant.cu).  An element's value is formed in fp32 (code times
// scale, one rounding), multiplied by alpha (one more) and rounded to the
// output type; alpha = 1 changes nothing, which is how the dequantiser of
// 4-bit matrices uses this kernel, with row t itself in the place of a token.
// A token outside [0, V) gives a row of zeros and reads nothing.
//
// A thread handles pieces of 16 output bytes, consecutive lanes consecutive
// pieces, four pieces' loads in flight; a block takes a run of consecutive
// pieces, so the division that finds a piece's row is 32 bits wide whatever
// the size of the output.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "lowbit.h"

namespace bsg {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr int kRun = kThreads * kUnroll;  // pieces per block

enum class Fmt { kBF16, kF32, kE4M3, kE4M3E8M0, kInt4 };

__device__ __forceinline__ float e8m0_value(uint8_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : static_cast<uint32_t>(b) << 23);  // 2^-127 is subnormal
}

__device__ __forceinline__ long long token_at(const LookupArgs& a, long long t) {
  if (!a.tokens) return t;
  return a.tokens64 ? static_cast<const long long*>(a.tokens)[t] : static_cast<const int*>(a.tokens)[t];
}

__device__ __forceinline__ float int4_scale(const Int4Matrix& w, long long r, long long g) {
  return w.scale_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w.scale)[r * w.lds + g])
                      : static_cast<const float*>(w.scale)[r * w.lds + g];
}

// Elements d .. d+E-1 of row r as fp32 (those at or past D are not used).
// `vec`: the row starts on a 16-byte boundary and the piece lies inside it.
template <Fmt F, int E>
__device__ __forceinline__ void read_piece(const LookupArgs& a, long long r, long long d, bool vec, float (&v)[E]) {
  if constexpr (F == Fmt::kBF16) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.table) + r * a.ld + d;
    if (vec) {
      uint32_t w[E / 2];
      if constexpr (E == 8) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
      } else {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
        w[0] = u.x, w[1] = u.y;
      }
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = d + i < a.D ? __bfloat162float(p[i]) : 0.f;
    }
  } else if constexpr (F == Fmt::kF32) {
    const float* p = static_cast<const float*>(a.table) + r * a.ld + d;
    if (vec) {
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        const float4 u = __ldg(reinterpret_cast<const float4*>(p) + i);
        v[4 * i] = u.x, v[4 * i + 1] = u.y, v[4 * i + 2] = u.z, v[4 * i + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = d + i < a.D ? p[i] : 0.f;
    }
  } else if constexpr (F == Fmt::kE4M3 || F == Fmt::kE4M3E8M0) {
    const uint8_t* p = static_cast<const uint8_t*>(a.table) + r * a.ld + d;
    uint32_t w[E / 4] = {};
    if (vec) {
      if constexpr (E == 8) {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
        w[0] = u.x, w[1] = u.y;
      } else {
        w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (d + i < a.D) w[i / 4] |= static_cast<uint32_t>(p[i]) << (8 * (i % 4));
    }
    const long long g = r * a.lds + (d >> 7);  // a piece never straddles a group of 128
    const float s = F == Fmt::kE4M3 ? static_cast<const float*>(a.scale)[g]
                                    : e8m0_value(static_cast<const uint8_t*>(a.scale)[g]);
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const __half2_raw h =
          __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i / 4] >> (8 * (i % 4))), __NV_E4M3);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      v[i] = f.x * s;
      v[i + 1] = f.y * s;
    }
  } else {
    const uint8_t* p = a.w.q + r * a.w.ldq + d / 2;
    uint32_t w = 0;
    if (vec) {
      w = E == 8 ? __ldg(reinterpret_cast<const uint32_t*>(p)) : __ldg(reinterpret_cast<const uint16_t*>(p));
    } else {
#pragma unroll
      for (int i = 0; i < E / 2; ++i)
        if (d + 2 * i < a.D) w |= static_cast<uint32_t>(p[i]) << (8 * i);
    }
    const long long g = d / a.w.group;  // nor one of 32
    const float s = int4_scale(a.w, r, g);
    const int z = a.w.zero ? a.w.zero[r * a.w.ldz + g] : 8;
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = static_cast<float>(static_cast<int>((w >> (4 * i)) & 15u) - z) * s;
  }
}

template <typename OutT, int E>
__device__ __forceinline__ void write_piece(OutT* p, const float (&v)[E], long long left, bool vec) {
  if constexpr (sizeof(OutT) == 2) {
    if (vec) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
      return;
    }
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i < left) p[i] = __float2bfloat16_rn(v[i]);
  } else {
    if (vec) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
      return;
    }
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i < left) p[i] = v[i];
  }
}

// tvec / ovec: table rows and output rows start on 16-byte boundaries.
template <Fmt F, typename OutT>
__global__ void __launch_bounds__(kThreads) lookup_kernel(const LookupArgs a, uint32_t pieces, bool tvec, bool ovec) {
  constexpr int E = 16 / sizeof(OutT);
  const long long total = a.T * static_cast<long long>(pieces);
  const long long run0 = blockIdx.x * static_cast<long long>(kRun);
  const long long t0 = run0 / pieces;
  const uint32_t rem = static_cast<uint32_t>(run0 - t0 * pieces);
  float v[kUnroll][E];
  long long t[kUnroll], d[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const uint32_t i = threadIdx.x + u * kThreads;
    const uint32_t off = rem + i, row = off / pieces;  // rem < pieces < 2^31
    t[u] = t0 + row;
    d[u] = static_cast<long long>(off - row * pieces) * E;
    if (run0 + i >= total) t[u] = -1;
    if (t[u] < 0) continue;
    const long long r = token_at(a, t[u]);
    if (r >= 0 && r < a.V) {
      read_piece<F, E>(a, r, d[u], tvec && d[u] + E <= a.D, v[u]);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) v[u][e] = 0.f;
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (t[u] < 0) continue;
#pragma unroll
    for (int e = 0; e < E; ++e) v[u][e] *= a.alpha;
    write_piece<OutT, E>(static_cast<OutT*>(a.out) + t[u] * a.ldo + d[u], v[u], a.D - d[u], ovec && d[u] + E <= a.D);
  }
}

bool rows16(const void* base, long long ld_bytes) {
  return (reinterpret_cast<uintptr_t>(base) & 15u) == 0 && ld_bytes % 16 == 0;
}

template <Fmt F, typename OutT>
cudaError_t launch_fmt(const LookupArgs& a, cudaStream_t stream) {
  constexpr int E = 16 / sizeof(OutT);
  const long long pieces = (a.D + E - 1) / E;
  const long long blocks = (a.T * pieces + kRun - 1) / kRun;
  const bool tvec = F == Fmt::kInt4 ? rows16(a.w.q, a.w.ldq)
                                    : rows16(a.table, a.ld * (F == Fmt::kBF16 ? 2 : F == Fmt::kF32 ? 4 : 1));
  const bool ovec = rows16(a.out, a.ldo * static_cast<long long>(sizeof(OutT)));
  lookup_kernel<F, OutT><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a, static_cast<uint32_t>(pieces),
                                                                                 tvec, ovec);
  return cudaGetLastError();
}

template <Fmt F>
cudaError_t launch_out(const LookupArgs& a, cudaStream_t stream) {
  return a.out_bf16 ? launch_fmt<F, __nv_bfloat16>(a, stream) : launch_fmt<F, float>(a, stream);
}

}  // namespace

cudaError_t launch_lookup(const LookupArgs& a, cudaStream_t stream) {
  switch (a.fmt) {
    case BS_TABLE_BF16: return launch_out<Fmt::kBF16>(a, stream);
    case BS_TABLE_F32: return launch_out<Fmt::kF32>(a, stream);
    case BS_TABLE_E4M3: return launch_out<Fmt::kE4M3>(a, stream);
    case BS_TABLE_E4M3_E8M0: return launch_out<Fmt::kE4M3E8M0>(a, stream);
    case BS_TABLE_INT4: return launch_out<Fmt::kInt4>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace bsg
