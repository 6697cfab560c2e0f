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
// A lane handles pieces of 16 output bytes, the lanes of a warp side by side in
// a row (in several where rows are short), the loads of one to eight pieces in
// flight (unroll_of); a warp stays in its rows, so addresses are worked out once
// per row.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "lowbit.h"
#include "sm100.cuh"

namespace bsg {

namespace {

constexpr int kThreads = 256;

enum class Fmt { kBF16, kF32, kE4M3, kE4M3E8M0, kInt4 };

__device__ __forceinline__ long long token_at(const LookupArgs& a, long long t) {
  if (!a.tokens) return t;
  return a.tokens64 ? static_cast<const long long*>(a.tokens)[t] : static_cast<const int*>(a.tokens)[t];
}

// A table row: where its elements, scales and zero points start.
template <Fmt F>
struct Row {
  const uint8_t *data, *scale, *zero;
  bool scale_bf16;
  int group_shift;

  __device__ __forceinline__ Row(const LookupArgs& a, long long r) : scale(nullptr), zero(nullptr) {
    if constexpr (F == Fmt::kInt4) {
      data = a.w.q + r * a.w.ldq;
      scale_bf16 = a.w.scale_bf16;
      scale = static_cast<const uint8_t*>(a.w.scale) + r * a.w.lds * (scale_bf16 ? 2 : 4);
      if (a.w.zero) zero = a.w.zero + r * a.w.ldz;
      group_shift = a.group_shift;
    } else {
      data = static_cast<const uint8_t*>(a.table) + r * a.ld * (F == Fmt::kBF16 ? 2 : (F == Fmt::kF32 ? 4 : 1));
      if constexpr (F == Fmt::kE4M3 || F == Fmt::kE4M3E8M0)
        scale = static_cast<const uint8_t*>(a.scale) + r * a.lds * (F == Fmt::kE4M3 ? 4 : 1);
    }
  }
};

// A piece as read: its bits, and its group's scale (as stored) and zero point.
template <Fmt F, int E>
struct Piece {
  static constexpr int kBytes = F == Fmt::kF32 ? 4 * E : (F == Fmt::kBF16 ? 2 * E : (F == Fmt::kInt4 ? E / 2 : E));
  static constexpr int kWords = (kBytes + 3) / 4;
  uint32_t w[kWords];
  uint32_t s, z;

  // Elements d .. d+E-1 of the row, `left` of which exist (the bits of the others
  // are zero).  `vec`: the row starts on a 16-byte boundary.  A piece never
  // straddles a group (of 32 elements or more).
  __device__ __forceinline__ void load(const Row<F>& row, int d, int left, bool vec) {
    const uint8_t* p = row.data + (F == Fmt::kInt4 ? d / 2 : static_cast<long long>(d) * (kBytes / E));
    if constexpr (F == Fmt::kInt4) {
      const int g = d >> row.group_shift;
      s = row.scale_bf16 ? __ldg(reinterpret_cast<const uint16_t*>(row.scale + 2LL * g))
                         : __ldg(reinterpret_cast<const uint32_t*>(row.scale + 4LL * g));
      z = row.zero ? __ldg(row.zero + g) : 8u;
    }
    if constexpr (F == Fmt::kE4M3) s = __ldg(reinterpret_cast<const uint32_t*>(row.scale) + (d >> 7));
    if constexpr (F == Fmt::kE4M3E8M0) s = __ldg(row.scale + (d >> 7));
    if (vec && left >= E) {
      if constexpr (kBytes >= 16) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) {
          const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + i);
          w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
        }
      } else if constexpr (kBytes == 8) {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
        w[0] = u.x, w[1] = u.y;
      } else if constexpr (kBytes == 4) {
        w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
      } else {
        w[0] = __ldg(reinterpret_cast<const uint16_t*>(p));
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
    if constexpr (F == Fmt::kF32) {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (i < left) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
    } else if constexpr (F == Fmt::kBF16) {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (i < left) w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[i]) << (16 * (i % 2));
    } else if constexpr (F == Fmt::kInt4) {
#pragma unroll
      for (int i = 0; i < E / 2; ++i)
        if (2 * i < left) w[0] |= static_cast<uint32_t>(p[i]) << (8 * i);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (i < left) w[i / 4] |= static_cast<uint32_t>(p[i]) << (8 * (i % 4));
    }
  }

  // Its values in fp32.
  __device__ __forceinline__ void values(const Row<F>& row, float (&v)[E]) const {
    if constexpr (F == Fmt::kF32) {
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = __uint_as_float(w[i]);
    } else if constexpr (F == Fmt::kBF16) {
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    } else if constexpr (F == Fmt::kInt4) {
      const float f = __uint_as_float(row.scale_bf16 ? s << 16 : s);
      // a nibble in the mantissa of 2^23 gives 2^23 + c; less 2^23 + z, exactly
      const float off = -__uint_as_float(0x4B000000u | (z & 15u));
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        uint32_t lo, hi;  // (w >> 4 i) & 15 | 2^23 as one three-input operation after the shift
        asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(lo) : "r"(w[0] >> (4 * i)), "r"(15u), "r"(0x4B000000u));
        asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(hi) : "r"(w[0] >> (4 * i + 4)), "r"(15u), "r"(0x4B000000u));
        const float2 c = __fadd2_rn(make_float2(__uint_as_float(lo), __uint_as_float(hi)), make_float2(off, off));
        const float2 x = __fmul2_rn(c, make_float2(f, f));
        v[i] = x.x;
        v[i + 1] = x.y;
      }
    } else {
      const float f = F == Fmt::kE4M3 ? __uint_as_float(s) : e8m0_to_f32(s);
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        const __half2_raw h =
            __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i / 4] >> (8 * (i % 4))), __NV_E4M3);
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
        v[i] = x.x * f;
        v[i + 1] = x.y * f;
      }
    }
  }
};

template <typename OutT, int E>
__device__ __forceinline__ void write_piece(OutT* p, const float (&v)[E], int left, bool vec) {
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

// U pieces of a row, the first at element d, E * lpr elements apart.  WHOLE: all
// of them exist, on 16-byte boundaries, and lpr is 32 (so that their distances
// are constants).
template <Fmt F, typename OutT, int U, bool WHOLE>
__device__ __forceinline__ void run_pieces(const LookupArgs& a, const Row<F>& row, bool named, int d, int lpr, int D,
                                           bool tvec, bool ovec, OutT* out) {
  constexpr int E = 16 / sizeof(OutT);
  const int apart = WHOLE ? E * 32 : E * lpr;
  Piece<F, E> piece[U];
  if (named) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = d + u * apart;
      if (WHOLE) piece[u].load(row, at, E, true);
      else if (at < D) piece[u].load(row, at, D - at, tvec);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int at = d + u * apart;
    if (!WHOLE && at >= D) break;
    float v[E] = {};
    if (named) {
      piece[u].values(row, v);
      if (a.alpha != 1.f) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] *= a.alpha;
      }
    }
    write_piece<OutT, E>(out + at, v, WHOLE ? E : D - at, WHOLE || (ovec && D - at >= E));
  }
}

// A warp's item: U pieces per lane of 32 / lpr rows, lpr lanes side by side in
// a row.  blockIdx.x: kThreads / 32 items' rows; blockIdx.y: the run of U * lpr
// pieces (gridDim.y runs apart).  tvec / ovec: table rows and output rows start
// on 16-byte boundaries.
template <Fmt F, typename OutT, int U>
__global__ void __launch_bounds__(kThreads, 4) lookup_kernel(const LookupArgs a, int lpr_log2, bool tvec, bool ovec) {
  constexpr int E = 16 / sizeof(OutT);
  const int lane = threadIdx.x & 31, lpr = 1 << lpr_log2;
  const long long t = ((blockIdx.x * static_cast<long long>(kThreads / 32) + threadIdx.x / 32) << (5 - lpr_log2)) + (lane >> lpr_log2);
  if (t >= a.T) return;
  const long long r = token_at(a, t);
  const bool named = r >= 0 && r < a.V;
  const int D = static_cast<int>(a.D);
  OutT* out = static_cast<OutT*>(a.out) + t * a.ldo;
  const Row<F> row(a, named ? r : 0);
  const int step = U * E * lpr;
  for (long long d0 = static_cast<long long>(blockIdx.y) * step; d0 < D; d0 += static_cast<long long>(gridDim.y) * step) {
    const int d = static_cast<int>(d0) + E * (lane & (lpr - 1));
    if (lpr_log2 == 5 && tvec && ovec && D - static_cast<int>(d0) >= step) {
      run_pieces<F, OutT, U, true>(a, row, named, d, 32, D, true, true, out);
    } else {
      run_pieces<F, OutT, U, false>(a, row, named, d, lpr, D, tvec, ovec, out);
    }
  }
}

bool rows16(const void* base, long long ld_bytes) {
  return (reinterpret_cast<uintptr_t>(base) & 15u) == 0 && ld_bytes % 16 == 0;
}

template <Fmt F, typename OutT, int U>
cudaError_t launch_unroll(const LookupArgs& a, cudaStream_t stream) {
  constexpr int E = 16 / sizeof(OutT);
  const long long pieces = (a.D + E - 1) / E;
  int lpr_log2 = 0;
  while (lpr_log2 < 5 && (1 << lpr_log2) < pieces) ++lpr_log2;
  const long long rows = static_cast<long long>(kThreads) >> lpr_log2;  // per block
  const long long runs = (pieces + (U << lpr_log2) - 1) / (U << lpr_log2);
  const bool tvec = F == Fmt::kInt4 ? rows16(a.w.q, a.w.ldq)
                                    : rows16(a.table, a.ld * (F == Fmt::kBF16 ? 2 : F == Fmt::kF32 ? 4 : 1));
  const bool ovec = rows16(a.out, a.ldo * static_cast<long long>(sizeof(OutT)));
  const dim3 grid(static_cast<unsigned>((a.T + rows - 1) / rows), static_cast<unsigned>(runs < 65535 ? runs : 65535));
  lookup_kernel<F, OutT, U><<<grid, kThreads, 0, stream>>>(a, lpr_log2, tvec, ovec);
  return cudaGetLastError();
}

// Pieces per lane of outputs above 4 MB.  More hide the loads' latency until the
// words they hold no longer fit the 64 registers of four blocks per SM: an fp32
// table's piece for bf16 outputs is 8 words, an e4m3 one's 2 and its scale.  16640
// rows of 5120 (and 8192 of 1001), us: fp32 to bf16 2 pieces 80.1 (25.6), 4
// pieces, which spilled, 86.3 (31.9); e4m3 to bf16 4 pieces 48.6 (27.9), 8, which
// spilled, 49.8 (31.2); e4m3 to fp32, no spill, 8 pieces 72.2, 4 pieces 82.6.
// 4-bit tables keep 8, although that spills 64 bytes: 5120 x 8192 read whole to
// bf16 22.2 against 23.7 with 4, to fp32 36.9 against 41.1, 16640 rows of 5120 to
// fp32 78.5 against 86.1, to bf16 51.8 against 50.1.
template <Fmt F, typename OutT>
constexpr int unroll_of() {
  constexpr bool bf16_out = sizeof(OutT) == 2;
  if (F == Fmt::kBF16) return 4;
  if (F == Fmt::kF32) return bf16_out ? 2 : 4;
  if (F == Fmt::kE4M3 || F == Fmt::kE4M3E8M0) return bf16_out ? 4 : 8;
  return 8;
}

// Small lookups spread over as many warps as there are (one piece per lane).
template <Fmt F, typename OutT>
cudaError_t launch_fmt(const LookupArgs& a, cudaStream_t stream) {
  const double bytes = static_cast<double>(a.T) * static_cast<double>(a.D) * sizeof(OutT);
  return bytes <= 4e6 ? launch_unroll<F, OutT, 1>(a, stream) : launch_unroll<F, OutT, unroll_of<F, OutT>()>(a, stream);
}

template <Fmt F>
cudaError_t launch_out(const LookupArgs& a, cudaStream_t stream) {
  return a.out_bf16 ? launch_fmt<F, __nv_bfloat16>(a, stream) : launch_fmt<F, float>(a, stream);
}

}  // namespace

cudaError_t launch_lookup(const LookupArgs& args, cudaStream_t stream) {
  LookupArgs a = args;
  a.group_shift = a.w.group == 32 ? 5 : a.w.group == 64 ? 6 : 7;
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
