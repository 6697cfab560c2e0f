// Quantisation of a matrix to 4-bit codes with one scale (and zero point) per
// group of 32, 64 or 128 consecutive elements of a row (HBM-bound).
//
//   symmetric:  s = fp32(amax / 7), c = clamp(rne(fp32(x / s)), -8, 7) + 8
//   asymmetric: lo = min(0, min x), hi = max(0, max x),
//               s = fp32(fp32(hi / 15) - fp32(lo / 15)),
//               z = clamp(rne(fp32(-lo / s)), 0, 15),
//               c = clamp(rne(fp32(x / s)) + z, 0, 15)
// s is rounded to bf16 first where the scales are bf16 (the codes then go by
// the rounded scale, the one they will be multiplied by), and is 1 where it
// would be 0.  The quotient is the correctly rounded fp32 one, by the same
// correction step as the e4m3 quantisers' (group_quant.cuh).
//
// A lane holds 16 consecutive elements, so group / 16 lanes share a group and
// reduce its range with shuffles; a warp covers 512 elements of a row per
// pass and has one or two passes' loads in flight.  5120 x 8192 bf16 in groups
// of 128 takes 21.9 us, 4.8 TB/s; 5120 x 8192 fp32 in groups of 32 with zero points
// 31.4 us, 6.2 TB/s.  Elements past K read as zero,
// which changes no range and whose code is the zero point, so the unused
// nibble of an odd row's last byte stands for the value zero.
#include <cuda_bf16.h>

#include "group_quant.cuh"
#include "lowbit.h"

namespace bsg {

namespace {

constexpr int kThreads = 256;
constexpr int kWarpElems = 512;

// Elements k .. k+15 of a row, as stored.
template <typename InT>
struct Sixteen {
  uint4 r[sizeof(InT)];

  // Those at or past K are zero; `vec`: all inside the row and 16-byte aligned.
  __device__ __forceinline__ void load(const InT* row, long long k, long long K, bool vec) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(InT)); ++i) r[i] = __ldg(reinterpret_cast<const uint4*>(row + k) + i);
      return;
    }
    uint32_t w[4 * sizeof(InT)] = {};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (k + i >= K) continue;
      if constexpr (sizeof(InT) == 4) w[i] = __float_as_uint(row[k + i]);
      else w[i / 2] |= static_cast<uint32_t>(__bfloat16_as_ushort(row[k + i])) << (16 * (i % 2));
    }
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(InT)); ++i) r[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }

  // Their largest magnitude (of bf16 pairs two at a time).
  __device__ __forceinline__ float amax() const {
    if constexpr (sizeof(InT) == 4) {
      float v[16], m = 0.f;
      values(v);
#pragma unroll
      for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v[i]));
      return m;
    } else {
      uint32_t m = max_abs_bf16x2(max_abs_bf16x2(r[0].x, r[0].y), max_abs_bf16x2(r[0].z, r[0].w));
      m = max_abs_bf16x2(m, max_abs_bf16x2(max_abs_bf16x2(r[1].x, r[1].y), max_abs_bf16x2(r[1].z, r[1].w)));
      return fmaxf(__uint_as_float((m << 16) & 0x7FFFFFFFu), __uint_as_float(m & 0x7FFF0000u));
    }
  }

  __device__ __forceinline__ void values(float (&v)[16]) const {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(InT)); ++i) {
      const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(InT) == 4) {
          v[4 * i + j] = __uint_as_float(w[j]);
        } else {
          v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
          v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
      }
    }
  }
};

// a / 7 and a / 15, correctly rounded, by Markstein's correction step (see
// quotient_rn in group_quant.cuh) where nothing under- or overflows: the
// divisor's reciprocal is a constant, and every significand was checked.
template <int DIV>
__device__ __forceinline__ float over_const(float a) {
  static_assert(DIV == 7 || DIV == 15, "constants below");
  constexpr float r = DIV == 7 ? 0x1.24924ap-3f : 0x1.111112p-4f;
  if (!(fabsf(a) >= 0x1p-100f && fabsf(a) <= 3.40282347e38f)) return __fdiv_rn(a, static_cast<float>(DIV));
  const float q1 = __fmul_rn(a, r);
  return __fmaf_rn(__fmaf_rn(-q1, static_cast<float>(DIV), a), r, q1);
}

// The codes of a lane's 16 elements, eight to a word: rne(v / s) + z clamped to
// 0..15.  Adding 1.5 * 2^23 to a quotient rounds it to an integer, ties to even,
// in the low bits of the sum, and a further z (an integer) is added exactly; so
// a code is the low nibble of its sum, and a Horner chain in 16 collects them:
// the sums' common high bits add up to a constant.  FAST: packed two-wide
// operations on the fp32 correction step, for scales in its range -- where a
// symmetric group's quotients lie in [-7.03, 7.03] (7 and half a bf16 step of the
// scale) and need no clamp; otherwise any scale.
template <bool ASYM, bool FAST>
__device__ __forceinline__ void codes16(const float (&v)[16], float s, float z, uint32_t (&w)[2]) {
  constexpr float kRound = 12582912.f;  // 1.5 * 2^23
  float2 q[8];
  if constexpr (FAST) {
    const float r = __frcp_rn(s);
    const float2 r2 = make_float2(r, r), ns2 = make_float2(-s, -s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = make_float2(v[2 * i], v[2 * i + 1]);
      const float2 q1 = __fmul2_rn(x, r2);
      q[i] = __ffma2_rn(__ffma2_rn(q1, ns2, x), r2, q1);
    }
  } else {
    const double rinv = __drcp_rn(static_cast<double>(s));
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = make_float2(over_scale(v[2 * i], rinv), over_scale(v[2 * i + 1], rinv));
  }
  uint32_t c[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (ASYM || !FAST) {  // both ends are integers, so clamping before the rounding is the same
      q[i].x = fminf(fmaxf(q[i].x, -z), 15.f - z);
      q[i].y = fminf(fmaxf(q[i].y, -z), 15.f - z);
    }
    float2 n;
    if constexpr (ASYM) {
      n = __fadd2_rn(__fadd2_rn(q[i], make_float2(kRound, kRound)), make_float2(z, z));
    } else {
      n = __fadd2_rn(q[i], make_float2(kRound + 8.f, kRound + 8.f));  // 8 is even: ties go the same way
    }
    c[2 * i] = __float_as_uint(n.x);
    c[2 * i + 1] = __float_as_uint(n.y);
  }
  constexpr uint32_t kHigh = 0x4B400000u;  // the bits of 1.5 * 2^23
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t t = c[8 * h + 7];
#pragma unroll
    for (int i = 6; i >= 0; --i) t = t * 16u + c[8 * h + i];
    w[h] = t - kHigh * 0x11111111u;
  }
}

template <typename InT, typename ScaleT, bool ASYM, int LANES, int kPasses>
__global__ void __launch_bounds__(kThreads, kPasses == 1 || sizeof(InT) == 2 ? 6 : 5)
    quantize_int4_kernel(const InT* __restrict__ x, long long N, long long K, long long ldx, uint8_t* __restrict__ q,
                         long long ldq, ScaleT* __restrict__ scale, long long lds, uint8_t* __restrict__ zero,
                         long long ldz) {
  constexpr int kGroup = 16 * LANES;
  const int lane = threadIdx.x & 31;
  const long long per_row = (K + kPasses * kWarpElems - 1) / (kPasses * kWarpElems);
  const long long it = blockIdx.x * static_cast<long long>(kThreads / 32) + threadIdx.x / 32;
  const long long n = it / per_row;
  if (n >= N) return;  // the whole warp
  const long long k0 = (it - n * per_row) * (kPasses * kWarpElems) + 16 * lane;
  const InT* row = x + n * ldx;
  uint8_t* qrow = q + n * ldq;
  const bool row_vec = (reinterpret_cast<uintptr_t>(row) & 15u) == 0;
  const bool q_vec = (reinterpret_cast<uintptr_t>(qrow) & 7u) == 0;
  Sixteen<InT> raw[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const long long k = k0 + p * kWarpElems;
    raw[p].load(row, k, K, row_vec && k + 16 <= K);
  }
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const long long k = k0 + p * kWarpElems;
    float v[16];
    raw[p].values(v);
    float lo = 0.f, hi = 0.f;
    if constexpr (ASYM) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        lo = fminf(lo, v[i]);
        hi = fmaxf(hi, v[i]);
      }
    } else {
      hi = raw[p].amax();
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      if constexpr (ASYM) lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    }
    float s = ASYM ? __fsub_rn(over_const<15>(hi), over_const<15>(lo)) : over_const<7>(hi);
    if constexpr (sizeof(ScaleT) == 2) s = __bfloat162float(__float2bfloat16_rn(s));
    if (s == 0.f) s = 1.f;
    float z = 8.f;  // the code of zero
    if constexpr (ASYM) z = fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.f), 15.f);
    uint32_t w[2];
    if (__all_sync(0xffffffffu, quotient_fast_range(s) && hi <= 3.40282347e38f)) {
      codes16<ASYM, true>(v, s, z, w);
    } else {
      codes16<ASYM, false>(v, s, z, w);
    }
    if (k < K) {
      if (lane % LANES == 0) {
        const long long g = k / kGroup;
        if constexpr (sizeof(ScaleT) == 2) {
          scale[n * lds + g] = __float2bfloat16_rn(s);
        } else {
          scale[n * lds + g] = s;
        }
        if constexpr (ASYM) zero[n * ldz + g] = static_cast<uint8_t>(z);
      }
      uint8_t* dst = qrow + k / 2;
      if (q_vec && k + 16 <= K) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (k + 2 * i < K) dst[i] = static_cast<uint8_t>(w[i / 4] >> (8 * (i % 4)));
      }
    }
  }
}

template <typename InT, typename ScaleT, bool ASYM, int LANES, int PASSES>
cudaError_t launch_passes(const void* x, long long N, long long K, long long ldx, uint8_t* q, long long ldq, void* scale,
                          long long lds, uint8_t* zero, long long ldz, cudaStream_t stream) {
  const long long items = N * ((K + PASSES * kWarpElems - 1) / (PASSES * kWarpElems));
  const long long blocks = (items + kThreads / 32 - 1) / (kThreads / 32);
  quantize_int4_kernel<InT, ScaleT, ASYM, LANES, PASSES><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(
      static_cast<const InT*>(x), N, K, ldx, q, ldq, static_cast<ScaleT*>(scale), lds, zero, ldz);
  return cudaGetLastError();
}

// Two passes per warp for large matrices, one for up to 2^24 elements: more warps
// (1024 x 4096 fp32 5.5 against 6.2 us, 2085 x 4099 bf16 7.5 against 9.1; 5120 x
// 8192 bf16 25.3 against 21.9).
template <typename InT, typename ScaleT, bool ASYM, int LANES>
cudaError_t launch_one(const void* x, long long N, long long K, long long ldx, uint8_t* q, long long ldq, void* scale,
                       long long lds, uint8_t* zero, long long ldz, cudaStream_t stream) {
  return N * K <= (1 << 24)
             ? launch_passes<InT, ScaleT, ASYM, LANES, 1>(x, N, K, ldx, q, ldq, scale, lds, zero, ldz, stream)
             : launch_passes<InT, ScaleT, ASYM, LANES, 2>(x, N, K, ldx, q, ldq, scale, lds, zero, ldz, stream);
}

template <typename InT, typename ScaleT, bool ASYM, typename... A>
cudaError_t launch_group(int group, A... a) {
  if (group == 32) return launch_one<InT, ScaleT, ASYM, 2>(a...);
  return group == 64 ? launch_one<InT, ScaleT, ASYM, 4>(a...) : launch_one<InT, ScaleT, ASYM, 8>(a...);
}

template <typename InT, typename ScaleT, typename... A>
cudaError_t launch_asym(bool asym, A... a) {
  return asym ? launch_group<InT, ScaleT, true>(a...) : launch_group<InT, ScaleT, false>(a...);
}

}  // namespace

cudaError_t launch_quantize_int4(const void* x, bool x_bf16, long long N, long long K, long long ldx, uint8_t* q,
                                 long long ldq, void* scale, bool scale_bf16, long long lds, uint8_t* zero,
                                 long long ldz, int group, cudaStream_t stream) {
  const bool asym = zero != nullptr;
  if (x_bf16)
    return scale_bf16 ? launch_asym<__nv_bfloat16, __nv_bfloat16>(asym, group, x, N, K, ldx, q, ldq, scale, lds, zero,
                                                                  ldz, stream)
                      : launch_asym<__nv_bfloat16, float>(asym, group, x, N, K, ldx, q, ldq, scale, lds, zero, ldz,
                                                          stream);
  return scale_bf16
             ? launch_asym<float, __nv_bfloat16>(asym, group, x, N, K, ldx, q, ldq, scale, lds, zero, ldz, stream)
             : launch_asym<float, float>(asym, group, x, N, K, ldx, q, ldq, scale, lds, zero, ldz, stream);
}

}  // namespace bsg
