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
// pass and has two passes' loads in flight.  Elements past K read as zero,
// which changes no range and whose code is the zero point, so the unused
// nibble of an odd row's last byte stands for the value zero.
#include <cuda_bf16.h>

#include "group_quant.cuh"
#include "lowbit.h"

namespace bsg {

namespace {

constexpr int kThreads = 256;
constexpr int kPasses = 2;
constexpr int kWarpElems = 512;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// Elements k .. k+15 of a row (zero at or past K); `vec`: all inside the row
// and 16-byte aligned.
template <typename InT>
__device__ __forceinline__ void load16(const InT* row, long long k, long long K, bool vec, float (&v)[16]) {
  if (vec) {
    constexpr int kPer = 16 / sizeof(InT);
#pragma unroll
    for (int i = 0; i < 16 / kPer; ++i) {
      const uint4 t = __ldg(reinterpret_cast<const uint4*>(row + k) + i);
      const uint32_t w[4] = {t.x, t.y, t.z, t.w};
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
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = k + i < K ? to_f32(row[k + i]) : 0.f;
  }
}

// The integer nearest to y (ties to even) in the low bits of the result, for
// |y| < 2^22: 1.5 * 2^23 + y has an ulp of one.
__device__ __forceinline__ int rne_bits(float y) { return __float_as_int(__fadd_rn(y, 12582912.f)); }

template <typename InT, typename ScaleT, bool ASYM, int LANES>
__global__ void __launch_bounds__(kThreads)
    quantize_int4_kernel(const InT* __restrict__ x, long long N, long long K, long long ldx, uint8_t* __restrict__ q,
                         long long ldq, ScaleT* __restrict__ scale, long long lds, uint8_t* __restrict__ zero,
                         long long ldz) {
  constexpr int kGroup = 16 * LANES;
  const int lane = threadIdx.x & 31;
  const long long per_row = (K + kPasses * kWarpElems - 1) / (kPasses * kWarpElems);
  const long long items = N * per_row;
  const long long warps = static_cast<long long>(gridDim.x) * (kThreads / 32);
  for (long long it = blockIdx.x * static_cast<long long>(kThreads / 32) + threadIdx.x / 32; it < items; it += warps) {
    const long long n = it / per_row;
    const long long k0 = (it - n * per_row) * (kPasses * kWarpElems) + 16 * lane;
    const InT* row = x + n * ldx;
    uint8_t* qrow = q + n * ldq;
    const bool row_vec = (reinterpret_cast<uintptr_t>(row) & 15u) == 0;
    float v[kPasses][16];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const long long k = k0 + p * kWarpElems;
      load16<InT>(row, k, K, row_vec && k + 16 <= K, v[p]);
    }
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const long long k = k0 + p * kWarpElems;
      float lo = 0.f, hi = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if constexpr (ASYM) {
          lo = fminf(lo, v[p][i]);
          hi = fmaxf(hi, v[p][i]);
        } else {
          hi = fmaxf(hi, fabsf(v[p][i]));
        }
      }
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) {
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        if constexpr (ASYM) lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      }
      float s = ASYM ? __fsub_rn(__fdiv_rn(hi, 15.f), __fdiv_rn(lo, 15.f)) : __fdiv_rn(hi, 7.f);
      if constexpr (sizeof(ScaleT) == 2) s = __bfloat162float(__float2bfloat16_rn(s));
      if (s == 0.f) s = 1.f;
      float z = 8.f;  // the code of zero
      if constexpr (ASYM) {
        z = fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.f), 15.f);
      }
      float y[16];
      code_quotients<16>(v[p], s, y);
      uint32_t w[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        // rne(y) + z clamped to 0..15: clamping y to [-z, 15 - z] first is the
        // same, both ends being integers
        const int c = rne_bits(fminf(fmaxf(y[i], -z), 15.f - z)) + static_cast<int>(z);
        w[i / 8] |= static_cast<uint32_t>(c & 15) << (4 * (i % 8));
      }
      if (k >= K) continue;
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
      if (k + 16 <= K && (reinterpret_cast<uintptr_t>(dst) & 7u) == 0) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (k + 2 * i < K) dst[i] = static_cast<uint8_t>(w[i / 4] >> (8 * (i % 4)));
      }
    }
  }
}

template <typename InT, typename ScaleT, bool ASYM, int LANES>
cudaError_t launch_one(const void* x, long long N, long long K, long long ldx, uint8_t* q, long long ldq, void* scale,
                       long long lds, uint8_t* zero, long long ldz, int sms, cudaStream_t stream) {
  const long long items = N * ((K + kPasses * kWarpElems - 1) / (kPasses * kWarpElems));
  long long blocks = (items + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 8LL * sms) blocks = 8LL * sms;
  quantize_int4_kernel<InT, ScaleT, ASYM, LANES><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(
      static_cast<const InT*>(x), N, K, ldx, q, ldq, static_cast<ScaleT*>(scale), lds, zero, ldz);
  return cudaGetLastError();
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
                                 long long ldz, int group, int sms, cudaStream_t stream) {
  const bool asym = zero != nullptr;
  if (x_bf16)
    return scale_bf16 ? launch_asym<__nv_bfloat16, __nv_bfloat16>(asym, group, x, N, K, ldx, q, ldq, scale, lds, zero,
                                                                  ldz, sms, stream)
                      : launch_asym<__nv_bfloat16, float>(asym, group, x, N, K, ldx, q, ldq, scale, lds, zero, ldz,
                                                          sms, stream);
  return scale_bf16
             ? launch_asym<float, __nv_bfloat16>(asym, group, x, N, K, ldx, q, ldq, scale, lds, zero, ldz, sms, stream)
             : launch_asym<float, float>(asym, group, x, N, K, ldx, q, ldq, scale, lds, zero, ldz, sms, stream);
}

}  // namespace bsg
