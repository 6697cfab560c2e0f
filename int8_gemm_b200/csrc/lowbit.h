// Internal interface of the 4-bit weight kernels (kernels_int4_quant.cu,
// kernels_int4_gemv.cu) and the row lookup and its gradient
// (kernels_lookup.cu, kernels_lookup_grad.cu) for the C-ABI layer
// (api_lowbit.cu).  Not part of the public header.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bsgemm.h"

namespace bsg {

// ---- shared with api.cu -----------------------------------------------------
// The calling thread's error message, and the current device's facts (its SM
// count and the error word of the bounded waits).
bs_status api_fail(bs_status st, const char* fmt, ...);
void api_clear();
bs_status api_device(int* sms, uint32_t** err);
bs_status api_launched(cudaError_t e, const char* what);
// Tensor map of N rows of `bytes` bytes, ldq apart, in boxes of box_bytes x
// box_rows.
bs_status api_map_codes(CUtensorMap* map, const void* q, int64_t bytes, int64_t N, int64_t ldq, uint32_t box_bytes,
                        uint32_t box_rows, CUtensorMapSwizzle swizzle);

// ---- 4-bit matrices ---------------------------------------------------------
// Codes 0..15 of a matrix [N, K], two to a byte (even k in the low nibble),
// row n at q + n * ldq; one scale (and zero point, 8 where `zero` is null) per
// row and `group` consecutive k: value = scale * (code - zero).
struct Int4Matrix {
  const uint8_t* q;
  long long ldq;
  const void* scale;
  bool scale_bf16;
  long long lds;
  const uint8_t* zero;
  long long ldz;
  int group;  // 32, 64 or 128
};

cudaError_t launch_quantize_int4(const void* x, bool x_bf16, long long N, long long K, long long ldx, uint8_t* q,
                                 long long ldq, void* scale, bool scale_bf16, long long lds, uint8_t* zero,
                                 long long ldz, int group, cudaStream_t stream);

constexpr int kInt4MaxM = 32;  // activation rows of one product
struct Int4Product {
  const void* x;
  bool x_bf16;
  long long ldx;
  Int4Matrix w;
  const float* bias;
  void* out;
  bool out_bf16;
  long long ldo;
  int M;
  long long N, K;
};
constexpr int kInt4BoxBytes = 64;  // bytes of a matrix row per tensor copy (64-byte swizzle)
cudaError_t launch_gemv_int4(const Int4Product& p, int sms, uint32_t* err, cudaStream_t stream);

// ---- lookup -----------------------------------------------------------------
// out[t, :] = alpha * table[tokens[t], :]; tokens null: row t itself.
struct LookupArgs {
  const void* tokens;
  bool tokens64;
  long long T;
  const void* table;  // unused for 4-bit tables (`w` describes them)
  bs_table_fmt fmt;
  long long ld;       // elements (bytes for e4m3)
  const void* scale;  // e4m3: one per row and 128 elements
  long long lds;
  Int4Matrix w;
  long long V, D;
  float alpha;
  void* out;
  bool out_bf16;
  long long ldo;
  int group_shift;  // filled in by launch_lookup
};
cudaError_t launch_lookup(const LookupArgs& a, cudaStream_t stream);

struct LookupGradArgs {
  const void* tokens;
  bool tokens64;
  long long T;
  const void* grad;
  bool grad_bf16;
  long long ldg;
  long long V, D;
  float alpha;
  long long padding_idx;  // negative: none
  void* out;
  bool out_bf16;
  long long ldo;
  bool accumulate;
  void* workspace;
};
size_t lookup_grad_workspace(long long T, long long V, long long D);
cudaError_t launch_lookup_grad(const LookupGradArgs& a, int sms, cudaStream_t stream);

}  // namespace bsg
