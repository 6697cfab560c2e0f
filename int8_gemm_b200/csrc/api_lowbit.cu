// C-ABI layer of the 4-bit weight operators and the row lookup with its
// gradient: argument validation and launches, in the manner of api.cu.
#include "launch.h"
#include "lowbit.h"

using namespace bsg;

namespace {

constexpr int64_t kMaxDim = 0x7FFFFFFF;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
uintptr_t in_size(bs_in_dtype t) { return t == BS_IN_BF16 ? 2 : 4; }
bool in_known(bs_in_dtype t) { return t == BS_IN_BF16 || t == BS_IN_F32; }
uintptr_t out_size(bs_out_dtype t) { return t == BS_OUT_BF16 ? 2 : 4; }
bool out_known(bs_out_dtype t) { return t == BS_OUT_BF16 || t == BS_OUT_F32; }

// Whether `rows` rows of `ld` elements of `size` bytes stay within 63 bits of
// address arithmetic.
bool extent_ok(int64_t rows, int64_t ld, int64_t size) {
  return ld <= (INT64_MAX / 16) / (rows > 0 ? rows : 1) / size;
}

// The checks that every operator on a 4-bit matrix shares.
bs_status check_int4(const void* q, int64_t ldq, const void* scale, bs_in_dtype scale_dtype, int64_t ld_scale,
                     const uint8_t* zero, int64_t ld_zero, int32_t group, int64_t N, int64_t K) {
  if (!in_known(scale_dtype)) return api_fail(BS_ERR_DTYPE, "scales must be bf16 or f32");
  if (group != 32 && group != 64 && group != 128)
    return api_fail(BS_ERR_SHAPE, "group=%d: groups of 32, 64 or 128 elements", group);
  if (N == 0 || K == 0) return BS_OK;
  if (!q || !scale) return api_fail(BS_ERR_NULL, "q and scale must be non-NULL");
  const int64_t bytes = (K + 1) / 2, groups = (K + group - 1) / group;
  if (ldq < bytes || ld_scale < groups || (zero && ld_zero < groups))
    return api_fail(BS_ERR_LAYOUT, "ldq must be >= ceil(K/2) = %lld, ld_scale and ld_zero >= ceil(K/group) = %lld",
                    (long long)bytes, (long long)groups);
  if (!extent_ok(N, ldq, 1) || !extent_ok(N, ld_scale, 4) || (zero && !extent_ok(N, ld_zero, 1)))
    return api_fail(BS_ERR_LAYOUT, "a stride times the number of rows is out of range");
  if (!aligned(scale, in_size(scale_dtype))) return api_fail(BS_ERR_ALIGNMENT, "scales must be aligned to their size");
  return BS_OK;
}

Int4Matrix int4_matrix(const void* q, int64_t ldq, const void* scale, bs_in_dtype scale_dtype, int64_t ld_scale,
                       const uint8_t* zero, int64_t ld_zero, int32_t group) {
  Int4Matrix w;
  w.q = static_cast<const uint8_t*>(q);
  w.ldq = ldq;
  w.scale = scale;
  w.scale_bf16 = scale_dtype == BS_IN_BF16;
  w.lds = ld_scale;
  w.zero = zero;
  w.ldz = ld_zero;
  w.group = group;
  return w;
}

// Checks of a lookup's output and size: [T, D] with 16-byte pieces counted in
// 31-bit blocks.
bs_status check_rows_out(const void* out, bs_out_dtype out_dtype, int64_t ldo, int64_t T, int64_t D) {
  if (!out) return api_fail(BS_ERR_NULL, "out is NULL");
  if (ldo < D) return api_fail(BS_ERR_LAYOUT, "ldo=%lld < %lld", (long long)ldo, (long long)D);
  if (!extent_ok(T, ldo, 4)) return api_fail(BS_ERR_LAYOUT, "a stride times the number of rows is out of range");
  if (!aligned(out, out_size(out_dtype))) return api_fail(BS_ERR_ALIGNMENT, "out must be aligned to its element size");
  if (D > (kMaxDim >> 1)) return api_fail(BS_ERR_SHAPE, "rows of more than 2^30-1 elements");
  if (T * ((D + 3) / 4) / 1024 >= kMaxDim)
    return api_fail(BS_ERR_SHAPE, "rows of %lld elements, %lld of them: about 2^43 elements or more", (long long)D, (long long)T);
  return BS_OK;
}

}  // namespace

extern "C" {

bs_status bs_quantize_int4(const void* x, bs_in_dtype x_dtype, int64_t N, int64_t K, int64_t ldx, void* q, int64_t ldq,
                           void* scale, bs_in_dtype scale_dtype, int64_t ld_scale, uint8_t* zero, int64_t ld_zero,
                           int32_t group, void* stream) {
  api_clear();
  if (N < 0 || K < 0) return api_fail(BS_ERR_SHAPE, "negative size N=%lld K=%lld", (long long)N, (long long)K);
  if (N > kMaxDim || K > kMaxDim) return api_fail(BS_ERR_SHAPE, "size exceeds 2^31-1");
  if (!in_known(x_dtype)) return api_fail(BS_ERR_DTYPE, "x must be bf16 or f32");
  bs_status st = check_int4(q, ldq, scale, scale_dtype, ld_scale, zero, ld_zero, group, N, K);
  if (st != BS_OK) return st;
  if (N == 0 || K == 0) return BS_OK;
  if (!x) return api_fail(BS_ERR_NULL, "x is NULL");
  if (ldx < K) return api_fail(BS_ERR_LAYOUT, "ldx=%lld < K=%lld", (long long)ldx, (long long)K);
  if (!extent_ok(N, ldx, 4)) return api_fail(BS_ERR_LAYOUT, "a stride times the number of rows is out of range");
  if (!aligned(x, in_size(x_dtype))) return api_fail(BS_ERR_ALIGNMENT, "x must be aligned to its element size");
  if (N * ((K + 1023) / 1024) / 8 >= kMaxDim) return api_fail(BS_ERR_SHAPE, "more than 2^44 elements");
  int sms = 0;
  uint32_t* err = nullptr;
  if ((st = api_device(&sms, &err)) != BS_OK) return st;
  return api_launched(
      launch_quantize_int4(x, x_dtype == BS_IN_BF16, N, K, ldx, static_cast<uint8_t*>(q), ldq, scale,
                           scale_dtype == BS_IN_BF16, ld_scale, zero, ld_zero, group,
                           static_cast<cudaStream_t>(stream)),
      "4-bit quantise launch");
}

bs_status bs_dequantize_int4(const void* q, int64_t ldq, const void* scale, bs_in_dtype scale_dtype, int64_t ld_scale,
                             const uint8_t* zero, int64_t ld_zero, int32_t group, void* out, bs_out_dtype out_dtype,
                             int64_t ldo, int64_t N, int64_t K, void* stream) {
  api_clear();
  if (N < 0 || K < 0) return api_fail(BS_ERR_SHAPE, "negative size N=%lld K=%lld", (long long)N, (long long)K);
  if (N > kMaxDim || K > kMaxDim) return api_fail(BS_ERR_SHAPE, "size exceeds 2^31-1");
  if (!out_known(out_dtype)) return api_fail(BS_ERR_DTYPE, "bs_dequantize_int4 writes bf16 or f32 only");
  bs_status st = check_int4(q, ldq, scale, scale_dtype, ld_scale, zero, ld_zero, group, N, K);
  if (st != BS_OK) return st;
  if (N == 0 || K == 0) return BS_OK;
  if ((st = check_rows_out(out, out_dtype, ldo, N, K)) != BS_OK) return st;
  int sms = 0;
  uint32_t* err = nullptr;
  if ((st = api_device(&sms, &err)) != BS_OK) return st;
  LookupArgs a = {};
  a.T = a.V = N;
  a.D = K;
  a.fmt = BS_TABLE_INT4;
  a.w = int4_matrix(q, ldq, scale, scale_dtype, ld_scale, zero, ld_zero, group);
  a.alpha = 1.f;
  a.out = out;
  a.out_bf16 = out_dtype == BS_OUT_BF16;
  a.ldo = ldo;
  return api_launched(launch_lookup(a, static_cast<cudaStream_t>(stream)), "4-bit dequantise launch");
}

bs_status bs_gemv_int4(const void* x, bs_in_dtype x_dtype, int64_t ldx, const void* q, int64_t ldq, const void* scale,
                       bs_in_dtype scale_dtype, int64_t ld_scale, const uint8_t* zero, int64_t ld_zero, int32_t group,
                       const float* bias, void* out, bs_out_dtype out_dtype, int64_t ldo, int64_t M, int64_t N,
                       int64_t K, void* stream) {
  api_clear();
  if (M < 0 || N < 0 || K < 0)
    return api_fail(BS_ERR_SHAPE, "negative size M=%lld N=%lld K=%lld", (long long)M, (long long)N, (long long)K);
  if (M > kInt4MaxM)
    return api_fail(BS_ERR_SHAPE, "M=%lld: at most %d rows (bs_dequantize_int4 and a GEMM serve more)", (long long)M,
                    kInt4MaxM);
  if (N > (kMaxDim >> 1) || K > (kMaxDim >> 1)) return api_fail(BS_ERR_SHAPE, "size exceeds 2^30-1");
  if (!in_known(x_dtype)) return api_fail(BS_ERR_DTYPE, "x must be bf16 or f32");
  if (!out_known(out_dtype)) return api_fail(BS_ERR_DTYPE, "bs_gemv_int4 writes bf16 or f32 only");
  bs_status st = check_int4(q, ldq, scale, scale_dtype, ld_scale, zero, ld_zero, group, N, K);
  if (st != BS_OK) return st;
  if (M == 0 || N == 0) return BS_OK;
  if ((st = check_rows_out(out, out_dtype, ldo, M, N)) != BS_OK) return st;
  if (bias && !aligned(bias, 4)) return api_fail(BS_ERR_ALIGNMENT, "bias must be 4-byte aligned");
  if (K > 0) {
    if (!x) return api_fail(BS_ERR_NULL, "x is NULL");
    if (ldx < K) return api_fail(BS_ERR_LAYOUT, "ldx=%lld < K=%lld", (long long)ldx, (long long)K);
    if (!extent_ok(M, ldx, 4)) return api_fail(BS_ERR_LAYOUT, "a stride times the number of rows is out of range");
    if (!aligned(x, in_size(x_dtype))) return api_fail(BS_ERR_ALIGNMENT, "x must be aligned to its element size");
    if (!aligned(q, 16) || ldq % 16 != 0)
      return api_fail(BS_ERR_ALIGNMENT, "q must be 16-byte aligned with ldq a multiple of 16");
    if (ldq >= (int64_t{1} << 40)) return api_fail(BS_ERR_LAYOUT, "ldq must be below 2^40");  // tensor map strides
  }
  int sms = 0;
  uint32_t* err = nullptr;
  if ((st = api_device(&sms, &err)) != BS_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (K == 0)
    return api_launched(launch_fill_zero(out, static_cast<int>(out_size(out_dtype)), M, N, ldo, 1, 0, cs, bias),
                        "bias-fill launch");
  Int4Product p;
  p.x = x;
  p.x_bf16 = x_dtype == BS_IN_BF16;
  p.ldx = ldx;
  p.w = int4_matrix(q, ldq, scale, scale_dtype, ld_scale, zero, ld_zero, group);
  p.bias = bias;
  p.out = out;
  p.out_bf16 = out_dtype == BS_OUT_BF16;
  p.ldo = ldo;
  p.M = static_cast<int>(M);
  p.N = N;
  p.K = K;
  return api_launched(launch_gemv_int4(p, sms, err, cs), "4-bit product launch");
}

bs_status bs_embedding(const void* tokens, bs_index_dtype token_dtype, int64_t T, const void* table, bs_table_fmt format,
                       int64_t ld_table, const void* scale, bs_in_dtype scale_dtype, int64_t ld_scale,
                       const uint8_t* zero, int64_t ld_zero, int32_t group, int64_t V, int64_t D, float alpha, void* out,
                       bs_out_dtype out_dtype, int64_t ldo, void* stream) {
  api_clear();
  if (T < 0 || V < 0 || D < 0) return api_fail(BS_ERR_SHAPE, "negative size T=%lld V=%lld D=%lld", (long long)T,
                                               (long long)V, (long long)D);
  if (T > kMaxDim || V > kMaxDim || D > kMaxDim) return api_fail(BS_ERR_SHAPE, "size exceeds 2^31-1");
  if (token_dtype != BS_INDEX_I32 && token_dtype != BS_INDEX_I64)
    return api_fail(BS_ERR_DTYPE, "tokens must be int32 or int64");
  if (!out_known(out_dtype)) return api_fail(BS_ERR_DTYPE, "bs_embedding writes bf16 or f32 only");
  bs_status st = BS_OK;
  switch (format) {
    case BS_TABLE_INT4:
      st = check_int4(table, ld_table, scale, scale_dtype, ld_scale, zero, ld_zero, group, V, D);
      if (st != BS_OK) return st;
      break;
    case BS_TABLE_BF16:
    case BS_TABLE_F32:
    case BS_TABLE_E4M3:
    case BS_TABLE_E4M3_E8M0: {
      if (V == 0 || D == 0) break;
      const uintptr_t size = format == BS_TABLE_BF16 ? 2 : (format == BS_TABLE_F32 ? 4 : 1);
      if (!table) return api_fail(BS_ERR_NULL, "table is NULL");
      if (ld_table < D) return api_fail(BS_ERR_LAYOUT, "ld_table=%lld < D=%lld", (long long)ld_table, (long long)D);
      if (!extent_ok(V, ld_table, 4)) return api_fail(BS_ERR_LAYOUT, "a stride times the number of rows is out of range");
      if (!aligned(table, size)) return api_fail(BS_ERR_ALIGNMENT, "table must be aligned to its element size");
      if (size == 1) {
        const int64_t groups = (D + 127) / 128;
        if (!scale) return api_fail(BS_ERR_NULL, "an e4m3 table needs its scales");
        if (ld_scale < groups) return api_fail(BS_ERR_LAYOUT, "ld_scale must be >= ceil(D/128) = %lld", (long long)groups);
        if (!extent_ok(V, ld_scale, 4))
          return api_fail(BS_ERR_LAYOUT, "a stride times the number of rows is out of range");
        if (format == BS_TABLE_E4M3 && !aligned(scale, 4))
          return api_fail(BS_ERR_ALIGNMENT, "fp32 scales must be 4-byte aligned");
      }
      break;
    }
    default: return api_fail(BS_ERR_DTYPE, "unknown table format %d", static_cast<int>(format));
  }
  if (T == 0 || D == 0) return BS_OK;
  if (!tokens) return api_fail(BS_ERR_NULL, "tokens is NULL");
  if (!aligned(tokens, token_dtype == BS_INDEX_I64 ? 8 : 4))
    return api_fail(BS_ERR_ALIGNMENT, "tokens must be aligned to their size");
  if ((st = check_rows_out(out, out_dtype, ldo, T, D)) != BS_OK) return st;
  int sms = 0;
  uint32_t* err = nullptr;
  if ((st = api_device(&sms, &err)) != BS_OK) return st;
  LookupArgs a = {};
  a.tokens = tokens;
  a.tokens64 = token_dtype == BS_INDEX_I64;
  a.T = T;
  a.table = table;
  a.fmt = format;
  a.ld = ld_table;
  a.scale = scale;
  a.lds = ld_scale;
  if (format == BS_TABLE_INT4)
    a.w = int4_matrix(table, ld_table, scale, scale_dtype, ld_scale, zero, ld_zero, group);
  a.V = V;
  a.D = D;
  a.alpha = alpha;
  a.out = out;
  a.out_bf16 = out_dtype == BS_OUT_BF16;
  a.ldo = ldo;
  return api_launched(launch_lookup(a, static_cast<cudaStream_t>(stream)), "lookup launch");
}

size_t bs_embedding_grad_workspace(int64_t T, int64_t V, int64_t D) {
  if (T < 0 || V < 0 || D < 0 || T > kMaxDim || V > kMaxDim || D > kMaxDim) return 0;
  return lookup_grad_workspace(T, V, D);
}

bs_status bs_embedding_grad(const void* tokens, bs_index_dtype token_dtype, int64_t T, const void* grad,
                            bs_in_dtype grad_dtype, int64_t ldg, int64_t V, int64_t D, float alpha, int64_t padding_idx,
                            void* d, bs_out_dtype d_dtype, int64_t ldd, int32_t accumulate, void* workspace,
                            size_t workspace_bytes, void* stream) {
  api_clear();
  if (T < 0 || V < 0 || D < 0) return api_fail(BS_ERR_SHAPE, "negative size T=%lld V=%lld D=%lld", (long long)T,
                                               (long long)V, (long long)D);
  if (T > kMaxDim || V > kMaxDim || D > kMaxDim) return api_fail(BS_ERR_SHAPE, "size exceeds 2^31-1");
  if (token_dtype != BS_INDEX_I32 && token_dtype != BS_INDEX_I64)
    return api_fail(BS_ERR_DTYPE, "tokens must be int32 or int64");
  if (!in_known(grad_dtype)) return api_fail(BS_ERR_DTYPE, "grad must be bf16 or f32");
  if (!out_known(d_dtype)) return api_fail(BS_ERR_DTYPE, "bs_embedding_grad writes bf16 or f32 only");
  if (V == 0 || D == 0) return BS_OK;
  bs_status st = check_rows_out(d, d_dtype, ldd, V, D);
  if (st != BS_OK) return st;
  if (T > 0) {
    const size_t need = lookup_grad_workspace(T, V, D);
    if (!tokens || !grad || (need > 0 && !workspace))
      return api_fail(BS_ERR_NULL, "tokens, grad and a workspace of that size must be non-NULL");
    if (!aligned(tokens, token_dtype == BS_INDEX_I64 ? 8 : 4))
      return api_fail(BS_ERR_ALIGNMENT, "tokens must be aligned to their size");
    if (ldg < D) return api_fail(BS_ERR_LAYOUT, "ldg=%lld < D=%lld", (long long)ldg, (long long)D);
    if (!extent_ok(T, ldg, 4)) return api_fail(BS_ERR_LAYOUT, "a stride times the number of rows is out of range");
    if (!aligned(grad, in_size(grad_dtype))) return api_fail(BS_ERR_ALIGNMENT, "grad must be aligned to its element size");
    if (!aligned(workspace, 256)) return api_fail(BS_ERR_ALIGNMENT, "the workspace must be 256-byte aligned");
    if (workspace_bytes < need)
      return api_fail(BS_ERR_WORKSPACE, "workspace of %zu bytes; this call needs %zu (bs_embedding_grad_workspace)",
                      workspace_bytes, need);
    // chunks of pairs times column slices, one CTA each
    if ((T + 31) / 32 * ((D + 1023) / 1024) >= kMaxDim / 2) return api_fail(BS_ERR_SHAPE, "T * D is out of range");
  }
  int sms = 0;
  uint32_t* err = nullptr;
  if ((st = api_device(&sms, &err)) != BS_OK) return st;
  LookupGradArgs a = {};
  a.tokens = tokens;
  a.tokens64 = token_dtype == BS_INDEX_I64;
  a.T = T;
  a.grad = grad;
  a.grad_bf16 = grad_dtype == BS_IN_BF16;
  a.ldg = ldg;
  a.V = V;
  a.D = D;
  a.alpha = alpha;
  a.padding_idx = padding_idx;
  a.out = d;
  a.out_bf16 = d_dtype == BS_OUT_BF16;
  a.ldo = ldd;
  a.accumulate = accumulate != 0;
  a.workspace = workspace;
  return api_launched(launch_lookup_grad(a, sms, static_cast<cudaStream_t>(stream)), "lookup gradient launch");
}

}  // extern "C"
