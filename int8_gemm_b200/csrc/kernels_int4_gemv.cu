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
// Eight warps share a CTA's tile of matrix rows, KW of them splitting K; each
// works alone until its sums meet the others' in shared memory (added in warp
// order).  A warp keeps a ring of its own tensor copies in flight, 16 RT rows x
// 64 bytes (128 k) each, and runs ahead into the CTA's next tile; persistent
// CTAs take every gridDim.x-th tile.  For a 128-deep block it holds the
// activations of 128 k as MMA fragments and passes its RT 16-row tiles by them.
// In a block a thread takes, for rows g and g + 8 of a tile (g = lane / 4), the
// word of 8 codes at k = 32 u + 8 (lane % 4) for u = 0 .. 3: all lanes' word u
// lies in the same 32 k, so every MMA sums inside one group whatever the group
// size, and under the copy's 64-byte swizzle (16-byte piece c of row r at
// c ^ (r / 2 % 4)) the lanes' words fall on different banks.  A word's nibbles
// j and j + 4 form the MMA's k pairs, and the activations are paired the same
// way.  The four lanes of a row load four consecutive groups' scales and zero
// points at once, one span of blocks ahead, and pass them round by shuffles.
//
// What bounds it: latency, with few warps to cover it.  A word of 8 codes costs 26
// warp instructions at 16 rows (11 unpack it: 3 shifts, 4 three-input logical, 4
// bf16 subtractions; the others are MMAs, activations, scales, sums and the ring),
// which 131072 x 5120 in groups of 128 could issue in 66 us; but fragments, sums and
// scales take 128 registers, so an SM holds 16 warps, and they issue in 54 % of the
// cycles, no pipe above 50 %.  One row takes 85 us, 16 rows 125, 32 rows (8 warps on
// an SM) 266, where the copies alone take 52.
#include <cuda_bf16.h>

#include "lowbit.h"
#include "quantize.h"
#include "sm100.cuh"

namespace bsg {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnits = 4;  // 32-k units per block
static_assert(kUnits * 16 == kInt4BoxBytes, "block and box agree");

// d = a b + (first ? 0 : d)
__device__ __forceinline__ void mma_bf16_16x8x16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                                 bool first) {
  if (first) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

// Codes j and j + 4 of a word less `off` = (128 + z, 128 + z), as a bf16 pair.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int j, uint32_t off) {
  uint32_t m;  // (w >> 4 j) & 0x000F000F | 0x43004300 in one three-input operation after the shift
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(m) : "r"(w >> (4 * j)), "r"(0x000F000Fu), "r"(0x43004300u));
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&m), *reinterpret_cast<const __nv_bfloat162*>(&off));
  return *reinterpret_cast<const uint32_t*>(&d);
}

template <int W>
struct Width {
  static constexpr int value = W;
};

// Eight consecutive activations of a row, as read.
template <typename XT>
struct Eight {
  uint32_t r[2 * sizeof(XT)];

  // All of them from a boundary of W bytes, or zeros.  W = 2 (bf16): whole words
  // and, where the row starts between two, an element at either end.
  template <int W>
  __device__ __forceinline__ void load_whole(const XT* p, bool in) {
    constexpr int kWords = static_cast<int>(2 * sizeof(XT));
    if constexpr (W == 16) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 u = in ? __ldg(reinterpret_cast<const uint4*>(p) + i / 4) : make_uint4(0, 0, 0, 0);
        r[i] = u.x, r[i + 1] = u.y, r[i + 2] = u.z, r[i + 3] = u.w;
      }
    } else if constexpr (W == 4) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) r[i] = in ? __ldg(reinterpret_cast<const uint32_t*>(p) + i) : 0u;
    } else {
      static_assert(W == 2 && sizeof(XT) == 2, "fp32 rows start on 4-byte boundaries");
      const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
      const bool odd = (reinterpret_cast<uintptr_t>(p) & 2u) != 0;
      const uint32_t* w = reinterpret_cast<const uint32_t*>(h + (odd ? 1 : 0));
      const uint32_t head = in && odd ? static_cast<uint32_t>(__ldg(h)) << 16 : 0u;
      const uint32_t w0 = in ? __ldg(w) : 0u, w1 = in ? __ldg(w + 1) : 0u, w2 = in ? __ldg(w + 2) : 0u;
      uint32_t tail = in && odd ? __ldg(h + 7) : 0u;
      if (in && !odd) tail = __ldg(w + 3);
      const uint32_t shift = odd ? 16 : 0;
      r[0] = __funnelshift_l(head, w0, shift);
      r[1] = __funnelshift_l(w0, w1, shift);
      r[2] = __funnelshift_l(w1, w2, shift);
      r[3] = __funnelshift_l(w2, tail, shift);
    }
  }

  // The first `left` of them; the others are zero.
  __device__ __forceinline__ void load(const XT* p, int left) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(2 * sizeof(XT)); ++i) r[i] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= left) continue;
      if constexpr (sizeof(XT) == 2) {
        r[i / 2] |= static_cast<uint32_t>(__bfloat16_as_ushort(p[i])) << (16 * (i % 2));
      } else {
        r[i] = __float_as_uint(p[i]);
      }
    }
  }

  // The k pairs (j, j + 4) of the bf16 parts that add up to the values, one
  // uint4 per part.  A truncated value leaves an exact remainder, so three
  // parts of 8 bits hold an fp32 value whole; a value that is not finite is its
  // own first part (a NaN kept one) and leaves no remainder.
  template <int PARTS>
  __device__ __forceinline__ void pairs(uint4 (&b)[PARTS]) const {
    if constexpr (PARTS == 1) {
      b[0] = make_uint4(__byte_perm(r[0], r[2], 0x5410), __byte_perm(r[0], r[2], 0x7632),
                        __byte_perm(r[1], r[3], 0x5410), __byte_perm(r[1], r[3], 0x7632));
    } else {
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (r[i] & 0x7FFFFFFFu) > 0x7F800000u ? 0x7FC00000u : r[i];
#pragma unroll
      for (int p = 0; p < PARTS; ++p) {
        b[p] = make_uint4(__byte_perm(v[0], v[4], 0x7632), __byte_perm(v[1], v[5], 0x7632),
                          __byte_perm(v[2], v[6], 0x7632), __byte_perm(v[3], v[7], 0x7632));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float f = __uint_as_float(v[i]), h = __uint_as_float(v[i] & 0xFFFF0000u);
          v[i] = (v[i] & 0x7F800000u) == 0x7F800000u ? 0u : __float_as_uint(__fsub_rn(f, h));
        }
      }
    }
  }
};

// GPB: groups per 128-deep block (1, 2 or 4); NT: tiles of 8 activation rows;
// RT: 16-row tiles of the matrix per warp; ZERO: the matrix has zero points.
// The ring is as deep as leaves room for kCtas CTAs on an SM (a third stage of 64
// rows, which cost the second CTA: 131072 x 5120, one row 101 us in place of 85, 16
// rows 157 in place of 125).
template <typename XT, int NT, int RT>
struct Config {
  static constexpr int kParts = sizeof(XT) == 2 ? 1 : 3;
  static constexpr int kCtas = NT * kParts == 1 && RT == 1 ? 3 : (NT * kParts <= 2 ? 2 : 1);  // per SM
  static constexpr int kBoxBytes = 16 * RT * kInt4BoxBytes;
  static constexpr int kStages = RT == 4 ? 2 : (RT == 2 ? 3 : 4);
  static constexpr int kPitch = 16 * RT + 4;  // floats between the activation rows of a warp's sums
  static constexpr int kRingBytes = kWarps * kStages * kBoxBytes;
  static constexpr int kSmem = kRingBytes + kWarps * 8 * NT * kPitch * 4 + 1024;  // 1024: the first box's alignment
};

// Scales (raw bits) or zero points of a lane's 2 RT rows for one of four
// consecutive groups.
template <int RT>
struct Side {
  uint32_t s[2 * RT], z[2 * RT];
};

template <typename XT, int GPB, int NT, int RT, bool ZERO>
__global__ void __launch_bounds__(kThreads, Config<XT, NT, RT>::kCtas)
    gemv_int4_kernel(const __grid_constant__ CUtensorMap tmq, const Int4Product p, int kw, uint32_t tiles, int xwidth,
                     uint32_t* err) {
  using C = Config<XT, NT, RT>;
  constexpr int PARTS = C::kParts;
  constexpr int kSpan = 4 / GPB;  // blocks that a load of scales serves
  constexpr int kUnitsPerGroup = kUnits / GPB;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kWarps][C::kStages];
  __shared__ int abort_flag;
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  if (pad + C::kSmem - 1024 > dynamic_smem_bytes()) {  // never touch memory the launch did not provide
    if (threadIdx.x == 0) record_error(err, kErrSmemTooSmall);
    return;
  }
  uint8_t* base = smem_raw + pad;
  float* sums = reinterpret_cast<float*>(base + C::kRingBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t = lane & 3;
  uint8_t* ring = base + warp * C::kStages * C::kBoxBytes;
  // this warp's K blocks [kb_lo, kb_lo + nb) and its rows within a tile
  const int KB = static_cast<int>((p.K + 127) / 128);
  const int part_k = warp & (kw - 1), row0 = 16 * RT * (warp / kw);
  const int kb_lo = static_cast<int>(static_cast<long long>(KB) * part_k / kw);
  const int nb = static_cast<int>(static_cast<long long>(KB) * (part_k + 1) / kw) - kb_lo;
  const int tile_rows = 16 * RT * (kWarps / kw);

  if (lane == 0) {
    for (int s = 0; s < C::kStages; ++s) mbar_init(&full[warp][s], 1);
    if (warp == 0) {
      abort_flag = 0;
      tma_prefetch_desc(&tmq);
    }
    fence_mbar_init();
  }
  __syncthreads();
  grid_dependency_wait();  // every operand may come from the previous kernel in the stream
  grid_launch_dependents();

  // the next box to copy, and the stage it goes to
  uint32_t copy_tile = blockIdx.x;
  int copy_b = 0, copy_st = 0;
  auto copy = [&]() {
    if (copy_tile < tiles && nb > 0) {
      if (lane == 0) {
        mbar_arrive_expect_tx(&full[warp][copy_st], C::kBoxBytes);
        tma_load_3d(ring + copy_st * C::kBoxBytes, &tmq, &full[warp][copy_st], (kb_lo + copy_b) * kInt4BoxBytes,
                    static_cast<int>(copy_tile) * tile_rows + row0, 0);
      }
      if (++copy_st == C::kStages) copy_st = 0;
      if (++copy_b == nb) copy_b = 0, copy_tile += gridDim.x;
    }
  };
  for (int s = 0; s < C::kStages; ++s) copy();

  const int K = static_cast<int>(p.K), G = static_cast<int>((p.K + p.w.group - 1) / p.w.group);
  const XT* xrow[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) xrow[j] = static_cast<const XT*>(p.x) + (8 * j + gr < p.M ? 8 * j + gr : 0) * p.ldx + 8 * t;
  // scales and zero points of the span that begins with block kb of `tile`
  const int scale_bytes = p.w.scale_bf16 ? 2 : 4;
  const long long step_s = 8 * p.w.lds * scale_bytes, step_z = 8 * p.w.ldz;
  const char* scale_g = static_cast<const char*>(p.w.scale) + t * scale_bytes;
  auto load_side = [&](Side<RT>& f, uint32_t tile, int kb) {
    const int n = static_cast<int>(tile) * tile_rows + row0 + gr;
    // rows left from n, none where the group or the tile does not exist
    const int left = tile < tiles && kb * GPB + t < G ? static_cast<int>(p.N) - n : 0;
    const char* sp = scale_g + (n * p.w.lds + kb * GPB) * scale_bytes;
    if (p.w.scale_bf16) {
#pragma unroll
      for (int i = 0; i < 2 * RT; ++i, sp += step_s) f.s[i] = left > 8 * i ? __ldg(reinterpret_cast<const uint16_t*>(sp)) : 0u;
    } else {
#pragma unroll
      for (int i = 0; i < 2 * RT; ++i, sp += step_s) f.s[i] = left > 8 * i ? __ldg(reinterpret_cast<const uint32_t*>(sp)) : 0u;
    }
    if constexpr (ZERO) {
      const uint8_t* zp = p.w.zero + n * p.w.ldz + kb * GPB + t;
#pragma unroll
      for (int i = 0; i < 2 * RT; ++i, zp += step_z) f.z[i] = left > 8 * i ? __ldg(zp) : 8u;
    }
  };
  uint32_t word_off[kUnits];  // word u of row gr of a 16-row tile
#pragma unroll
  for (int u = 0; u < kUnits; ++u) word_off[u] = gr * kInt4BoxBytes + 4 * t + ((u ^ ((gr >> 1) & 3)) << 4);

  Side<RT> now, next;
  if (nb > 0) load_side(next, blockIdx.x, kb_lo);
  const uint32_t scale_shift = p.w.scale_bf16 ? 16 : 0;
  int st = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    float acc[RT][NT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
#pragma unroll 1
    for (int b = 0; b < nb; ++b) {
      const int slot = (b % kSpan) * GPB;  // of this block's first group among the four loaded
      if (slot == 0) {
        now = next;
        if (b + kSpan < nb) load_side(next, tile, kb_lo + b + kSpan);
        else load_side(next, tile + gridDim.x, kb_lo);
      }
      // the block's activations
      uint4 x[kUnits][NT][PARTS];
      {
        const int k0 = (kb_lo + b) * 128;
        auto whole = [&](auto width) {
          Eight<XT> v[kUnits][NT];
#pragma unroll
          for (int u = 0; u < kUnits; ++u)
#pragma unroll
            for (int j = 0; j < NT; ++j)
              v[u][j].template load_whole<decltype(width)::value>(xrow[j] + k0 + 32 * u, 8 * j + gr < p.M);
#pragma unroll
          for (int u = 0; u < kUnits; ++u)
#pragma unroll
            for (int j = 0; j < NT; ++j) v[u][j].template pairs<PARTS>(x[u][j]);
        };
        if (k0 + 128 <= K && xwidth == 16) {
          whole(Width<16>());
        } else if (k0 + 128 <= K && (sizeof(XT) == 4 ? RT > 1 : xwidth == 4)) {
          whole(Width<4>());
        } else if (sizeof(XT) == 2 && k0 + 128 <= K) {
          if constexpr (sizeof(XT) == 2) whole(Width<2>());
        } else {
#pragma unroll
          for (int u = 0; u < kUnits; ++u)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              Eight<XT> v;
              v.load(xrow[j] + k0 + 32 * u, 8 * j + gr < p.M ? K - k0 - 32 * u - 8 * t : 0);
              v.template pairs<PARTS>(x[u][j]);
            }
        }
      }
      if (ok) ok = wait_bounded(&full[warp][st], phase, &abort_flag, err, kErrTimeout | kRoleConsumer | kWaitStageFull);
      ok = __all_sync(0xffffffffu, ok);  // the lanes of a warp go on, or give up, together
      if (!ok) break;
      const uint8_t* box = ring + st * C::kBoxBytes;
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        float part[NT][4];
        uint32_t off0 = 0x43084308u, off1 = 0x43084308u;  // 128 + z, twice: one unit of the last place of bf16's 128 is 1
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
          const bool first = u % kUnitsPerGroup == 0, last = u % kUnitsPerGroup == kUnitsPerGroup - 1;
          if (first) {
            const int src = (lane & ~3) | (slot + u / kUnitsPerGroup);
            s0 = __uint_as_float(__shfl_sync(0xffffffffu, now.s[2 * i], src) << scale_shift);
            s1 = __uint_as_float(__shfl_sync(0xffffffffu, now.s[2 * i + 1], src) << scale_shift);
            if constexpr (ZERO) {
              off0 = ((__shfl_sync(0xffffffffu, now.z[2 * i], src) & 15u) | 0x4300u) * 0x10001u;
              off1 = ((__shfl_sync(0xffffffffu, now.z[2 * i + 1], src) & 15u) | 0x4300u) * 0x10001u;
            }
          }
          const uint32_t w0 = *reinterpret_cast<const uint32_t*>(box + word_off[u] + 16 * i * kInt4BoxBytes);
          const uint32_t w1 = *reinterpret_cast<const uint32_t*>(box + word_off[u] + (16 * i + 8) * kInt4BoxBytes);
          uint32_t a[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            a[h][0] = code_pair(w0, 2 * h, off0);
            a[h][1] = code_pair(w1, 2 * h, off1);
            a[h][2] = code_pair(w0, 2 * h + 1, off0);
            a[h][3] = code_pair(w1, 2 * h + 1, off1);
          }
#pragma unroll
          for (int c = PARTS - 1; c >= 0; --c) {  // the smallest parts first
#pragma unroll
            for (int j = 0; j < NT; ++j) mma_bf16_16x8x16(part[j], a[0], x[u][j][c].x, x[u][j][c].y, first && c == PARTS - 1);
#pragma unroll
            for (int j = 0; j < NT; ++j) mma_bf16_16x8x16(part[j], a[1], x[u][j][c].z, x[u][j][c].w, false);
          }
          if (last) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(e < 2 ? s0 : s1, part[j][e], acc[i][j][e]);
          }
        }
      }
      if (++st == C::kStages) st = 0, phase ^= 1;
      __syncwarp();  // every lane has read the box
      copy();
    }
    // the warps' sums [activation row][matrix row], added in order of K
    float* mine = sums + warp * 8 * NT * C::kPitch;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mine[(8 * j + 2 * t + e % 2) * C::kPitch + 16 * i + 8 * (e / 2) + gr] = acc[i][j][e];
    __syncthreads();
    const int rows_log2 = __ffs(tile_rows) - 1;  // a power of two
    for (int i = threadIdx.x; i < p.M << rows_log2; i += kThreads) {
      const int m = i >> rows_log2, r = i & (tile_rows - 1);
      const long long n = static_cast<long long>(tile) * tile_rows + r;
      if (n >= p.N) continue;
      const float* from = sums + ((r / (16 * RT)) * kw * 8 * NT + m) * C::kPitch + (r & (16 * RT - 1));
      float y = from[0];
      for (int w = 1; w < kw; ++w) y += from[w * 8 * NT * C::kPitch];
      if (p.bias) y += p.bias[n];
      const long long o = m * p.ldo + n;
      if (p.out_bf16) static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(y);
      else static_cast<float*>(p.out)[o] = y;
    }
    __syncthreads();
  }
  // a wait that gave up leaves copies in flight: let them land before the CTA retires
  if (!ok) pause_ns(1000000);
}

template <typename XT, int GPB, int NT, int RT, bool ZERO>
cudaError_t launch_zero(const Int4Product& p, int sms, uint32_t* err, cudaStream_t stream) {
  using C = Config<XT, NT, RT>;
  int per_sm = 0;
  cudaError_t e = ctas_per_sm_once<gemv_int4_kernel<XT, GPB, NT, RT, ZERO>>(kThreads, C::kSmem, &per_sm);
  if (e != cudaSuccess) return e;
  CUtensorMap map;
  if (api_map_codes(&map, p.w.q, (p.K + 1) / 2, p.N, p.w.ldq, kInt4BoxBytes, 16 * RT, CU_TENSOR_MAP_SWIZZLE_64B) != BS_OK)
    return cudaErrorInvalidValue;
  // Bytes of a load of activations: 16 where every row starts on such a boundary
  // (the distance of rows says nothing about a single one), else 4, and 2 for bf16
  // rows that start between words.  32768 x 8198, contiguous rows, 1 / 16 / 32 rows:
  // 43 / 66 / 147 us in words, 44 / 77 / 189 as rows that may start between them, 48
  // / 100 / 569 element by element; rows padded to 16 bytes 43 / 62 / 121.  8197: 43 /
  // 82 / 217 against 48 / 100 / 534.  (Loads of 8 bytes as well: 129 against 150 for
  // 32 rows of 8196, but 87 against 78 for 17 fp32 rows of 8208.)  fp32, whose split
  // needs the registers, goes by words where a warp has 64 matrix rows (8192 x 4098, 9
  // rows 27.9 against 29.0) and word by word, each eight split before the next are
  // read, where it has 16 (179 x 8982, 9 rows 28.2 against 32.5).
  const uintptr_t starts = reinterpret_cast<uintptr_t>(p.x) | (p.M > 1 ? static_cast<uintptr_t>(p.ldx) * sizeof(XT) : 0);
  const int xwidth = starts % 16 == 0 ? 16 : (starts % 4 == 0 ? 4 : 2);
  const long long blocks = (p.K + 127) / 128;
  int kw = 1;  // warps that split K: all eight where there are as many blocks
  while (kw < kWarps && 2 * kw <= blocks) kw *= 2;
  const long long rows = 16 * RT * (kWarps / kw), tiles = (p.N + rows - 1) / rows;
  const long long slots = static_cast<long long>(per_sm) * sms;
  cudaLaunchAttribute attr[1];
  // programmatic dependent launch: the prologue may overlap the previous kernel
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles < slots ? tiles : slots), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gemv_int4_kernel<XT, GPB, NT, RT, ZERO>, map, p, kw, static_cast<uint32_t>(tiles), xwidth, err);
}

template <typename XT, int GPB, int NT, int RT>
cudaError_t launch_one(const Int4Product& p, int sms, uint32_t* err, cudaStream_t stream) {
  return p.w.zero ? launch_zero<XT, GPB, NT, RT, true>(p, sms, err, stream) : launch_zero<XT, GPB, NT, RT, false>(p, sms, err, stream);
}

// Rows per warp: 64 (32 with four tiles of activation rows, whose fragments take
// the registers) share a block's activations, 16 give more CTAs; fp32 activations,
// split in registers, pay for 64 earlier.  Many rows / 16, us, groups of 128:
//   bf16, K = 4096   1 row       8 rows      16 rows     32 rows
//     N = 2048       7.9 / 5.5   8.8 / 6.4   11.1 / 6.8  10.4 / 8.7
//     N = 4736       8.5 / 9.7   9.5 / 9.9   11.9 / 8.8  11.2 / 15.5
//     N = 8192       9.5 / 13.2  10.7 / 13.7 12.9 / 14.1 19.3 / 27.9
//     131072 x 5120  85 / 133                125 / 192   267 / 423
//   fp32, K = 4096
//     N = 2048       12.5 / 9.1  14.0 / 10.5 21.0 / 14.6
//     N = 2368       12.6 / 9.3  14.0 / 10.7 21.1 / 14.7
//     N = 4096       13.0 / 15.4 14.5 / 16.8 21.6 / 25.5
//     N = 8192       14.1 / 28.1 15.8 / 29.7 22.8 / 48.4
// The rule looks at N alone.  Where K is short, so that fewer warps share it and a
// CTA takes up to 512 rows, 16 stay ahead for longer: 5000 x 128 3.0 / 2.4, 3.9 /
// 2.7, 5.3 / 3.3, 5.6 / 4.2; 8192 x 256 3.0 / 2.6, 4.4 / 3.0, 6.7 / 3.5, 6.3 / 4.7;
// 16384 x 512 3.8 / 5.0, 4.5 / 5.5, 6.0 / 6.4, 9.3 / 11.8.
template <typename XT, int GPB, int NT>
cudaError_t launch_rows(const Int4Product& p, int sms, uint32_t* err, cudaStream_t stream) {
  constexpr int RT = NT == 4 ? 2 : 4;
  const long long enough = (sizeof(XT) == 2 ? 32LL : 16LL) * sms;
  return p.N >= enough ? launch_one<XT, GPB, NT, RT>(p, sms, err, stream) : launch_one<XT, GPB, NT, 1>(p, sms, err, stream);
}

template <typename XT, int GPB>
cudaError_t launch_tiles(const Int4Product& p, int sms, uint32_t* err, cudaStream_t stream) {
  if (p.M <= 8) return launch_rows<XT, GPB, 1>(p, sms, err, stream);
  if constexpr (sizeof(XT) == 2) {
    if (p.M > 16) return launch_rows<XT, GPB, 4>(p, sms, err, stream);
  }
  return launch_rows<XT, GPB, 2>(p, sms, err, stream);
}

template <typename XT>
cudaError_t launch_group(const Int4Product& p, int sms, uint32_t* err, cudaStream_t stream) {
  if (p.w.group == 128) return launch_tiles<XT, 1>(p, sms, err, stream);
  return p.w.group == 64 ? launch_tiles<XT, 2>(p, sms, err, stream) : launch_tiles<XT, 4>(p, sms, err, stream);
}

}  // namespace

cudaError_t launch_gemv_int4(const Int4Product& p, int sms, uint32_t* err, cudaStream_t stream) {
  if (p.x_bf16) return launch_group<__nv_bfloat16>(p, sms, err, stream);
  // fp32: 16 activation rows per launch (three parts of more would not fit the registers)
  for (int m = 0; m < p.M; m += 16) {
    Int4Product h = p;
    h.x = static_cast<const float*>(p.x) + m * p.ldx;
    h.out = static_cast<char*>(p.out) + m * p.ldo * (p.out_bf16 ? 2 : 4);
    h.M = p.M - m < 16 ? p.M - m : 16;
    const cudaError_t e = launch_group<float>(h, sms, err, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace bsg
