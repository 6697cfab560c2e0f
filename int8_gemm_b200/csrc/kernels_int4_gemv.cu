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
// A CTA owns 128 matrix rows and a run of 128-deep K blocks, which pass
// through a ring of stages in shared memory.  One thread fetches a block's
// codes (128 rows x 64 bytes) with a tensor copy; four staging warps write its
// activations in the order of the MMA's fragments (fp32 split on the way) and
// its scales and zero points as (scale, 128 + z) pairs; four warps multiply,
// 32 rows each, so that a fragment of activations serves two 16-row tiles.
// In a block a thread takes, for rows g and g + 8 of a tile (g = lane / 4), the
// word of 8 codes at k = 32 u + 8 (lane % 4) for u = 0 .. 3: all lanes' word u
// lies in the same 32 k, so every MMA sums inside one group whatever the group
// size, and under the copy's 64-byte swizzle (16-byte piece c of row r at
// c ^ (r / 2 % 4)) the lanes' words fall on different banks.  A word's nibbles
// j and j + 4 form the MMA's k pairs, and the activations are paired the same
// way.  With few row tiles K is split over the CTAs of a cluster, whose partial
// tiles meet in distributed shared memory and are added in rank order.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "lowbit.h"
#include "quantize.h"
#include "sm100.cuh"

namespace bsg {

namespace {

namespace cg = cooperative_groups;

constexpr int kMmaWarps = 4;    // 32 rows each
constexpr int kStageWarps = 4;  // one 32-k unit of activations and 32 rows of scales each
constexpr int kThreads = 32 * (kMmaWarps + kStageWarps);
constexpr int kTiles = 2;  // 16-row tiles per warp
constexpr int kUnits = 4;  // 32-k units per block
constexpr int kCodeBytes = kInt4TileRows * kInt4TileBytes;
constexpr int kPitch = kInt4TileRows + 4;  // floats between the rows of a partial tile
static_assert(kMmaWarps * kTiles * 16 == kInt4TileRows && kUnits * 16 == kInt4TileBytes, "tile and box agree");

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

// Eight activations of a row, k .. k+7 (zero at or past K), as read.
template <typename XT>
struct Eight {
  uint32_t r[2 * sizeof(XT)];

  __device__ __forceinline__ void load(const XT* row, long long k, long long K, bool vec) {
    if (vec && k + 8 <= K) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(XT)) / 2; ++i) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(row + k) + i);
        r[4 * i] = u.x, r[4 * i + 1] = u.y, r[4 * i + 2] = u.z, r[4 * i + 3] = u.w;
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < static_cast<int>(2 * sizeof(XT)); ++i) r[i] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (k + i >= K) continue;
      if constexpr (sizeof(XT) == 2) {
        r[i / 2] |= static_cast<uint32_t>(__bfloat16_as_ushort(row[k + i])) << (16 * (i % 2));
      } else {
        r[i] = __float_as_uint(row[k + i]);
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

// GPB: groups per 128-deep block (1, 2 or 4); NT: tiles of 8 activation rows.
template <typename XT, int GPB, int NT>
struct Config {
  static constexpr int kParts = sizeof(XT) == 2 ? 1 : 3;
  static constexpr int kXBytes = kUnits * NT * kParts * 512;  // fragments: 16 bytes per lane
  static constexpr int kScaleBytes = GPB * kInt4TileRows * 8;
  static constexpr int kStageBytes = kCodeBytes + kXBytes + kScaleBytes;
  static constexpr int kStages = 4;
  static constexpr int kSmem = kStages * kStageBytes + 1024;  // and the alignment of the first stage
  static_assert(kStages * kStageBytes >= 8 * NT * kPitch * 4, "the partial tile takes the ring's place");
};

// Grid: S consecutive CTAs (a cluster) per 128-row tile, splitting its K blocks.
template <typename XT, int GPB, int NT>
__global__ void __launch_bounds__(kThreads, NT <= 2 && sizeof(XT) == 2 ? 3 : 2)
    gemv_int4_kernel(const __grid_constant__ CUtensorMap tmq, const Int4Product p, int S, bool xvec, uint32_t* err) {
  using C = Config<XT, GPB, NT>;
  constexpr int PARTS = C::kParts;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[C::kStages], empty[C::kStages];
  __shared__ int abort_flag;
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x) % S;
  const long long n0 = static_cast<long long>(blockIdx.x / S) * kInt4TileRows;
  const int KB = static_cast<int>((p.K + 127) / 128);
  const int kb_lo = static_cast<int>(static_cast<long long>(KB) * rank / S);
  const int kb_hi = static_cast<int>(static_cast<long long>(KB) * (rank + 1) / S);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1 + kStageWarps);  // the tensor copy's arrival and each staging warp's
      mbar_init(&empty[s], kMmaWarps);
    }
    abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmq);
  }
  __syncthreads();
  grid_dependency_wait();  // every operand may come from the previous kernel in the stream
  grid_launch_dependents();

  float acc[kTiles][NT][4] = {};
  if (warp < kMmaWarps) {
    const int gr = lane >> 2, t = lane & 3;
    const uint32_t row_off = (32 * warp + gr) * kInt4TileBytes + 4 * t;
    const uint32_t swz = (gr >> 1) & 3;
    int it = 0;
    for (int kb = kb_lo; kb < kb_hi; ++kb, ++it) {
      const int st = it % C::kStages;
      if (!wait_bounded(&full[st], (it / C::kStages) & 1u, &abort_flag, err, kErrTimeout | kRoleConsumer | kWaitStageFull))
        break;
      const uint8_t* codes = ring + st * C::kStageBytes + row_off;
      const uint4* xs = reinterpret_cast<const uint4*>(ring + st * C::kStageBytes + kCodeBytes) + lane;
      const uint2* sc = reinterpret_cast<const uint2*>(ring + st * C::kStageBytes + kCodeBytes + C::kXBytes) + 32 * warp + gr;
      constexpr int kUnitsPerGroup = kUnits / GPB;
      uint2 so[kTiles][2];  // (scale, 128 + z) of rows gr and gr + 8 of each tile
      float part[kTiles][NT][4];
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        if (u % kUnitsPerGroup == 0) {
#pragma unroll
          for (int i = 0; i < kTiles; ++i) {
            so[i][0] = sc[(u / kUnitsPerGroup) * kInt4TileRows + 16 * i];
            so[i][1] = sc[(u / kUnitsPerGroup) * kInt4TileRows + 16 * i + 8];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) part[i][j][e] = 0.f;
          }
        }
        uint32_t a[kTiles][2][4];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          const uint8_t* c = codes + 16 * i * kInt4TileBytes + ((u ^ swz) << 4);
          const uint32_t w0 = *reinterpret_cast<const uint32_t*>(c);
          const uint32_t w1 = *reinterpret_cast<const uint32_t*>(c + 8 * kInt4TileBytes);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            a[i][h][0] = code_pair(w0, 2 * h, so[i][0].y);
            a[i][h][1] = code_pair(w1, 2 * h, so[i][1].y);
            a[i][h][2] = code_pair(w0, 2 * h + 1, so[i][0].y);
            a[i][h][3] = code_pair(w1, 2 * h + 1, so[i][1].y);
          }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
          for (int c = PARTS - 1; c >= 0; --c) {  // the smallest parts first
            const uint4 b = xs[((u * NT + j) * PARTS + c) * 32];
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
              mma_bf16_16x8x16(part[i][j], a[i][0], b.x, b.y);
              mma_bf16_16x8x16(part[i][j], a[i][1], b.z, b.w);
            }
          }
        }
        if (u % kUnitsPerGroup == kUnitsPerGroup - 1) {
#pragma unroll
          for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                acc[i][j][e] = fmaf(__uint_as_float(so[i][e / 2].x), part[i][j][e], acc[i][j][e]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
  } else {
    const int a = warp - kMmaWarps;  // unit of activations, and 32 rows of scales
    const XT* x = static_cast<const XT*>(p.x);
    const int gr = lane >> 2, t = lane & 3;
    const long long n = n0 + 32 * a + lane;
    const bool in_row = n < p.N;
    // a block's activations and scales are in registers one block ahead
    Eight<XT> v[NT];
    float s[GPB];
    uint32_t z[GPB];
    auto fetch = [&](int kb) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int m = 8 * j + gr;
        v[j].load(x + (m < p.M ? m : 0) * p.ldx, static_cast<long long>(kb) * 128 + 32 * a + 8 * t, m < p.M ? p.K : 0, xvec);
      }
#pragma unroll
      for (int g = 0; g < GPB; ++g) {
        const long long j = static_cast<long long>(kb) * GPB + g;
        s[g] = 0.f;
        z[g] = 8;
        if (in_row && j * p.w.group < p.K) {
          s[g] = p.w.scale_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.w.scale)[n * p.w.lds + j])
                                : static_cast<const float*>(p.w.scale)[n * p.w.lds + j];
          if (p.w.zero) z[g] = p.w.zero[n * p.w.ldz + j] & 15u;
        }
      }
    };
    if (kb_lo < kb_hi) fetch(kb_lo);
    int it = 0;
    for (int kb = kb_lo; kb < kb_hi; ++kb, ++it) {
      const int st = it % C::kStages;
      if (it >= C::kStages && !wait_bounded(&empty[st], (it / C::kStages - 1) & 1u, &abort_flag, err,
                                            kErrTimeout | kRoleProducer | kWaitStageEmpty))
        break;
      uint8_t* stage = ring + st * C::kStageBytes;
      if (a == 0 && lane == 0) {
        mbar_arrive_expect_tx(&full[st], kCodeBytes);
        tma_load_3d(stage, &tmq, &full[st], kb * kInt4TileBytes, static_cast<int>(n0), 0);
      }
      uint4* xs = reinterpret_cast<uint4*>(stage + kCodeBytes) + lane;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint4 b[PARTS];
        v[j].template pairs<PARTS>(b);
#pragma unroll
        for (int c = 0; c < PARTS; ++c) xs[((a * NT + j) * PARTS + c) * 32] = b[c];
      }
      uint2* sc = reinterpret_cast<uint2*>(stage + kCodeBytes + C::kXBytes) + 32 * a + lane;
#pragma unroll
      for (int g = 0; g < GPB; ++g)  // one unit of the last place of bf16's 128 is 1
        sc[g * kInt4TileRows] = make_uint2(__float_as_uint(s[g]), (0x4300u + z[g]) * 0x10001u);
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[st]);
      if (kb + 1 < kb_hi) fetch(kb + 1);
    }
    // a wait that gave up leaves copies in flight: let them land before the CTA retires
    if (a == 0 && lane == 0 && abort_flag) pause_ns(1000000);
  }

  // the warps' sums as a partial tile [activation row][matrix row], over the ring
  __syncthreads();
  float* tile = reinterpret_cast<float*>(ring);
  if (warp < kMmaWarps) {
    const int gr = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          tile[(8 * j + 2 * t + e % 2) * kPitch + 32 * warp + 16 * i + 8 * (e / 2) + gr] = acc[i][j][e];
  }
  cg::cluster_group cluster = cg::this_cluster();
  if (S > 1) cluster.sync();
  else __syncthreads();
  // CTA `rank` finishes its share of the activation rows
  for (int i = threadIdx.x; i < p.M * kInt4TileRows; i += kThreads) {
    const int m = i / kInt4TileRows, r = i % kInt4TileRows;
    if (m % S != rank || n0 + r >= p.N) continue;
    float y = 0.f;
    if (S > 1) {
      for (int c = 0; c < S; ++c) y += *cluster.map_shared_rank(tile + m * kPitch + r, c);
    } else {
      y = tile[m * kPitch + r];
    }
    if (p.bias) y += p.bias[n0 + r];
    const long long o = m * p.ldo + n0 + r;
    if (p.out_bf16) static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(y);
    else static_cast<float*>(p.out)[o] = y;
  }
  if (S > 1) cluster.sync();  // a CTA's tile stays until every rank has read it
}

// K splits of a row tile: enough CTAs for two per SM, at most eight to a
// cluster, each with two K blocks at least.
int splits_for(long long tiles, long long blocks, int sms) {
  int S = 1;
  while (S < 8 && 2 * S * tiles <= 2LL * sms && blocks >= 4 * S) S *= 2;
  return S;
}

template <typename XT, int GPB, int NT>
cudaError_t launch_one(const Int4Product& p, const CUtensorMap& q, int sms, uint32_t* err, cudaStream_t stream) {
  using C = Config<XT, GPB, NT>;
  int per_sm = 0;
  cudaError_t e = ctas_per_sm_once<gemv_int4_kernel<XT, GPB, NT>>(kThreads, C::kSmem, &per_sm);
  if (e != cudaSuccess) return e;
  const bool xvec = (reinterpret_cast<uintptr_t>(p.x) & 15u) == 0 && (p.ldx * sizeof(XT)) % 16 == 0;
  const long long tiles = (p.N + kInt4TileRows - 1) / kInt4TileRows;
  const int S = splits_for(tiles, (p.K + 127) / 128, sms);
  cudaLaunchAttribute attr[2];
  // programmatic dependent launch: the prologue may overlap the previous kernel
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(S);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * S), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gemv_int4_kernel<XT, GPB, NT>, q, p, S, xvec, err);
}

template <typename XT, int GPB>
cudaError_t launch_tiles(const Int4Product& p, const CUtensorMap& q, int sms, uint32_t* err, cudaStream_t stream) {
  if (p.M <= 8) return launch_one<XT, GPB, 1>(p, q, sms, err, stream);
  return p.M <= 16 ? launch_one<XT, GPB, 2>(p, q, sms, err, stream) : launch_one<XT, GPB, 4>(p, q, sms, err, stream);
}

template <typename XT>
cudaError_t launch_group(const Int4Product& p, const CUtensorMap& q, int sms, uint32_t* err, cudaStream_t stream) {
  if (p.w.group == 128) return launch_tiles<XT, 1>(p, q, sms, err, stream);
  return p.w.group == 64 ? launch_tiles<XT, 2>(p, q, sms, err, stream) : launch_tiles<XT, 4>(p, q, sms, err, stream);
}

}  // namespace

cudaError_t launch_gemv_int4(const Int4Product& p, const CUtensorMap& q, int sms, uint32_t* err, cudaStream_t stream) {
  return p.x_bf16 ? launch_group<__nv_bfloat16>(p, q, sms, err, stream) : launch_group<float>(p, q, sms, err, stream);
}

}  // namespace bsg
