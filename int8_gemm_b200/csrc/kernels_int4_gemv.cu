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
// A CTA owns 256 matrix rows and a run of 128-deep K blocks, which pass
// through a ring of stages in shared memory.  One thread fetches a block's
// codes (256 rows x 64 bytes) with a tensor copy; four staging warps write its
// activations in the order of the MMA's fragments (fp32 split on the way) and
// its scales and zero points as (scale, 128 + z) pairs; eight warps multiply,
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

constexpr int kMmaWarps = 8;    // 32 rows each
constexpr int kFillWarps = 3;   // staging activations and scales; one warp more issues the tensor copies
constexpr int kThreads = 32 * (kMmaWarps + 1 + kFillWarps);
constexpr int kTiles = 2;  // 16-row tiles per warp
constexpr int kUnits = 4;  // 32-k units per block
constexpr int kCodeBytes = kInt4TileRows * kInt4TileBytes;
constexpr int kScaleGroups = 4;  // groups of a slot of scales: 4, 2 or 1 blocks
constexpr int kScalePitch = kInt4TileRows * 8 + 64;  // bytes between a slot's groups (64: a load's groups store to different banks)
constexpr int kScaleBytes = kScaleGroups * kScalePitch;
constexpr int kScaleStages = 3;
constexpr int kPitch = kInt4TileRows + 4;  // floats between the rows of a partial tile
static_assert(kMmaWarps * kTiles * 16 == kInt4TileRows && kUnits * 16 == kInt4TileBytes, "tile and box agree");

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

// Eight consecutive activations of a row, as read.
template <typename XT>
struct Eight {
  uint32_t r[2 * sizeof(XT)];

  // From a 16-byte boundary, or zeros.
  __device__ __forceinline__ void load16(const XT* p, bool in) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(XT)) / 2; ++i) {
      const uint4 u = in ? __ldg(reinterpret_cast<const uint4*>(p) + i) : make_uint4(0, 0, 0, 0);
      r[4 * i] = u.x, r[4 * i + 1] = u.y, r[4 * i + 2] = u.z, r[4 * i + 3] = u.w;
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

// GPB: groups per 128-deep block (1, 2 or 4); NT: tiles of 8 activation rows.
template <typename XT, int GPB, int NT>
struct Config {
  static constexpr int kParts = sizeof(XT) == 2 ? 1 : 3;
  static constexpr int kXBytes = kUnits * NT * kParts * 512;  // fragments: 16 bytes per lane
  static constexpr int kStageBytes = kCodeBytes + kXBytes;
  static constexpr int kCtas = NT <= 2 && sizeof(XT) == 2 ? 2 : 1;  // per SM
  static constexpr int kRoom = 225 * 1024 / kCtas - kScaleStages * kScaleBytes - 2048;
  static constexpr int kStages = kRoom / kStageBytes < 8 ? kRoom / kStageBytes : 8;
  static constexpr int kSmem = kStages * kStageBytes + kScaleStages * kScaleBytes + 1024;  // 1024: the first stage's alignment
  static_assert(kStages >= 3, "a ring");
  static_assert(kStages * kStageBytes >= 8 * NT * kPitch * 4, "the partial tile takes the ring's place");
};

// Grid: S consecutive CTAs (a cluster) per row tile, splitting its K blocks.
template <typename XT, int GPB, int NT>
__global__ void __launch_bounds__(kThreads, Config<XT, GPB, NT>::kCtas)
    gemv_int4_kernel(const __grid_constant__ CUtensorMap tmq, const Int4Product p, int S, bool xvec, uint32_t* err) {
  using C = Config<XT, GPB, NT>;
  constexpr int PARTS = C::kParts;
  constexpr int kSpan = kScaleGroups / GPB;  // blocks per scale slot
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[C::kStages], empty[C::kStages], sfull[kScaleStages], sempty[kScaleStages];
  __shared__ int abort_flag;
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* scales = ring + C::kStages * C::kStageBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(blockIdx.x) % S;
  const long long n0 = static_cast<long long>(blockIdx.x / S) * kInt4TileRows;
  const int KB = static_cast<int>((p.K + 127) / 128);
  const int kb_lo = static_cast<int>(static_cast<long long>(KB) * rank / S);
  const int blocks = static_cast<int>(static_cast<long long>(KB) * (rank + 1) / S) - kb_lo;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 2);  // the tensor copy's arrival and the activations'
      mbar_init(&empty[s], kMmaWarps);
    }
    for (int s = 0; s < kScaleStages; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&sempty[s], kMmaWarps);
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
    constexpr int kUnitsPerGroup = kUnits / GPB;
    uint32_t word_off[kUnits];  // word u of row gr of the warp's first tile
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
      word_off[u] = (32 * warp + gr) * kInt4TileBytes + 4 * t + ((u ^ ((gr >> 1) & 3)) << 4);
    int st = 0, sst = 0, in_slot = 0;
    uint32_t phase = 0, sphase = 0;
    for (int b = 0; b < blocks; ++b) {
      if (in_slot == 0 &&
          !wait_bounded(&sfull[sst], sphase, &abort_flag, err, kErrTimeout | kRoleConsumer | kWaitScaleFull))
        break;
      if (!wait_bounded(&full[st], phase, &abort_flag, err, kErrTimeout | kRoleConsumer | kWaitStageFull)) break;
      const uint8_t* stage = ring + st * C::kStageBytes;
      const uint4* xs = reinterpret_cast<const uint4*>(stage + kCodeBytes) + lane;
      const uint2* sc = reinterpret_cast<const uint2*>(scales + sst * kScaleBytes + in_slot * GPB * kScalePitch) + 32 * warp + gr;
      uint2 so[kTiles][2];  // (scale, 128 + z) of rows gr and gr + 8 of each tile
      float part[kTiles][NT][4];
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const bool first = u % kUnitsPerGroup == 0, last = u % kUnitsPerGroup == kUnitsPerGroup - 1;
        uint32_t a[kTiles][2][4];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          if (first) {
            so[i][0] = sc[(u / kUnitsPerGroup) * (kScalePitch / 8) + 16 * i];
            so[i][1] = sc[(u / kUnitsPerGroup) * (kScalePitch / 8) + 16 * i + 8];
          }
          const uint8_t* c = stage + word_off[u] + 16 * i * kInt4TileBytes;
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
            const uint4 x = xs[((u * NT + j) * PARTS + c) * 32];
#pragma unroll
            for (int i = 0; i < kTiles; ++i) mma_bf16_16x8x16(part[i][j], a[i][0], x.x, x.y, first && c == PARTS - 1);
#pragma unroll
            for (int i = 0; i < kTiles; ++i) mma_bf16_16x8x16(part[i][j], a[i][1], x.z, x.w, false);
          }
        }
        if (last) {
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
      if (++st == C::kStages) st = 0, phase ^= 1;
      if (++in_slot == kSpan) {
        if (lane == 0) mbar_arrive(&sempty[sst]);
        in_slot = 0;
        if (++sst == kScaleStages) sst = 0, sphase ^= 1;
      }
    }
  } else if (warp == kMmaWarps) {
    if (lane == 0) {
      int st = 0;
      uint32_t phase = 1;  // of the stage's previous use
      for (int b = 0; b < blocks; ++b) {
        if (b >= C::kStages &&
            !wait_bounded(&empty[st], phase, &abort_flag, err, kErrTimeout | kRoleProducer | kWaitStageEmpty))
          break;
        mbar_arrive_expect_tx(&full[st], kCodeBytes);
        tma_load_3d(ring + st * C::kStageBytes, &tmq, &full[st], (kb_lo + b) * kInt4TileBytes, static_cast<int>(n0), 0);
        if (++st == C::kStages) st = 0, phase ^= 1;
      }
      // a wait that gave up leaves copies in flight: let them land before the CTA retires
      if (abort_flag) pause_ns(1000000);
    }
  } else {
    // block b's activations are warp b % 3's, and so are the scales of slot s;
    // each warp takes its tasks in the order of the blocks they belong to
    const int a = warp - kMmaWarps - 1;
    const int K = static_cast<int>(p.K), G = static_cast<int>((p.K + p.w.group - 1) / p.w.group);
    const XT* xrow[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) xrow[j] = static_cast<const XT*>(p.x) + (8 * j + gr < p.M ? 8 * j + gr : 0) * p.ldx;
    const int col = lane % kScaleGroups, row = lane / kScaleGroups;  // 4 groups of 8 rows per load
    for (int b = 0; b < blocks; ++b) {
      if (b % kSpan == 0 && (b / kSpan) % kFillWarps == a) {
        const int slot = b / kSpan, sst = slot % kScaleStages;
        const int g = (kb_lo + b) * GPB + col;
        uint8_t* dst = scales + sst * kScaleBytes + col * kScalePitch + row * 8;
        bool waited = slot < kScaleStages;
#pragma unroll 1
        for (int r0 = 0; r0 < kInt4TileRows; r0 += 128) {
          // all loads first (a conversion beside its load would wait for it)
          uint32_t sv[16], zv[16];
          const long long n = n0 + r0 + row;
          const bool g_in = g < G;
          if (p.w.scale_bf16) {
            const uint16_t* sp = static_cast<const uint16_t*>(p.w.scale) + n * p.w.lds + g;
#pragma unroll
            for (int i = 0; i < 16; ++i) sv[i] = g_in && n + 8 * i < p.N ? __ldg(sp + 8 * i * p.w.lds) : 0u;
          } else {
            const uint32_t* sp = static_cast<const uint32_t*>(p.w.scale) + n * p.w.lds + g;
#pragma unroll
            for (int i = 0; i < 16; ++i) sv[i] = g_in && n + 8 * i < p.N ? __ldg(sp + 8 * i * p.w.lds) : 0u;
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) zv[i] = 8;
          if (p.w.zero) {
            const uint8_t* zp = p.w.zero + n * p.w.ldz + g;
#pragma unroll
            for (int i = 0; i < 16; ++i) zv[i] = g_in && n + 8 * i < p.N ? __ldg(zp + 8 * i * p.w.ldz) : 8u;
          }
          if (!waited) {
            waited = wait_bounded(&sempty[sst], (slot / kScaleStages - 1) & 1u, &abort_flag, err,
                                  kErrTimeout | kRoleScale | kWaitScaleEmpty);
            if (!waited) break;
          }
#pragma unroll
          for (int i = 0; i < 16; ++i)  // one unit of the last place of bf16's 128 is 1
            *reinterpret_cast<uint2*>(dst + (r0 + 8 * i) * 8) = make_uint2(p.w.scale_bf16 ? sv[i] << 16 : sv[i], (0x4300u + (zv[i] & 15u)) * 0x10001u);
        }
        if (!waited) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfull[sst]);
      }
      if (b % kFillWarps != a) continue;
      const int st = b % C::kStages;
      const int k0 = (kb_lo + b) * 128 + 8 * t;
      uint4* xs = reinterpret_cast<uint4*>(ring + st * C::kStageBytes + kCodeBytes) + lane;
      const bool whole = xvec && (kb_lo + b) * 128 + 128 <= K;
      bool waited = b < C::kStages;
      constexpr int kAhead = NT * sizeof(XT) <= 8 ? kUnits : 2;  // units whose loads are in flight together
#pragma unroll 1
      for (int u0 = 0; u0 < kUnits; u0 += kAhead) {
        Eight<XT> v[kAhead][NT];
        if (whole) {
#pragma unroll
          for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int j = 0; j < NT; ++j) v[u][j].load16(xrow[j] + k0 + 32 * (u0 + u), 8 * j + gr < p.M);
        } else {
#pragma unroll
          for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              const int k = k0 + 32 * (u0 + u);
              v[u][j].load(xrow[j] + k, 8 * j + gr < p.M ? K - k : 0);
            }
        }
        if (!waited) {
          waited = wait_bounded(&empty[st], (b / C::kStages - 1) & 1u, &abort_flag, err,
                                kErrTimeout | kRoleProducer | kWaitStageEmpty);
          if (!waited) break;
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            uint4 x[PARTS];
            v[u][j].template pairs<PARTS>(x);
#pragma unroll
            for (int c = 0; c < PARTS; ++c) xs[(((u0 + u) * NT + j) * PARTS + c) * 32] = x[c];
          }
      }
      if (!waited) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[st]);
    }
  }

  // the warps' sums as a partial tile [activation row][matrix row], over the ring
  __syncthreads();
  float* tile = reinterpret_cast<float*>(ring);
  if (warp < kMmaWarps) {
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

// K splits of a row tile (a power of two up to 8) on a GPU that holds `slots`
// CTAs: the one with the least K blocks on the busiest slot, counting a CTA's
// fixed costs as two blocks.
int splits_for(long long tiles, long long blocks, long long slots) {
  int best = 1;
  long long least = 0;
  for (int S = 1; S <= 8 && S <= blocks; S *= 2) {
    const long long cost = ((tiles * S + slots - 1) / slots) * ((blocks + S - 1) / S + 2);
    if (S == 1 || cost < least) best = S, least = cost;
  }
  return best;
}

template <typename XT, int GPB, int NT>
cudaError_t launch_one(const Int4Product& p, const CUtensorMap& q, int sms, uint32_t* err, cudaStream_t stream) {
  using C = Config<XT, GPB, NT>;
  int per_sm = 0;
  cudaError_t e = ctas_per_sm_once<gemv_int4_kernel<XT, GPB, NT>>(kThreads, C::kSmem, &per_sm);
  if (e != cudaSuccess) return e;
  const bool xvec = (reinterpret_cast<uintptr_t>(p.x) & 15u) == 0 && (p.ldx * sizeof(XT)) % 16 == 0;
  const long long tiles = (p.N + kInt4TileRows - 1) / kInt4TileRows;
  const int S = splits_for(tiles, (p.K + 127) / 128, static_cast<long long>(per_sm) * sms);
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
