// Weight gradients of the gated feed-forward block:
//   dWg[o][i] = add + sum_t dgate[t][o] x[t][i],  dWu likewise from dup.
//
// One tcgen05 GEMM over the tokens for both (their tiles are dealt as those of one
// matrix of twice the outputs), both operands MN-major as they lie in memory: a
// token's row holds 64 outputs or inputs in 128 bytes. A CTA pair computes 256
// outputs x 256 inputs. The tensor core's fp32 sums cut off instead of rounding,
// which bends a long sum towards zero in proportion to its length, so TMEM holds the
// sum of at most 512 tokens at a time (two buffers in turn), and the epilogue warps add
// each to the tile's running sum in their registers, rounded. The last round's tiles
// are cut into ranges of tokens where they fill it badly (wgrad_plan.h).
#include <algorithm>

#include "glu.h"
#include "launch.h"
#include "pair_roles.cuh"
#include "row_ops.cuh"
#include "wgrad_plan.h"

namespace grpo {
namespace {

constexpr int kStages = 5;
constexpr int kBox = kTok * 128;     // 64 tokens x 64 columns
constexpr int kOperand = 2 * kBox;   // a CTA's 128 outputs, or 128 inputs
// Stages summed in TMEM: 512 tokens of bf16, 256 of fp16, whose products have 22
// significant bits against 16, so that more of each is cut off (512 tokens of one sign:
// bf16 9e-7 off, fp16 2.8e-6; 256 of them in bf16 cost 5541 x 1536 x 8960 262 us
// against 250).
__host__ __device__ __forceinline__ int segment_of(const GluWgradArgs& a) {
  return a.fp16 ? 4 : 8;
}
constexpr int kEpilogueWarps = 8;
constexpr int kFirstEpilogue = 4;  // warps 0 TMA, 1 MMA, 2 and 3 idle
constexpr int kThreads = 32 * (kFirstEpilogue + kEpilogueWarps);
// dW leaves, and what is added to it comes, by TMA in boxes of 32 outputs x 16 inputs,
// four a warp in turn: a thread's own accesses, 16 bytes of a row each, held the next
// tile's sums up (4096 tokens x 4096 x 14336: 672 us without `add`, 862 with it).
constexpr int kBoxBytes = 32 * 64, kBoxes = 4, kBoxesOfTile = kTileN / 2 / 16;
constexpr int kSmem = 1024 + 2 * kStages * kOperand + kEpilogueWarps * kBoxes * kBoxBytes;
static_assert(kSmem <= 227 * 1024 - 1024, "shared memory of a CTA");
static_assert(kBoxesOfTile == 2 * kBoxes, "each box is loaded twice a tile");
constexpr uint32_t kTmemCols = 512;
constexpr int kSlotFloats = kTileM * kTileN;
// Self-test: from here on `lost` counts boxes to add of the first CTA's first tile.
constexpr uint32_t kLostBox = 1u << 29;

// Row tiles of one weight: the first half of the plan's are the gate's.
__host__ __device__ __forceinline__ int half_tiles(int f) { return (f + kTileM - 1) / kTileM; }

// Where a tile's rows are: of which weight, from which output on.
struct Side {
  bool up;
  int o0;
};
__device__ __forceinline__ Side side_of(const GluWgradArgs& a, int tm) {
  const int half = half_tiles(a.f);
  const bool up = tm >= half;
  return {up, (up ? tm - half : tm) * kTileM};
}

__global__ void __launch_bounds__(kThreads, 1)
    glu_wgrad_kernel(const __grid_constant__ CUtensorMap map_gate,
                     const __grid_constant__ CUtensorMap map_up,
                     const __grid_constant__ CUtensorMap map_x,
                     const __grid_constant__ CUtensorMap map_dw0,
                     const __grid_constant__ CUtensorMap map_dw1,
                     const __grid_constant__ CUtensorMap map_add0,
                     const __grid_constant__ CUtensorMap map_add1, const GluWgradArgs args,
                     const WgradPlan plan) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[kStages];  // leader: both CTAs' tiles are there
  __shared__ __align__(8) uint64_t done_bar[kStages];  // the stage's MMAs are done
  __shared__ __align__(8) uint64_t tfull_bar[2], tempty_bar[2];
  __shared__ __align__(8) uint64_t add_bar[kEpilogueWarps][kBoxes];  // a box to add landed
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;

  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* const ring = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* const boxes = ring + 2 * kStages * kOperand;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(blockIdx.x) / 2, pairs = static_cast<int>(gridDim.x) / 2;
  volatile int* abort_flag = &abort_sh;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    // The status word of this call. Nothing writes it before a wait runs out.
    if (blockIdx.x == 0) *args.status = GRPO_OK;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_bar[s], 2);
      mbar_init(&done_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], 2 * kEpilogueWarps);  // both CTAs' epilogue warps
    }
    for (int w = 0; w < kEpilogueWarps; ++w)
      for (int b = 0; b < kBoxes; ++b) mbar_init(&add_bar[w][b], 1);
    mbar_init(&drain_bar, 1);
    abort_sh = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&map_gate);
    tma_prefetch_desc(&map_up);
    tma_prefetch_desc(&map_x);
  }
  if (warp == 1) {
    tmem_alloc_pair(&tmem_base_sh, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = tmem_base_sh;

  WgradWork work;
  WgradItem it;
  bool ok = true;
  const int segment = segment_of(args);
  // One lane of each role walks through the work, waits and issues; the others are
  // at the warp barrier before the closing cluster barrier.
  if (warp == 0) {
    // ------------------------------------------------------ tiles by TMA --
    if (elect_one()) {
      uint32_t n = 0;  // stages issued
      while (ok && work.next(plan, pair, pairs, it)) {
        int tm, tn;
        tile_place(plan, it.tile, tm, tn);
        const Side side = side_of(args, tm);
        const CUtensorMap* ma = side.up ? &map_up : &map_gate;
        const int o0 = side.o0 + static_cast<int>(rank) * (kTileM / 2);
        const int i0 = tn * kTileN + static_cast<int>(rank) * (tile_cols(args.d, tn) / 2);
        for (int k = it.kb; k < it.ke; ++k, ++n) {
          const uint32_t s = n % kStages;
          if (!mbar_wait(&done_bar[s], ((n / kStages) & 1u) ^ 1u, abort_flag, args.status)) {
            ok = false;
            break;
          }
          if (n == args.lost && blockIdx.x == 0) continue;
          const uint32_t lead = mapa_shared(smem_u32(&full_bar[s]), 0);
          mbar_arrive_expect_tx_cluster(lead, 2 * kOperand);
          uint8_t* a = ring + s * 2 * kOperand;
          tma_load_2d_pair_nohint(a, ma, lead, o0, k * kTok);
          tma_load_2d_pair_nohint(a + kBox, ma, lead, o0 + 64, k * kTok);
          tma_load_2d_pair_nohint(a + kOperand, &map_x, lead, i0, k * kTok);
          tma_load_2d_pair_nohint(a + kOperand + kBox, &map_x, lead, i0 + 64, k * kTok);
        }
      }
      // After a timeout: let the copies in flight land before the CTA exits.
      if (!ok && rank == 0)
        for (uint32_t j = n >= kStages ? n - kStages : 0; j < n; ++j)
          drain(&full_bar[j % kStages], (j / kStages) & 1u);
    }
  } else if (warp == 1 && rank == 0) {
    // -------------------------------------------------------- MMA issuer --
    if (elect_one()) {
      uint32_t n = 0, seg = 0;  // stages, segments issued
      const uint32_t type_bits = args.fp16 ? (1u << 7) | (1u << 10) : 0u;
      while (ok && work.next(plan, pair, pairs, it)) {
        int tm, tn;
        tile_place(plan, it.tile, tm, tn);
        const uint32_t idesc = idesc_bf16(kTileM, tile_cols(args.d, tn), true, true) & ~type_bits;
        for (int k = it.kb; k < it.ke; ++k, ++n) {
          const bool first = ((k - it.kb) & (segment - 1)) == 0;
          const bool last = ((k - it.kb + 1) & (segment - 1)) == 0 || k == it.ke - 1;
          const uint32_t buf = seg & 1u;
          if (first &&
              !mbar_wait(&tempty_bar[buf], ((seg >> 1) & 1u) ^ 1u, abort_flag, args.status)) {
            ok = false;
            break;
          }
          const uint32_t s = n % kStages;
          if (!mbar_wait(&full_bar[s], (n / kStages) & 1u, abort_flag, args.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t dcol = tmem_base + buf * kTileN;
          const uint32_t a = smem_u32(ring + s * 2 * kOperand), b = a + kOperand;
#pragma unroll
          for (int kk = 0; kk < kTok / 16; ++kk)
            // 64-wide blocks of outputs or inputs 8 KB apart, 8 tokens 1 KB.
            tc_mma_bf16_pair(dcol, sdesc_sw128(a + kk * 2048, kBox, 1024),
                             sdesc_sw128(b + kk * 2048, kBox, 1024), idesc,
                             first && kk == 0 ? 0u : 1u);
          tc_commit_pair_multicast(&done_bar[s], 0x3);
          if (last) tc_commit_pair_multicast(&tfull_bar[buf], 0x3);
          seg += last ? 1 : 0;
        }
      }
      tc_commit_pair(&drain_bar);
      drain(&drain_bar, 0);
    }
  } else if (warp >= kFirstEpilogue) {
    // ---------------------------------------------------------- epilogue --
    // A thread holds one output's sums over half of the tile's inputs.
    const int q = warp & 3;  // TMEM lane quarter of this warp
    const int half = (warp - kFirstEpilogue) >> 2;
    const uint32_t tempty0 = mapa_shared(smem_u32(&tempty_bar[0]), 0);
    const uint32_t t0 =
        tmem_base + (static_cast<uint32_t>(q * 32) << 16) + half * (kTileN / 2);
    uint32_t seg = 0;
    const int wid = warp - kFirstEpilogue;
    uint8_t* const box0 = boxes + wid * kBoxes * kBoxBytes;
    const uint32_t lane_row = smem_u32(box0) + lane * 64, swizzle = (lane >> 1) & 3;
    // Of the current tile: boxes of `add` asked for, and waited for. Each tile has all
    // of its boxes loaded, so a box's first load of a tile ends phase 0, its second 1.
    int asked = 0, had = 0;
    const uint32_t lost_box =
        args.lost != kNoneLost && args.lost >= kLostBox && blockIdx.x == 0 && wid == 0
            ? args.lost - kLostBox
            : kNoneLost;
    while (ok && work.next(plan, pair, pairs, it)) {
      int tm, tn;
      tile_place(plan, it.tile, tm, tn);
      const Side side = side_of(args, tm);
      const int row0 = side.o0 + static_cast<int>(rank) * 128 + q * 32;
      const int col0 = tn * kTileN + half * (kTileN / 2);
      const CUtensorMap* const map_add = side.up ? &map_add1 : &map_add0;
      const bool whole = it.slot < 0 && row0 < args.f && col0 < args.d;
      const bool adds = whole && (side.up ? args.add_up : args.add_gate) != nullptr;
      auto ask = [&](int b) {
        if (lane == 0 && (static_cast<uint32_t>(b) != lost_box || it.tile != 0)) {
          uint64_t* bar = &add_bar[wid][b % kBoxes];
          mbar_arrive_expect_tx(bar, kBoxBytes);
          tma_load_2d(box0 + (b % kBoxes) * kBoxBytes, map_add, bar, col0 + 16 * b, row0);
        }
      };
      asked = had = 0;
      if (adds) {  // the first boxes come while the tile's sums do
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
        for (; asked < kBoxes; ++asked) ask(asked);
      }
      float sum[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 32; ++j) sum[c][j] = 0.f;
      for (int k = it.kb; k < it.ke; k += segment, ++seg) {
        const uint32_t buf = seg & 1u;
        if (!warp_wait(&tfull_bar[buf], (seg >> 1) & 1u, abort_flag, args.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            float v[8];
            tmem_ld8(t0 + buf * kTileN + c * 32 + h * 8, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[c][8 * h + j] += v[j];
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty0 + buf * 8u);
      }
      if (!ok) break;
      if (it.slot >= 0) {
        const int lrow = static_cast<int>(rank) * 128 + q * 32 + lane;  // row of the tile
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (col0 + c * 32 >= args.d) break;
          float* p = args.partials + static_cast<long long>(it.slot) * kSlotFloats +
                     ((half * 4 + c) * 8 * kTileM + lrow) * 4;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<float4*>(p + j * kTileM * 4) = make_float4(
                sum[c][4 * j], sum[c][4 * j + 1], sum[c][4 * j + 2], sum[c][4 * j + 3]);
        }
        __syncwarp();
        continue;
      }
      if (!whole) continue;
#pragma unroll
      for (int b = 0; b < kBoxesOfTile; ++b) {
        float* const v = &sum[b / 2][16 * (b % 2)];
        const uint32_t at = lane_row + (b % kBoxes) * kBoxBytes;
        if (adds) {
          ok = ok && warp_wait(&add_bar[wid][b % kBoxes], b / kBoxes, abort_flag, args.status);
          if (ok) had = b + 1;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 x = lds_v4(at + ((j ^ swizzle) << 4));
            v[4 * j] += __uint_as_float(x.x);
            v[4 * j + 1] += __uint_as_float(x.y);
            v[4 * j + 2] += __uint_as_float(x.z);
            v[4 * j + 3] += __uint_as_float(x.w);
          }
        } else {
          if (lane == 0) bulk_wait_group_read<kBoxes - 1>();
          __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          sts_v4(at + ((j ^ swizzle) << 4), __float_as_uint(v[4 * j]),
                 __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]),
                 __float_as_uint(v[4 * j + 3]));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (ok && col0 + 16 * b < args.d)
            tma_store_2d(side.up ? &map_dw1 : &map_dw0, box0 + (b % kBoxes) * kBoxBytes,
                         col0 + 16 * b, row0);
          bulk_commit_group();
        }
        if (adds && ok && b > 0 && asked < kBoxesOfTile) {  // into the box before this one
          if (lane == 0) bulk_wait_group_read<1>();
          ask(asked++);
        }
      }
      if (!ok) break;
    }
    // Copies in flight land before the CTA exits.
    if (!ok && lane == 0)
      for (; had < asked; ++had) drain(&add_bar[wid][had % kBoxes], had / kBoxes);
    // A tile, or a piece of one, is whole or NaN: so are this one and the rest. Boxes of
    // this one that are on their way out land first.
    if (!ok) {
      if (lane == 0) bulk_wait_group<0>();
      __syncwarp();
      do {
        int tm, tn;
        tile_place(plan, it.tile, tm, tn);
        const Side side = side_of(args, tm);
        const int lrow = static_cast<int>(rank) * 128 + q * 32 + lane;
        const int row = side.o0 + lrow;
        float* dw = side.up ? args.dw_up : args.dw_gate;
#pragma unroll 1
        for (int c4 = half * 32; c4 < half * 32 + 32; ++c4) {
          const int i0 = tn * kTileN + 4 * c4;
          float* p = it.slot >= 0
                         ? args.partials + static_cast<long long>(it.slot) * kSlotFloats +
                               (c4 * kTileM + lrow) * 4
                     : row < args.f && i0 < args.d
                         ? dw + static_cast<long long>(row) * args.d + i0
                         : nullptr;
          if (p != nullptr) *reinterpret_cast<float4*>(p) = make_float4(kNaN, kNaN, kNaN, kNaN);
        }
      } while (work.next(plan, pair, pairs, it));
    }
    if (lane == 0) bulk_wait_group<0>();
  }

  // Neither CTA may leave while the other's tensor core reads its shared memory
  // or an arrival is on its way to it: every thread arrives for itself here.
  __syncwarp();
  tc_fence_before();
  cluster_sync_threads();
  tc_fence_after();
  __syncwarp();
  if (warp == 1) tmem_dealloc_pair(tmem_base, kTmemCols);
}

// The cut tiles: the sum of each tile's pieces in the order of their tokens, and
// `add`. A CTA takes 16 columns and 256 / G rows of a tile; thread (row, g) adds the
// pieces g, g + G, ..., and the G sums are then added in their order.
template <int G>
__global__ void __launch_bounds__(kTileM) glu_wgrad_join_kernel(const GluWgradArgs args,
                                                                const WgradPlan plan) {
  constexpr int kRows = kTileM / G;
  __shared__ float4 part[G > 1 ? G : 1][G > 1 ? 4 : 1][G > 1 ? kRows : 1];
  const int t = static_cast<int>(blockIdx.x);
  const int qa = first_piece(plan, t), qb = last_piece(plan, t);
  int tm, tn;
  tile_place(plan, plan.whole + t, tm, tn);
  const Side side = side_of(args, tm);
  const int r = static_cast<int>(threadIdx.x) % kRows, g = static_cast<int>(threadIdx.x) / kRows;
  const int lrow = static_cast<int>(blockIdx.z) * kRows + r;
  const int row = side.o0 + lrow;
  const int c0 = static_cast<int>(blockIdx.y) * 16;  // column of the tile
  const int i0 = tn * kTileN + c0;
  const bool valid = row < args.f && i0 < args.d;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the pieces are there
  float4 v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (valid) {
#pragma unroll 4
    for (int q = qa + g; q <= qb; q += G) {
      const float* p = args.partials +
                       static_cast<long long>(piece_slot(plan, t, q)) * kSlotFloats +
                       (c0 / 4 * kTileM + lrow) * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 x = *reinterpret_cast<const float4*>(p + j * kTileM * 4);
        v[j].x += x.x;
        v[j].y += x.y;
        v[j].z += x.z;
        v[j].w += x.w;
      }
    }
  }
  if constexpr (G > 1) {
#pragma unroll
    for (int j = 0; j < 4; ++j) part[g][j][r] = v[j];
    __syncthreads();
    if (g != 0) return;
    for (int k = 1; k < G; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 x = part[k][j][r];
        v[j].x += x.x;
        v[j].y += x.y;
        v[j].z += x.z;
        v[j].w += x.w;
      }
  }
  if (!valid) return;
  const long long at = static_cast<long long>(row) * args.d + i0;
  const float* add = side.up ? args.add_up : args.add_gate;
  float* dw = side.up ? args.dw_up : args.dw_gate;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (i0 + 4 * j >= args.d) break;
    if (add != nullptr) {
      const float4 x = *reinterpret_cast<const float4*>(add + at + 4 * j);
      v[j].x += x.x;
      v[j].y += x.y;
      v[j].z += x.z;
      v[j].w += x.w;
    }
    *reinterpret_cast<float4*>(dw + at + 4 * j) = v[j];
  }
}

}  // namespace

size_t glu_wgrad_workspace(long long n, int f, int d) {
  return 256 + partial_tiles(n, 2 * half_tiles(f) * kTileM, d) * kSlotFloats * sizeof(float);
}

cudaError_t prepare_glu_wgrad() {
  return cudaFuncSetAttribute(glu_wgrad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kSmem);
}

cudaError_t launch_glu_wgrad(const GluWgradArgs& a, int sms, cudaStream_t st) {
  const int pairs = std::min(sms / 2, kRefPairs);
  CUtensorMap map_gate, map_up, map_x;
  auto map = [&](CUtensorMap* m, const void* base, int cols, long long ld) {
    return encode_map_2d(m, base, static_cast<uint64_t>(cols), static_cast<uint64_t>(a.n),
                         static_cast<uint64_t>(ld) * 2, 64, kTok, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                         CU_TENSOR_MAP_SWIZZLE_128B);
  };
  if (!map(&map_gate, a.dgate, a.f, a.ldg) || !map(&map_up, a.dup, a.f, a.ldu) ||
      !map(&map_x, a.x, a.d, a.ldx))
    return cudaErrorInvalidValue;
  // dW and what is added to it, by 16 inputs.
  CUtensorMap out[4];
  const float* const base[4] = {a.dw_gate, a.dw_up, a.add_gate, a.add_up};
  for (int i = 0; i < 4; ++i) {
    if (base[i] == nullptr)
      out[i] = out[0];
    else if (!encode_map_2d(&out[i], base[i], static_cast<uint64_t>(a.d),
                            static_cast<uint64_t>(a.f), static_cast<uint64_t>(a.d) * 4, 16, 32,
                            CU_TENSOR_MAP_DATA_TYPE_FLOAT32, CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
  }
  WgradPlan plan = make_plan(a.n, 2 * half_tiles(a.f) * kTileM, a.d, pairs);
  plan.group = kGluGroup;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * launch_pairs(plan, pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  {
    LaunchTimer timer("glu_wgrad_kernel", st);
    e = cudaLaunchKernelEx(&cfg, glu_wgrad_kernel, map_gate, map_up, map_x, out[0], out[1], out[2],
                           out[3], a, plan);
  }
  if (e != cudaSuccess || plan.cut == 0) return e;
  // Its launch overlaps the end of the other (it waits for that itself).
  const int pieces = (plan.kt + plan.per_pair - 1) / plan.per_pair + 1;  // of a tile, at most
  const int groups = pieces > 4 ? 8 : 1;
  cudaLaunchConfig_t join = {};
  join.gridDim = dim3(plan.cut, kTileN / 16, groups);
  join.blockDim = dim3(kTileM);
  join.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  join.attrs = attr;
  join.numAttrs = 1;
  LaunchTimer timer("glu_wgrad_join_kernel", st);
  return groups == 8 ? cudaLaunchKernelEx(&join, glu_wgrad_join_kernel<8>, a, plan)
                     : cudaLaunchKernelEx(&join, glu_wgrad_join_kernel<1>, a, plan);
}

}  // namespace grpo
