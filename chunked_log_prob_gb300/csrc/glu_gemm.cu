// The gated feed-forward block's matrix products, with what belongs to them in the
// epilogue:
//   forward   h = act(x Wg^T) * (x Wu^T)
//   again     dgate = dh u act'(g), dup = dh act(g) from g = x Wg^T, u = x Wu^T
//   dx        dgate Wg + dup Wu
//
// One tcgen05 GEMM. A CTA pair computes 256 rows x 256 accumulator columns: of the
// first two, 128 columns of the gate and the same 128 of the other projection. Each
// CTA of a pair brings half of the second operand, so one loads Wg's rows and the
// other Wu's, and both projections of a value end up in the same thread's TMEM
// lane. They leave TMEM once, as h (or as the gradients): against two GEMMs and an
// elementwise pass, x is read once and the fp32 projections are never written. dx
// is one sum over 2 f columns, its first half from (dgate, Wg) and its second from
// (dup, Wu); where its tiles fill no round of the SM pairs, or the last one badly, they
// are cut along that sum, and a second kernel adds the pieces. TMEM holds two tiles, so an
// epilogue runs beside the next tile's MMAs.
//
// The tensor core's fp32 sums cut off instead of rounding: a unit of 2^-23 of the sum so
// far, at most, every 16 products, which bends a long sum towards zero (2^20 products of
// one sign: 7e-3). A sum of more than kSumStages is therefore made of sums of that many
// stages, added with rounding by the epilogue warps.
#include <algorithm>
#include <type_traits>

#include "glu.h"
#include "glu_act.cuh"
#include "launch.h"
#include "pair_roles.cuh"
#include "row_ops.cuh"
#include "wgrad_plan.h"

namespace grpo {
namespace {

constexpr int kFwd = 0, kAgain = 1, kDx = 2;

constexpr int kStages = 5;
constexpr int kBK = 64;                  // columns of a stage: 128 bytes
constexpr int kOperand = 128 * kBK * 2;  // a CTA's 128 rows of either operand
constexpr int kBox = kBK * 128;          // 64 rows x 64 columns of an MN-major operand
constexpr int kEpilogueWarps = 8;
constexpr int kFirstEpilogue = 4;  // warps 0 TMA, 1 MMA, 2 and 3 zeros of masked segments
constexpr int kThreads = 32 * (kFirstEpilogue + kEpilogueWarps);
constexpr int kSeg = 16;               // rows of a segment
constexpr int kTileSegs = 256 / kSeg;
// Segments that a CTA lists (2 bytes each): 131072 rows. Beyond them masked rows are
// computed like the others, and their zeros written in the epilogue.
constexpr int kMostSegs = 8192;
// Outputs leave by TMA from boxes of 32 rows x 32 columns, three a warp in turn: a
// thread's own stores, 16 bytes of a row each, took longer than a tile's MMAs
// (8192 x 1536 x 8960 padded, h and the projections: 254 us).
constexpr int kOutBox = 32 * 64, kOutBoxes = 3;
constexpr int kSmem = 1024 + 2 * kStages * kOperand + kEpilogueWarps * kOutBoxes * kOutBox +
                      2 * kMostSegs;
static_assert(kSmem <= 227 * 1024 - 1024, "shared memory of a CTA");
constexpr uint32_t kTmemCols = 512;
constexpr int kSlotFloats = kTileM * kTileN;  // of a piece of a cut tile
// Stages of one sum in TMEM: 1024 products. Values of random sign, of which a wrong sum now
// and then sends one to the other 16-bit neighbour: h at 16384 x 4096 x 14336 is not the
// nearest to its value in 64 bits in 1.2e-3 of them (6.7e-4 where fp32 sums round), dx at
// 8192 x 1536 x 8960 in 1.2e-3 (1.5e-3); with whole sums in TMEM 4.2e-3 and 7.8e-3. Stages
// of one sum, forward / backward again there and forward padded (us, one box): all 2185 /
// 4671 / 234, 32 2204 / 4706 / 234, 16 2214 / 4808 / 240, 8 2248 / 4895 / 252.
constexpr int kSumStages = 16;

// The launch's tiles: 256 rows x `cols` columns of f (of d for dx), dealt to the pairs
// by `work`; its kt counts the stages of a tile, for dx those of both operand pairs.
struct GluPlan {
  WgradPlan work;
  int half;  // dx: stages of the first operand pair
  int cols;  // forward and again: 128, 96 or 64; dx: 256 or 128
  int segs;  // segments to list, 0: tiles are of consecutive rows
};

// Whether a segment holds a row that counts.
__device__ __forceinline__ bool segment_lives(const uint8_t* mask, long long n, int seg) {
  const long long r0 = static_cast<long long>(seg) * kSeg;
  const uint8_t* p = mask + r0;
  if (r0 + kSeg <= n && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    return (v.x | v.y | v.z | v.w) != 0;
  }
  bool any = false;
  for (int i = 0; i < kSeg && r0 + i < n; ++i) any = any || p[i] != 0;
  return any;
}

// Lists the segments of all rows: those that live first, in order, then the others.
// All threads of the CTA call this. Returns how many live.
__device__ __forceinline__ int list_segments(const uint8_t* mask, long long n, int segs,
                                             uint16_t* list, int* scratch) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int each = (segs + kThreads - 1) / kThreads;
  const int a = least(static_cast<int>(threadIdx.x) * each, segs), b = least(a + each, segs);
  int mine = 0;
  for (int s = a; s < b; ++s) mine += segment_lives(mask, n, s) ? 1 : 0;
  int before = mine;  // inclusive sums, of the warp and then of the warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) scratch[warp] = before;
  __syncthreads();
  int live = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == warp) before += live - mine;
    live += scratch[w];
  }
  int other = live + a - before;  // where this thread's first dead one goes
  for (int s = a; s < b; ++s) {
    if (segment_lives(mask, n, s))
      list[before++] = static_cast<uint16_t>(s);
    else
      list[other++] = static_cast<uint16_t>(s);
  }
  __syncthreads();
  return live;
}

template <typename T>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  return std::is_same_v<T, __half> ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}
template <typename T>
__device__ __forceinline__ void unpack16(uint32_t w, float& lo, float& hi) {
  if constexpr (std::is_same_v<T, __half>) {
    unpack_f16x2(w, lo, hi);
  } else {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xffff0000u);
  }
}

// A warp's boxes on their way out, through the 64-byte swizzle: the lane's row of 32
// columns, 16 at a time. The rows are two segments, of 16 lanes each.
struct OutBoxes {
  uint8_t* base;
  uint32_t turn;
  int lane;

  // The next box, free again.
  __device__ __forceinline__ uint32_t begin() {
    if (lane == 0) bulk_wait_group_read<kOutBoxes - 1>();
    __syncwarp();
    return smem_u32(base + turn * kOutBox);
  }
  __device__ __forceinline__ void put16(uint32_t box, int half, const uint32_t* w) const {
    const uint32_t row = box + lane * 64, x = (lane >> 1) & 3;
    sts_v4(row + (((2 * half) ^ x) << 4), w[0], w[1], w[2], w[3]);
    sts_v4(row + (((2 * half + 1) ^ x) << 4), w[4], w[5], w[6], w[7]);
  }
  // Sends it to column `col`, rows r0 and r1 on (n: not there).
  __device__ __forceinline__ void end(const CUtensorMap* map, int col, int r0, int r1, int n) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (r0 < n) tma_store_2d(map, base + turn * kOutBox, col, r0);
      if (r1 < n) tma_store_2d(map, base + turn * kOutBox + kOutBox / 2, col, r1);
      bulk_commit_group();
    }
    turn = turn == kOutBoxes - 1 ? 0 : turn + 1;
  }
};

template <typename T>
__device__ __forceinline__ void load16(const T* p, uint32_t (&w)[8], int left) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (8 * j < left) x = *reinterpret_cast<const uint4*>(p + 8 * j);
    w[4 * j] = x.x;
    w[4 * j + 1] = x.y;
    w[4 * j + 2] = x.z;
    w[4 * j + 3] = x.w;
  }
}

// 16 TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
      "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
      "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// A checkpoint block that one thread holds: 32 values as stored.
template <typename T>
__device__ __forceinline__ void ckpt_store32(const uint32_t (&w)[16], uint8_t* q, uint8_t* ex,
                                             int left) {
  float a = 0.f;
  bool special = false;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float lo, hi;
    unpack16<T>(w[j], lo, hi);
    const float m0 = fabsf(lo), m1 = fabsf(hi);
    if (m0 <= FLT_MAX) a = fmaxf(a, m0);
    if (m1 <= FLT_MAX) a = fmaxf(a, m1);
    special = special || !(m0 <= FLT_MAX) || !(m1 <= FLT_MAX);
  }
  const int k = ckpt_exponent(a);
  const float inv = pow2(-k);
  special = special || k >= CkptTop<T>::k;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float lo, hi;
      unpack16<T>(w[8 * j + i], lo, hi);
      o[i] = special ? pack_e4m3x2(ckpt_scaled<T>(lo, inv, k), ckpt_scaled<T>(hi, inv, k))
                     : pack_e4m3x2(lo * inv, hi * inv);
    }
    // A row's bytes are padded to 16.
    if (16 * j < left)
      st_global_v4(q + 16 * j, __byte_perm(o[0], o[1], 0x5410), __byte_perm(o[2], o[3], 0x5410),
                   __byte_perm(o[4], o[5], 0x5410), __byte_perm(o[6], o[7], 0x5410));
  }
  *ex = static_cast<uint8_t>(k + kCkptBias);
}

// Columns of a dx tile's MMAs: half of them where no more are left.
__device__ __forceinline__ int dx_cols(const GluPlan& p, int d, int tn) {
  return p.cols == kTileN ? tile_cols(d, tn) : p.cols;
}

// LONG: tiles of more than kSumStages stages.
template <int MODE, typename T, bool LONG>
__global__ void __launch_bounds__(kThreads, 1)
    glu_gemm_kernel(const __grid_constant__ CUtensorMap map_a0,
                    const __grid_constant__ CUtensorMap map_a1,
                    const __grid_constant__ CUtensorMap map_s0,
                    const __grid_constant__ CUtensorMap map_s1,
                    const __grid_constant__ CUtensorMap map_b0,
                    const __grid_constant__ CUtensorMap map_b1,
                    const __grid_constant__ CUtensorMap map_o0,
                    const __grid_constant__ CUtensorMap map_o1,
                    const __grid_constant__ CUtensorMap map_o2, const GluArgs args,
                    const GluPlan plan) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[kStages];  // leader: both CTAs' tiles are there
  __shared__ __align__(8) uint64_t done_bar[kStages];  // the stage's MMAs are done
  __shared__ __align__(8) uint64_t tfull_bar[2], tempty_bar[2];
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh, status_sh;
  __shared__ int scratch[kThreads / 32];

  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* const ring = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* const boxes = ring + 2 * kStages * kOperand;
  uint16_t* const list =
      reinterpret_cast<uint16_t*>(boxes + kEpilogueWarps * kOutBoxes * kOutBox);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(blockIdx.x) / 2, pairs = static_cast<int>(gridDim.x) / 2;
  volatile int* abort_flag = &abort_sh;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_bar[s], 2);
      mbar_init(&done_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], 2 * kEpilogueWarps);  // both CTAs' epilogue warps
    }
    mbar_init(&drain_bar, 1);
    abort_sh = 0;
    status_sh = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&map_a0);
    tma_prefetch_desc(rank == 0 ? &map_b0 : &map_b1);
  }
  if (warp == 1) {
    tmem_alloc_pair(&tmem_base_sh, kTmemCols);
    tmem_relinquish_pair();
  }
  const int live_segs =
      plan.segs > 0 ? list_segments(args.mask, args.n, plan.segs, list, scratch) : 0;
  WgradPlan wp = plan.work;
  if (plan.segs > 0) {  // nothing is cut then
    wp.n_m = (live_segs + kTileSegs - 1) / kTileSegs;
    wp.whole = wp.n_m * wp.n_n;
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if constexpr (MODE == kDx)
    asm volatile("griddepcontrol.wait;" ::: "memory");  // dgate and dup are there
  if constexpr (MODE != kFwd) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem_base = tmem_base_sh;
  WgradWork work;
  WgradItem it;
  // Row of this CTA's row i of a row tile; args.n where there is none.
  auto row_of = [&](int tm, int i) -> long long {
    if (plan.segs == 0)
      return min(static_cast<long long>(tm) * kTileM + static_cast<int>(rank) * 128 + i, args.n);
    const int s = tm * kTileSegs + static_cast<int>(rank) * (kTileSegs / 2) + i / kSeg;
    return s < live_segs
               ? min(static_cast<long long>(list[s]) * kSeg + (i & (kSeg - 1)), args.n)
               : args.n;
  };

  bool ok = true;
  // One lane of each role walks through the work, waits and issues; the others are
  // at the warp barrier before the closing cluster barrier.
  if (warp == 0) {
    // ------------------------------------------------------ tiles by TMA --
    if (elect_one()) {
      uint32_t n = 0;  // stages issued
      // dx: half a tile's columns are a box of 64, or two
      const bool two = MODE == kDx && plan.cols == kTileN;
      const uint32_t b_bytes =
          MODE == kDx ? (two ? kOperand : kBox) : static_cast<uint32_t>(plan.cols) * kBK * 2;
      while (ok && work.next(wp, pair, pairs, it)) {
        int tm, tn;
        tile_place(wp, it.tile, tm, tn);
        int rows[kTileSegs / 2];  // where the tile's segments begin
#pragma unroll
        for (int j = 0; j < kTileSegs / 2; ++j) rows[j] = static_cast<int>(row_of(tm, j * kSeg));
        // One box holds them where the last one is there, and that far from the first.
        const int last = rows[kTileSegs / 2 - 1];
        const bool together = plan.segs == 0 || (last < args.n && last - rows[0] == 128 - kSeg);
        const int n0 = tn * plan.cols + (MODE == kDx ? static_cast<int>(rank) *
                                                           (dx_cols(plan, args.d, tn) / 2)
                                                     : 0);
        for (int k = it.kb; k < it.ke; ++k, ++n) {
          const uint32_t s = n % kStages;
          if (!mbar_wait(&done_bar[s], ((n / kStages) & 1u) ^ 1u, abort_flag, &status_sh)) {
            ok = false;
            break;
          }
          if (n == args.lost && blockIdx.x == 0) continue;
          const uint32_t lead = mapa_shared(smem_u32(&full_bar[s]), 0);
          mbar_arrive_expect_tx_cluster(lead, kOperand + b_bytes);
          uint8_t* a = ring + s * 2 * kOperand;
          uint8_t* b = a + kOperand;
          const bool second = MODE == kDx && k >= plan.half;
          const int k0 = (second ? k - plan.half : k) * kBK;
          if (together) {
            tma_load_2d_pair_nohint(a, second ? &map_a1 : &map_a0, lead, k0, rows[0]);
          } else {
            const CUtensorMap* ms = second ? &map_s1 : &map_s0;
#pragma unroll
            for (int j = 0; j < kTileSegs / 2; ++j)
              tma_load_2d_pair_nohint(a + j * kSeg * kBK * 2, ms, lead, k0, rows[j]);
          }
          if constexpr (MODE == kDx) {
            const CUtensorMap* mb = second ? &map_b1 : &map_b0;
            tma_load_2d_pair_nohint(b, mb, lead, n0, k0);
            if (two) tma_load_2d_pair_nohint(b + kBox, mb, lead, n0 + 64, k0);
          } else {
            tma_load_2d_pair_nohint(b, rank == 0 ? &map_b0 : &map_b1, lead, k0, n0);
          }
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
      uint32_t n = 0, t = 0;  // stages, sums issued
      const uint32_t type_bits = args.fp16 ? (1u << 7) | (1u << 10) : 0u;
      while (ok && work.next(wp, pair, pairs, it)) {
        int tm, tn;
        tile_place(wp, it.tile, tm, tn);
        const uint32_t idesc =
            idesc_bf16(kTileM, MODE == kDx ? dx_cols(plan, args.d, tn) : 2 * plan.cols, false,
                       MODE == kDx) &
            ~type_bits;
        for (int k0 = it.kb; ok && k0 < it.ke; ++t) {
          const int k1 = LONG ? least(k0 + kSumStages, it.ke) : it.ke;
          const uint32_t buf = t & 1u;
          if (!mbar_wait(&tempty_bar[buf], ((t >> 1) & 1u) ^ 1u, abort_flag, &status_sh)) {
            ok = false;
            break;
          }
          const uint32_t dcol = tmem_base + buf * kTileN;
          for (int k = k0; k < k1; ++k, ++n) {
            const uint32_t s = n % kStages;
            if (!mbar_wait(&full_bar[s], (n / kStages) & 1u, abort_flag, &status_sh)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a = smem_u32(ring + s * 2 * kOperand), b = a + kOperand;
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk)
              tc_mma_bf16_pair(dcol, sdesc_sw128(a + kk * 32, 16, 1024),
                               MODE == kDx ? sdesc_sw128(b + kk * 2048, kBox, 1024)
                                           : sdesc_sw128(b + kk * 32, 16, 1024),
                               idesc, k == k0 && kk == 0 ? 0u : 1u);
            tc_commit_pair_multicast(&done_bar[s], 0x3);
          }
          if (ok) tc_commit_pair_multicast(&tfull_bar[buf], 0x3);
          k0 = k1;
        }
      }
      tc_commit_pair(&drain_bar);
      drain(&drain_bar, 0);
    }
  } else if (warp < kFirstEpilogue && warp > 1) {
    // ------------------------------------- zeros of the masked segments --
    const int width = MODE == kDx ? args.d : args.f;
    for (int i = live_segs + static_cast<int>(blockIdx.x); i < plan.segs;
         i += static_cast<int>(gridDim.x)) {
#pragma unroll 1
      for (int r = 0; r < kSeg; ++r) {
        const long long row = static_cast<long long>(list[i]) * kSeg + r;
        if (row >= args.n) break;
        for (int c = (static_cast<int>(threadIdx.x) - 64) * 8; c < width; c += 64 * 8) {
          if (MODE == kDx) {
            st_global_v4(static_cast<T*>(args.dx) + row * args.lddx + c, 0u, 0u, 0u, 0u);
            continue;
          }
          if (args.h != nullptr)
            st_global_v4(static_cast<T*>(args.h) + row * args.ldh + c, 0u, 0u, 0u, 0u);
          if (args.gate != nullptr)
            st_global_v4(static_cast<T*>(args.gate) + row * args.ldg + c, 0u, 0u, 0u, 0u);
          if (args.up != nullptr)
            st_global_v4(static_cast<T*>(args.up) + row * args.ldu + c, 0u, 0u, 0u, 0u);
          if (args.ck.q != nullptr) {
            *reinterpret_cast<uint2*>(args.ck.q + row * args.ck.ldq + c) = make_uint2(0u, 0u);
            args.ck.ex[row * args.ck.lde + c / kCkptBlock] =
                static_cast<uint8_t>(kCkptMinExp + kCkptBias);
          }
        }
      }
    }
  } else if (warp >= kFirstEpilogue) {
    // ---------------------------------------------------------- epilogue --
    // A thread holds one row's half of the tile's columns.
    const int q = warp & 3;  // TMEM lane quarter of this warp
    const int half = (warp - kFirstEpilogue) >> 2;
    const uint32_t tempty0 = mapa_shared(smem_u32(&tempty_bar[0]), 0);
    const uint32_t t0 = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    uint32_t t = 0;
    OutBoxes out = {boxes + (warp - kFirstEpilogue) * kOutBoxes * kOutBox, 0u, lane};
    const int n = static_cast<int>(args.n);
    for (; work.next(wp, pair, pairs, it); ++t) {
      int tm, tn;
      tile_place(wp, it.tile, tm, tn);
      const long long row = row_of(tm, q * 32 + lane);
      const int r0 = static_cast<int>(row_of(tm, q * 32)),
                r1 = static_cast<int>(row_of(tm, q * 32 + 16));
      const bool there = row < args.n;
      const bool live = there && (args.mask == nullptr || args.mask[row] != 0);
      // The first of dh comes while the tile's (last) sum does, each next one a step ahead.
      uint32_t ahead[8];
      const T* dh = nullptr;
      auto bring_dh = [&] {
        const int f0 = tn * plan.cols;
        dh = static_cast<const T*>(args.dh) + row * args.lddh + f0;
        load16<T>(dh + half * 32, ahead,
                  live && half * 32 < plan.cols ? args.f - f0 - half * 32 : 0);
      };
      if constexpr (MODE == kAgain && !LONG) bring_dh();
      if constexpr (LONG) {
        // The sums before the tile's last are added up in registers, and then to that in
        // TMEM. Chunk c of this warp's 32 columns: of dx, or of either projection.
        float sum[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[c][j] = 0.f;
        auto chunk = [&](int c) {
          const int col = half * 32 + 64 * (MODE == kDx ? c : c & 1);
          return MODE == kDx ? col : col + (c >> 1) * plan.cols;
        };
        int k = it.kb;
        for (; ok && k + kSumStages < it.ke; k += kSumStages, ++t) {
          const uint32_t buf = t & 1u;
          if (!warp_wait(&tfull_bar[buf], (t >> 1) & 1u, abort_flag, &status_sh)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              float v[8];
              tmem_ld8(t0 + buf * kTileN + chunk(c) + 8 * h, v);
#pragma unroll
              for (int j = 0; j < 8; ++j) sum[c][8 * h + j] += v[j];
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(tempty0 + buf * 8u);
        }
        const uint32_t buf = t & 1u;
        if (!ok || !warp_wait(&tfull_bar[buf], (t >> 1) & 1u, abort_flag, &status_sh)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (k != it.kb) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              if (half * 32 + 64 * (MODE == kDx ? c : c & 1) >= plan.cols) continue;
              const uint32_t at = t0 + buf * kTileN + chunk(c) + 8 * h;
              float v[8];
              tmem_ld8(at, v);
#pragma unroll
              for (int j = 0; j < 8; ++j) v[j] += sum[c][8 * h + j];
              tmem_st8(at, v);
            }
          }
          tmem_wait_st();
        }
        if constexpr (MODE == kAgain) bring_dh();
      } else {
        if (!warp_wait(&tfull_bar[t & 1u], (t >> 1) & 1u, abort_flag, &status_sh)) {
          ok = false;
          break;
        }
        tc_fence_after();
      }
      const uint32_t buf = t & 1u;
      const uint32_t acc = t0 + buf * kTileN;
      const int width = MODE == kDx ? args.d : args.f;
      // The two halves of the warps take turns with the tile's 32 columns each.
#pragma unroll 1
      for (int col = half * 32; col < plan.cols; col += 64) {
        const int at = tn * plan.cols + col, left = width - at;
        if (left <= 0) break;
        if constexpr (MODE == kDx) {
          float v[32];
          tmem_ld32(acc + col, v);
          if (it.slot >= 0) {  // a piece of a cut tile
            float* p = args.partials + static_cast<long long>(it.slot) * kSlotFloats +
                       (col / 4 * kTileM + static_cast<int>(rank) * 128 + q * 32 + lane) * 4;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<float4*>(p + j * kTileM * 4) =
                  make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          } else {
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = live ? pack16<T>(v[2 * j], v[2 * j + 1]) : 0u;
            const uint32_t box = out.begin();
            out.put16(box, 0, w);
            out.put16(box, 1, w + 8);
            out.end(&map_o0, at, r0, r1, n);
          }
        } else if constexpr (MODE == kAgain) {
          // Three boxes at once: dgate, dup and (should it be wanted) h.
          const int outs = args.h != nullptr ? 3 : 2;
          const uint32_t box = smem_u32(out.base);
#pragma unroll 1
          for (int s = 0; s < 2; ++s) {
            float g[16], u[16];
            tmem_ld16(acc + col + 16 * s, g);
            tmem_ld16(acc + plan.cols + col + 16 * s, u);
            uint32_t d[8], dg[8], du[8], hw[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = ahead[j];
            const int next = s == 0 ? 16 : 64;  // columns on
            load16<T>(dh + col + next, ahead,
                      live && col + next < plan.cols ? left - next : 0);
            with_act(args.act, [&](auto tag) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                float d0, d1, s0, s1;
                unpack16<T>(d[j], d0, d1);
                const float a0 = activate<decltype(tag)::value, true>(g[2 * j], s0);
                const float a1 = activate<decltype(tag)::value, true>(g[2 * j + 1], s1);
                const float u0 = u[2 * j], u1 = u[2 * j + 1];
                dg[j] = live ? pack16<T>(d0 * u0 * s0, d1 * u1 * s1) : 0u;
                du[j] = live ? pack16<T>(d0 * a0, d1 * a1) : 0u;
                hw[j] = live ? pack16<T>(a0 * u0, a1 * u1) : 0u;
              }
            });
            if (s == 0) {  // the boxes before them have been read
              if (lane == 0) bulk_wait_group_read<0>();
              __syncwarp();
            }
            out.put16(box, s, dg);
            out.put16(box + kOutBox, s, du);
            if (outs == 3) out.put16(box + 2 * kOutBox, s, hw);
            __syncwarp();  // the next load is the whole warp's
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            const CUtensorMap* const to[3] = {&map_o0, &map_o1, &map_o2};
            for (int o = 0; o < outs; ++o) {
              if (r0 < n) tma_store_2d(to[o], out.base + o * kOutBox, at, r0);
              if (r1 < n) tma_store_2d(to[o], out.base + o * kOutBox + kOutBox / 2, at, r1);
            }
            bulk_commit_group();
          }
        } else {
          float g[32], u[32];
          tmem_ld32(acc + col, g);
          tmem_ld32(acc + plan.cols + col, u);
          uint32_t w[16];
          if (args.gate != nullptr) {
            uint32_t box = out.begin();
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = live ? pack16<T>(g[2 * j], g[2 * j + 1]) : 0u;
            out.put16(box, 0, w);
            out.put16(box, 1, w + 8);
            out.end(&map_o1, at, r0, r1, n);
            box = out.begin();
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = live ? pack16<T>(u[2 * j], u[2 * j + 1]) : 0u;
            out.put16(box, 0, w);
            out.put16(box, 1, w + 8);
            out.end(&map_o2, at, r0, r1, n);
          }
          with_act(args.act, [&](auto tag) {
            float s;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float h0 = activate<decltype(tag)::value, false>(g[2 * j], s) * u[2 * j];
              const float h1 =
                  activate<decltype(tag)::value, false>(g[2 * j + 1], s) * u[2 * j + 1];
              w[j] = live ? pack16<T>(h0, h1) : 0u;
            }
          });
          const uint32_t box = out.begin();
          out.put16(box, 0, w);
          out.put16(box, 1, w + 8);
          out.end(&map_o0, at, r0, r1, n);
          if (args.ck.q != nullptr && there)
            ckpt_store32<T>(w, args.ck.q + row * args.ck.ldq + at,
                            args.ck.ex + row * args.ck.lde + at / kCkptBlock, left);
        }
        __syncwarp();  // the next load is the whole warp's
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty0 + buf * 8u);
    }
    // A tile is whole or NaN: so are this one and the rest after a wait that ran out.
    if (!ok) {
      do {
        int tm, tn;
        tile_place(wp, it.tile, tm, tn);
        if (MODE == kDx && it.slot >= 0) {
          float* p = args.partials + static_cast<long long>(it.slot) * kSlotFloats +
                     (static_cast<int>(rank) * 128 + q * 32 + lane) * 4;
#pragma unroll 1
          for (int c4 = half * 32; c4 < half * 32 + 32; ++c4)
            *reinterpret_cast<float4*>(p + c4 * kTileM * 4) = make_float4(kNaN, kNaN, kNaN, kNaN);
          continue;
        }
        const long long row = row_of(tm, q * 32 + lane);
        if (row >= args.n) continue;
        const uint32_t w = pack16<T>(kNaN, kNaN);
        const int width = MODE == kDx ? args.d : args.f, cols = plan.cols / 2;
        const int c0 = tn * plan.cols + half * cols;  // any half: a multiple of 8
#pragma unroll 1
        for (int c = c0; c < least(c0 + cols, width); c += 8) {
          if (MODE == kDx) {
            st_global_v4(static_cast<T*>(args.dx) + row * args.lddx + c, w, w, w, w);
            continue;
          }
          if (args.h != nullptr)
            st_global_v4(static_cast<T*>(args.h) + row * args.ldh + c, w, w, w, w);
          if (args.gate != nullptr)
            st_global_v4(static_cast<T*>(args.gate) + row * args.ldg + c, w, w, w, w);
          if (args.up != nullptr)
            st_global_v4(static_cast<T*>(args.up) + row * args.ldu + c, w, w, w, w);
          if (args.ck.q != nullptr) {
            *reinterpret_cast<uint2*>(args.ck.q + row * args.ck.ldq + c) =
                make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
            args.ck.ex[row * args.ck.lde + c / kCkptBlock] = kCkptBias;
          }
        }
      } while (work.next(wp, pair, pairs, it));
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

// dx of the cut tiles: the sum of each tile's pieces in their order. A CTA takes 16
// columns and 256 / G rows of a tile; thread (row, g) adds the pieces g, g + G, ..., and
// the G sums are then added in their order.
template <typename T, int G>
__global__ void __launch_bounds__(kTileM) glu_dx_join_kernel(const GluArgs args,
                                                             const WgradPlan plan) {
  constexpr int kRows = kTileM / G;
  __shared__ float4 part[G > 1 ? G : 1][G > 1 ? 4 : 1][G > 1 ? kRows : 1];
  const int t = static_cast<int>(blockIdx.x);
  int tm, tn;
  tile_place(plan, plan.whole + t, tm, tn);
  const int r = static_cast<int>(threadIdx.x) % kRows, g = static_cast<int>(threadIdx.x) / kRows;
  const int lrow = static_cast<int>(blockIdx.z) * kRows + r;
  const long long row = static_cast<long long>(tm) * kTileM + lrow;
  const int c0 = static_cast<int>(blockIdx.y) * 16;  // column of the tile
  const int i0 = tn * kTileN + c0;
  const bool valid = row < args.n && i0 < args.d;
  const bool live = valid && (args.mask == nullptr || args.mask[row] != 0);
  const int qa = first_piece(plan, t), qb = last_piece(plan, t);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the pieces are there
  float v[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = 0.f;
  if (live) {
#pragma unroll 4
    for (int q = qa + g; q <= qb; q += G) {
      const float* p = args.partials +
                       static_cast<long long>(piece_slot(plan, t, q)) * kSlotFloats +
                       (c0 / 4 * kTileM + lrow) * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 x = *reinterpret_cast<const float4*>(p + j * kTileM * 4);
        v[4 * j] += x.x;
        v[4 * j + 1] += x.y;
        v[4 * j + 2] += x.z;
        v[4 * j + 3] += x.w;
      }
    }
  }
  if constexpr (G > 1) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      part[g][j][r] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    __syncthreads();
    if (g != 0) return;
    for (int k = 1; k < G; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 x = part[k][j][r];
        v[4 * j] += x.x;
        v[4 * j + 1] += x.y;
        v[4 * j + 2] += x.z;
        v[4 * j + 3] += x.w;
      }
  }
  if (!valid) return;
  T* const out = static_cast<T*>(args.dx) + row * args.lddx + i0;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (i0 + 8 * j < args.d)
      st_global_v4(out + 8 * j, pack16<T>(v[8 * j], v[8 * j + 1]),
                   pack16<T>(v[8 * j + 2], v[8 * j + 3]), pack16<T>(v[8 * j + 4], v[8 * j + 5]),
                   pack16<T>(v[8 * j + 6], v[8 * j + 7]));
}

template <typename T>
cudaError_t launch_dx_join(const GluArgs& args, const WgradPlan& plan, cudaStream_t st) {
  const int pieces = (plan.kt + plan.per_pair - 1) / plan.per_pair + 1;  // of a tile, at most
  const int groups = pieces > 4 ? 8 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(plan.cut, kTileN / 16, groups);
  cfg.blockDim = dim3(kTileM);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  LaunchTimer timer("glu_dx_join_kernel", st);
  return groups == 8 ? cudaLaunchKernelEx(&cfg, glu_dx_join_kernel<T, 8>, args, plan)
                     : cudaLaunchKernelEx(&cfg, glu_dx_join_kernel<T, 1>, args, plan);
}

template <int MODE, typename T, bool LONG>
cudaError_t launch(const CUtensorMap (&a)[4], const CUtensorMap (&b)[2],
                   const CUtensorMap (&o)[3], const GluArgs& args,
                   const GluPlan& plan, int sms, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * launch_pairs(plan.work, std::min(sms / 2, kRefPairs)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  // dx starts while the kernel before it ends (and waits for that itself).
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = MODE == kDx ? 2 : 1;
  cudaError_t e;
  {
    LaunchTimer timer(MODE == kFwd     ? "glu_gemm_kernel<fwd>"
                      : MODE == kAgain ? "glu_gemm_kernel<again>"
                                       : "glu_gemm_kernel<dx>",
                      st);
    e = cudaLaunchKernelEx(&cfg, glu_gemm_kernel<MODE, T, LONG>, a[0], a[1], a[2], a[3], b[0], b[1],
                           o[0], o[1], o[2], args, plan);
  }
  if (MODE != kDx || e != cudaSuccess || plan.work.cut == 0) return e;
  return launch_dx_join<T>(args, plan.work, st);
}

bool map16(CUtensorMap* map, const void* base, int cols, long long rows, long long ld,
           uint32_t box_rows) {
  return encode_map_2d(map, base, static_cast<uint64_t>(cols), static_cast<uint64_t>(rows),
                       static_cast<uint64_t>(ld) * 2, kBK, box_rows,
                       CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Columns of a tile: fewer where the rounds of the SM pairs then come out shorter. A
// stage of fewer columns brings as many rows of the first operand, so a tile of half
// the columns takes 0.70 to 0.73 of the time (16384 x 4096 x 14336 forward 2193 us with
// 128, 3076 with 64; 33 rows, which the weights bound, 62 in two rounds, 68 in three).
int tile_columns(int n_m, int width, int most, int pairs) {
  const int choice[3] = {most, most / 4 * 3, most / 2};
  const int cost[3] = {100, 86, 72};
  int best = most;
  long long least = 0;
  for (int i = 0; i < 3; ++i) {
    if (choice[i] == 192) continue;  // dx: its weights come in boxes of 64 columns
    const long long tiles = static_cast<long long>(n_m) * ((width + choice[i] - 1) / choice[i]);
    const long long time = (tiles + pairs - 1) / pairs * cost[i];
    if (i == 0 || time < least) {
      best = choice[i];
      least = time;
    }
  }
  return best;
}

// dx as a sum over the columns of dgate and of dup, dealt like that of a weight gradient
// over its tokens. Pieces of different tiles share no operands while they run, and a stage
// of them takes some 1.6 times as long, so tiles are cut only where that and the join (25
// stages) still save 24 of them, which the host's part of the join costs, and up to
// four whole rounds before them (16384 x 4096 x 14336, 13 rounds: 2453 and 2520 us).
// Uncut and cut, with the pass before it: 64 rows x 4096 x 14336 132 and 59 us, 512 rows
// 141 and 121, 35 x 496 x 6976 62 and 18, 3 x 48 x 12800 105 and 15; not cut by this rule
// (with whole sums in TMEM): 5888 x 1536 x 8960 255 and 312, 2048 rows 121 and 120, 1024 x
// 2880 x 2880 41 and 43.
WgradPlan dx_plan(long long n, int f, int d, int pairs) {
  const long long stages = 2LL * ((f + kBK - 1) / kBK);
  WgradPlan p = make_plan(stages * kTok, static_cast<int>(n), d, pairs);
  if (p.cut > 0 && (p.whole > 4 * kRefPairs || 8LL * p.per_pair + 5 * (25 + 24) > 5LL * p.kt ||
                    // the workspace is sized for kRefPairs
                    (pairs < kRefPairs && dx_plan(n, f, d, kRefPairs).cut == 0)))
    p.cut = 0;
  return p;
}

template <int MODE>
cudaError_t launch_mode(const GluArgs& args, int sms, cudaStream_t st) {
  CUtensorMap a[4], b[2];
  GluPlan plan;
  const int pairs = std::min(sms / 2, kRefPairs);
  const long long segs = (args.n + kSeg - 1) / kSeg;
  plan.segs = args.mask != nullptr && segs <= kMostSegs ? static_cast<int>(segs) : 0;
  const int n_m = static_cast<int>((args.n + kTileM - 1) / kTileM);
  const int width = MODE == kDx ? args.d : args.f, depth = MODE == kDx ? args.f : args.d;
  plan.half = (depth + kBK - 1) / kBK;
  const int stages = MODE == kDx ? 2 * plan.half : plan.half;
  plan.work = {};
  if (MODE == kDx && args.partials != nullptr) {
    // Tiles that fill no round, or the last one badly, are cut along their long sum.
    // Segments are not listed then (masked rows are zeros already, and few).
    plan.work = dx_plan(args.n, args.f, args.d, pairs);
    if (plan.work.cut > 0 && plan.segs > 0 && plan.work.whole > 0) plan.work.cut = 0;
  }
  if (plan.work.cut > 0) {
    plan.cols = kTileN;
    plan.segs = 0;
  } else {
    plan.cols = tile_columns(n_m, width, MODE == kDx ? kTileN : 128, pairs);
    plan.work = {};
    plan.work.n_m = n_m;
    plan.work.n_n = (width + plan.cols - 1) / plan.cols;
    plan.work.kt = stages;
    plan.work.whole = n_m * plan.work.n_n;
  }
  plan.work.group = kGluGroup;
  // The first operand's rows by 128 and by segments; the weights' by columns of f.
  const void* first[2] = {MODE == kDx ? args.gate : args.x, MODE == kDx ? args.up : args.x};
  const long long ld[2] = {MODE == kDx ? args.ldg : args.ldx, MODE == kDx ? args.ldu : args.ldx};
  const uint32_t b_rows = MODE == kDx ? kBK : static_cast<uint32_t>(plan.cols);
  for (int i = 0; i < 2; ++i) {
    if (MODE != kDx && i == 1) {
      a[1] = a[0];
      a[3] = a[2];
      continue;
    }
    if (!map16(&a[i], first[i], depth, args.n, ld[i], 128)) return cudaErrorInvalidValue;
    a[2 + i] = a[i];
    if (plan.segs > 0 && !map16(&a[2 + i], first[i], depth, args.n, ld[i], kSeg))
      return cudaErrorInvalidValue;
  }
  if (!map16(&b[0], args.w_gate, args.d, args.f, args.ldwg, b_rows) ||
      !map16(&b[1], args.w_up, args.d, args.f, args.ldwu, b_rows))
    return cudaErrorInvalidValue;
  // What leaves: dx; or h, gate and up; or dgate, dup and h.
  CUtensorMap o[3];
  void* const out[3] = {MODE == kDx ? args.dx : MODE == kFwd ? args.h : args.gate,
                        MODE == kFwd ? args.gate : args.up, MODE == kFwd ? args.up : args.h};
  const long long ldo[3] = {MODE == kDx ? args.lddx : MODE == kFwd ? args.ldh : args.ldg,
                            MODE == kFwd ? args.ldg : args.ldu, MODE == kFwd ? args.ldu : args.ldh};
  for (int i = 0; i < 3; ++i) {
    if (i > 0 && (MODE == kDx || out[i] == nullptr))
      o[i] = o[0];
    else if (!encode_map_2d(&o[i], out[i], static_cast<uint64_t>(width),
                            static_cast<uint64_t>(args.n), static_cast<uint64_t>(ldo[i]) * 2, 32,
                            kSeg, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
  }
  auto run = [&](auto type) {
    using T = decltype(type);
    return stages > kSumStages ? launch<MODE, T, true>(a, b, o, args, plan, sms, st)
                                  : launch<MODE, T, false>(a, b, o, args, plan, sms, st);
  };
  return args.fp16 ? run(__half()) : run(__nv_bfloat16());
}

// ---------------------------------------- from the projections as kept ----

constexpr int kRowThreads = 256;

// dgate = dh u act'(g), dup = dh act(g), h = act(g) u: memory bound, 8 values of a
// row a thread. 4096 x 14336: 90 us, 6.5 TB/s, with 32 CTAs an SM, four rounds of them
// (110 with 8, which all run at once, 101 with a thread for each 8 values).
template <typename T>
__global__ void __launch_bounds__(kRowThreads) glu_bwd_kept_kernel(const GluArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // Steps of all threads' groups of 8; the place moves on without a division.
  const int per_row = a.f / 8;
  const long long step = static_cast<long long>(gridDim.x) * kRowThreads;
  const long long rows = step / per_row;
  const int more = static_cast<int>(step - rows * per_row);
  const long long first = static_cast<long long>(blockIdx.x) * kRowThreads + threadIdx.x;
  long long row = first / per_row;
  int group = static_cast<int>(first - row * per_row);
  for (; row < a.n; row += rows, group += more) {
    if (group >= per_row) {
      group -= per_row;
      if (++row >= a.n) break;
    }
    const int col = group * 8;
    const bool live = a.mask == nullptr || a.mask[row] != 0;
    uint4 d = make_uint4(0, 0, 0, 0), g = d, u = d;
    if (live) {
      d = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.dh) + row * a.lddh + col);
      g = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.gate_in) + row * a.ldgi + col);
      u = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.up_in) + row * a.ldui + col);
    }
    const uint32_t dw[4] = {d.x, d.y, d.z, d.w}, gw[4] = {g.x, g.y, g.z, g.w},
                   uw[4] = {u.x, u.y, u.z, u.w};
    uint32_t og[4], ou[4], oh[4];
    with_act(a.act, [&](auto tag) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float d0, d1, g0, g1, u0, u1, s0, s1;
        unpack16<T>(dw[j], d0, d1);
        unpack16<T>(gw[j], g0, g1);
        unpack16<T>(uw[j], u0, u1);
        const float a0 = activate<decltype(tag)::value, true>(g0, s0);
        const float a1 = activate<decltype(tag)::value, true>(g1, s1);
        og[j] = pack16<T>(d0 * u0 * s0, d1 * u1 * s1);
        ou[j] = pack16<T>(d0 * a0, d1 * a1);
        oh[j] = pack16<T>(a0 * u0, a1 * u1);
      }
    });
    st_global_v4(static_cast<T*>(a.gate) + row * a.ldg + col, og[0], og[1], og[2], og[3]);
    st_global_v4(static_cast<T*>(a.up) + row * a.ldu + col, ou[0], ou[1], ou[2], ou[3]);
    if (a.h != nullptr)
      st_global_v4(static_cast<T*>(a.h) + row * a.ldh + col, oh[0], oh[1], oh[2], oh[3]);
  }
}

}  // namespace

template <int MODE, typename T>
cudaError_t prepare() {
  cudaError_t e = cudaSuccess;
  for (const void* k : {reinterpret_cast<const void*>(glu_gemm_kernel<MODE, T, false>),
                        reinterpret_cast<const void*>(glu_gemm_kernel<MODE, T, true>)})
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  return e;
}

cudaError_t prepare_glu_gemm() {
  for (const auto f : {prepare<kFwd, __nv_bfloat16>, prepare<kFwd, __half>,
                       prepare<kAgain, __nv_bfloat16>, prepare<kAgain, __half>,
                       prepare<kDx, __nv_bfloat16>, prepare<kDx, __half>}) {
    const cudaError_t e = f();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

size_t glu_dx_workspace(long long n, int f, int d) {
  if (n == 0 || dx_plan(n, f, d, kRefPairs).cut == 0) return 0;
  return 2 * kRefPairs * kSlotFloats * sizeof(float);
}

cudaError_t launch_glu_fwd(const GluArgs& a, int sms, cudaStream_t st) {
  return launch_mode<kFwd>(a, sms, st);
}
cudaError_t launch_glu_bwd_again(const GluArgs& a, int sms, cudaStream_t st) {
  return launch_mode<kAgain>(a, sms, st);
}
cudaError_t launch_glu_dx(const GluArgs& a, int sms, cudaStream_t st) {
  return launch_mode<kDx>(a, sms, st);
}

cudaError_t launch_glu_bwd_kept(const GluArgs& a, int sms, cudaStream_t st) {
  const long long all = a.n * (a.f / 8);
  const unsigned grid = static_cast<unsigned>(
      std::min<long long>((all + kRowThreads - 1) / kRowThreads, 32LL * sms));
  LaunchTimer timer("glu_bwd_kept_kernel", st);
  if (a.fp16)
    glu_bwd_kept_kernel<__half><<<grid, kRowThreads, 0, st>>>(a);
  else
    glu_bwd_kept_kernel<__nv_bfloat16><<<grid, kRowThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace grpo
