// Weight gradient of a linear layer from the 8-bit checkpoint of its input:
//   dW[o][i] = add[o][i] + sum_t dY[t][o] X[t][i],  X = q 2^k.
//
// A tcgen05 GEMM over the tokens, both operands MN-major (a token's row holds
// 64 outputs or inputs in 128 bytes). X never exists in memory: its e4m3 tiles
// arrive by TMA, converter warps widen them on chip to bf16 - exactly,
// since 2^k is a power of two and e4m3 has 4 significant bits - into the
// 128-byte-swizzled layout that a bf16 TMA load would have left, and the tensor
// cores read them from there. Against expanding X first (16384 x 4096: 69 MB
// read, 134 MB written, 134 MB read again) the operand costs 1.03 bytes a value.
//
// A CTA pair computes 256 outputs x 256 inputs. The tensor core's fp32 sums cut
// off instead of rounding, which bends a long sum towards zero in proportion to
// its length (measured against fp64: 3.1e-6 at 5541 tokens, 1.1e-5 at 16384), so
// TMEM holds the sum of kSegment stages at a time (two buffers in turn), and the
// epilogue warps add each to the tile's running sum in their registers, rounded
// (4.2e-7 at 16384 tokens).
//
// 16384 x 4096 x 4096: 322 us, 1707 TFLOP/s (0.89 of cuBLAS's measured burst), 353
// to 368 us in a row under the power cap. Bound by the tensor cores and, close behind,
// by the widening (a stage of 64 tokens takes the former 512 cycles, measured
// about 640).
#include <algorithm>
#include <cstring>

#include "launch.h"
#include "norm.h"
#include "row_ops.cuh"
#include "wgrad_plan.h"

namespace grpo {
namespace {

// Rings: a slot's way round (barrier to barrier, TMA or widening, the MMAs)
// takes several stages' MMA time, so each of them is as deep as memory allows.
constexpr int kDy = 5;             // dY tiles
constexpr int kX = 4;              // widened X tiles
constexpr int kRaw = 6;            // e4m3 tiles with their exponents
// The converters' two groups take turns with the stages. A slot must stay with
// one of them: a group that waits for a phase of its barrier has then seen the
// phase before (a parity alone cannot tell that one apart from the one after).
static_assert(kRaw % 2 == 0, "a raw slot belongs to one converter group");
constexpr int kBoxBytes = kTok * 128;      // 64 tokens x 64 bf16 columns
constexpr int kOperand = 2 * kBoxBytes;    // a CTA's 128 outputs, or 128 inputs
constexpr int kRawQ = kTok * 128;          // 64 tokens x 128 e4m3
constexpr int kRawBytes = kRawQ + kTok * 16;  // and 16 exponents, ours among them
constexpr int kStoreBuf = 32 * 64;         // 32 x 16 fp32 on its way out
constexpr int kSegment = 16;       // stages summed in TMEM: 1024 tokens
// Warps: 0 dY by TMA, 1 MMA, 2 the checkpoint by TMA, 3 idle, then two
// warpgroups that hold the sums and four that widen. The latter work in two
// halves that take turns with the stages: widening is short dependent chains
// between barriers, so it wants many warps (16384 x 4096 x 4096: 397 us with
// eight of them, 372 with sixteen).
constexpr int kEpilogueWarps = 8, kConvertWarps = 16;
constexpr int kConvertGroup = 8;  // warps that share a stage
constexpr int kFirstEpilogue = 4, kFirstConvert = kFirstEpilogue + kEpilogueWarps;
constexpr int kThreads = 32 * (kFirstConvert + kConvertWarps);
// Registers of a thread: 72 at launch (896 x 72 = 64512), moved to the epilogue,
// whose threads hold 128 sums: 128 x 24 + 256 x 144 + 512 x 48 = 64512.
constexpr int kLaunchRegs = 72, kControlRegs = 24, kEpilogueRegs = 144, kConvertRegs = 48;
static_assert(128 * kControlRegs + 32 * kEpilogueWarps * kEpilogueRegs +
                      32 * kConvertWarps * kConvertRegs <=
                  kThreads * kLaunchRegs,
              "registers of a CTA");
constexpr int kSmem = 1024 + (kDy + kX) * kOperand + kRaw * kRawBytes +
                      kEpilogueWarps * kStoreBuf;
constexpr uint32_t kTmemCols = 512;
static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
constexpr int kSlotFloats = kTileM * kTileN;

__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > kWaitLimitCycles) return;
}

// A warp's wait: one answer for all lanes, before steps of the whole warp. Each
// polls for itself, and one may give up (or see the abort flag) as another finds
// the phase done.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                          int* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status)) != 0;
}

// True in one lane of the (whole) warp. The compiler then knows that one thread
// runs what follows and feeds tcgen05 and TMA their uniform operands directly;
// behind `lane == 0` it cannot, and a stage took its issuing thread twice as
// long as the tensor core (16384 x 4096 x 4096: 518 us against 407).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "elect.sync _|P, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, P;\n\t}"
      : "=r"(p));
  return p != 0;
}

template <int N>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Twice 16 e4m3 of one block each, with their exponent bytes, to bf16, exactly.
// Where both 2^k are fp16 (k in [-24, 15], or all values 0: the usual
// activations), a value costs one mixed multiply-add of two fp16 into fp32.
__device__ __forceinline__ void widen32(const uint4 (&w)[2], const uint32_t (&e)[2],
                                        uint32_t (&o)[2][8]) {
  uint16_t f16[2];
  bool small = e[0] - 103u <= 39u && e[1] - 103u <= 39u;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    asm("cvt.rn.f16.f32 %0, %1;" : "=h"(f16[h]) : "f"(__uint_as_float(e[h] << 23)));
  if (!small) {
    small = true;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (e[h] - 103u <= 39u) continue;
      f16[h] = 0;
      small = small && (w[h].x | w[h].y | w[h].z | w[h].w) == 0u;
    }
  }
  if (small) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t in[4] = {w[h].x, w[h].y, w[h].z, w[h].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float lo, hi;
        asm("{\n\t.reg .b32 t;\n\t.reg .b16 l, h;\n\t"
            "cvt.rn.f16x2.e4m3x2 t, %2;\n\t"
            "mov.b32 {l, h}, t;\n\t"
            "fma.rn.f32.f16 %0, l, %3, %4;\n\t"
            "fma.rn.f32.f16 %1, h, %3, %4;\n\t}"
            : "=f"(lo), "=f"(hi)
            : "h"(static_cast<uint16_t>(in[j >> 1] >> (16 * (j & 1)))), "h"(f16[h]), "f"(0.f));
        o[h][j] = pack_bf16x2(lo, hi);
      }
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t in[4] = {w[h].x, w[h].y, w[h].z, w[h].w};
      const float f = ckpt_factor(e[h]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 v = unpack_e4m3x2(in[j >> 1] >> (16 * (j & 1)));
        o[h][j] = pack_bf16x2(v.x * f, v.y * f);
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    ckpt_wgrad_kernel(const __grid_constant__ CUtensorMap map_dy,
                      const __grid_constant__ CUtensorMap map_q,
                      const __grid_constant__ CUtensorMap map_ex,
                      const __grid_constant__ CUtensorMap map_dw, const WgradArgs args,
                      const WgradPlan plan) {
  extern __shared__ uint8_t smem_raw[];
  // By stage, in turns of kDy. The X ring is shorter: a converter waits for the
  // MMAs of the stage kX before its own, whose barrier cannot go round again
  // before that stage's X tile is there.
  __shared__ __align__(8) uint64_t full_bar[kDy];  // leader: both CTAs' dY and X tiles are there
  __shared__ __align__(8) uint64_t done_bar[kDy];  // the stage's MMAs are done
  __shared__ __align__(8) uint64_t raw_full[kRaw];   // this CTA's e4m3 tile landed
  __shared__ __align__(8) uint64_t raw_empty[kRaw];  // its converter warps have read it
  __shared__ __align__(8) uint64_t tfull_bar[2], tempty_bar[2];
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;

  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* const ring = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* const xring = ring + kDy * kOperand;
  uint8_t* const raw = xring + kX * kOperand;
  uint8_t* const out = raw + kRaw * kRawBytes;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(blockIdx.x) / 2, pairs = static_cast<int>(gridDim.x) / 2;
  volatile int* abort_flag = &abort_sh;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    // The status word of this call. Nothing writes it before a wait runs out.
    if (blockIdx.x == 0) *args.status = GRPO_OK;
    for (int s = 0; s < kDy; ++s) {
      mbar_init(&full_bar[s], 2 + 2 * kConvertGroup);  // dY's TMA threads, converter warps
      mbar_init(&done_bar[s], 1);
    }
    for (int s = 0; s < kRaw; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], kConvertGroup);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], 2 * kEpilogueWarps);  // both CTAs' epilogue warps
    }
    mbar_init(&drain_bar, 1);
    abort_sh = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&map_dy);
    tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_ex);
    tma_prefetch_desc(&map_dw);
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

  // Each role moves its registers inside its own branch: the compiler holds what
  // follows to the new count only where the instruction dominates it.
  if (warp < kFirstEpilogue) {
    give_registers<kControlRegs>();
    // One lane of each role walks through the work, waits and issues; the others
    // are at the warp barrier before the closing cluster barrier. (No step inside
    // is the whole warp's: lanes that waited each for itself could part at a wait
    // that runs out, and the two halves then wait for each other without end.)
    if (warp == 0) {
      // -------------------------------------------------- dY's tiles by TMA --
      if (elect_one()) {
        uint32_t n = 0;  // stages issued
        while (ok && work.next(plan, pair, pairs, it)) {
          int tm, tn;
          tile_place(plan, it.tile, tm, tn);
          const int o0 = tm * kTileM + static_cast<int>(rank) * (kTileM / 2);
          for (int k = it.kb; k < it.ke; ++k, ++n) {
            const uint32_t s = n % kDy;
            if (!mbar_wait(&done_bar[s], ((n / kDy) & 1u) ^ 1u, abort_flag, args.status)) {
              ok = false;
              break;
            }
            const uint32_t lead = mapa_shared(smem_u32(&full_bar[s]), 0);
            mbar_arrive_expect_tx_cluster(lead, kOperand);
            uint8_t* a = ring + s * kOperand;
            tma_load_2d_pair_nohint(a, &map_dy, lead, o0, k * kTok);
            tma_load_2d_pair_nohint(a + kBoxBytes, &map_dy, lead, o0 + 64, k * kTok);
          }
        }
        // After a timeout: let the copies in flight land before the CTA exits (the
        // peer passes the closing cluster barrier only after this). Their barriers
        // also wait for converters that may have given up: the drain ends by its
        // own limit then, long after any copy.
        if (!ok && rank == 0)
          for (uint32_t j = n >= kDy ? n - kDy : 0; j < n; ++j)
            drain(&full_bar[j % kDy], (j / kDy) & 1u);
      }
    } else if (warp == 2) {
      // -------------------------------------------- checkpoint tiles by TMA --
      if (elect_one()) {
        uint32_t n = 0;
        while (ok && work.next(plan, pair, pairs, it)) {
          int tm, tn;
          tile_place(plan, it.tile, tm, tn);
          const int i0 = tn * kTileN + static_cast<int>(rank) * (tile_cols(args.in, tn) / 2);
          // Exponents come 16 at a time (a TMA copy starts on 16 bytes).
          const int x0 = (i0 / kCkptBlock) & ~15;
          for (int k = it.kb; k < it.ke; ++k, ++n) {
            const uint32_t r = n % kRaw;
            if (!mbar_wait(&raw_empty[r], ((n / kRaw) & 1u) ^ 1u, abort_flag, args.status)) {
              ok = false;
              break;
            }
            if (n == args.lost && blockIdx.x == 0) continue;
            mbar_arrive_expect_tx(&raw_full[r], kRawBytes);
            tma_load_2d(raw + r * kRawBytes, &map_q, &raw_full[r], i0, k * kTok);
            tma_load_2d(raw + r * kRawBytes + kRawQ, &map_ex, &raw_full[r], x0, k * kTok);
          }
        }
        if (!ok)
          for (uint32_t j = n >= kRaw ? n - kRaw : 0; j < n; ++j)
            drain(&raw_full[j % kRaw], (j / kRaw) & 1u);
      }
    } else if (warp == 1 && rank == 0) {
      // ------------------------------------------------------ MMA issuer --
      if (elect_one()) {
        uint32_t n = 0, seg = 0;  // stages, segments issued
        while (ok && work.next(plan, pair, pairs, it)) {
          int tm, tn;
          tile_place(plan, it.tile, tm, tn);
          const uint32_t idesc = idesc_bf16(kTileM, tile_cols(args.in, tn), true, true);
          for (int k = it.kb; k < it.ke; ++k, ++n) {
            const bool first = (k - it.kb) % kSegment == 0;
            const bool last = (k - it.kb) % kSegment == kSegment - 1 || k == it.ke - 1;
            const uint32_t buf = seg & 1u;
            if (first &&
                !mbar_wait(&tempty_bar[buf], ((seg >> 1) & 1u) ^ 1u, abort_flag, args.status)) {
              ok = false;
              break;
            }
            const uint32_t sa = n % kDy;
            if (!mbar_wait(&full_bar[sa], (n / kDy) & 1u, abort_flag, args.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t d = tmem_base + buf * kTileN;
            const uint32_t a = smem_u32(ring + sa * kOperand);
            const uint32_t b = smem_u32(xring + n % kX * kOperand);
#pragma unroll
            for (int kk = 0; kk < kTok / 16; ++kk)
              // 64-wide blocks of outputs or inputs 8 KB apart, 8 tokens 1 KB.
              tc_mma_bf16_pair(d, sdesc_sw128(a + kk * 2048, kBoxBytes, 1024),
                               sdesc_sw128(b + kk * 2048, kBoxBytes, 1024), idesc,
                               first && kk == 0 ? 0u : 1u);
            tc_commit_pair_multicast(&done_bar[sa], 0x3);
            if (last) tc_commit_pair_multicast(&tfull_bar[buf], 0x3);
            seg += last ? 1 : 0;
          }
        }
        tc_commit_pair(&drain_bar);
        drain(&drain_bar, 0);
      }
    }
  } else if (warp >= kFirstConvert) {
    // -------------------------------------------------------- converters --
    give_registers<kConvertRegs>();
    // A thread widens 16 columns of two tokens, 32 apart, of every second stage:
    // piece c of the 64 columns of one box. Eight lanes that load or store at
    // once take 4 pieces of the rows rho and rho ^ 5 of 8: the 128-byte swizzle
    // (raw tile: piece c at c ^ row; X tile: pieces 2c and 2c + 1 at theirs ^
    // row) puts them in eight different banks both times.
    const int wid = warp - kFirstConvert;
    const uint32_t group = wid / kConvertGroup;
    const int box = wid & 1;
    const int c = lane & 3;
    const int row = ((wid & (kConvertGroup - 1)) >> 1) * 8 +
                    ((lane >> 3) ^ (((lane >> 2) & 1) * 5));
    const uint32_t src0 = smem_u32(raw) + row * 128 + (((box * 4 + c) ^ (row & 7)) << 4);
    const uint32_t exp0 = smem_u32(raw) + kRawQ + row * 16 + box * 2 + (c >> 1);
    const uint32_t dst0 =
        smem_u32(xring) + box * kBoxBytes + row * 128 + (((2 * c) ^ (row & 7)) << 4);
    const uint32_t full0 = mapa_shared(smem_u32(&full_bar[0]), 0);
    // Ring positions of stage n, and of stage n - kX in the ring of done_bar.
    uint32_t n = 0, r = group, r_par = 0, f = group;
    uint32_t d = 2 * kDy - kX + group, d_par = 1;
    while (d >= kDy) d -= kDy;
    while (__all_sync(0xffffffffu, ok) && work.next(plan, pair, pairs, it)) {
      int tm, tn;
      tile_place(plan, it.tile, tm, tn);
      const int i0 = tn * kTileN + static_cast<int>(rank) * (tile_cols(args.in, tn) / 2);
      const uint32_t ex = exp0 + ((i0 / kCkptBlock) & 15);  // our exponent of the 16
      const uint32_t n_end = n + (it.ke - it.kb);
      // A lane whose wait ran out stays with its warp up to the tile's end (no
      // vote on the way: 1 to 3 % of the whole): it waits no more, what it stores
      // is not its values, and its CTA's abort flag is up.
      for (uint32_t m = n + ((n ^ group) & 1u); m < n_end; m += 2) {
        ok = ok && mbar_wait(&raw_full[r], r_par, abort_flag, args.status);
        uint4 w[2];
        uint32_t e[2], o[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          w[h] = lds_v4(src0 + r * kRawBytes + h * 32 * 128);
          e[h] = lds_u8(ex + r * kRawBytes + h * 32 * 16);
        }
        widen32(w, e, o);
        // Widened before the slot is waited for: only the stores, the fence and
        // the barriers lie on the slot's way round.
        if (m >= kX) ok = ok && mbar_wait(&done_bar[d], d_par, abort_flag, args.status);
        const uint32_t dst = dst0 + (m % kX) * kOperand;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          sts_v4(dst + h * 32 * 128, o[h][0], o[h][1], o[h][2], o[h][3]);
          sts_v4((dst + h * 32 * 128) ^ 16u, o[h][4], o[h][5], o[h][6], o[h][7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && ok) {
          mbar_arrive(&raw_empty[r]);
          mbar_arrive_cluster(full0 + f * 8u);
        }
        if ((r += 2) >= kRaw) {
          r -= kRaw;
          r_par ^= 1u;
        }
        if ((f += 2) >= kDy) f -= kDy;
        if ((d += 2) >= kDy) {
          d -= kDy;
          d_par ^= 1u;
        }
      }
      n = n_end;
    }
  } else {
    // ---------------------------------------------------------- epilogue --
    // A thread holds one output's sums over half of the tile's inputs.
    take_registers<kEpilogueRegs>();
    const int q = warp & 3;  // TMEM lane quarter of this warp
    const int half = (warp - kFirstEpilogue) >> 2;
    const uint32_t tempty0 = mapa_shared(smem_u32(&tempty_bar[0]), 0);
    uint8_t* const stage = out + (warp - kFirstEpilogue) * kStoreBuf;
    const uint32_t t0 =
        tmem_base + (static_cast<uint32_t>(q * 32) << 16) + half * (kTileN / 2);
    uint32_t seg = 0;
    const uint32_t peer_abort = mapa_shared(smem_u32(&abort_sh), rank ^ 1u);
    while (ok && work.next(plan, pair, pairs, it)) {
      int tm, tn;
      tile_place(plan, it.tile, tm, tn);
      float sum[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 32; ++j) sum[c][j] = 0.f;
      // Where a wait of either CTA ran out, X may hold what a converter lane did
      // not widen; its CTA's abort flag was up before that stage reached the
      // tensor core.
      uint32_t gave_up = 0;
      for (int k = it.kb; k < it.ke; k += kSegment, ++seg) {
        const uint32_t buf = seg & 1u;
        if (!warp_wait(&tfull_bar[buf], (seg >> 1) & 1u, abort_flag, args.status)) {
          ok = false;
          break;
        }
        if (k + kSegment >= it.ke)
          gave_up = static_cast<uint32_t>(*abort_flag) | ld_cluster_u32(peer_abort);
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
      if (__any_sync(0xffffffffu, !ok || gave_up != 0)) {
        ok = false;
        break;
      }
      const int lrow = static_cast<int>(rank) * 128 + q * 32 + lane;  // row of the tile
      const int row0 = tm * kTileM + static_cast<int>(rank) * 128 + q * 32;
      const int row = row0 + lane;
      if (row0 >= args.out) continue;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int cb = half * 4 + c;
        const int i0 = tn * kTileN + cb * 32;
        if (i0 >= args.in) break;
        if (it.slot >= 0) {
          float* p = args.partials + static_cast<long long>(it.slot) * kSlotFloats +
                     (cb * 8 * kTileM + lrow) * 4;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            st_global_v4(p + j * kTileM * 4, __float_as_uint(sum[c][4 * j]),
                         __float_as_uint(sum[c][4 * j + 1]), __float_as_uint(sum[c][4 * j + 2]),
                         __float_as_uint(sum[c][4 * j + 3]));
          continue;
        }
        if (args.add != nullptr && row < args.out) {
          const float* a = args.add + row * args.ldadd + i0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (i0 + 4 * j >= args.in) break;
            const float4 x = *reinterpret_cast<const float4*>(a + 4 * j);
            sum[c][4 * j] += x.x;
            sum[c][4 * j + 1] += x.y;
            sum[c][4 * j + 2] += x.z;
            sum[c][4 * j + 3] += x.w;
          }
        }
        // Two boxes of 16 inputs, through the 64-byte swizzle.
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (i0 + 16 * h >= args.in) break;
          if (lane == 0) bulk_wait_group_read<0>();  // the last box has been read
          __syncwarp();
          uint4* srow = reinterpret_cast<uint4*>(stage + lane * 64);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float* v = &sum[c][16 * h + 4 * j];
            srow[j ^ ((lane >> 1) & 3)] =
                make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                           __float_as_uint(v[3]));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&map_dw, stage, i0 + 16 * h, row0);
            bulk_commit_group();
          }
        }
      }
    }
    // A tile, or a piece of one, is whole or NaN: so are this one and the rest.
    if (!ok) {
      do {
        int tm, tn;
        tile_place(plan, it.tile, tm, tn);
        const int lrow = static_cast<int>(rank) * 128 + q * 32 + lane;
        const int row = tm * kTileM + lrow;
#pragma unroll 1
        for (int c4 = half * 32; c4 < half * 32 + 32; ++c4) {
          const int i0 = tn * kTileN + 4 * c4;
          float* p = it.slot >= 0
                         ? args.partials + static_cast<long long>(it.slot) * kSlotFloats +
                               (c4 * kTileM + lrow) * 4
                     : row < args.out && i0 < args.in ? args.dw + row * args.lddw + i0
                                                      : nullptr;
          if (p != nullptr) st_global_v4(p, 0x7fc00000u, 0x7fc00000u, 0x7fc00000u, 0x7fc00000u);
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

// dW of the cut tiles: the sum of each tile's pieces, and `add`. A CTA takes 16
// columns and 256 / G rows of a tile; thread (row, g) adds the pieces g, g + G, ...
// in their order, and the G sums are then added in theirs: always the same order,
// so the result does not change from call to call. G = 8 where a tile may have
// more than 4 pieces, which one thread would wait for in a row. Whole calls, tokens
// x out x in, with G = 1 and with G = 8: 32768 x 256 x 512 59 and 27 us, 4096 x 256 x
// 256 20 and 17, 2000 x 512 x 512 (5 pieces) 19.1 and 17.1; but 8192 x 1536 x 1536
// (36 tiles of up to 4 pieces, most of the 8 threads idle) 48 and 53.
template <int G>
__global__ void __launch_bounds__(kTileM) ckpt_wgrad_join_kernel(const WgradArgs args,
                                                                 const WgradPlan plan) {
  constexpr int kRows = kTileM / G;
  __shared__ float4 part[G > 1 ? G : 1][G > 1 ? 4 : 1][G > 1 ? kRows : 1];
  const int t = static_cast<int>(blockIdx.x);
  const int qa = first_piece(plan, t), qb = last_piece(plan, t);
  int tm, tn;
  tile_place(plan, plan.whole + t, tm, tn);
  const int r = static_cast<int>(threadIdx.x) % kRows, g = static_cast<int>(threadIdx.x) / kRows;
  const int lrow = static_cast<int>(blockIdx.z) * kRows + r;
  const int row = tm * kTileM + lrow;
  const int c0 = static_cast<int>(blockIdx.y) * 16;  // column of the tile
  const int i0 = tn * kTileN + c0;
  const bool valid = row < args.out && i0 < args.in;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the pieces are there
  float4 v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (valid) {
#pragma unroll 4
    for (int q = qa + g; q <= qb; q += G) {
      const int slot = piece_slot(plan, t, q);
      const float* p = args.partials + static_cast<long long>(slot) * kSlotFloats +
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
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (i0 + 4 * j >= args.in) break;
    if (args.add != nullptr) {
      const float4 x = *reinterpret_cast<const float4*>(args.add + row * args.ldadd + i0 + 4 * j);
      v[j].x += x.x;
      v[j].y += x.y;
      v[j].z += x.z;
      v[j].w += x.w;
    }
    *reinterpret_cast<float4*>(args.dw + row * args.lddw + i0 + 4 * j) = v[j];
  }
}

}  // namespace

size_t ckpt_wgrad_workspace(long long n, int out, int in) {
  return 256 + partial_tiles(n, out, in) * kSlotFloats * sizeof(float);
}

cudaError_t prepare_ckpt_wgrad() {
  return cudaFuncSetAttribute(ckpt_wgrad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kSmem);
}

cudaError_t launch_ckpt_wgrad(const WgradArgs& a, int sms, cudaStream_t st) {
  const int pairs = std::min(sms / 2, kRefPairs);
  CUtensorMap map_dy, map_q, map_ex, map_dw;
  if (!encode_map_2d(&map_dy, a.dy, a.out, a.n, a.lddy * 2, 64, kTok,
                     CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_map_2d(&map_q, a.ck.q, a.in, a.n, a.ck.ldq, 128, kTok, CU_TENSOR_MAP_DATA_TYPE_UINT8,
                     CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_map_2d(&map_ex, a.ck.ex, a.ck.lde, a.n, a.ck.lde, 16, kTok,
                     CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !encode_map_2d(&map_dw, a.dw, a.in, a.out, a.lddw * 4, 16, 32,
                     CU_TENSOR_MAP_DATA_TYPE_FLOAT32, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  const WgradPlan plan = make_plan(a.n, a.out, a.in, pairs);
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
    LaunchTimer timer("ckpt_wgrad_kernel", st);
    e = cudaLaunchKernelEx(&cfg, ckpt_wgrad_kernel, map_dy, map_q, map_ex, map_dw, a, plan);
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
  LaunchTimer timer("ckpt_wgrad_join_kernel", st);
  return groups == 8 ? cudaLaunchKernelEx(&join, ckpt_wgrad_join_kernel<8>, a, plan)
                     : cudaLaunchKernelEx(&join, ckpt_wgrad_join_kernel<1>, a, plan);
}

}  // namespace grpo
