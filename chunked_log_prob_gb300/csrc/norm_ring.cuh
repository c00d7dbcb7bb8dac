// What the norms' forward and backward kernels share: the ring of rows in
// shared memory and the shapes of their launches.
#pragma once

#include <algorithm>

#include "kernel_fit.h"
#include "launch.h"
#include "norm.h"
#include "row_ops.cuh"

namespace grpo {
namespace {

constexpr int kRowThreads = 256;  // threads of a CTA whose rows are short

__device__ __forceinline__ bool row_live(const uint8_t* mask, long long row, long long n) {
  return row < n && (mask == nullptr || mask[row] != 0);
}

// Each row of the CTA (threadIdx.y) has a ring of `slots` rows in shared memory,
// filled by bulk copies; a slot is filled again as soon as the row's sum has
// been taken, when every thread holds its values. Bulk copies start and end on
// 16 bytes: of a row that does not, the 16 bytes around its ends come too, and
// its values are read one by one (VEC false).
// The bytes in flight come from the ring, so what is left is issue slots: a
// thread holds up to 32 values, so that a row's fixed work (barriers, sums,
// addresses) is shared by few warps, and works on pairs of them.
struct Ring {
  int slots;           // rows in flight for each row of the CTA
  uint32_t row_bytes;  // of a slot
  int part;            // backward, two CTAs to a row: columns of the first
};

// Shared memory: barriers, then the parameters as fp32, then the rings.
constexpr int kMaxSlots = 8;
constexpr int kMaxRows = 8;  // rows of a CTA
constexpr uint32_t kRingBars = kMaxRows * kMaxSlots * sizeof(uint64_t);

// Threads of a CTA at most.
constexpr int kRingThreads = 512;

// After a timeout: lets the copies still in flight land (within the same limit).
__device__ __forceinline__ void land(uint64_t* bars, int slots, uint32_t parity, uint32_t pending) {
  for (int s = 0; s < slots; ++s)
    if ((pending >> s) & 1u) row_wait(&bars[s], (parity >> s) & 1u);
}

// Two sums into the peer CTA's shared memory, counted on its barrier there.
// `at`, `bar`: addresses in this CTA of what is meant in the peer's.
__device__ __forceinline__ void send_sums(uint32_t at, uint32_t bar, uint32_t peer, float a,
                                          float b) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%2, %3}, [%1];" ::"r"(
          mapa_shared(at, peer)),
      "r"(mapa_shared(bar, peer)), "f"(a), "f"(b)
      : "memory");
}

__device__ __forceinline__ int param_width(int type) { return type == GRPO_DTYPE_FP32 ? 4 : 2; }

// Rows of the group that begins at `row`.
__device__ __forceinline__ int row_count(long long row, long long n, long long step) {
  return row < n ? static_cast<int>((n - 1 - row) / step) + 1 : 0;
}

// How many of them are fetched: up to the self-test's lost row.
__device__ __forceinline__ int fetch_count(int count, long long row0, long long step,
                                           uint32_t lost) {
  if (lost == kNoneLost) return count;
  const long long past = static_cast<long long>(lost) - row0;
  return past >= 0 && past % step == 0 && past / step < count ? static_cast<int>(past / step)
                                                              : count;
}

// Threads of a row and rows of a CTA for D columns held in registers.
struct RowShape {
  int tpr, rows, ch;
};
// The most values a thread, up to 8 `most`, that leave no more than a
// tenth of the threads idle (else the fewest idle ones); CTAs of about
// `threads` threads.
RowShape ring_shape(int d, int most, int threads) {
  RowShape best = {0, 0, 0};
  int best_room = 0;
  for (int ch = most; ch >= 1; --ch) {
    const int tpr = (d + 256 * ch - 1) / (256 * ch) * 32;
    const int room = tpr * 8 * ch;
    if (tpr > kRingThreads || (best.ch != 0 && room >= best_room)) continue;
    best = {tpr, std::min(kMaxRows, std::max(1, threads / tpr)), ch};
    best_room = room;
    if (10 * room <= 11 * d) break;
  }
  return best;
}

constexpr size_t kSmemMax = 227 * 1024 - 22528;  // less the kernels' static arrays
constexpr size_t kSmemTarget = 72 * 1024;       // of a CTA: three to an SM

// Rows in flight of a CTA: as many slots as fit kSmemTarget beside the
// parameters, at most kMaxSlots and at least 2 (1 for rows that fit but once).
Ring make_ring(uint32_t row_bytes, int rows, size_t fixed) {
  const size_t slot = static_cast<size_t>(row_bytes) * rows;
  const size_t room = kSmemTarget > fixed ? kSmemTarget - fixed : 0;
  size_t slots = std::min<size_t>(kMaxSlots, std::max<size_t>(2, room / slot));
  if (fixed + slots * slot > kSmemMax) slots = 1;
  Ring r;
  r.slots = static_cast<int>(slots);
  r.row_bytes = row_bytes;
  r.part = 0;
  return r;
}

// CTAs of a kernel that fit an SM of the current device, which is opted in to
// large shared memory for it first. What was found is kept for each device.
template <auto Kernel>
cudaError_t ctas_per_sm(int threads, size_t smem, int* n) {
  static KernelFit fit;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess || fit.find(device, threads, smem, n)) return e;
  if (!fit.opted_in(device)) {
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmemMax));
    if (e != cudaSuccess) return e;
    fit.set_opted_in(device);
  }
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, Kernel, threads, smem);
  if (e == cudaSuccess) fit.keep(device, threads, smem, *n);
  return e;
}

}  // namespace
}  // namespace grpo
