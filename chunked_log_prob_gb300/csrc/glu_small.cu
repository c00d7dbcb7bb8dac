// The gated feed-forward block's forward pass for a few rows (a decoded token, or one
// of each of a group of completions): every weight is read once, and that is all the
// time there is to spend (4096 x 14336: 235 MB, 34.6 us at the measured copy rate; 36.2
// us, 6.49 TB/s, with one row, 36.7 with eight).
//
// A CTA takes 8 columns f of both projections, a warp of it a share of k. One
// mma.sync of 16 x 8 x 16 has Wg's rows f to f + 7 as its first eight rows and Wu's as
// its last, up to 8 tokens as its columns, so a thread ends up with both projections
// of the same values. k is dealt out of order, the same way for both operands: a
// thread's 16 bytes of a row are its operands of two instructions, so weights go from
// memory to the tensor core without shared memory or shuffles, and four lanes read 64
// bytes of a row. The warps of a CTA split k, interleaved, and their sums are added in
// shared memory in the order of the warps. (tcgen05 has nothing to give here: its
// least tile is 128 rows, and memory is the bound.)
#include <algorithm>
#include <type_traits>

#include "glu.h"
#include "glu_act.cuh"
#include "launch.h"
#include "wgrad_plan.h"

namespace grpo {
namespace {

constexpr int kBlockK = 64;  // of a warp's step: 128 bytes of a row
// Steps of one sum of the tensor core, which cuts off instead of rounding: 2048 products,
// 1.5e-5 off at most. A warp adds longer ones up with rounding.
constexpr int kSumSteps = 32;

__device__ __forceinline__ uint4 stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <typename T>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same_v<T, __half>)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kMostWarps = 16;
constexpr int kCols = 8;                      // of f, a CTA
constexpr int kSums = 2 * kCols * kGluSmallRows;  // of a warp

// LONG: a warp's share of k is more than one sum (all sizes in that form: 1 to 3 % slower).
template <typename T, bool LONG>
__global__ void __launch_bounds__(32 * kMostWarps) glu_small_kernel(const GluArgs a) {
  __shared__ float part[kMostWarps][2][kCols][kGluSmallRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int r = lane >> 2, c = lane & 3;
  const int f0 = static_cast<int>(blockIdx.x) * kCols;
  const int n = static_cast<int>(a.n);
  const T* const wg = static_cast<const T*>(a.w_gate) + (f0 + r) * a.ldwg + c * 8;
  const T* const wu = static_cast<const T*>(a.w_up) + (f0 + r) * a.ldwu + c * 8;
  const T* const x = static_cast<const T*>(a.x) + r * a.ldx + c * 8;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto add_step = [&](int k0) {
    uint4 g[2], u[2], b[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = k0 + 32 * h;
      const bool in = k + c * 8 < a.d;
      g[h] = in ? stream16(wg + k) : zero;
      u[h] = in ? stream16(wu + k) : zero;
      b[h] = in && r < n ? __ldg(reinterpret_cast<const uint4*>(x + k)) : zero;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mma16<T>(acc, g[h].x, u[h].x, g[h].y, u[h].y, b[h].x, b[h].y);
      mma16<T>(acc, g[h].z, u[h].z, g[h].w, u[h].w, b[h].z, b[h].w);
    }
  };
  if constexpr (LONG) {
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    int k0 = warp * kBlockK;
    while (k0 < a.d) {
      const int end = least(a.d, k0 + kSumSteps * warps * kBlockK);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = 0.f;
#pragma unroll 4
      for (; k0 < end; k0 += warps * kBlockK) add_step(k0);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] += acc[j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = sum[j];
  } else {
#pragma unroll 4
    for (int k0 = warp * kBlockK; k0 < a.d; k0 += warps * kBlockK) add_step(k0);
  }
  *reinterpret_cast<float2*>(&part[warp][0][r][2 * c]) = make_float2(acc[0], acc[1]);
  *reinterpret_cast<float2*>(&part[warp][1][r][2 * c]) = make_float2(acc[2], acc[3]);
  __syncthreads();
  // A thread finishes one value: neighbours take neighbouring columns of a row.
  for (int i = threadIdx.x; i < kCols * n; i += blockDim.x) {
    const int row = i / kCols, col = i % kCols;
    float g = 0.f, u = 0.f, h = 0.f, slope;
    for (int w = 0; w < warps; ++w) {
      g += part[w][0][col][row];
      u += part[w][1][col][row];
    }
    if (a.mask == nullptr || a.mask[row] != 0)
      with_act(a.act,
               [&](auto tag) { h = activate<decltype(tag)::value, false>(g, slope) * u; });
    else
      g = u = 0.f;
    const int f = f0 + col;
    static_cast<T*>(a.h)[row * a.ldh + f] = static_cast<T>(h);
    if (a.gate != nullptr) {
      static_cast<T*>(a.gate)[row * a.ldg + f] = static_cast<T>(g);
      static_cast<T*>(a.up)[row * a.ldu + f] = static_cast<T>(u);
    }
  }
}

template <typename T>
cudaError_t launch(const GluArgs& a, int sms, cudaStream_t st) {
  const int groups = a.f / kCols;
  // As many warps to a CTA as k has steps, but fewer where there are CTAs enough to
  // fill the device. With 4, 8 and 16 (us): 4096 x 14336 (1792 CTAs) 36.2, 36.2, 38.0;
  // 1536 x 8960 (1120) 11.3, 12.5, 13.5; 4096 x 4096 (512) 19.1, 14.0, 15.8; 2880 x
  // 2880 (360) 14.4, 9.4, 8.0.
  const int steps = (a.d + kBlockK - 1) / kBlockK;
  const int most = groups >= 6 * sms ? 4 : groups >= 3 * sms ? 8 : kMostWarps;
  const int warps = std::max(1, std::min(most, steps));
  LaunchTimer timer("glu_small_kernel", st);
  if (a.d > warps * kSumSteps * kBlockK)
    glu_small_kernel<T, true><<<groups, 32 * warps, 0, st>>>(a);
  else
    glu_small_kernel<T, false><<<groups, 32 * warps, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_glu_small(const GluArgs& a, int sms, cudaStream_t st) {
  return a.fp16 ? launch<__half>(a, sms, st) : launch<__nv_bfloat16>(a, sms, st);
}

}  // namespace grpo
