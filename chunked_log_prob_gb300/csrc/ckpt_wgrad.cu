// Weight gradient of a linear layer from the 8-bit checkpoint of its input:
//   dW[o][i] = add[o][i] + sum_t dY[t][o] X[t][i],  X = q 2^k exactly.
#include "launch.h"
#include "norm.h"
#include "row_ops.cuh"

namespace grpo {
namespace {

constexpr int kTile = 64;   // outputs x inputs of a CTA
constexpr int kDepth = 32;  // tokens staged at a time

// 256 threads, 4 x 4 sums each, fp32.
__global__ void __launch_bounds__(256) ckpt_wgrad_kernel(const WgradArgs a) {
  __shared__ float sy[kDepth][kTile + 1], sx[kDepth][kTile + 1];
  const int o0 = blockIdx.y * kTile, i0 = blockIdx.x * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const __nv_bfloat16* dy = static_cast<const __nv_bfloat16*>(a.dy);
  float acc[4][4] = {};
  for (long long t0 = 0; t0 < a.n; t0 += kDepth) {
    for (int e = threadIdx.x; e < kDepth * kTile; e += 256) {
      const int r = e / kTile, c = e % kTile;
      const long long t = t0 + r;
      sy[r][c] = t < a.n && o0 + c < a.out ? to_f32(dy[t * a.lddy + o0 + c]) : 0.f;
      float v = 0.f;
      if (t < a.n && i0 + c < a.in)
        v = unpack_e4m3x2(a.ck.q[t * a.ck.ldq + i0 + c]).x *
            ckpt_factor(a.ck.ex[t * a.ck.lde + (i0 + c) / kCkptBlock]);
      sx[r][c] = v;
    }
    __syncthreads();
#pragma unroll 4
    for (int r = 0; r < kDepth; ++r) {
      float y[4], x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        y[k] = sy[r][ty + 16 * k];
        x[k] = sx[r][tx + 16 * k];
      }
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[p][k] += y[p] * x[k];
    }
    __syncthreads();
  }
#pragma unroll
  for (int p = 0; p < 4; ++p)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int o = o0 + ty + 16 * p, i = i0 + tx + 16 * k;
      if (o >= a.out || i >= a.in) continue;
      const float add = a.add != nullptr ? a.add[o * a.ldadd + i] : 0.f;
      a.dw[o * a.lddw + i] = add + acc[p][k];
    }
}

}  // namespace

cudaError_t launch_ckpt_wgrad(const WgradArgs& a, int sms, cudaStream_t st) {
  (void)sms;
  LaunchTimer timer("ckpt_wgrad_kernel", st);
  ckpt_wgrad_kernel<<<dim3((a.in + kTile - 1) / kTile, (a.out + kTile - 1) / kTile), 256, 0, st>>>(a);
  return cudaGetLastError();
}

size_t ckpt_wgrad_workspace(long long n, int out, int in) {
  (void)n;
  (void)out;
  (void)in;
  return 256;
}

}  // namespace grpo
