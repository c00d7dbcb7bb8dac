// Internal launch interface of the gated feed-forward operators.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "grpo_gb300.h"
#include "norm.h"

namespace grpo {

// Row tiles that the block's GEMMs walk together. 16384 x 4096 x 14336, forward / backward
// again / weight gradients (us, under the power cap, two boxes): 4 2348 / 4829 / 2377, 8
// 2231 / 4667 / 2335, 16 2174 / 4636 / 2325; 16 2118 / 4513 / 2270, 20 2110 / 4579 / 2346,
// 32 2227 / 4751 / 2424. At 8192 x 1536 x 8960, 8 241 / 549 / 282, 16 234 / 545 / 281, 20
// 234 / 547 / 284; 4096 x 4096 x 14336, 8 536 / 1175 / 610, 16 534 / 1141 / 618, 20 528 /
// 1140 / 620; 2048 x 2880 x 2880 all within the 5 % that runs of one differ by.
constexpr int kGluGroup = 16;

// One call's tensors, [n][d] and [n][f] with row strides in elements; the weights
// are [f][d]. Which of them a launch reads and writes depends on it.
struct GluArgs {
  const void* x;
  const void* w_gate;
  const void* w_up;
  const void* dh;
  const void* gate_in;  // backward: the projections as they were kept, or null
  const void* up_in;
  void* h;     // forward; backward: optional
  void* gate;  // forward: the projections (optional); backward: their gradients
  void* up;
  void* dx;
  const uint8_t* mask;
  CkptView ck;  // forward: of h; ck.q null: none
  long long n, ldx, ldwg, ldwu, lddh, ldgi, ldui, ldh, ldg, ldu, lddx;
  int d, f;
  int fp16;  // the 16-bit type: 0 bf16, 1 fp16
  int act;
  float* partials;  // dx: pieces of cut tiles, or null (nothing is cut)
  uint32_t lost;  // self-test: the first CTA's stage whose copies are left out, or kNoneLost
};

// act(x Wg^T) * (x Wu^T) for any number of rows.
cudaError_t launch_glu_fwd(const GluArgs& a, int sms, cudaStream_t st);
// The same (but no checkpoint) for up to kGluSmallRows of them.
constexpr int kGluSmallRows = 8;
cudaError_t launch_glu_small(const GluArgs& a, int sms, cudaStream_t st);
// The gradients of the projections, which are computed again.
cudaError_t launch_glu_bwd_again(const GluArgs& a, int sms, cudaStream_t st);
// The same from the projections as they were kept.
cudaError_t launch_glu_bwd_kept(const GluArgs& a, int sms, cudaStream_t st);
// dx = a.gate Wg + a.up Wu. Bytes of partials that help it (host only; 0: none).
size_t glu_dx_workspace(long long n, int f, int d);
cudaError_t launch_glu_dx(const GluArgs& a, int sms, cudaStream_t st);
cudaError_t prepare_glu_gemm();

// Both weight gradients, fp32 [f][d], packed.
struct GluWgradArgs {
  const void* dgate;
  const void* dup;
  const void* x;
  const float* add_gate;  // or null
  const float* add_up;
  float* dw_gate;
  float* dw_up;
  float* partials;
  int* status;
  long long n, ldg, ldu, ldx;
  int f, d;
  int fp16;
  uint32_t lost;  // as above
};
size_t glu_wgrad_workspace(long long n, int f, int d);
cudaError_t launch_glu_wgrad(const GluWgradArgs& a, int sms, cudaStream_t st);
cudaError_t prepare_glu_wgrad();

}  // namespace grpo
