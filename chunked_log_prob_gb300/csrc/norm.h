// Internal launch interface of the norm and checkpoint operators.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "grpo_gb300.h"

namespace grpo {

// A checkpoint in its buffer: q [n][ldq] bytes, exponents [n][lde] bytes.
struct CkptView {
  uint8_t* q = nullptr;
  uint8_t* ex = nullptr;
  long long ldq = 0, lde = 0;
};

struct CkptLayout {
  long long ldq, lde;
  size_t off_ex, total;
};
// ldq: D up to 16; lde: a byte per 32 columns, up to 16 (TMA row strides).
CkptLayout ckpt_layout(long long n, int hidden);
CkptView ckpt_view(const void* buf, long long n, int hidden);

struct NormFwdArgs {
  const void* x;
  const void* res;  // or null
  const void* weight;
  const void* bias;
  const uint8_t* mask;
  void* y;
  void* z;
  float* mean;
  float* rstd;
  CkptView ck;  // ck.q null: none
  long long n, ldx, ldr, ldy, ldz;
  int d, wtype, kind;
  float eps;
  uint32_t lost;  // self-test: the row from which on its CTA copies none, or kNoneLost
};

struct NormBwdArgs {
  const void* dy;
  const void* x;  // or null: from ck
  CkptView ck;
  const void* weight;
  const float* mean;
  const float* rstd;
  const uint8_t* mask;
  const void* dres;
  void* dx;
  float* dweight;
  float* dbias;
  const float* add_dweight;
  const float* add_dbias;
  float* partials;  // [rows of partials][d], those of dbias behind them
  long long n, lddy, ldx, lddres, lddx;
  int d, wtype, kind;
  uint32_t lost;  // as above (where two CTAs share a row: the first)
};

struct CkptArgs {
  const void* x;  // pack: in
  void* out;      // unpack: out
  const uint8_t* mask;
  CkptView ck;
  long long n, ld;
  int d;
};

// No copy is left out (grpo_selftest_lose_copy).
constexpr uint32_t kNoneLost = 0xffffffffu;

// Largest D of the kernels that hold a whole row in registers (forward: of rows on
// 16 bytes; others up to 8192).
constexpr int kNormRegisterRow = 16384;
// Rows of partial weight gradients of one backward call: at most this many.
constexpr int kNormMaxPartials = 608;

int norm_bwd_partials(long long n, int d);  // upper bound for a call
cudaError_t launch_norm_fwd(const NormFwdArgs& a, int dtype, bool vec, int sms, cudaStream_t st);
cudaError_t launch_norm_bwd(const NormBwdArgs& a, int dtype, bool vec, int sms, cudaStream_t st);
cudaError_t launch_ckpt_pack(const CkptArgs& a, int dtype, bool vec, int sms, cudaStream_t st);
cudaError_t launch_ckpt_unpack(const CkptArgs& a, int dtype, bool vec, int sms, cudaStream_t st);

struct WgradArgs {
  const void* dy;
  CkptView ck;
  const float* add;
  float* dw;
  float* partials;
  int* status;
  long long n, lddy, lddw, ldadd;
  int out, in;
  uint32_t lost;  // self-test: the first CTA's stage whose copy is left out, or kNoneLost
};
size_t ckpt_wgrad_workspace(long long n, int out, int in);
cudaError_t launch_ckpt_wgrad(const WgradArgs& a, int sms, cudaStream_t st);

}  // namespace grpo
