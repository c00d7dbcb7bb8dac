// Host side of the gated feed-forward entry points: argument checks and launches.
#include <cstdint>

#include "glu.h"
#include "launch.h"

namespace grpo {
namespace {

constexpr int64_t kMaxRows = 1LL << 30;
constexpr int32_t kMaxFeatures = 1 << 20;
constexpr int64_t kMaxTiles = 1LL << 30;

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool on(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int64_t stride_or(int64_t s, int64_t packed) { return s != 0 ? s : packed; }

int check_sizes(int64_t n, int32_t inner, int32_t hidden) {
  if (n < 0 || inner <= 0 || hidden <= 0) return GRPO_ERR_INVALID_ARG;
  if (inner % 8 != 0 || hidden % 8 != 0 || n > kMaxRows || inner > kMaxFeatures ||
      hidden > kMaxFeatures)
    return GRPO_ERR_UNSUPPORTED_SHAPE;
  // Tiles of 128 columns at least, counted in 32 bits.
  const int64_t rows = (n + 255) / 256, wide = inner > hidden ? inner : hidden;
  return rows * ((wide + 127) / 128) > kMaxTiles ? GRPO_ERR_UNSUPPORTED_SHAPE : GRPO_OK;
}

int check_desc(const grpo_glu_desc* d) {
  if (d == nullptr) return GRPO_ERR_INVALID_ARG;
  if ((d->dtype != GRPO_DTYPE_BF16 && d->dtype != GRPO_DTYPE_FP16) || d->act < GRPO_ACT_SILU ||
      d->act > GRPO_ACT_RELU)
    return GRPO_ERR_INVALID_ARG;
  const int r = check_sizes(d->n_tokens, d->inner, d->hidden);
  if (r != GRPO_OK) return r;
  for (const int64_t s : {d->x_stride, d->w_gate_stride, d->w_up_stride, d->dx_stride}) {
    if (s != 0 && s < d->hidden) return GRPO_ERR_INVALID_ARG;
    if (s % 8 != 0) return GRPO_ERR_UNSUPPORTED_SHAPE;
  }
  for (const int64_t s : {d->h_stride, d->gate_stride, d->up_stride, d->dh_stride, d->dgate_stride,
                          d->dup_stride}) {
    if (s != 0 && s < d->inner) return GRPO_ERR_INVALID_ARG;
    if (s % 8 != 0) return GRPO_ERR_UNSUPPORTED_SHAPE;
  }
  return GRPO_OK;
}

// What the calls share.
GluArgs args_of(const grpo_glu_desc* d) {
  GluArgs a = {};
  a.n = d->n_tokens;
  a.d = d->hidden;
  a.f = d->inner;
  a.fp16 = d->dtype == GRPO_DTYPE_FP16;
  a.act = d->act;
  a.ldx = stride_or(d->x_stride, d->hidden);
  a.ldwg = stride_or(d->w_gate_stride, d->hidden);
  a.ldwu = stride_or(d->w_up_stride, d->hidden);
  a.lddx = stride_or(d->dx_stride, d->hidden);
  a.lddh = stride_or(d->dh_stride, d->inner);
  a.ldh = stride_or(d->h_stride, d->inner);
  a.lost = kNoneLost;
  return a;
}

}  // namespace
}  // namespace grpo

using namespace grpo;

extern "C" {

int grpo_glu_fwd(const void* x, const void* w_gate, const void* w_up, const uint8_t* mask, void* h,
                 void* gate, void* up, void* ckpt, const grpo_glu_desc* desc, void* stream) {
  const CallRange range("grpo_glu_fwd");
  int r = check_desc(desc);
  if (r != GRPO_OK) return r;
  if (w_gate == nullptr || w_up == nullptr || (gate == nullptr) != (up == nullptr) ||
      (desc->n_tokens > 0 && (x == nullptr || h == nullptr)))
    return GRPO_ERR_INVALID_ARG;
  if (!on16(x) || !on16(w_gate) || !on16(w_up) || !on16(h) || !on16(gate) || !on16(up) ||
      !on(ckpt, 256))
    return GRPO_ERR_MISALIGNED;
  int sms = 0;
  if ((r = setup_device(&sms)) != GRPO_OK) return r;
  if (desc->n_tokens == 0) return GRPO_OK;
  GluArgs a = args_of(desc);
  a.x = x;
  a.w_gate = w_gate;
  a.w_up = w_up;
  a.mask = mask;
  a.h = h;
  a.gate = gate;
  a.up = up;
  a.ldg = stride_or(desc->gate_stride, desc->inner);
  a.ldu = stride_or(desc->up_stride, desc->inner);
  a.ck = ckpt_view(ckpt, desc->n_tokens, desc->inner);
  a.lost = take_lost();
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.n > kGluSmallRows)
    return launch_glu_fwd(a, sms, st) == cudaSuccess ? GRPO_OK : GRPO_ERR_CUDA;
  if (launch_glu_small(a, sms, st) != cudaSuccess) return GRPO_ERR_CUDA;
  if (ckpt == nullptr) return GRPO_OK;
  CkptArgs c;  // few rows are seldom kept: a launch of its own
  c.x = h;
  c.out = h;
  c.mask = mask;
  c.ck = a.ck;
  c.n = a.n;
  c.ld = a.ldh;
  c.d = a.f;
  return launch_ckpt_pack(c, desc->dtype, true, sms, st) == cudaSuccess ? GRPO_OK : GRPO_ERR_CUDA;
}

int grpo_glu_bwd(const void* dh, const void* x, const void* w_gate, const void* w_up,
                 const void* gate, const void* up, const uint8_t* mask, void* dgate, void* dup,
                 void* dx, void* h, const grpo_glu_desc* desc, void* workspace,
                 size_t workspace_bytes, void* stream) {
  const CallRange range("grpo_glu_bwd");
  int r = check_desc(desc);
  if (r != GRPO_OK) return r;
  const bool kept = gate != nullptr;
  if (kept != (up != nullptr) || w_gate == nullptr || w_up == nullptr ||
      (desc->n_tokens > 0 &&
       (dh == nullptr || dgate == nullptr || dup == nullptr || (!kept && x == nullptr))))
    return GRPO_ERR_INVALID_ARG;
  for (const void* p : {dh, x, w_gate, w_up, gate, up, static_cast<const void*>(dgate),
                        static_cast<const void*>(dup), static_cast<const void*>(dx),
                        static_cast<const void*>(h)})
    if (!on16(p)) return GRPO_ERR_MISALIGNED;
  if (!on(workspace, 256)) return GRPO_ERR_MISALIGNED;
  const size_t need = glu_dx_workspace(desc->n_tokens, desc->inner, desc->hidden);
  if (workspace != nullptr && dx != nullptr && workspace_bytes < need)
    return GRPO_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  if ((r = setup_device(&sms)) != GRPO_OK) return r;
  if (desc->n_tokens == 0) return GRPO_OK;
  GluArgs a = args_of(desc);
  a.x = x;
  a.w_gate = w_gate;
  a.w_up = w_up;
  a.dh = dh;
  a.gate_in = gate;
  a.up_in = up;
  a.ldgi = stride_or(desc->gate_stride, desc->inner);
  a.ldui = stride_or(desc->up_stride, desc->inner);
  a.mask = mask;
  a.h = h;
  a.gate = dgate;
  a.up = dup;
  a.ldg = stride_or(desc->dgate_stride, desc->inner);
  a.ldu = stride_or(desc->dup_stride, desc->inner);
  a.dx = dx;
  a.partials = need > 0 ? static_cast<float*>(workspace) : nullptr;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const uint32_t lost = take_lost();
  if (!kept) a.lost = lost;
  if ((kept ? launch_glu_bwd_kept(a, sms, st) : launch_glu_bwd_again(a, sms, st)) != cudaSuccess)
    return GRPO_ERR_CUDA;
  if (dx == nullptr) return GRPO_OK;
  a.lost = kept ? lost : kNoneLost;
  return launch_glu_dx(a, sms, st) == cudaSuccess ? GRPO_OK : GRPO_ERR_CUDA;
}

int grpo_glu_bwd_workspace_size(int64_t n_tokens, int32_t inner, int32_t hidden, size_t* bytes) {
  if (bytes == nullptr) return GRPO_ERR_INVALID_ARG;
  const int r = check_sizes(n_tokens, inner, hidden);
  if (r != GRPO_OK) return r;
  *bytes = glu_dx_workspace(n_tokens, inner, hidden);
  return GRPO_OK;
}

int grpo_glu_wgrad_workspace_size(int64_t n_tokens, int32_t inner, int32_t hidden, size_t* bytes) {
  if (bytes == nullptr) return GRPO_ERR_INVALID_ARG;
  const int r = check_sizes(n_tokens, inner, hidden);
  if (r != GRPO_OK) return r;
  *bytes = glu_wgrad_workspace(n_tokens, inner, hidden);
  return GRPO_OK;
}

int grpo_glu_wgrad(const void* dgate, const void* dup, const void* x, const float* add_gate,
                   const float* add_up, float* dw_gate, float* dw_up, const grpo_glu_desc* desc,
                   void* workspace, size_t workspace_bytes, void* stream) {
  const CallRange range("grpo_glu_wgrad");
  int r = check_desc(desc);
  if (r != GRPO_OK) return r;
  const int64_t n = desc->n_tokens;
  if (dw_gate == nullptr || dw_up == nullptr || workspace == nullptr ||
      (n > 0 && (dgate == nullptr || dup == nullptr || x == nullptr)))
    return GRPO_ERR_INVALID_ARG;
  if (!on16(dgate) || !on16(dup) || !on16(x) || !on16(add_gate) || !on16(add_up) ||
      !on16(dw_gate) || !on16(dw_up) || !on(workspace, 256))
    return GRPO_ERR_MISALIGNED;
  if (workspace_bytes < glu_wgrad_workspace(n, desc->inner, desc->hidden))
    return GRPO_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  if ((r = setup_device(&sms)) != GRPO_OK) return r;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (n == 0) {  // empty sums
    const size_t bytes = static_cast<size_t>(desc->inner) * desc->hidden * sizeof(float);
    cudaError_t e = cudaMemsetAsync(workspace, 0, 64, st);
    const float* add[] = {add_gate, add_up};
    float* out[] = {dw_gate, dw_up};
    for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
      if (add[i] == nullptr)
        e = cudaMemsetAsync(out[i], 0, bytes, st);
      else if (add[i] != out[i])
        e = cudaMemcpyAsync(out[i], add[i], bytes, cudaMemcpyDeviceToDevice, st);
    }
    return e == cudaSuccess ? GRPO_OK : GRPO_ERR_CUDA;
  }
  GluWgradArgs a;
  a.dgate = dgate;
  a.dup = dup;
  a.x = x;
  a.add_gate = add_gate;
  a.add_up = add_up;
  a.dw_gate = dw_gate;
  a.dw_up = dw_up;
  a.status = static_cast<int*>(workspace);
  a.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + 256);
  a.n = n;
  a.ldg = stride_or(desc->dgate_stride, desc->inner);
  a.ldu = stride_or(desc->dup_stride, desc->inner);
  a.ldx = stride_or(desc->x_stride, desc->hidden);
  a.f = desc->inner;
  a.d = desc->hidden;
  a.fp16 = desc->dtype == GRPO_DTYPE_FP16;
  a.lost = take_lost();
  return launch_glu_wgrad(a, sms, st) == cudaSuccess ? GRPO_OK : GRPO_ERR_CUDA;
}

}  // extern "C"
