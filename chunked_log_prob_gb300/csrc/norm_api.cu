// Host side of the norm and checkpoint entry points: argument checks, the
// choice between the aligned and the general kernels, and the launches.
#include <climits>
#include <cstdint>

#include "launch.h"
#include "norm.h"

namespace grpo {
namespace {

constexpr int64_t kMaxRows = 1LL << 30;
constexpr int32_t kMaxHidden = 1 << 27;
constexpr int32_t kMaxWgrad = 1 << 20;  // features of a linear layer

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool known_dtype(int t) { return t >= GRPO_DTYPE_BF16 && t <= GRPO_DTYPE_FP32; }
size_t dtype_bytes(int t) { return t == GRPO_DTYPE_FP32 ? 4 : 2; }

int check_rows(int64_t n, int32_t hidden) {
  if (n < 0 || hidden <= 0) return GRPO_ERR_INVALID_ARG;
  if (n > kMaxRows || hidden > kMaxHidden) return GRPO_ERR_UNSUPPORTED_SHAPE;
  return GRPO_OK;
}

int check_desc(const grpo_norm_desc* d) {
  if (d == nullptr || d->reserved != 0) return GRPO_ERR_INVALID_ARG;
  if (!known_dtype(d->dtype) ||
      (d->weight_dtype != d->dtype && d->weight_dtype != GRPO_DTYPE_FP32) ||
      (d->kind != GRPO_NORM_LAYER && d->kind != GRPO_NORM_RMS) || !(d->eps >= 0.f))
    return GRPO_ERR_INVALID_ARG;
  for (const int64_t s : {d->x_stride, d->residual_stride, d->y_stride, d->z_stride, d->dy_stride,
                          d->dres_stride, d->dx_stride})
    if (s != 0 && s < d->hidden) return GRPO_ERR_INVALID_ARG;
  return check_rows(d->n_tokens, d->hidden);
}

// A tensor's rows: its stride, and whether all of them start on 16 bytes.
struct Rows {
  const void* p;
  int64_t stride;
};
bool rows_on_16(const Rows* r, int count, int hidden, int dtype) {
  if (hidden % 8 != 0) return false;
  for (int i = 0; i < count; ++i)
    if (r[i].p != nullptr &&
        (!aligned(r[i].p, 16) || r[i].stride * static_cast<int64_t>(dtype_bytes(dtype)) % 16 != 0))
      return false;
  return true;
}
bool rows_on_element(const Rows* r, int count, int dtype) {
  for (int i = 0; i < count; ++i)
    if (!aligned(r[i].p, dtype_bytes(dtype))) return false;
  return true;
}

int check_wgrad(int64_t n, int32_t out, int32_t in, int64_t dy_stride) {
  if (n < 0 || out <= 0 || in <= 0 || (dy_stride != 0 && dy_stride < out))
    return GRPO_ERR_INVALID_ARG;
  if (out % 8 != 0 || in % 8 != 0 || dy_stride % 8 != 0 || n > kMaxRows || out > kMaxWgrad ||
      in > kMaxWgrad)
    return GRPO_ERR_UNSUPPORTED_SHAPE;
  return GRPO_OK;
}

thread_local uint32_t t_lost = kNoneLost;

int64_t stride_or(int64_t s, int64_t hidden) { return s != 0 ? s : hidden; }

size_t norm_workspace(const grpo_norm_desc* d) {
  const size_t rows = static_cast<size_t>(norm_bwd_partials(d->n_tokens, d->hidden));
  return (2 * rows * static_cast<size_t>(d->hidden) * sizeof(float) + 255) / 256 * 256;
}

}  // namespace

uint32_t take_lost() {
  const uint32_t v = t_lost;
  t_lost = kNoneLost;
  return v;
}

}  // namespace grpo

using namespace grpo;

extern "C" {

int grpo_norm_fwd(const void* x, const void* residual, const void* weight, const void* bias,
                  const uint8_t* mask, void* y, void* z, float* mean, float* rstd, void* ckpt,
                  const grpo_norm_desc* desc, void* stream) {
  const CallRange range("grpo_norm_fwd");
  int r = check_desc(desc);
  if (r != GRPO_OK) return r;
  const int64_t n = desc->n_tokens, hid = desc->hidden;
  if (n > 0 && (x == nullptr || y == nullptr)) return GRPO_ERR_INVALID_ARG;
  if (z != nullptr && residual == nullptr) return GRPO_ERR_INVALID_ARG;  // z is x
  if (mean != nullptr && desc->kind == GRPO_NORM_RMS) return GRPO_ERR_INVALID_ARG;
  const Rows rows[] = {{x, stride_or(desc->x_stride, hid)},
                       {residual, stride_or(desc->residual_stride, hid)},
                       {y, stride_or(desc->y_stride, hid)},
                       {z, stride_or(desc->z_stride, hid)}};
  if (!rows_on_element(rows, 4, desc->dtype) || !aligned(weight, dtype_bytes(desc->weight_dtype)) ||
      !aligned(bias, dtype_bytes(desc->weight_dtype)) || !aligned(mean, 4) || !aligned(rstd, 4) ||
      !aligned(ckpt, 256))
    return GRPO_ERR_MISALIGNED;
  int sms = 0;
  if ((r = setup_device(&sms)) != GRPO_OK) return r;
  if (n == 0) return GRPO_OK;
  NormFwdArgs a;
  a.x = x;
  a.res = residual;
  a.weight = weight;
  a.bias = bias;
  a.mask = mask;
  a.y = y;
  a.z = z;
  a.mean = mean;
  a.rstd = rstd;
  a.ck = ckpt_view(ckpt, n, desc->hidden);
  a.n = n;
  a.ldx = rows[0].stride;
  a.ldr = rows[1].stride;
  a.ldy = rows[2].stride;
  a.ldz = rows[3].stride;
  a.d = desc->hidden;
  a.wtype = desc->weight_dtype;
  a.kind = desc->kind;
  a.eps = desc->eps;
  a.lost = take_lost();
  const bool vec = rows_on_16(rows, 4, desc->hidden, desc->dtype);
  return launch_norm_fwd(a, desc->dtype, vec, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? GRPO_OK
             : GRPO_ERR_CUDA;
}

int grpo_norm_workspace_size(const grpo_norm_desc* desc, size_t* bytes) {
  if (bytes == nullptr) return GRPO_ERR_INVALID_ARG;
  const int r = check_desc(desc);
  if (r != GRPO_OK) return r;
  *bytes = norm_workspace(desc);
  return GRPO_OK;
}

int grpo_norm_bwd(const void* dy, const void* x, const void* ckpt, const void* weight,
                  const float* mean, const float* rstd, const uint8_t* mask, const void* dres,
                  void* dx, float* dweight, float* dbias, const float* add_dweight,
                  const float* add_dbias, const grpo_norm_desc* desc, void* workspace,
                  size_t workspace_bytes, void* stream) {
  const CallRange range("grpo_norm_bwd");
  int r = check_desc(desc);
  if (r != GRPO_OK) return r;
  const int64_t n = desc->n_tokens, hid = desc->hidden;
  if (n > 0 && (dy == nullptr || dx == nullptr || rstd == nullptr ||
                (x == nullptr) == (ckpt == nullptr)))
    return GRPO_ERR_INVALID_ARG;
  if (n > 0 && (mean == nullptr) != (desc->kind == GRPO_NORM_RMS)) return GRPO_ERR_INVALID_ARG;
  if ((add_dweight != nullptr && dweight == nullptr) || (add_dbias != nullptr && dbias == nullptr))
    return GRPO_ERR_INVALID_ARG;
  const bool grads = dweight != nullptr || dbias != nullptr;
  if (grads && workspace == nullptr) return GRPO_ERR_INVALID_ARG;
  const Rows rows[] = {{dy, stride_or(desc->dy_stride, hid)},
                       {x, stride_or(desc->x_stride, hid)},
                       {dres, stride_or(desc->dres_stride, hid)},
                       {dx, stride_or(desc->dx_stride, hid)}};
  if (!rows_on_element(rows, 4, desc->dtype) || !aligned(weight, dtype_bytes(desc->weight_dtype)) ||
      !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(ckpt, 256) || !aligned(dweight, 4) ||
      !aligned(dbias, 4) || !aligned(add_dweight, 4) || !aligned(add_dbias, 4) ||
      !aligned(workspace, 256))
    return GRPO_ERR_MISALIGNED;
  if (grads && workspace_bytes < norm_workspace(desc)) return GRPO_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  if ((r = setup_device(&sms)) != GRPO_OK) return r;
  NormBwdArgs a;
  a.dy = dy;
  a.x = x;
  a.ck = ckpt_view(ckpt, n, desc->hidden);
  a.weight = weight;
  a.mean = mean;
  a.rstd = rstd;
  a.mask = mask;
  a.dres = dres;
  a.dx = dx;
  a.dweight = dweight;
  a.dbias = dbias;
  a.add_dweight = add_dweight;
  a.add_dbias = add_dbias;
  a.partials = static_cast<float*>(workspace);
  a.n = n;
  a.lddy = rows[0].stride;
  a.ldx = rows[1].stride;
  a.lddres = rows[2].stride;
  a.lddx = rows[3].stride;
  a.d = desc->hidden;
  a.wtype = desc->weight_dtype;
  a.kind = desc->kind;
  a.lost = take_lost();
  const bool vec = rows_on_16(rows, 4, desc->hidden, desc->dtype);
  return launch_norm_bwd(a, desc->dtype, vec, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? GRPO_OK
             : GRPO_ERR_CUDA;
}

int grpo_ckpt_size(int64_t n_tokens, int32_t hidden, size_t* bytes) {
  if (bytes == nullptr) return GRPO_ERR_INVALID_ARG;
  const int r = check_rows(n_tokens, hidden);
  if (r != GRPO_OK) return r;
  *bytes = ckpt_layout(n_tokens, hidden).total;
  return GRPO_OK;
}

int grpo_ckpt_layout(int64_t n_tokens, int32_t hidden, int64_t* q_stride, int64_t* exponent_offset,
                     int64_t* exponent_stride) {
  if (q_stride == nullptr || exponent_offset == nullptr || exponent_stride == nullptr)
    return GRPO_ERR_INVALID_ARG;
  const int r = check_rows(n_tokens, hidden);
  if (r != GRPO_OK) return r;
  const CkptLayout l = ckpt_layout(n_tokens, hidden);
  *q_stride = l.ldq;
  *exponent_offset = static_cast<int64_t>(l.off_ex);
  *exponent_stride = l.lde;
  return GRPO_OK;
}

namespace {

// Shared by packing and unpacking: `x` is the tensor in its own type.
int ckpt_call(const void* x, bool pack, const uint8_t* mask, const void* ckpt, int64_t n,
              int32_t hidden, int32_t dtype, int64_t stride, void* stream) {
  int r = check_rows(n, hidden);
  if (r != GRPO_OK) return r;
  if (!known_dtype(dtype) || (stride != 0 && stride < hidden)) return GRPO_ERR_INVALID_ARG;
  if (n > 0 && (x == nullptr || ckpt == nullptr)) return GRPO_ERR_INVALID_ARG;
  const Rows rows = {x, stride_or(stride, hidden)};
  if (!rows_on_element(&rows, 1, dtype) || !aligned(ckpt, 256)) return GRPO_ERR_MISALIGNED;
  int sms = 0;
  if ((r = setup_device(&sms)) != GRPO_OK) return r;
  if (n == 0) return GRPO_OK;
  CkptArgs a;
  a.x = x;
  a.out = const_cast<void*>(x);
  a.mask = mask;
  a.ck = ckpt_view(ckpt, n, hidden);
  a.n = n;
  a.ld = rows.stride;
  a.d = hidden;
  const bool vec = rows_on_16(&rows, 1, hidden, dtype);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = pack ? launch_ckpt_pack(a, dtype, vec, sms, st)
                             : launch_ckpt_unpack(a, dtype, vec, sms, st);
  return e == cudaSuccess ? GRPO_OK : GRPO_ERR_CUDA;
}

}  // namespace

int grpo_ckpt_pack(const void* x, const uint8_t* mask, void* ckpt, int64_t n_tokens,
                   int32_t hidden, int32_t dtype, int64_t x_stride, void* stream) {
  const CallRange range("grpo_ckpt_pack");
  return ckpt_call(x, true, mask, ckpt, n_tokens, hidden, dtype, x_stride, stream);
}

int grpo_ckpt_unpack(const void* ckpt, void* x, int64_t n_tokens, int32_t hidden, int32_t dtype,
                     int64_t x_stride, void* stream) {
  const CallRange range("grpo_ckpt_unpack");
  return ckpt_call(x, false, nullptr, ckpt, n_tokens, hidden, dtype, x_stride, stream);
}

int grpo_selftest_lose_copy(int64_t index) {
  if (index < -1 || index >= kMaxRows) return GRPO_ERR_INVALID_ARG;
  t_lost = index < 0 ? kNoneLost : static_cast<uint32_t>(index);
  return GRPO_OK;
}

int grpo_ckpt_wgrad_workspace_size(int64_t n_tokens, int32_t out, int32_t in, size_t* bytes) {
  if (bytes == nullptr) return GRPO_ERR_INVALID_ARG;
  const int r = check_wgrad(n_tokens, out, in, 0);
  if (r != GRPO_OK) return r;
  *bytes = ckpt_wgrad_workspace(n_tokens, out, in);
  return GRPO_OK;
}

int grpo_ckpt_wgrad(const void* dy, const void* ckpt, const float* add, float* dW, int64_t n_tokens,
                    int32_t out, int32_t in, int64_t dy_stride, void* workspace,
                    size_t workspace_bytes, void* stream) {
  const CallRange range("grpo_ckpt_wgrad");
  int r = check_wgrad(n_tokens, out, in, dy_stride);
  if (r != GRPO_OK) return r;
  if (dW == nullptr || workspace == nullptr ||
      (n_tokens > 0 && (dy == nullptr || ckpt == nullptr)))
    return GRPO_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(ckpt, 256) || !aligned(add, 16) || !aligned(dW, 16) ||
      !aligned(workspace, 256))
    return GRPO_ERR_MISALIGNED;
  if (workspace_bytes < ckpt_wgrad_workspace(n_tokens, out, in))
    return GRPO_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  if ((r = setup_device(&sms)) != GRPO_OK) return r;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t bytes = static_cast<size_t>(out) * in * sizeof(float);
  if (n_tokens == 0) {  // an empty sum
    if (cudaMemsetAsync(workspace, 0, 64, st) != cudaSuccess) return GRPO_ERR_CUDA;
    const cudaError_t e = add == nullptr ? cudaMemsetAsync(dW, 0, bytes, st)
                          : add != dW    ? cudaMemcpyAsync(dW, add, bytes, cudaMemcpyDeviceToDevice, st)
                                         : cudaSuccess;
    return e == cudaSuccess ? GRPO_OK : GRPO_ERR_CUDA;
  }
  WgradArgs a;
  a.dy = dy;
  a.ck = ckpt_view(ckpt, n_tokens, in);
  a.add = add;
  a.dw = dW;
  a.status = static_cast<int*>(workspace);
  a.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + 256);
  a.n = n_tokens;
  a.lddy = stride_or(dy_stride, out);
  a.lddw = in;
  a.ldadd = in;
  a.out = out;
  a.in = in;
  a.lost = take_lost();
  return launch_ckpt_wgrad(a, sms, st) == cudaSuccess ? GRPO_OK : GRPO_ERR_CUDA;
}

}  // extern "C"
