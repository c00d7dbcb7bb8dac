// Activations to 8 bits and back: e4m3 values, one power of two per 32 columns
// of a row (the format is described in row_ops.cuh). Memory bound: one read and
// one write of everything, about 5 operations per value.
#include <algorithm>

#include "launch.h"
#include "norm.h"
#include "row_ops.cuh"

namespace grpo {

CkptLayout ckpt_layout(long long n, int hidden) {
  CkptLayout l;
  l.ldq = (hidden + 15LL) / 16 * 16;
  l.lde = ((hidden + kCkptBlock - 1LL) / kCkptBlock + 15) / 16 * 16;
  l.off_ex = (static_cast<size_t>(n) * l.ldq + 255) / 256 * 256;
  l.total = l.off_ex + (static_cast<size_t>(n) * l.lde + 255) / 256 * 256;
  return l;
}

CkptView ckpt_view(const void* buf, long long n, int hidden) {
  CkptView v;
  if (buf == nullptr) return v;
  const CkptLayout l = ckpt_layout(n, hidden);
  v.q = static_cast<uint8_t*>(const_cast<void*>(buf));
  v.ex = v.q + l.off_ex;
  v.ldq = l.ldq;
  v.lde = l.lde;
  return v;
}

namespace {

constexpr int kTpr = 32;   // a warp's part of a row: 256 columns
constexpr int kWarps = 8;

// One warp per (row, 256 columns).
template <typename T, bool VEC>
__global__ void __launch_bounds__(kTpr* kWarps) ckpt_pack_kernel(const CkptArgs a, int slabs,
                                                                 long long units) {
  const int t = threadIdx.x & 31;
  const long long step = static_cast<long long>(gridDim.x) * kWarps;
  for (long long u = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units;
       u += step) {
    const long long row = u / slabs;
    const int first = static_cast<int>(u - row * slabs) * (8 * kTpr);
    const int d = min(a.d - first, 8 * kTpr);
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (a.mask == nullptr || a.mask[row] != 0)
      widen(load_chunk<T, VEC>(static_cast<const T*>(a.x) + row * a.ld + first, 0, t, kTpr, d), v);
    ckpt_store_chunk<T, VEC>(v, a.ck.q + row * a.ck.ldq + first,
                             a.ck.ex + row * a.ck.lde + first / kCkptBlock, 0, t, kTpr, d);
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kTpr* kWarps) ckpt_unpack_kernel(const CkptArgs a, int slabs,
                                                                   long long units) {
  const int t = threadIdx.x & 31;
  const long long step = static_cast<long long>(gridDim.x) * kWarps;
  for (long long u = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units;
       u += step) {
    const long long row = u / slabs;
    const int first = static_cast<int>(u - row * slabs) * (8 * kTpr);
    const int d = min(a.d - first, 8 * kTpr);
    float v[8];
    ckpt_widen<VEC>(ckpt_load_chunk<VEC>(a.ck.q + row * a.ck.ldq + first,
                                         a.ck.ex + row * a.ck.lde + first / kCkptBlock, 0, t, kTpr,
                                         d),
                    v);
    store_chunk<T, VEC>(static_cast<T*>(a.out) + row * a.ld + first, narrow<T>(v), 0, t, kTpr, d);
  }
}

template <typename T, bool VEC, bool PACK>
cudaError_t run(const CkptArgs& a, int sms, cudaStream_t st) {
  const int slabs = (a.d + 8 * kTpr - 1) / (8 * kTpr);
  const long long units = a.n * slabs;
  const int grid = static_cast<int>(std::min<long long>((units + kWarps - 1) / kWarps, 8LL * sms));
  LaunchTimer timer(PACK ? "ckpt_pack_kernel" : "ckpt_unpack_kernel", st);
  if (PACK)
    ckpt_pack_kernel<T, VEC><<<grid, kTpr * kWarps, 0, st>>>(a, slabs, units);
  else
    ckpt_unpack_kernel<T, VEC><<<grid, kTpr * kWarps, 0, st>>>(a, slabs, units);
  return cudaGetLastError();
}

template <bool PACK>
cudaError_t run_any(const CkptArgs& a, int dtype, bool vec, int sms, cudaStream_t st) {
  switch (dtype) {
    case GRPO_DTYPE_BF16:
      return vec ? run<__nv_bfloat16, true, PACK>(a, sms, st)
                 : run<__nv_bfloat16, false, PACK>(a, sms, st);
    case GRPO_DTYPE_FP16:
      return vec ? run<__half, true, PACK>(a, sms, st) : run<__half, false, PACK>(a, sms, st);
    default:
      return vec ? run<float, true, PACK>(a, sms, st) : run<float, false, PACK>(a, sms, st);
  }
}

}  // namespace

cudaError_t launch_ckpt_pack(const CkptArgs& a, int dtype, bool vec, int sms, cudaStream_t st) {
  return run_any<true>(a, dtype, vec, sms, st);
}

cudaError_t launch_ckpt_unpack(const CkptArgs& a, int dtype, bool vec, int sms, cudaStream_t st) {
  return run_any<false>(a, dtype, vec, sms, st);
}

}  // namespace grpo
