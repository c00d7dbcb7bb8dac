// Layer norm and RMS norm, forward and backward, with the residual add, the
// row mask and the 8-bit checkpoint of the normed stream fused in.
//
//   z = round(x + r);  mu = mean z (layer), 0 (rms);
//   rstd = (mean (z - mu)^2 + eps)^-1/2;  y = (z - mu) rstd w + b
//   h = (z - mu) rstd, u = dy w:
//   dx = rstd (u - mean u - h mean(u h)) + dres   (rms: without mean u)
//   dw = sum_t dy h, db = sum_t dy
//
// Memory bound: about 10 operations per value against 4 to 9 bytes. A row is
// read once and held in registers (up to 8192 columns); statistics are fp32.
#include <algorithm>
#include <atomic>

#include "launch.h"
#include "norm.h"
#include "row_ops.cuh"

namespace grpo {

namespace {

constexpr int kRowThreads = 256;  // threads of a CTA whose rows are short

__device__ __forceinline__ bool row_live(const uint8_t* mask, long long row, long long n) {
  return row < n && (mask == nullptr || mask[row] != 0);
}

// Mean and centred sum of squares of a row. Layer norm: each warp centres its
// values on their own mean, then the warps' sums are joined exactly as if one
// had centred on the row's (no difference of large squares). `cnt`: valid
// values of this warp, shared by all warps in cnt_sh.
template <int CH, bool VEC>
__device__ __forceinline__ float2 row_moments(const float (&v)[CH][8], int kind, int t, int tpr,
                                              int d, int bar, float2* sh, const float* cnt_sh,
                                              int& phase) {
  float s = 0.f;
  if (kind == GRPO_NORM_RMS) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[c][j] * v[c][j];
    return make_float2(0.f, row_sum2(make_float2(s, 0.f), t, tpr, bar, sh, phase).x);
  }
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) s += v[c][j];
  s = warp_sum(s);
  const int warp = t >> 5, lane = t & 31;
  const float cnt = cnt_sh[warp];
  const float mw = cnt > 0.f ? s / cnt : 0.f;
  float m2 = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float e = v[c][j] - mw;
      if (chunk_col<VEC>(c, j, t, tpr) < d) m2 += e * e;
    }
  m2 = warp_sum(m2);
  if (tpr == 32) return make_float2(mw, m2);
  float2* p = sh + phase * 32;
  phase ^= 1;
  if (lane == 0) p[warp] = make_float2(s, m2);
  named_barrier(bar, tpr);
  const bool in = lane < (tpr >> 5);
  const float2 o = in ? p[lane] : make_float2(0.f, 0.f);
  const float n = in ? cnt_sh[lane] : 0.f;
  const float mean = warp_sum(o.x) / static_cast<float>(d);
  const float e = n > 0.f ? o.x / n - mean : 0.f;
  return make_float2(mean, warp_sum(o.y + n * e * e));
}

// Valid columns of each warp of a row into cnt_sh; followed by a barrier.
template <int CH, bool VEC>
__device__ __forceinline__ void count_columns(int t, int tpr, int d, float* cnt_sh) {
  float n = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) n += chunk_col<VEC>(c, j, t, tpr) < d ? 1.f : 0.f;
  n = warp_sum(n);
  if ((t & 31) == 0) cnt_sh[t >> 5] = n;
}

// blockDim = (tpr, rows of the CTA). The next row's loads are issued before
// this row's sums, so that they are in flight during its barrier and stores.
template <typename T, bool VEC, int CH>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const NormFwdArgs a) {
  __shared__ float2 red[8][2 * 32];
  __shared__ float cnt_all[8][32];
  const int t = threadIdx.x, tpr = blockDim.x, g = threadIdx.y, d = a.d;
  int phase = 0;
  float w[CH][8], b[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = chunk_col<VEC>(c, j, t, tpr);
      w[c][j] = a.weight != nullptr && col < d ? load_param(a.weight, a.wtype, col) : 1.f;
      b[c][j] = a.bias != nullptr && col < d ? load_param(a.bias, a.wtype, col) : 0.f;
    }
  count_columns<CH, VEC>(t, tpr, d, cnt_all[g]);
  __syncthreads();

  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.res);
  T* y = static_cast<T*>(a.y);
  T* z = static_cast<T*>(a.z);
  const long long step = static_cast<long long>(gridDim.x) * blockDim.y;
  long long row = static_cast<long long>(blockIdx.x) * blockDim.y + g;
  bool live = row_live(a.mask, row, a.n);
  bool live1 = row_live(a.mask, row + step, a.n);
  Raw8<T> rx[CH], rr[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    if (live) rx[c] = load_chunk<T, VEC>(x + row * a.ldx, c, t, tpr, d);
    if (live && res != nullptr) rr[c] = load_chunk<T, VEC>(res + row * a.ldr, c, t, tpr, d);
  }
  for (; row < a.n; row += step) {
    const bool live2 = row_live(a.mask, row + 2 * step, a.n);
    const long long next = row + step;
    float v[CH][8];
    if (live) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        widen(rx[c], v[c]);
        if (res != nullptr) {
          float r[8];
          widen(rr[c], r);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[c][j] += r[j];
          // The stream holds z rounded; the norm is taken of what it holds.
          const Raw8<T> o = narrow<T>(v[c]);
          if (z != nullptr) store_chunk<T, VEC>(z + row * a.ldz, o, c, t, tpr, d);
          widen(o, v[c]);
        }
      }
    }
    if (live1) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        rx[c] = load_chunk<T, VEC>(x + next * a.ldx, c, t, tpr, d);
        if (res != nullptr) rr[c] = load_chunk<T, VEC>(res + next * a.ldr, c, t, tpr, d);
      }
    }
    float mean = 0.f, rstd = 0.f;
    if (live) {
      const float2 m = row_moments<CH, VEC>(v, a.kind, t, tpr, d, g + 1, red[g], cnt_all[g], phase);
      mean = m.x;
      rstd = 1.f / sqrtf(m.y / static_cast<float>(d) + a.eps);
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] = 0.f;
        if (z != nullptr && res != nullptr)
          store_chunk<T, VEC>(z + row * a.ldz, narrow<T>(v[c]), c, t, tpr, d);
      }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (a.ck.q != nullptr)
        ckpt_store_chunk<T, VEC>(v[c], a.ck.q + row * a.ck.ldq, a.ck.ex + row * a.ck.lde, c, t, tpr,
                                 d);
      if (live) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] = (v[c][j] - mean) * rstd * w[c][j] + b[c][j];
      }
      store_chunk<T, VEC>(y + row * a.ldy, narrow<T>(v[c]), c, t, tpr, d);
    }
    if (t == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    live = live1;
    live1 = live2;
  }
}

// The aligned form. Each row of the CTA (threadIdx.y) has a ring of `slots`
// rows in shared memory, filled by bulk copies; a slot is filled again as soon
// as the row's sum has been taken, when every thread holds its values.
// The bytes in flight come from the ring, so what is left is issue slots: a
// thread holds up to 32 values, so that a row's fixed work (barriers, sums,
// addresses) is shared by few warps, and works on pairs of them.
struct Ring {
  int slots;           // rows in flight for each row of the CTA
  uint32_t row_bytes;  // of a slot
};

// Shared memory: barriers, then the parameters as fp32, then the rings.
constexpr int kMaxSlots = 8;
constexpr int kMaxRows = 8;  // rows of a CTA
constexpr uint32_t kRingBars = kMaxRows * kMaxSlots * sizeof(uint64_t);

// Threads of a CTA with 8 ch values a thread, at most (kNormRegisterRow columns).
constexpr int ring_threads(int ch) { return ch == 4 ? 256 : ch == 3 ? 352 : 512; }

// After a timeout: lets the copies still in flight land (within the same limit).
__device__ __forceinline__ void land(uint64_t* bars, int slots, uint32_t parity, uint32_t pending) {
  for (int s = 0; s < slots; ++s)
    if ((pending >> s) & 1u) row_wait(&bars[s], (parity >> s) & 1u);
}

// Columns that warp k of a row holds (VEC layout).
template <int CH>
__device__ __forceinline__ float warp_columns(int k, int tpr, int d) {
  int n = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) n += max(0, min(256, d - (c * tpr + k * 32) * 8));
  return static_cast<float>(n);
}

// Rows of the group that begins at `row`.
__device__ __forceinline__ int row_count(long long row, long long n, long long step) {
  return row < n ? static_cast<int>((n - 1 - row) / step) + 1 : 0;
}

template <typename T, int CH, int KIND>
__global__ void __launch_bounds__(ring_threads(CH)) norm_fwd_ring_kernel(const NormFwdArgs a, const Ring ring) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float red[kMaxRows][2 * 2 * 16];
  const int t = threadIdx.x, tpr = blockDim.x, g = threadIdx.y, d = a.d;
  const int warps = tpr >> 5;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem) + g * kMaxSlots;
  float* const sw = reinterpret_cast<float*>(smem + kRingBars);
  float* const sb = sw + (a.weight != nullptr ? d : 0);
  const uint32_t sw32 = smem_u32(sw), sb32 = smem_u32(sb);
  const uint32_t rows0 = smem_u32(sb + (a.bias != nullptr ? d : 0)) +
                         g * ring.slots * ring.row_bytes;
  const uint32_t x_bytes = d * sizeof(T);
  const bool res = a.res != nullptr;
  const long long step = static_cast<long long>(gridDim.x) * blockDim.y;
  const long long row0 = static_cast<long long>(blockIdx.x) * blockDim.y + g;
  const int count = row_count(row0, a.n, step);
  const uint8_t* const mask = a.mask;
  // Thread 0: slots whose copies have not been waited for, and the next row to fetch.
  uint32_t pending = 0;
  int fetched = 0;
  const auto fetch = [&](int slot) {
    if (fetched >= count) return;
    const long long r = row0 + step * fetched++;
    if (mask != nullptr && mask[r] == 0) return;
    pending |= 1u << slot;
    const uint32_t dst = rows0 + slot * ring.row_bytes;
    mbar_arrive_expect_tx(&bars[slot], res ? 2 * x_bytes : x_bytes);
    bulk_load(dst, static_cast<const T*>(a.x) + r * a.ldx, x_bytes, &bars[slot]);
    if (res) bulk_load(dst + x_bytes, static_cast<const T*>(a.res) + r * a.ldr, x_bytes, &bars[slot]);
  };
  if (t == 0) {
    for (int s = 0; s < ring.slots; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
    for (int s = 0; s < ring.slots; ++s) fetch(s);
  }
  for (int k = t; k < 2 * 2 * 16; k += tpr) red[g][k] = 0.f;
  if (a.weight != nullptr) stage_param(sw, a.weight, a.wtype, d, g * tpr + t, tpr * blockDim.y);
  if (a.bias != nullptr) stage_param(sb, a.bias, a.wtype, d, g * tpr + t, tpr * blockDim.y);
  __syncthreads();

  const float inv_d = 1.f / static_cast<float>(d);
  // Values of this warp that are columns: its chunks before d.
  float warp_n = 0.f;
  if (KIND == GRPO_NORM_LAYER) {
#pragma unroll
    for (int c = 0; c < CH; ++c) warp_n += (c * tpr + t) * 8 < d ? 8.f : 0.f;
    warp_n = warp_sum(warp_n);
  }
  const float inv_warp_n = warp_n > 0.f ? 1.f / warp_n : 0.f;
  T* y = static_cast<T*>(a.y) + row0 * a.ldy;
  T* z = res && a.z != nullptr ? static_cast<T*>(a.z) + row0 * a.ldz : nullptr;
  uint8_t* q = a.ck.q != nullptr ? a.ck.q + row0 * a.ck.ldq : nullptr;
  uint8_t* ex = a.ck.ex + row0 * a.ck.lde;
  int phase = 0, slot = 0;
  uint32_t parity = 0;  // a bit per slot
  bool ok = true;
  bool live = count > 0 && (mask == nullptr || mask[row0] != 0);
  for (int i = 0; i < count; ++i) {
    const bool live1 =
        i + 1 < count && (mask == nullptr || mask[row0 + step * (i + 1)] != 0);
    f32x2 v[CH][4];
    float mean = 0.f, rstd = 0.f;
    if (live) {
      ok = ok && row_wait(&bars[slot], (parity >> slot) & 1u);
      if (ok) {
        parity ^= 1u << slot;
        pending &= ~(1u << slot);
      }
      const uint32_t src = rows0 + slot * ring.row_bytes + t * sizeof(Raw8<T>);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[c][j] = 0ull;
        if ((c * tpr + t) * 8 >= d) continue;
        const uint32_t at = src + c * tpr * sizeof(Raw8<T>);
        widen2(lds_raw<T>(at), v[c]);
        if (res) {
          f32x2 r[4];
          widen2(lds_raw<T>(at + x_bytes), r);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[c][j] = add2(v[c][j], r[j]);
          // The stream holds z rounded; the norm is taken of what it holds.
          const Raw8<T> o = narrow2<T>(v[c]);
          if (z != nullptr) store_raw(z + (c * tpr + t) * 8, o);
          widen2(o, v[c]);
        }
      }
      if (KIND == GRPO_NORM_RMS) {
        f32x2 s[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[j & 1] = fma2(v[c][j], v[c][j], s[j & 1]);
        float m[1] = {warp_sum(sum_of(add2(s[0], s[1])))};
        join_warps(m, t, warps, g + 1, red[g], phase);
        rstd = rsqrtf(m[0] * inv_d + a.eps);
      } else {
        // Each warp centres its values on their own mean; the warps' sums are
        // then joined as if all had been centred on the row's.
        f32x2 s[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[j & 1] = add2(v[c][j], s[j & 1]);
        const float sum = warp_sum(sum_of(add2(s[0], s[1])));
        const float mw = sum * inv_warp_n;
        const f32x2 nmw = pair(-mw, -mw);
        s[0] = s[1] = 0ull;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          if ((c * tpr + t) * 8 >= d) continue;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x2 e = add2(v[c][j], nmw);
            s[j & 1] = fma2(e, e, s[j & 1]);
          }
        }
        const float m2 = warp_sum(sum_of(add2(s[0], s[1])));
        float total = sum, centred = m2;
        if (warps > 1) {
          float* sh = red[g] + phase * 2 * 16;
          phase ^= 1;
          if ((t & 31) == 0) {
            sh[t >> 5] = sum;
            sh[16 + (t >> 5)] = m2;
          }
          named_barrier(g + 1, tpr);
          total = 0.f;
          for (int k = 0; k < warps; ++k) total += sh[k];
          const float mu = total * inv_d;
          centred = 0.f;
          for (int k = 0; k < warps; ++k) {
            const float nk = warp_columns<CH>(k, tpr, d);
            const float e = nk > 0.f ? sh[k] / nk - mu : 0.f;
            centred += sh[16 + k] + nk * e * e;
          }
        } else {
          __syncwarp();
        }
        mean = total * inv_d;
        rstd = rsqrtf(centred * inv_d + a.eps);
      }
      if (!ok) rstd = __uint_as_float(0x7fc00000u);
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[c][j] = 0ull;
        if (z != nullptr && (c * tpr + t) * 8 < d)
          store_raw(z + (c * tpr + t) * 8, narrow2<T>(v[c]));
      }
    }
    // Every thread has its values (the sum's barrier, or the warp's).
    if (t == 0 && ok) fetch(slot);
    if (++slot == ring.slots) slot = 0;
    const f32x2 scale = pair(rstd, rstd), shift = pair(-mean, -mean);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int at = c * tpr + t;
      if (q != nullptr) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) split(v[c][j], f[2 * j], f[2 * j + 1]);
        ckpt_store_chunk<T, true>(f, q, ex, c, t, tpr, d);
      }
      if (8 * at >= d) continue;
      if (live) {
        f32x2 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[c][j] = mul2(KIND == GRPO_NORM_LAYER ? add2(v[c][j], shift) : v[c][j], scale);
        if (a.weight != nullptr) {
          read_param(sw32, at, 2 * d, w);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[c][j] = mul2(v[c][j], w[j]);
        }
        if (a.bias != nullptr) {
          read_param(sb32, at, 2 * d, w);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[c][j] = add2(v[c][j], w[j]);
        }
      }
      store_raw(y + 8 * at, narrow2<T>(v[c]));
    }
    if (t == 0) {
      const long long row = row0 + step * i;
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    y += step * a.ldy;
    if (z != nullptr) z += step * a.ldz;
    if (q != nullptr) {
      q += step * a.ck.ldq;
      ex += step * a.ck.lde;
    }
    live = live1;
  }
  land(bars, ring.slots, parity, pending);
}

// Rows beyond kNormRegisterRow columns: the CTA walks over the row three times
// (sum, centred squares, output); the second and third walk find it in L2. A
// thread rereads only what it stored itself, so outputs may lie on the inputs.
template <typename T, bool VEC>
__global__ void __launch_bounds__(512) norm_fwd_long_kernel(const NormFwdArgs a) {
  __shared__ float2 red[2 * 32];
  const int t = threadIdx.x, tpr = blockDim.x, d = a.d;
  const int chunks = (d + 8 * tpr - 1) / (8 * tpr);
  int phase = 0;
  for (long long row = blockIdx.x; row < a.n; row += gridDim.x) {
    const bool live = row_live(a.mask, row, a.n);
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* res = a.res != nullptr ? static_cast<const T*>(a.res) + row * a.ldr : nullptr;
    T* z = a.z != nullptr && res != nullptr ? static_cast<T*>(a.z) + row * a.ldz : nullptr;
    T* y = static_cast<T*>(a.y) + row * a.ldy;
    const auto stream = [&](int c, float(&v)[8]) {
      if (!live) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f;
        return;
      }
      widen(load_chunk<T, VEC>(x, c, t, tpr, d), v);
      if (res != nullptr) {
        float r[8];
        widen(load_chunk<T, VEC>(res, c, t, tpr, d), r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += r[j];
        widen(narrow<T>(v), v);
      }
    };
    float mean = 0.f, rstd = 0.f;
    if (live) {
      float v[8];
      if (a.kind != GRPO_NORM_RMS) {
        float s = 0.f;
        for (int c = 0; c < chunks; ++c) {
          stream(c, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) s += v[j];
        }
        mean = row_sum2(make_float2(s, 0.f), t, tpr, 1, red, phase).x / static_cast<float>(d);
      }
      float m2 = 0.f;
      for (int c = 0; c < chunks; ++c) {
        stream(c, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float e = v[j] - mean;
          if (chunk_col<VEC>(c, j, t, tpr) < d) m2 += e * e;
        }
      }
      m2 = row_sum2(make_float2(m2, 0.f), t, tpr, 1, red, phase).x;
      rstd = 1.f / sqrtf(m2 / static_cast<float>(d) + a.eps);
    }
    for (int c = 0; c < chunks; ++c) {
      float v[8];
      stream(c, v);
      if (z != nullptr) store_chunk<T, VEC>(z, narrow<T>(v), c, t, tpr, d);
      if (a.ck.q != nullptr)
        ckpt_store_chunk<T, VEC>(v, a.ck.q + row * a.ck.ldq, a.ck.ex + row * a.ck.lde, c, t, tpr,
                                 d);
      if (live) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int col = chunk_col<VEC>(c, j, t, tpr);
          if (col >= d) continue;
          const float w = a.weight != nullptr ? load_param(a.weight, a.wtype, col) : 1.f;
          const float b = a.bias != nullptr ? load_param(a.bias, a.wtype, col) : 0.f;
          v[j] = (v[j] - mean) * rstd * w + b;
        }
      }
      store_chunk<T, VEC>(y, narrow<T>(v), c, t, tpr, d);
    }
    if (t == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
  }
}

// One chunk of the stream for the backward pass, as loaded.
template <typename T, bool VEC, bool CK>
struct RawStream {
  Raw8<T> r;
  __device__ __forceinline__ void load(const NormBwdArgs& a, long long row, int c, int t, int tpr) {
    r = load_chunk<T, VEC>(static_cast<const T*>(a.x) + row * a.ldx, c, t, tpr, a.d);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const { widen(r, v); }
};
template <typename T, bool VEC>
struct RawStream<T, VEC, true> {
  RawCkpt<VEC> r;
  __device__ __forceinline__ void load(const NormBwdArgs& a, long long row, int c, int t, int tpr) {
    r = ckpt_load_chunk<VEC>(a.ck.q + row * a.ck.ldq, a.ck.ex + row * a.ck.lde, c, t, tpr, a.d);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const { ckpt_widen<VEC>(r, v); }
};

// dx, and this CTA's sums over its rows for dw (and db), which each thread
// keeps in registers for its own columns: the rows' order is fixed by the grid,
// so the sums are the same on every run.
template <typename T, bool VEC, int CH, bool CK, bool DB>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormBwdArgs a) {
  __shared__ float2 red[8][2 * 32];
  extern __shared__ float col_sums[];  // [d], [d] when the CTA has several rows in flight
  const int t = threadIdx.x, tpr = blockDim.x, g = threadIdx.y, d = a.d;
  int phase = 0;
  float w[CH][8], dw[CH][8], db[DB ? CH : 1][8];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = chunk_col<VEC>(c, j, t, tpr);
      w[c][j] = a.weight != nullptr && col < d ? load_param(a.weight, a.wtype, col) : 1.f;
      dw[c][j] = 0.f;
      if (DB) db[DB ? c : 0][j] = 0.f;
    }
  const T* dy = static_cast<const T*>(a.dy);
  const T* dres = static_cast<const T*>(a.dres);
  T* dx = static_cast<T*>(a.dx);
  const long long step = static_cast<long long>(gridDim.x) * blockDim.y;
  long long row = static_cast<long long>(blockIdx.x) * blockDim.y + g;
  bool live = row_live(a.mask, row, a.n);
  bool live1 = row_live(a.mask, row + step, a.n);
  const float inv_d = 1.f / static_cast<float>(d);
  Raw8<T> ry[CH], rr[CH];
  RawStream<T, VEC, CK> rx[CH];
  float mean = 0.f, rstd = 0.f;
  const auto fetch = [&](long long r) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      ry[c] = load_chunk<T, VEC>(dy + r * a.lddy, c, t, tpr, d);
      rx[c].load(a, r, c, t, tpr);
      if (dres != nullptr) rr[c] = load_chunk<T, VEC>(dres + r * a.lddres, c, t, tpr, d);
    }
    rstd = a.rstd[r];
    mean = a.kind != GRPO_NORM_RMS ? a.mean[r] : 0.f;
  };
  if (live) fetch(row);
  for (; row < a.n; row += step) {
    const bool live2 = row_live(a.mask, row + 2 * step, a.n);
    if (!live) {
      const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < CH; ++c)
        store_chunk<T, VEC>(dx + row * a.lddx, narrow<T>(zero), c, t, tpr, d);
      if (live1) fetch(row + step);
    } else {
      float u[CH][8], h[CH][8];
      Raw8<T> cur_res[CH];
      float2 s = make_float2(0.f, 0.f);
      const float rs = rstd;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        widen(ry[c], u[c]);
        rx[c].get(h[c]);
        if (dres != nullptr) cur_res[c] = rr[c];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          h[c][j] = (h[c][j] - mean) * rs;
          dw[c][j] += u[c][j] * h[c][j];
          if (DB) db[DB ? c : 0][j] += u[c][j];
          u[c][j] *= w[c][j];
          s.x += u[c][j];
          s.y += u[c][j] * h[c][j];
        }
      }
      if (live1) fetch(row + step);
      s = row_sum2(s, t, tpr, g + 1, red[g], phase);
      const float c1 = a.kind != GRPO_NORM_RMS ? s.x * inv_d : 0.f;
      const float c2 = s.y * inv_d;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) u[c][j] = rs * (u[c][j] - c1 - h[c][j] * c2);
        if (dres != nullptr) {
          float r[8];
          widen(cur_res[c], r);
#pragma unroll
          for (int j = 0; j < 8; ++j) u[c][j] += r[j];
        }
        store_chunk<T, VEC>(dx + row * a.lddx, narrow<T>(u[c]), c, t, tpr, d);
      }
    }
    live = live1;
    live1 = live2;
  }
  if (a.dweight == nullptr && !DB) return;
  // The CTA's rows in flight, added in their order.
  if (blockDim.y > 1) {
    float* sw = col_sums;
    float* sb = col_sums + d;
    for (int k = 0; k < static_cast<int>(blockDim.y); ++k) {
      if (g == k) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int col = chunk_col<VEC>(c, j, t, tpr);
            if (col < d) {
              sw[col] = k == 0 ? dw[c][j] : sw[col] + dw[c][j];
              if (DB) sb[col] = k == 0 ? db[DB ? c : 0][j] : sb[col] + db[DB ? c : 0][j];
            }
          }
      }
      __syncthreads();
    }
    float* pw = a.partials + static_cast<long long>(blockIdx.x) * d;
    float* pb = pw + static_cast<long long>(gridDim.x) * d;
    for (int col = g * tpr + t; col < d; col += tpr * blockDim.y) {
      pw[col] = sw[col];
      if (DB) pb[col] = sb[col];
    }
  } else {
    float* pw = a.partials + static_cast<long long>(blockIdx.x) * d;
    float* pb = pw + static_cast<long long>(gridDim.x) * d;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int col = chunk_col<VEC>(c, j, t, tpr);
        if (col < d) {
          pw[col] = dw[c][j];
          if (DB) pb[col] = db[DB ? c : 0][j];
        }
      }
  }
}

// The aligned form of norm_bwd_kernel, its rows in flight as in
// norm_fwd_ring_kernel. A slot holds dy, then x (or its bytes and exponents),
// then dres. FULL: layer norm, or a bias gradient; else neither.
template <typename T, int CH, bool CK, bool FULL>
__global__ void __launch_bounds__(ring_threads(CH)) norm_bwd_ring_kernel(const NormBwdArgs a, const Ring ring) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float red[kMaxRows][2 * 2 * 16];
  const int t = threadIdx.x, tpr = blockDim.x, g = threadIdx.y, d = a.d;
  const int warps = tpr >> 5;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem) + g * kMaxSlots;
  float* const sw = reinterpret_cast<float*>(smem + kRingBars);
  uint8_t* const ring0 = reinterpret_cast<uint8_t*>(sw + (a.weight != nullptr ? d : 0));
  const uint32_t sw32 = smem_u32(sw);
  const uint32_t rows0 = smem_u32(ring0) + g * ring.slots * ring.row_bytes;
  const uint32_t t_bytes = d * sizeof(T);
  const uint32_t q_bytes = static_cast<uint32_t>(a.ck.ldq), e_bytes = static_cast<uint32_t>(a.ck.lde);
  const uint32_t x_bytes = CK ? q_bytes + e_bytes : t_bytes;  // rows of 16 bytes
  const bool res = a.dres != nullptr, layer = FULL && a.kind == GRPO_NORM_LAYER;
  const long long step = static_cast<long long>(gridDim.x) * blockDim.y;
  const long long row0 = static_cast<long long>(blockIdx.x) * blockDim.y + g;
  const int count = row_count(row0, a.n, step);
  const uint8_t* const mask = a.mask;
  uint32_t pending = 0;
  int fetched = 0;
  const auto fetch = [&](int slot) {
    if (fetched >= count) return;
    const long long r = row0 + step * fetched++;
    if (mask != nullptr && mask[r] == 0) return;
    pending |= 1u << slot;
    const uint32_t dst = rows0 + slot * ring.row_bytes;
    mbar_arrive_expect_tx(&bars[slot], t_bytes + x_bytes + (res ? t_bytes : 0));
    bulk_load(dst, static_cast<const T*>(a.dy) + r * a.lddy, t_bytes, &bars[slot]);
    if (CK) {
      bulk_load(dst + t_bytes, a.ck.q + r * a.ck.ldq, q_bytes, &bars[slot]);
      bulk_load(dst + t_bytes + q_bytes, a.ck.ex + r * a.ck.lde, e_bytes, &bars[slot]);
    } else {
      bulk_load(dst + t_bytes, static_cast<const T*>(a.x) + r * a.ldx, t_bytes, &bars[slot]);
    }
    if (res)
      bulk_load(dst + t_bytes + x_bytes, static_cast<const T*>(a.dres) + r * a.lddres, t_bytes,
                &bars[slot]);
  };
  if (t == 0) {
    for (int s = 0; s < ring.slots; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
    for (int s = 0; s < ring.slots; ++s) fetch(s);
  }
  for (int k = t; k < 2 * 2 * 16; k += tpr) red[g][k] = 0.f;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (a.weight != nullptr) stage_param(sw, a.weight, a.wtype, d, g * tpr + t, tpr * blockDim.y);
  __syncthreads();

  f32x2 dw[CH][4], db[FULL ? CH : 1][4];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      dw[c][j] = 0ull;
      if (FULL) db[FULL ? c : 0][j] = 0ull;
    }
  const float inv_d = 1.f / static_cast<float>(d);
  T* dx = static_cast<T*>(a.dx) + row0 * a.lddx;
  int phase = 0, slot = 0;
  uint32_t parity = 0;
  bool ok = true;
  bool live = count > 0 && (mask == nullptr || mask[row0] != 0);
  float rstd1 = live ? a.rstd[row0] : 0.f;
  float mean1 = live && layer ? a.mean[row0] : 0.f;
  for (int i = 0; i < count; ++i) {
    const long long next = row0 + step * (i + 1);
    const bool live1 = i + 1 < count && (mask == nullptr || mask[next] != 0);
    const float rstd = rstd1, mean = mean1;
    rstd1 = live1 ? a.rstd[next] : 0.f;
    mean1 = live1 && layer ? a.mean[next] : 0.f;
    if (!live) {
      const f32x2 zero[4] = {0ull, 0ull, 0ull, 0ull};
      if (t == 0 && ok) fetch(slot);
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if ((c * tpr + t) * 8 < d) store_raw(dx + (c * tpr + t) * 8, narrow2<T>(zero));
    } else {
      ok = ok && row_wait(&bars[slot], (parity >> slot) & 1u);
      if (ok) {
        parity ^= 1u << slot;
        pending &= ~(1u << slot);
      }
      const uint32_t src = rows0 + slot * ring.row_bytes;
      const f32x2 scale = pair(rstd, rstd), shift = pair(-mean, -mean);
      f32x2 u[CH][4], h[CH][4];
      Raw8<T> rr[CH];
      f32x2 su = 0ull, suh = 0ull;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int at = c * tpr + t;
        if (8 * at >= d) continue;
        const uint32_t off = at * sizeof(Raw8<T>);
        widen2(lds_raw<T>(src + off), u[c]);
        if (CK) {
          ckpt_widen2(lds_v2(src + t_bytes + 8 * at),
                      ckpt_factor(lds_u8(src + t_bytes + q_bytes + at / 4)), h[c]);
        } else {
          widen2(lds_raw<T>(src + t_bytes + off), h[c]);
        }
        if (res) rr[c] = lds_raw<T>(src + t_bytes + x_bytes + off);
        f32x2 w[4];
        if (a.weight != nullptr) read_param(sw32, at, 2 * d, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (FULL) h[c][j] = add2(h[c][j], shift);
          h[c][j] = mul2(h[c][j], scale);
          dw[c][j] = fma2(u[c][j], h[c][j], dw[c][j]);
          if (FULL) db[FULL ? c : 0][j] = add2(u[c][j], db[FULL ? c : 0][j]);
          if (a.weight != nullptr) u[c][j] = mul2(u[c][j], w[j]);
          if (FULL) su = add2(u[c][j], su);
          suh = fma2(u[c][j], h[c][j], suh);
        }
      }
      float s[FULL ? 2 : 1];
      s[0] = warp_sum(sum_of(suh));
      if (FULL) s[FULL ? 1 : 0] = warp_sum(sum_of(su));
      join_warps(s, t, warps, g + 1, red[g], phase);
      if (t == 0 && ok) fetch(slot);
      const float c1 = layer ? s[FULL ? 1 : 0] * inv_d : 0.f;
      const float c2 = ok ? s[0] * inv_d : __uint_as_float(0x7fc00000u);
      const f32x2 n1 = pair(-c1, -c1), n2 = pair(-c2, -c2);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int at = c * tpr + t;
        if (8 * at >= d) continue;
        f32x2 r[4] = {0ull, 0ull, 0ull, 0ull};
        if (res) widen2(rr[c], r);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (FULL) u[c][j] = add2(u[c][j], n1);
          u[c][j] = fma2(fma2(h[c][j], n2, u[c][j]), scale, r[j]);
        }
        store_raw(dx + 8 * at, narrow2<T>(u[c]));
      }
      if (!ok) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            dw[c][j] = ~0ull;  // NaN
            if (FULL) db[FULL ? c : 0][j] = ~0ull;
          }
      }
    }
    if (++slot == ring.slots) slot = 0;
    dx += step * a.lddx;
    live = live1;
  }
  land(bars, ring.slots, parity, pending);
  const bool want_db = FULL && a.dbias != nullptr;
  if (a.dweight == nullptr && !want_db) return;
  // The CTA's rows in flight, added in their order; the rings have been read.
  float* const cw = blockDim.y > 1 ? reinterpret_cast<float*>(ring0) : nullptr;
  float* const cb = cw != nullptr ? cw + d : nullptr;
  float* pw = a.partials + static_cast<long long>(blockIdx.x) * d;
  float* pb = pw + static_cast<long long>(gridDim.x) * d;
  if (cw == nullptr) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int at = c * tpr + t;
      if (8 * at >= d) continue;
      store_raw(pw + 8 * at, narrow2<float>(dw[c]));
      if (want_db) store_raw(pb + 8 * at, narrow2<float>(db[FULL ? c : 0]));
    }
    return;
  }
  __syncthreads();
  for (int k = 0; k < static_cast<int>(blockDim.y); ++k) {
    if (g == k) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int at = c * tpr + t;
        if (8 * at >= d) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f32x2* pc = reinterpret_cast<f32x2*>(cw + 8 * at + 2 * j);
          *pc = k == 0 ? dw[c][j] : add2(*pc, dw[c][j]);
          if (want_db) {
            f32x2* pd = reinterpret_cast<f32x2*>(cb + 8 * at + 2 * j);
            *pd = k == 0 ? db[FULL ? c : 0][j] : add2(*pd, db[FULL ? c : 0][j]);
          }
        }
      }
    }
    __syncthreads();
  }
  for (int col = g * tpr + t; col < d; col += tpr * blockDim.y) {
    pw[col] = cw[col];
    if (want_db) pb[col] = cb[col];
  }
}

// Rows beyond kNormRegisterRow columns: dx in two walks over the row.
template <typename T, bool VEC, bool CK>
__global__ void __launch_bounds__(512) norm_bwd_long_kernel(const NormBwdArgs a) {
  __shared__ float2 red[2 * 32];
  const int t = threadIdx.x, tpr = blockDim.x, d = a.d;
  const int chunks = (d + 8 * tpr - 1) / (8 * tpr);
  int phase = 0;
  for (long long row = blockIdx.x; row < a.n; row += gridDim.x) {
    T* dx = static_cast<T*>(a.dx) + row * a.lddx;
    const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
    const bool live = row_live(a.mask, row, a.n);
    float u[8], h[8];
    float2 s = make_float2(0.f, 0.f);
    const float rs = live ? a.rstd[row] : 0.f;
    const float mean = live && a.kind != GRPO_NORM_RMS ? a.mean[row] : 0.f;
    const auto terms = [&](int c) {
      RawStream<T, VEC, CK> rx;
      rx.load(a, row, c, t, tpr);
      rx.get(h);
      widen(load_chunk<T, VEC>(dy, c, t, tpr, d), u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int col = chunk_col<VEC>(c, j, t, tpr);
        h[j] = (h[j] - mean) * rs;
        if (col < d && a.weight != nullptr) u[j] *= load_param(a.weight, a.wtype, col);
      }
    };
    if (live) {
      for (int c = 0; c < chunks; ++c) {
        terms(c);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s.x += u[j];
          s.y += u[j] * h[j];
        }
      }
      s = row_sum2(s, t, tpr, 1, red, phase);
    }
    const float c1 = a.kind != GRPO_NORM_RMS ? s.x / static_cast<float>(d) : 0.f;
    const float c2 = s.y / static_cast<float>(d);
    for (int c = 0; c < chunks; ++c) {
      if (live) {
        terms(c);
        float r[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (a.dres != nullptr)
          widen(load_chunk<T, VEC>(static_cast<const T*>(a.dres) + row * a.lddres, c, t, tpr, d), r);
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = rs * (u[j] - c1 - h[j] * c2) + r[j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = 0.f;
      }
      store_chunk<T, VEC>(dx, narrow<T>(u), c, t, tpr, d);
    }
  }
}

// The weight gradients of such rows, before dx is written (dx may lie on dy):
// a CTA takes 8 x 32 columns (VEC) or 32 x 8 and every gridDim.y-th group of 8
// rows, one row to each of its 8 warps.
template <typename T, bool VEC, bool CK>
__global__ void __launch_bounds__(256) norm_bwd_cols_kernel(const NormBwdArgs a) {
  __shared__ float sh[2][8][256];
  const int t = threadIdx.x, g = threadIdx.y, d = a.d;
  const int first = blockIdx.x * 256;  // columns [first, first + 256)
  float dw[8], db[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[j] = db[j] = 0.f;
  const int dd = min(d - first, 256);
  const T* dy = static_cast<const T*>(a.dy) + first;
  NormBwdArgs s = a;  // the same rows, from this column on
  s.d = dd;
  if (CK) {
    s.ck.q += first;
    s.ck.ex += first / kCkptBlock;
  } else {
    s.x = static_cast<const T*>(a.x) + first;
  }
  for (long long row = static_cast<long long>(blockIdx.y) * 8 + g; row < a.n;
       row += static_cast<long long>(gridDim.y) * 8) {
    if (!row_live(a.mask, row, a.n)) continue;
    float u[8], h[8];
    widen(load_chunk<T, VEC>(dy + row * a.lddy, 0, t, 32, dd), u);
    RawStream<T, VEC, CK> rx;
    rx.load(s, row, 0, t, 32);
    rx.get(h);
    const float rs = a.rstd[row];
    const float mean = a.kind != GRPO_NORM_RMS ? a.mean[row] : 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dw[j] += u[j] * ((h[j] - mean) * rs);
      db[j] += u[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int col = chunk_col<VEC>(0, j, t, 32);
    sh[0][g][col] = dw[j];
    sh[1][g][col] = db[j];
  }
  __syncthreads();
  const int col = g * 32 + t;
  if (col >= dd) return;
  float w = 0.f, b = 0.f;
  for (int k = 0; k < 8; ++k) {
    w += sh[0][k][col];
    b += sh[1][k][col];
  }
  a.partials[static_cast<long long>(blockIdx.y) * d + first + col] = w;
  if (a.dbias != nullptr)
    a.partials[static_cast<long long>(gridDim.y + blockIdx.y) * d + first + col] = b;
}

// dw and db from the CTAs' partial sums: 32 columns a CTA, the partial rows
// dealt to its 16 warps, whose sums are added in warp order. Launched while the
// backward kernel still runs (it waits for its end here): 3 us less a call.
__global__ void __launch_bounds__(512) norm_bwd_finish_kernel(const float* __restrict__ partials,
                                                              int rows, int d, float* dweight,
                                                              float* dbias, const float* add_dw,
                                                              const float* add_db) {
  __shared__ float sh[16][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const bool bias = blockIdx.y == 1;
  const float* p = partials + (bias ? static_cast<long long>(rows) * d : 0);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float s = 0.f;
  if (col < d) {
#pragma unroll 8
    for (int r = g; r < rows; r += 16) s += p[static_cast<long long>(r) * d + col];
  }
  sh[g][lane] = s;
  __syncthreads();
  if (g != 0 || col >= d) return;
  for (int k = 1; k < 16; ++k) s += sh[k][lane];
  const float* add = bias ? add_db : add_dw;
  float* out = bias ? dbias : dweight;
  if (out != nullptr) out[col] = add != nullptr ? add[col] + s : s;
}

// Threads of a row and rows of a CTA for D columns held in registers.
struct RowShape {
  int tpr, rows, ch;
};
// One by one: 16 values a thread (8 up to 256 columns).
RowShape row_shape(int d) {
  RowShape s;
  s.ch = d <= 256 ? 1 : 2;
  const int per = 8 * s.ch;
  s.tpr = (d + per * 32 - 1) / (per * 32) * 32;
  s.rows = s.tpr >= kRowThreads ? 1 : kRowThreads / s.tpr;
  return s;
}
// Aligned: the most values a thread, up to 8 `most`, that leave no more than a
// tenth of the threads idle (else the fewest idle ones); CTAs of about
// `threads` threads.
RowShape ring_shape(int d, int most, int threads) {
  RowShape best = {0, 0, 0};
  int best_room = 0;
  for (int ch = most; ch >= 1; --ch) {
    const int tpr = (d + 256 * ch - 1) / (256 * ch) * 32;
    const int room = tpr * 8 * ch;
    if (tpr > 512 || (best.ch != 0 && room >= best_room)) continue;
    best = {tpr, std::min(kMaxRows, std::max(1, threads / tpr)), ch};
    best_room = room;
    if (10 * room <= 11 * d) break;
  }
  return best;
}

// CTAs of `threads` threads resident on the device, looked up once per kernel.
template <auto Kernel>
int resident(int threads, size_t smem, int sms) {
  static std::atomic<int> known[33];
  std::atomic<int>& k = known[threads / 32];
  int n = k.load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, Kernel, threads, smem) != cudaSuccess ||
        n < 1)
      n = 1;
    k.store(n, std::memory_order_relaxed);
  }
  return n * sms;
}

constexpr size_t kSmemMax = 227 * 1024 - 8192;  // less the kernels' static arrays
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
  return r;
}

// Opts a kernel in to large shared memory, once.
template <auto Kernel>
bool opted_in() {
  static const bool ok = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              static_cast<int>(kSmemMax)) == cudaSuccess;
  return ok;
}

template <auto Kernel>
cudaError_t ctas_per_sm(int threads, size_t smem, int* n) {
  if (!opted_in<Kernel>()) return cudaErrorInvalidValue;
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, Kernel, threads, smem);
}

template <typename T, int CH, int KIND>
cudaError_t fwd_ring(const NormFwdArgs& a, const RowShape& s, int sms, cudaStream_t st) {
  constexpr auto kernel = norm_fwd_ring_kernel<T, CH, KIND>;
  const size_t fixed = kRingBars + sizeof(float) * a.d *
                                       ((a.weight != nullptr) + (a.bias != nullptr));
  const Ring ring = make_ring(a.d * sizeof(T) * (a.res != nullptr ? 2 : 1), s.rows, fixed);
  const size_t smem = fixed + static_cast<size_t>(ring.slots) * ring.row_bytes * s.rows;
  int per_sm = 0;
  cudaError_t e = ctas_per_sm<kernel>(s.tpr * s.rows, smem, &per_sm);
  if (e != cudaSuccess) return e;
  const long long units = (a.n + s.rows - 1) / s.rows;
  const int grid = static_cast<int>(std::min<long long>(units, std::max(1, per_sm) * sms));
  LaunchTimer timer("norm_fwd_kernel", st);
  kernel<<<grid, dim3(s.tpr, s.rows), smem, st>>>(a, ring);
  return cudaGetLastError();
}

template <typename T, int KIND>
cudaError_t fwd_aligned(const NormFwdArgs& a, int sms, cudaStream_t st) {
  const RowShape s = ring_shape(a.d, 4, kRowThreads);
  switch (s.ch) {
    case 1: return fwd_ring<T, 1, KIND>(a, s, sms, st);
    case 2: return fwd_ring<T, 2, KIND>(a, s, sms, st);
    case 3: return fwd_ring<T, 3, KIND>(a, s, sms, st);
    default: return fwd_ring<T, 4, KIND>(a, s, sms, st);
  }
}

template <typename T, bool VEC, int CH>
cudaError_t fwd(const NormFwdArgs& a, const RowShape& s, int sms, cudaStream_t st) {
  constexpr auto kernel = norm_fwd_kernel<T, VEC, CH>;
  const long long units = (a.n + s.rows - 1) / s.rows;
  const int grid = static_cast<int>(
      std::min<long long>(units, resident<kernel>(s.tpr * s.rows, 0, sms)));
  LaunchTimer timer("norm_fwd_kernel", st);
  kernel<<<grid, dim3(s.tpr, s.rows), 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T, bool VEC>
cudaError_t fwd_any(const NormFwdArgs& a, int sms, cudaStream_t st) {
  if (a.d > kNormRegisterRow) {
    const int grid = static_cast<int>(std::min<long long>(a.n, 3LL * sms));
    LaunchTimer timer("norm_fwd_long_kernel", st);
    norm_fwd_long_kernel<T, VEC><<<grid, 512, 0, st>>>(a);
    return cudaGetLastError();
  }
  if constexpr (VEC) {
    return a.kind == GRPO_NORM_RMS ? fwd_aligned<T, GRPO_NORM_RMS>(a, sms, st)
                                   : fwd_aligned<T, GRPO_NORM_LAYER>(a, sms, st);
  } else {
    const RowShape s = row_shape(a.d);
    return s.ch == 1 ? fwd<T, false, 1>(a, s, sms, st) : fwd<T, false, 2>(a, s, sms, st);
  }
}

cudaError_t finish(const NormBwdArgs& a, int rows, cudaStream_t st) {
  if (a.dweight == nullptr && a.dbias == nullptr) return cudaSuccess;
  const dim3 grid((a.d + 31) / 32, a.dbias != nullptr ? 2 : 1);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(512);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  LaunchTimer timer("norm_bwd_finish_kernel", st);
  return cudaLaunchKernelEx(&cfg, norm_bwd_finish_kernel, static_cast<const float*>(a.partials), rows,
                            a.d, a.dweight, a.dbias, a.add_dweight, a.add_dbias);
}

template <typename T, int CH, bool CK, bool FULL>
cudaError_t bwd_ring(const NormBwdArgs& a, const RowShape& s, int sms, cudaStream_t st) {
  constexpr auto kernel = norm_bwd_ring_kernel<T, CH, CK, FULL>;
  const size_t fixed = kRingBars + (a.weight != nullptr ? sizeof(float) * a.d : 0);
  const uint32_t t_bytes = a.d * sizeof(T);
  const Ring ring =
      make_ring(t_bytes * (a.dres != nullptr ? 2 : 1) +
                    (CK ? static_cast<uint32_t>(a.ck.ldq + a.ck.lde) : t_bytes),
                s.rows, fixed);
  size_t smem = static_cast<size_t>(ring.slots) * ring.row_bytes * s.rows;
  if (s.rows > 1) smem = std::max(smem, static_cast<size_t>(a.d) * 8);
  smem += fixed;
  int per_sm = 0;
  cudaError_t e = ctas_per_sm<kernel>(s.tpr * s.rows, smem, &per_sm);
  if (e != cudaSuccess) return e;
  const long long units = (a.n + s.rows - 1) / s.rows;
  const int grid = static_cast<int>(std::min<long long>(
      std::min<long long>(units, kNormMaxPartials), std::max(1, per_sm) * sms));
  {
    LaunchTimer timer("norm_bwd_kernel", st);
    kernel<<<grid, dim3(s.tpr, s.rows), smem, st>>>(a, ring);
  }
  e = cudaGetLastError();
  return e != cudaSuccess ? e : finish(a, grid, st);
}

template <typename T, bool CK, bool FULL>
cudaError_t bwd_aligned(const NormBwdArgs& a, int sms, cudaStream_t st) {
  const RowShape s = ring_shape(a.d, 2, kRowThreads);
  switch (s.ch) {
    case 1: return bwd_ring<T, 1, CK, FULL>(a, s, sms, st);
    default: return bwd_ring<T, 2, CK, FULL>(a, s, sms, st);
  }
}

template <typename T, bool VEC, int CH, bool CK, bool DB>
cudaError_t bwd(const NormBwdArgs& a, const RowShape& s, int sms, cudaStream_t st) {
  constexpr auto kernel = norm_bwd_kernel<T, VEC, CH, CK, DB>;
  const long long units = (a.n + s.rows - 1) / s.rows;
  const size_t smem = s.rows > 1 ? static_cast<size_t>(a.d) * (DB ? 8 : 4) : 0;
  // Occupancy is asked for the largest such buffer (rows > 1: at most 2048 columns).
  const int grid = static_cast<int>(std::min<long long>(
      std::min<long long>(units, kNormMaxPartials),
      resident<kernel>(s.tpr * s.rows, s.rows > 1 ? 2048 * 8 : 0, sms)));
  {
    LaunchTimer timer("norm_bwd_kernel", st);
    kernel<<<grid, dim3(s.tpr, s.rows), smem, st>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : finish(a, grid, st);
}

template <typename T, bool VEC, bool CK>
cudaError_t bwd_any(const NormBwdArgs& a, int sms, cudaStream_t st) {
  if (a.d > kNormRegisterRow) {
    const int slabs = (a.d + 255) / 256;
    const int groups = norm_bwd_partials(a.n, a.d);
    if (a.dweight != nullptr || a.dbias != nullptr) {
      LaunchTimer timer("norm_bwd_cols_kernel", st);
      norm_bwd_cols_kernel<T, VEC, CK><<<dim3(slabs, groups), dim3(32, 8), 0, st>>>(a);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    {
      LaunchTimer timer("norm_bwd_long_kernel", st);
      const int grid = static_cast<int>(std::min<long long>(a.n, 3LL * sms));
      norm_bwd_long_kernel<T, VEC, CK><<<grid, 512, 0, st>>>(a);
    }
    e = cudaGetLastError();
    return e != cudaSuccess ? e : finish(a, groups, st);
  }
  const bool db = a.dbias != nullptr;
  if constexpr (VEC) {
    return db || a.kind == GRPO_NORM_LAYER ? bwd_aligned<T, CK, true>(a, sms, st)
                                           : bwd_aligned<T, CK, false>(a, sms, st);
  } else {
    const RowShape s = row_shape(a.d);
    if (s.ch == 1)
      return db ? bwd<T, false, 1, CK, true>(a, s, sms, st)
                : bwd<T, false, 1, CK, false>(a, s, sms, st);
    return db ? bwd<T, false, 2, CK, true>(a, s, sms, st)
              : bwd<T, false, 2, CK, false>(a, s, sms, st);
  }
}

template <typename T>
cudaError_t bwd_typed(const NormBwdArgs& a, bool vec, int sms, cudaStream_t st) {
  if (a.x != nullptr)
    return vec ? bwd_any<T, true, false>(a, sms, st) : bwd_any<T, false, false>(a, sms, st);
  return vec ? bwd_any<T, true, true>(a, sms, st) : bwd_any<T, false, true>(a, sms, st);
}

}  // namespace

int norm_bwd_partials(long long n, int d) {
  if (d > kNormRegisterRow) {
    // Row groups of norm_bwd_cols_kernel: 8 CTAs an SM.
    return static_cast<int>(std::min<long long>(std::max(1, 8 * 152 / ((d + 255) / 256)),
                                                std::max<long long>(1, (n + 7) / 8)));
  }
  // A CTA takes one row at least.
  return static_cast<int>(std::min<long long>(kNormMaxPartials, std::max<long long>(1, n)));
}

cudaError_t launch_norm_fwd(const NormFwdArgs& a, int dtype, bool vec, int sms, cudaStream_t st) {
  switch (dtype) {
    case GRPO_DTYPE_BF16:
      return vec ? fwd_any<__nv_bfloat16, true>(a, sms, st)
                 : fwd_any<__nv_bfloat16, false>(a, sms, st);
    case GRPO_DTYPE_FP16:
      return vec ? fwd_any<__half, true>(a, sms, st) : fwd_any<__half, false>(a, sms, st);
    default:
      return vec ? fwd_any<float, true>(a, sms, st) : fwd_any<float, false>(a, sms, st);
  }
}

cudaError_t launch_norm_bwd(const NormBwdArgs& a, int dtype, bool vec, int sms, cudaStream_t st) {
  if (a.n == 0) return finish(a, 0, st);
  switch (dtype) {
    case GRPO_DTYPE_BF16: return bwd_typed<__nv_bfloat16>(a, vec, sms, st);
    case GRPO_DTYPE_FP16: return bwd_typed<__half>(a, vec, sms, st);
    default: return bwd_typed<float>(a, vec, sms, st);
  }
}

}  // namespace grpo
