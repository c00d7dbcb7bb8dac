// Row-wise building blocks shared by the norm and the activation checkpoint
// kernels: a thread's share of a row, loads and stores of 8 values at a time,
// sums over the threads of a row, and the 8-bit checkpoint format.
//
// A row of D values is spread over `tpr` threads (a multiple of 32); thread t
// holds chunks of 8 values. Where every row starts on 16 bytes and D % 8 == 0
// (VEC), chunk c of thread t is the 8 consecutive columns from (c tpr + t) 8.
// Otherwise its value j is column (8 c + j) tpr + t, loaded one by one: any D,
// stride and alignment. In both, the 32 columns of a checkpoint block are held
// by one warp: by 4 neighbouring lanes (VEC), or one column to a lane.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cstdint>

#include "ptx.cuh"

namespace grpo {

constexpr int kCkptBlock = 32;     // columns that share a power of two
constexpr int kCkptMinExp = -117;  // 2^-117 2^-9 is a normal bf16: every value
                                   // of the format expands to bf16 exactly
constexpr int kCkptBias = 127;

constexpr uint8_t kCkptNaN = 0x7f;  // an e4m3 NaN
constexpr float kNaN = __builtin_nanf("");

template <typename T>
struct alignas(16) Raw8 {
  T e[8];
};

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  return static_cast<float>(v);
}

// Two values rounded to T, to nearest even.
__device__ __forceinline__ void from_f32x2(float a, float b, __nv_bfloat16* o) {
  *reinterpret_cast<__nv_bfloat162*>(o) = __floats2bfloat162_rn(a, b);
}
__device__ __forceinline__ void from_f32x2(float a, float b, __half* o) {
  *reinterpret_cast<__half2*>(o) = __floats2half2_rn(a, b);
}
__device__ __forceinline__ void from_f32x2(float a, float b, float* o) {
  o[0] = a;
  o[1] = b;
}

template <bool VEC>
__device__ __forceinline__ int chunk_col(int c, int j, int t, int tpr) {
  return VEC ? (c * tpr + t) * 8 + j : (c * 8 + j) * tpr + t;
}

// Chunk c of this thread's share of a row; zeros past column d.
template <typename T, bool VEC>
__device__ __forceinline__ Raw8<T> load_chunk(const T* row, int c, int t, int tpr, int d) {
  Raw8<T> r;
  if (VEC) {
    const int col = chunk_col<true>(c, 0, t, tpr);
    uint4* w = reinterpret_cast<uint4*>(&r);
    if (col < d) {
      const uint4* p = reinterpret_cast<const uint4*>(row + col);
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(r) / 16); ++i) w[i] = p[i];
    } else {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(r) / 16); ++i) w[i] = make_uint4(0, 0, 0, 0);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = chunk_col<false>(c, j, t, tpr);
      r.e[j] = col < d ? row[col] : T(0.f);
    }
  }
  return r;
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_chunk(T* row, const Raw8<T>& r, int c, int t, int tpr,
                                            int d) {
  if (VEC) {
    const int col = chunk_col<true>(c, 0, t, tpr);
    if (col < d) {
      uint4* p = reinterpret_cast<uint4*>(row + col);
      const uint4* w = reinterpret_cast<const uint4*>(&r);
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(r) / 16); ++i) p[i] = w[i];
    }
  } else if (8 * (c + 1) * tpr <= d) {  // the whole row's chunk
    T* p = row + 8 * c * tpr + t;
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j * tpr] = r.e[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = chunk_col<false>(c, j, t, tpr);
      if (col < d) row[col] = r.e[j];
    }
  }
}

template <typename T>
__device__ __forceinline__ void widen(const Raw8<T>& r, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = to_f32(r.e[j]);
}

template <typename T>
__device__ __forceinline__ Raw8<T> narrow(const float (&v)[8]) {
  Raw8<T> r;
#pragma unroll
  for (int j = 0; j < 8; j += 2) from_f32x2(v[j], v[j + 1], &r.e[j]);
  return r;
}

// A weight or bias of either type; `type` is a grpo_dtype.
__device__ __forceinline__ float load_param(const void* p, int type, int col) {
  if (type == GRPO_DTYPE_FP32) return static_cast<const float*>(p)[col];
  if (type == GRPO_DTYPE_BF16) return to_f32(static_cast<const __nv_bfloat16*>(p)[col]);
  return to_f32(static_cast<const __half*>(p)[col]);
}

__device__ __forceinline__ float2 warp_sum2(float2 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Sum of a pair over the `tpr` threads of a row, given to all of them, in a
// fixed order. tpr == 32: shuffles alone. Otherwise one named barrier (`bar`,
// 1-15) of the row's threads; `sh` holds 2 x 32 pairs, used in turn (`phase`).
__device__ __forceinline__ float2 row_sum2(float2 v, int t, int tpr, int bar, float2* sh,
                                           int& phase) {
  v = warp_sum2(v);
  if (tpr == 32) return v;
  float2* s = sh + phase * 32;
  phase ^= 1;
  if ((t & 31) == 0) s[t >> 5] = v;
  named_barrier(bar, tpr);
  const int lane = t & 31;
  return warp_sum2(lane < (tpr >> 5) ? s[lane] : make_float2(0.f, 0.f));
}

// ------------------------------------------------------- rows in flight ----
// Rows come to shared memory by bulk copies, several rows ahead: the bytes in
// flight do not cost registers.

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Waits for a phase of `bar`; false after about a second, then after `gave_up()`
// (no status word here: the caller gives NaN).
template <typename F>
__device__ __forceinline__ bool row_wait(uint64_t* bar, uint32_t parity, F gave_up,
                                         long long limit = kWaitLimitCycles) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > limit) {
      gave_up();
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool row_wait(uint64_t* bar, uint32_t parity) {
  return row_wait(bar, parity, [] {});
}

// Two fp32 in one 64-bit register: Blackwell multiplies and adds them with one
// instruction, and these kernels are near the issue limit.
using f32x2 = unsigned long long;

__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float sum_of(f32x2 v) {
  float a, b;
  split(v, a, b);
  return a + b;
}

// 8 values of a chunk as four pairs.
__device__ __forceinline__ void widen2(const Raw8<__nv_bfloat16>& r, f32x2 (&v)[4]) {
  const uint32_t* u = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = pair(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xffff0000u));
}
__device__ __forceinline__ void widen2(const Raw8<__half>& r, f32x2 (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = pair(to_f32(r.e[2 * j]), to_f32(r.e[2 * j + 1]));
}
__device__ __forceinline__ void widen2(const Raw8<float>& r, f32x2 (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = pair(r.e[2 * j], r.e[2 * j + 1]);
}
template <typename T>
__device__ __forceinline__ Raw8<T> narrow2(const f32x2 (&v)[4]) {
  Raw8<T> r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a, b;
    split(v[j], a, b);
    from_f32x2(a, b, &r.e[2 * j]);
  }
  return r;
}

// A row of d values in a slot of shared memory: its bytes, or (VEC false) those
// of the 16-byte pieces that it touches; where in them it begins; the slot.
template <typename T, bool VEC>
__device__ __forceinline__ uint32_t row_shift(const T* p) {
  return VEC ? 0u : static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
}
template <typename T, bool VEC>
__device__ __forceinline__ uint32_t row_span(const T* p, int d) {
  const uint32_t bytes = d * static_cast<uint32_t>(sizeof(T));
  return VEC ? bytes : (row_shift<T, false>(p) + bytes + 15u) & ~15u;
}
template <typename T, bool VEC>
__host__ __device__ constexpr uint32_t row_slot(int d) {
  const uint32_t bytes = d * static_cast<uint32_t>(sizeof(T));
  return VEC ? bytes : ((bytes + 15u) & ~15u) + 16u;
}
// Every 16 bytes that are read hold at least one byte of the row.
template <typename T, bool VEC>
__device__ __forceinline__ void bulk_row(uint32_t dst, const T* p, int d, uint64_t* bar) {
  bulk_load(dst, reinterpret_cast<const uint8_t*>(p) - row_shift<T, VEC>(p), row_span<T, VEC>(p, d),
            bar);
}

template <typename T>
__device__ __forceinline__ void store_raw(T* p, const Raw8<T>& r) {
  const uint4* w = reinterpret_cast<const uint4*>(&r);
#pragma unroll
  for (int k = 0; k < static_cast<int>(sizeof(r) / 16); ++k) reinterpret_cast<uint4*>(p)[k] = w[k];
}

__device__ __forceinline__ __nv_bfloat16 lds_value(uint32_t p, __nv_bfloat16) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(p) : "memory");
  return __ushort_as_bfloat16(v);
}
__device__ __forceinline__ __half lds_value(uint32_t p, __half) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(p) : "memory");
  return __ushort_as_half(v);
}
__device__ __forceinline__ float lds_value(uint32_t p, float) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(p) : "memory");
  return v;
}

// Chunk c of a row in shared memory; zeros past column d.
template <typename T, bool VEC>
__device__ __forceinline__ Raw8<T> lds_chunk(uint32_t row, int c, int t, int tpr, int d) {
  Raw8<T> r;
  if (VEC) {
    uint4* w = reinterpret_cast<uint4*>(&r);
    const int i = c * tpr + t;
#pragma unroll
    for (int k = 0; k < static_cast<int>(sizeof(r) / 16); ++k)
      w[k] = 8 * i < d ? lds_v4(row + i * sizeof(r) + 16 * k) : make_uint4(0, 0, 0, 0);
  } else if (8 * (c + 1) * tpr <= d) {
    const uint32_t p = row + (8 * c * tpr + t) * sizeof(T);
#pragma unroll
    for (int j = 0; j < 8; ++j) r.e[j] = lds_value(p + j * tpr * static_cast<int>(sizeof(T)), T());
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = chunk_col<false>(c, j, t, tpr);
      r.e[j] = col < d ? lds_value(row + col * sizeof(T), T()) : T(0.f);
    }
  }
  return r;
}
template <typename T, bool VEC>
__device__ __forceinline__ void lds_values(uint32_t row, int c, int t, int tpr, int d,
                                           f32x2 (&v)[4]) {
  widen2(lds_chunk<T, VEC>(row, c, t, tpr, d), v);
}

// fp32 sums of a chunk to a row of fp32 (VEC: on 16 bytes, d % 8 == 0).
template <bool VEC>
__device__ __forceinline__ void store_sums(float* row, const f32x2 (&v)[4], int c, int t, int tpr,
                                           int d) {
  store_chunk<float, VEC>(row, narrow2<float>(v), c, t, tpr, d);
}

// A weight or bias vector as fp32 in shared memory. VEC: the first four columns
// of every chunk, then the other four, so that neighbouring threads read
// neighbouring 16 bytes.
__host__ __device__ constexpr uint32_t param_bytes(int d) {
  return (4u * static_cast<uint32_t>(d) + 15u) & ~15u;
}
template <bool VEC>
__device__ __forceinline__ void stage_param(float* dst, const void* p, int type, int d, int thread,
                                            int threads) {
  const int half = d / 2;
  if (VEC && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    for (int i = thread; 8 * i < d; i += threads) {
      float v[8];
      if (type == GRPO_DTYPE_FP32)
        widen(load_chunk<float, true>(static_cast<const float*>(p), 0, i, 0, d), v);
      else if (type == GRPO_DTYPE_BF16)
        widen(load_chunk<__nv_bfloat16, true>(static_cast<const __nv_bfloat16*>(p), 0, i, 0, d), v);
      else
        widen(load_chunk<__half, true>(static_cast<const __half*>(p), 0, i, 0, d), v);
      *reinterpret_cast<float4*>(dst + 4 * i) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(dst + half + 4 * i) = make_float4(v[4], v[5], v[6], v[7]);
    }
    return;
  }
#pragma unroll 4
  for (int col = thread; col < d; col += threads) {
    const int j = col & 7;
    const int at = VEC ? (j >= 4 ? half : 0) + (col >> 3) * 4 + (j & 3) : col;
    dst[at] = load_param(p, type, col);
  }
}
template <bool VEC>
__device__ __forceinline__ void read_param(uint32_t s, int c, int t, int tpr, int d,
                                           f32x2 (&w)[4]) {
  if (VEC) {
    const uint32_t p = s + 16 * (c * tpr + t);
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(w[0]), "=l"(w[1]) : "r"(p) : "memory");
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];"
                 : "=l"(w[2]), "=l"(w[3])
                 : "r"(p + 2 * d)
                 : "memory");
  } else {
    widen2(lds_chunk<float, false>(s, c, t, tpr, d), w);
  }
}

// Joins NV sums of a row's warps (each after warp_sum): every thread gets the
// totals, added in warp order. One named barrier; `sh` holds 2 x NV x 16 sums,
// used in turn (`phase`), those beyond the last warp 0.
template <int NV>
__device__ __forceinline__ void join_warps(float (&v)[NV], int t, int warps, int bar, float* sh,
                                           int& phase) {
  if (warps == 1) {
    __syncwarp();
    return;
  }
  float* s = sh + phase * NV * 16;
  phase ^= 1;
  if ((t & 31) == 0) {
#pragma unroll
    for (int k = 0; k < NV; ++k) s[k * 16 + (t >> 5)] = v[k];
  }
  named_barrier(bar, warps * 32);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    v[k] = 0.f;
#pragma unroll
    for (int w = 0; w < 16; w += 4) {
      if (w >= warps) break;
      const float4 x = *reinterpret_cast<const float4*>(s + k * 16 + w);
      v[k] += (x.x + x.y) + (x.z + x.w);
    }
  }
}

// ---------------------------------------------------- 8-bit checkpoints ----
// Blocks of 32 columns of a row share 2^k; a value is q 2^k with q = e4m3 of
// x / 2^k, rounded to nearest even (half a step: 2^-4 relative for |q| >=
// 2^-6, 2^-10 2^k below). With a = max |x| over the block's finite values,
// a = m 2^e, 1 <= m < 2: k = e - 8 if m <= 1.75 (a / 2^k <= 448, e4m3's
// largest), else e - 7. A power of two makes x / 2^k and q 2^k exact.
// Infinities and NaN are kept as NaN. Where m > 1.75 at the type's largest
// exponent, rounding up to 256 2^k would leave the type: held to 240 there.

template <typename T>
struct CkptTop;  // the k at which 256 2^k is beyond the type's largest value
template <>
struct CkptTop<__nv_bfloat16> {
  static constexpr int k = 120;
};
template <>
struct CkptTop<__half> {
  static constexpr int k = 8;
};
template <>
struct CkptTop<float> {
  static constexpr int k = 120;
};

// k of a block whose largest finite magnitude is `a` (a >= 0, finite).
__device__ __forceinline__ int ckpt_exponent(float a) {
  const uint32_t u = __float_as_uint(a);
  const int k = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(k, kCkptMinExp);
}

// 2^k for k in [-126, 127].
__device__ __forceinline__ float pow2(int k) {
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

// |v| maxima that keep a NaN.
__device__ __forceinline__ float max_abs_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Two e4m3 (low byte first), to nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two e4m3 (low byte first) widened.
__device__ __forceinline__ float2 unpack_e4m3x2(uint32_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w)));
  float2 f;
  unpack_f16x2(h, f.x, f.y);
  return f;
}

// One value for the checkpoint, with everything that can be special about it.
template <typename T>
__device__ __forceinline__ float ckpt_scaled(float v, float inv, int k) {
  if (!(fabsf(v) <= FLT_MAX)) return __uint_as_float(0x7fc00000u);
  v *= inv;
  if (k >= CkptTop<T>::k) v = fminf(fmaxf(v, -240.f), 240.f);
  return v;
}

// 8 columns of a block, of which 4 neighbouring lanes hold one, as e4m3, and the
// block's exponent byte. Every lane of the warp calls this (0 where there is no
// column).
template <typename T>
__device__ __forceinline__ uint2 ckpt_encode(const f32x2 (&p)[4], int& ex) {
  float v[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) split(p[j], v[2 * j], v[2 * j + 1]);
  float a = max_abs_nan(v[0], v[1], v[2]);
  a = max_abs_nan(a, v[3], v[4]);
  a = max_abs_nan(max_abs_nan(a, v[5], v[6]), v[7], v[7]);
  const float b = __shfl_xor_sync(0xffffffffu, a, 1);
  a = max_abs_nan(a, b, b);
  const float c = __shfl_xor_sync(0xffffffffu, a, 2);
  a = max_abs_nan(a, c, c);
  uint2 w;
  int k = ckpt_exponent(a);
  // Nothing in the warp's blocks is special (the usual case): scale and round.
  // The branch keeps some ten instructions per value out of the path.
  if (__all_sync(0xffffffffu, a <= FLT_MAX && k < CkptTop<T>::k)) {
    const float inv = pow2(-k);
    const f32x2 ii = pair(inv, inv);
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float lo, hi;
      split(mul2(p[j], ii), lo, hi);
      h[j] = pack_e4m3x2(lo, hi);
    }
    w.x = __byte_perm(h[0], h[1], 0x5410);
    w.y = __byte_perm(h[2], h[3], 0x5410);
  } else {
    a = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float m = fabsf(v[j]);
      if (m <= FLT_MAX) a = fmaxf(a, m);
    }
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
    k = ckpt_exponent(a);
    const float inv = pow2(-k);
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      h[j] = pack_e4m3x2(ckpt_scaled<T>(v[2 * j], inv, k), ckpt_scaled<T>(v[2 * j + 1], inv, k));
    w.x = __byte_perm(h[0], h[1], 0x5410);
    w.y = __byte_perm(h[2], h[3], 0x5410);
  }
  ex = k + kCkptBias;
  return w;
}

// 1 KB of shared memory a warp, for blocks between a column to a lane and 8
// columns to a lane.
struct BlockTurn {
  float at[8][33];
};

// Writes chunk c of a row to its checkpoint. Every lane of the warp calls this
// (values past column d are 0, and so is what the padding behind d gets). q: the
// row's bytes; ex: its exponents; turn: VEC false only, this warp's.
template <typename T, bool VEC>
__device__ __forceinline__ void ckpt_store_chunk(const f32x2 (&v)[4], uint8_t* q, uint8_t* ex,
                                                 int c, int t, int tpr, int d, BlockTurn* turn) {
  int e, col;
  uint2 w;
  if (VEC) {
    col = chunk_col<true>(c, 0, t, tpr);
    w = ckpt_encode<T>(v, e);
  } else {
    // The warp holds 8 blocks, one to each j.
    const int lane = t & 31;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float lo, hi;
      split(v[j], lo, hi);
      turn->at[2 * j][lane] = lo;
      turn->at[2 * j + 1][lane] = hi;
    }
    __syncwarp();
    const float* const b = turn->at[lane >> 2] + 8 * (lane & 3);
    const f32x2 p[4] = {pair(b[0], b[1]), pair(b[2], b[3]), pair(b[4], b[5]), pair(b[6], b[7])};
    w = ckpt_encode<T>(p, e);
    col = (8 * c + (lane >> 2)) * tpr + (t - lane) + 8 * (lane & 3);
  }
  if (col < d) {
    *reinterpret_cast<uint2*>(q + col) = w;
    if ((t & 3) == 0) ex[col / kCkptBlock] = static_cast<uint8_t>(e);
  }
}

// A chunk of a checkpoint row as loaded: its bytes and its exponents.
template <bool VEC>
struct RawCkpt {
  uint2 w;
  uint8_t ex[VEC ? 1 : 8];
};

template <bool VEC>
__device__ __forceinline__ RawCkpt<VEC> ckpt_load_chunk(const uint8_t* q, const uint8_t* ex, int c,
                                                        int t, int tpr, int d) {
  RawCkpt<VEC> r;
  if (VEC) {
    const int col = chunk_col<true>(c, 0, t, tpr);
    r.w = make_uint2(0, 0);
    r.ex[0] = kCkptBias;
    if (col < d) {
      r.w = *reinterpret_cast<const uint2*>(q + col);
      r.ex[0] = ex[col / kCkptBlock];
    }
  } else {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = chunk_col<false>(c, j, t, tpr);
      r.ex[VEC ? 0 : j] = kCkptBias;
      if (col < d) {
        w[j >> 2] |= static_cast<uint32_t>(q[col]) << (8 * (j & 3));
        r.ex[VEC ? 0 : j] = ex[col / kCkptBlock];
      }
    }
    r.w = make_uint2(w[0], w[1]);
  }
  return r;
}

// The stored exponent byte as the factor 2^k. Bytes outside what packing
// writes (10 to 247) are held to [1, 254], where the factor is a normal fp32.
__device__ __forceinline__ float ckpt_factor(uint32_t byte) {
  return __uint_as_float(min(max(byte, 1u), 254u) << 23);
}

template <bool VEC>
__device__ __forceinline__ void ckpt_widen(const RawCkpt<VEC>& r, float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const uint32_t w = (h < 2 ? r.w.x : r.w.y) >> (16 * (h & 1));
    const float2 f = unpack_e4m3x2(w & 0xffffu);
    v[2 * h] = f.x * ckpt_factor(r.ex[VEC ? 0 : 2 * h]);
    v[2 * h + 1] = f.y * ckpt_factor(r.ex[VEC ? 0 : 2 * h + 1]);
  }
}

// The same of a checkpoint row in shared memory.
template <bool VEC>
__device__ __forceinline__ void lds_ckpt(uint32_t q, uint32_t ex, int c, int t, int tpr, int d,
                                         f32x2 (&v)[4]) {
  if (VEC) {
    const int i = c * tpr + t;
    if (8 * i >= d) {
#pragma unroll
      for (int h = 0; h < 4; ++h) v[h] = 0ull;
      return;
    }
    const uint2 w = lds_v2(q + 8 * i);
    const float f = ckpt_factor(lds_u8(ex + i / 4));
    const f32x2 ff = pair(f, f);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const float2 x = unpack_e4m3x2((h < 2 ? w.x : w.y) >> (16 * (h & 1)));
      v[h] = mul2(pair(x.x, x.y), ff);
    }
  } else {
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = chunk_col<false>(c, j, t, tpr);
      x[j] = col < d ? unpack_e4m3x2(lds_u8(q + col)).x * ckpt_factor(lds_u8(ex + col / kCkptBlock))
                     : 0.f;
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) v[h] = pair(x[2 * h], x[2 * h + 1]);
  }
}

}  // namespace grpo
