// One AdamW step over many tensors, and the norm of all their gradients.
//
// Memory bound: every value is read and written once (fp32 moments: 28 bytes a
// parameter with fp32 gradients and parameters; 8-bit moments: 16), so many tensors
// share a launch and their table travels in the kernel's parameters: no copy to the
// device, nothing kept from one call for the next, and a captured launch holds it.
// A CTA takes a chunk of one tensor, which it finds by bisection; a warp takes 256
// consecutive values at a time, 8 to a lane in 16-byte loads.
//
// Moments in 8 bits: 128 consecutive values share a scale, and 16 lanes hold them, so
// the largest is four shuffles away. With round to nearest, a second moment that
// changes by a thousandth a step would stand still (e4m3's neighbours are a sixteenth
// to an eighth apart); rounded at random it is right in the mean.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "launch.h"
#include "norm.h"
#include "row_ops.cuh"

namespace grpo {
namespace {

constexpr int kThreads = 256;  // of the norm's kernels
constexpr int kWarps = kThreads / 32;
// Of the step's, its CTAs of an SM (which set its registers), and the most values that
// one takes. With moments in 8 bits the instructions bound it, and short CTAs give their
// places up sooner: 2^28 values in 720 us with CTAs of 256 threads, 676 with 128, 673 with
// 64 (bf16 parameters, before the roundings were made exact; fp32 791, 735 and 687); exact,
// 14 of them an SM 739 and 718, 16 738 and 786, 12 745 and 736. In 32 bits, which memory
// bounds: 1023, 1017 and 997 us with 16384, 8192 and 4096 values.
template <int BITS>
constexpr int kStepThreads = BITS == 8 ? 64 : 256;
template <int BITS>
constexpr int kStepCtas = BITS == 8 ? 14 : 4;
template <int BITS>
constexpr int kStepChunk = BITS == 8 ? 16384 : 4096;
constexpr int kGroup = 256;  // values of a warp's step
constexpr int kBlock = 128;  // values that share a scale
constexpr float kTop = 448.f;              // the largest e4m3
constexpr float kLeast = 3.0092655e-36f;   // 2^-118: blocks below it are kept as zeros
constexpr int kSmallTable = 24, kLargeTable = 256;

struct AdamwEntry {
  void* param;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  void* copy;
  long long numel;
  long long place;  // of its first value in the random numbers' count
  float lr, decay;
  int chunk;        // its first chunk of the launch
  uint8_t ptype, gtype, ctype;
};

template <int N>
struct AdamwTable {
  AdamwEntry e[N];
};

struct AdamwArgs {
  int count;
  int chunk;  // values of a chunk, a multiple of kGroup
  float beta1, beta2, rest1, rest2, eps;
  float log1, log2;  // of the betas
  float fix1, fix2;  // 1 / (1 - beta1^step), 1 / sqrt(1 - beta2^step)
  uint64_t seed;
  long long step;
  const float* scale;
  const float* lr_factor;
  const int64_t* step_on_device;
};

// ------------------------------------------------------- random numbers ----

// A 32-bit number to another, all bits mixed (multiply and fold; the multipliers are
// the fractions of the roots of 2 and 3).
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

struct Keys {
  uint32_t k0, k1;
};
__device__ __forceinline__ Keys keys_of(uint64_t seed, uint64_t step) {
  const uint32_t a =
      mix(static_cast<uint32_t>(seed) ^ mix(static_cast<uint32_t>(seed >> 32) + 0x3C6EF372u));
  const uint32_t b =
      mix(static_cast<uint32_t>(step) ^ mix(static_cast<uint32_t>(step >> 32) + a));
  return {b, mix(b + 0x510E527Fu)};
}

// The keys of the 2^32 places that begin at a multiple of it: the step's own for the
// first of them (mix(0) is 0).
__device__ __forceinline__ Keys keys_at(const Keys& k, uint32_t high) {
  const uint32_t far = mix(high);
  return {k.k0 ^ far, k.k1 + mix(far * 0x1F83D9ABu)};
}

// The first hash of a place: 16 bits for either moment.
__device__ __forceinline__ uint32_t bits_after(const Keys& k, uint32_t x) {
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x = x * 0xBB67AE85u + k.k1 * 0xBB67AE85u;
  return x ^ (x >> 16);
}
__device__ __forceinline__ uint32_t bits_at(const Keys& k, uint32_t i) {
  const uint32_t x = i ^ k.k0;
  return bits_after(k, x ^ (x >> 16));
}
// And the second, from the first: 16 bits for the parameter.
__device__ __forceinline__ uint32_t more_bits(const Keys& k, uint32_t x) {
  const uint32_t y = (x ^ k.k1) * 0x5BE0CD19u;
  return (y ^ (y >> 16)) & 0xffffu;
}

// ----------------------------------------------------------- conversions ----

// The high bytes of four words, the first one's lowest.
__device__ __forceinline__ uint32_t high_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

// Eight values y scaled by f to e4m3 at random: a = |y f| (448 at most) goes to its
// lower neighbour lo, or to the upper one hi where u < 2^16 (a - lo) / (hi - lo), u
// the low 16 bits of x. The comparison is exact.
//
// 2^-120 takes e4m3's normal range to fp32's, and its subnormals to fp32's: bits 20 to
// 26 of the word are lo's code and the 20 below them (a - lo) / (hi - lo), for every
// a. Adding 2^20 - 1 - 16 u carries into the code where those are more than 16 u.
__device__ __forceinline__ uint2 codes_of(const float (&y)[8], float f, const uint32_t (&x)[8]) {
  uint32_t s[8], t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t w = __float_as_uint(fminf(fabsf(y[j] * f), kTop) * 0x1p-120f);
    t[j] = ((w + 0xfffffu) - 16u * (x[j] & 0xffffu)) * 16u;
    s[j] = __float_as_uint(y[j]);
  }
  constexpr uint32_t kSigns = 0x80808080u;
  return make_uint2(high_bytes(t[0], t[1], t[2], t[3]) | (high_bytes(s[0], s[1], s[2], s[3]) & kSigns),
                    high_bytes(t[4], t[5], t[6], t[7]) | (high_bytes(s[4], s[5], s[6], s[7]) & kSigns));
}

// The same of roots (y >= 0) by their squares: u < 2^16 (a^2 - lo^2) / (hi^2 - lo^2), u
// the high 16 bits of x. A y beyond `some` never becomes 0.
__device__ __forceinline__ uint2 codes_of_roots(const float (&y)[8], float f,
                                                const uint32_t (&x)[8], float some) {
  uint32_t t[8], least = 0xffffffffu;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float a = fminf(y[j] * f, kTop);
    const uint32_t w = __float_as_uint(a * 0x1p-120f);
    const uint32_t lo = w & 0xfff00000u, hi = lo + 0x100000u;
    const float l = __uint_as_float(lo) * 0x1p120f, h = __uint_as_float(hi) * 0x1p120f;
    const float q = __uint_as_float(((x[j] >> 9) & 0x007fff80u) | 0x3f800000u) - 1.f;  // u / 2^16
    t[j] = (q * ((h - l) * (h + l)) < (a - l) * (a + l) ? hi : lo) * 16u;
    least = min(least, w);
  }
  if (least < 0x100000u) {  // rare: a value, or a zero, below the least code
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (y[j] > some) t[j] = max(t[j], 0x1000000u);
  }
  return make_uint2(high_bytes(t[0], t[1], t[2], t[3]), high_bytes(t[4], t[5], t[6], t[7]));
}

// Codes whose values are not finite, as NaN.
__device__ __forceinline__ void lose(const float (&y)[8], uint2& q) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t& w = j < 4 ? q.x : q.y;
    const int at = 8 * (j & 3);
    if (!(fabsf(y[j]) <= FLT_MAX))
      w = (w & ~(0xffu << at)) | static_cast<uint32_t>(kCkptNaN) << at;
  }
}

// Off by 2^-23 of itself at most; where v is subnormal too.
__device__ __forceinline__ float quick_root(float v) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// Off by 2^-22 of itself at most, for 2^-126 and more.
__device__ __forceinline__ float quick_inverse_root(float v) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// Off by 2^-23 of itself at most, for 0 and 2^-126 to 2^126.
__device__ __forceinline__ float quick_inverse(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

template <typename T>
__device__ __forceinline__ float load1(const void* p, long long i) {
  return to_f32(static_cast<const T*>(p)[i]);
}

// 8 consecutive values from 16-byte loads.
template <typename T>
__device__ __forceinline__ void load8(const void* p, long long i, float (&v)[8]) {
  Raw8<T> r;
  const uint4* s = reinterpret_cast<const uint4*>(static_cast<const T*>(p) + i);
  uint4* w = reinterpret_cast<uint4*>(&r);
#pragma unroll
  for (int k = 0; k < static_cast<int>(sizeof(r) / 16); ++k) w[k] = __ldcs(s + k);
  widen(r, v);
}
template <typename T>
__device__ __forceinline__ void store8(void* p, long long i, const float (&v)[8]) {
  const Raw8<T> r = narrow<T>(v);
  uint4* d = reinterpret_cast<uint4*>(static_cast<T*>(p) + i);
  const uint4* w = reinterpret_cast<const uint4*>(&r);
#pragma unroll
  for (int k = 0; k < static_cast<int>(sizeof(r) / 16); ++k) __stcs(d + k, w[k]);
}

// ------------------------------------------------------------------ step ----

// What a chunk's threads share.
struct StepOf {
  float scale, fade, rate, beta1, beta2, rest1, rest2, fix2, eps;
  Keys keys;  // of the chunk's places where they are all `near` one another, or the step's
  bool near;
};

// The largest |y| of a lane, and over the 16 lanes of a block; NaN where one of them is.
__device__ __forceinline__ float lane_top(const float (&y)[8]) {
  float a = max_abs_nan(y[0], y[1], y[2]);
  a = max_abs_nan(a, y[3], y[4]);
  return max_abs_nan(max_abs_nan(a, y[5], y[6]), y[7], y[7]);
}
__device__ __forceinline__ float block_top(const float (&y)[8]) {
  float a = lane_top(y);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const float b = __shfl_xor_sync(0xffffffffu, a, o);
    a = max_abs_nan(a, b, b);
  }
  return a;
}
// The largest finite one.
__device__ __noinline__ float block_top_finite(float y0, float y1, float y2, float y3, float y4,
                                               float y5, float y6, float y7) {
  const float y[8] = {y0, y1, y2, y3, y4, y5, y6, y7};
  float a = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) a = fabsf(y[j]) <= FLT_MAX ? fmaxf(a, fabsf(y[j])) : a;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

// A chunk of a tensor: its values' parts, how many they are, and the place of the first.
template <int BITS, typename P, typename G>
struct Chunk {
  using M = std::conditional_t<BITS == 8, uint8_t, float>;
  P* param;
  const G* grad;
  M* m;
  M* v;
  float* m_scale;
  float* v_scale;
  void* copy;  // 2 bytes a value
  int count;
  uint32_t place;  // its low 32 bits
  uint32_t high;   // the others, of the first value
  int ctype;

  __device__ __forceinline__ Chunk(const AdamwEntry& e, long long begin, int chunk)
      : param(static_cast<P*>(e.param) + begin),
        grad(static_cast<const G*>(e.grad) + begin),
        m(static_cast<M*>(e.m) + begin),
        v(static_cast<M*>(e.v) + begin),
        m_scale(BITS == 8 ? e.m_scale + begin / kBlock : nullptr),
        v_scale(BITS == 8 ? e.v_scale + begin / kBlock : nullptr),
        copy(e.copy == nullptr ? nullptr : static_cast<uint16_t*>(e.copy) + begin),
        count(static_cast<int>(min(static_cast<long long>(chunk), e.numel - begin))),
        place(static_cast<uint32_t>(e.place + begin)),
        high(static_cast<uint32_t>(static_cast<uint64_t>(e.place + begin) >> 32)),
        ctype(e.ctype) {}
};

// A lane's 8 values: consecutive from `first` on (VEC, all there), or every 16th of
// their block, as far as the chunk goes.
template <int BITS, typename P, typename G, bool VEC>
__device__ __forceinline__ void step8(const Chunk<BITS, P, G>& e, const StepOf& s, int first,
                                      int lane) {
  constexpr int kEvery = VEC ? 1 : 16;
  float p[8], g[8], m[8], v[8];
  bool have[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) have[j] = VEC || first + j * kEvery < e.count;
  const int block = first / kBlock;  // BITS 8: this lane's
  float ms = 0.f, vs = 0.f;
  if (BITS == 8 && have[0]) {
    ms = e.m_scale[block];
    vs = e.v_scale[block];
  }
  if constexpr (VEC) {
    load8<P>(e.param, first, p);
    load8<G>(e.grad, first, g);
    if constexpr (BITS == 32) {
      load8<float>(e.m, first, m);
      load8<float>(e.v, first, v);
    } else {
      const uint2 mq = __ldcs(reinterpret_cast<const uint2*>(e.m + first));
      const uint2 vq = __ldcs(reinterpret_cast<const uint2*>(e.v + first));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 a = unpack_e4m3x2((j < 2 ? mq.x : mq.y) >> (16 * (j & 1)));
        const float2 b = unpack_e4m3x2((j < 2 ? vq.x : vq.y) >> (16 * (j & 1)));
        m[2 * j] = a.x;
        m[2 * j + 1] = a.y;
        v[2 * j] = b.x;
        v[2 * j + 1] = b.y;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = first + j * kEvery;
      p[j] = g[j] = m[j] = v[j] = 0.f;
      if (have[j]) {
        p[j] = to_f32(e.param[i]);
        g[j] = to_f32(e.grad[i]);
        if constexpr (BITS == 32) {
          m[j] = e.m[i];
          v[j] = e.v[i];
        } else {
          m[j] = unpack_e4m3x2(e.m[i]).x;
          v[j] = unpack_e4m3x2(e.v[i]).x;
        }
      }
    }
  }
  float root[8];
  {
    const f32x2 scale = pair(s.scale, s.scale), beta1 = pair(s.beta1, s.beta1),
                beta2 = pair(s.beta2, s.beta2), rest1 = pair(s.rest1, s.rest1),
                rest2 = pair(s.rest2, s.rest2), fix2 = pair(s.fix2, s.fix2),
                eps = pair(s.eps, s.eps), rate = pair(-s.rate, -s.rate),
                fade = pair(-s.fade, -s.fade), ms2 = pair(ms, ms), vs2 = pair(vs, vs);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      f32x2 m2 = pair(m[j], m[j + 1]), v2 = pair(v[j], v[j + 1]);
      if (BITS == 8) {
        m2 = mul2(m2, ms2);
        v2 = mul2(v2, vs2);
        v2 = mul2(v2, v2);
      }
      const f32x2 x2 = mul2(pair(g[j], g[j + 1]), scale);
      const f32x2 dm = mul2(rest1, x2), dv = mul2(rest2, mul2(x2, x2));
      if (BITS == 8) {
        // Each product and sum rounded (and the root below): which of two neighbours a
        // moment goes to then follows from the formula's own fp32 values. (The
        // assembler makes one fused step of a product and a sum of pairs.)
        float a, b, c, d;
        split(m2, a, b);
        split(dm, c, d);
        m2 = pair(__fadd_rn(__fmul_rn(s.beta1, a), c), __fadd_rn(__fmul_rn(s.beta1, b), d));
        split(v2, a, b);
        split(dv, c, d);
        v2 = pair(__fadd_rn(__fmul_rn(s.beta2, a), c), __fadd_rn(__fmul_rn(s.beta2, b), d));
      } else {
        m2 = fma2(beta1, m2, dm);
        v2 = fma2(beta2, v2, dv);
      }
      split(m2, m[j], m[j + 1]);
      split(v2, v[j], v[j + 1]);
      if (BITS == 8) {
        // y about v^-1/2 to 2^-22, g = v y; then Newton's step for the root, g + (v -
        // g^2) y / 2, which is right to the last bit but for one in a million.
        const f32x2 y = pair(quick_inverse_root(v[j]), quick_inverse_root(v[j + 1]));
        const f32x2 minus = pair(-1.f, -1.f), half = pair(-0.5f, -0.5f);
        const f32x2 g2 = mul2(v2, y);
        split(fma2(fma2(g2, g2, mul2(v2, minus)), mul2(y, half), g2), root[j], root[j + 1]);
      } else {
        root[j] = quick_root(v[j]);
        root[j + 1] = quick_root(v[j + 1]);
      }
    }
    if (BITS == 8 && !(lane_top(root) <= FLT_MAX)) {  // 0, subnormal or not finite: no y
#pragma unroll
      for (int j = 0; j < 8; ++j) root[j] = __fsqrt_rn(v[j]);
    }
    auto step_of = [&](int j) {  // of values j and j + 1
      float d0, d1;
      split(fma2(pair(root[j], root[j + 1]), fix2, eps), d0, d1);
      // d is 0 or normal: a root of at least 2^-75, or eps
      return mul2(mul2(rate, pair(m[j], m[j + 1])), pair(quick_inverse(d0), quick_inverse(d1)));
    };
    // Decay and step are added up before the parameter takes them: 1 - lr decay as an
    // fp32 would round the decay itself to a multiple of 2^-24, each step the same way.
    if (lane_top(p) <= FLT_MAX) {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const f32x2 q = pair(p[j], p[j + 1]);
        split(add2(q, fma2(fade, q, step_of(j))), p[j], p[j + 1]);
      }
    } else {  // an infinity has no decay: it stays
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        float d0, d1;
        split(step_of(j), d0, d1);
        p[j] += fabsf(p[j]) <= FLT_MAX ? fmaf(-s.fade, p[j], d0) : d0;
        p[j + 1] += fabsf(p[j + 1]) <= FLT_MAX ? fmaf(-s.fade, p[j + 1], d1) : d1;
      }
    }
  }
  if constexpr (BITS == 32 && VEC) {
    store8<float>(e.m, first, m);
    store8<float>(e.v, first, v);
  } else if constexpr (BITS == 32) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (have[j]) {
        e.m[first + j * kEvery] = m[j];
        e.v[first + j * kEvery] = v[j];
      }
  }
  uint32_t x[8];
  constexpr bool kRandom = BITS == 8 || sizeof(P) == 2;
  Keys keys = s.keys;
  if constexpr (kRandom) {
    // A lane's values lie in one block, which no multiple of 2^32 parts.
    const uint32_t place = e.place + static_cast<uint32_t>(first);
    if (!s.near) keys = keys_at(s.keys, e.high + (place < e.place ? 1u : 0u));
    // Consecutive places, from a multiple of 8 on, differ below what the first fold
    // moves.
    const uint32_t head = place ^ keys.k0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      x[j] = VEC ? bits_after(keys, (head ^ (head >> 16)) ^ j)
                 : bits_at(keys, place + j * kEvery);
  }
  if constexpr (BITS == 8) {
    float mt = block_top(m), vt = block_top(root);
    // Nothing in the warp's blocks is special (the usual case).
    const bool plain = __all_sync(0xffffffffu, mt <= FLT_MAX && vt <= FLT_MAX);
    if (!plain) {
      mt = block_top_finite(m[0], m[1], m[2], m[3], m[4], m[5], m[6], m[7]);
      vt = block_top_finite(root[0], root[1], root[2], root[3], root[4], root[5], root[6], root[7]);
    }
    mt = mt >= kLeast ? mt : 0.f;
    vt = vt >= kLeast ? vt : 0.f;
    // 448 / top: of m in the even lanes, of the root in the odd ones, and then for all.
    // The top of a block of zeros is 0, and so is its factor.
    const float top = (lane & 1) == 0 ? mt : vt;
    const float factor = top > 0.f ? __frcp_rn(top) * kTop : 0.f;
    const float mi = __shfl_sync(0xffffffffu, factor, lane & 16);
    const float vi = __shfl_sync(0xffffffffu, factor, (lane & 16) + 1);
    uint2 mq = codes_of(m, mi, x);
    uint2 vq = codes_of_roots(root, vi, x, vt > 0.f ? 0.f : FLT_MAX);
    if (!plain) {
      lose(m, mq);
      lose(root, vq);
    }
    if constexpr (VEC) {
      __stcs(reinterpret_cast<uint2*>(e.m + first), mq);
      __stcs(reinterpret_cast<uint2*>(e.v + first), vq);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (have[j]) {
          e.m[first + j * kEvery] =
              static_cast<uint8_t>((j < 4 ? mq.x : mq.y) >> (8 * (j & 3)));
          e.v[first + j * kEvery] =
              static_cast<uint8_t>((j < 4 ? vq.x : vq.y) >> (8 * (j & 3)));
        }
    }
    if ((lane & 14) == 0 && block * kBlock < e.count)
      ((lane & 1) == 0 ? e.m_scale : e.v_scale)[block] = top * (1.f / kTop);
  }
  if constexpr (sizeof(P) == 2) {
    // To bf16 at random: 16 random bits below the kept ones, then cut off; infinities
    // and NaN as they are.
    float top = max_abs_nan(p[0], p[1], p[2]);
    top = max_abs_nan(max_abs_nan(top, p[3], p[4]), max_abs_nan(p[5], p[6], p[7]), p[0]);
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      w[j] = (__float_as_uint(p[j]) + more_bits(keys, x[j])) & 0xffff0000u;
    if (!(top <= FLT_MAX)) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!(fabsf(p[j]) <= FLT_MAX)) w[j] = __float_as_uint(p[j]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = __uint_as_float(w[j]);
  }
  if constexpr (VEC) {
    if constexpr (sizeof(P) == 2) {  // already bf16s
      uint4 w;
      w.x = __byte_perm(__float_as_uint(p[0]), __float_as_uint(p[1]), 0x7632);
      w.y = __byte_perm(__float_as_uint(p[2]), __float_as_uint(p[3]), 0x7632);
      w.z = __byte_perm(__float_as_uint(p[4]), __float_as_uint(p[5]), 0x7632);
      w.w = __byte_perm(__float_as_uint(p[6]), __float_as_uint(p[7]), 0x7632);
      __stcs(reinterpret_cast<uint4*>(e.param + first), w);
    } else {
      store8<P>(e.param, first, p);
    }
    if (e.copy != nullptr) {
      if (e.ctype == GRPO_DTYPE_BF16)
        store8<__nv_bfloat16>(e.copy, first, p);
      else
        store8<__half>(e.copy, first, p);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!have[j]) continue;
      const int i = first + j * kEvery;
      e.param[i] = static_cast<P>(p[j]);
      if (e.copy != nullptr) {
        if (e.ctype == GRPO_DTYPE_BF16)
          static_cast<__nv_bfloat16*>(e.copy)[i] = __float2bfloat16_rn(p[j]);
        else
          static_cast<__half*>(e.copy)[i] = __float2half_rn(p[j]);
      }
    }
  }
}

__device__ __forceinline__ bool on(const void* p, int a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

template <int BITS, typename P, typename G>
__device__ __forceinline__ void step_chunk(const AdamwEntry& e, const StepOf& s, long long begin,
                                           int chunk) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kState = BITS == 8 ? 8 : 16;
  constexpr int kStep = kStepThreads<BITS> / 32 * kGroup;
  const bool vec = on(e.param, 16) && on(e.grad, 16) && on(e.m, kState) && on(e.v, kState) &&
                   on(e.copy, 16);
  const Chunk<BITS, P, G> c(e, begin, chunk);
  for (int at = warp * kGroup; at < c.count; at += kStep) {
    if (vec && at + kGroup <= c.count)
      step8<BITS, P, G, true>(c, s, at + lane * 8, lane);
    else
      step8<BITS, P, G, false>(c, s, at + (lane >> 4) * kBlock + (lane & 15), lane);
  }
}

template <int BITS, typename P>
__device__ __forceinline__ void step_grad(const AdamwEntry& e, const StepOf& s, long long begin,
                                          int chunk) {
  if (e.gtype == GRPO_DTYPE_FP32)
    step_chunk<BITS, P, float>(e, s, begin, chunk);
  else if (e.gtype == GRPO_DTYPE_BF16)
    step_chunk<BITS, P, __nv_bfloat16>(e, s, begin, chunk);
  else
    step_chunk<BITS, P, __half>(e, s, begin, chunk);
}

// The last entry whose first chunk is at most c.
template <typename E>
__device__ __forceinline__ int find_entry(const E* e, int count, int c) {
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (e[mid].chunk <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

template <int N, int BITS>
__global__ void __launch_bounds__(kStepThreads<BITS>, kStepCtas<BITS>)
    adamw_kernel(const __grid_constant__ AdamwTable<N> table, const AdamwArgs args) {
  const float scale = args.scale != nullptr ? *args.scale : 1.f;
  if (!(fabsf(scale) <= FLT_MAX)) return;  // the step is skipped
  const int c = static_cast<int>(blockIdx.x);
  const AdamwEntry& e = table.e[find_entry(table.e, args.count, c)];
  StepOf s;
  float fix1 = args.fix1;
  s.fix2 = args.fix2;
  long long step = args.step;
  if (args.step_on_device != nullptr) {
    step = max(static_cast<long long>(*args.step_on_device), 1LL);
    // 1 - beta^t without its cancellation.
    const float t = static_cast<float>(step);
    fix1 = 1.f / -expm1f(t * args.log1);
    s.fix2 = rsqrtf(-expm1f(t * args.log2));
  }
  const float lr = e.lr * (args.lr_factor != nullptr ? *args.lr_factor : 1.f);
  s.scale = scale;
  s.fade = lr * e.decay;
  s.rate = lr * fix1;
  s.beta1 = args.beta1;
  s.beta2 = args.beta2;
  s.rest1 = args.rest1;
  s.rest2 = args.rest2;
  s.eps = args.eps;
  s.keys = keys_of(args.seed, static_cast<uint64_t>(step));
  const long long begin = static_cast<long long>(c - e.chunk) * args.chunk;
  const uint64_t place = static_cast<uint64_t>(e.place + begin);
  s.near = (place >> 32) == ((place + static_cast<uint64_t>(args.chunk) - 1) >> 32);
  if (s.near) s.keys = keys_at(s.keys, static_cast<uint32_t>(place >> 32));
  if (e.ptype == GRPO_DTYPE_FP32)
    step_grad<BITS, float>(e, s, begin, args.chunk);
  else
    step_grad<BITS, __nv_bfloat16>(e, s, begin, args.chunk);
}

// ------------------------------------------------------------------ norm ----

constexpr int kNormTable = 1024;
constexpr int kNormCtas = 1216;  // 8 an SM
constexpr int kNormChunk = 16384;

struct NormEntry {
  const void* grad;
  long long numel;
  int chunk;
  int type;
};
template <int N>
struct NormTable {
  NormEntry e[N];
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The sum over the CTA, in thread 0.
__device__ __forceinline__ double cta_sum(double v) {
  __shared__ double part[kWarps];
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < kWarps; ++w) v += part[w];
  return v;
}

// A sum of fp32 values in two parts, two such sums side by side: what the sum's
// rounding leaves is found exactly and kept (the sum of two floating-point numbers and
// its error: Knuth), so that the norm is right to fp32's last bit however many there are;
// fp64 for every value would take three times as long as reading it. Its range is that of
// values up to 2^50 (2^25 of their squares are below 2^126) beside one of 2^-50 at least
// (the others' squares may be subnormal, off by 2^-149 each); the rest is summed in fp64.
struct Squares {
  f32x2 sum = 0ull, rest = 0ull;
  double far = 0.0;

  __device__ __forceinline__ void add(f32x2 q) {
    const f32x2 minus = pair(-1.f, -1.f);
    const f32x2 t = add2(sum, q);
    const f32x2 b = fma2(sum, minus, t);                           // t - sum
    const f32x2 c = add2(fma2(b, minus, q), fma2(fma2(b, minus, t), minus, sum));
    sum = t;
    rest = add2(rest, c);
  }
  // Two values' squares; EXACT: they are fp32 numbers themselves (16-bit values').
  template <bool EXACT>
  __device__ __forceinline__ void square(float x, float y) {
    const f32x2 v = pair(x, y), q = pair(__fmul_rn(x, x), __fmul_rn(y, y));
    add(q);
    if (!EXACT) rest = add2(rest, fma2(v, v, mul2(q, pair(-1.f, -1.f))));
  }
  // A thread's eight values at a time, N of them: whether they are in range.
  template <int N>
  static __device__ __forceinline__ bool in_range(const float (&v)[N][8]) {
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int j = 0; j < 8; j += 2) top = max_abs_nan(top, v[k][j], v[k][j + 1]);
    return (top >= 0x1p-50f && top <= 0x1p50f) || top == 0.f;
  }
  template <bool EXACT, int N>
  __device__ __forceinline__ void take(const float (&v)[N][8]) {
    if (in_range(v)) {
#pragma unroll
      for (int k = 0; k < N; ++k)
#pragma unroll
        for (int j = 0; j < 8; j += 2) square<EXACT>(v[k][j], v[k][j + 1]);
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x = v[k][j], q = __fmul_rn(x, x);
          // beyond fp32: infinity, or NaN
          far += q <= FLT_MAX ? static_cast<double>(x) * static_cast<double>(x)
                              : static_cast<double>(q);
        }
    }
  }
  __device__ __forceinline__ double total() const {
    float a, b, c, d;
    split(sum, a, b);
    split(rest, c, d);
    return (static_cast<double>(a) + static_cast<double>(c)) +
           (static_cast<double>(b) + static_cast<double>(d)) + far;
  }
};

// A thread's squares of a chunk.
template <typename T>
__device__ __forceinline__ void squares(const void* p, long long begin, long long end,
                                        Squares& s) {
  constexpr bool kExact = sizeof(T) == 2;
  long long at = begin;
  if (on(p, 16)) {  // begin is a multiple of the chunk
    constexpr int kStep = kThreads * 8;
    for (; at + 4 * kStep <= end; at += 4 * kStep) {
      float v[4][8];
#pragma unroll
      for (int k = 0; k < 4; ++k) load8<T>(p, at + k * kStep + threadIdx.x * 8, v[k]);
      s.take<kExact>(v);
    }
  }
  for (; at < end; at += 8 * kThreads) {
    float v[1][8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const long long i = at + k * kThreads + threadIdx.x;
      v[0][k] = i < end ? load1<T>(p, i) : 0.f;
    }
    s.take<kExact>(v);
  }
}

// One partial sum a CTA; CTAs take the chunks round robin.
template <int N>
__global__ void __launch_bounds__(kThreads)
    grad_norm_kernel(const __grid_constant__ NormTable<N> table, int count, int chunks,
                     double* partials) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Squares s;
  for (int c = static_cast<int>(blockIdx.x); c < chunks; c += static_cast<int>(gridDim.x)) {
    const NormEntry& e = table.e[find_entry(table.e, count, c)];
    const long long begin = static_cast<long long>(c - e.chunk) * kNormChunk;
    const long long end = min(begin + kNormChunk, e.numel);
    if (e.type == GRPO_DTYPE_FP32)
      squares<float>(e.grad, begin, end, s);
    else if (e.type == GRPO_DTYPE_BF16)
      squares<__nv_bfloat16>(e.grad, begin, end, s);
    else
      squares<__half>(e.grad, begin, end, s);
  }
  const double sum = cta_sum(s.total());
  if (threadIdx.x == 0) partials[blockIdx.x] = sum;
}

// norm and scale from the partial sums, in their order.
__global__ void __launch_bounds__(kThreads)
    grad_norm_finish_kernel(const double* partials, int count, double max_norm, float* out) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial sums are there
  double sum = 0.0;
  for (int i = static_cast<int>(threadIdx.x); i < count; i += kThreads) sum += partials[i];
  sum = cta_sum(sum);
  if (threadIdx.x != 0) return;
  const double norm = sqrt(sum);
  out[0] = static_cast<float>(norm);
  float scale = 1.f;
  if (!(out[0] <= FLT_MAX))
    scale = kNaN;
  else if (max_norm > 0.0)
    scale = static_cast<float>(fmin(1.0, max_norm / (norm + 1e-6)));
  out[1] = scale;
}

template <int N, int BITS>
cudaError_t launch_adamw(const AdamwEntry* e, const AdamwArgs& a, int chunks, cudaStream_t st) {
  AdamwTable<N> table;
  std::copy(e, e + a.count, table.e);
  std::fill(table.e + a.count, table.e + N, AdamwEntry());
  LaunchTimer timer("adamw_kernel", st);
  adamw_kernel<N, BITS><<<chunks, kStepThreads<BITS>, 0, st>>>(table, a);
  return cudaGetLastError();
}

template <int N>
cudaError_t launch_norm(const NormEntry* e, int count, int chunks, double* partials,
                        cudaStream_t st) {
  NormTable<N> table;
  std::copy(e, e + count, table.e);
  std::fill(table.e + count, table.e + N, NormEntry());
  LaunchTimer timer("grad_norm_kernel", st);
  grad_norm_kernel<N><<<std::min(chunks, kNormCtas), kThreads, 0, st>>>(table, count, chunks,
                                                                       partials);
  return cudaGetLastError();
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t dtype_bytes(int t) { return t == GRPO_DTYPE_FP32 ? 4 : 2; }
bool known_dtype(int t) { return t >= GRPO_DTYPE_BF16 && t <= GRPO_DTYPE_FP32; }
constexpr int64_t kMaxValues = 1LL << 40;

size_t norm_workspace(int32_t count) {
  const size_t launches = (static_cast<size_t>(count) + kNormTable - 1) / kNormTable;
  return std::max<size_t>(1, launches) * ((kNormCtas * sizeof(double) + 255) / 256 * 256);
}

int check_tensor(const grpo_adamw_tensor& t) {
  if (t.numel < 0) return GRPO_ERR_INVALID_ARG;
  if (t.numel > kMaxValues) return GRPO_ERR_UNSUPPORTED_SHAPE;
  if ((t.param_dtype != GRPO_DTYPE_FP32 && t.param_dtype != GRPO_DTYPE_BF16) ||
      !known_dtype(t.grad_dtype) || (t.state_bits != 8 && t.state_bits != 32) ||
      !(std::fabs(t.lr) <= 3e38f) || !(std::fabs(t.weight_decay) <= 3e38f))
    return GRPO_ERR_INVALID_ARG;
  if (t.copy_or_null != nullptr &&
      (t.param_dtype != GRPO_DTYPE_FP32 ||
       (t.copy_dtype != GRPO_DTYPE_BF16 && t.copy_dtype != GRPO_DTYPE_FP16)))
    return GRPO_ERR_INVALID_ARG;
  if (t.numel == 0 || t.grad == nullptr) return GRPO_OK;
  if (t.param == nullptr || t.m == nullptr || t.v == nullptr ||
      (t.state_bits == 8 && (t.m_scale == nullptr || t.v_scale == nullptr)))
    return GRPO_ERR_INVALID_ARG;
  const size_t state = t.state_bits == 8 ? 1 : 4;
  if (!aligned(t.param, dtype_bytes(t.param_dtype)) || !aligned(t.grad, dtype_bytes(t.grad_dtype)) ||
      !aligned(t.m, state) || !aligned(t.v, state) || !aligned(t.m_scale, 4) ||
      !aligned(t.v_scale, 4) || !aligned(t.copy_or_null, 2))
    return GRPO_ERR_MISALIGNED;
  return GRPO_OK;
}

}  // namespace
}  // namespace grpo

using namespace grpo;

extern "C" {

int grpo_grad_norm_workspace_size(int32_t count, size_t* bytes) {
  if (bytes == nullptr || count < 0) return GRPO_ERR_INVALID_ARG;
  *bytes = norm_workspace(count);
  return GRPO_OK;
}

int grpo_grad_norm(const grpo_grad* grads, int32_t count, double max_norm, float* out,
                   void* workspace, size_t workspace_bytes, void* stream) {
  const CallRange range("grpo_grad_norm");
  if (count < 0 || (count > 0 && grads == nullptr) || out == nullptr || workspace == nullptr ||
      max_norm != max_norm)
    return GRPO_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i) {
    if (grads[i].numel < 0 || grads[i].reserved != 0 || !known_dtype(grads[i].dtype))
      return GRPO_ERR_INVALID_ARG;
    if (grads[i].numel > kMaxValues) return GRPO_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(grads[i].data, dtype_bytes(grads[i].dtype))) return GRPO_ERR_MISALIGNED;
  }
  if (!aligned(out, 4) || !aligned(workspace, 256)) return GRPO_ERR_MISALIGNED;
  if (workspace_bytes < norm_workspace(count)) return GRPO_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  const int r = setup_device(&sms);
  if (r != GRPO_OK) return r;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  double* partials = static_cast<double*>(workspace);
  NormEntry e[kNormTable];
  int used = 0, sums = 0;
  int64_t chunks = 0;
  auto flush = [&]() {
    if (used == 0) return cudaSuccess;
    const int c = static_cast<int>(chunks);
    const cudaError_t err = used <= 64 ? launch_norm<64>(e, used, c, partials + sums, st)
                                       : launch_norm<kNormTable>(e, used, c, partials + sums, st);
    sums += std::min(c, kNormCtas);
    used = 0;
    chunks = 0;
    return err;
  };
  for (int i = 0; i < count; ++i) {
    if (grads[i].numel == 0 || grads[i].data == nullptr) continue;
    const int64_t more = (grads[i].numel + kNormChunk - 1) / kNormChunk;
    if (used == kNormTable && flush() != cudaSuccess) return GRPO_ERR_CUDA;
    e[used++] = {grads[i].data, grads[i].numel, static_cast<int>(chunks), grads[i].dtype};
    chunks += more;
    if (chunks > (1LL << 30)) return GRPO_ERR_UNSUPPORTED_SHAPE;
  }
  if (flush() != cudaSuccess) return GRPO_ERR_CUDA;
  // Its launch overlaps the end of the other (it waits for that itself).
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  LaunchTimer timer("grad_norm_finish_kernel", st);
  return cudaLaunchKernelEx(&cfg, grad_norm_finish_kernel,
                            static_cast<const double*>(partials), sums, max_norm,
                            out) == cudaSuccess
             ? GRPO_OK
             : GRPO_ERR_CUDA;
}

int grpo_adamw_step(const grpo_adamw_tensor* tensors, int32_t count,
                    const grpo_adamw_params* params, void* stream) {
  const CallRange range("grpo_adamw_step");
  if (count < 0 || (count > 0 && tensors == nullptr) || params == nullptr)
    return GRPO_ERR_INVALID_ARG;
  const grpo_adamw_params& q = *params;
  if (!(q.beta1 >= 0.0 && q.beta1 < 1.0) || !(q.beta2 >= 0.0 && q.beta2 < 1.0) ||
      !(q.eps >= 0.0) || (q.step_on_device == nullptr && q.step < 1))
    return GRPO_ERR_INVALID_ARG;
  if (!aligned(q.scale, 4) || !aligned(q.lr_factor, 4) || !aligned(q.step_on_device, 8))
    return GRPO_ERR_MISALIGNED;
  int64_t values = 0;
  for (int i = 0; i < count; ++i) {
    const int r = check_tensor(tensors[i]);
    if (r != GRPO_OK) return r;
    if (tensors[i].grad != nullptr) values += tensors[i].numel;
  }
  int sms = 0;
  const int r = setup_device(&sms);
  if (r != GRPO_OK) return r;
  AdamwArgs a;
  a.beta1 = static_cast<float>(q.beta1);
  a.beta2 = static_cast<float>(q.beta2);
  a.rest1 = static_cast<float>(1.0 - q.beta1);
  a.rest2 = static_cast<float>(1.0 - q.beta2);
  // An eps above 0 stays so, and normal (the step's quick inverse takes no subnormals); no
  // root but 0 is that small.
  a.eps = q.eps > 0.0 ? std::max(static_cast<float>(q.eps), FLT_MIN) : 0.f;
  // beta 0: its power is 0 (the logarithm a number that expm1 takes to -1).
  a.log1 = q.beta1 > 0.0 ? static_cast<float>(std::log(q.beta1)) : -200.f;
  a.log2 = q.beta2 > 0.0 ? static_cast<float>(std::log(q.beta2)) : -200.f;
  const double t = static_cast<double>(q.step_on_device == nullptr ? q.step : 1);
  a.fix1 = static_cast<float>(1.0 / (1.0 - std::pow(q.beta1, t)));
  a.fix2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(q.beta2, t)));
  a.seed = q.seed;
  a.step = q.step;
  a.scale = q.scale;
  a.lr_factor = q.lr_factor;
  a.step_on_device = q.step_on_device;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Tensors with moments of either kind have launches of their own.
  AdamwEntry e[kLargeTable];
  for (const int bits : {32, 8}) {
    // The largest chunk that still gives every SM eight CTAs: long chunks find their
    // tensor and work out the step less often, short ones fill the device.
    a.chunk = bits == 8 ? kStepChunk<8> : kStepChunk<32>;
    while (a.chunk > (bits == 8 ? 4 : 8) * kGroup && values / a.chunk < 8LL * sms) a.chunk /= 2;
    int64_t chunks = 0, place = 0;
    a.count = 0;
    auto flush = [&]() {
      if (a.count == 0) return cudaSuccess;
      const int c = static_cast<int>(chunks);
      const bool few = a.count <= kSmallTable;
      const cudaError_t err = bits == 32 ? (few ? launch_adamw<kSmallTable, 32>(e, a, c, st)
                                                : launch_adamw<kLargeTable, 32>(e, a, c, st))
                                         : (few ? launch_adamw<kSmallTable, 8>(e, a, c, st)
                                                : launch_adamw<kLargeTable, 8>(e, a, c, st));
      a.count = 0;
      chunks = 0;
      return err;
    };
    for (int i = 0; i < count; ++i) {
      const grpo_adamw_tensor& x = tensors[i];
      const int64_t at = place;
      place += (x.numel + kBlock - 1) / kBlock * kBlock;
      if (x.numel == 0 || x.grad == nullptr || x.state_bits != bits) continue;
      const int64_t more = (x.numel + a.chunk - 1) / a.chunk;
      if ((a.count == kLargeTable || chunks + more > (1LL << 30)) && flush() != cudaSuccess)
        return GRPO_ERR_CUDA;
      AdamwEntry& d = e[a.count++];
      d.param = x.param;
      d.grad = x.grad;
      d.m = x.m;
      d.v = x.v;
      d.m_scale = x.m_scale;
      d.v_scale = x.v_scale;
      d.copy = x.copy_or_null;
      d.numel = x.numel;
      d.place = at;
      d.lr = x.lr;
      d.decay = x.weight_decay;
      d.chunk = static_cast<int>(chunks);
      d.ptype = static_cast<uint8_t>(x.param_dtype);
      d.gtype = static_cast<uint8_t>(x.grad_dtype);
      d.ctype = static_cast<uint8_t>(x.copy_dtype);
      chunks += more;
    }
    if (flush() != cudaSuccess) return GRPO_ERR_CUDA;
  }
  return GRPO_OK;
}

}  // extern "C"
