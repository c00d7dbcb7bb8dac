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

// Each row of the CTA (threadIdx.y) has a ring of `slots` rows in shared memory,
// filled by bulk copies; a slot is filled again as soon as the row's sum has
// been taken, when every thread holds its values. Bulk copies start and end on
// 16 bytes: of a row that does not, the 16 bytes around its ends come too, and
// its values are read one by one (VEC false).
// The bytes in flight come from the ring, so what is left is issue slots: a
// thread holds up to 32 values, so that a row's fixed work (barriers, sums,
// addresses) is shared by few warps, and works on pairs of them.
struct Ring {
  int slots;           // rows in flight for each row of the CTA
  uint32_t row_bytes;  // of a slot
  int split;           // backward: CTAs of a row (a cluster of 2 beyond 8192 columns)
  int part;            // and columns of the first
};

// Shared memory: barriers, then the parameters as fp32, then the rings.
constexpr int kMaxSlots = 8;
constexpr int kMaxRows = 8;  // rows of a CTA
constexpr uint32_t kRingBars = kMaxRows * kMaxSlots * sizeof(uint64_t);

// Threads of a CTA at most.
constexpr int kRingThreads = 512;

// After a timeout: lets the copies still in flight land (within the same limit).
__device__ __forceinline__ void land(uint64_t* bars, int slots, uint32_t parity, uint32_t pending) {
  for (int s = 0; s < slots; ++s)
    if ((pending >> s) & 1u) row_wait(&bars[s], (parity >> s) & 1u);
}

// Two sums into the peer CTA's shared memory, counted on its barrier there.
// `at`, `bar`: addresses in this CTA of what is meant in the peer's.
__device__ __forceinline__ void send_sums(uint32_t at, uint32_t bar, uint32_t peer, float a,
                                          float b) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%2, %3}, [%1];" ::"r"(
          mapa_shared(at, peer)),
      "r"(mapa_shared(bar, peer)), "f"(a), "f"(b)
      : "memory");
}

__device__ __forceinline__ int param_width(int type) { return type == GRPO_DTYPE_FP32 ? 4 : 2; }

// Rows of the group that begins at `row`.
__device__ __forceinline__ int row_count(long long row, long long n, long long step) {
  return row < n ? static_cast<int>((n - 1 - row) / step) + 1 : 0;
}

template <typename T, bool VEC, int CH, int KIND>
__global__ void __launch_bounds__(kRingThreads) norm_fwd_kernel(const NormFwdArgs a, const Ring ring) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float red[kMaxRows][2 * 2 * 16];
  __shared__ float warp_n[2][16];
  __shared__ BlockTurn turns[VEC ? 1 : kRingThreads / 32];
  const int t = threadIdx.x, tpr = blockDim.x, g = threadIdx.y, d = a.d;
  const int warps = tpr >> 5;
  BlockTurn* const turn = turns + (VEC ? 0 : g * warps + (t >> 5));
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem) + g * kMaxSlots;
  float* const sw = reinterpret_cast<float*>(smem + kRingBars);
  float* const sb = sw + (a.weight != nullptr ? param_bytes(d) / 4 : 0);
  const uint32_t sw32 = smem_u32(sw), sb32 = smem_u32(sb);
  const uint32_t rows0 = smem_u32(sb + (a.bias != nullptr ? param_bytes(d) / 4 : 0)) +
                         g * ring.slots * ring.row_bytes;
  const uint32_t x_bytes = row_slot<T, VEC>(d);
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
    const T* px = static_cast<const T*>(a.x) + r * a.ldx;
    const T* pr = static_cast<const T*>(a.res) + r * a.ldr;
    mbar_arrive_expect_tx(&bars[slot],
                          row_span<T, VEC>(px, d) + (res ? row_span<T, VEC>(pr, d) : 0));
    bulk_row<T, VEC>(dst, px, d, &bars[slot]);
    if (res) bulk_row<T, VEC>(dst + x_bytes, pr, d, &bars[slot]);
  };
  if (t == 0) {
    for (int s = 0; s < ring.slots; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
    for (int s = 0; s < ring.slots; ++s) fetch(s);
  }
  for (int k = t; k < 2 * 2 * 16; k += tpr) red[g][k] = 0.f;
  if (a.weight != nullptr)
    stage_param<VEC>(sw, a.weight, a.wtype, d, g * tpr + t, tpr * blockDim.y);
  if (a.bias != nullptr) stage_param<VEC>(sb, a.bias, a.wtype, d, g * tpr + t, tpr * blockDim.y);
  // Columns that each warp of a row holds, and their inverse.
  if (KIND == GRPO_NORM_LAYER) {
    float n = 0.f;
#pragma unroll
    for (int k = 0; k < 8 * CH; ++k) n += chunk_col<VEC>(k >> 3, k & 7, t, tpr) < d ? 1.f : 0.f;
    n = warp_sum(n);
    if ((t & 31) == 0) {
      warp_n[0][t >> 5] = n;
      warp_n[1][t >> 5] = n > 0.f ? 1.f / n : 0.f;
    }
  }
  __syncthreads();

  const float inv_d = 1.f / static_cast<float>(d);
  const float inv_warp_n = KIND == GRPO_NORM_LAYER ? warp_n[1][t >> 5] : 0.f;
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
      const long long row = row0 + step * i;
      const uint32_t src =
          rows0 + slot * ring.row_bytes + row_shift<T, VEC>(static_cast<const T*>(a.x) + row * a.ldx);
      const uint32_t src_r = rows0 + slot * ring.row_bytes + x_bytes +
                             row_shift<T, VEC>(static_cast<const T*>(a.res) + row * a.ldr);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        lds_values<T, VEC>(src, c, t, tpr, d, v[c]);
        if (res) {
          f32x2 r[4];
          lds_values<T, VEC>(src_r, c, t, tpr, d, r);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[c][j] = add2(v[c][j], r[j]);
          // The stream holds z rounded; the norm is taken of what it holds.
          const Raw8<T> o = narrow2<T>(v[c]);
          if (z != nullptr) store_chunk<T, VEC>(z, o, c, t, tpr, d);
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
          if (VEC ? (c * tpr + t) * 8 >= d : 8 * c * tpr >= d) continue;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f32x2 e = add2(v[c][j], nmw);
            if (!VEC) {
              float lo, hi;
              split(e, lo, hi);
              e = pair(chunk_col<false>(c, 2 * j, t, tpr) < d ? lo : 0.f,
                       chunk_col<false>(c, 2 * j + 1, t, tpr) < d ? hi : 0.f);
            }
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
            const float e = sh[k] * warp_n[1][k] - mu;
            centred += sh[16 + k] + warp_n[0][k] * e * e;
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
        if (z != nullptr) store_chunk<T, VEC>(z, narrow2<T>(v[c]), c, t, tpr, d);
      }
    }
    // Every thread has its values (the sum's barrier, or the warp's).
    if (t == 0 && ok) fetch(slot);
    if (++slot == ring.slots) slot = 0;
    const f32x2 scale = pair(rstd, rstd), shift = pair(-mean, -mean);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (q != nullptr) {
        ckpt_store_chunk<T, VEC>(v[c], q, ex, c, t, tpr, d, turn);
      }
      if (VEC ? (c * tpr + t) * 8 >= d : 8 * c * tpr >= d) continue;
      if (live) {
        f32x2 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[c][j] = mul2(KIND == GRPO_NORM_LAYER ? add2(v[c][j], shift) : v[c][j], scale);
        if (a.weight != nullptr) {
          read_param<VEC>(sw32, c, t, tpr, d, w);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[c][j] = mul2(v[c][j], w[j]);
        }
        if (a.bias != nullptr) {
          read_param<VEC>(sb32, c, t, tpr, d, w);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[c][j] = add2(v[c][j], w[j]);
        }
      }
      store_chunk<T, VEC>(y, narrow2<T>(v[c]), c, t, tpr, d);
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
  __shared__ BlockTurn turns[VEC ? 1 : 16];
  const int t = threadIdx.x, tpr = blockDim.x, d = a.d;
  BlockTurn* const turn = turns + (VEC ? 0 : t >> 5);
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
        ckpt_store_chunk<T, VEC>({pair(v[0], v[1]), pair(v[2], v[3]), pair(v[4], v[5]), pair(v[6], v[7])},
                                 a.ck.q + row * a.ck.ldq, a.ck.ex + row * a.ck.lde, c, t, tpr, d, turn);
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
// so the sums are the same on every run. Rows in flight as in norm_fwd_kernel; a
// slot holds dy, then x (or its bytes and exponents), then dres. FULL: layer
// norm, or a bias gradient; else neither. 16 values a thread: with 32 the sums
// alone take 64 to 128 registers (131072 x 2880 layer norm: 789 us against 545).
template <typename T, bool VEC, int CH, bool CK, bool FULL>
__global__ void __launch_bounds__(kRingThreads) norm_bwd_kernel(const NormBwdArgs a, const Ring ring) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float red[kMaxRows][2 * 2 * 16];
  __shared__ __align__(8) uint64_t sums_bar[2];
  __shared__ __align__(8) float peer_sums[2][2];
  const int t = threadIdx.x, tpr = blockDim.x, g = threadIdx.y;
  // This CTA's columns [col0, col0 + d) of the row.
  const bool halved = ring.split == 2;
  const uint32_t rank = halved ? cluster_ctarank() : 0u;
  const int col0 = rank != 0 ? ring.part : 0;
  const int d = halved ? (rank != 0 ? a.d - ring.part : ring.part) : a.d;
  const int blk = static_cast<int>(blockIdx.x) / ring.split;
  const int blks = static_cast<int>(gridDim.x) / ring.split;
  const int warps = tpr >> 5;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem) + g * kMaxSlots;
  float* const sw = reinterpret_cast<float*>(smem + kRingBars);
  uint8_t* const ring0 =
      reinterpret_cast<uint8_t*>(sw + (a.weight != nullptr ? param_bytes(d) / 4 : 0));
  const uint32_t sw32 = smem_u32(sw);
  const uint32_t rows0 = smem_u32(ring0) + g * ring.slots * ring.row_bytes;
  const uint32_t t_bytes = row_slot<T, VEC>(d);
  // Of a checkpoint's row up to its padding, or (first of two CTAs) to `part`.
  const bool ends = !halved || rank != 0;
  const uint32_t q_bytes = static_cast<uint32_t>(ends ? a.ck.ldq - col0 : d);
  const uint32_t e_bytes =
      static_cast<uint32_t>(ends ? a.ck.lde - col0 / kCkptBlock : d / kCkptBlock);
  const uint32_t x_bytes = CK ? q_bytes + e_bytes : t_bytes;  // rows of 16 bytes
  const T* const g_dy = static_cast<const T*>(a.dy) + col0;
  const T* const g_x = static_cast<const T*>(a.x) + col0;
  const T* const g_res = static_cast<const T*>(a.dres) + col0;
  const bool res = a.dres != nullptr, layer = FULL && a.kind == GRPO_NORM_LAYER;
  const long long step = static_cast<long long>(blks) * blockDim.y;
  const long long row0 = static_cast<long long>(blk) * blockDim.y + g;
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
    const T* py = g_dy + r * a.lddy;
    const T* px = g_x + r * a.ldx;
    const T* pr = g_res + r * a.lddres;
    mbar_arrive_expect_tx(&bars[slot], row_span<T, VEC>(py, d) +
                                           (CK ? x_bytes : row_span<T, VEC>(px, d)) +
                                           (res ? row_span<T, VEC>(pr, d) : 0));
    bulk_row<T, VEC>(dst, py, d, &bars[slot]);
    if (CK) {
      bulk_load(dst + t_bytes, a.ck.q + r * a.ck.ldq + col0, q_bytes, &bars[slot]);
      bulk_load(dst + t_bytes + q_bytes, a.ck.ex + r * a.ck.lde + col0 / kCkptBlock, e_bytes,
                &bars[slot]);
    } else {
      bulk_row<T, VEC>(dst + t_bytes, px, d, &bars[slot]);
    }
    if (res) bulk_row<T, VEC>(dst + t_bytes + x_bytes, pr, d, &bars[slot]);
  };
  if (t == 0) {
    for (int s = 0; s < ring.slots; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
    for (int s = 0; s < ring.slots; ++s) fetch(s);
  }
  for (int k = t; k < 2 * 2 * 16; k += tpr) red[g][k] = 0.f;
  if (t == 0 && g == 0 && halved) {
    mbar_init(&sums_bar[0], 1);
    mbar_init(&sums_bar[1], 1);
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (a.weight != nullptr)
    stage_param<VEC>(sw, static_cast<const uint8_t*>(a.weight) + col0 * param_width(a.wtype),
                     a.wtype, d, g * tpr + t, tpr * blockDim.y);
  __syncwarp();
  if (halved) cluster_sync();  // the peer's barriers are there
  __syncthreads();

  f32x2 dw[CH][4], db[FULL ? CH : 1][4];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      dw[c][j] = 0ull;
      if (FULL) db[FULL ? c : 0][j] = 0ull;
    }
  const float inv_d = 1.f / static_cast<float>(a.d);
  T* dx = static_cast<T*>(a.dx) + row0 * a.lddx + col0;
  uint32_t swaps = 0;  // rows whose sums the two CTAs have told each other
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
      for (int c = 0; c < CH; ++c) store_chunk<T, VEC>(dx, narrow2<T>(zero), c, t, tpr, d);
    } else {
      ok = ok && row_wait(&bars[slot], (parity >> slot) & 1u);
      if (ok) {
        parity ^= 1u << slot;
        pending &= ~(1u << slot);
      }
      const long long row = row0 + step * i;
      const uint32_t src = rows0 + slot * ring.row_bytes;
      const uint32_t src_y = src + row_shift<T, VEC>(g_dy + row * a.lddy);
      const uint32_t src_x = src + t_bytes + (CK ? 0 : row_shift<T, VEC>(g_x + row * a.ldx));
      const uint32_t src_r = src + t_bytes + x_bytes + row_shift<T, VEC>(g_res + row * a.lddres);
      const f32x2 scale = pair(rstd, rstd), shift = pair(-mean, -mean);
      f32x2 u[CH][4], h[CH][4];
      Raw8<T> rr[CH];
      f32x2 su = 0ull, suh = 0ull;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (VEC ? (c * tpr + t) * 8 >= d : 8 * c * tpr >= d) continue;
        lds_values<T, VEC>(src_y, c, t, tpr, d, u[c]);
        if (CK)
          lds_ckpt<VEC>(src_x, src_x + q_bytes, c, t, tpr, d, h[c]);
        else
          lds_values<T, VEC>(src_x, c, t, tpr, d, h[c]);
        if (res) rr[c] = lds_chunk<T, VEC>(src_r, c, t, tpr, d);
        f32x2 w[4];
        if (a.weight != nullptr) read_param<VEC>(sw32, c, t, tpr, d, w);
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
      __syncwarp();
      if (halved) {
        // Tell the peer, and wait for its part (two places in turn: it cannot
        // be two rows ahead). Both add in the same order.
        const uint32_t b = swaps & 1u;
        if (t == 0) {
          mbar_arrive_expect_tx(&sums_bar[b], 8);
          send_sums(smem_u32(&peer_sums[b][0]), smem_u32(&sums_bar[b]), rank ^ 1u, s[0],
                    FULL ? s[FULL ? 1 : 0] : 0.f);
        }
        ok = ok && row_wait(&sums_bar[b], (swaps >> 1) & 1u);
        ++swaps;
#pragma unroll
        for (int k = 0; k < (FULL ? 2 : 1); ++k)
          s[k] = rank == 0 ? s[k] + peer_sums[b][k] : peer_sums[b][k] + s[k];
      }
      const float c1 = layer ? s[FULL ? 1 : 0] * inv_d : 0.f;
      const float c2 = ok ? s[0] * inv_d : __uint_as_float(0x7fc00000u);
      const f32x2 n1 = pair(-c1, -c1), n2 = pair(-c2, -c2);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (VEC ? (c * tpr + t) * 8 >= d : 8 * c * tpr >= d) continue;
        f32x2 r[4] = {0ull, 0ull, 0ull, 0ull};
        if (res) widen2(rr[c], r);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (FULL) u[c][j] = add2(u[c][j], n1);
          u[c][j] = fma2(fma2(h[c][j], n2, u[c][j]), scale, r[j]);
        }
        store_chunk<T, VEC>(dx, narrow2<T>(u[c]), c, t, tpr, d);
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
  __syncwarp();
  if (halved) cluster_sync();  // nothing more arrives from the peer
  const bool want_db = FULL && a.dbias != nullptr;
  if (a.dweight == nullptr && !want_db) return;
  // The CTA's rows in flight, added in their order; the rings have been read.
  float* const cw = reinterpret_cast<float*>(ring0);
  float* const cb = cw + d;
  float* pw = a.partials + static_cast<long long>(blk) * a.d + col0;
  float* pb = pw + static_cast<long long>(blks) * a.d;
  if (blockDim.y == 1) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      store_sums<VEC>(pw, dw[c], c, t, tpr, d);
      if (want_db) store_sums<VEC>(pb, db[FULL ? c : 0], c, t, tpr, d);
    }
    return;
  }
  __syncthreads();
  for (int k = 0; k < static_cast<int>(blockDim.y); ++k) {
    if (g == k) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c0 = chunk_col<VEC>(c, 2 * j, t, tpr), c1 = chunk_col<VEC>(c, 2 * j + 1, t, tpr);
          float lo, hi;
          split(dw[c][j], lo, hi);
          if (c0 < d) cw[c0] = k == 0 ? lo : cw[c0] + lo;
          if (c1 < d) cw[c1] = k == 0 ? hi : cw[c1] + hi;
          if (want_db) {
            split(db[FULL ? c : 0][j], lo, hi);
            if (c0 < d) cb[c0] = k == 0 ? lo : cb[c0] + lo;
            if (c1 < d) cb[c1] = k == 0 ? hi : cb[c1] + hi;
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
#pragma unroll 4
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
  // Four rows' loads at a time, in flight together.
  const long long step = static_cast<long long>(gridDim.y) * 8;
  for (long long row = static_cast<long long>(blockIdx.y) * 8 + g; row < a.n; row += 4 * step) {
    Raw8<T> ry[4];
    RawStream<T, VEC, CK> rx[4];
    float rs[4], mean[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const long long r = row + k * step;
      rs[k] = mean[k] = 0.f;
      if (!row_live(a.mask, r, a.n)) continue;
      ry[k] = load_chunk<T, VEC>(dy + r * a.lddy, 0, t, 32, dd);
      rx[k].load(s, r, 0, t, 32);
      rs[k] = a.rstd[r];
      if (a.kind != GRPO_NORM_RMS) mean[k] = a.mean[r];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (!row_live(a.mask, row + k * step, a.n)) continue;
      float u[8], h[8];
      widen(ry[k], u);
      rx[k].get(h);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dw[j] += u[j] * ((h[j] - mean[k]) * rs[k]);
        db[j] += u[j];
      }
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
// The most values a thread, up to 8 `most`, that leave no more than a
// tenth of the threads idle (else the fewest idle ones); CTAs of about
// `threads` threads.
RowShape ring_shape(int d, int most, int threads) {
  RowShape best = {0, 0, 0};
  int best_room = 0;
  for (int ch = most; ch >= 1; --ch) {
    const int tpr = (d + 256 * ch - 1) / (256 * ch) * 32;
    const int room = tpr * 8 * ch;
    if (tpr > kRingThreads || (best.ch != 0 && room >= best_room)) continue;
    best = {tpr, std::min(kMaxRows, std::max(1, threads / tpr)), ch};
    best_room = room;
    if (10 * room <= 11 * d) break;
  }
  return best;
}

constexpr size_t kSmemMax = 227 * 1024 - 22528;  // less the kernels' static arrays
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
  r.split = 1;
  r.part = 0;
  return r;
}

// Opts a kernel in to large shared memory, once.
template <auto Kernel>
bool opted_in() {
  static const bool ok = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              static_cast<int>(kSmemMax)) == cudaSuccess;
  return ok;
}

// CTAs of a kernel that fit an SM; the last answer is kept for calls of one shape.
template <auto Kernel>
cudaError_t ctas_per_sm(int threads, size_t smem, int* n) {
  static std::atomic<uint64_t> last{0};
  const uint64_t key = (static_cast<uint64_t>(smem) << 24) | (static_cast<uint64_t>(threads) << 8);
  const uint64_t seen = last.load(std::memory_order_relaxed);
  if (seen != 0 && (seen & ~uint64_t{0xff}) == key) {
    *n = static_cast<int>(seen & 0xff);
    return cudaSuccess;
  }
  if (!opted_in<Kernel>()) return cudaErrorInvalidValue;
  const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, Kernel, threads, smem);
  if (e == cudaSuccess) last.store(key | static_cast<uint64_t>(*n), std::memory_order_relaxed);
  return e;
}

template <typename T, bool VEC>
cudaError_t fwd_long(const NormFwdArgs& a, int sms, cudaStream_t st) {
  const int grid = static_cast<int>(std::min<long long>(a.n, 3LL * sms));
  LaunchTimer timer("norm_fwd_long_kernel", st);
  norm_fwd_long_kernel<T, VEC><<<grid, 512, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T, bool VEC, int CH, int KIND>
cudaError_t fwd_ring(const NormFwdArgs& a, const RowShape& s, int sms, cudaStream_t st) {
  constexpr auto kernel = norm_fwd_kernel<T, VEC, CH, KIND>;
  const size_t fixed =
      kRingBars + param_bytes(a.d) * ((a.weight != nullptr) + (a.bias != nullptr));
  const Ring ring = make_ring(row_slot<T, VEC>(a.d) * (a.res != nullptr ? 2 : 1), s.rows, fixed);
  const size_t smem = fixed + static_cast<size_t>(ring.slots) * ring.row_bytes * s.rows;
  if (smem > kSmemMax) return fwd_long<T, VEC>(a, sms, st);
  int per_sm = 0;
  cudaError_t e = ctas_per_sm<kernel>(s.tpr * s.rows, smem, &per_sm);
  if (e != cudaSuccess) return e;
  const long long units = (a.n + s.rows - 1) / s.rows;
  const int grid = static_cast<int>(std::min<long long>(units, std::max(1, per_sm) * sms));
  LaunchTimer timer("norm_fwd_kernel", st);
  kernel<<<grid, dim3(s.tpr, s.rows), smem, st>>>(a, ring);
  return cudaGetLastError();
}

template <typename T, bool VEC, int KIND>
cudaError_t fwd_kind(const NormFwdArgs& a, int sms, cudaStream_t st) {
  // One by one, 16 values a thread: 32 take 228 registers.
  const RowShape s = ring_shape(a.d, VEC ? 4 : 2, kRowThreads);
  switch (s.ch) {
    case 1: return fwd_ring<T, VEC, 1, KIND>(a, s, sms, st);
    case 2: return fwd_ring<T, VEC, 2, KIND>(a, s, sms, st);
    case 3:
      if constexpr (VEC) return fwd_ring<T, VEC, 3, KIND>(a, s, sms, st);
    case 4:
      if constexpr (VEC) return fwd_ring<T, VEC, 4, KIND>(a, s, sms, st);
    default: return fwd_long<T, VEC>(a, sms, st);
  }
}

template <typename T, bool VEC>
cudaError_t fwd_any(const NormFwdArgs& a, int sms, cudaStream_t st) {
  return a.kind == GRPO_NORM_RMS ? fwd_kind<T, VEC, GRPO_NORM_RMS>(a, sms, st)
                                 : fwd_kind<T, VEC, GRPO_NORM_LAYER>(a, sms, st);
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

template <typename T, bool VEC, int CH, bool CK, bool FULL>
cudaError_t bwd_ring(const NormBwdArgs& a, const RowShape& s, int part, int sms, cudaStream_t st) {
  constexpr auto kernel = norm_bwd_kernel<T, VEC, CH, CK, FULL>;
  const int d = part != 0 ? part : a.d;  // columns of a CTA
  const size_t fixed = kRingBars + (a.weight != nullptr ? param_bytes(d) : 0);
  const uint32_t t_bytes = row_slot<T, VEC>(d);
  const uint32_t ck_bytes = static_cast<uint32_t>(
      part != 0 ? part + part / 32 : a.ck.ldq + a.ck.lde);
  Ring ring = make_ring(t_bytes * (a.dres != nullptr ? 2 : 1) + (CK ? ck_bytes : t_bytes), s.rows,
                        fixed);
  ring.split = part != 0 ? 2 : 1;
  ring.part = part;
  size_t smem = static_cast<size_t>(ring.slots) * ring.row_bytes * s.rows;
  if (s.rows > 1) smem = std::max(smem, static_cast<size_t>(d) * 8);
  smem += fixed;
  int per_sm = 0;
  cudaError_t e = ctas_per_sm<kernel>(s.tpr * s.rows, smem, &per_sm);
  if (e != cudaSuccess) return e;
  const long long units = (a.n + s.rows - 1) / s.rows;
  const int groups = static_cast<int>(
      std::min<long long>(std::min<long long>(units, kNormMaxPartials),
                          std::max(1, per_sm) * (sms / ring.split)));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(groups * ring.split);
  cfg.blockDim = dim3(s.tpr, s.rows);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ring.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ring.split == 2 ? 1 : 0;
  {
    LaunchTimer timer("norm_bwd_kernel", st);
    e = cudaLaunchKernelEx(&cfg, kernel, a, ring);
  }
  return e != cudaSuccess ? e : finish(a, groups, st);
}

template <typename T, bool VEC, bool CK, bool FULL>
cudaError_t bwd_kind(const NormBwdArgs& a, int sms, cudaStream_t st) {
  // Beyond 8192 columns two CTAs share a row, at a multiple of 512 columns (16
  // exponents: 16 bytes).
  const int part = a.d > kRingThreads * 16 ? ((a.d + 1) / 2 + 511) / 512 * 512 : 0;
  const RowShape s = ring_shape(part != 0 ? part : a.d, 2, kRowThreads);
  if (s.ch == 1) return bwd_ring<T, VEC, 1, CK, FULL>(a, s, part, sms, st);
  return bwd_ring<T, VEC, 2, CK, FULL>(a, s, part, sms, st);
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
  return a.dbias != nullptr || a.kind == GRPO_NORM_LAYER
             ? bwd_kind<T, VEC, CK, true>(a, sms, st)
             : bwd_kind<T, VEC, CK, false>(a, sms, st);
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
