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
// read once and held in registers: up to 16384 columns where rows start on 16
// bytes and shared memory holds one of them beside the parameters (not fp32 of
// 16384 columns with residual, weight and bias), else up to 8192; longer rows are
// walked three times. Statistics are fp32.
// What it took, at 131072 x 2880 in bf16 with residual and checkpoint (3.41 GB):
// loads into registers one row ahead 1615 us; rows in flight in shared memory
// 610; pairs of values and 32 of them a thread 568 to 580 (5.9 to 6.0 TB/s, of
// 6.8 measured for a copy; it follows how the five streams meet in DRAM).
#include <climits>

#include "norm_ring.cuh"

namespace grpo {
namespace {

// `lost` holds each warp's first row whose copy did not come, and one of them all.
__device__ __forceinline__ void gave_up(int* lost, int i) {
  atomicMin(&lost[(threadIdx.y * blockDim.x + threadIdx.x) >> 5], i);
  lost[kRingThreads / 32] = i;
}

// After the rows: a warp whose wait ran out has stored into z and the checkpoint
// what its copies did not bring, in that row and in all since. NaN over it, here:
// a branch for it in each row, or its state in registers, cost 3 to 5 % (131072
// x 2880 without a residual).
template <typename T, bool VEC, int CH>
__device__ __forceinline__ void lost_rows(const NormFwdArgs& a, const int* lost) {
  const int first = lost[(threadIdx.y * blockDim.x + threadIdx.x) >> 5];
  if (first == INT_MAX) return;
  const long long step = static_cast<long long>(gridDim.x) * blockDim.y;
  for (long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y + step * first;
       row < a.n; row += step) {
    if (!row_live(a.mask, row, a.n)) continue;
#pragma unroll 1
    for (int k = 0; k < 8 * CH; ++k) {
      const int col = chunk_col<VEC>(k >> 3, k & 7, threadIdx.x, blockDim.x);
      if (col >= a.d) continue;
      if (a.res != nullptr && a.z != nullptr) static_cast<T*>(a.z)[row * a.ldz + col] = T(kNaN);
      if (a.ck.q != nullptr) a.ck.q[row * a.ck.ldq + col] = kCkptNaN;
    }
  }
}

template <typename T, bool VEC, int CH, int KIND>
__global__ void __launch_bounds__(kRingThreads) norm_fwd_kernel(const NormFwdArgs a, const Ring ring) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float red[kMaxRows][2 * 2 * 16];
  __shared__ float warp_n[2][16];
  __shared__ int lost[kRingThreads / 32 + 1];
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
  const int fetches = fetch_count(count, row0, step, a.lost);
  const uint8_t* const mask = a.mask;
  // Thread 0: slots whose copies have not been waited for, and the next row to fetch.
  uint32_t pending = 0;
  int fetched = 0;
  const auto fetch = [&](int slot) {
    if (fetched >= fetches) return;
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
  for (int k = g * tpr + t; k <= kRingThreads / 32; k += tpr * blockDim.y) lost[k] = INT_MAX;
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
      ok = ok && row_wait(&bars[slot], (parity >> slot) & 1u,
                          [&] { gave_up(lost, i); });
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
        // A thread whose copy did not come has NaN: so has then all of the row.
        float m[1] = {warp_sum(ok ? sum_of(add2(s[0], s[1])) : kNaN)};
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
        const float sum = warp_sum(ok ? sum_of(add2(s[0], s[1])) : kNaN);
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
  __syncwarp();
  if (lost[kRingThreads / 32] != INT_MAX) lost_rows<T, VEC, CH>(a, lost);
}

// Rows that leave registers (unaligned ones beyond 8192 columns, others beyond
// kNormRegisterRow, and those that shared memory has no room for): the CTA walks
// over the row three times (sum, centred squares, output); the second and third
// walk find it in L2. A thread rereads only what it stored itself, so outputs may
// lie on the inputs. With residual and checkpoint in bf16: 4096 x 20480 203 us
// (3.7 TB/s), 4096 x 9001 160 us (2.1), 4096 x 16384 in registers 107 (5.7).
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
  // CTAs of up to 512 threads: the most rows under way on an SM (131072 x 2880
  // without a residual: 256 us, with 256 threads 289). Few rows go one to a CTA.
  RowShape s = ring_shape(a.d, VEC ? 4 : 2, kRingThreads);
  s.rows = static_cast<int>(std::max<long long>(1, std::min<long long>(s.rows, a.n / sms)));
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

}  // namespace

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

}  // namespace grpo
