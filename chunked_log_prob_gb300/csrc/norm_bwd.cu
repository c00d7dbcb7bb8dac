// Layer norm and RMS norm, backward (formulas in norm_fwd.cu).
//
// Memory bound, and near the issue limit: some 20 instructions a value with the
// sums for dw in registers, 12 to 16 warps an SM. At 131072 x 2880, layer norm
// from the stream (3.02 GB): loads into registers 1876 us, rows in flight in
// shared memory 646, pairs of values 542 to 560 (5.4 to 5.6 TB/s). Reading the row
// a second time from shared memory instead of holding it over the sum was slower
// (582: its instructions cost more than its registers save).
#include "norm_ring.cuh"

namespace grpo {
namespace {

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
template <typename T, bool VEC, int CH, bool CK, bool FULL, int SPLIT>
__global__ void __launch_bounds__(kRingThreads) norm_bwd_kernel(const NormBwdArgs a, const Ring ring) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float red[kMaxRows][2 * 2 * 16];
  __shared__ __align__(8) uint64_t sums_bar[2];
  __shared__ __align__(8) float peer_sums[2][2];
  const int t = threadIdx.x, tpr = blockDim.x, g = threadIdx.y;
  // This CTA's columns [col0, col0 + d) of the row.
  constexpr bool halved = SPLIT == 2;
  const uint32_t rank = halved ? cluster_ctarank() : 0u;
  const int col0 = rank != 0 ? ring.part : 0;
  const int d = halved ? (rank != 0 ? a.d - ring.part : ring.part) : a.d;
  const int blk = static_cast<int>(blockIdx.x) / SPLIT;
  const int blks = static_cast<int>(gridDim.x) / SPLIT;
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
  const int fetches = fetch_count(count, row0, step, rank == 0 ? a.lost : kNoneLost);
  const uint8_t* const mask = a.mask;
  uint32_t pending = 0;
  int fetched = 0;
  const auto fetch = [&](int slot) {
    if (fetched >= fetches) return;
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
  bool heard = true;  // the peer's sums have come so far
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
      // A thread whose copy did not come has NaN: so has then all of the row's dx.
      s[0] = warp_sum(ok ? sum_of(suh) : kNaN);
      if (FULL) s[FULL ? 1 : 0] = warp_sum(sum_of(su));
      join_warps(s, t, warps, g + 1, red[g], phase);
      if (t == 0 && ok) fetch(slot);
      __syncwarp();
      if (halved) {
        // Tell the peer, and wait for its part (two places in turn: it cannot
        // be two rows ahead). Both add in the same order. This goes on when a
        // copy did not come, or the CTAs would lose count of each other: a row
        // then takes the peer up to kWaitLimitCycles, and this waits longer.
        const uint32_t b = swaps & 1u;
        if (t == 0) {
          if (heard) mbar_arrive_expect_tx(&sums_bar[b], 8);
          send_sums(smem_u32(&peer_sums[b][0]), smem_u32(&sums_bar[b]), rank ^ 1u, s[0],
                    FULL ? s[FULL ? 1 : 0] : 0.f);
        }
        heard = heard && row_wait(&sums_bar[b], (swaps >> 1) & 1u, [] {}, 4 * kWaitLimitCycles);
        ++swaps;
#pragma unroll
        for (int k = 0; k < (FULL ? 2 : 1); ++k)
          s[k] = rank == 0 ? s[k] + peer_sums[b][k] : peer_sums[b][k] + s[k];
      }
      const float c1 = layer ? s[FULL ? 1 : 0] * inv_d : 0.f;
      const float c2 = heard ? s[0] * inv_d : kNaN;
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
    }
    if (++slot == ring.slots) slot = 0;
    dx += step * a.lddx;
    live = live1;
  }
  land(bars, ring.slots, parity, pending);
  __syncwarp();
  if (halved) {
    cluster_sync();  // nothing more arrives from the peer
    if (!heard)      // or what it sent last is on its way: half a millisecond
      for (const long long t0 = clock64(); clock64() - t0 < (1 << 20);) {
      }
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

// Rows beyond kNormRegisterRow columns: dx in two walks over the row. From a
// checkpoint with dres, bf16, weight gradients included: 4096 x 20480 265 us (2.2
// TB/s), 4096 x 20001 865 us (one value a load), 4096 x 16384 in registers 99 (4.8).
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
// `partials` is written by that kernel after this one has started, so it must not
// be read as constant data (no __restrict__ here).
__global__ void __launch_bounds__(512) norm_bwd_finish_kernel(const float* partials,
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

template <typename T, bool VEC, int CH, bool CK, bool FULL, int SPLIT>
cudaError_t bwd_ring(const NormBwdArgs& a, const RowShape& s, int part, int sms, cudaStream_t st) {
  constexpr auto kernel = norm_bwd_kernel<T, VEC, CH, CK, FULL, SPLIT>;
  const int d = part != 0 ? part : a.d;  // columns of a CTA
  const size_t fixed = kRingBars + (a.weight != nullptr ? param_bytes(d) : 0);
  const uint32_t t_bytes = row_slot<T, VEC>(d);
  const uint32_t ck_bytes = static_cast<uint32_t>(
      part != 0 ? part + part / 32 : a.ck.ldq + a.ck.lde);
  Ring ring = make_ring(t_bytes * (a.dres != nullptr ? 2 : 1) + (CK ? ck_bytes : t_bytes), s.rows,
                        fixed);
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
                          std::max(1, per_sm) * (sms / SPLIT)));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(groups * SPLIT);
  cfg.blockDim = dim3(s.tpr, s.rows);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = SPLIT;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT == 2 ? 1 : 0;
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
  if (part != 0) return bwd_ring<T, VEC, 2, CK, FULL, 2>(a, s, part, sms, st);
  if (s.ch == 1) return bwd_ring<T, VEC, 1, CK, FULL, 1>(a, s, part, sms, st);
  return bwd_ring<T, VEC, 2, CK, FULL, 1>(a, s, part, sms, st);
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

cudaError_t launch_norm_bwd(const NormBwdArgs& a, int dtype, bool vec, int sms, cudaStream_t st) {
  if (a.n == 0) return finish(a, 0, st);
  switch (dtype) {
    case GRPO_DTYPE_BF16: return bwd_typed<__nv_bfloat16>(a, vec, sms, st);
    case GRPO_DTYPE_FP16: return bwd_typed<__half>(a, vec, sms, st);
    default: return bwd_typed<float>(a, vec, sms, st);
  }
}

}  // namespace grpo
