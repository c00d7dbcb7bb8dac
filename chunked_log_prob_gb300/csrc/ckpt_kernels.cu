// Activations to 8 bits and back: e4m3 values, one power of two per 32 columns
// of a row (the format is described in row_ops.cuh).
//
// Memory bound: one read and one write of everything (131072 x 2880 in bf16, 1.15
// GB: packing 201 us, unpacking 187; 5.7 and 6.1 TB/s). Four neighbouring lanes
// hold a block, 8 columns each; the blocks of all rows are dealt to the warps in
// order, so that no lane idles but in a row's last block. A thread has kAhead
// blocks' loads in flight. Rows that are not on 16 bytes go through 1 KB of
// shared memory a warp, so that their loads and stores are of neighbouring
// elements.
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

constexpr int kThreads = 256;
constexpr int kAhead = 4;

// Blocks are walked in steps of all threads' blocks; the place (row, block in
// the row) moves on without a division.
struct Walk {
  long long rows;  // of a step
  int blocks;      // and blocks beyond them
  int per_row;     // blocks of a row
};
struct Place {
  long long row;
  int block;
  __device__ __forceinline__ void next(const Walk& w) {
    row += w.rows;
    block += w.blocks;
    if (block >= w.per_row) {
      block -= w.per_row;
      ++row;
    }
  }
};
// The place of this thread's first block.
__device__ __forceinline__ Place first_place(const Walk& w) {
  const long long b = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) >> 2;
  return {b / w.per_row, static_cast<int>(b % w.per_row)};
}

// Rows that are not on 16 bytes: the warp's 8 blocks are loaded or stored one
// after the other, a column to a lane. Where they are, from the lanes that hold
// them: the block's offset in elements, and its columns.
__device__ __forceinline__ long long block_offset(long long mine, int j) {
  return __shfl_sync(0xffffffffu, mine, 4 * j);
}
__device__ __forceinline__ int block_columns(int mine, int j) {
  return __shfl_sync(0xffffffffu, mine, 4 * j);
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) ckpt_pack_kernel(const CkptArgs a, const Walk walk) {
  // VEC false: the warp's 8 blocks on their way between the two orders.
  __shared__ float turn[VEC ? 1 : kThreads / 4][VEC ? 1 : 33];
  const int sub = threadIdx.x & 3, lane = threadIdx.x & 31;
  float(*const blocks)[VEC ? 1 : 33] = turn + (VEC ? 0 : (threadIdx.x >> 5) * 8);
  Place p = first_place(walk);
  // All lanes of a warp stay in the loop together (shuffles): while its first
  // lane's block exists.
  while (__shfl_sync(0xffffffffu, p.row < a.n ? 1 : 0, 0)) {
    Place at[kAhead];
    Raw8<T> raw[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      at[k] = p;
      const int col = p.block * kCkptBlock + sub * 8;
      const bool read = p.row < a.n && (a.mask == nullptr || a.mask[p.row] != 0);
      const T* row = static_cast<const T*>(a.x) + p.row * a.ld;
      if (VEC) {
        uint4* w = reinterpret_cast<uint4*>(&raw[k]);
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(raw[k]) / 16); ++i)
          w[i] = read && col < a.d ? reinterpret_cast<const uint4*>(row + col)[i]
                                   : make_uint4(0, 0, 0, 0);
      } else {
        const long long off = p.row * a.ld + p.block * kCkptBlock;
        const int columns = read ? min(kCkptBlock, a.d - p.block * kCkptBlock) : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const long long o = block_offset(off, j);
          raw[k].e[j] = lane < block_columns(columns, j)
                            ? static_cast<const T*>(a.x)[o + lane]
                            : T(0.f);
        }
      }
      p.next(walk);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      f32x2 v[4];
      widen2(raw[k], v);
      if (!VEC) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float lo, hi;
          split(v[j >> 1], lo, hi);
          blocks[j][lane] = (j & 1) ? hi : lo;
        }
        __syncwarp();
        const float* const b = blocks[lane >> 2] + 8 * sub;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = pair(b[2 * j], b[2 * j + 1]);
      }
      int e;
      const uint2 w = ckpt_encode<T>(v, e);
      const int col = at[k].block * kCkptBlock + sub * 8;
      if (at[k].row < a.n && col < a.d) {
        uint8_t* q = a.ck.q + at[k].row * a.ck.ldq + col;
        *reinterpret_cast<uint2*>(q) = w;  // zeros into the padding behind d
        if (sub == 0) a.ck.ex[at[k].row * a.ck.lde + at[k].block] = static_cast<uint8_t>(e);
      }
    }
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) ckpt_unpack_kernel(const CkptArgs a, const Walk walk) {
  __shared__ float turn[VEC ? 1 : kThreads / 4][VEC ? 1 : 33];
  const int sub = threadIdx.x & 3, lane = threadIdx.x & 31;
  float(*const blocks)[VEC ? 1 : 33] = turn + (VEC ? 0 : (threadIdx.x >> 5) * 8);
  Place p = first_place(walk);
  while (__shfl_sync(0xffffffffu, p.row < a.n ? 1 : 0, 0)) {
    Place at[kAhead];
    uint2 w[kAhead];
    uint32_t e[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      at[k] = p;
      const int col = p.block * kCkptBlock + sub * 8;
      w[k] = make_uint2(0, 0);
      e[k] = kCkptBias;
      // A row's bytes are padded to 16: the last piece is read whole.
      if (p.row < a.n && col < a.d) {
        w[k] = *reinterpret_cast<const uint2*>(a.ck.q + p.row * a.ck.ldq + col);
        e[k] = a.ck.ex[p.row * a.ck.lde + p.block];
      }
      p.next(walk);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      f32x2 v[4];
      const float f = ckpt_factor(e[k]);
      const f32x2 ff = pair(f, f);
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const float2 x = unpack_e4m3x2((h < 2 ? w[k].x : w[k].y) >> (16 * (h & 1)));
        v[h] = mul2(pair(x.x, x.y), ff);
      }
      const int col = at[k].block * kCkptBlock + sub * 8;
      const bool write = at[k].row < a.n;
      if (VEC) {
        if (write && col < a.d)
          store_raw(static_cast<T*>(a.out) + at[k].row * a.ld + col, narrow2<T>(v));
      } else {
        __syncwarp();
        float* const b = blocks[lane >> 2] + 8 * sub;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float lo, hi;
          split(v[j], lo, hi);
          b[2 * j] = lo;
          b[2 * j + 1] = hi;
        }
        __syncwarp();
        const long long off = at[k].row * a.ld + at[k].block * kCkptBlock;
        const int columns = write ? min(kCkptBlock, a.d - at[k].block * kCkptBlock) : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const long long o = block_offset(off, j);
          if (lane < block_columns(columns, j)) static_cast<T*>(a.out)[o + lane] = T(blocks[j][lane]);
        }
      }
    }
  }
}

template <typename T, bool VEC, bool PACK>
cudaError_t run(const CkptArgs& a, int sms, cudaStream_t st) {
  const int per_row = (a.d + kCkptBlock - 1) / kCkptBlock;
  const long long threads = 4 * a.n * per_row;
  const int grid = static_cast<int>(std::min<long long>(
      (threads + kThreads - 1) / kThreads, 8LL * sms));
  const long long step = static_cast<long long>(grid) * kThreads / 4;
  const Walk walk = {step / per_row, static_cast<int>(step % per_row), per_row};
  LaunchTimer timer(PACK ? "ckpt_pack_kernel" : "ckpt_unpack_kernel", st);
  if (PACK)
    ckpt_pack_kernel<T, VEC><<<grid, kThreads, 0, st>>>(a, walk);
  else
    ckpt_unpack_kernel<T, VEC><<<grid, kThreads, 0, st>>>(a, walk);
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
