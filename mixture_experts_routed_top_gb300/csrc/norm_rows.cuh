// Device code that the norms share (block_norm.cu, layer_norm.cu): rows in registers,
// sums over a row, the ring of rows in shared memory and its edges.
#pragma once

#include <math.h>

#include <algorithm>
#include <atomic>

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

// Eight consecutive elements of a row as floats.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint4 u;
  u.x = pack_bf16x2(v[0], v[1]);
  u.y = pack_bf16x2(v[2], v[3]);
  u.z = pack_bf16x2(v[4], v[5]);
  u.w = pack_bf16x2(v[6], v[7]);
  *reinterpret_cast<uint4*>(p) = u;
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ float get(const float* p) { return *p; }
__device__ __forceinline__ float get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// The columns of a row that a thread holds: NV pieces of 8.  VEC: piece v is
// columns 8 (tx + TX v) .. +7, moved in 16-byte vectors (H % 8 == 0, rows
// 16-byte aligned); otherwise single columns TX apart, for any H and stride.
template <bool VEC, int NV>
struct Cols {
  int tx, TX, H;
  __device__ __forceinline__ int col(int v, int e) const {
    return VEC ? (tx + TX * v) * 8 + e : tx + TX * (v * 8 + e);
  }
  template <typename T>
  __device__ __forceinline__ void load(const T* row, int v, float (&x)[8], float fill) const {
    if (VEC) {
      if (col(v, 0) < H) {
        load8(row + col(v, 0), x);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fill;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = col(v, e) < H ? get(row + col(v, e)) : fill;
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, int v, const float (&x)[8]) const {
    if (VEC) {
      if (col(v, 0) < H) store8(row + col(v, 0), x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col(v, e) < H) put(row + col(v, e), x[e]);
    }
  }
  // a vector of fp32 or bf16 weights (16-byte aligned where VEC)
  __device__ __forceinline__ void load_any(const void* p, bool bf16, int v, float (&x)[8],
                                           float fill) const {
    if (bf16) load(static_cast<const __nv_bfloat16*>(p), v, x, fill);
    else load(static_cast<const float*>(p), v, x, fill);
  }
};

// Sums of N values over a block of whole warps.  Every thread gets the
// same bits: the warps' sums are added in warp order.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* s_red, int warps) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v[n] += __shfl_xor_sync(0xffffffffu, v[n], off);
  if (warps == 1) return;
  const int warp = threadIdx.x >> 5;
  __syncthreads();  // the previous sums have been read
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) s_red[warp * N + n] = v[n];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = 0.f;
  for (int w = 0; w < warps; ++w)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += s_red[w * N + n];
}

constexpr int kMaxRed = 32 * 4;  // warps of a block x values of a reduction

// Sums of the blocks' partial rows: 32 columns x 8 slices of the blocks per
// thread block, each slice added in block order, then the 8 slices in order.
__global__ void __launch_bounds__(256)
    norm_partials_kernel(const float* __restrict__ partials, int blocks, int n_part, int H,
                               float* o0, float* o1, float* o2) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float s[8][33];
  const int x = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + x, p = blockIdx.y;
  float sum = 0.f;
  if (col < H)
#pragma unroll 8
    for (int b = sl; b < blocks; b += 8)
      sum += partials[(static_cast<long>(b) * n_part + p) * H + col];
  s[sl][x] = sum;
  __syncthreads();
  if (sl == 0 && col < H) {
#pragma unroll
    for (int i = 1; i < 8; ++i) sum += s[i][x];
    (p == 0 ? o0 : p == 1 ? o1 : o2)[col] = sum;
  }
}

// ------------------------------------------------------------ streamed rows
// Rows of H <= 8192 columns.  Blocks of up to 512 threads stay on their SM and
// walk over the rows; a thread holds the same NV pieces of 8 columns of every
// row (so weights and sums over tokens stay in registers), and the next rows
// are copied into a ring in shared memory (cp.async), so loads run while the
// block computes.  Where H % 8 == 0 and rows start at 16 bytes, a thread copies
// its own pieces into its own slots: no thread reads another's, so the ring
// needs no barrier; the block meets only for the sums.
constexpr int kRingBytes = 200 * 1024;   // rings of an SM's blocks together, at most

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// `bytes` of the 16 from memory, zeros for the others.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const F2 (&v)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 q = parts(v[i]);
    w[i] = pack_bf16x2(q.x, q.y);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const F2 (&v)[4]) {
  const float2 a = parts(v[0]), b = parts(v[1]), c = parts(v[2]), d = parts(v[3]);
  reinterpret_cast<float4*>(p)[0] = make_float4(a.x, a.y, b.x, b.y);
  reinterpret_cast<float4*>(p)[1] = make_float4(c.x, c.y, d.x, d.y);
}
// 8 weights (or per-channel gates) of a thread's columns, next to each other or
// (EDGE) 32 apart; 1 where p is null and 0 past the row's end.
template <bool EDGE>
__device__ __forceinline__ void weights8(const void* p, bool bf16, int col, int H, F2 (&v)[4]) {
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = col + (EDGE ? 32 * e : 0) < H ? 1.f : 0.f;
  if (EDGE) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = col + 32 * e;
      if (p != nullptr && c < H)
        f[e] = bf16 ? get(static_cast<const __nv_bfloat16*>(p) + c)
                    : get(static_cast<const float*>(p) + c);
    }
  } else if (p != nullptr && col < H) {
    if (bf16) load8(static_cast<const __nv_bfloat16*>(p) + col, f);
    else load8(static_cast<const float*>(p) + col, f);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = f2(f[2 * e], f[2 * e + 1]);
}

// A thread's 16-byte pieces of one stage; piece p lies p * kRingThreads pieces
// further on (a constant, so that offsets are part of the instructions).
constexpr int kRingThreads = 512;
struct Slots {
  uint4* at;
  // 8 elements of bf16 (one piece) or fp32 (two)
  template <typename T>
  __device__ __forceinline__ void fetch8(int p, const T* src) const {
    cp_async16(smem_u32(at + p * kRingThreads), src);
    if (sizeof(T) == 4) cp_async16(smem_u32(at + (p + 1) * kRingThreads), src + 4);
  }
  __device__ __forceinline__ void fetch8_any(int p, const void* src, long off, bool bf16) const {
    if (bf16) fetch8(p, static_cast<const __nv_bfloat16*>(src) + off);
    else fetch8(p, static_cast<const float*>(src) + off);
  }
  __device__ __forceinline__ void read8(int p, bool f32, F2 (&v)[4]) const {
    const uint4 a = at[p * kRingThreads];
    if (f32) {
      const uint4 b = at[(p + 1) * kRingThreads];
      v[0] = f2(__uint_as_float(a.x), __uint_as_float(a.y));
      v[1] = f2(__uint_as_float(a.z), __uint_as_float(a.w));
      v[2] = f2(__uint_as_float(b.x), __uint_as_float(b.y));
      v[3] = f2(__uint_as_float(b.z), __uint_as_float(b.w));
    } else {
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
  }
};

// Rows of any length and stride (EDGE).  They are copied as the aligned 16 bytes
// that they touch, from the one in which the row begins (none lies before the
// tensor, whose first row is aligned), into a ring of whole rows that the block
// shares, and read from there element by element: a warp has 256 NV columns
// side by side, a lane every 32nd of them, so that loads from the ring and
// stores are runs of 32 elements whatever the alignment, in few instructions
// (aligned vectors with the columns shifted into place took three times as
// many and twice the time).  Past the row's end the ring holds zeros.
__device__ __forceinline__ uint32_t byte_in_16(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
}
// Bytes in the ring of a row of `threads` times 8 NV elements.
__host__ __device__ constexpr int edge_bytes(int threads, int nv, int size) {
  return threads * 8 * nv * size + 16;
}
template <typename T>
__device__ __forceinline__ void edge_fetch(char* to, const T* row, int H) {
  const int lead = static_cast<int>(byte_in_16(row)), bytes = H * static_cast<int>(sizeof(T));
  const char* from = reinterpret_cast<const char*>(row) - lead;
  // as many pieces for every row, so that none keeps an earlier row's end
  const int n = (16 - static_cast<int>(sizeof(T)) + bytes) / 16 + 1;
  for (int i = threadIdx.x; i < n; i += blockDim.x)
    cp_async16(smem_u32(to + 16 * i), from + 16 * i, min(max(lead + bytes - 16 * i, 0), 16));
}
// 8 of a thread's columns of the row that begins at byte `sh` of the ring's row
// at `at`.
__device__ __forceinline__ void edge_read(const char* at, bool f32, uint32_t sh, int col,
                                          F2 (&v)[4]) {
  if (f32) {
    const float* p = reinterpret_cast<const float*>(at + sh) + col;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2(p[64 * i], p[64 * i + 32]);
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(at + sh) + col;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = f2(__uint_as_float(static_cast<uint32_t>(p[64 * i]) << 16),
                __uint_as_float(static_cast<uint32_t>(p[64 * i + 32]) << 16));
  }
}
// Columns col .. of a row: 8 next to each other, or (EDGE) 32 apart.
template <bool EDGE, typename T>
__device__ __forceinline__ void put8(T* row, int col, int H, const F2 (&v)[4]) {
  if (!EDGE) {
    store8(row + col, v);
    return;
  }
  T* const to = row + col;
  if ((col & ~31) + 256 <= H) {  // the same in a warp
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 q = parts(v[i]);
      put(to + 64 * i, q.x);
      put(to + 64 * i + 32, q.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 q = parts(v[i]);
      if (col + 64 * i < H) put(to + 64 * i, q.x);
      if (col + 64 * i + 32 < H) put(to + 64 * i + 32, q.y);
    }
  }
}

// Sums over a row's warps, one barrier each: two buffers in turn, so a buffer
// is written again only after a barrier that follows its reads.  s_red:
// [2][rows][16] pairs, zero from the row's warp count on.  Two sums travel as
// a pair: in the first shuffle each half of the warp hands over the sum that
// the other half goes on with, so 5 shuffles do for both, and the warps' pairs
// are added with packed instructions.
constexpr int kRedPairs = 2 * 8 * 16;  // at most 8 rows of two to 16 warps in a block
__device__ __forceinline__ F2 ring_sums2(float a, float b, F2* s_red, int& turn) {
  const int lane = threadIdx.x & 31;
  const bool low = lane < 16;
  float v = (low ? a : b) + __shfl_xor_sync(0xffffffffu, low ? b : a, 16);
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  // lanes 0..15 hold the sum of a, the others that of b
  const int warps = blockDim.x >> 5;
  if (warps == 1) return f2(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 16));
  F2* buf = s_red + (turn * 8 + threadIdx.y) * 16;
  turn ^= 1;
  if ((lane & 15) == 0) reinterpret_cast<float*>(buf + (threadIdx.x >> 5))[lane >> 4] = v;
  __syncthreads();
  ulonglong2 t = *reinterpret_cast<const ulonglong2*>(buf);
  F2 x{t.x}, y{t.y};
  for (int w = 2; w < warps; w += 2) {
    t = *reinterpret_cast<const ulonglong2*>(buf + w);
    x = add2(x, F2{t.x});
    y = add2(y, F2{t.y});
  }
  return add2(x, y);
}
__device__ __forceinline__ float ring_sum(float a, F2* s_red, int& turn) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return a;
  float* buf = reinterpret_cast<float*>(s_red + (turn * 8 + threadIdx.y) * 16);
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = a;
  __syncthreads();
  ulonglong2 t = *reinterpret_cast<const ulonglong2*>(buf);
  F2 x{t.x}, y{t.y};
  for (int w = 4; w < warps; w += 4) {
    t = *reinterpret_cast<const ulonglong2*>(buf + w);
    x = add2(x, F2{t.x});
    y = add2(y, F2{t.y});
  }
  return sum2(add2(x, y));
}

// Threads of a row and rows of a block: NV = 1 up to 2048 columns, 2 above; rows
// side by side up to 512 threads, fewer where that would leave blocks idle.
dim3 ring_block(int T, int H, int nv, int blocks) {
  const int tx = ceil_div(H, 256 * nv) * 32;
  const int most = tx == 32 ? 16 : std::min(512 / tx, 8);
  const int ty = std::max(1, std::min(most, ceil_div(T, blocks)));
  return dim3(tx, ty);
}

template <typename K>
cudaError_t ring_ready(K kern, std::atomic<int>* ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (e != cudaSuccess) return e;
    ready[dev].store(1, std::memory_order_release);
  }
  return cudaSuccess;
}

// Bytes of one stage: pv pieces for each of the NV column sets of a thread.
constexpr size_t stage_bytes(int pv, int nv) { return static_cast<size_t>(pv) * nv * kRingThreads * 16; }

// The same for EDGE: whole rows of n32 fp32 and n16 bf16 tensors.
size_t edge_stage_bytes(int n32, int n16, int nv, dim3 block) {
  return static_cast<size_t>(block.y) *
         (static_cast<size_t>(n32) * edge_bytes(block.x, nv, 4) + n16 * edge_bytes(block.x, nv, 2));
}

}  // namespace
}  // namespace moe
