// The norms after and before a block in one pass, with the block's gate and
// residual scale, and their gradient.
//
// Forward, for one token's stream r, block output y [H]:
//   z  = y / rms(y) * w_post            (or y: no norm after the block)
//   r' = r + scale * g * z              g: per channel, per token, per element or 1
//   n  = r' / rms(r') * w_pre           rms(v) = sqrt(mean v^2 + eps)
// r' and n leave rounded once each; n is made from the unrounded r'.
//
// Backward, from dL/dr' (dr) and dL/dn (dn), with the r' that was stored:
//   q   = dn * w_pre / rms(r'),   d  = dr + q - r' mean(q r') / rms(r')^2   (dL/dr)
//   dz  = scale * g * d,          dg = scale * z * d, summed over what shares g
//   q2  = dz * w_post / rms(y),   dy = q2 - y mean(q2 y) / rms(y)^2
//   dw_pre = sum_t dn r' / rms(r'),   dw_post = sum_t dz y / rms(y)
// The norms' statistics are computed again from the rows, which have to be
// read anyway: two more sums in reductions that run in any case, against
// storing and loading them.
//
// Both are bound by memory: a row is read once into registers, every
// reduction runs over the registers, and sums are held in fp32.
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

// Forward, the rows that the streamed kernels below do not take (above 8192
// columns): a row per block, held in registers.  4778 x 12288 bf16
// with both norms and a gate per channel 142 us (3.3 TB/s), bound by the
// latency of its three dependent trips with one row per block in flight; 12289
// columns, in single elements and with 250 bytes of spills a thread, 334.
template <typename RT, bool VEC, int NV>
__global__ void __launch_bounds__(1024) block_norm_kernel(const BlockNormArgs a) {
  pdl_launch_dependents();
  __shared__ float s_red[kMaxRed];
  const Cols<VEC, NV> c{static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x), a.H};
  const int warps = blockDim.x >> 5;
  const float inv_h = 1.f / static_cast<float>(a.H);
  pdl_wait();
  const long t = blockIdx.x;
  const RT* r_in = static_cast<const RT*>(a.residual) + t * a.ld_res;
  const __nv_bfloat16* y_in =
      a.y ? static_cast<const __nv_bfloat16*>(a.y) + t * a.ld_y : nullptr;
  float r[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) c.load(r_in, v, r[v], 0.f);
  if (y_in != nullptr) {
    float y[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) c.load(y_in, v, y[v], 0.f);
    float coef = a.scale;
    if (a.gate_kind == MOE_GATE_TOKEN)
      coef *= a.gate_bf16 ? get(static_cast<const __nv_bfloat16*>(a.gate) + t)
                          : get(static_cast<const float*>(a.gate) + t);
    float rstd = 1.f;
    if (a.post_norm) {
      float sum[1] = {0.f};
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[0] += y[v][e] * y[v][e];
      row_sums<1>(sum, s_red, warps);
      rstd = rsqrtf(sum[0] * inv_h + a.eps);
    }
    coef *= rstd;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float m[8];
      if (a.post_norm && a.post_weight != nullptr) {
        c.load_any(a.post_weight, a.weight_bf16, v, m, 0.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[v][e] *= m[e];
      }
      if (a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_ELEMENT) {
        const long off = a.gate_kind == MOE_GATE_ELEMENT ? t * a.ld_gate : 0;
        const void* g = a.gate_bf16
                            ? static_cast<const void*>(static_cast<const __nv_bfloat16*>(a.gate) + off)
                            : static_cast<const void*>(static_cast<const float*>(a.gate) + off);
        c.load_any(g, a.gate_bf16, v, m, 0.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[v][e] *= m[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) r[v][e] += coef * y[v][e];
      c.store(static_cast<RT*>(a.residual_out) + t * a.H, v, r[v]);
    }
  }
  if (a.pre_norm) {
    float sum[1] = {0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[0] += r[v][e] * r[v][e];
    row_sums<1>(sum, s_red, warps);
    const float rstd = rsqrtf(sum[0] * inv_h + a.eps);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float m[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) r[v][e] *= rstd;
      if (a.pre_weight != nullptr) {
        c.load_any(a.pre_weight, a.weight_bf16, v, m, 0.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[v][e] *= m[e];
      }
      c.store(static_cast<__nv_bfloat16*>(a.normed) + t * a.H, v, r[v]);
    }
  }
}

// Backward.  One block per row at a time, blocks striding over the rows;
// each thread keeps the sums over its rows for its own columns (dw_pre,
// dw_post and a per-channel dg) and leaves them as one partial row per
// block; block_norm_partials_kernel adds those in block order, so the
// result does not depend on timing.  For rows above 8192 columns, and rows of
// 2049 columns or more whose ring of two stages would not fit: fp32 streams with
// both gradients and a gate per element, of either type.  4778 x 12288 bf16 with
// both norms and a gate per channel 537 us (1.3 TB/s): a column's sums and values
// take more registers than its threads have (1 KB of spills a thread; 4.5 KB where
// rows are not whole vectors, 1945 us at 12289 columns).  An fp32 stream with a
// gate per element 134 us at 4096 x 4096, 229 at 4096 x 7168 (2.8 TB/s).
template <typename RT, bool VEC, int NV>
__global__ void __launch_bounds__(512) block_norm_backward_kernel(const BlockNormBwdArgs a) {
  pdl_launch_dependents();
  __shared__ float s_red[kMaxRed];
  const Cols<VEC, NV> c{static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x), a.H};
  const int warps = blockDim.x >> 5;
  const float inv_h = 1.f / static_cast<float>(a.H);
  float acc_pre[NV][8] = {}, acc_post[NV][8] = {}, acc_gate[NV][8] = {};
  pdl_wait();
  for (long t = blockIdx.x; t < a.T; t += gridDim.x) {
    float d[NV][8], r[NV][8];
    if (a.grad_res != nullptr) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
        c.load(static_cast<const RT*>(a.grad_res) + t * a.ld_gres, v, d[v], 0.f);
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) d[v][e] = 0.f;
    }
    if (a.grad_normed != nullptr) {
      float q[NV][8], sum[2] = {0.f, 0.f};
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float m[8];
        c.load(static_cast<const RT*>(a.residual) + t * a.ld_res, v, r[v], 0.f);
        c.load(static_cast<const __nv_bfloat16*>(a.grad_normed) + t * a.ld_gn, v, q[v], 0.f);
        if (a.pre_weight != nullptr) c.load_any(a.pre_weight, a.weight_bf16, v, m, 0.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          sum[0] += r[v][e] * r[v][e];
          sum[1] += q[v][e] * r[v][e] * (a.pre_weight != nullptr ? m[e] : 1.f);
        }
      }
      row_sums<2>(sum, s_red, warps);
      const float rstd = rsqrtf(sum[0] * inv_h + a.eps);
      const float corr = sum[1] * inv_h * rstd * rstd * rstd;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float m[8];
        if (a.pre_weight != nullptr) c.load_any(a.pre_weight, a.weight_bf16, v, m, 0.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float qn = q[v][e] * rstd;
          acc_pre[v][e] += qn * r[v][e];
          d[v][e] += qn * (a.pre_weight != nullptr ? m[e] : 1.f) - r[v][e] * corr;
        }
      }
    }
    if (a.d_res != nullptr) {
#pragma unroll
      for (int v = 0; v < NV; ++v) c.store(static_cast<RT*>(a.d_res) + t * a.H, v, d[v]);
    }
    if (a.y == nullptr) continue;
    // dz (without the gate and scale: coef and m below), and the sums
    //   0: y^2   1: dz w_post y (the norm's projection)   2: z' d (a per-token dg)
    float y[NV][8], sum[3] = {0.f, 0.f, 0.f};
    float gt = 1.f;
    if (a.gate_kind == MOE_GATE_TOKEN)
      gt = a.gate_bf16 ? get(static_cast<const __nv_bfloat16*>(a.gate) + t)
                       : get(static_cast<const float*>(a.gate) + t);
    const long goff = a.gate_kind == MOE_GATE_ELEMENT ? t * a.ld_gate : 0;
    const void* grow = a.gate_bf16
                           ? static_cast<const void*>(static_cast<const __nv_bfloat16*>(a.gate) + goff)
                           : static_cast<const void*>(static_cast<const float*>(a.gate) + goff);
    const bool gvec = a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_ELEMENT;
    const bool pw = a.post_norm && a.post_weight != nullptr;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float m[8], w[8];
      c.load(static_cast<const __nv_bfloat16*>(a.y) + t * a.ld_y, v, y[v], 0.f);
      if (gvec) c.load_any(grow, a.gate_bf16, v, m, 0.f);
      if (pw) c.load_any(a.post_weight, a.weight_bf16, v, w, 0.f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float wd = d[v][e] * (pw ? w[e] : 1.f);
        sum[0] += y[v][e] * y[v][e];
        sum[2] += wd * y[v][e];
        sum[1] += wd * y[v][e] * (gvec ? m[e] : 1.f);
      }
    }
    float rstd = 1.f;
    if (a.post_norm || a.gate_kind == MOE_GATE_TOKEN) row_sums<3>(sum, s_red, warps);
    if (a.post_norm) rstd = rsqrtf(sum[0] * inv_h + a.eps);
    if (a.gate_kind == MOE_GATE_TOKEN && threadIdx.x == 0) {
      const float dg = a.scale * rstd * sum[2];
      if (a.gate_bf16) put(static_cast<__nv_bfloat16*>(a.d_gate) + t, dg);
      else put(static_cast<float*>(a.d_gate) + t, dg);
    }
    const float coef = a.scale * gt * rstd;  // dL/d(y * w_post) per unit of g d
    const float corr = a.post_norm ? sum[1] * inv_h * rstd * rstd * coef : 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float m[8], w[8], dgv[8];
      if (gvec) c.load_any(grow, a.gate_bf16, v, m, 0.f);
      if (pw) c.load_any(a.post_weight, a.weight_bf16, v, w, 0.f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float gd = d[v][e] * (gvec ? m[e] : 1.f) * coef;
        const float wv = pw ? w[e] : 1.f;
        dgv[e] = a.scale * rstd * y[v][e] * wv * d[v][e];
        acc_post[v][e] += gd * y[v][e];
        acc_gate[v][e] += dgv[e];
        y[v][e] = gd * wv - y[v][e] * corr;
      }
      c.store(static_cast<__nv_bfloat16*>(a.d_y) + t * a.H, v, y[v]);
      if (a.gate_kind == MOE_GATE_ELEMENT) {
        if (a.gate_bf16) c.store(static_cast<__nv_bfloat16*>(a.d_gate) + t * a.H, v, dgv);
        else c.store(static_cast<float*>(a.d_gate) + t * a.H, v, dgv);
      }
    }
  }
  float* part = a.partials + static_cast<long>(blockIdx.x) * a.n_part * a.H;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    int p = 0;
    if (a.d_pre != nullptr) c.store(part + static_cast<long>(p++) * a.H, v, acc_pre[v]);
    if (a.d_post != nullptr) c.store(part + static_cast<long>(p++) * a.H, v, acc_post[v]);
    if (a.gate_kind == MOE_GATE_CHANNEL) c.store(part + static_cast<long>(p++) * a.H, v, acc_gate[v]);
  }
}

// Sums of the blocks' partial rows: 32 columns x 8 slices of the blocks per
// thread block, each slice added in block order, then the 8 slices in order.
__global__ void __launch_bounds__(256)
    block_norm_partials_kernel(const float* __restrict__ partials, int blocks, int n_part, int H,
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

// Pairs of floats, for the packed fp32 instructions (two lanes of work in one
// issue slot: these kernels are held back by issue as much as by memory).
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ float2 parts(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ float sum2(F2 a) {
  const float2 p = parts(a);
  return p.x + p.y;
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

// Forward blocks on an SM: rows above 2048 columns fill a block by themselves, and
// one block with a deep ring and registers for its weights is faster than two
// (8192 x 7168 80 us against 86); shorter rows share one, and two are (4099 x
// 2048 22 us against 29).
constexpr int ring_blocks(int nv) { return nv == 1 ? 2 : 1; }

// MID: a call between two blocks (y given, norm before the next block, no
// gate per element), whose options are then constants of the code.
// 8192 x 7168 bf16 with both norms and a gate per channel: 80 us (470 MB, 5.9
// TB/s, 86 % of a copy), bound by memory; 4099 x 2048 with an fp32 stream 22 (101
// MB, 4.6 TB/s: a block walks over seven steps of two rows that share its barriers,
// so filling and draining the ring counts); one token 3.7, three dependent trips
// (row, two sums).  EDGE: 8192 x 7167 137 us (3.4 TB/s), bound by issue; a row per block without a
// ring 309.
template <typename RT, int NV, int STAGES, bool MID, bool EDGE>
__global__ void __launch_bounds__(kRingThreads, ring_blocks(NV))
    block_norm_ring_kernel(const BlockNormArgs a) {
  pdl_launch_dependents();
  extern __shared__ uint4 s_ring[];
  __shared__ __align__(16) F2 s_red[kRedPairs];
  constexpr bool R32 = sizeof(RT) == 4;
  constexpr int PR = R32 ? 2 : 1;                 // pieces of a residual row
  const bool has_y = MID || a.y != nullptr, pre_norm = MID || a.pre_norm;
  const bool elem = !MID && a.gate_kind == MOE_GATE_ELEMENT;
  const int nthr = blockDim.x * blockDim.y, tid = threadIdx.x + threadIdx.y * blockDim.x;
  // pieces of 8 columns: residual, y, gate
  const int pv = PR + (has_y ? 1 : 0) + (elem ? (a.gate_bf16 ? 1 : 2) : 0);
  for (int i = tid; i < kRedPairs; i += nthr) s_red[i] = f2(0.f);
  __syncthreads();
  const int H = a.H;
  const RT* const res = static_cast<const RT*>(a.residual);
  const __nv_bfloat16* const ys = static_cast<const __nv_bfloat16*>(a.y);
  // EDGE: a row's tensors one behind the other
  const int row32 = edge_bytes(blockDim.x, NV, 4), row16 = edge_bytes(blockDim.x, NV, 2);
  const int o_y = R32 ? row32 : row16, o_g = o_y + (has_y ? row16 : 0),
            row_bytes = o_g + (elem ? (a.gate_bf16 ? row16 : row32) : 0);
  // EDGE: elements past the row's end read as zeros
  auto col = [&](int v) {
    return EDGE ? static_cast<int>(threadIdx.x >> 5) * (256 * NV) + (threadIdx.x & 31) + 256 * v
                : static_cast<int>(threadIdx.x + blockDim.x * v) * 8;
  };
  auto in = [&](int v) { return EDGE || col(v) < H; };
  const float inv_h = 1.f / static_cast<float>(H);
  const long step = static_cast<long>(gridDim.x) * blockDim.y;
  auto edge_row = [&](int st) {
    return reinterpret_cast<char*>(s_ring) + (st * blockDim.y + threadIdx.y) * row_bytes;
  };
  if (EDGE) {
    for (int i = tid; i < STAGES * static_cast<int>(blockDim.y) * row_bytes / 16; i += nthr)
      s_ring[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
  auto fetch = [&](long t, int st) {
    if (EDGE && t < a.T) {
      char* const to = edge_row(st);
      edge_fetch(to, res + t * a.ld_res, H);
      if (has_y) edge_fetch(to + o_y, ys + t * a.ld_y, H);
      if (elem && a.gate_bf16)
        edge_fetch(to + o_g, static_cast<const __nv_bfloat16*>(a.gate) + t * a.ld_gate, H);
      else if (elem) edge_fetch(to + o_g, static_cast<const float*>(a.gate) + t * a.ld_gate, H);
    } else if (t < a.T) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (in(v)) {
          const Slots sl{s_ring + (st * NV + v) * pv * kRingThreads + tid};
          sl.fetch8(0, static_cast<const RT*>(a.residual) + t * a.ld_res + col(v));
          if (has_y) sl.fetch8(PR, static_cast<const __nv_bfloat16*>(a.y) + t * a.ld_y + col(v));
          if (elem) sl.fetch8_any(PR + 1, a.gate, t * a.ld_gate + col(v), a.gate_bf16);
        }
      }
    }
    cp_async_commit();
  };
  pdl_wait();
  long t = static_cast<long>(blockIdx.x) * blockDim.y + threadIdx.y;
#pragma unroll
  for (int st = 0; st < STAGES - 1; ++st) fetch(t + st * step, st);
  // weights of this thread's columns: m = post_weight * per-channel gate
  F2 m[NV][4], wp[NV][4];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    weights8<EDGE>(a.post_weight, a.weight_bf16, col(v), H, m[v]);
    if (a.gate_kind == MOE_GATE_CHANNEL) {
      weights8<EDGE>(a.gate, a.gate_bf16, col(v), H, wp[v]);
#pragma unroll
      for (int e = 0; e < 4; ++e) m[v][e] = mul2(m[v][e], wp[v][e]);
    }
    weights8<EDGE>(a.pre_weight, a.weight_bf16, col(v), H, wp[v]);
  }
  auto gate_byte = [&](long t) {
    return a.gate_bf16 ? byte_in_16(static_cast<const __nv_bfloat16*>(a.gate) + t * a.ld_gate)
                       : byte_in_16(static_cast<const float*>(a.gate) + t * a.ld_gate);
  };
  auto read_y = [&](uint4* slot, const char* erow, int v, F2 (&y)[4]) {
    if (EDGE) edge_read(erow + o_y, false, byte_in_16(ys + t * a.ld_y), col(v), y);
    else Slots{slot + v * pv * kRingThreads}.read8(PR, false, y);
  };
  int st = 0, turn = 0;
  for (long base = static_cast<long>(blockIdx.x) * blockDim.y; base < a.T; base += step, t += step) {
    if (EDGE) {  // this row's copies, everyone's, and the last row is done with
      cp_async_wait<STAGES - 2>();
      __syncthreads();
    }
    fetch(t + (STAGES - 1) * step, st == 0 ? STAGES - 1 : st - 1);
    if (!EDGE) cp_async_wait<STAGES - 1>();
    const bool on = t < a.T;
    uint4* const slot = s_ring + st * NV * pv * kRingThreads + tid;
    const char* const erow = edge_row(st);
    if (++st == STAGES) st = 0;
    F2 r[NV][4];
    float coef = a.scale;
    if (has_y) {
      if (a.gate_kind == MOE_GATE_TOKEN && on)
        coef *= a.gate_bf16 ? get(static_cast<const __nv_bfloat16*>(a.gate) + t)
                            : get(static_cast<const float*>(a.gate) + t);
      if (a.post_norm) {
        F2 sq = f2(0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          if (on && in(v)) {
            F2 y[4];
            read_y(slot, erow, v, y);
#pragma unroll
            for (int e = 0; e < 4; ++e) sq = fma2(y[e], y[e], sq);
          }
        }
        coef *= rsqrtf(ring_sum(sum2(sq), s_red, turn) * inv_h + a.eps);
      }
    }
    F2 sq = f2(0.f);
    const F2 coef2 = f2(coef);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const Slots sl{slot + v * pv * kRingThreads};
#pragma unroll
      for (int e = 0; e < 4; ++e) r[v][e] = f2(0.f);
      if (on && in(v)) {
        if (EDGE) edge_read(erow, R32, byte_in_16(res + t * a.ld_res), col(v), r[v]);
        else sl.read8(0, R32, r[v]);
        if (has_y) {
          F2 y[4];
          read_y(slot, erow, v, y);
          if (elem) {
            F2 g[4];
            if (EDGE) edge_read(erow + o_g, !a.gate_bf16, gate_byte(t), col(v), g);
            else sl.read8(PR + 1, !a.gate_bf16, g);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = mul2(y[e], g[e]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) r[v][e] = fma2(coef2, mul2(y[e], m[v][e]), r[v][e]);
          put8<EDGE>(static_cast<RT*>(a.residual_out) + t * H, col(v), H, r[v]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) sq = fma2(r[v][e], r[v][e], sq);
      }
    }
    if (pre_norm) {
      const F2 rstd = f2(rsqrtf(ring_sum(sum2(sq), s_red, turn) * inv_h + a.eps));
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (on && in(v)) {
#pragma unroll
          for (int e = 0; e < 4; ++e) r[v][e] = mul2(mul2(r[v][e], rstd), wp[v][e]);
          put8<EDGE>(static_cast<__nv_bfloat16*>(a.normed) + t * H, col(v), H, r[v]);
        }
      }
    }
  }
}

// Backward on the same ring, one block per SM.  Two sums over tokens stay in
// registers per column: acc_pre = sum dn r' / rms(r'), and acc = sum g_t d y /
// rms(y) (g_t: the per-token or per-element gate), of which a per-channel
// gate's dg = scale * w_post * acc and dw_post = scale * g * acc are
// multiples, since w_post and that gate do not depend on the token.
// MID: both gradients and y given, no gate per element.
// 8192 x 7168 bf16 with both norms and a gate per channel: 117 us and 7 for the
// partial rows' sums (705 MB, 5.7 TB/s over both, 84 % of a copy), bound by
// memory and nearly as much by issue.  EDGE: 8192 x 7167 246 us (2.9 TB/s), by
// issue; without a ring 1684.
template <typename RT, int NV, int STAGES, bool MID, bool EDGE>
__global__ void __launch_bounds__(kRingThreads, 1)
    block_norm_backward_ring_kernel(const BlockNormBwdArgs a) {
  pdl_launch_dependents();
  extern __shared__ uint4 s_ring[];
  __shared__ __align__(16) F2 s_red[kRedPairs];
  constexpr bool R32 = sizeof(RT) == 4;
  constexpr int PR = R32 ? 2 : 1;
  const bool has_y = MID || a.y != nullptr, has_gr = MID || a.grad_res != nullptr,
             has_gn = MID || a.grad_normed != nullptr;
  const bool elem = !MID && a.gate_kind == MOE_GATE_ELEMENT;
  const bool gch = a.gate_kind == MOE_GATE_CHANNEL;
  // pieces: residual, grad_residual, grad_normed, y, gate
  const int p_gr = has_gn ? PR : 0, p_gn = p_gr + (has_gr ? PR : 0), p_y = p_gn + (has_gn ? 1 : 0),
            p_g = p_y + (has_y ? 1 : 0);
  const int pv = p_g + (elem ? (a.gate_bf16 ? 1 : 2) : 0);
  const int nthr = blockDim.x * blockDim.y, tid = threadIdx.x + threadIdx.y * blockDim.x;
  for (int i = tid; i < kRedPairs; i += nthr) s_red[i] = f2(0.f);
  __syncthreads();
  const int H = a.H;
  const RT* const res = static_cast<const RT*>(a.residual);
  const RT* const grs = static_cast<const RT*>(a.grad_res);
  const __nv_bfloat16* const gns = static_cast<const __nv_bfloat16*>(a.grad_normed);
  const __nv_bfloat16* const ys = static_cast<const __nv_bfloat16*>(a.y);
  // EDGE: a row's tensors one behind the other
  const int row32 = edge_bytes(blockDim.x, NV, 4), row16 = edge_bytes(blockDim.x, NV, 2);
  const int rowR = R32 ? row32 : row16;
  const int o_gr = has_gn ? rowR : 0, o_gn = o_gr + (has_gr ? rowR : 0),
            o_y = o_gn + (has_gn ? row16 : 0), o_g = o_y + (has_y ? row16 : 0),
            row_bytes = o_g + (elem ? (a.gate_bf16 ? row16 : row32) : 0);
  // EDGE: elements past the row's end read as zeros
  auto col = [&](int v) {
    return EDGE ? static_cast<int>(threadIdx.x >> 5) * (256 * NV) + (threadIdx.x & 31) + 256 * v
                : static_cast<int>(threadIdx.x + blockDim.x * v) * 8;
  };
  auto in = [&](int v) { return EDGE || col(v) < H; };
  const float inv_h = 1.f / static_cast<float>(H);
  const long step = static_cast<long>(gridDim.x) * blockDim.y;
  auto edge_row = [&](int st) {
    return reinterpret_cast<char*>(s_ring) + (st * blockDim.y + threadIdx.y) * row_bytes;
  };
  if (EDGE) {
    for (int i = tid; i < STAGES * static_cast<int>(blockDim.y) * row_bytes / 16; i += nthr)
      s_ring[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
  auto fetch = [&](long t, int st) {
    if (EDGE && t < a.T) {
      char* const to = edge_row(st);
      if (has_gn) {
        edge_fetch(to, res + t * a.ld_res, H);
        edge_fetch(to + o_gn, gns + t * a.ld_gn, H);
      }
      if (has_gr) edge_fetch(to + o_gr, grs + t * a.ld_gres, H);
      if (has_y) edge_fetch(to + o_y, ys + t * a.ld_y, H);
      if (elem && a.gate_bf16)
        edge_fetch(to + o_g, static_cast<const __nv_bfloat16*>(a.gate) + t * a.ld_gate, H);
      else if (elem) edge_fetch(to + o_g, static_cast<const float*>(a.gate) + t * a.ld_gate, H);
    } else if (t < a.T) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (in(v)) {
          const Slots sl{s_ring + (st * NV + v) * pv * kRingThreads + tid};
          if (has_gn) {
            sl.fetch8(0, static_cast<const RT*>(a.residual) + t * a.ld_res + col(v));
            sl.fetch8(p_gn, static_cast<const __nv_bfloat16*>(a.grad_normed) + t * a.ld_gn + col(v));
          }
          if (has_gr) sl.fetch8(p_gr, static_cast<const RT*>(a.grad_res) + t * a.ld_gres + col(v));
          if (has_y) sl.fetch8(p_y, static_cast<const __nv_bfloat16*>(a.y) + t * a.ld_y + col(v));
          if (elem) sl.fetch8_any(p_g, a.gate, t * a.ld_gate + col(v), a.gate_bf16);
        }
      }
    }
    cp_async_commit();
  };
  pdl_wait();
  long t = static_cast<long>(blockIdx.x) * blockDim.y + threadIdx.y;
#pragma unroll
  for (int st = 0; st < STAGES - 1; ++st) fetch(t + st * step, st);
  const void* post_w = a.post_norm ? a.post_weight : nullptr;
  F2 m[NV][4], wp[NV][4];  // scale * post_weight * per-channel gate, pre_weight
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    weights8<EDGE>(post_w, a.weight_bf16, col(v), H, m[v]);
    weights8<EDGE>(gch ? a.gate : nullptr, a.gate_bf16, col(v), H, wp[v]);
#pragma unroll
    for (int e = 0; e < 4; ++e) m[v][e] = mul2(f2(a.scale), mul2(m[v][e], wp[v][e]));
    weights8<EDGE>(a.pre_weight, a.weight_bf16, col(v), H, wp[v]);
  }
  F2 acc_pre[NV][4], acc[NV][4];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc_pre[v][e] = acc[v][e] = f2(0.f);
  auto gate_byte = [&](long t) {
    return a.gate_bf16 ? byte_in_16(static_cast<const __nv_bfloat16*>(a.gate) + t * a.ld_gate)
                       : byte_in_16(static_cast<const float*>(a.gate) + t * a.ld_gate);
  };
  auto read_rq = [&](uint4* slot, const char* erow, int v, F2 (&r)[4], F2 (&q)[4]) {
    if (EDGE) {
      edge_read(erow, R32, byte_in_16(res + t * a.ld_res), col(v), r);
      edge_read(erow + o_gn, false, byte_in_16(gns + t * a.ld_gn), col(v), q);
    } else {
      const Slots sl{slot + v * pv * kRingThreads};
      sl.read8(0, R32, r);
      sl.read8(p_gn, false, q);
    }
  };
  auto read_y = [&](uint4* slot, const char* erow, int v, F2 (&y)[4]) {
    if (EDGE) edge_read(erow + o_y, false, byte_in_16(ys + t * a.ld_y), col(v), y);
    else Slots{slot + v * pv * kRingThreads}.read8(p_y, false, y);
  };
  auto read_g = [&](uint4* slot, const char* erow, int v, F2 (&g)[4]) {
    if (EDGE) edge_read(erow + o_g, !a.gate_bf16, gate_byte(t), col(v), g);
    else Slots{slot + v * pv * kRingThreads}.read8(p_g, !a.gate_bf16, g);
  };
  int st = 0, turn = 0;
  for (long base = static_cast<long>(blockIdx.x) * blockDim.y; base < a.T; base += step, t += step) {
    if (EDGE) {  // this row's copies, everyone's, and the last row is done with
      cp_async_wait<STAGES - 2>();
      __syncthreads();
    }
    fetch(t + (STAGES - 1) * step, st == 0 ? STAGES - 1 : st - 1);
    if (!EDGE) cp_async_wait<STAGES - 1>();
    const bool on = t < a.T;
    uint4* const slot = s_ring + st * NV * pv * kRingThreads + tid;
    const char* const erow = edge_row(st);
    if (++st == STAGES) st = 0;
    float rstd = 1.f, corr = 0.f;
    if (has_gn) {
      F2 s0 = f2(0.f), s1 = f2(0.f);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (on && in(v)) {
          const Slots sl{slot + v * pv * kRingThreads};
          F2 r[4], q[4];
          read_rq(slot, erow, v, r, q);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s0 = fma2(r[e], r[e], s0);
            s1 = fma2(mul2(q[e], wp[v][e]), r[e], s1);
          }
        }
      }
      const float2 sum = parts(ring_sums2(sum2(s0), sum2(s1), s_red, turn));
      rstd = rsqrtf(sum.x * inv_h + a.eps);
      corr = sum.y * inv_h * rstd * rstd * rstd;
    }
    F2 d[NV][4];
    F2 s0 = f2(0.f), s1 = f2(0.f);  // y^2; scale * the norm's projection, which a per-token dg needs too
    {
      const F2 rstd2 = f2(rstd), ncorr = f2(-corr);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const Slots sl{slot + v * pv * kRingThreads};
#pragma unroll
        for (int e = 0; e < 4; ++e) d[v][e] = f2(0.f);
        if (!(on && in(v))) continue;
        if (has_gr && EDGE)
          edge_read(erow + o_gr, R32, byte_in_16(grs + t * a.ld_gres), col(v), d[v]);
        else if (has_gr) sl.read8(p_gr, R32, d[v]);
        if (has_gn) {
          F2 r[4], q[4];
          read_rq(slot, erow, v, r, q);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const F2 qn = mul2(q[e], rstd2);
            acc_pre[v][e] = fma2(qn, r[e], acc_pre[v][e]);
            d[v][e] = fma2(qn, wp[v][e], fma2(r[e], ncorr, d[v][e]));
          }
        }
        if (a.d_res != nullptr) put8<EDGE>(static_cast<RT*>(a.d_res) + t * H, col(v), H, d[v]);
        if (has_y) {
          F2 y[4];
          read_y(slot, erow, v, y);
#pragma unroll
          for (int e = 0; e < 4; ++e) s0 = fma2(y[e], y[e], s0);
          if (elem) {
            F2 g[4];
            read_g(slot, erow, v, g);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = mul2(y[e], g[e]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) s1 = fma2(mul2(d[v][e], m[v][e]), y[e], s1);
        }
      }
    }
    if (!has_y) continue;
    float gt = 1.f;
    rstd = 1.f, corr = 0.f;
    if (a.gate_kind == MOE_GATE_TOKEN && on)
      gt = a.gate_bf16 ? get(static_cast<const __nv_bfloat16*>(a.gate) + t)
                       : get(static_cast<const float*>(a.gate) + t);
    if (a.post_norm || a.gate_kind == MOE_GATE_TOKEN) {
      const float2 sum = parts(ring_sums2(sum2(s0), sum2(s1), s_red, turn));
      if (a.post_norm) {
        rstd = rsqrtf(sum.x * inv_h + a.eps);
        corr = sum.y * inv_h * rstd * rstd * gt * rstd;
      }
      if (a.gate_kind == MOE_GATE_TOKEN && threadIdx.x == 0 && on) {
        const float dg = rstd * sum.y;
        if (a.gate_bf16) put(static_cast<__nv_bfloat16*>(a.d_gate) + t, dg);
        else put(static_cast<float*>(a.d_gate) + t, dg);
      }
    }
    const F2 gr = f2(gt * rstd), ncorr = f2(-corr);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const Slots sl{slot + v * pv * kRingThreads};
      if (!(on && in(v))) continue;
      F2 y[4];
      read_y(slot, erow, v, y);
      if (elem) {
        F2 g[4], dg[4];
        read_g(slot, erow, v, g);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dg[e] = mul2(mul2(gr, m[v][e]), mul2(y[e], d[v][e]));
          d[v][e] = mul2(d[v][e], g[e]);
        }
        if (a.gate_bf16) put8<EDGE>(static_cast<__nv_bfloat16*>(a.d_gate) + t * H, col(v), H, dg);
        else put8<EDGE>(static_cast<float*>(a.d_gate) + t * H, col(v), H, dg);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const F2 gd = mul2(gr, d[v][e]);
        acc[v][e] = fma2(gd, y[e], acc[v][e]);
        y[e] = fma2(m[v][e], gd, mul2(y[e], ncorr));
      }
      put8<EDGE>(static_cast<__nv_bfloat16*>(a.d_y) + t * H, col(v), H, y);
    }
  }
  if (a.n_part == 0) return;
  // the block's rows side by side added in order, through the ring's memory
  cp_async_wait<0>();
  float* sum = reinterpret_cast<float*>(s_ring);   // [threads in y][n_part][H]
  __syncthreads();
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (!in(v)) continue;
    float* to = sum + static_cast<long>(threadIdx.y) * a.n_part * H;
    F2 w[4];
    if (a.d_pre != nullptr) {
      put8<EDGE>(to, col(v), H, acc_pre[v]);
      to += H;
    }
    if (a.d_post != nullptr) {
      weights8<EDGE>(gch ? a.gate : nullptr, a.gate_bf16, col(v), H, w);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = mul2(mul2(f2(a.scale), w[e]), acc[v][e]);
      put8<EDGE>(to, col(v), H, w);
      to += H;
    }
    if (gch) {
      weights8<EDGE>(post_w, a.weight_bf16, col(v), H, w);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = mul2(mul2(f2(a.scale), w[e]), acc[v][e]);
      put8<EDGE>(to, col(v), H, w);
    }
  }
  __syncthreads();
  float* part = a.partials + static_cast<long>(blockIdx.x) * a.n_part * H;
  const int total = a.n_part * H;
  if (EDGE) {
    for (int i = tid; i < total; i += nthr) {
      float v = sum[i];
      for (int y = 1; y < blockDim.y; ++y) v += sum[y * total + i];
      part[i] = v;
    }
  } else {
    for (int i = tid * 4; i < total; i += nthr * 4) {  // H % 8 == 0
      float4 v = *reinterpret_cast<const float4*>(sum + i);
      for (int y = 1; y < blockDim.y; ++y) {
        const float4 o = *reinterpret_cast<const float4*>(sum + static_cast<long>(y) * total + i);
        v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
      }
      *reinterpret_cast<float4*>(part + i) = v;
    }
  }
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

template <typename RT, int NV, int STAGES, bool MID, bool EDGE = false>
cudaError_t fwd_ring(const BlockNormArgs& a, dim3 block, size_t smem, int grid, cudaStream_t s) {
  static std::atomic<int> ready[64] = {};
  const cudaError_t e = ring_ready(block_norm_ring_kernel<RT, NV, STAGES, MID, EDGE>, ready);
  if (e != cudaSuccess) return e;
  return launch_pdl(block_norm_ring_kernel<RT, NV, STAGES, MID, EDGE>, dim3(grid), block, smem, s,
                    a);
}
template <typename RT, int NV, int STAGES, bool MID, bool EDGE = false>
cudaError_t bwd_ring(const BlockNormBwdArgs& a, dim3 block, size_t smem, int grid, cudaStream_t s) {
  static std::atomic<int> ready[64] = {};
  const cudaError_t e = ring_ready(block_norm_backward_ring_kernel<RT, NV, STAGES, MID, EDGE>, ready);
  if (e != cudaSuccess) return e;
  return launch_pdl(block_norm_backward_ring_kernel<RT, NV, STAGES, MID, EDGE>, dim3(grid), block,
                    smem, s, a);
}

// Bytes of one stage: pv pieces for each of the NV column sets of a thread.
constexpr size_t stage_bytes(int pv, int nv) { return static_cast<size_t>(pv) * nv * kRingThreads * 16; }

// The same for EDGE: whole rows of n32 fp32 and n16 bf16 tensors.
size_t edge_stage_bytes(int n32, int n16, int nv, dim3 block) {
  return static_cast<size_t>(block.y) *
         (static_cast<size_t>(n32) * edge_bytes(block.x, nv, 4) + n16 * edge_bytes(block.x, nv, 2));
}

template <typename RT, int NV, bool VEC>
cudaError_t fwd_nv(const BlockNormArgs& a, int num_sms, cudaStream_t s) {
  constexpr int PER_SM = ring_blocks(NV), PR = static_cast<int>(sizeof(RT) / 2);
  const dim3 block = ring_block(a.T, a.H, NV, PER_SM * num_sms);
  const bool elem = a.gate_kind == MOE_GATE_ELEMENT;
  const int grid = std::min(PER_SM * num_sms, ceil_div(a.T, block.y));
  if (!VEC) {
    const int g32 = elem && !a.gate_bf16, g16 = elem && a.gate_bf16, y16 = a.y != nullptr;
    const size_t stage = edge_stage_bytes((PR == 2) + g32, (PR == 1) + y16 + g16, NV, block);
    return 4 * stage * PER_SM <= kRingBytes
               ? fwd_ring<RT, NV, 4, false, true>(a, block, 4 * stage, grid, s)
               : fwd_ring<RT, NV, 2, false, true>(a, block, 2 * stage, grid, s);
  }
  if (a.y != nullptr && a.pre_norm && !elem) {
    // 160 of 200 KB for bf16 rows; one stage more was slower at each width
    // (81.7 against 80.2 us at 8192 x 7168, 23.2 against 22.0 at 4099 x 2048)
    constexpr int ST = NV == 1 ? 3 : PR == 1 ? 5 : 4;
    static_assert(ST * stage_bytes(PR + 1, NV) * PER_SM <= kRingBytes, "a ring");
    return fwd_ring<RT, NV, ST, true>(a, block, ST * stage_bytes(PR + 1, NV), grid, s);
  }
  const size_t stage = stage_bytes(PR + (a.y != nullptr) + (elem ? (a.gate_bf16 ? 1 : 2) : 0), NV);
  return fwd_ring<RT, NV, 2, false>(a, block, 2 * stage, grid, s);
}
size_t bwd_edge_stage(const BlockNormBwdArgs& a, bool r32, int nv, dim3 block) {
  const bool elem = a.gate_kind == MOE_GATE_ELEMENT;
  const int r = (a.grad_normed != nullptr) + (a.grad_res != nullptr);
  return edge_stage_bytes((r32 ? r : 0) + (elem && !a.gate_bf16),
                          (r32 ? 0 : r) + (a.grad_normed != nullptr) + (a.y != nullptr) +
                              (elem && a.gate_bf16),
                          nv, block);
}
template <typename RT, int NV, bool VEC>
cudaError_t bwd_nv(const BlockNormBwdArgs& a, int num_sms, int pv, int* blocks, cudaStream_t s) {
  const dim3 block = ring_block(a.T, a.H, NV, num_sms);
  const size_t stage = VEC ? stage_bytes(pv, NV) : bwd_edge_stage(a, sizeof(RT) == 4, NV, block);
  const size_t sums = static_cast<size_t>(block.y) * a.n_part * a.H * 4;  // <= 96 KB
  const int grid = *blocks = std::min(std::min(num_sms, kNormBwdBlocks), ceil_div(a.T, block.y));
  if (!VEC)
    return 3 * stage <= kRingBytes
               ? bwd_ring<RT, NV, 3, false, true>(a, block, std::max(3 * stage, sums), grid, s)
               : bwd_ring<RT, NV, 2, false, true>(a, block, std::max(2 * stage, sums), grid, s);
  if (a.grad_res != nullptr && a.grad_normed != nullptr && a.y != nullptr &&
      a.gate_kind != MOE_GATE_ELEMENT)
    return 3 * stage <= kRingBytes
               ? bwd_ring<RT, NV, 3, true>(a, block, std::max(3 * stage, sums), grid, s)
               : bwd_ring<RT, NV, 2, true>(a, block, std::max(2 * stage, sums), grid, s);
  return bwd_ring<RT, NV, 2, false>(a, block, std::max(2 * stage, sums), grid, s);
}

template <typename RT, bool VEC>
cudaError_t fwd(const BlockNormArgs& a, int num_sms, cudaStream_t s) {
  if (a.H <= 8192)
    return a.H <= 2048 ? fwd_nv<RT, 1, VEC>(a, num_sms, s) : fwd_nv<RT, 2, VEC>(a, num_sms, s);
  // two pieces of 8 columns per thread
  const dim3 block(ceil_div(ceil_div(a.H, 8), 64) * 32);
  return launch_pdl(block_norm_kernel<RT, VEC, 2>, dim3(a.T), block, 0, s, a);
}

template <typename RT, bool VEC>
cudaError_t bwd(const BlockNormBwdArgs& a, int num_sms, int* blocks_used, cudaStream_t s) {
  if (a.H <= 8192) {
    const int pr = static_cast<int>(sizeof(RT) / 2);
    const int pv = (a.grad_normed ? pr + 1 : 0) + (a.grad_res ? pr : 0) + (a.y != nullptr) +
                   (a.gate_kind == MOE_GATE_ELEMENT ? (a.gate_bf16 ? 1 : 2) : 0);
    // two stages fit: every case up to 2048 columns; above, all but fp32 streams with both
    // gradients and a gate per element: 7 or 8 pieces, 224 or 256 KB, as a stage is laid out
    // for 512 threads whatever the block has.  Rows that are not whole vectors take what
    // they need, and of the same calls only those of 2049 to 2560, 3585 to 4096 and 7169 to
    // 8192 columns (fp32 gates: from 3073 and from 6145) do not fit.
    const int nv = a.H <= 2048 ? 1 : 2;
    const size_t stage =
        VEC ? stage_bytes(pv, nv)
            : bwd_edge_stage(a, pr == 2, nv, ring_block(a.T, a.H, nv, num_sms));
    if (2 * stage <= kRingBytes)
      return nv == 1 ? bwd_nv<RT, 1, VEC>(a, num_sms, pv, blocks_used, s)
                     : bwd_nv<RT, 2, VEC>(a, num_sms, pv, blocks_used, s);
  }
  const int blocks = *blocks_used =
      static_cast<int>(std::min<long>(std::min(2 * num_sms, kNormBwdBlocks), a.T));
  const int pieces = ceil_div(a.H, 8);
  const int nv = pieces <= 512 ? 1 : pieces <= 1024 ? 2 : 4;
  const dim3 block(ceil_div(ceil_div(pieces, nv), 32) * 32);
  if (nv == 1) return launch_pdl(block_norm_backward_kernel<RT, VEC, 1>, dim3(blocks), block, 0, s, a);
  if (nv == 2) return launch_pdl(block_norm_backward_kernel<RT, VEC, 2>, dim3(blocks), block, 0, s, a);
  return launch_pdl(block_norm_backward_kernel<RT, VEC, 4>, dim3(blocks), block, 0, s, a);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& a, bool res_bf16, bool vec, int num_sms,
                              cudaStream_t s) {
  cudaError_t e;
  if (res_bf16)
    e = vec ? fwd<__nv_bfloat16, true>(a, num_sms, s) : fwd<__nv_bfloat16, false>(a, num_sms, s);
  else
    e = vec ? fwd<float, true>(a, num_sms, s) : fwd<float, false>(a, num_sms, s);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_block_norm_backward(const BlockNormBwdArgs& a, bool res_bf16, bool vec,
                                       int num_sms, cudaStream_t s) {
  cudaError_t e;
  int blocks = 0;
  if (res_bf16)
    e = vec ? bwd<__nv_bfloat16, true>(a, num_sms, &blocks, s)
            : bwd<__nv_bfloat16, false>(a, num_sms, &blocks, s);
  else
    e = vec ? bwd<float, true>(a, num_sms, &blocks, s) : bwd<float, false>(a, num_sms, &blocks, s);
  count_launches(1);
  if (e != cudaSuccess) return e;
  if (a.n_part > 0) {
    float* o[3] = {nullptr, nullptr, nullptr};
    int p = 0;
    if (a.d_pre != nullptr) o[p++] = a.d_pre;
    if (a.d_post != nullptr) o[p++] = a.d_post;
    if (a.gate_kind == MOE_GATE_CHANNEL) o[p++] = static_cast<float*>(a.d_gate);
    e = launch_pdl(block_norm_partials_kernel, dim3(ceil_div(a.H, 32), a.n_part), dim3(256), 0, s,
                   static_cast<const float*>(a.partials), blocks, a.n_part, a.H, o[0], o[1], o[2]);
    count_launches(1);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
