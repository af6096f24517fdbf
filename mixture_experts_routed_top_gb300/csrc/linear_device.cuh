// Device code that the dense products share (linear.cu, linear_fp8.cu): operand
// descriptors, bounded waits, 8-wide loads and stores, activations, the
// epilogues and the joining of a split contraction.
#pragma once

#include <algorithm>
#include <type_traits>

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int BK = 64;  // bf16 elements per 128-byte swizzled row

// Shared-memory descriptor of an MN-major tile with 128-byte swizzling: 64
// rows (of M or N) contiguous in a 128-byte line, lines along the
// contraction, 8 lines (1024 bytes) per swizzle atom; the next 64 rows
// `slab_bytes` away.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t slab_bytes) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);    // start address / 16
  d |= static_cast<uint64_t>(slab_bytes >> 4) << 16;      // leading byte offset: next 64 rows
  d |= static_cast<uint64_t>(1024 >> 4) << 32;            // stride byte offset: next 8 lines
  d |= static_cast<uint64_t>(1) << 46;                    // descriptor version (sm_100 family)
  d |= static_cast<uint64_t>(2) << 61;                    // swizzle mode: 128 B
  return d;
}

// Instruction descriptor of idesc_bf16_f32 with the operands' orders.
__host__ __device__ constexpr uint32_t idesc_bf16_order(int M, int N, bool a_mn, bool b_mn) {
  return idesc_bf16_f32(M, N) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
}

// Bounded waits as mbar_wait_bounded, on the SM's cycle counter: reading the
// global timer takes longer than most of these waits.  2e9 cycles are a second
// at the card's 2 GHz; each try itself blocks for a while.
constexpr long long kWaitCycles = 2000000000ll, kDrainCycles = 40000000ll;
enum class WaitScope { kCta, kPair, kPairRelaxed };
template <WaitScope S>
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  return S == WaitScope::kCta    ? mbar_try_wait(bar, parity)
         : S == WaitScope::kPair ? mbar_try_wait_cluster(bar, parity)
                                 : mbar_try_wait_cluster_relaxed(bar, parity);
}
template <WaitScope S>
__device__ __forceinline__ bool wait_cycles(uint32_t bar, uint32_t parity, volatile int* abort,
                                            int* err, int code, long long limit) {
  long long t0 = 0;
  for (int i = 0;; ++i) {
    if (try_wait<S>(bar, parity)) return true;
    if ((i & 15) == 15) {
      if (*abort) return false;
      const long long now = clock64();
      if (i == 15) t0 = now;
      else if (now - t0 > limit) {
        atomicOr(err, code);
        *abort = 1;
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait_pair(uint32_t bar, uint32_t parity, volatile int* abort,
                                          int* err, int code, long long limit = kWaitCycles) {
  return wait_cycles<WaitScope::kPair>(bar, parity, abort, err, code, limit);
}
// Where nothing but reads and writes of TMEM is ordered, or with fence_acquire_shared_cluster.
__device__ __forceinline__ bool wait_pair_relaxed(uint32_t bar, uint32_t parity, volatile int* abort,
                                                  int* err, int code, long long limit = kWaitCycles) {
  return wait_cycles<WaitScope::kPairRelaxed>(bar, parity, abort, err, code, limit);
}
__device__ __forceinline__ bool wait_cta(uint32_t bar, uint32_t parity, volatile int* abort,
                                         int* err, int code, long long limit = kWaitCycles) {
  return wait_cycles<WaitScope::kCta>(bar, parity, abort, err, code, limit);
}

// 2-D load counted on an mbarrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(const CUtensorMap* map, uint32_t bar,
                                                 uint32_t dst, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

__device__ __forceinline__ float ldf(const void* p, long i, bool bf16) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
              : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void stf(void* p, long i, bool f32, float v) {
  if (f32) static_cast<float*>(p)[i] = v;
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}
__device__ __forceinline__ void ld8(const void* p, long i, bool bf16, float (&v)[8]) {
  if (bf16) {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = q[0], b = q[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}
__device__ __forceinline__ void st8(void* p, long i, bool f32, const float (&v)[8]) {
  if (f32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint4 u;
    u.x = pack_bf16x2(v[0], v[1]);
    u.y = pack_bf16x2(v[2], v[3]);
    u.z = pack_bf16x2(v[4], v[5]);
    u.w = pack_bf16x2(v[6], v[7]);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) = u;
  }
}

// The activation in fp32; silu_f's fast division only where the result is
// rounded to bf16.
__device__ __forceinline__ float act_f(float z, int act, bool f32) {
  if (act == MOE_ACT_NONE) return z;
  if (act == MOE_ACT_SILU && f32) return z / (1.f + expf(-z));
  return gate_act(z, act);
}
// 8 elements from 16 bytes of bf16 or 32 of fp32.
template <bool F32>
__device__ __forceinline__ void bits8(const uint4 (&x)[F32 ? 2 : 1], float (&v)[8]) {
  const uint4 a = x[0], b = x[F32 ? 1 : 0];
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = __uint_as_float(F32 ? w[j] : j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
}
// A result and the residual.  REST (the gradients' products): the residual is the
// product of what rounding an operand left, and it joins only finite results.  Times
// an infinity that rest, 0 or of either sign, would make the infinite result a NaN.
template <bool REST>
__device__ __forceinline__ float plus(float v, float r) {
  return REST && !(fabsf(v) < INFINITY) ? v : v + r;
}
// The epilogue on 8 consecutive columns n.. of row m (m < M) where N % 8 == 0 and
// every row is 16-byte aligned: pre-activation z = v + bias, y = residual +
// act(z).  ACT and F32 are constants of the code: kernels hold several copies of
// this, and with every activation and type in each the code was so long that
// fetching it took longer than a small product (33 us for 64 x 256 x 256),
// while one copy called as a function took 300 ns a call.
// b: the bias there; x: the residual's bits.
template <int ACT, bool F32, bool REST>
__device__ __forceinline__ void epilogue8(const LinearEpi& p, long m, int n, const float (&b)[8],
                                          const uint4 (&x)[F32 ? 2 : 1], float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] += b[j];
  if (p.preact != nullptr) st8(p.preact, m * p.ld_out + n, F32, v);
  if (ACT != MOE_ACT_NONE) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = act_f(v[j], ACT, F32);
  }
  if (p.residual != nullptr) {
    float r[8];
    bits8<F32>(x, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = plus<REST>(v[j], r[j]);
  }
  st8(p.out, m * p.ld_out + n, F32, v);
}
// 32 consecutive columns of 32 rows from a warp's TMEM load (lane: row m).  The
// values go through `buf` (32 x 32 floats of this warp, 16-byte pieces of a row
// in the order of their index xor the row's, so that neither side meets a bank
// twice), after which lanes hold neighbouring columns: 4 lanes of 8 columns a
// row, or where rows are not whole aligned vectors (p.vec off) 32 of one.
// Straight from the lanes every access touched 32 rows, and the epilogue of a
// 256 x 256 tile took 6 us, as long as 1152 of the contraction.
constexpr int kTurn = 32 * 32;
template <int ACT, bool F32, bool REST>
__device__ __forceinline__ void epilogue32(const LinearEpi& p, long m, int n,
                                           const uint32_t (&v)[32], float* buf,
                                           const int lane = threadIdx.x & 31) {
  const long m0 = m - lane;
  // bias and residual of 8 columns of 4 rows, every load on its way before the
  // first store, which the compiler may not move loads across
  const int nv = n + 8 * (lane & 3);
  float bv[8] = {};
  uint4 xv[4][F32 ? 2 : 1] = {};
  if (p.vec && nv < p.N) {
    if (p.residual != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const long row = m0 + 8 * i + (lane >> 2);
        if (row < p.M) {
          const uint4* q = reinterpret_cast<const uint4*>(
              static_cast<const char*>(p.residual) + (row * p.ld_res + nv) * (F32 ? 4 : 2));
          xv[i][0] = q[0];
          if (F32) xv[i][F32 ? 1 : 0] = q[1];
        }
      }
    }
    if (p.bias != nullptr) ld8(p.bias, nv, p.bias_bf16, bv);
  }
  __syncwarp();  // the previous step's values have been read
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<uint4*>(buf + lane * 32 + 4 * (c ^ (lane & 7))) =
        make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
  __syncwarp();
  if (p.vec) {
    const int c = 2 * (lane & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 8 * i + (lane >> 2);
      const float4 x = *reinterpret_cast<const float4*>(buf + row * 32 + 4 * (c ^ (row & 7)));
      const float4 y = *reinterpret_cast<const float4*>(buf + row * 32 + 4 * ((c + 1) ^ (row & 7)));
      float f[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
      if (m0 + row < p.M && nv < p.N) epilogue8<ACT, F32, REST>(p, m0 + row, nv, bv, xv[i], f);
    }
  } else if (n + lane < p.N) {
    const int rows = static_cast<int>(min(32l, p.M - m0)), col = n + lane;
    const float b = p.bias != nullptr ? ldf(p.bias, col, p.bias_bf16) : 0.f;
    using U = std::conditional_t<F32, uint32_t, uint16_t>;  // the residual's bits
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 8) {
      U x[8] = {};
      if (p.residual != nullptr) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (r0 + k < rows) x[k] = static_cast<const U*>(p.residual)[(m0 + r0 + k) * p.ld_res + col];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = r0 + k;
        if (r >= rows) break;
        const float z = buf[r * 32 + 4 * ((lane >> 2) ^ k) + (lane & 3)] + b;
        const float res = __uint_as_float(static_cast<uint32_t>(x[k]) << (F32 ? 0 : 16));
        if (p.preact != nullptr) stf(p.preact, (m0 + r) * p.ld_out + col, F32, z);
        stf(p.out, (m0 + r) * p.ld_out + col, F32, __fadd_rn(act_f(z, ACT, F32), res));
      }
    }
  }
  __syncwarp();
}

// Joining a split contraction.  The CTAs of a cluster share a tile and each owns
// some of its rows.  A CTA has its sums in its shared memory ([128][STRIDE]
// floats); it writes the other owners' rows to its part of the workspace
// ([CTA][128][8 * CHUNKS] floats, whole lines, into L2), and after a cluster
// barrier each owner adds its rows over all CTAs in their order (so the
// result does not depend on timing), its own from shared memory, and runs the
// epilogue on them: 8 columns of a row per thread, neighbouring threads along
// the row, the loads of two rows from up to four CTAs in flight together.
// Through distributed shared memory instead, reading or writing, the same
// exchange ran at 17 to 30 GB/s per SM and took 5 us of a router product of
// 8192 tokens and 10 of a 256 x 2048 x 2048 one.
template <int THREADS, int CHUNKS, int STRIDE>
__device__ __forceinline__ void hand_over(const float* stg, float* part, int row0, int rows) {
  constexpr int C4 = 2 * CHUNKS;  // float4s of a row
  for (int i = threadIdx.x; i < (128 - rows) * C4; i += THREADS) {
    int row = i / C4;
    row += row >= row0 ? rows : 0;  // the rows before and after the CTA's own
    const int c = (i % C4) * 4;
    __stcg(reinterpret_cast<float4*>(part + row * (4 * C4) + c),
           *reinterpret_cast<const float4*>(stg + row * STRIDE + c));
  }
}
// v[row][8] += parts k0 .. k0 + PARTS - 1 of the first R of a thread's 4 rows,
// `count` of which there are.  own: its columns of the rows in shared memory,
// other: in the first CTA's part of the workspace, the next one's `step`
// floats further on; `mine` is the part in shared memory.
template <int R, int PARTS>
__device__ __forceinline__ void add_parts(const float* own, int own_step, const float* other,
                                          int other_step, long step, int k0, int mine, int count,
                                          float (&v)[4][8]) {
  float4 x[PARTS][R][2];
#pragma unroll
  for (int i = 0; i < PARTS; ++i)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      x[i][r][0] = x[i][r][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r >= count) continue;
      if (k0 + i == mine) {
        const float4* q = reinterpret_cast<const float4*>(own + r * own_step);
        x[i][r][0] = q[0];
        x[i][r][1] = q[1];
      } else {
        const float4* q = reinterpret_cast<const float4*>(other + step * (k0 + i) + r * other_step);
        x[i][r][0] = __ldcg(q);
        x[i][r][1] = __ldcg(q + 1);
      }
    }
#pragma unroll
  for (int i = 0; i < PARTS; ++i)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      v[r][0] += x[i][r][0].x, v[r][1] += x[i][r][0].y, v[r][2] += x[i][r][0].z;
      v[r][3] += x[i][r][0].w, v[r][4] += x[i][r][1].x, v[r][5] += x[i][r][1].y;
      v[r][6] += x[i][r][1].z, v[r][7] += x[i][r][1].w;
    }
}
// RB rows of a warp, a lane every 32nd column: sums `from` (this lane's, rows
// `stride` apart; -1: no row), bias b.  The type and whether there is an
// activation are constants: tested per element they took most of its time.
template <bool F32, bool ACT, int RB>
__device__ __forceinline__ void single_rows(const LinearEpi& p, const float* from, int stride,
                                            const int (&row)[RB], long m0, int n0,
                                            const float (&b)[8]) {
  constexpr int COLS = 8 / RB;
  using T = std::conditional_t<F32, float, __nv_bfloat16>;
  const int n = n0 + (threadIdx.x & 31);
  // the residual's bits, every load on its way before the first is used (with the
  // conversion beside the load each waited for its own, 7 us at 391 x 224 x 706)
  using U = std::conditional_t<F32, uint32_t, uint16_t>;
  U y[RB][COLS];
#pragma unroll
  for (int k = 0; k < RB; ++k)
#pragma unroll
    for (int j = 0; j < COLS; ++j) y[k][j] = 0;
  if (p.residual != nullptr) {
#pragma unroll
    for (int k = 0; k < RB; ++k)
#pragma unroll
      for (int j = 0; j < COLS; ++j)
        if (row[k] >= 0 && n + 32 * j < p.N)
          y[k][j] = static_cast<const U*>(p.residual)[(m0 + row[k]) * p.ld_res + n + 32 * j];
  }
#pragma unroll
  for (int k = 0; k < RB; ++k) {
    if (row[k] < 0) continue;
    const float* const v = from + row[k] * stride;
    const long at = (m0 + row[k]) * p.ld_out + n;
#pragma unroll
    for (int j = 0; j < COLS; ++j) {
      if (n + 32 * j >= p.N) continue;
      const float z = v[32 * j] + b[j];
      if (p.preact != nullptr) stf(static_cast<T*>(p.preact) + at, 32 * j, F32, z);
      // not fused into the activation, which would depend on the other options
      const float res = __uint_as_float(static_cast<uint32_t>(y[k][j]) << (F32 ? 0 : 16));
      stf(static_cast<T*>(p.out) + at, 32 * j, F32, __fadd_rn(res, ACT ? act_f(z, p.act, F32) : z));
    }
  }
}

// The rows row0 .. row0 + rows of a tile whose first row is m0, columns n0 ..
// n0 + 8 * CHUNKS.  parts: number of CTAs (1, 2, 4 or 8), mine: this one's place
// among them; part0: the first one's part of the workspace, the next ones'
// `step` floats further on.  Rows that are not whole aligned vectors go back into
// stg and leave it with a warp's lanes along a row (391 x 224 x 706 from the
// threads' 8 columns 22.5 us, so 12.1; x 704 9.2).
template <int THREADS, int CHUNKS, int STRIDE, bool REST>
__device__ __forceinline__ void join_rows(const LinearEpi& p, float* stg, const float* part0,
                                          long step, int parts, int mine, int row0, int rows,
                                          long m0, int n0) {
  static_assert(THREADS % CHUNKS == 0 && 32 % CHUNKS == 0, "a thread keeps its columns");
  constexpr int STEP = THREADS / CHUNKS, WROWS = 32 / CHUNKS, WCOLS = CHUNKS / 4;
  constexpr int RB = 8 / WCOLS;
  const int lane = threadIdx.x & 31;
  const int col = (threadIdx.x % CHUNKS) * 8, n = n0 + col;
  if (p.vec && n >= p.N) return;
  float b[8];  // of the thread's columns; without vectors of lane, lane + 32, ..
#pragma unroll
  for (int j = 0; j < 8; ++j) b[j] = 0.f;
  if (p.bias != nullptr) {
    if (p.vec) {
      ld8(p.bias, n, p.bias_bf16, b);
    } else {
#pragma unroll
      for (int j = 0; j < WCOLS; ++j)
        if (n0 + lane + 32 * j < p.N) b[j] = ldf(p.bias, n0 + lane + 32 * j, p.bias_bf16);
    }
  }
  // rows in flight: 4 of up to two parts, 2 of four (twice as many measured slower)
  const int R = parts <= 2 ? 4 : 2;
  const int end = static_cast<int>(min(static_cast<long>(rows), p.M - m0 - row0));
#pragma unroll 1
  for (int iw = threadIdx.x / 32 * WROWS; iw < end; iw += R * STEP) {  // the warp's first row
    const int i = iw + lane / CHUNKS;
    const int count = max(0, min(R, (end - i + STEP - 1) / STEP)), ra = row0 + i;
    float* const own = stg + ra * STRIDE + col;
    const float* const other = part0 + ra * (8 * CHUNKS) + col;
    constexpr int OS = STEP * STRIDE, PS = STEP * 8 * CHUNKS;
    float v[4][8];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[r][j] = 0.f;
    if (parts == 1) add_parts<4, 1>(own, OS, other, PS, step, 0, mine, count, v);
    else if (parts == 2) add_parts<4, 2>(own, OS, other, PS, step, 0, mine, count, v);
    else
      for (int k = 0; k < parts; k += 4)
        add_parts<2, 4>(own, OS, other, PS, step, k, mine, count, v);
    if (!p.vec) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (r >= count) continue;
        float4* q = reinterpret_cast<float4*>(own + r * OS);
        q[0] = make_float4(v[r][0], v[r][1], v[r][2], v[r][3]);
        q[1] = make_float4(v[r][4], v[r][5], v[r][6], v[r][7]);
      }
      __syncwarp();
      for (int r = 0; r < R * WROWS; r += RB) {
        int rows_at[RB];
#pragma unroll
        for (int k = 0; k < RB; ++k) {
          const int row = iw + (r + k) / WROWS * STEP + (r + k) % WROWS;
          rows_at[k] = row < end ? row0 + row : -1;
        }
        const float* from = stg + lane;
        if (p.out_f32) {
          if (p.act == MOE_ACT_NONE) single_rows<true, false>(p, from, STRIDE, rows_at, m0, n0, b);
          else single_rows<true, true>(p, from, STRIDE, rows_at, m0, n0, b);
        } else {
          if (p.act == MOE_ACT_NONE) single_rows<false, false>(p, from, STRIDE, rows_at, m0, n0, b);
          else single_rows<false, true>(p, from, STRIDE, rows_at, m0, n0, b);
        }
      }
      continue;
    }
#pragma unroll 1
    for (int r = 0; r < count; ++r) {
      const long m = m0 + ra + r * STEP;
      float z[8], y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        z[j] = (r == 0 ? v[0][j] : r == 1 ? v[1][j] : r == 2 ? v[2][j] : v[3][j]) + b[j];
        y[j] = 0.f;
      }
      if (p.residual != nullptr) ld8(p.residual, m * p.ld_res + n, !p.out_f32, y);
      if (p.preact != nullptr) st8(p.preact, m * p.ld_out + n, p.out_f32, z);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = plus<REST>(act_f(z[j], p.act, p.out_f32), y[j]);
      st8(p.out, m * p.ld_out + n, p.out_f32, y);
    }
  }
}

// ------------------------------------------------------ gated products
// Weights [2 N, K], gate rows first: a tile of N' output columns has their N' gate
// columns and then their N' up columns, and its epilogue makes
//   zg = g + bias[n],  zu = u + bias[N + n],  out = act(zg) zu
// of them.  p.preact, rows 2 N apart, takes zg and zu rounded once each.
template <int ACT>
__device__ __forceinline__ float gated_f(float zg, float zu, int act) {
  return gate_act(zg, ACT == MOE_ACT_NONE ? act : ACT) * zu;
}
// 8 consecutive columns n.. of row m, every row of whole aligned vectors.
// ACT: a constant activation, or MOE_ACT_NONE: the arguments'.
template <int ACT>
__device__ __forceinline__ void gated8(const LinearEpi& p, long m, int n, const float (&bg)[8],
                                       const float (&bu)[8], float (&zg)[8], float (&zu)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) zg[j] += bg[j], zu[j] += bu[j];
  if (p.preact != nullptr) {
    st8(p.preact, m * (2l * p.N) + n, false, zg);
    st8(p.preact, m * (2l * p.N) + p.N + n, false, zu);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) zg[j] = gated_f<ACT>(zg[j], zu[j], p.act);
  st8(p.out, m * p.ld_out + n, false, zg);
}
// One column n < N of row m.
template <int ACT>
__device__ __forceinline__ void gated1(const LinearEpi& p, long m, int n, float zg, float zu) {
  if (p.preact != nullptr) {
    stf(p.preact, m * (2l * p.N) + n, false, zg);
    stf(p.preact, m * (2l * p.N) + p.N + n, false, zu);
  }
  stf(p.out, m * p.ld_out + n, false, gated_f<ACT>(zg, zu, p.act));
}
// As epilogue32, of 32 gate and the 32 up columns of the outputs n .. n + 31: both go
// through the turn buffer one after the other, as many passes a tile as without a gate.
template <int ACT>
__device__ __forceinline__ void epilogue32_gated(const LinearEpi& p, long m, int n,
                                                 const uint32_t (&g)[32], const uint32_t (&u)[32],
                                                 float* buf) {
  const int lane = threadIdx.x & 31;
  const long m0 = m - lane;
  auto turn = [&](const uint32_t (&v)[32]) {
    __syncwarp();  // the previous values have been read
#pragma unroll
    for (int c = 0; c < 8; ++c)
      *reinterpret_cast<uint4*>(buf + lane * 32 + 4 * (c ^ (lane & 7))) =
          make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    __syncwarp();
  };
  if (p.vec) {
    const int nv = n + 8 * (lane & 3), c = 2 * (lane & 3);
    float bg[8] = {}, bu[8] = {};
    if (p.bias != nullptr && nv < p.N) {
      ld8(p.bias, nv, p.bias_bf16, bg);
      ld8(p.bias, p.N + nv, p.bias_bf16, bu);
    }
    auto take = [&](int row, float (&f)[8]) {
      const float4 x = *reinterpret_cast<const float4*>(buf + row * 32 + 4 * (c ^ (row & 7)));
      const float4 y = *reinterpret_cast<const float4*>(buf + row * 32 + 4 * ((c + 1) ^ (row & 7)));
      f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w;
      f[4] = y.x, f[5] = y.y, f[6] = y.z, f[7] = y.w;
    };
    float zg[4][8];
    turn(g);
#pragma unroll
    for (int i = 0; i < 4; ++i) take(8 * i + (lane >> 2), zg[i]);
    turn(u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 8 * i + (lane >> 2);
      float zu[8];
      take(row, zu);
      if (m0 + row < p.M && nv < p.N) gated8<ACT>(p, m0 + row, nv, bg, bu, zg[i], zu);
    }
  } else {  // rows that are not whole aligned vectors: a lane a column
    const int col = n + lane, rows = static_cast<int>(min(32l, p.M - m0));
    const bool on = col < p.N;
    const float bg = on && p.bias != nullptr ? ldf(p.bias, col, p.bias_bf16) : 0.f;
    const float bu = on && p.bias != nullptr ? ldf(p.bias, p.N + col, p.bias_bf16) : 0.f;
    float zg[32];
    turn(g);
#pragma unroll
    for (int r = 0; r < 32; ++r) zg[r] = buf[r * 32 + 4 * ((lane >> 2) ^ (r & 7)) + (lane & 3)] + bg;
    turn(u);
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      const float zu = buf[r * 32 + 4 * ((lane >> 2) ^ (r & 7)) + (lane & 3)] + bu;
      if (on && r < rows) gated1<ACT>(p, m0 + r, col, zg[r], zu);
    }
  }
}
// As join_rows, of a tile of 64 gate and 64 up columns of the outputs n0 .. n0 + 63: a
// thread joins 8 of each.
template <int THREADS, int STRIDE>
__device__ __forceinline__ void join_rows_gated(const LinearEpi& p, float* stg, const float* part0,
                                                long step, int parts, int mine, int row0, int rows,
                                                long m0, int n0) {
  constexpr int CHUNKS = 8, STEP = THREADS / CHUNKS, WROWS = 32 / CHUNKS;
  static_assert(THREADS % CHUNKS == 0, "a thread keeps its columns");
  const int lane = threadIdx.x & 31;
  const int col = (threadIdx.x % CHUNKS) * 8, n = n0 + col;
  if (p.vec && n >= p.N) return;
  float bg[8] = {}, bu[8] = {};  // without vectors: of the columns lane and lane + 32
  if (p.bias != nullptr) {
    if (p.vec) {
      ld8(p.bias, n, p.bias_bf16, bg);
      ld8(p.bias, p.N + n, p.bias_bf16, bu);
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (n0 + lane + 32 * j < p.N) {
          bg[j] = ldf(p.bias, n0 + lane + 32 * j, p.bias_bf16);
          bu[j] = ldf(p.bias, p.N + n0 + lane + 32 * j, p.bias_bf16);
        }
    }
  }
  const int R = 2;  // rows of a thread in flight
  const int end = static_cast<int>(min(static_cast<long>(rows), p.M - m0 - row0));
#pragma unroll 1
  for (int iw = threadIdx.x / 32 * WROWS; iw < end; iw += R * STEP) {  // the warp's first row
    const int i = iw + lane / CHUNKS;
    const int count = max(0, min(R, (end - i + STEP - 1) / STEP)), ra = row0 + i;
    float* const own = stg + ra * STRIDE + col;
    const float* const other = part0 + ra * 128 + col;
    constexpr int OS = STEP * STRIDE, PS = STEP * 128;
    float g[4][8], u[4][8];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < 8; ++j) g[r][j] = u[r][j] = 0.f;
    if (parts == 1) {
      add_parts<2, 1>(own, OS, other, PS, step, 0, mine, count, g);
      add_parts<2, 1>(own + 64, OS, other + 64, PS, step, 0, mine, count, u);
    } else {
      for (int k = 0; k < parts; k += 2) {
        add_parts<2, 2>(own, OS, other, PS, step, k, mine, count, g);
        add_parts<2, 2>(own + 64, OS, other + 64, PS, step, k, mine, count, u);
      }
    }
    if (p.vec) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r < count) gated8<MOE_ACT_NONE>(p, m0 + ra + r * STEP, n, bg, bu, g[r], u[r]);
      continue;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= count) continue;
      float4* q = reinterpret_cast<float4*>(own + r * OS);
      q[0] = make_float4(g[r][0], g[r][1], g[r][2], g[r][3]);
      q[1] = make_float4(g[r][4], g[r][5], g[r][6], g[r][7]);
      q[16] = make_float4(u[r][0], u[r][1], u[r][2], u[r][3]);
      q[17] = make_float4(u[r][4], u[r][5], u[r][6], u[r][7]);
    }
    __syncwarp();
    for (int r = 0; r < R * WROWS; ++r) {  // a warp's lanes along a row
      const int row = iw + r / WROWS * STEP + r % WROWS;
      if (row >= end) continue;
      const float* v = stg + (row0 + row) * STRIDE + lane;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (n0 + lane + 32 * j < p.N)
          gated1<MOE_ACT_NONE>(p, m0 + row0 + row, n0 + lane + 32 * j, v[32 * j] + bg[j],
                               v[64 + 32 * j] + bu[j]);
    }
  }
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// The end of the kernels of few tokens.  s_part: each warp's sums [token][row] of its
// tile of 16 weight rows; `wpr` warps of each of the S blocks of a cluster share a
// tile.  The warps' sums are added in order, then the blocks', through the
// cluster's shared memory (half a kilobyte each), and the results shared out.
constexpr int kStreamWarps = 8;
template <int TOK, bool GATED>
__device__ __forceinline__ void stream_results(const LinearEpi& p, float (&s_part)[kStreamWarps][TOK][17],
                                               float (&s_sum)[kStreamWarps][TOK][16], const int wpr,
                                               const int S, const int rank, const int tiles,
                                               const int tile0, const int N, const int T) {
  constexpr int OUT = GATED ? 8 : 16;  // outputs of a tile
  const int count = tiles * TOK * 16;  // (tile, token, row), the row fastest
  if (S > 1) {
    for (int i = threadIdx.x; i < count; i += kStreamWarps * 32) {
      const int tl = i / (TOK * 16), tok = i / 16 % TOK, r = i % 16;
      float z = 0.f;
      for (int q = 0; q < wpr; ++q) z += s_part[tl * wpr + q][tok][r];
      (&s_sum[0][0][0])[i] = z;
    }
    __syncwarp();
    cluster_sync_all();
  }
  // the blocks of a cluster share the results out among them
  for (int i = threadIdx.x + rank * (kStreamWarps * 32); i < (GATED ? count / 2 : count);
       i += S * (kStreamWarps * 32)) {
    const int tl = i / (TOK * OUT), tok = i / OUT % TOK, r = i % OUT, n = (tile0 + tl) * OUT + r;
    if (n >= N || tok >= T) continue;
    float z = 0.f, zu = 0.f;  // GATED: rows r and 8 + r
    if (S > 1) {
      const uint32_t at = smem_u32(&s_sum[0][0][0] + (GATED ? (tl * TOK + tok) * 16 + r : i));
#pragma unroll 8
      for (int q = 0; q < S; ++q) {
        z += ld_cluster_f32(mapa_shared(at, q));
        if (GATED) zu += ld_cluster_f32(mapa_shared(at + 32u, q));
      }
    } else {
      for (int q = 0; q < wpr; ++q) {
        z += s_part[tl * wpr + q][tok][r];
        if (GATED) zu += s_part[tl * wpr + q][tok][8 + r];
      }
    }
    if (p.bias != nullptr) z += ldf(p.bias, n, p.bias_bf16);
    if (GATED) {
      if (p.bias != nullptr) zu += ldf(p.bias, N + n, p.bias_bf16);
      gated1<MOE_ACT_NONE>(p, tok, n, z, zu);
      continue;
    }
    if (p.preact != nullptr) stf(p.preact, tok * p.ld_out + n, p.out_f32, z);
    z = act_f(z, p.act, p.out_f32);
    if (p.residual != nullptr) z += ldf(p.residual, tok * p.ld_res + n, !p.out_f32);
    stf(p.out, tok * p.ld_out + n, p.out_f32, z);
  }
  if (S > 1) {
    __syncwarp();
    cluster_sync_all();  // the others have read this block's sums
  }
}

// Tile order: groups of `group` row tiles, all column tiles of a group
// before the next, so the tiles in flight share operand rows in L2.
__device__ __forceinline__ void pair_tile(int tile, int mt, int nt, int group, int* mi, int* ni) {
  const int per = group * nt;
  const int g = tile / per;
  const int rows = min(group, mt - g * group);
  const int r = tile - g * per;
  *ni = r / rows;
  *mi = g * group + (r - *ni * rows);
}

}  // namespace
}  // namespace moe
