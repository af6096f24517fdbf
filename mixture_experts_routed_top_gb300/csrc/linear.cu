// Dense products beside the experts: y = residual + act(x w^T + bias) with
// the bias, activation and residual in the epilogue, and the two products
// of its gradient, dx = dz w and dw = dz^T x.
//
// All three are D[M, N] = A B^T over a contraction of length K; what differs
// is which index of an operand is contiguous in memory:
//   forward  A = x  [T, K]   K contiguous        B = w [N, K]  K contiguous
//   dx       A = dz [T, N]   contraction N       B = w [N, K]  its rows run along the contraction
//   dw       A = dz [T, N]   rows along it       B = x [T, K]  rows along it
// Operands whose contraction index is contiguous are "K-major", the others
// "MN-major"; the tensor core reads both from 128-byte swizzled shared
// memory, so no operand is ever transposed in memory.  A K-major tile is
// loaded as boxes of 64 (contraction) x 128 rows, an MN-major one as boxes of
// 64 (rows) x the contraction length of a stage; both land in 128-byte rows.
// Edges in any direction read as zeros (TMA) and are not stored.
//
// The kernels, chosen by linear_streams() and linear_path():
//   linear_pair_kernel   256 x 256 tiles on CTA pairs, persistent: large products
//   linear_sums_kernel   the same tiles with sums in registers: large fp32
//                        results, and tiles that two pairs share
//   linear_tile_kernel   128 x 128 tiles, the contraction split over the CTAs
//                        of a cluster: few tiles
//   linear_stream_kernel a few tokens: the weights streamed into registers, and
//   linear_vector_kernel for one token
#include <algorithm>
#include <atomic>
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
template <bool kCluster>
__device__ __forceinline__ bool wait_cycles(uint32_t bar, uint32_t parity, volatile int* abort,
                                            int* err, int code, long long limit) {
  long long t0 = 0;
  for (int i = 0;; ++i) {
    if (kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
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
  return wait_cycles<true>(bar, parity, abort, err, code, limit);
}
__device__ __forceinline__ bool wait_cta(uint32_t bar, uint32_t parity, volatile int* abort,
                                         int* err, int code, long long limit = kWaitCycles) {
  return wait_cycles<false>(bar, parity, abort, err, code, limit);
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
                                           const uint32_t (&v)[32], float* buf) {
  const int lane = threadIdx.x & 31;
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

// ====================================================== CTA-pair kernel
// tcgen05.mma.cta_group::2, M = 256 (128 rows of A in each CTA), N = 256
// (128 rows of B in each CTA), 128 of the contraction per stage.  Roles in
// each CTA (320 threads): warp 0 TMA producer (ring of 3 stages, 32 KB of A
// and of B each), warp 1 TMEM and, on rank 0, the MMA issuer (two
// 256-column accumulators, so a tile's epilogue runs under the next tile's
// products), warps 2-9 epilogue (32 rows, half of the columns).  Both CTAs'
// loads complete on rank 0's stage barrier; rank 0's commits arrive on both
// CTAs' stage-free and accumulator-full barriers; both epilogues arrive on rank
// 0's accumulator-free barrier.  Every mbarrier wait is bounded.
//
// Bound by the tensor cores, which are busy 88 % of the time: 8192 x 7168 x
// 4096 with bias and gelu 254 us from a cool start (1.89 PFLOP/s) and 306 in an
// endless loop, where the power limit lowers the clock.  Six stages of 64 keep
// more loads in flight, but cost 2 % (a barrier and a commit per 4 products);
// waits without cluster scope, streaming stores and groups of 4, 6, 11, 12, 16
// or 32 row tiles are no faster.
constexpr int kPStages = 3;
constexpr int kPThreads = 320;
constexpr int kPSlab = 128 * BK * 2;        // 16 KB: 128 rows x 64, or 64 rows x 128
constexpr int kPOper = 2 * kPSlab;          // one operand's part of a stage
constexpr int kPOffB = kPStages * kPOper;
constexpr int kPOffBar = 2 * kPStages * kPOper;
constexpr int kPBars = 2 * kPStages + 2 + 2 + 1;
constexpr int kPOffMisc = kPOffBar + kPBars * 8;
constexpr int kPOffTurn = kPOffMisc + 8 + 64;  // a buffer per epilogue warp
static_assert(kPOffTurn % 16 == 0 && kPOffMisc % 8 == 0, "aligned");
constexpr int kPSmem = kPOffTurn + 8 * kTurn * 4 + 1024;
static_assert(kPSmem <= 227 * 1024, "shared memory budget");

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

template <bool A_MN, bool B_MN, int ACT>
__global__ void __launch_bounds__(kPThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tm_a,
                       const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ LinearDev p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kPOffBar);
  uint64_t* full = bars;                  // rank 0: both CTAs' loads of a stage landed
  uint64_t* empty = bars + kPStages;      // both: the stage's MMAs are done
  uint64_t* tfull = bars + 2 * kPStages;  // both: accumulator complete
  uint64_t* tempty = tfull + 2;           // rank 0: both CTAs drained it
  uint64_t* fin = tempty + 2;             // rank 0: every MMA done
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kPOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kPOffMisc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank() & 1u;
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kPStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&tfull[a]), 1);
      mbar_init(smem_u32(&tempty[a]), 16);
    }
    mbar_init(smem_u32(fin), 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
  }
  cluster_sync_all();  // the pair's barriers are up
  if (warp == 1) tmem_alloc_pair(smem_u32(s_tmem), 512);
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the pair's TMEM is allocated in both CTAs
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  const int mt = (p.epi.M + 255) >> 8, nt = (p.epi.N + 255) >> 8;
  const int total = mt * nt;
  const int KB = (p.K + 2 * BK - 1) / (2 * BK);
  const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t ph = 0, issued = 0, last_par = 0;
      bool ok = true;
      for (int tile = cid; ok && tile < total; tile += ncl) {
        int mi, ni;
        pair_tile(tile, mt, nt, p.group, &mi, &ni);
        const int arow = mi * 256 + 128 * static_cast<int>(rank);
        const int brow = ni * 256 + 128 * static_cast<int>(rank);
        for (int kb = 0; kb < KB; ++kb) {
          if (!wait_pair(smem_u32(&empty[stage]), ph ^ 1u, s_abort, p.err,
                                             ERR_TIMEOUT_PRODUCER)) {
            ok = false;
            break;
          }
          const uint32_t fb_local = smem_u32(&full[stage]);
          if (rank == 0) mbar_arrive_expect_tx(fb_local, 2u * 2u * kPOper);
          const uint32_t fb = mapa_shared(fb_local, 0);
          const uint32_t a_dst = smem_u32(smem + stage * kPOper);
          const uint32_t b_dst = smem_u32(smem + kPOffB + stage * kPOper);
          const int k0 = kb * 2 * BK;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (A_MN) tma_load_2d_pair(&tm_a, fb, a_dst + h * kPSlab, arow + BK * h, k0);
            else tma_load_2d_pair(&tm_a, fb, a_dst + h * kPSlab, k0 + BK * h, arow);
            if (B_MN) tma_load_2d_pair(&tm_b, fb, b_dst + h * kPSlab, brow + BK * h, k0);
            else tma_load_2d_pair(&tm_b, fb, b_dst + h * kPSlab, k0 + BK * h, brow);
          }
          issued |= 1u << stage;
          last_par = (last_par & ~(1u << stage)) | (ph << stage);
          if (++stage == kPStages) {
            stage = 0;
            ph ^= 1u;
          }
        }
      }
      // drain: rank 0 until every issued stage's loads (both CTAs') landed,
      // rank 1 until its last loads of each stage were consumed
      for (int s = 0; s < kPStages; ++s) {
        if ((issued >> s) & 1u) {
          volatile int no_abort = 0;
          const uint32_t par = (last_par >> s) & 1u;
          wait_pair(smem_u32(rank == 0 ? &full[s] : &empty[s]), par, &no_abort,
                                        p.err, ERR_TIMEOUT_PRODUCER, kDrainCycles);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_bf16_order(256, 256, A_MN, B_MN);
      int stage = 0, it = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = cid; ok && tile < total; tile += ncl, ++it) {
        const int acc = it & 1;
        if (!wait_pair(smem_u32(&tempty[acc]), ((it >> 1) & 1) ^ 1u, s_abort,
                                           p.err, ERR_TIMEOUT_MMA))
          break;
        tc_fence_after();
        for (int kb = 0; kb < KB; ++kb) {
          if (!wait_pair(smem_u32(&full[stage]), ph, s_abort, p.err,
                                             ERR_TIMEOUT_MMA)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t as = smem_u32(smem + stage * kPOper);
          const uint32_t bs = smem_u32(smem + kPOffB + stage * kPOper);
          const uint64_t ad = A_MN ? sdesc_mn_sw128(as, kPSlab) : sdesc_k_sw128(as);
          const uint64_t bd = B_MN ? sdesc_mn_sw128(bs, kPSlab) : sdesc_k_sw128(bs);
#pragma unroll
          for (int kk = 0; kk < 2 * BK / 16; ++kk) {
            // 16 of the contraction: 32 bytes along a K-major row (the next
            // slab after 64), 16 lines of an MN-major tile
            const uint32_t koff = ((kk >> 2) * kPSlab >> 4) + 2 * (kk & 3), moff = kk * 128;
            umma_f16_pair(tmem + acc * 256, ad + (A_MN ? moff : koff), bd + (B_MN ? moff : koff),
                          idesc, (kb | kk) != 0 ? 1u : 0u);
          }
          umma_commit_pair_both(smem_u32(&empty[stage]));
          if (++stage == kPStages) {
            stage = 0;
            ph ^= 1u;
          }
        }
        if (ok) umma_commit_pair_both(smem_u32(&tfull[acc]));
      }
      if (it > 0) {
        umma_commit_pair_local(smem_u32(fin));
        volatile int no_abort = 0;
        wait_pair(smem_u32(fin), 0, &no_abort, p.err, ERR_TIMEOUT_MMA);
      }
    }
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;  // TMEM lane quarter, column half
    const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16) + 128 * half;
    float* const turn = reinterpret_cast<float*>(smem + kPOffTurn) + (warp - 2) * kTurn;
    int it = 0;
    for (int tile = cid; tile < total; tile += ncl, ++it) {
      int mi, ni;
      pair_tile(tile, mt, nt, p.group, &mi, &ni);
      const int acc = it & 1;
      int ok = 1;
      if (lane == 0)
        ok = wait_pair(smem_u32(&tfull[acc]), (it >> 1) & 1, s_abort, p.err,
                                           ERR_TIMEOUT_EPILOGUE);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const long m = static_cast<long>(mi) * 256 + 128 * rank + 32 * q + lane;
      const int n0 = ni * 256 + 128 * half;
#pragma unroll 1
      for (int s = 0; s < 4; ++s) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(tl + acc * 256 + 32 * s, v);
        tmem_ld_wait();
        if (s == 3) {  // every column read: hand the accumulator back
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (rank == 0) mbar_arrive(smem_u32(&tempty[acc]));
            else mbar_arrive_remote(mapa_shared(smem_u32(&tempty[acc]), 0));
          }
        }
        if (n0 + 32 * s < p.epi.N) epilogue32<ACT, false, B_MN>(p.epi, m, n0 + 32 * s, v, turn);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither CTA leaves while the other may touch its shared memory
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ========================================= CTA pairs, sums in registers
// The same 256 x 256 pair tiles for two cases.
//
// fp32 results.  The tensor core truncates each addition into its fp32
// accumulator, a bias toward zero that grows with the number of additions:
// measured 1.0e-6 of the result per 1024 of the contraction (7.9e-6 at 7168,
// where fp32 arithmetic has 0.9e-6).  So an accumulator takes 768 of the
// contraction, and the epilogue warps add each such part in registers,
// rounding to nearest, while the other accumulator is filled: 7e-7 at any
// length.  8192 x 2048 x 7168 takes 165 us against 142 with bf16 results (whose
// rounding hides the truncation, so linear_pair_kernel takes them).  A thread's
// 128 sums leave 40 of its 168 registers to the epilogue, which stores 264
// bytes of them in local memory; silu with its accurate division 452, and 202 us.
//
// Few tiles.  A cluster of two pairs shares a tile: pair i takes the i-th part
// of the contraction, and the pairs' sums are joined as said above.  8192 x
// 7168 x 256 34 us (0.88 PFLOP/s): 64 pairs, the tensor cores busy half of the
// time, the rest first stages, the join and the epilogue.
//
// 320 threads: producer, MMA, 8 epilogue warps (a thread: one row, 128 columns).
constexpr int kAThreads = 320;
constexpr int kASeg = 6;          // stages (of 128) per part; with 4 the parts cost 2 % more time
constexpr int kAStride = 260;     // floats per staged row: 256 + 4 (no bank conflicts)
static_assert(128 * kAStride * 4 <= kPOffBar, "staged tile fits the ring");

// Arrive on the mbarrier at shared offset `bar` in the CTAs of `mask` when
// this thread's tcgen05 operations so far have completed.
__device__ __forceinline__ void umma_commit_pair_mask(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar), "h"(mask)
      : "memory");
}

// ACT: the activation without a split (fp32 results); with one it is read from
// the arguments, in the single copy of the joining epilogue.
template <bool A_MN, bool B_MN, bool SPLIT, int ACT>
__global__ void __launch_bounds__(kAThreads, 1)
    linear_sums_kernel(const __grid_constant__ CUtensorMap tm_a,
                       const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ LinearDev p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kPOffBar);
  uint64_t* full = bars;                  // leader: both CTAs' loads of a stage landed
  uint64_t* empty = bars + kPStages;      // both: the stage's MMAs are done
  uint64_t* tfull = bars + 2 * kPStages;  // both: a part is complete
  uint64_t* tempty = tfull + 2;           // leader: both CTAs have read it
  uint64_t* fin = tempty + 2;             // leader: every MMA done
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kPOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kPOffMisc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int crank = static_cast<int>(cluster_ctarank());
  const int rank = crank & 1, pair = crank >> 1, S = SPLIT ? p.split : 1;
  const uint32_t lead = static_cast<uint32_t>(crank & ~1);
  const uint16_t both = static_cast<uint16_t>(3u << lead);
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kPStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&tfull[a]), 1);
      mbar_init(smem_u32(&tempty[a]), 16);
    }
    mbar_init(smem_u32(fin), 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
  }
  cluster_sync_all();
  if (warp == 1) tmem_alloc_pair(smem_u32(s_tmem), 512);
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  const int mt = (p.epi.M + 255) >> 8, nt = (p.epi.N + 255) >> 8;
  const int total = mt * nt;
  const int KB = (p.K + 2 * BK - 1) / (2 * BK);
  const int kb0 = static_cast<int>(static_cast<long>(KB) * pair / S);
  const int kb1 = static_cast<int>(static_cast<long>(KB) * (pair + 1) / S);
  const int cid = blockIdx.x / (2 * S), ncl = gridDim.x / (2 * S);

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t ph = 0, issued = 0, last_par = 0;
      bool ok = true;
      for (int tile = cid; ok && tile < total; tile += ncl) {
        int mi, ni;
        pair_tile(tile, mt, nt, p.group, &mi, &ni);
        const int arow = mi * 256 + 128 * rank, brow = ni * 256 + 128 * rank;
        // tiles begin at different places of their part, so that the tiles in
        // flight do not all ask for the same lines of the other operand at once
        int kb = kb0 + static_cast<int>(static_cast<long>(tile) * 5 % (kb1 - kb0));
        for (int left = kb1 - kb0; left > 0; --left) {
          if (!wait_pair(smem_u32(&empty[stage]), ph ^ 1u, s_abort, p.err,
                                             ERR_TIMEOUT_PRODUCER)) {
            ok = false;
            break;
          }
          const uint32_t fb_local = smem_u32(&full[stage]);
          if (rank == 0) mbar_arrive_expect_tx(fb_local, 2u * 2u * kPOper);
          const uint32_t fb = mapa_shared(fb_local, lead);
          const uint32_t a_dst = smem_u32(smem + stage * kPOper);
          const uint32_t b_dst = smem_u32(smem + kPOffB + stage * kPOper);
          const int k0 = kb * 2 * BK;
          if (++kb == kb1) kb = kb0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (A_MN) tma_load_2d_pair(&tm_a, fb, a_dst + h * kPSlab, arow + BK * h, k0);
            else tma_load_2d_pair(&tm_a, fb, a_dst + h * kPSlab, k0 + BK * h, arow);
            if (B_MN) tma_load_2d_pair(&tm_b, fb, b_dst + h * kPSlab, brow + BK * h, k0);
            else tma_load_2d_pair(&tm_b, fb, b_dst + h * kPSlab, k0 + BK * h, brow);
          }
          issued |= 1u << stage;
          last_par = (last_par & ~(1u << stage)) | (ph << stage);
          if (++stage == kPStages) {
            stage = 0;
            ph ^= 1u;
          }
        }
      }
      // drain: the leader until every issued stage's loads (both CTAs')
      // landed, the other until its last loads of each stage were consumed
      for (int s = 0; s < kPStages; ++s) {
        if ((issued >> s) & 1u) {
          volatile int no_abort = 0;
          const uint32_t par = (last_par >> s) & 1u;
          wait_pair(smem_u32(rank == 0 ? &full[s] : &empty[s]), par, &no_abort,
                                        p.err, ERR_TIMEOUT_PRODUCER, kDrainCycles);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_bf16_order(256, 256, A_MN, B_MN);
      int stage = 0, it = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = cid; ok && tile < total; tile += ncl) {
        for (int kb = kb0; ok && kb < kb1; ++it) {
          const int acc = it & 1;
          if (!wait_pair(smem_u32(&tempty[acc]), ((it >> 1) & 1) ^ 1u, s_abort,
                                             p.err, ERR_TIMEOUT_MMA)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int end = min(kb + kASeg, kb1);
          for (bool first = true; kb < end; ++kb, first = false) {
            if (!wait_pair(smem_u32(&full[stage]), ph, s_abort, p.err,
                                               ERR_TIMEOUT_MMA)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t as = smem_u32(smem + stage * kPOper);
            const uint32_t bs = smem_u32(smem + kPOffB + stage * kPOper);
            const uint64_t ad = A_MN ? sdesc_mn_sw128(as, kPSlab) : sdesc_k_sw128(as);
            const uint64_t bd = B_MN ? sdesc_mn_sw128(bs, kPSlab) : sdesc_k_sw128(bs);
#pragma unroll
            for (int kk = 0; kk < 2 * BK / 16; ++kk) {
              const uint32_t koff = ((kk >> 2) * kPSlab >> 4) + 2 * (kk & 3), moff = kk * 128;
              umma_f16_pair(tmem + acc * 256, ad + (A_MN ? moff : koff), bd + (B_MN ? moff : koff),
                            idesc, (!first || kk != 0) ? 1u : 0u);
            }
            umma_commit_pair_mask(smem_u32(&empty[stage]), both);
            if (++stage == kPStages) {
              stage = 0;
              ph ^= 1u;
            }
          }
          if (ok) umma_commit_pair_mask(smem_u32(&tfull[acc]), both);
        }
      }
      if (it > 0) {
        umma_commit_pair_local(smem_u32(fin));
        volatile int no_abort = 0;
        wait_pair(smem_u32(fin), 0, &no_abort, p.err, ERR_TIMEOUT_MMA);
      }
    }
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;  // TMEM lane quarter, column half
    const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16) + 128 * half;
    float* const turn = reinterpret_cast<float*>(smem + kPOffTurn) + (warp - 2) * kTurn;
    auto release = [&](int buf) {  // this warp has read the part
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(smem_u32(&tempty[buf]));
        else mbar_arrive_remote(mapa_shared(smem_u32(&tempty[buf]), lead));
      }
    };
    int it = 0;
    for (int tile = cid; tile < total; tile += ncl) {
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.f;
      int ok = 1;
#pragma unroll 1
      for (int kb = kb0; kb < kb1; kb += kASeg, ++it) {
        const int buf = it & 1;
        if (lane == 0)
          ok = wait_pair(smem_u32(&tfull[buf]), (it >> 1) & 1, s_abort, p.err, ERR_TIMEOUT_EPILOGUE);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(tl + buf * 256 + 32 * s, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[32 * s + i] += __uint_as_float(v[i]);
        }
        release(buf);
      }
      if (!ok) break;
      if (SPLIT) {
        // one tile per cluster: the last part has been read, so every load
        // has landed and every product is done
        float* row = reinterpret_cast<float*>(smem) + (32 * q + lane) * kAStride + 128 * half;
#pragma unroll
        for (int j = 0; j < 128; j += 4)
          *reinterpret_cast<float4*>(row + j) =
              make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
      } else {
        int mi, ni;
        pair_tile(tile, mt, nt, p.group, &mi, &ni);
        const long m = static_cast<long>(mi) * 256 + 128 * rank + 32 * q + lane;
        const int n0 = ni * 256 + 128 * half;
#pragma unroll
        for (int s = 0; s < 4; ++s) {  // the accumulators are free: the next tile runs on
          uint32_t v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(acc[32 * s + i]);
          if (n0 + 32 * s < p.epi.N) epilogue32<ACT, true, false>(p.epi, m, n0 + 32 * s, v, turn);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  float* const stg = reinterpret_cast<float*>(smem);
  const int rows = 128 / S;
  if (SPLIT)
    hand_over<kAThreads, 32, kAStride>(stg, p.parts + static_cast<long>(blockIdx.x) * 128 * 256,
                                       pair * rows, rows);
  __syncwarp();
  cluster_sync_all();  // sums handed over; without a split: nobody is still signalling
  tc_fence_after();
  if (SPLIT && !*s_abort) {
    int mi, ni;
    pair_tile(cid, mt, nt, p.group, &mi, &ni);
    // the CTAs of this rank of each pair, two apart
    join_rows<kAThreads, 32, kAStride, B_MN>(
        p.epi, stg, p.parts + static_cast<long>(blockIdx.x - 2 * pair) * 128 * 256, 2l * 128 * 256,
        S, pair, pair * rows, rows, static_cast<long>(mi) * 256 + 128 * rank, ni * 256);
  }
  __syncwarp();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ====================================================== split tile kernel
// One 128 x 128 tile per cluster of S CTAs; CTA r takes the r-th part of the
// contraction (at least one stage), in two accumulators, which halves the
// tensor core's truncation; the CTAs' sums are joined as said above.  Two CTAs
// fit an SM (with 256 TMEM columns each).  Bound by latency: the way of the first
// and the last stage, and the exchange of the sums.  1024 x 2048 x 2048 15.3 us
// (0.56 PFLOP/s), 64 x 2048 x 7168 13.4, of which the weights take 4.3.
constexpr int kTStages = 3;
constexpr int kTThreads = 192;
constexpr int kTOper = 128 * BK * 2;             // 16 KB: one operand's part of a stage
constexpr int kTOffB = kTStages * kTOper;
constexpr int kTOffBar = 2 * kTStages * kTOper;
constexpr int kTBars = 2 * kTStages + 1;
constexpr int kTOffMisc = kTOffBar + kTBars * 8;
constexpr int kTSmem = kTOffMisc + 16 + 1024;
constexpr int kTStride = 132;                    // floats per staged row: 128 + 4 (no bank conflicts)
static_assert(128 * kTStride * 4 <= kTOffBar, "staged tile fits the ring");

template <bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kTThreads)
    linear_tile_kernel(const __grid_constant__ CUtensorMap tm_a,
                       const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ LinearDev p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kTOffBar);
  uint64_t* empty = full + kTStages;
  uint64_t* done = empty + kTStages;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kTOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kTOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.split;
  const int rank = static_cast<int>(cluster_ctarank());
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kTStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(done), 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
  }
  if (warp == 1) tmem_alloc(smem_u32(s_tmem), 256);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  const uint32_t tmem = *s_tmem;
  const int mt = (p.epi.M + 127) >> 7;
  const int tile = blockIdx.x / S;
  const int mi = tile % mt, ni = tile / mt;
  const int KB = (p.K + BK - 1) / BK;
  const int kb0 = static_cast<int>(static_cast<long>(KB) * rank / S);
  const int kb1 = static_cast<int>(static_cast<long>(KB) * (rank + 1) / S);
  const int kmid = kb0 + (kb1 - kb0 + 1) / 2;  // from here on the second accumulator
  int ok = 1;
  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t ph = 0, issued = 0, last_par = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait_cta(smem_u32(&empty[stage]), ph ^ 1u, s_abort, p.err,
                                     ERR_TIMEOUT_PRODUCER))
          break;
        const uint32_t fb = smem_u32(&full[stage]);
        mbar_arrive_expect_tx(fb, 2u * kTOper);
        const uint32_t a_dst = smem_u32(smem + stage * kTOper);
        const uint32_t b_dst = smem_u32(smem + kTOffB + stage * kTOper);
        const int k0 = kb * BK;
        if (A_MN) {  // two boxes of 64 rows x 64 lines
          tma_load_2d(&tm_a, fb, a_dst, mi * 128, k0);
          tma_load_2d(&tm_a, fb, a_dst + kTOper / 2, mi * 128 + BK, k0);
        } else {
          tma_load_2d(&tm_a, fb, a_dst, k0, mi * 128);
        }
        if (B_MN) {
          tma_load_2d(&tm_b, fb, b_dst, ni * 128, k0);
          tma_load_2d(&tm_b, fb, b_dst + kTOper / 2, ni * 128 + BK, k0);
        } else {
          tma_load_2d(&tm_b, fb, b_dst, k0, ni * 128);
        }
        issued |= 1u << stage;
        last_par = (last_par & ~(1u << stage)) | (ph << stage);
        if (++stage == kTStages) {
          stage = 0;
          ph ^= 1u;
        }
      }
      for (int s = 0; s < kTStages; ++s) {  // nothing in flight when the ring is reused
        if ((issued >> s) & 1u) {
          volatile int no_abort = 0;
          wait_cta(smem_u32(&full[s]), (last_par >> s) & 1u, &no_abort, p.err,
                                  ERR_TIMEOUT_PRODUCER, kDrainCycles);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_order(128, 128, A_MN, B_MN);
      int stage = 0;
      uint32_t ph = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait_cta(smem_u32(&full[stage]), ph, s_abort, p.err, ERR_TIMEOUT_MMA))
          break;
        tc_fence_after();
        const uint32_t as = smem_u32(smem + stage * kTOper);
        const uint32_t bs = smem_u32(smem + kTOffB + stage * kTOper);
        const uint64_t ad = A_MN ? sdesc_mn_sw128(as, kTOper / 2) : sdesc_k_sw128(as);
        const uint64_t bd = B_MN ? sdesc_mn_sw128(bs, kTOper / 2) : sdesc_k_sw128(bs);
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          umma_f16(tmem + (kb < kmid ? 0 : 128), ad + (A_MN ? kk * 128 : kk * 2),
                   bd + (B_MN ? kk * 128 : kk * 2), idesc,
                   (kk > 0 || (kb != kb0 && kb != kmid)) ? 1u : 0u);
        umma_commit(smem_u32(&empty[stage]));
        if (++stage == kTStages) {
          stage = 0;
          ph ^= 1u;
        }
      }
      umma_commit(smem_u32(done));
    }
  }
  // every thread waits for the last product: after it the ring is free
  if (!wait_cta(smem_u32(done), 0, s_abort, p.err, ERR_TIMEOUT_EPILOGUE) || *s_abort)
    ok = 0;
  __syncthreads();
  __syncwarp();
  tc_fence_after();
  if (warp >= 2) {
    const int q = warp & 3;
    float* row = reinterpret_cast<float*>(smem) + (32 * q + lane) * kTStride;
#pragma unroll 1
    for (int s = 0; s < 4; ++s) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(q * 32) << 16) + 32 * s, v);
      tmem_ld_wait();
      if (kmid < kb1) {
        uint32_t u[32];
        tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(q * 32) << 16) + 128 + 32 * s, u);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j)
          v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(u[j]));
      }
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        *reinterpret_cast<float4*>(row + 32 * s + j) =
            make_float4(__uint_as_float(v[j]), __uint_as_float(v[j + 1]), __uint_as_float(v[j + 2]),
                        __uint_as_float(v[j + 3]));
    }
    tc_fence_before();
  }
  __syncthreads();
  float* const stg = reinterpret_cast<float*>(smem);
  const int rows = 128 / S;
  if (S > 1) {
    hand_over<kTThreads, 16, kTStride>(stg, p.parts + static_cast<long>(blockIdx.x) * 128 * 128,
                                       rank * rows, rows);
    __syncwarp();
    cluster_sync_all();  // sums handed over
  }
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 256);
  if (ok)
    join_rows<kTThreads, 16, kTStride, B_MN>(
        p.epi, stg, p.parts + static_cast<long>(blockIdx.x - rank) * 128 * 128, 128l * 128, S, rank,
        rank * rows, rows, static_cast<long>(mi) * 128, ni * 128);
}

// ====================================================== one token
// The weights [N, K] are read once, and that is what it costs: WPR warps of a
// block share two rows of w, each lane multiplying 16-byte pieces of them with
// the token's, and add their sums in order.  2048 x 7168 6.3 us from memory
// (4.7 TB/s, 2 us more than the bytes need), 3.7 from L2.
template <int WPR>
__global__ void __launch_bounds__(256)
    linear_vector_kernel(const __grid_constant__ LinearStreamArgs a) {
  constexpr int R = 2;                // rows of w per warp: they share the token's loads
  constexpr int GROUPS = 8 / WPR;     // row pairs per block
  pdl_launch_dependents();
  __shared__ float s_part[8][R];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = warp / WPR, part = warp % WPR;
  const int n0 = (blockIdx.x * GROUPS + grp) * R;
  pdl_wait();
  float acc[R] = {};
  const int chunks = a.K / 8;
  if (n0 < a.epi.N) {
    const __nv_bfloat16* w0 = a.w + static_cast<long>(n0) * a.ld_w;
    const __nv_bfloat16* w1 = a.w + static_cast<long>(min(n0 + 1, a.epi.N - 1)) * a.ld_w;
#pragma unroll 4
    for (int c = part * 32 + lane; c < chunks; c += WPR * 32) {
      float f[R][8], x[8];
      ld8(w0, c * 8, true, f[0]);
      ld8(w1, c * 8, true, f[1]);
      ld8(a.x, c * 8, true, x);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[r] = fmaf(f[r][j], x[j], acc[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], off);
    if (lane == 0) s_part[warp][r] = acc[r];
  }
  __syncthreads();
  const int i = threadIdx.x, n = blockIdx.x * GROUPS * R + i;
  if (i < GROUPS * R && n < a.epi.N) {
    float z = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) z += s_part[i / R * WPR + w][i % R];
    const LinearEpi& p = a.epi;
    if (p.bias != nullptr) z += ldf(p.bias, n, p.bias_bf16);
    if (p.preact != nullptr) stf(p.preact, n, p.out_f32, z);
    z = act_f(z, p.act, p.out_f32);
    if (p.residual != nullptr) z += ldf(p.residual, n, !p.out_f32);
    stf(p.out, n, p.out_f32, z);
  }
}

// ====================================================== few tokens
// 2 to 16 tokens, to 32 where there are few rows: the weights [N, K] are again
// read once, straight from memory into the registers that multiply them.  So
// no tiles in shared memory and no TMEM: a thread's 16-byte loads are operand
// fragments of the warp-level product (16 weight rows x 8 tokens x 16), whose
// contraction index may be counted in any order as long as both operands do
// it alike: of 32 consecutive elements of a row, lane 4 g + t holds 8 t .. 8 t + 7
// of row g (and of row g + 8, and of token g), the first four of them in one
// instruction and the others in the next.  8 tokens at 2048 x 7168 (weights that
// take 4.3 us to arrive) 9.4 us, against 24 on CUDA cores, most of it unpacking,
// and 15 in tiles with a split contraction; 16 tokens 10.6 against 15; 32 tokens
// at 256 x 7168 5.6 against 10.4, but at 7168 x 2048 14.3 against 13.4.
//
// A tile of 16 rows is shared by `wpr` warps of each of the S blocks of a cluster,
// which take groups of 32 G of the contraction in turn and ask for a whole
// group before they use any of it; the more of them, the more of the weights
// are on their way at once.  After each group its sums are added to fp32
// registers (the tensor core truncates its additions); at the end the warps'
// sums are added in order, then the blocks', through the cluster's shared
// memory (half a kilobyte each).
__device__ __forceinline__ uint4 ld_stream(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void warp_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

constexpr int kStreamWarps = 8;
// NT: groups of 8 tokens; G: steps of 32 of the contraction per group.
template <int NT>
struct StreamLay {
  static constexpr int G = NT == 1 ? 8 : 4, TOK = 8 * NT;
};
template <int NT>
__global__ void __launch_bounds__(kStreamWarps * 32)
    linear_stream_kernel(const __grid_constant__ LinearStreamArgs a) {
  constexpr int G = StreamLay<NT>::G, TOK = StreamLay<NT>::TOK;
  pdl_launch_dependents();
  __shared__ float s_part[kStreamWarps][TOK][17];
  __shared__ float s_sum[kStreamWarps][TOK][16];  // of a tile, over this block's warps
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int wpr = a.wpr, S = a.split, rank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tiles = kStreamWarps / wpr;  // of a block
  const int tile0 = blockIdx.x / S * tiles, part = rank * wpr + warp % wpr;
  const int n0 = (tile0 + warp / wpr) * 16;
  const int N = a.epi.N, T = a.epi.M, K = a.K;
  pdl_wait();
  float sum[NT][4] = {};
  if (n0 < N) {
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const bool on0 = n0 + g < N, on1 = n0 + 8 + g < N;
    const __nv_bfloat16* w0 = a.w + static_cast<long>(n0 + g) * a.ld_w;
    const __nv_bfloat16* w1 = w0 + 8 * a.ld_w;
#pragma unroll 1
    for (int k0 = part * (32 * G); k0 < K; k0 += wpr * S * (32 * G)) {
      uint4 wv[G][2], xv[G][NT];
#pragma unroll
      for (int s = 0; s < G; ++s) {
        const int k = k0 + 32 * s + 8 * t;
        wv[s][0] = on0 && k < K ? ld_stream(w0 + k) : zero;
        wv[s][1] = on1 && k < K ? ld_stream(w1 + k) : zero;
      }
#pragma unroll
      for (int s = 0; s < G; ++s) {
        const int k = k0 + 32 * s + 8 * t;
#pragma unroll
        for (int q = 0; q < NT; ++q)
          xv[s][q] = 8 * q + g < T && k < K
                         ? __ldg(reinterpret_cast<const uint4*>(a.x + (8 * q + g) * a.ld_x + k))
                         : zero;
      }
      float c[NT][4] = {};
#pragma unroll
      for (int s = 0; s < G; ++s)
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          const uint4 lo = wv[s][0], hi = wv[s][1], x = xv[s][q];
          warp_mma(c[q], lo.x, hi.x, lo.y, hi.y, x.x, x.y);
          warp_mma(c[q], lo.z, hi.z, lo.w, hi.w, x.z, x.w);
        }
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[q][i] += c[q][i];
    }
  }
  // a lane's sums: rows g and g + 8, tokens 2 t and 2 t + 1 of each 8
#pragma unroll
  for (int q = 0; q < NT; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) s_part[warp][8 * q + 2 * t + (i & 1)][g + 8 * (i >> 1)] = sum[q][i];
  __syncthreads();
  const LinearEpi& p = a.epi;
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
  for (int i = threadIdx.x + rank * (kStreamWarps * 32); i < count; i += S * (kStreamWarps * 32)) {
    const int tl = i / (TOK * 16), tok = i / 16 % TOK, r = i % 16, n = (tile0 + tl) * 16 + r;
    if (n >= N || tok >= T) continue;
    float z = 0.f;
    if (S > 1) {
      const uint32_t at = smem_u32(&s_sum[0][0][0] + i);
#pragma unroll 8
      for (int q = 0; q < S; ++q) z += ld_cluster_f32(mapa_shared(at, q));
    } else {
      for (int q = 0; q < wpr; ++q) z += s_part[tl * wpr + q][tok][r];
    }
    if (p.bias != nullptr) z += ldf(p.bias, n, p.bias_bf16);
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

// ====================================================== dz and dbias
// dz = dy * act'(z) rounded to bf16 for the two products (their operands are
// bf16 tiles), and the column sums of the unrounded dz.  A block covers 256
// columns (8 per thread) and a slice of the rows; the slices' sums are added
// in order by linear_colsum_kernel.
// One exponential per slope, with the fast exponential and division: at most
// a few units of 2^-22, far below the rounding of dz (2^-9 on average) and
// averaged out in the sums.  With the accurate forms the kernel took 40 us for
// 8191 x 2048 with silu, three times what its loads and stores need; now 22
// (100 MB, 4.6 TB/s, 19 instructions an element).
// SPLIT, the second part of few dz, is a constant of the code: as a test in the
// loop that large gradients run it cost 15 registers and 12 us.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if (ACT == MOE_ACT_SILU) {  // s (1 + z (1 - s)), 1 - s = e^-z s; below -80 (-1.4e-33) as at -80
    z = z < -80.f ? -80.f : z;
    const float e = __expf(-z), s = __fdividef(1.f, 1.f + e);
    return s * fmaf(z, e * s, 1.f);
  }
  if (ACT == MOE_ACT_GELU)  // Phi(z) + z phi(z); the second term is 0 long before z^2 overflows
    return fmaf(z * __expf(-0.5f * fminf(z * z, 1000.f)), 0.39894228040143268f,
                0.5f * (1.f + erff(z * 0.70710678118654752f)));
  return z > 0.f ? 1.f : 0.f;
}

template <int ACT, bool F32, bool SPLIT>
__global__ void __launch_bounds__(256) linear_dz_kernel(const LinearDzArgs a) {
  pdl_launch_dependents();
  __shared__ float s_sum[8][256];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int n = blockIdx.x * 256 + x * 8;
  pdl_wait();
  const long t0 = static_cast<long>(a.T) * blockIdx.y / gridDim.y;
  const long t1 = static_cast<long>(a.T) * (blockIdx.y + 1) / gridDim.y;
  float sum[8] = {};
  auto row = [&](long t, float (&d)[8], float (&z)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (ACT != MOE_ACT_NONE) d[j] *= act_slope<ACT>(z[j]);
      sum[j] += d[j];
    }
    if (a.dz != nullptr) st8(a.dz, t * a.ld_dz + n, false, d);  // rows padded to 8: always whole
    if (SPLIT) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // nothing is left of one that bf16 has no finite value for
        const float hi = __bfloat162float(__float2bfloat16_rn(d[j]));
        d[j] = fabsf(hi) < INFINITY ? d[j] - hi : 0.f;
      }
      st8(a.dz_lo, t * a.ld_dz + n, false, d);
    }
  };
  if (n < a.N && a.vec) {
#pragma unroll 4
    for (long t = t0 + y; t < t1; t += 8) {
      float d[8], z[8];
      ld8(a.dy, t * a.ld_dy + n, !F32, d);
      if (ACT != MOE_ACT_NONE) ld8(a.preact, t * a.ld_z + n, !F32, z);
      row(t, d, z);
    }
  } else if (n < a.N) {
    for (long t = t0 + y; t < t1; t += 8) {
      float d[8], z[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool in = n + j < a.N;
        d[j] = in ? ldf(a.dy, t * a.ld_dy + n + j, !F32) : 0.f;
        z[j] = in && ACT != MOE_ACT_NONE ? ldf(a.preact, t * a.ld_z + n + j, !F32) : 0.f;
      }
      row(t, d, z);
    }
  }
  if (a.partials == nullptr) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) s_sum[y][x * 8 + j] = sum[j];
  __syncthreads();
  const int col = blockIdx.x * 256 + threadIdx.x;
  if (col < a.N) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += s_sum[i][threadIdx.x];
    a.partials[static_cast<long>(blockIdx.y) * a.N + col] = v;
  }
}

// Sums of the slices' partial rows: 32 columns x 8 parts of the slices per
// block, each part added in order, then the parts.
__global__ void __launch_bounds__(256)
    linear_colsum_kernel(const float* __restrict__ partials, int slices, int N, float* out) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float s[8][33];
  const int x = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int n = blockIdx.x * 32 + x;
  float v = 0.f;
  if (n < N) {
#pragma unroll 8
    for (int i = part; i < slices; i += 8) v += partials[static_cast<long>(i) * N + n];
  }
  s[part][x] = v;
  __syncthreads();
  if (part == 0 && n < N) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += s[i][x];
    out[n] = v;
  }
}

template <bool A_MN, bool B_MN, int ACT>
cudaError_t launch_pair(const CUtensorMap& tm_a, const CUtensorMap& tm_b, LinearDev p,
                        cudaStream_t s) {
  auto kern = linear_pair_kernel<A_MN, B_MN, ACT>;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64) return cudaErrorInvalidDevice;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(kPThreads);
  cfg.dynamicSmemBytes = kPSmem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static std::atomic<int> max_clusters[64] = {};
  int nc = max_clusters[dev].load(std::memory_order_acquire);
  if (nc == 0) {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kPSmem);
    if (err != cudaSuccess) return err;
    err = cudaOccupancyMaxActiveClusters(&nc, kern, &cfg);
    if (err != cudaSuccess) return err;
    if (nc < 1) return cudaErrorLaunchOutOfResources;
    max_clusters[dev].store(nc, std::memory_order_release);
  }
  const long tiles = static_cast<long>(ceil_div(p.epi.M, 256)) * ceil_div(p.epi.N, 256);
  p.group = 8;
  cfg.gridDim = dim3(2 * static_cast<int>(std::min<long>(nc, tiles)));
  cfg.stream = s;
  cfg.numAttrs = 2;
  err = cudaLaunchKernelEx(&cfg, kern, tm_a, tm_b, p);
  count_launches(1);
  return err != cudaSuccess ? err : cudaGetLastError();
}

template <bool A_MN, bool B_MN, bool SPLIT, int ACT>
cudaError_t launch_sums(const CUtensorMap& tm_a, const CUtensorMap& tm_b, LinearDev p, int split,
                        cudaStream_t s) {
  auto kern = linear_sums_kernel<A_MN, B_MN, SPLIT, ACT>;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64) return cudaErrorInvalidDevice;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * split);
  cfg.blockDim = dim3(kAThreads);
  cfg.dynamicSmemBytes = kPSmem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static std::atomic<int> max_clusters[64] = {};  // pairs without a split
  int nc = max_clusters[dev].load(std::memory_order_acquire);
  if (nc == 0) {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kPSmem);
    if (err != cudaSuccess) return err;
    cfg.gridDim = dim3(2);
    attr[0].val.clusterDim.x = 2;
    err = cudaOccupancyMaxActiveClusters(&nc, kern, &cfg);
    if (err != cudaSuccess) return err;
    if (nc < 1) return cudaErrorLaunchOutOfResources;
    max_clusters[dev].store(nc, std::memory_order_release);
    attr[0].val.clusterDim.x = 2 * split;
  }
  const long tiles = static_cast<long>(ceil_div(p.epi.M, 256)) * ceil_div(p.epi.N, 256);
  p.group = 8;
  p.split = split;
  // without a split the pairs stay and walk over the tiles; with one a
  // cluster takes one tile
  cfg.gridDim = dim3(2 * split * static_cast<int>(split > 1 ? tiles : std::min<long>(nc, tiles)));
  cfg.stream = s;
  cfg.numAttrs = 2;
  err = cudaLaunchKernelEx(&cfg, kern, tm_a, tm_b, p);
  count_launches(1);
  return err != cudaSuccess ? err : cudaGetLastError();
}

template <bool A_MN, bool B_MN>
cudaError_t launch_tile(const CUtensorMap& tm_a, const CUtensorMap& tm_b, LinearDev p, int split,
                        cudaStream_t s) {
  auto kern = linear_tile_kernel<A_MN, B_MN>;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64) return cudaErrorInvalidDevice;
  static std::atomic<int> ready[64] = {};
  if (!ready[dev].load(std::memory_order_acquire)) {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kTSmem);
    if (err != cudaSuccess) return err;
    ready[dev].store(1, std::memory_order_release);
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  p.split = split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ceil_div(p.epi.M, 128) * ceil_div(p.epi.N, 128) * split);
  cfg.blockDim = dim3(kTThreads);
  cfg.dynamicSmemBytes = kTSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  err = cudaLaunchKernelEx(&cfg, kern, tm_a, tm_b, p);
  count_launches(1);
  return err != cudaSuccess ? err : cudaGetLastError();
}

template <int WPR>
cudaError_t launch_vector_w(const LinearStreamArgs& a, cudaStream_t s) {
  return launch_pdl(linear_vector_kernel<WPR>, dim3(ceil_div(a.epi.N, 8 / WPR * 2)), dim3(256), 0, s, a);
}
cudaError_t launch_vector(const LinearStreamArgs& a, int num_sms, cudaStream_t s) {
  // warps per row pair: enough that every SM has 40 warps, at most 8
  const long pairs = (a.epi.N + 1) / 2, want = 40L * num_sms;
  if (pairs >= want) return launch_vector_w<1>(a, s);
  if (2 * pairs >= want) return launch_vector_w<2>(a, s);
  if (4 * pairs >= want) return launch_vector_w<4>(a, s);
  return launch_vector_w<8>(a, s);
}

template <int ACT>
cudaError_t launch_dz(const LinearDzArgs& a, dim3 grid, cudaStream_t s) {
  const dim3 block(256);
  if (a.dz_lo != nullptr) {
    if (a.f32) return launch_pdl(linear_dz_kernel<ACT, true, true>, grid, block, 0, s, a);
    if constexpr (ACT == MOE_ACT_SILU || ACT == MOE_ACT_GELU)
      return launch_pdl(linear_dz_kernel<ACT, false, true>, grid, block, 0, s, a);
    return cudaErrorInvalidValue;  // bf16 gradients times 0 or 1 have no second part
  }
  return a.f32 ? launch_pdl(linear_dz_kernel<ACT, true, false>, grid, block, 0, s, a)
               : launch_pdl(linear_dz_kernel<ACT, false, false>, grid, block, 0, s, a);
}

template <int NT>
cudaError_t launch_stream(LinearStreamArgs a, int num_sms, cudaStream_t s) {
  // warps of a block per tile, then blocks: until every SM has WANT warps, as
  // long as each has a group of the contraction
  constexpr long WANT = 16;
  constexpr int kGroup = 32 * StreamLay<NT>::G;
  const long tiles = ceil_div(a.epi.N, 16);
  a.wpr = a.split = 1;
  while (a.wpr < kStreamWarps && tiles * a.wpr < WANT * num_sms && a.wpr * kGroup < a.K) a.wpr *= 2;
  while (a.split < 8 && tiles * a.wpr * a.split < WANT * num_sms && a.wpr * a.split * kGroup < a.K)
    a.split *= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ceil_div(tiles, kStreamWarps / a.wpr) * a.split);
  cfg.blockDim = dim3(kStreamWarps * 32);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = a.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, linear_stream_kernel<NT>, a);
}

}  // namespace

// Which kernel, and how many parts of the contraction.  256 x 256 tiles on
// persistent pairs from half a wave of them (measured, bf16: 512 x 2048 x 7168,
// 56 tiles, 20.2 us against 21.6 in 128 x 128 tiles).  Below, 128 x 128 tiles
// with the contraction split until the grid covers the GPU twice (two such
// CTAs fit an SM), each part at least 4 stages long: 64 x 7168 x 4096 21 us
// against 29 on split pairs, 1024 x 2048 x 2048 15.3 against 16.9.  Two pairs
// per tile where that gives most of a wave of full tiles and the contraction
// is long, so that reading the operands counts (8192 x 7168 x 256 34 us against
// 36, but 8192 x 7168 x 64 31 against 28), or where an fp32 result would have more
// than 1024 of the contraction in one accumulator (unless the split of the small
// tiles is at its end: from K = 16384 on, with few tiles, it has more).
LinearPath linear_path(long M, long N, long K, bool out_f32, int num_sms) {
  LinearPath r;
  const long big = static_cast<long>(ceil_div(M, 256)) * ceil_div(N, 256);
  const long pairs = std::min(num_sms, kLinearMaxParts / 2) / 2;
  r.split = 1;
  if (big >= pairs / 2) {
    r.kind = out_f32 ? LinearPath::kSums : LinearPath::kPair;
    return r;
  }
  r.kind = LinearPath::kTile;
  const long tiles = static_cast<long>(ceil_div(M, 128)) * ceil_div(N, 128);
  while (r.split < 8 && tiles * r.split * 2 <= 4 * pairs && K / (r.split * 2) >= 4 * BK)
    r.split *= 2;
  if ((big * 8 >= pairs * 3 && 3 * big <= tiles && K >= 64 * BK) ||
      (out_f32 && K / (2 * r.split) > 16 * BK && r.split < 8)) {
    r.kind = LinearPath::kSums;  // 2 * big <= pairs here
    r.split = 2;
  }
  return r;
}

cudaError_t launch_linear(const CUtensorMap& tm_a, const CUtensorMap& tm_b, const LinearDev& p,
                          bool a_mn, bool b_mn, const LinearPath& path, cudaStream_t s) {
  constexpr int kNone = MOE_ACT_NONE;
  const int act = p.epi.act;
  // what each kernel supports, whatever chose the path: the CTA-pair kernel
  // stores bf16, the register sums fp32 unless they are joined, a split has
  // no empty part and its sums fit the workspace
  const bool sums = path.kind == LinearPath::kSums;
  const long parts = static_cast<long>(path.split) *
                     (sums ? 4l * ceil_div(p.epi.M, 256) * ceil_div(p.epi.N, 256)
                           : static_cast<long>(ceil_div(p.epi.M, 128)) * ceil_div(p.epi.N, 128));
  const int stages = ceil_div(p.K, sums ? 2 * BK : BK);
  if ((path.kind == LinearPath::kPair && p.epi.out_f32) ||
      (sums && (path.split > 2 || (path.split == 1 && (!p.epi.out_f32 || a_mn || b_mn)))) ||
      (path.split != 1 && path.split != 2 && path.split != 4 && path.split != 8) ||
      (path.split > 1 && (path.split > stages || parts > kLinearMaxParts)))
    return cudaErrorInvalidValue;
  if (path.kind == LinearPath::kPair) {
    if (a_mn) return launch_pair<true, true, kNone>(tm_a, tm_b, p, s);
    if (b_mn) return launch_pair<false, true, kNone>(tm_a, tm_b, p, s);
    if (act == MOE_ACT_SILU) return launch_pair<false, false, MOE_ACT_SILU>(tm_a, tm_b, p, s);
    if (act == MOE_ACT_GELU) return launch_pair<false, false, MOE_ACT_GELU>(tm_a, tm_b, p, s);
    if (act == MOE_ACT_RELU) return launch_pair<false, false, MOE_ACT_RELU>(tm_a, tm_b, p, s);
    return launch_pair<false, false, kNone>(tm_a, tm_b, p, s);
  }
  if (path.kind == LinearPath::kSums) {
    const int n = path.split;
    // without a split only for fp32 results, which the gradients' products have not
    if (a_mn) return launch_sums<true, true, true, kNone>(tm_a, tm_b, p, n, s);
    if (b_mn) return launch_sums<false, true, true, kNone>(tm_a, tm_b, p, n, s);
    if (n > 1) return launch_sums<false, false, true, kNone>(tm_a, tm_b, p, n, s);
    if (act == MOE_ACT_SILU)
      return launch_sums<false, false, false, MOE_ACT_SILU>(tm_a, tm_b, p, n, s);
    if (act == MOE_ACT_GELU)
      return launch_sums<false, false, false, MOE_ACT_GELU>(tm_a, tm_b, p, n, s);
    if (act == MOE_ACT_RELU)
      return launch_sums<false, false, false, MOE_ACT_RELU>(tm_a, tm_b, p, n, s);
    return launch_sums<false, false, false, kNone>(tm_a, tm_b, p, n, s);
  }
  if (a_mn) return launch_tile<true, true>(tm_a, tm_b, p, path.split, s);
  if (b_mn) return launch_tile<false, true>(tm_a, tm_b, p, path.split, s);
  return launch_tile<false, false>(tm_a, tm_b, p, path.split, s);
}

bool linear_streams(int T, int N) { return T <= 16 || (T <= 32 && N <= 1024); }

cudaError_t launch_linear_stream(const LinearStreamArgs& a, int num_sms, cudaStream_t s) {
  cudaError_t e;
  if (a.epi.M == 1) e = launch_vector(a, num_sms, s);
  else if (a.epi.M <= 8) e = launch_stream<1>(a, num_sms, s);
  else if (a.epi.M <= 16) e = launch_stream<2>(a, num_sms, s);
  else e = launch_stream<4>(a, num_sms, s);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

int linear_dz_slices(long T, long N, int num_sms) {
  const long cols = ceil_div(N, 256);
  const long want = std::max<long>(1, 4L * num_sms / cols);
  return static_cast<int>(std::max<long>(1, std::min<long>(want, T / 32)));
}

cudaError_t launch_linear_dz(const LinearDzArgs& a, int slices, float* dbias, cudaStream_t s) {
  const dim3 grid(ceil_div(a.N, 256), slices);
  cudaError_t e;
  if (a.act == MOE_ACT_SILU) e = launch_dz<MOE_ACT_SILU>(a, grid, s);
  else if (a.act == MOE_ACT_GELU) e = launch_dz<MOE_ACT_GELU>(a, grid, s);
  else if (a.act == MOE_ACT_RELU) e = launch_dz<MOE_ACT_RELU>(a, grid, s);
  else e = launch_dz<MOE_ACT_NONE>(a, grid, s);
  count_launches(1);
  if (e != cudaSuccess) return e;
  if (dbias != nullptr && slices > 1) {  // one slice has written dbias itself
    e = launch_pdl(linear_colsum_kernel, dim3(ceil_div(a.N, 32)), dim3(256), 0, s,
                   static_cast<const float*>(a.partials), slices, a.N, dbias);
    count_launches(1);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
