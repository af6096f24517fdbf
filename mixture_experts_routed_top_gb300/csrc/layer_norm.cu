// Layer norm with the residual sum before it in one pass, and its gradient.
//
// Forward, for one token's stream x, block output y [H]:
//   r = x + y  (or x),  n = (r - mean) / sqrt(var + eps) * w + b
// r and n leave rounded once each; n is made from the unrounded r.  The variance is the
// mean of (r - mean)^2 over the row in registers, so a stream far from zero loses
// nothing, at the price of a second sum over the row.  The mean is the sum divided by H, not
// times a rounded 1 / H, which would leave a row of equal numbers 2^-24 of them.
//
// Backward, from dL/dr (dr) and dL/dn (dn), with the r that was stored; h = (r - mean) rs,
// rs = 1 / sqrt(var + eps), q = dn * w:
//   d  = dr + rs (q - mean(q) - h mean(q h))
//   dw = sum_t dn h,   db = sum_t dn
// The statistics are computed again from the row, which has to be read anyway: the sums of
// r and q in one reduction, those of (r - mean)^2 and q (r - mean) in the next.
//
// Both are bound by memory and use the ring of rows of the rms norms.
#include "norm_rows.cuh"

namespace moe {
namespace {

// Where a thread's 8 columns from `col` on end inside a row of any length: those past
// the end count as none.
__device__ __forceinline__ void mask_edge(int col, int H, F2 (&v)[4]) {
  if ((col & ~31) + 256 <= H) return;  // the same in a warp
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 q = parts(v[i]);
    v[i] = f2(col + 64 * i < H ? q.x : 0.f, col + 64 * i + 32 < H ? q.y : 0.f);
  }
}
template <bool EDGE>
__device__ __forceinline__ void bias8(const void* p, bool bf16, int col, int H, F2 (&v)[4]) {
  if (p != nullptr) {
    weights8<EDGE>(p, bf16, col, H, v);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = f2(0.f);
  }
}

constexpr int ln_blocks(int nv) { return nv == 1 ? 2 : 1; }  // on an SM

// 8192 x 7168 bf16 with the residual sum 77 us (470 MB, 6.1 TB/s, 91 % of a copy), bound by
// memory, with an fp32 stream 132 (705 MB, 5.3 TB/s); 8 tokens 3.2, three dependent trips (row,
// two sums).  EDGE: 8192 x 7167 bf16 127 us (3.7 TB/s), fp32 143 (4.9 TB/s), bound by issue.
template <typename RT, int NV, int STAGES, bool EDGE>
__global__ void __launch_bounds__(kRingThreads, ln_blocks(NV))
    layer_norm_ring_kernel(const LayerNormArgs a) {
  pdl_launch_dependents();
  extern __shared__ uint4 s_ring[];
  __shared__ __align__(16) F2 s_red[kRedPairs];
  constexpr bool R32 = sizeof(RT) == 4;
  constexpr int PR = R32 ? 2 : 1;  // pieces of a residual row
  const bool has_y = a.y != nullptr;
  const int nthr = blockDim.x * blockDim.y, tid = threadIdx.x + threadIdx.y * blockDim.x;
  const int pv = PR + (has_y ? 1 : 0);
  for (int i = tid; i < kRedPairs; i += nthr) s_red[i] = f2(0.f);
  __syncthreads();
  const int H = a.H;
  const RT* const res = static_cast<const RT*>(a.residual);
  const __nv_bfloat16* const ys = static_cast<const __nv_bfloat16*>(a.y);
  const int o_y = edge_bytes(blockDim.x, NV, sizeof(RT)),
            row_bytes = o_y + (has_y ? edge_bytes(blockDim.x, NV, 2) : 0);
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
    } else if (t < a.T) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (in(v)) {
          const Slots sl{s_ring + (st * NV + v) * pv * kRingThreads + tid};
          sl.fetch8(0, res + t * a.ld_res + col(v));
          if (has_y) sl.fetch8(PR, ys + t * a.ld_y + col(v));
        }
      }
    }
    cp_async_commit();
  };
  pdl_wait();
  long t = static_cast<long>(blockIdx.x) * blockDim.y + threadIdx.y;
#pragma unroll
  for (int st = 0; st < STAGES - 1; ++st) fetch(t + st * step, st);
  F2 w[NV][4], b[NV][4];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    weights8<EDGE>(a.weight, a.weight_bf16, col(v), H, w[v]);
    bias8<EDGE>(a.bias, a.weight_bf16, col(v), H, b[v]);
  }
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
    F2 r[NV][4], s = f2(0.f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const Slots sl{slot + v * pv * kRingThreads};
#pragma unroll
      for (int e = 0; e < 4; ++e) r[v][e] = f2(0.f);
      if (!(on && in(v))) continue;
      if (EDGE) edge_read(erow, R32, byte_in_16(res + t * a.ld_res), col(v), r[v]);
      else sl.read8(0, R32, r[v]);
      if (has_y) {
        F2 y[4];
        if (EDGE) edge_read(erow + o_y, false, byte_in_16(ys + t * a.ld_y), col(v), y);
        else sl.read8(PR, false, y);
#pragma unroll
        for (int e = 0; e < 4; ++e) r[v][e] = add2(r[v][e], y[e]);
        put8<EDGE>(static_cast<RT*>(a.residual_out) + t * H, col(v), H, r[v]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) s = add2(s, r[v][e]);
    }
    const F2 mean = f2(-ring_sum(sum2(s), s_red, turn) / static_cast<float>(H));  // negative: added
    s = f2(0.f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!in(v)) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) r[v][e] = add2(r[v][e], mean);
      if (EDGE) mask_edge(col(v), H, r[v]);
#pragma unroll
      for (int e = 0; e < 4; ++e) s = fma2(r[v][e], r[v][e], s);
    }
    const F2 rstd = f2(rsqrtf(ring_sum(sum2(s), s_red, turn) * inv_h + a.eps));
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!(on && in(v))) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) r[v][e] = fma2(mul2(r[v][e], rstd), w[v][e], b[v][e]);
      put8<EDGE>(static_cast<__nv_bfloat16*>(a.normed) + t * H, col(v), H, r[v]);
    }
  }
}

// The sums over tokens of a thread's columns stay in registers; a block leaves them as one
// partial row, and norm_partials_kernel adds those in block order.
// GR: a gradient of the stream beside the norm's, a constant of the code.
// 8192 x 7168 bf16 with it 94 us and 6 for the partial rows' sums (470 MB, 4.7 TB/s over
// both), held back by issue (0.54 instructions a cycle and scheduler, 27 a column and row
// over all) more than by memory; a row's first sums taken together with the last ones of
// the row before, a barrier a row less, changed nothing.  EDGE: 4099 x 2050 with an fp32
// stream 34 us with both results (134 MB, 4.0 TB/s).
template <typename RT, int NV, int STAGES, bool EDGE, bool GR>
__global__ void __launch_bounds__(kRingThreads, 1)
    layer_norm_backward_ring_kernel(const LayerNormBwdArgs a) {
  pdl_launch_dependents();
  extern __shared__ uint4 s_ring[];
  __shared__ __align__(16) F2 s_red[kRedPairs];
  constexpr bool R32 = sizeof(RT) == 4;
  constexpr int PR = R32 ? 2 : 1;
  constexpr bool has_gr = GR;
  // pieces: residual, grad_normed, grad_residual
  constexpr int pv = PR + 1 + (has_gr ? PR : 0);
  const int nthr = blockDim.x * blockDim.y, tid = threadIdx.x + threadIdx.y * blockDim.x;
  for (int i = tid; i < kRedPairs; i += nthr) s_red[i] = f2(0.f);
  __syncthreads();
  const int H = a.H;
  const RT* const res = static_cast<const RT*>(a.residual);
  const RT* const grs = static_cast<const RT*>(a.grad_res);
  const __nv_bfloat16* const gns = static_cast<const __nv_bfloat16*>(a.grad_normed);
  const int rowR = edge_bytes(blockDim.x, NV, sizeof(RT));
  const int o_gn = rowR, o_gr = o_gn + edge_bytes(blockDim.x, NV, 2), row_bytes = o_gr + (has_gr ? rowR : 0);
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
      edge_fetch(to + o_gn, gns + t * a.ld_gn, H);
      if (has_gr) edge_fetch(to + o_gr, grs + t * a.ld_gres, H);
    } else if (t < a.T) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (in(v)) {
          const Slots sl{s_ring + (st * NV + v) * pv * kRingThreads + tid};
          sl.fetch8(0, res + t * a.ld_res + col(v));
          sl.fetch8(PR, gns + t * a.ld_gn + col(v));
          if (has_gr) sl.fetch8(PR + 1, grs + t * a.ld_gres + col(v));
        }
      }
    }
    cp_async_commit();
  };
  pdl_wait();
  long t = static_cast<long>(blockIdx.x) * blockDim.y + threadIdx.y;
#pragma unroll
  for (int st = 0; st < STAGES - 1; ++st) fetch(t + st * step, st);
  F2 w[NV][4], acc_w[NV][4], acc_b[NV][4];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    weights8<EDGE>(a.weight, a.weight_bf16, col(v), H, w[v]);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc_w[v][e] = acc_b[v][e] = f2(0.f);
  }
  int st = 0, turn = 0;
  for (long base = static_cast<long>(blockIdx.x) * blockDim.y; base < a.T; base += step, t += step) {
    if (EDGE) {
      cp_async_wait<STAGES - 2>();
      __syncthreads();
    }
    fetch(t + (STAGES - 1) * step, st == 0 ? STAGES - 1 : st - 1);
    if (!EDGE) cp_async_wait<STAGES - 1>();
    const bool on = t < a.T;
    uint4* const slot = s_ring + st * NV * pv * kRingThreads + tid;
    const char* const erow = edge_row(st);
    if (++st == STAGES) st = 0;
    F2 r[NV][4], g[NV][4], s0 = f2(0.f), s1 = f2(0.f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const Slots sl{slot + v * pv * kRingThreads};
#pragma unroll
      for (int e = 0; e < 4; ++e) r[v][e] = g[v][e] = f2(0.f);
      if (!(on && in(v))) continue;
      if (EDGE) {
        edge_read(erow, R32, byte_in_16(res + t * a.ld_res), col(v), r[v]);
        edge_read(erow + o_gn, false, byte_in_16(gns + t * a.ld_gn), col(v), g[v]);
      } else {
        sl.read8(0, R32, r[v]);
        sl.read8(PR, false, g[v]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s0 = add2(s0, r[v][e]);
        s1 = fma2(g[v][e], w[v][e], s1);
      }
    }
    float2 sum = parts(ring_sums2(sum2(s0), sum2(s1), s_red, turn));
    const F2 mean = f2(-sum.x / static_cast<float>(H));  // negative: added
    const float mean_q = sum.y * inv_h;
    s0 = s1 = f2(0.f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!in(v)) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) r[v][e] = add2(r[v][e], mean);
      if (EDGE) mask_edge(col(v), H, r[v]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s0 = fma2(r[v][e], r[v][e], s0);
        s1 = fma2(mul2(g[v][e], w[v][e]), r[v][e], s1);
      }
    }
    sum = parts(ring_sums2(sum2(s0), sum2(s1), s_red, turn));
    const float rstd = rsqrtf(sum.x * inv_h + a.eps);
    const F2 rs = f2(rstd), shift = f2(-rstd * mean_q), corr = f2(-sum.y * inv_h * rstd * rstd);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!(on && in(v))) continue;
      F2 d[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) d[e] = f2(0.f);
      if (has_gr && EDGE) edge_read(erow + o_gr, R32, byte_in_16(grs + t * a.ld_gres), col(v), d);
      else if (has_gr) Slots{slot + v * pv * kRingThreads}.read8(PR + 1, R32, d);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const F2 h = mul2(r[v][e], rs);
        acc_w[v][e] = fma2(g[v][e], h, acc_w[v][e]);
        acc_b[v][e] = add2(acc_b[v][e], g[v][e]);
        const F2 q = fma2(mul2(g[v][e], w[v][e]), rs, shift);
        d[e] = add2(d[e], fma2(h, corr, q));
      }
      put8<EDGE>(static_cast<RT*>(a.d_res) + t * H, col(v), H, d);
      if (a.d_y != nullptr) put8<EDGE>(static_cast<__nv_bfloat16*>(a.d_y) + t * H, col(v), H, d);
    }
  }
  if (a.n_part == 0) return;
  // the block's rows side by side added in order, through the ring's memory
  cp_async_wait<0>();
  float* sum = reinterpret_cast<float*>(s_ring);  // [threads in y][n_part][H]
  __syncthreads();
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (!in(v)) continue;
    float* to = sum + static_cast<long>(threadIdx.y) * a.n_part * H;
    if (a.d_w != nullptr) {
      put8<EDGE>(to, col(v), H, acc_w[v]);
      to += H;
    }
    if (a.d_b != nullptr) put8<EDGE>(to, col(v), H, acc_b[v]);
  }
  __syncthreads();
  float* part = a.partials + static_cast<long>(blockIdx.x) * a.n_part * H;
  const int total = a.n_part * H;
  for (int i = tid; i < total; i += nthr) {
    float v = sum[i];
    for (int y = 1; y < blockDim.y; ++y) v += sum[y * total + i];
    part[i] = v;
  }
}

// Rows above 8192 columns: one per block, held in registers.  Forward 8192 x 12288 bf16 151 us
// (805 MB, 5.3 TB/s), 8192 x 16384 191 (5.6 TB/s); single columns where rows are not whole
// vectors: 8192 x 12287 353 (2.3 TB/s).
template <typename RT, bool VEC>
__global__ void __launch_bounds__(1024) layer_norm_kernel(const LayerNormArgs a) {
  pdl_launch_dependents();
  constexpr int NV = 2;
  __shared__ float s_red[kMaxRed];
  const Cols<VEC, NV> c{static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x), a.H};
  const int warps = blockDim.x >> 5;
  const float inv_h = 1.f / static_cast<float>(a.H);
  pdl_wait();
  const long t = blockIdx.x;
  float r[NV][8], sum[1] = {0.f};
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    c.load(static_cast<const RT*>(a.residual) + t * a.ld_res, v, r[v], 0.f);
    if (a.y != nullptr) {
      float y[8];
      c.load(static_cast<const __nv_bfloat16*>(a.y) + t * a.ld_y, v, y, 0.f);
#pragma unroll
      for (int e = 0; e < 8; ++e) r[v][e] += y[e];
      c.store(static_cast<RT*>(a.residual_out) + t * a.H, v, r[v]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[0] += r[v][e];
  }
  row_sums<1>(sum, s_red, warps);
  const float mean = sum[0] / static_cast<float>(a.H);
  sum[0] = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      r[v][e] = c.col(v, e) < a.H ? r[v][e] - mean : 0.f;
      sum[0] += r[v][e] * r[v][e];
    }
  row_sums<1>(sum, s_red, warps);
  const float rstd = rsqrtf(sum[0] * inv_h + a.eps);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    float m[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[v][e] *= rstd;
    if (a.weight != nullptr) {
      c.load_any(a.weight, a.weight_bf16, v, m, 0.f);
#pragma unroll
      for (int e = 0; e < 8; ++e) r[v][e] *= m[e];
    }
    if (a.bias != nullptr) {
      c.load_any(a.bias, a.weight_bf16, v, m, 0.f);
#pragma unroll
      for (int e = 0; e < 8; ++e) r[v][e] += m[e];
    }
    c.store(static_cast<__nv_bfloat16*>(a.normed) + t * a.H, v, r[v]);
  }
}

// The sums over tokens and the values of a column take more registers than its threads have: 328
// to 432 bytes of spill stores a thread and 472 to 648 of loads, in the loop over rows, and one row
// in flight an SM (19 % of the warps).  That is what bounds it, at a quarter of the issue slots:
// 8192 x 12288 bf16 600 us (1.3 TB/s), 8192 x 16384 630, 8192 x 12287 1807.
template <typename RT, bool VEC>
__global__ void __launch_bounds__(512) layer_norm_backward_kernel(const LayerNormBwdArgs a) {
  pdl_launch_dependents();
  constexpr int NV = 4;
  __shared__ float s_red[kMaxRed];
  const Cols<VEC, NV> c{static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x), a.H};
  const int warps = blockDim.x >> 5;
  const float inv_h = 1.f / static_cast<float>(a.H);
  float acc_w[NV][8] = {}, acc_b[NV][8] = {};
  pdl_wait();
  for (long t = blockIdx.x; t < a.T; t += gridDim.x) {
    const RT* const res = static_cast<const RT*>(a.residual) + t * a.ld_res;
    const __nv_bfloat16* const gn = static_cast<const __nv_bfloat16*>(a.grad_normed) + t * a.ld_gn;
    float r[NV][8], g[NV][8], sum[2] = {0.f, 0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float m[8];
      c.load(res, v, r[v], 0.f);
      c.load(gn, v, g[v], 0.f);
      if (a.weight != nullptr) c.load_any(a.weight, a.weight_bf16, v, m, 0.f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum[0] += r[v][e];
        sum[1] += g[v][e] * (a.weight != nullptr ? m[e] : 1.f);
      }
    }
    row_sums<2>(sum, s_red, warps);
    const float mean = sum[0] / static_cast<float>(a.H), mean_q = sum[1] * inv_h;
    sum[0] = sum[1] = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float m[8];
      if (a.weight != nullptr) c.load_any(a.weight, a.weight_bf16, v, m, 0.f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        r[v][e] = c.col(v, e) < a.H ? r[v][e] - mean : 0.f;
        sum[0] += r[v][e] * r[v][e];
        sum[1] += g[v][e] * (a.weight != nullptr ? m[e] : 1.f) * r[v][e];
      }
    }
    row_sums<2>(sum, s_red, warps);
    const float rstd = rsqrtf(sum[0] * inv_h + a.eps);
    const float shift = rstd * mean_q, corr = sum[1] * inv_h * rstd * rstd;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float m[8], d[8];
      if (a.weight != nullptr) c.load_any(a.weight, a.weight_bf16, v, m, 0.f);
      if (a.grad_res != nullptr) {
        c.load(static_cast<const RT*>(a.grad_res) + t * a.ld_gres, v, d, 0.f);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float h = r[v][e] * rstd;
        acc_w[v][e] += g[v][e] * h;
        acc_b[v][e] += g[v][e];
        d[e] += g[v][e] * (a.weight != nullptr ? m[e] : 1.f) * rstd - shift - h * corr;
      }
      c.store(static_cast<RT*>(a.d_res) + t * a.H, v, d);
      if (a.d_y != nullptr) c.store(static_cast<__nv_bfloat16*>(a.d_y) + t * a.H, v, d);
    }
  }
  float* part = a.partials + static_cast<long>(blockIdx.x) * a.n_part * a.H;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (a.d_w != nullptr) c.store(part, v, acc_w[v]);
    if (a.d_b != nullptr) c.store(part + (a.d_w != nullptr ? a.H : 0), v, acc_b[v]);
  }
}

template <typename RT, int NV, int STAGES, bool EDGE>
cudaError_t fwd_ring(const LayerNormArgs& a, dim3 block, size_t smem, int grid, cudaStream_t s) {
  static std::atomic<int> ready[64] = {};
  const cudaError_t e = ring_ready(layer_norm_ring_kernel<RT, NV, STAGES, EDGE>, ready);
  if (e != cudaSuccess) return e;
  return launch_pdl(layer_norm_ring_kernel<RT, NV, STAGES, EDGE>, dim3(grid), block, smem, s, a);
}
template <typename RT, int NV, int STAGES, bool EDGE, bool GR>
cudaError_t bwd_ring(const LayerNormBwdArgs& a, dim3 block, size_t smem, int grid, cudaStream_t s) {
  static std::atomic<int> ready[64] = {};
  const cudaError_t e = ring_ready(layer_norm_backward_ring_kernel<RT, NV, STAGES, EDGE, GR>, ready);
  if (e != cudaSuccess) return e;
  return launch_pdl(layer_norm_backward_ring_kernel<RT, NV, STAGES, EDGE, GR>, dim3(grid), block, smem, s, a);
}

template <typename RT, int NV, bool VEC>
cudaError_t fwd_nv(const LayerNormArgs& a, int num_sms, cudaStream_t s) {
  constexpr int PER_SM = ln_blocks(NV), PR = static_cast<int>(sizeof(RT) / 2);
  const dim3 block = ring_block(a.T, a.H, NV, PER_SM * num_sms);
  const int grid = std::min(PER_SM * num_sms, ceil_div(a.T, block.y));
  if (!VEC) {
    const size_t stage = edge_stage_bytes(PR == 2, (PR == 1) + (a.y != nullptr), NV, block);
    return 4 * stage * PER_SM <= kRingBytes ? fwd_ring<RT, NV, 4, true>(a, block, 4 * stage, grid, s)
                                            : fwd_ring<RT, NV, 2, true>(a, block, 2 * stage, grid, s);
  }
  constexpr int ST = NV == 1 ? 3 : PR == 1 ? 5 : 4;  // as the rms norms
  static_assert(ST * stage_bytes(PR + 1, NV) * PER_SM <= kRingBytes, "a ring");
  return fwd_ring<RT, NV, ST, false>(a, block, ST * stage_bytes(PR + (a.y != nullptr), NV), grid, s);
}
template <typename RT, int NV, bool VEC, bool GR>
cudaError_t bwd_nv(const LayerNormBwdArgs& a, int num_sms, int* blocks, cudaStream_t s) {
  constexpr int PR = static_cast<int>(sizeof(RT) / 2), ROWS = 1 + GR;
  const dim3 block = ring_block(a.T, a.H, NV, num_sms);
  const size_t stage = VEC ? stage_bytes(PR * ROWS + 1, NV)
                           : edge_stage_bytes(PR == 2 ? ROWS : 0, (PR == 1 ? ROWS : 0) + 1, NV, block);
  const size_t sums = static_cast<size_t>(block.y) * a.n_part * a.H * 4;  // <= 64 KB
  const int grid = *blocks = std::min(std::min(num_sms, kNormBwdBlocks), ceil_div(a.T, block.y));
  if (VEC) {  // whole stages of 512 threads, as many as fit: four 99 us at 8192 x 7168, three 102
    constexpr size_t kStage = stage_bytes(PR * ROWS + 1, NV);
    constexpr int ST = 4 * kStage <= kRingBytes ? 4 : 3 * kStage <= kRingBytes ? 3 : 2;
    static_assert(2 * kStage <= kRingBytes, "a ring");
    return bwd_ring<RT, NV, ST, false, GR>(a, block, std::max(ST * kStage, sums), grid, s);
  }
  return 3 * stage <= kRingBytes
             ? bwd_ring<RT, NV, 3, true, GR>(a, block, std::max(3 * stage, sums), grid, s)
             : bwd_ring<RT, NV, 2, true, GR>(a, block, std::max(2 * stage, sums), grid, s);
}

template <typename RT, bool VEC>
cudaError_t fwd(const LayerNormArgs& a, int num_sms, cudaStream_t s) {
  if (a.H <= 8192)
    return a.H <= 2048 ? fwd_nv<RT, 1, VEC>(a, num_sms, s) : fwd_nv<RT, 2, VEC>(a, num_sms, s);
  const dim3 block(ceil_div(ceil_div(a.H, 8), 64) * 32);
  return launch_pdl(layer_norm_kernel<RT, VEC>, dim3(a.T), block, 0, s, a);
}
template <typename RT, bool VEC>
cudaError_t bwd(const LayerNormBwdArgs& a, int num_sms, int* blocks, cudaStream_t s) {
  if (a.H <= 8192)
    return a.grad_res != nullptr
               ? (a.H <= 2048 ? bwd_nv<RT, 1, VEC, true>(a, num_sms, blocks, s)
                              : bwd_nv<RT, 2, VEC, true>(a, num_sms, blocks, s))
               : (a.H <= 2048 ? bwd_nv<RT, 1, VEC, false>(a, num_sms, blocks, s)
                              : bwd_nv<RT, 2, VEC, false>(a, num_sms, blocks, s));
  *blocks = static_cast<int>(std::min<long>(std::min(num_sms, kNormBwdBlocks), a.T));
  const dim3 block(ceil_div(ceil_div(ceil_div(a.H, 8), 4), 32) * 32);
  return launch_pdl(layer_norm_backward_kernel<RT, VEC>, dim3(*blocks), block, 0, s, a);
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormArgs& a, bool res_bf16, bool vec, int num_sms,
                              cudaStream_t s) {
  cudaError_t e;
  if (res_bf16)
    e = vec ? fwd<__nv_bfloat16, true>(a, num_sms, s) : fwd<__nv_bfloat16, false>(a, num_sms, s);
  else
    e = vec ? fwd<float, true>(a, num_sms, s) : fwd<float, false>(a, num_sms, s);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_layer_norm_backward(const LayerNormBwdArgs& a, bool res_bf16, bool vec,
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
    e = launch_pdl(norm_partials_kernel, dim3(ceil_div(a.H, 32), a.n_part), dim3(256), 0, s,
                   static_cast<const float*>(a.partials), blocks, a.n_part, a.H,
                   a.d_w != nullptr ? a.d_w : a.d_b, a.d_b, static_cast<float*>(nullptr));
    count_launches(1);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
