// Routing by scores: softmax or sigmoid scores of the router's logits, a
// balance bias that moves the choice but not the weights, expert groups of
// which only the best are eligible, top-k, weights renormalised and scaled;
// and the gradient of the weights with respect to the logits.
//
// Forward, for one token with logits l_e:
//   s_e = 1 / (1 + exp(-l_e))               sigmoid scores, or
//   s_e = exp(l_e - max l) / S              softmax scores; S sums the E terms
//         by halves (term i + term i + P/2, and so on, P = E rounded up to a
//         power of two), a fixed tree, so the scores do not depend on how
//         the terms are spread over threads
//   c_e = s_e + b_e in 32 bits; -inf where the expert is masked (l_e or b_e
//         -inf, or NaN)
//   a group's score is the sum of its one or two largest live c_e; the
//   topk_group best groups (ties: lower group) keep their c, the others' is
//   -inf; the k largest c are taken, ties to the lower expert index
//   w_j = s_j (0 where c_j = -inf), divided by their sum if renormalised
//         (1/k each where that sum is 0), times scale
// The scores use expf and IEEE division, not the fast forms: the choice
// compares them bit by bit, so that a tie and a near-tie come out the same
// in any implementation of the formulas in 32 bits.
#include <math.h>

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kWarps = 8;  // tokens (warps) per block

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float v, float* o) { *o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16* o) { *o = __float2bfloat16_rn(v); }

// Order-preserving map of floats (no NaN, no -0) to unsigned; -inf maps to
// 0x007fffff, and 0 is below every float.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
constexpr uint32_t kKeyNegInf = 0x007fffffu;
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ uint32_t warp_max_u32(uint32_t v) {
  return __reduce_max_sync(0xffffffffu, v);
}

// Where a lane's NPL values lie in a row: runs of C = min(NPL, 4) neighbours,
// the lanes' runs next to each other, so that a row is read in whole lines
// (16 bytes of fp32 or 8 of bf16 per lane).  Blocks of NPL neighbours per
// lane instead ran 1024 experts 5 times slower: every load touched 32 lines.
template <int NPL>
struct Lay {
  static constexpr int C = NPL < 4 ? NPL : 4;
  static __device__ __forceinline__ int expert(int lane, int i) {
    return (i / C) * (32 * C) + lane * C + i % C;
  }
};

template <typename T, int NPL>
__device__ __forceinline__ void load_row(const T* __restrict__ row, int E, int lane, bool vec,
                                         float (&v)[NPL]) {
  if (NPL >= 4 && vec) {  // E % 4 == 0: a run is inside the row or outside it
#pragma unroll
    for (int i = 0; i < NPL; i += 4) {
      const int e = Lay<NPL>::expert(lane, i);
      T t[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) t[j] = T(0.f);
      if (e < E) {
        if (sizeof(T) == 4) *reinterpret_cast<uint4*>(t) = __ldg(reinterpret_cast<const uint4*>(row + e));
        else *reinterpret_cast<uint2*>(t) = __ldg(reinterpret_cast<const uint2*>(row + e));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i + j] = to_f(t[j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = Lay<NPL>::expert(lane, i);
      v[i] = e < E ? to_f(row[e]) : 0.f;
    }
  }
}

// Softmax numerators of a row (NaN and -inf count as masked: 0; the largest
// logit gives 1 even when it is +inf) and their sum by halves.
template <int NPL>
__device__ __forceinline__ float softmax_terms(float (&v)[NPL], int E, int lane) {
  constexpr int C = Lay<NPL>::C;
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NPL; ++i)
    if (Lay<NPL>::expert(lane, i) < E) m = fmaxf(m, v[i]);  // fmaxf drops NaN
  m = key_value(warp_max_u32(order_key(m + 0.f)));
  float t[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const bool live = Lay<NPL>::expert(lane, i) < E && v[i] > -INFINITY;
    v[i] = live ? expf(v[i] == m ? 0.f : __fsub_rn(v[i], m)) : 0.f;
    t[i] = v[i];
  }
  // halves: the highest bits of an expert's index are its run's, then the
  // lane's, then its place in the run
#pragma unroll
  for (int n = NPL / 2; n >= C; n /= 2)
#pragma unroll
    for (int i = 0; i < n; ++i) t[i] = __fadd_rn(t[i], t[i + n]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int i = 0; i < C; ++i) t[i] = __fadd_rn(t[i], __shfl_xor_sync(0xffffffffu, t[i], off));
#pragma unroll
  for (int n = C / 2; n > 0; n /= 2)
#pragma unroll
    for (int i = 0; i < n; ++i) t[i] = __fadd_rn(t[i], t[i + n]);
  return t[0];
}

// __frcp_rn is the correctly rounded 1 / v, the same bits as IEEE division.
__device__ __forceinline__ float sigmoid_score(float x) {
  return __frcp_rn(__fadd_rn(1.f, expf(-x)));
}

// The k largest of the warp's keys in (key descending, expert ascending)
// order, written to s_idx / s_val; value 0 where the key is that of -inf.
//
// Up to kRankK of them by rank: the k-th largest of the 32 lane maxima is a
// bound that at least k keys reach and few others do; those are gathered (at
// most 32) as one 64-bit number each, key above, complement of the expert
// below, and each lane counts the numbers above its own.  At 256 experts and
// k = 8 about 12 are gathered.  The other cases, more than kRankK or more
// than 32 keys at the bound (ties, masked experts), take k rounds of a
// warp-wide maximum that remove one key each, 2 us more at 8192 x 256.
constexpr int kRankK = 16;
struct __align__(16) Cand {
  unsigned long long num[32];
  float val[32];
};
template <int NPL>
__device__ __forceinline__ void select_top(uint32_t (&key)[NPL], const float (&s)[NPL], int k,
                                           int lane, Cand& c, int* s_idx, float* s_val) {
  if (k <= kRankK) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < NPL; ++i) best = max(best, key[i]);
    uint32_t bound = 0;
    for (int taken = 0; taken < k;) {  // equal maxima leave together
      bound = warp_max_u32(best);
      const bool mine = best == bound;
      taken += __popc(__ballot_sync(0xffffffffu, mine));
      if (mine) best = 0u;
      if (bound == 0u) break;  // fewer lanes than k hold an expert
    }
    c.num[lane] = 0ull;
    __syncwarp();
    int n = 0;
    const uint32_t below = (1u << lane) - 1u;
    if (bound != 0u) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const bool in = key[i] >= bound;
        const uint32_t b = __ballot_sync(0xffffffffu, in);
        const int at = n + __popc(b & below);
        if (in && at < 32) {
          c.num[at] = static_cast<unsigned long long>(key[i]) << 32 |
                      static_cast<uint32_t>(~Lay<NPL>::expert(lane, i));
          c.val[at] = s[i];
        }
        n += __popc(b);
      }
    }
    __syncwarp();
    if (bound != 0u && n <= 32) {
      const unsigned long long mine = c.num[lane];
      int rank = 0;
      for (int j = 0; j < n; j += 2) {  // 0 past the last
        const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(&c.num[j]);
        rank += o.x > mine;
        rank += o.y > mine;
      }
      if (lane < n && rank < k) {
        s_idx[rank] = static_cast<int>(~static_cast<uint32_t>(mine));
        s_val[rank] = static_cast<uint32_t>(mine >> 32) == kKeyNegInf ? 0.f : c.val[lane];
      }
      __syncwarp();
      return;
    }
  }
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) best = max(best, key[i]);
    const uint32_t top = warp_max_u32(best);
    int at = NPL;  // this lane's first value that is the maximum
#pragma unroll
    for (int i = NPL - 1; i >= 0; --i)
      if (key[i] == top) at = i;
    const uint32_t mine = at < NPL ? Lay<NPL>::expert(lane, at) : 0xffffffffu;
    if (__reduce_min_sync(0xffffffffu, mine) == mine && at < NPL) {
      float sv = 0.f;
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (i == at) {
          sv = s[i];
          key[i] = 0u;
        }
      s_idx[j] = static_cast<int>(mine);
      s_val[j] = top == kKeyNegInf ? 0.f : sv;
    }
  }
  __syncwarp();
}

// Shared rows have a gap after every 32 experts, so that groups of 32 do not
// all begin in one bank.
__device__ __forceinline__ int padded(int e) { return e + (e >> 5); }

// One warp per token, so that no step needs a barrier.  Bound by issue, not by
// its bytes: 8192 x 256 sigmoid scores, 4 of 8 groups, k = 8: 10.7 us, two thirds
// of the issue slots taken, where its 8.9 MB need 1.3; 4099 x 60 softmax 4.0, one
// token 3.9 (the depth of its dependent steps).  Registers are held to what
// leaves 5 blocks on an SM; 7 spill.
template <typename T, int NPL>
__global__ void __launch_bounds__(kWarps * 32, NPL <= 8 ? 5 : NPL == 16 ? 4 : 2)
    route_scored_kernel(const RouteScoredArgs a) {
  pdl_launch_dependents();
  __shared__ int s_idx[kWarps][kMaxK];
  __shared__ float s_val[kWarps][kMaxK];
  __shared__ Cand s_cand[kWarps];
  extern __shared__ float s_row[];  // [kWarps][33 * NPL], with groups
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long t = static_cast<long>(blockIdx.x) * kWarps + warp;
  pdl_wait();
  if (t >= a.T) return;
  const int E = a.E;
  auto expert = [&](int i) { return Lay<NPL>::expert(lane, i); };
  float s[NPL], b[NPL];
  load_row<T, NPL>(static_cast<const T*>(a.logits) + t * a.ld, E, lane, a.vec, s);
#pragma unroll
  for (int i = 0; i < NPL; ++i) b[i] = 0.f;
  if (a.bias != nullptr) load_row<float, NPL>(a.bias, E, lane, E % 4 == 0, b);
  uint32_t dead = 0;  // bit i: the lane's i-th expert is masked (or there is none)
#pragma unroll
  for (int i = 0; i < NPL; ++i)
    if (expert(i) >= E || !(s[i] > -INFINITY)) dead |= 1u << i;
  if (a.softmax) {
    const float sum = softmax_terms<NPL>(s, E, lane);
#pragma unroll
    for (int i = 0; i < NPL; ++i) s[i] = (dead >> i) & 1u ? 0.f : __fdiv_rn(s[i], sum);
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) s[i] = (dead >> i) & 1u ? 0.f : sigmoid_score(s[i]);
  }
  uint32_t key[NPL];  // 0: no expert, or taken already
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const float c = __fadd_rn(s[i], b[i]);
    const bool live = !((dead >> i) & 1u) && c > -INFINITY;
    key[i] = expert(i) < E ? (live ? order_key(c + 0.f) : kKeyNegInf) : 0u;
  }
  if (a.n_group > 1) {
    // 32 / n_group lanes (a power of two) per group look through its keys in
    // shared memory and join their two largest by shuffles
    const int gs = E / a.n_group;
    const int lpg = 1 << (31 - __clz(32 / a.n_group));
    constexpr int C = Lay<NPL>::C;
    uint32_t* row = reinterpret_cast<uint32_t*>(s_row) + warp * 33 * NPL;
    const int at0 = lane * C + (lane * C >> 5);  // padded(expert(i)), i's part a constant
#pragma unroll
    for (int i = 0; i < NPL; ++i) row[at0 + (i / C) * (33 * C) + i % C] = key[i];
    __syncwarp();
    const int mine = lane / lpg;  // this lane's group
    uint32_t t1 = kKeyNegInf, t2 = kKeyNegInf;
    if (mine < a.n_group) {
#pragma unroll 4
      for (int j = lane % lpg; j < gs; j += lpg) {
        const uint32_t kx = row[padded(mine * gs + j)];
        t2 = max(t2, min(t1, kx));
        t1 = max(t1, kx);
      }
    }
    for (int off = 1; off < lpg; off <<= 1) {
      const uint32_t o1 = __shfl_xor_sync(0xffffffffu, t1, off);
      const uint32_t o2 = __shfl_xor_sync(0xffffffffu, t2, off);
      t2 = max(max(t2, o2), min(t1, o1));
      t1 = max(t1, o1);
    }
    // a masked second expert adds nothing
    float g = key_value(t1);
    if (a.group_top == 2 && t2 > kKeyNegInf) g = __fadd_rn(g, key_value(t2));
    // the topk_group largest, equal ones in group order; bit lpg * q: group q is kept
    uint32_t gkey = mine < a.n_group && lane % lpg == 0 ? order_key(g + 0.f) : 0u, kept = 0;
    for (int q = 0; q < a.topk_group; ++q) {
      const uint32_t top = warp_max_u32(gkey);
      const int first = __ffs(__ballot_sync(0xffffffffu, gkey == top)) - 1;
      kept |= 1u << first;
      if (lane == first) gkey = 0u;
    }
    // e / gs = e * ceil(2^20 / gs) >> 20 for e, gs <= 1024
    const uint32_t magic = ((1u << 20) + gs - 1) / gs;
    auto eligible = [&](int e) {
      const uint32_t q = (static_cast<uint32_t>(e) * magic) >> 20;
      return (kept >> min(q * lpg, 31u)) & 1u;
    };
    if (gs % C == 0) {  // a run lies in one group
#pragma unroll
      for (int i = 0; i < NPL; i += C) {
        const uint32_t cap = eligible(expert(i)) ? 0xffffffffu : kKeyNegInf;
#pragma unroll
        for (int c = 0; c < C; ++c) key[i + c] = min(key[i + c], cap);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (!eligible(expert(i))) key[i] = min(key[i], kKeyNegInf);
    }
  }
  select_top<NPL>(key, s, a.k, lane, s_cand[warp], s_idx[warp], s_val[warp]);
  const bool has = lane < a.k;
  float w = has ? s_val[warp][lane] : 0.f;
  if (a.renorm) {
    float sum = w;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    w = sum > 0.f ? w / sum : 1.f / static_cast<float>(a.k);
  }
  if (has) {
    a.idx[t * a.k + lane] = s_idx[warp][lane];
    a.w[t * a.k + lane] = w * a.scale;
  }
}

// Gradient.  With g_j = scale * dL/dw_j, r_j = s_j / sum of the chosen s,
// D = sum_j g_j r_j:
//   renormalised, sigmoid   dl_j = (g_j - D) r_j (1 - s_j)
//   renormalised, softmax   dl_j = (g_j - D) r_j    (the softmax's own
//                           denominator cancels: only the chosen logits count)
//   as they are, sigmoid    dl_j = g_j s_j (1 - s_j)
//   as they are, softmax    dl_e = s_e ([e chosen] g_e - sum_j g_j s_j), every e
// A slot whose weight is 0, or whose expert is masked, has no gradient.
// One warp per token; lane j holds slot j.  Three of the four forms read
// only the chosen logits and write one row, whose zeros and values are put
// together in shared memory so that the row leaves in 16-byte vectors.
// 8192 x 256 fp32 softmax as they are, the form with the most to read: 6.3 us
// (17.6 MB, 2.8 TB/s): the launch, then the choice and the row in turn.
template <typename T, int NPL>
__global__ void __launch_bounds__(kWarps * 32)
    route_scored_backward_kernel(const RouteScoredBwdArgs a) {
  pdl_launch_dependents();
  extern __shared__ float s_row[];  // [kWarps][32 * NPL]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long t = static_cast<long>(blockIdx.x) * kWarps + warp;
  pdl_wait();
  if (t >= a.T) return;
  const int E = a.E, k = a.k;
  const T* lrow = static_cast<const T*>(a.logits) + t * a.ld;
  float* row = s_row + warp * 32 * NPL;
  int e = -1;
  float g = 0.f, x = -INFINITY;
  if (lane < k) {
    e = __ldg(a.idx + t * k + lane);
    const float w = __ldg(a.w + t * k + lane);
    g = a.scale * __ldg(a.grad_w + t * k + lane);
    if (e < 0 || e >= E || w == 0.f) e = -1;
    if (e >= 0) x = to_f(lrow[e]);
    if (e >= 0 && a.bias != nullptr && !(__ldg(a.bias + e) > -INFINITY)) e = -1;
    if (!(x > -INFINITY)) e = -1;
    if (e < 0) g = 0.f;
  }
  const bool has = e >= 0;
  auto sum32 = [](float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
  };
  const bool dense = a.softmax && !a.renorm;
  float d = 0.f;
  if (!dense) {
    float s = 0.f, rest = 1.f;  // score (softmax: up to the common factor), 1 - s
    if (a.softmax) {
      float m = has ? x : -INFINITY;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      s = has ? expf(x == m ? 0.f : x - m) : 0.f;
    } else if (has) {
      s = sigmoid_score(x);
      rest = sigmoid_score(-x);  // 1 - s without its cancellation
    }
    if (a.renorm) {
      const float total = sum32(s);
      const float r = total > 0.f ? s / total : 0.f;
      d = (g - sum32(g * r)) * r * rest;
    } else {
      d = g * s * rest;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) row[i * 32 + lane] = 0.f;
    __syncwarp();
    if (has) row[e] = d;
    __syncwarp();
  } else {
    float p[NPL];
    load_row<T, NPL>(lrow, E, lane, a.vec, p);
    const float sum = softmax_terms<NPL>(p, E, lane);
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      p[i] = p[i] > 0.f ? p[i] / sum : 0.f;
      row[Lay<NPL>::expert(lane, i)] = p[i];
    }
    __syncwarp();
    const float ps = has ? row[e] : 0.f;
    const float dot = sum32(g * ps);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < NPL; ++i) row[Lay<NPL>::expert(lane, i)] = -p[i] * dot;
    __syncwarp();
    if (has) row[e] = ps * (g - dot);
    __syncwarp();
  }
  T* out = static_cast<T*>(a.grad_logits) + t * a.ldo;
  constexpr int PV = 16 / sizeof(T);
  if (a.vec_out) {
    for (int c = lane * PV; c < E; c += 32 * PV) {
      T o[PV];
#pragma unroll
      for (int j = 0; j < PV; ++j) from_f(row[c + j], &o[j]);
      *reinterpret_cast<uint4*>(out + c) = *reinterpret_cast<const uint4*>(o);
    }
  } else {
    for (int c = lane; c < E; c += 32) from_f(row[c], out + c);
  }
}

template <typename T, int NPL>
cudaError_t fwd(const RouteScoredArgs& a, cudaStream_t s) {
  const size_t smem = a.n_group > 1 ? sizeof(float) * kWarps * 33 * NPL : 0;
  return launch_pdl(route_scored_kernel<T, NPL>, dim3(ceil_div(a.T, kWarps)), dim3(kWarps * 32),
                    smem, s, a);
}
template <typename T, int NPL>
cudaError_t bwd(const RouteScoredBwdArgs& a, cudaStream_t s) {
  return launch_pdl(route_scored_backward_kernel<T, NPL>, dim3(ceil_div(a.T, kWarps)),
                    dim3(kWarps * 32), sizeof(float) * kWarps * 32 * NPL, s, a);
}

template <typename T>
cudaError_t fwd_t(const RouteScoredArgs& a, cudaStream_t s) {
  const int npl = ceil_div(a.E, 32);
  if (npl <= 1) return fwd<T, 1>(a, s);
  if (npl <= 2) return fwd<T, 2>(a, s);
  if (npl <= 4) return fwd<T, 4>(a, s);
  if (npl <= 8) return fwd<T, 8>(a, s);
  if (npl <= 16) return fwd<T, 16>(a, s);
  return fwd<T, 32>(a, s);
}
template <typename T>
cudaError_t bwd_t(const RouteScoredBwdArgs& a, cudaStream_t s) {
  const int npl = ceil_div(a.E, 32);
  if (npl <= 1) return bwd<T, 1>(a, s);
  if (npl <= 2) return bwd<T, 2>(a, s);
  if (npl <= 4) return bwd<T, 4>(a, s);
  if (npl <= 8) return bwd<T, 8>(a, s);
  if (npl <= 16) return bwd<T, 16>(a, s);
  return bwd<T, 32>(a, s);
}

}  // namespace

cudaError_t launch_route_scored(const RouteScoredArgs& a, bool bf16, cudaStream_t s) {
  const cudaError_t e = bf16 ? fwd_t<__nv_bfloat16>(a, s) : fwd_t<float>(a, s);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_route_scored_backward(const RouteScoredBwdArgs& a, bool bf16, cudaStream_t s) {
  const cudaError_t e = bf16 ? bwd_t<__nv_bfloat16>(a, s) : bwd_t<float>(a, s);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
