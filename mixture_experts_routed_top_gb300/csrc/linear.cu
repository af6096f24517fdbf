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
// Three kernels, chosen by linear_path():
//   linear_pair_kernel   256 x 256 tiles on CTA pairs, persistent: large products
//   linear_tile_kernel   128 x 128 tiles, the contraction split over the CTAs
//                        of a cluster: few tiles
//   linear_gemv_kernel   up to 8 tokens: the weights streamed through CUDA cores
#include <algorithm>
#include <atomic>

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

// The epilogue on 8 consecutive columns n.. of row m (m < M): pre-activation
// z = v + bias, y = residual + act(z).  The activation is computed in fp32
// with silu_f's fast division only where the result is rounded to bf16.
__device__ __forceinline__ float act_f(float z, int act, bool f32) {
  if (act == MOE_ACT_NONE) return z;
  if (act == MOE_ACT_SILU && f32) return z / (1.f + expf(-z));
  return gate_act(z, act);
}
__device__ __forceinline__ void epilogue8(const LinearEpi& p, long m, int n, float (&v)[8]) {
  if (n >= p.N) return;
  if (p.vec) {  // N % 8 == 0 and every row 16-byte aligned
    float b[8];
    if (p.bias != nullptr) {
      ld8(p.bias, n, p.bias_bf16, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += b[j];
    }
    if (p.preact != nullptr) st8(p.preact, m * p.ld_out + n, p.out_f32, v);
    if (p.act != MOE_ACT_NONE) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = act_f(v[j], p.act, p.out_f32);
    }
    if (p.residual != nullptr) {
      ld8(p.residual, m * p.ld_res + n, !p.out_f32, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += b[j];
    }
    st8(p.out, m * p.ld_out + n, p.out_f32, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (n + j < p.N) {
        float z = v[j];
        if (p.bias != nullptr) z += ldf(p.bias, n + j, p.bias_bf16);
        if (p.preact != nullptr) stf(p.preact, m * p.ld_out + n + j, p.out_f32, z);
        z = act_f(z, p.act, p.out_f32);
        if (p.residual != nullptr) z += ldf(p.residual, m * p.ld_res + n + j, !p.out_f32);
        stf(p.out, m * p.ld_out + n + j, p.out_f32, z);
      }
    }
  }
}

// ====================================================== CTA-pair kernel
// tcgen05.mma.cta_group::2, M = 256 (128 rows of A in each CTA), N = 256
// (128 rows of B in each CTA), 128 of the contraction per stage.  Roles in
// each CTA (192 threads): warp 0 TMA producer (ring of 3 stages, 32 KB of A
// and of B each), warp 1 TMEM and, on rank 0, the MMA issuer (two
// 256-column accumulators, so a tile's epilogue runs under the next tile's
// products), warps 2-5 epilogue.  Both CTAs' loads complete on rank 0's stage
// barrier; rank 0's commits arrive on both CTAs' stage-free and
// accumulator-full barriers; both epilogues arrive on rank 0's
// accumulator-free barrier.  Every mbarrier wait is bounded.
constexpr int kPStages = 3;
constexpr int kPThreads = 192;
constexpr int kPSlab = 128 * BK * 2;        // 16 KB: 128 rows x 64, or 64 rows x 128
constexpr int kPOper = 2 * kPSlab;          // one operand's part of a stage
constexpr int kPOffB = kPStages * kPOper;
constexpr int kPOffBar = 2 * kPStages * kPOper;
constexpr int kPBars = 2 * kPStages + 2 + 2 + 1;
constexpr int kPOffMisc = kPOffBar + kPBars * 8;
constexpr int kPSmem = kPOffMisc + 16 + 1024;
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

template <bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kPThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tm_a,
                       const __grid_constant__ CUtensorMap tm_b, const LinearDev p) {
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
      mbar_init(smem_u32(&tempty[a]), 8);
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
          if (!mbar_wait_bounded<true, true>(smem_u32(&empty[stage]), ph ^ 1u, s_abort, p.err,
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
          mbar_wait_bounded<true, true>(smem_u32(rank == 0 ? &full[s] : &empty[s]), par, &no_abort,
                                        p.err, ERR_TIMEOUT_PRODUCER, 20000000ull);
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
        if (!mbar_wait_bounded<true, true>(smem_u32(&tempty[acc]), ((it >> 1) & 1) ^ 1u, s_abort,
                                           p.err, ERR_TIMEOUT_MMA))
          break;
        tc_fence_after();
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait_bounded<true, true>(smem_u32(&full[stage]), ph, s_abort, p.err,
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
        mbar_wait_bounded<true, true>(smem_u32(fin), 0, &no_abort, p.err, ERR_TIMEOUT_MMA);
      }
    }
  } else {
    const int q = warp & 3;  // TMEM lane quarter this warp may access
    const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16);
    int it = 0;
    for (int tile = cid; tile < total; tile += ncl, ++it) {
      int mi, ni;
      pair_tile(tile, mt, nt, p.group, &mi, &ni);
      const int acc = it & 1;
      int ok = 1;
      if (lane == 0)
        ok = mbar_wait_bounded<true, true>(smem_u32(&tfull[acc]), (it >> 1) & 1, s_abort, p.err,
                                           ERR_TIMEOUT_EPILOGUE);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const long m = static_cast<long>(mi) * 256 + 128 * rank + 32 * q + lane;
      const int n0 = ni * 256;
      const int steps = min(8, (p.epi.N - n0 + 31) >> 5);
      for (int s = 0; s < steps; ++s) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(tl + acc * 256 + 32 * s, v);
        tmem_ld_wait();
        if (s == steps - 1) {  // every column read: hand the accumulator back
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (rank == 0) mbar_arrive(smem_u32(&tempty[acc]));
            else mbar_arrive_remote(mapa_shared(smem_u32(&tempty[acc]), 0));
          }
        }
        if (m < p.epi.M) {
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[j + i]);
            epilogue8(p.epi, m, n0 + 32 * s + j, f);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither CTA leaves while the other may touch its shared memory
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ====================================================== split tile kernel
// One 128 x 128 tile per cluster of S CTAs; CTA r takes the r-th part of the
// contraction.  The parts are added through distributed shared memory: each
// CTA leaves its accumulator in its own shared memory, and CTA r adds rows
// r * 128/S .. of all S in rank order (so the result does not depend on
// timing) and runs the epilogue on them.  No scratch in global memory, one
// launch.
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

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kTThreads)
    linear_tile_kernel(const __grid_constant__ CUtensorMap tm_a,
                       const __grid_constant__ CUtensorMap tm_b, const LinearDev p) {
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
  if (warp == 1) tmem_alloc(smem_u32(s_tmem), 128);
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
  int ok = 1;
  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t ph = 0, issued = 0, last_par = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait_bounded<true>(smem_u32(&empty[stage]), ph ^ 1u, s_abort, p.err,
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
          mbar_wait_bounded<true>(smem_u32(&full[s]), (last_par >> s) & 1u, &no_abort, p.err,
                                  ERR_TIMEOUT_PRODUCER, 20000000ull);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_order(128, 128, A_MN, B_MN);
      int stage = 0;
      uint32_t ph = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait_bounded<true>(smem_u32(&full[stage]), ph, s_abort, p.err, ERR_TIMEOUT_MMA))
          break;
        tc_fence_after();
        const uint32_t as = smem_u32(smem + stage * kTOper);
        const uint32_t bs = smem_u32(smem + kTOffB + stage * kTOper);
        const uint64_t ad = A_MN ? sdesc_mn_sw128(as, kTOper / 2) : sdesc_k_sw128(as);
        const uint64_t bd = B_MN ? sdesc_mn_sw128(bs, kTOper / 2) : sdesc_k_sw128(bs);
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          umma_f16(tmem, ad + (A_MN ? kk * 128 : kk * 2), bd + (B_MN ? kk * 128 : kk * 2), idesc,
                   (kb > kb0 || kk > 0) ? 1u : 0u);
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
  if (!mbar_wait_bounded<true>(smem_u32(done), 0, s_abort, p.err, ERR_TIMEOUT_EPILOGUE) || *s_abort)
    ok = 0;
  __syncthreads();
  __syncwarp();
  tc_fence_after();
  float* stg = reinterpret_cast<float*>(smem);
  if (warp >= 2) {
    const int q = warp & 3;
    const int row = 32 * q + lane;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(q * 32) << 16) + 32 * s, v);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        *reinterpret_cast<float4*>(stg + row * kTStride + 32 * s + j) =
            kb1 > kb0 ? make_float4(__uint_as_float(v[j]), __uint_as_float(v[j + 1]),
                                    __uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]))
                      : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    tc_fence_before();
  }
  __syncwarp();
  if (S > 1) cluster_sync_all();
  else __syncthreads();
  if (ok) {
    const int rows = 128 / S;
    for (int i = threadIdx.x; i < rows * 16; i += kTThreads) {
      const int row = rank * rows + (i >> 4), col = (i & 15) * 8;
      const long m = static_cast<long>(mi) * 128 + row;
      if (m >= p.epi.M || ni * 128 + col >= p.epi.N) continue;
      const uint32_t at = smem_u32(stg + row * kTStride + col);
      float f[8] = {};
      for (int r = 0; r < S; ++r) {
        const uint32_t o = mapa_shared(at, r);
        const float4 a = ld_cluster_f4(o), b = ld_cluster_f4(o + 16);
        f[0] += a.x, f[1] += a.y, f[2] += a.z, f[3] += a.w;
        f[4] += b.x, f[5] += b.y, f[6] += b.z, f[7] += b.w;
      }
      epilogue8(p.epi, m, ni * 128 + col, f);
    }
  }
  __syncwarp();
  if (S > 1) cluster_sync_all();  // the others have read this CTA's part
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 128);
}

// ====================================================== few tokens
// Weights [N, K] streamed once by CUDA cores: WPR warps of a block share R
// rows of w, each lane multiplying 16-byte pieces of them with the same
// pieces of the TT tokens (read through L1).
template <int TT, int WPR>
__global__ void __launch_bounds__(256) linear_gemv_kernel(const LinearGemvArgs a) {
  constexpr int R = 2;                // rows of w per warp: they share the token loads
  constexpr int GROUPS = 8 / WPR;     // row pairs per block
  pdl_launch_dependents();
  __shared__ float s_part[8][R * TT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = warp / WPR, part = warp % WPR;
  const int n0 = (blockIdx.x * GROUPS + grp) * R;
  pdl_wait();
  float acc[R][TT] = {};
  const int chunks = a.K / 8;
  if (n0 < a.epi.N) {
    const __nv_bfloat16* w0 = a.w + static_cast<long>(n0) * a.ld_w;
    const __nv_bfloat16* w1 = a.w + static_cast<long>(min(n0 + 1, a.epi.N - 1)) * a.ld_w;
#pragma unroll 4
    for (int c = part * 32 + lane; c < chunks; c += WPR * 32) {
      float f[R][8];
      ld8(w0, c * 8, true, f[0]);
      ld8(w1, c * 8, true, f[1]);
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        if (t < a.epi.M) {
          float x[8];
          ld8(a.x, t * a.ld_x + c * 8, true, x);
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[r][t] = fmaf(f[r][j], x[j], acc[r][t]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1)
        acc[r][t] += __shfl_xor_sync(0xffffffffu, acc[r][t], off);
      if (lane == 0) s_part[warp][r * TT + t] = acc[r][t];
    }
  __syncthreads();
  if (threadIdx.x < GROUPS * R * TT) {
    const int g = threadIdx.x / (R * TT), i = threadIdx.x % (R * TT);
    const int r = i / TT, t = i % TT;
    const int n = (blockIdx.x * GROUPS + g) * R + r;
    if (n < a.epi.N && t < a.epi.M) {
      float z = 0.f;
#pragma unroll
      for (int w = 0; w < WPR; ++w) z += s_part[g * WPR + w][i];
      const LinearEpi& p = a.epi;
      if (p.bias != nullptr) z += ldf(p.bias, n, p.bias_bf16);
      if (p.preact != nullptr) stf(p.preact, t * p.ld_out + n, p.out_f32, z);
      z = act_f(z, p.act, p.out_f32);
      if (p.residual != nullptr) z += ldf(p.residual, t * p.ld_res + n, !p.out_f32);
      stf(p.out, t * p.ld_out + n, p.out_f32, z);
    }
  }
}

// ====================================================== dz and dbias
// dz = dy * act'(z) rounded to bf16 for the two products (their operands are
// bf16 tiles), and the column sums of the unrounded dz.  A block covers 256
// columns (8 per thread) and a slice of the rows; the slices' sums are added
// in order by linear_colsum_kernel.
// One exponential per slope, with the fast exponential and division: at most
// a few units of 2^-22, far below the rounding of dz (2^-9 on average) and
// averaged out in the sums.  With the accurate forms the kernel spent 57
// instructions per element and took 40 us for 8191 x 2048, three times what
// its loads and stores need.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if (ACT == MOE_ACT_SILU) {  // s (1 + z (1 - s)), 1 - s = e^-z s; e^-z kept finite
    const float e = __expf(fminf(-z, 80.f)), s = __fdividef(1.f, 1.f + e);
    return s * fmaf(z, e * s, 1.f);
  }
  if (ACT == MOE_ACT_GELU)  // Phi(z) + z phi(z); the second term is 0 long before z^2 overflows
    return fmaf(z * __expf(-0.5f * fminf(z * z, 1000.f)), 0.39894228040143268f,
                0.5f * (1.f + erff(z * 0.70710678118654752f)));
  return z > 0.f ? 1.f : 0.f;
}

template <int ACT, bool F32>
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

template <bool A_MN, bool B_MN>
cudaError_t launch_pair(const CUtensorMap& tm_a, const CUtensorMap& tm_b, LinearDev p,
                        cudaStream_t s) {
  auto kern = linear_pair_kernel<A_MN, B_MN>;
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

template <int TT, int WPR>
cudaError_t launch_gemv_t(const LinearGemvArgs& a, cudaStream_t s) {
  const int rows = 8 / WPR * 2;
  return launch_pdl(linear_gemv_kernel<TT, WPR>, dim3(ceil_div(a.epi.N, rows)), dim3(256), 0, s, a);
}
template <int TT>
cudaError_t launch_gemv_w(const LinearGemvArgs& a, int num_sms, cudaStream_t s) {
  // warps per row pair: enough that every SM has 40 warps, at most 8
  const long pairs = (a.epi.N + 1) / 2, want = 40L * num_sms;
  if (pairs >= want) return launch_gemv_t<TT, 1>(a, s);
  if (2 * pairs >= want) return launch_gemv_t<TT, 2>(a, s);
  if (4 * pairs >= want) return launch_gemv_t<TT, 4>(a, s);
  return launch_gemv_t<TT, 8>(a, s);
}

}  // namespace

// Tiles of 256 x 256 on CTA pairs from half a wave of them; below, 128 x 128
// tiles whose contraction is split over up to 8 CTAs until the grid covers
// the GPU twice (two such CTAs fit an SM), each part at least 4 stages long.
LinearPath linear_path(long M, long N, long K, int num_sms) {
  LinearPath r;
  const long big = static_cast<long>(ceil_div(M, 256)) * ceil_div(N, 256);
  r.pair = big >= num_sms / 4;
  r.split = 1;
  const long tiles = static_cast<long>(ceil_div(M, 128)) * ceil_div(N, 128);
  while (r.split < 8 && tiles * r.split * 2 <= 2L * num_sms && K / (r.split * 2) >= 4 * BK)
    r.split *= 2;
  return r;
}

cudaError_t launch_linear(const CUtensorMap& tm_a, const CUtensorMap& tm_b, const LinearDev& p,
                          bool a_mn, bool b_mn, const LinearPath& path, cudaStream_t s) {
  if (path.pair) {
    if (!a_mn && !b_mn) return launch_pair<false, false>(tm_a, tm_b, p, s);
    if (!a_mn) return launch_pair<false, true>(tm_a, tm_b, p, s);
    return launch_pair<true, true>(tm_a, tm_b, p, s);
  }
  if (!a_mn && !b_mn) return launch_tile<false, false>(tm_a, tm_b, p, path.split, s);
  if (!a_mn) return launch_tile<false, true>(tm_a, tm_b, p, path.split, s);
  return launch_tile<true, true>(tm_a, tm_b, p, path.split, s);
}

cudaError_t launch_linear_gemv(const LinearGemvArgs& a, int num_sms, cudaStream_t s) {
  cudaError_t e;
  if (a.epi.M <= 1) e = launch_gemv_w<1>(a, num_sms, s);
  else if (a.epi.M <= 2) e = launch_gemv_w<2>(a, num_sms, s);
  else if (a.epi.M <= 4) e = launch_gemv_w<4>(a, num_sms, s);
  else e = launch_gemv_w<8>(a, num_sms, s);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

int linear_dz_slices(long T, long N, int num_sms) {
  const long cols = ceil_div(N, 256);
  const long want = std::max<long>(1, 4L * num_sms / cols);
  return static_cast<int>(std::max<long>(1, std::min<long>(want, T / 32)));
}

cudaError_t launch_linear_dz(const LinearDzArgs& a, int slices, float* dbias, cudaStream_t s) {
  const dim3 grid(ceil_div(a.N, 256), slices), block(256);
  cudaError_t e;
  auto go = [&](auto kern_f32, auto kern_bf16) {
    return a.f32 ? launch_pdl(kern_f32, grid, block, 0, s, a) : launch_pdl(kern_bf16, grid, block, 0, s, a);
  };
  if (a.act == MOE_ACT_SILU)
    e = go(linear_dz_kernel<MOE_ACT_SILU, true>, linear_dz_kernel<MOE_ACT_SILU, false>);
  else if (a.act == MOE_ACT_GELU)
    e = go(linear_dz_kernel<MOE_ACT_GELU, true>, linear_dz_kernel<MOE_ACT_GELU, false>);
  else if (a.act == MOE_ACT_RELU)
    e = go(linear_dz_kernel<MOE_ACT_RELU, true>, linear_dz_kernel<MOE_ACT_RELU, false>);
  else
    e = go(linear_dz_kernel<MOE_ACT_NONE, true>, linear_dz_kernel<MOE_ACT_NONE, false>);
  count_launches(1);
  if (e != cudaSuccess) return e;
  if (dbias != nullptr) {
    e = launch_pdl(linear_colsum_kernel, dim3(ceil_div(a.N, 32)), dim3(256), 0, s,
                   static_cast<const float*>(a.partials), slices, a.N, dbias);
    count_launches(1);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
