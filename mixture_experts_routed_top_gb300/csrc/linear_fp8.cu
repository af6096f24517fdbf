// Dense products of 8-bit operands: y = residual + act(x w^T + bias) with e4m3 codes, a
// scale per 1 x 128 of x (a token, 128 of the contraction) and one per 128 x 128 of w,
// and the quantiser of such rows:
//   z[t, n] = sum_kb sx[t, kb] sw[n / 128, kb] (sum_{k in kb} qx[t, k] qw[n, k])
// A block of 128 of the contraction is one 128-byte swizzled row of an operand and one
// scale of each: the inner sums come from the tensor core (products of e4m3 are exact
// in it), and are multiplied by their scales and added in fp32 registers.
//
// The kernels, chosen by fp8_streams() and fp8_path():
//   fp8_pair_kernel    256 x 256 tiles on CTA pairs, persistent: large products
//   fp8_tile_kernel    128 x 128 tiles, the contraction split over a cluster: few tiles
//   fp8_stream_kernel  a few tokens: the weights streamed into registers
//   fp8_rows_kernel    the rows' codes and scales, before the first two
#include <algorithm>
#include <atomic>

#include "linear_device.cuh"

namespace moe {
namespace {

constexpr int kB = 128;  // e4m3 per 128-byte swizzled row = one scale block

__device__ __forceinline__ float ue8m0_value(uint32_t b) {
  return b == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23);
}
__device__ __forceinline__ float scale_at(const void* base, long i, int ue8m0) {
  return ue8m0 ? ue8m0_value(__ldg(static_cast<const uint8_t*>(base) + i))
               : __ldg(static_cast<const float*>(base) + i);
}
// Of a block of a row from its absolute maximum, as the weights' quantiser, but no
// less than 2^-126, whose reciprocal is still a number; *stored: bits or exponent byte.
// An infinity or NaN makes an infinite or NaN scale (byte 255), which makes its row NaN.
__device__ __forceinline__ float row_scale(float amax, bool ue8m0, uint32_t* stored) {
  if (amax == 0.f) {
    *stored = ue8m0 ? 127u : __float_as_uint(1.0f);
    return 1.0f;
  }
  float q = amax / 448.0f;
  q = q < __uint_as_float(0x00800000u) ? __uint_as_float(0x00800000u) : q;  // a NaN stays one
  if (!ue8m0) {
    *stored = __float_as_uint(q);
    return q;
  }
  if (!(q < INFINITY)) {
    *stored = 255u;
    return INFINITY;
  }
  return ue8m0_ceil(q, stored);
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return static_cast<uint32_t>(e4m3x2(a, b)) | (static_cast<uint32_t>(e4m3x2(c, d)) << 16);
}
__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}
// The largest absolute value of 8, as bits: those of bf16 without a sign are ordered as
// integers, NaN above all.
__device__ __forceinline__ uint32_t amax8(const uint4& u) {
  const uint32_t m = 0x7fff7fffu;
  return __vmaxu2(__vmaxu2(u.x & m, u.y & m), __vmaxu2(u.z & m, u.w & m));
}
__device__ __forceinline__ float amax_value(uint32_t pair) {  // of both halves
  return __uint_as_float(max(pair << 16, pair & 0xffff0000u));
}
__device__ __forceinline__ uint2 codes8(const uint4& u, float inv) {
  float v[8];
  unpack8(u, v);
  return make_uint2(e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}

// ====================================================== rows of codes
// Bound by memory.  A block takes 32 rows x 512 columns; 16 lanes hold a 1 x 128 block,
// 16 bytes each, and a thread's 8 loads are on their way before the first is used; each
// scale is made by one lane.  8192 x 7168 31 us (176 MB, 5.7 TB/s).  The
// scales leave through shared memory, so that those of a K block are written in whole
// lines where they are neighbours.
__global__ void __launch_bounds__(256) fp8_rows_kernel(const __grid_constant__ Fp8RowsArgs a) {
  pdl_launch_dependents();
  __shared__ uint32_t s_scale[4][32];
  const int hw = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int t0 = blockIdx.x * 32, kb0 = blockIdx.y * 4;
  pdl_wait();
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int u = hw + 16 * i, t = t0 + (u >> 2), kb = kb0 + (u & 3);
    v[i] = t < a.T && kb < a.KB
               ? __ldg(reinterpret_cast<const uint4*>(a.x + t * a.ld_x + kb * kB) + l)
               : make_uint4(0u, 0u, 0u, 0u);
  }
  // lane l of the 16 keeps the maximum of unit l % 8, so that each scale is made once
  uint32_t mine = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t m = amax8(v[i]);
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, off));
    if ((l & 7) == i) mine = m;
  }
  uint32_t stored;
  const float inv_mine = 1.0f / row_scale(amax_value(mine), a.ue8m0, &stored);
  if (l < 8) {
    const int u = hw + 16 * l;
    s_scale[u & 3][u >> 2] = stored;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int u = hw + 16 * i, t = t0 + (u >> 2), kb = kb0 + (u & 3);
    const float inv = __shfl_sync(0xffffffffu, inv_mine, i, 16);
    if (t < a.T && kb < a.KB)
      reinterpret_cast<uint2*>(a.q + (static_cast<long>(t) * a.KB + kb) * kB)[l] = codes8(v[i], inv);
  }
  __syncthreads();
  const int i = threadIdx.x;
  if (i >= 128) return;
  const int t = t0 + (i & 31), kb = kb0 + (i >> 5);
  if (t >= a.T || kb >= a.KB) return;
  const long at = t * a.s_row + kb * a.s_kb;
  if (a.ue8m0) static_cast<uint8_t*>(a.scale)[at] = static_cast<uint8_t>(s_scale[i >> 5][i & 31]);
  else static_cast<uint32_t*>(a.scale)[at] = s_scale[i >> 5][i & 31];
}

// ====================================================== promotion
// 32 of a K block's sums in this thread's row, times s, added to acc[AT ..].
template <int AT, int N>
__device__ __forceinline__ void promote(const uint32_t (&v)[32], float s, float (&acc)[N]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) acc[AT + i] = fmaf(__uint_as_float(v[i]), s, acc[AT + i]);
}

// The scales of a row of x, four K blocks at a time: one 16-byte load where they lie side by
// side (fp32; 4 bytes of UE8M0), four loads where they do not.
struct ScaleRow {
  const char* x;
  long step;
  bool valid, side, ue8m0;
  __device__ __forceinline__ ScaleRow(const Fp8Scales& sc, long m, bool valid_)
      : valid(valid_), ue8m0(sc.ue8m0 != 0) {
    const int size = ue8m0 ? 1 : 4;
    x = static_cast<const char*>(sc.x) + m * sc.x_row * size;
    step = sc.x_kb * size;
    side = sc.x_kb == 1 && (reinterpret_cast<uintptr_t>(x) & (4 * size - 1)) == 0;
  }
  // of the blocks kb .. kb + 3, kb a multiple of 4, those below KB
  __device__ __forceinline__ void four(int kb, int KB, float (&s)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = 0.f;
    if (!valid) return;
    const char* p = x + kb * step;
    if (side && kb + 4 <= KB) {
      if (!ue8m0) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p));
        s[0] = v.x, s[1] = v.y, s[2] = v.z, s[3] = v.w;
      } else {
        const uint32_t v = __ldg(reinterpret_cast<const uint32_t*>(p));
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = ue8m0_value((v >> (8 * i)) & 255u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (kb + i < KB) s[i] = scale_at(p + i * step, 0, ue8m0);
    }
  }
};

// ====================================================== CTA-pair kernel
// 256 x 256 tiles, cta_group::2: each CTA holds 128 rows of x and 128 of w per stage, and
// 128 rows x 256 columns of the sums of two K blocks in TMEM, one of them being filled
// while the other is promoted.  Roles (384 threads):
//   warp 0     TMA producer
//   warp 1     MMA issuer (rank 0); the whole warp walks and one lane issues
//   warps 2-3  the scale products of 8 K blocks at a time, into a ring of two such slabs
//   warps 4-11 promotion and epilogue: thread = row, two halves of 128 columns.  Columns go
//              32 at a time, the next load on its way while the last one is multiplied,
//              also from one K block to the next.  128 sums and 64 loaded values take the
//              registers that the first four warps give up (4 x 56 + 8 x 224 a lane of the
//              12 x 168 that the block is launched with).
// Barriers as in the bf16 pair kernel.  Those that the other CTA signals are waited for at
// cluster scope: without an acquire where only TMEM changes hands, with one of shared memory
// where the loads' stages do.  An acquire of all memory empties the L1, which holds the scales
// that the warps 2-3 go on with: 8192 x 7168 x 4096 with UE8M0 scales 242 us, so 203.  The slabs'
// barriers, of one CTA, are waited for at its own scope.  Every wait is bounded.
//
// 8192 x 7168 x 4096 with either kind of scales 202 to 207 us (2.35 PFLOP/s).  Bound by the promotion beside
// the products: without it the same loop takes 138 (3.5 PFLOP/s).  128 multiply-adds a thread and
// block with two warps a scheduler, the reads of TMEM and the tensor core overlap only in
// part.  Plain multiply-adds: packed ones issue at half the rate and were 5 % slower here.
// Narrower tiles, which would leave four buffers in TMEM, are bound by shared memory (281 us),
// 16 promoting warps by their registers (248 and more).  The arrivals that hand a buffer back
// to rank 0, 8 a K block, are relaxed: released at cluster scope they doubled the time (406).
constexpr int kStages = 5;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr int kRegsFew = 56, kRegsMany = 224;
static_assert(4 * kRegsFew + kEpiWarps * kRegsMany <= (4 + kEpiWarps) * 168, "registers of the launch");
constexpr int kSlab = 8;                           // K blocks of scale products
constexpr int kOper = 128 * kB;                    // 16 KB: one operand's part of a stage
constexpr int kOffBar = 2 * kStages * kOper;
constexpr int kBars = 2 * kStages + 9;
constexpr int kOffMisc = kOffBar + kBars * 8;
constexpr int kOffTurn = (kOffMisc + 8 + 15) / 16 * 16;
constexpr int kOffScale = kOffTurn + kEpiWarps * kTurn * 4;  // [2][kSlab][2 halves][128 rows]
constexpr int kSmem = kOffScale + 2 * kSlab * 256 * 4 + 1024;
static_assert(kOffMisc % 8 == 0 && kSmem <= 227 * 1024, "shared memory");

// 64 columns of 32 rows of bf16 results without activation and residual, rows of whole
// aligned vectors: the bias where the sums are, 16-byte pieces of the rounded rows through
// the turn buffer (in the order of their index xor the row's), then 8 lanes along a row, so
// that a store fills lines.
__device__ __forceinline__ void epilogue64_bf16(const LinearEpi& p, int m0, int n, float* z, float* buf, int lane) {
  uint4* const b4 = reinterpret_cast<uint4*>(buf);
  __syncwarp();  // the previous step's values have been read
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    if (p.bias != nullptr && n + 8 * c < p.N) {
      float b[8];
      ld8(p.bias, n + 8 * c, p.bias_bf16, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) z[8 * c + j] += b[j];
    }
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(z[8 * c + 2 * j], z[8 * c + 2 * j + 1]);
    b4[lane * 8 + (c ^ (lane & 7))] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __syncwarp();
  const int c = lane & 7, r0 = lane >> 3;
  if (n + 8 * c >= p.N) return;
  __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.out) + (static_cast<long>(m0) + r0) * p.ld_out + n + 8 * c;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 4 * i;
    if (m0 + r < p.M) *reinterpret_cast<uint4*>(to + 4 * i * p.ld_out) = b4[r * 8 + (c ^ (r & 7))];
  }
}
// 32 columns of 32 rows of anything else, rows of whole aligned vectors, in little code: 8
// activations of a loop.  With all 128 of a thread's columns in line, fetching the code took
// longer than running it (4099 x 7168 x 2112 with gelu 112 us, so 92).
template <int ACT, bool F32>
__device__ __forceinline__ void epilogue32_small(const LinearEpi& p, int m0, int n, const uint32_t (&v)[32],
                                                 float* buf, int lane) {
  const int nv = n + 8 * (lane & 3), c = 2 * (lane & 3);
  float b[8] = {};
  if (p.bias != nullptr && nv < p.N) ld8(p.bias, nv, p.bias_bf16, b);
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<uint4*>(buf + lane * 32 + 4 * (c ^ (lane & 7))) =
        make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
  __syncwarp();
  if (nv >= p.N) return;
#pragma unroll 1
  for (int row = lane >> 2; row < 32 && m0 + row < p.M; row += 8) {
    const float4 x = *reinterpret_cast<const float4*>(buf + row * 32 + 4 * (c ^ (row & 7)));
    const float4 y = *reinterpret_cast<const float4*>(buf + row * 32 + 4 * ((c + 1) ^ (row & 7)));
    float f[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w}, r[8] = {};
    const long m = static_cast<long>(m0) + row;
    if (p.residual != nullptr) ld8(p.residual, m * p.ld_res + nv, !F32, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __fadd_rn(act_f(f[j] + b[j], ACT, F32), r[j]);
    st8(p.out, m * p.ld_out + nv, F32, f);
  }
}

template <int ACT, bool F32>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                    const __grid_constant__ Fp8LinearDev p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar);  // rank 0: both CTAs' loads landed
  uint64_t* empty = full + kStages;        // both: the stage's MMAs are done
  uint64_t* pfull = empty + kStages;       // both: sums of a K block complete
  uint64_t* pempty = pfull + 2;            // rank 0: both CTAs have read them
  uint64_t* fin = pempty + 2;              // rank 0: every MMA done
  uint64_t* sfull = fin + 1;               // a slab of scale products is there
  uint64_t* sempty = sfull + 2;            // it has been read
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank() & 1u);
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&pfull[b]), 1);
      mbar_init(smem_u32(&pempty[b]), 2 * kEpiWarps);
      mbar_init(smem_u32(&sfull[b]), 64);
      mbar_init(smem_u32(&sempty[b]), kEpiWarps);
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
  const int total = mt * nt, KB = p.KB;
  const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
  float* const slabs = reinterpret_cast<float*>(smem + kOffScale);

  if (warp < 4) {
    regs_fewer<kRegsFew>();
    if (warp == 0 && lane == 0) {
      int stage = 0;
      uint32_t ph = 0, issued = 0, last_par = 0;
      bool ok = true;
      for (int tile = cid; ok && tile < total; tile += ncl) {
        int mi, ni;
        pair_tile(tile, mt, nt, p.group, &mi, &ni);
        for (int kb = 0; kb < KB; ++kb) {
          if (!wait_pair_relaxed(smem_u32(&empty[stage]), ph ^ 1u, s_abort, p.err, ERR_TIMEOUT_PRODUCER)) {
            ok = false;
            break;
          }
          fence_acquire_shared_cluster();
          const uint32_t fb_local = smem_u32(&full[stage]);
          if (rank == 0) mbar_arrive_expect_tx(fb_local, 4u * kOper);
          const uint32_t fb = mapa_shared(fb_local, 0);
          const uint32_t a_dst = smem_u32(smem + 2 * stage * kOper);
          tma_load_2d_pair(&tm_a, fb, a_dst, kb * kB, mi * 256 + 128 * rank);
          tma_load_2d_pair(&tm_b, fb, a_dst + kOper, kb * kB, ni * 256 + 128 * rank);
          issued |= 1u << stage;
          last_par = (last_par & ~(1u << stage)) | (ph << stage);
          if (++stage == kStages) {
            stage = 0;
            ph ^= 1u;
          }
        }
      }
      // drain: rank 0 until every issued stage's loads (both CTAs') landed,
      // rank 1 until its last loads of each stage were consumed
      for (int s = 0; s < kStages; ++s) {
        if ((issued >> s) & 1u) {
          volatile int no_abort = 0;
          wait_pair(smem_u32(rank == 0 ? &full[s] : &empty[s]), (last_par >> s) & 1u, &no_abort,
                    p.err, ERR_TIMEOUT_PRODUCER, kDrainCycles);
        }
      }
    } else if (warp == 1 && rank == 0) {
      // one K block is like the next, whatever tile it is of
      constexpr uint32_t idesc = idesc_e4m3_f32(256, 256);
      const uint32_t count = static_cast<uint32_t>(cid < total ? (total - cid + ncl - 1) / ncl : 0) * KB;
      const uint64_t d0 = sdesc_k_sw128(smem_u32(smem));
      int stage = 0;
      uint32_t ph = 0;
      for (uint32_t g = 0; g < count; ++g) {
        const uint32_t b = g & 1, eph = ((g >> 1) & 1) ^ 1u;
        const uint32_t fbar = smem_u32(&full[stage]), ebar = smem_u32(&pempty[b]);
        const bool f = mbar_try_wait_cluster_relaxed(fbar, ph);  // both on their way
        const bool e = mbar_try_wait_cluster_relaxed(ebar, eph);
        const bool ok = (f || wait_pair_relaxed(fbar, ph, s_abort, p.err, ERR_TIMEOUT_MMA)) &&
                        (e || wait_pair_relaxed(ebar, eph, s_abort, p.err, ERR_TIMEOUT_MMA));
        if (!__all_sync(0xffffffffu, ok)) break;
        fence_acquire_shared_cluster();
        tc_fence_after();
        const uint64_t ad = d0 + static_cast<uint32_t>(stage * (2 * kOper >> 4)), bd = ad + (kOper >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kB / 32; ++kk)
            umma_f8_pair(tmem + b * 256, ad + 2 * kk, bd + 2 * kk, idesc, kk != 0 ? 1u : 0u);
          umma_commit_pair_both(smem_u32(&pfull[b]));
          umma_commit_pair_both(smem_u32(&empty[stage]));
        }
        __syncwarp();
        if (++stage == kStages) {
          stage = 0;
          ph ^= 1u;
        }
      }
      if (count > 0) {
        if (elect_one()) umma_commit_pair_local(smem_u32(fin));
        volatile int no_abort = 0;
        wait_pair(smem_u32(fin), 0, &no_abort, p.err, ERR_TIMEOUT_MMA);
      }
    } else if (warp >= 2) {
      const int r = threadIdx.x - 64;  // rows r and r + 64
      const int nb = (p.epi.N + kB - 1) / kB;  // rows of weight scales
      uint32_t slab = 0;
      bool ok = true;
      for (int tile = cid; ok && tile < total; tile += ncl) {
        int mi, ni;
        pair_tile(tile, mt, nt, p.group, &mi, &ni);
        const long m = static_cast<long>(mi) * 256 + 128 * rank + r;
        ScaleRow x0(p.sc, m, m < p.epi.M), x1(p.sc, m + 64, m + 64 < p.epi.M);
        const long w0 = static_cast<long>(min(2 * ni, nb - 1)) * KB, w1 = static_cast<long>(min(2 * ni + 1, nb - 1)) * KB;
        for (int kb = 0; kb < KB; kb += kSlab, ++slab) {
          const int b = slab & 1;
          if (!wait_cta(smem_u32(&sempty[b]), ((slab >> 1) & 1) ^ 1u, s_abort, p.err, ERR_TIMEOUT_EPILOGUE)) {
            ok = false;
            break;
          }
          float* to = slabs + b * kSlab * 256 + r;
#pragma unroll 1
          for (int j = 0; j < kSlab && kb + j < KB; j += 4) {
            float a[4], c[4];
            x0.four(kb + j, KB, a);
            x1.four(kb + j, KB, c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (kb + j + i >= KB) continue;
              const float u0 = scale_at(p.sc.w, w0 + kb + j + i, p.sc.ue8m0),
                          u1 = scale_at(p.sc.w, w1 + kb + j + i, p.sc.ue8m0);
              float* const at = to + (j + i) * 256;
              at[0] = a[i] * u0;
              at[64] = c[i] * u0;
              at[128] = a[i] * u1;
              at[192] = c[i] * u1;
            }
          }
          mbar_arrive(smem_u32(&sfull[b]));
        }
      }
    }
    __syncwarp();
  } else {
    regs_more<kRegsMany>();
    const int q = warp & 3, half = (warp - 4) >> 2;  // TMEM lane quarter, column half
    const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16) + 128 * half;
    float* const turn = reinterpret_cast<float*>(smem + kOffTurn) + (warp - 4) * kTurn;
    const uint32_t pempty0 = rank == 0 ? smem_u32(pempty) : mapa_shared(smem_u32(pempty), 0);
    const float* const mine = slabs + 128 * half + 32 * q + lane;
    uint32_t g = 0, slab = 0;  // K blocks and slabs so far
    uint32_t v[2][32];
    // waits for block g's sums and asks for the first 32 of them
    auto begin = [&] {
      const bool ready = wait_pair_relaxed(smem_u32(&pfull[g & 1]), (g >> 1) & 1, s_abort, p.err, ERR_TIMEOUT_EPILOGUE);
      if (!__all_sync(0xffffffffu, ready)) return false;
      tc_fence_after();
      tmem_ld_32x32b_x32(tl + (g & 1) * 256, v[0]);
      return true;
    };
    for (int tile = cid; tile < total; tile += ncl) {
      int mi, ni;
      pair_tile(tile, mt, nt, p.group, &mi, &ni);
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.f;
      bool ok = true;
      for (int kb0 = 0; ok && kb0 < KB; kb0 += kSlab, ++slab) {
        ok = wait_cta(smem_u32(&sfull[slab & 1]), (slab >> 1) & 1, s_abort, p.err, ERR_TIMEOUT_EPILOGUE);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const float* from = mine + (slab & 1) * kSlab * 256;
        const int count = min(kSlab, KB - kb0);
        if (kb0 == 0) ok = begin();
#pragma unroll 1
        for (int j = 0; ok && j < count; ++j) {
          const float s = from[j * 256];
          const uint32_t tb = tl + (g & 1) * 256;
          tmem_ld_wait_x32(v[0]);
          tmem_ld_32x32b_x32(tb + 32, v[1]);
          promote<0>(v[0], s, acc);
          tmem_ld_wait_x32(v[1]);
          tmem_ld_32x32b_x32(tb + 64, v[0]);
          promote<32>(v[1], s, acc);
          tmem_ld_wait_x32(v[0]);
          tmem_ld_32x32b_x32(tb + 96, v[1]);
          promote<64>(v[0], s, acc);
          tmem_ld_wait_x32(v[1]);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (rank == 0) mbar_arrive(pempty0 + 8 * (g & 1));
            else mbar_arrive_remote_relaxed(pempty0 + 8 * (g & 1));
          }
          ++g;
          if (kb0 + j + 1 < KB) ok = begin();
          promote<96>(v[1], s, acc);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sempty[slab & 1]));
      }
      if (!ok) break;
      // what the epilogue derives from these is not worth a register while blocks are promoted
      int ln = lane, n0 = ni * 256 + 128 * half;
      asm volatile("" : "+r"(mi), "+r"(n0), "+r"(ln));
      const int m0 = mi * 256 + 128 * rank + 32 * q;
      constexpr bool kPlain = ACT == MOE_ACT_NONE && !F32;
      if (kPlain && p.epi.vec && p.epi.residual == nullptr) {
        epilogue64_bf16(p.epi, m0, n0, acc, turn, ln);
        if (n0 + 64 < p.epi.N) epilogue64_bf16(p.epi, m0, n0 + 64, acc + 64, turn, ln);
        continue;
      }
      auto step = [&](const float* z, int n) {
        uint32_t u[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(z[i]);
        if (n >= p.epi.N) return;
        if (!kPlain && p.epi.vec) epilogue32_small<ACT, F32>(p.epi, m0, n, u, turn, ln);
        else epilogue32<ACT, F32, false>(p.epi, static_cast<long>(m0) + ln, n, u, turn, ln);
      };
      if (kPlain) {  // in a loop, as the others, it cost the promotion registers (222 us against 205)
#pragma unroll
        for (int s = 0; s < 4; ++s) step(acc + 32 * s, n0 + 32 * s);
      } else {
#pragma unroll 1
        for (int s = 0; s < 4; ++s) {
          step(acc, n0 + 32 * s);
#pragma unroll
          for (int i = 0; i < 96; ++i) acc[i] = acc[i + 32];
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither CTA leaves while the other may touch its shared memory
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ====================================================== split tile kernel
// One 128 x 128 tile per cluster of S CTAs; CTA r takes the r-th part of the contraction
// (at least one K block).  8 promotion
// warps: thread = row, two halves of 64 columns; the CTAs' sums are joined as the bf16
// kernel's.  Bound by latency: first stages, the exchange of sums, too few blocks.  Codes given
// and all caches cold 64 x 7168 x 2112 16 us on 68 blocks (15.7 MB, tensor cores busy 15 %), 512
// tokens 23 on 136 (19 MB, 19 %).
constexpr int kTStages = 5;
constexpr int kTEpiWarps = 8;
constexpr int kTThreads = 64 + 32 * kTEpiWarps;
constexpr int kTOffBar = 2 * kTStages * kOper;
constexpr int kTBars = 2 * kTStages + 4;
constexpr int kTOffMisc = kTOffBar + kTBars * 8;
constexpr int kTSmem = kTOffMisc + 16 + 1024;
constexpr int kTStride = 132;  // floats per staged row: 128 + 4 (no bank conflicts)
static_assert(128 * kTStride * 4 <= kTOffBar, "staged tile fits the ring");

__global__ void __launch_bounds__(kTThreads, 1)
    fp8_tile_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                    const __grid_constant__ Fp8LinearDev p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kTOffBar);
  uint64_t* empty = full + kTStages;
  uint64_t* pfull = empty + kTStages;
  uint64_t* pempty = pfull + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kTOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kTOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.split;
  const int rank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kTStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&pfull[b]), 1);
      mbar_init(smem_u32(&pempty[b]), kTEpiWarps);
    }
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
  const int kb0 = static_cast<int>(static_cast<long>(p.KB) * rank / S);
  const int kb1 = static_cast<int>(static_cast<long>(p.KB) * (rank + 1) / S);
  float* const stg = reinterpret_cast<float*>(smem);
  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t ph = 0, issued = 0, last_par = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait_cta(smem_u32(&empty[stage]), ph ^ 1u, s_abort, p.err, ERR_TIMEOUT_PRODUCER)) break;
        const uint32_t fb = smem_u32(&full[stage]);
        mbar_arrive_expect_tx(fb, 2u * kOper);
        const uint32_t a_dst = smem_u32(smem + 2 * stage * kOper);
        tma_load_2d(&tm_a, fb, a_dst, kb * kB, mi * 128);
        tma_load_2d(&tm_b, fb, a_dst + kOper, kb * kB, ni * 128);
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
          wait_cta(smem_u32(&full[s]), (last_par >> s) & 1u, &no_abort, p.err, ERR_TIMEOUT_PRODUCER,
                   kDrainCycles);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(128, 128);
      int stage = 0;
      uint32_t ph = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        const int g = kb - kb0, b = g & 1;
        if (!wait_cta(smem_u32(&pempty[b]), ((g >> 1) & 1) ^ 1u, s_abort, p.err, ERR_TIMEOUT_MMA) ||
            !wait_cta(smem_u32(&full[stage]), ph, s_abort, p.err, ERR_TIMEOUT_MMA))
          break;
        tc_fence_after();
        const uint32_t as = smem_u32(smem + 2 * stage * kOper);
        const uint64_t ad = sdesc_k_sw128(as), bd = sdesc_k_sw128(as + kOper);
#pragma unroll
        for (int kk = 0; kk < kB / 32; ++kk)
          umma_f8(tmem + b * 128, ad + 2 * kk, bd + 2 * kk, idesc, kk != 0 ? 1u : 0u);
        umma_commit(smem_u32(&empty[stage]));
        umma_commit(smem_u32(&pfull[b]));
        if (++stage == kTStages) {
          stage = 0;
          ph ^= 1u;
        }
      }
    }
  }
  float acc[64];
  const int q = warp & 3, half = (warp - 2) >> 2;
  if (warp >= 2) {
#pragma unroll
    for (int i = 0; i < 64; ++i) acc[i] = 0.f;
    const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16) + 64 * half;
    const long m = static_cast<long>(mi) * 128 + 32 * q + lane;
    const ScaleRow row(p.sc, m, m < p.epi.M);
    const long w_row = static_cast<long>(ni) * p.KB;  // ni * 128 < N
    uint32_t v[2][32];
    // waits for the sums of block g of this part and asks for the first 32 of them
    auto begin = [&](int g) {
      const bool ready = wait_cta(smem_u32(&pfull[g & 1]), (g >> 1) & 1, s_abort, p.err, ERR_TIMEOUT_EPILOGUE);
      if (!__all_sync(0xffffffffu, ready)) return false;
      tc_fence_after();
      tmem_ld_32x32b_x32(tl + (g & 1) * 128, v[0]);
      return true;
    };
    float sx[4], nx[4], sw = scale_at(p.sc.w, w_row + kb0, p.sc.ue8m0);
    row.four(kb0 & ~3, p.KB, nx);  // the scales of four blocks, those ahead on their way
    bool ok = true;
#pragma unroll 1
    for (int kb = kb0; ok && kb < kb1; ++kb) {
      const int g = kb - kb0, b = g & 1;
      if (g == 0 || (kb & 3) == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sx[i] = nx[i];
        if ((kb | 3) + 1 < kb1) row.four((kb | 3) + 1, p.KB, nx);
      }
      const float s = sw * ((kb & 2) ? ((kb & 1) ? sx[3] : sx[2]) : ((kb & 1) ? sx[1] : sx[0]));
      if (kb + 1 < kb1) sw = scale_at(p.sc.w, w_row + kb + 1, p.sc.ue8m0);
      if (g == 0) ok = begin(0);
      if (!ok) break;
      tmem_ld_wait_x32(v[0]);
      tmem_ld_32x32b_x32(tl + b * 128 + 32, v[1]);
      promote<0>(v[0], s, acc);
      tmem_ld_wait_x32(v[1]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&pempty[b]));
      if (kb + 1 < kb1) ok = begin(g + 1);
      promote<32>(v[1], s, acc);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();  // every K block has been promoted, so every load and product is done
  tc_fence_after();
  if (warp >= 2) {
    float* row = stg + (32 * q + lane) * kTStride + 64 * half;
#pragma unroll
    for (int j = 0; j < 64; j += 4)
      *reinterpret_cast<float4*>(row + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
  }
  __syncthreads();
  const int rows = 128 / S;
  if (S > 1) {
    hand_over<kTThreads, 16, kTStride>(stg, p.parts + static_cast<long>(blockIdx.x) * 128 * 128,
                                       rank * rows, rows);
    __syncwarp();
    cluster_sync_all();  // sums handed over
  }
  if (warp == 1) tmem_dealloc(tmem, 256);
  if (!*s_abort)
    join_rows<kTThreads, 16, kTStride, false>(
        p.epi, stg, p.parts + static_cast<long>(blockIdx.x - rank) * 128 * 128, 128l * 128, S, rank,
        rank * rows, rows, static_cast<long>(mi) * 128, ni * 128);
}

// ====================================================== few tokens
// As the bf16 kernel of few tokens: the codes of w go from memory into the registers of a
// warp-level product (16 weight rows x 8 tokens x 32).  A lane's 16-byte loads are its
// fragments: of 64 consecutive codes of a row, lane 4 g + t holds 16 t .. 16 t + 15 of
// row g, the first 8 of them in one instruction and the others in the next; any order of
// the contraction does, as long as both operands count it alike.  Tokens in bf16 are
// quantised on the way by every warp that multiplies them: the four lanes of a token
// hold a whole 1 x 128 block of it.  One token at 2048 x 7168 6.2 us, with its codes given
// 5.1 (14.7 MB, 2.9 TB/s): bound by the launch and one trip to memory.
__device__ __forceinline__ uint4 ld_codes(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void warp_mma_f8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT: groups of 8 tokens; G: K blocks that a warp asks for at once.
template <int NT, bool CODES, int G>
__global__ void __launch_bounds__(kStreamWarps * 32)
    fp8_stream_kernel(const __grid_constant__ Fp8StreamArgs a) {
  constexpr int TOK = 8 * NT;
  pdl_launch_dependents();
  __shared__ float s_part[kStreamWarps][TOK][17];
  __shared__ float s_sum[kStreamWarps][TOK][16];  // of a tile, over this block's warps
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int wpr = a.wpr, S = a.split, rank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tiles = kStreamWarps / wpr;  // of a block
  const int tile0 = blockIdx.x / S * tiles, part = rank * wpr + warp % wpr;
  const int n0 = (tile0 + warp / wpr) * 16;
  const int N = a.epi.N, T = a.epi.M, KB = a.KB;
  pdl_wait();
  float sum[NT][4] = {};
  if (n0 < N) {
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const bool on0 = n0 + g < N, on1 = n0 + 8 + g < N;
    const uint8_t* w0 = a.w + static_cast<long>(n0 + g) * a.ld_w + 16 * t;
    const uint8_t* w1 = w0 + 8 * a.ld_w;
    const long wbase = static_cast<long>(n0 / kB) * KB;  // 16 rows lie in one scale block
#pragma unroll 1
    for (int kb0 = part * G; kb0 < KB; kb0 += wpr * S * G) {
      uint4 wv[G][2][2];
      float sw[G];
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const bool in = kb0 + j < KB;
        const long k = static_cast<long>(kb0 + j) * kB;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          wv[j][h][0] = on0 && in ? ld_codes(w0 + k + 64 * h) : zero;
          wv[j][h][1] = on1 && in ? ld_codes(w1 + k + 64 * h) : zero;
        }
        sw[j] = in ? scale_at(a.sc.w, wbase + kb0 + j, a.sc.ue8m0) : 0.f;
      }
#pragma unroll
      for (int j = 0; j < G; ++j) {
        if (kb0 + j >= KB) break;  // the same for the whole warp
        const long k = static_cast<long>(kb0 + j) * kB + 16 * t;
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          const int tok = 8 * q + g;
          uint4 xc[2] = {zero, zero};
          float sx = 0.f;
          if (CODES) {
            if (tok < T) {
              const uint8_t* x = static_cast<const uint8_t*>(a.x) + tok * a.ld_x + k;
              xc[0] = __ldg(reinterpret_cast<const uint4*>(x));
              xc[1] = __ldg(reinterpret_cast<const uint4*>(x + 64));
              sx = scale_at(a.sc.x, tok * a.sc.x_row + (kb0 + j) * a.sc.x_kb, a.sc.ue8m0);
            }
          } else {
            uint4 v[4] = {zero, zero, zero, zero};
            if (tok < T) {
              const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x) + tok * a.ld_x + k;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                v[i] = __ldg(reinterpret_cast<const uint4*>(x + 64 * (i >> 1) + 8 * (i & 1)));
            }
            uint32_t m = __vmaxu2(__vmaxu2(amax8(v[0]), amax8(v[1])), __vmaxu2(amax8(v[2]), amax8(v[3])));
            m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
            uint32_t stored;
            sx = row_scale(amax_value(m), a.sc.ue8m0 != 0, &stored);
            const float inv = 1.0f / sx;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint2 lo = codes8(v[2 * h], inv), hi = codes8(v[2 * h + 1], inv);
              xc[h] = make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
          }
          float c[4] = {};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 lo = wv[j][h][0], hi = wv[j][h][1], x = xc[h];
            warp_mma_f8(c, lo.x, hi.x, lo.y, hi.y, x.x, x.y);
            warp_mma_f8(c, lo.z, hi.z, lo.w, hi.w, x.z, x.w);
          }
          // a lane's sums: rows g and g + 8, tokens 2 t and 2 t + 1 of each 8
          const float s0 = sw[j] * __shfl_sync(0xffffffffu, sx, 8 * t);
          const float s1 = sw[j] * __shfl_sync(0xffffffffu, sx, 8 * t + 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[q][i] = fmaf(c[i], i & 1 ? s1 : s0, sum[q][i]);
        }
      }
    }
  }
#pragma unroll
  for (int q = 0; q < NT; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) s_part[warp][8 * q + 2 * t + (i & 1)][g + 8 * (i >> 1)] = sum[q][i];
  __syncthreads();
  stream_results<TOK, false>(a.epi, s_part, s_sum, wpr, S, rank, tiles, tile0, N, T);
}

template <int ACT, bool F32>
cudaError_t launch_pair(const CUtensorMap& tm_a, const CUtensorMap& tm_b, Fp8LinearDev p, cudaStream_t s) {
  auto kern = fp8_pair_kernel<ACT, F32>;
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
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static std::atomic<int> max_clusters[64] = {};
  int nc = max_clusters[dev].load(std::memory_order_acquire);
  if (nc == 0) {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
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

template <int ACT>
cudaError_t launch_pair_act(const CUtensorMap& tm_a, const CUtensorMap& tm_b, const Fp8LinearDev& p,
                            cudaStream_t s) {
  return p.epi.out_f32 ? launch_pair<ACT, true>(tm_a, tm_b, p, s) : launch_pair<ACT, false>(tm_a, tm_b, p, s);
}

cudaError_t launch_tile(const CUtensorMap& tm_a, const CUtensorMap& tm_b, Fp8LinearDev p, int split,
                        cudaStream_t s) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64) return cudaErrorInvalidDevice;
  static std::atomic<int> ready[64] = {};
  if (!ready[dev].load(std::memory_order_acquire)) {
    err = cudaFuncSetAttribute(fp8_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTSmem);
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
  err = cudaLaunchKernelEx(&cfg, fp8_tile_kernel, tm_a, tm_b, p);
  count_launches(1);
  return err != cudaSuccess ? err : cudaGetLastError();
}

template <int NT, bool CODES, int G>
cudaError_t launch_stream(Fp8StreamArgs a, int num_sms, cudaStream_t s) {
  // warps of a block per tile until every SM has 16, then two blocks, as long as each has a
  // group of the contraction (8 tokens at 7168 x 2112: one block 10.9 us, two 8.4, up to
  // eight 11.1; at 2048 x 7168 8 warps 6.5 us, 4 warps 8.5)
  const long tiles = ceil_div(a.epi.N, 16);
  a.wpr = a.split = 1;
  while (a.wpr < kStreamWarps && tiles * a.wpr < 16l * num_sms && a.wpr * G < a.KB) a.wpr *= 2;
  if (tiles * a.wpr < 16l * num_sms && a.wpr * G < a.KB) a.split = 2;
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
  return cudaLaunchKernelEx(&cfg, fp8_stream_kernel<NT, CODES, G>, a);
}
template <bool CODES>
cudaError_t launch_stream_tokens(const Fp8StreamArgs& a, int num_sms, cudaStream_t s) {
  // 8 tokens and a long contraction: four K blocks at once, 8.4 us against 9.8 at 7168 x 2112
  // (at 2048 x 7168, where a warp has two, 7.8 against 6.5; 16 tokens 12.9 against 11.0)
  if (a.epi.M <= 8)
    return a.KB >= 32 ? launch_stream<1, CODES, 4>(a, num_sms, s) : launch_stream<1, CODES, 2>(a, num_sms, s);
  if constexpr (CODES)
    return a.epi.M <= 16 ? launch_stream<2, CODES, 2>(a, num_sms, s) : launch_stream<4, CODES, 2>(a, num_sms, s);
  return cudaErrorInvalidValue;  // more bf16 tokens come with their codes made before
}

}  // namespace

// As linear_path: pairs from half a wave of their tiles, below it 128 x 128 tiles with the
// contraction split until the grid covers the GPU, each part at least two K blocks long.
LinearPath fp8_path(long M, long N, long K, int num_sms) {
  LinearPath r;
  const long big = static_cast<long>(ceil_div(M, 256)) * ceil_div(N, 256);
  const long pairs = std::min(num_sms, kLinearMaxParts / 2) / 2;
  r.split = 1;
  if (big >= pairs / 2) {
    r.kind = LinearPath::kPair;
    return r;
  }
  r.kind = LinearPath::kTile;
  const long tiles = static_cast<long>(ceil_div(M, 128)) * ceil_div(N, 128);
  while (r.split < 4 && tiles * r.split * 2 <= 2 * pairs && K / (r.split * 2) >= 2 * kB) r.split *= 2;
  return r;
}

// How many of the last rows the kernel of few tokens takes: up to 16 beyond whole row tiles,
// where their tiles would begin another wave of pairs and a second reading of all weights costs
// less than that wave, whose time grows with K alone, the reading's with N and the rows too.
// With and without, us, 1 | 16 rows beyond whole tiles:
//   K 7168   N 2112 51, 68 | 54, 68   4096 58, 68 | 62, 68   7168 65, 68 | 73, 68
//            N 18432 95, 70 | 105, 70   36864 171, 128 | 208, 128
//   K 4096   N 2112 42, 48 | 42, 48   4096 42, 48 | 49, 48
//   K 2048   N 1024 32, 36 | 36, 36   4096 31, 33 | 36, 33 (8 rows 33, 33)   7168 31, 33 | 36, 33
//   K 512    N 2112 23, 21 | 27, 21   4096 25, 21 | 27, 21   (a launch is more than the wave)
//   K 16384  N 4096 101, 134 | 109, 134   9216 124, 134 | 136, 134   18432 170, 136 | 197, 136
// So up to 4096 columns and from a contraction of 2048 on, from 4096 on for more than 8 rows: no
// size was slower by more than the timer's step of 1 us.
int fp8_rest(int T, int N, int K, const LinearPath& path, int num_sms) {
  const int rest = T % 256, pairs = std::max(num_sms / 2, 1);
  if (path.kind != LinearPath::kPair || T < 256 || N > 4096 || K < 2048 || rest == 0 ||
      rest > (K < 4096 ? 8 : 16))
    return 0;
  const long nt = ceil_div(N, 256), tiles = (T / 256 + 1) * nt;
  return (tiles - nt + pairs - 1) / pairs < (tiles + pairs - 1) / pairs ? rest : 0;
}

cudaError_t launch_fp8_linear(const CUtensorMap& tm_x, const CUtensorMap& tm_w, const Fp8LinearDev& p,
                              const LinearPath& path, cudaStream_t s) {
  const long parts = static_cast<long>(path.split) * ceil_div(p.epi.M, 128) * ceil_div(p.epi.N, 128);
  if (path.kind == LinearPath::kSums || (path.kind == LinearPath::kPair && path.split != 1) ||
      (path.split != 1 && path.split != 2 && path.split != 4 && path.split != 8) ||
      (path.split > 1 && (path.split > p.KB || parts > kLinearMaxParts)))
    return cudaErrorInvalidValue;
  if (path.kind == LinearPath::kTile) return launch_tile(tm_x, tm_w, p, path.split, s);
  if (p.epi.act == MOE_ACT_SILU) return launch_pair_act<MOE_ACT_SILU>(tm_x, tm_w, p, s);
  if (p.epi.act == MOE_ACT_GELU) return launch_pair_act<MOE_ACT_GELU>(tm_x, tm_w, p, s);
  if (p.epi.act == MOE_ACT_RELU) return launch_pair_act<MOE_ACT_RELU>(tm_x, tm_w, p, s);
  return launch_pair_act<MOE_ACT_NONE>(tm_x, tm_w, p, s);
}

bool fp8_streams(int T, int N) { return T <= 16 || (T <= 32 && N <= 1024); }

cudaError_t launch_fp8_stream(const Fp8StreamArgs& a, int num_sms, cudaStream_t s) {
  const cudaError_t e = a.codes ? launch_stream_tokens<true>(a, num_sms, s)
                                : launch_stream_tokens<false>(a, num_sms, s);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_fp8_rows(const Fp8RowsArgs& a, cudaStream_t s) {
  const cudaError_t e = launch_pdl(fp8_rows_kernel, dim3(ceil_div(a.T, 32), ceil_div(a.KB, 4)), dim3(256), 0, s, a);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
