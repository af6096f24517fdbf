// C-ABI entry points of the operators around the experts (scored routing,
// block norms, linear): argument validation, tensor maps, kernel choice.
// Nothing here throws or allocates device memory; every error is a status.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstring>
#include <initializer_list>
#include <mutex>
#include <type_traits>
#include <utility>

#include "moe_internal.h"

using namespace moe;

namespace moe {

moe_status cuda_error(cudaError_t e, const char* what) {
  return set_last_error(MOE_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e),
                        cudaGetErrorString(e));
}

int device_sms() {
  static std::atomic<int> sms[64] = {};
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return 152;
  n = sms[dev].load(std::memory_order_relaxed);
  if (n) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 152;
  sms[dev].store(n, std::memory_order_relaxed);
  return n;
}

bool ptr_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

namespace {
moe_status make_map_2d(CUtensorMap* m, CUtensorMapDataType type, uint64_t size, const void* base,
                       uint64_t inner, uint64_t outer, uint64_t ld, uint32_t box_inner,
                       uint32_t box_outer) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  if (!fn)
    return set_last_error(MOE_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {ld * size};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(m, type, 2, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return set_last_error(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return MOE_OK;
}
}  // namespace

moe_status make_map_bf16_2d(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer,
                            uint64_t ld, uint32_t box_inner, uint32_t box_outer) {
  return make_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, inner, outer, ld, box_inner, box_outer);
}
moe_status make_map_u8_2d(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer,
                          uint64_t ld) {
  return make_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, base, inner, outer, ld, 128, 128);
}

}  // namespace moe

namespace {

bool is_dtype(int dt) { return dt == MOE_DT_BF16 || dt == MOE_DT_F32; }
int size_of(int dt) { return dt == MOE_DT_F32 ? 4 : 2; }

// Row starts of a 16-byte aligned buffer stay 16-byte aligned.
bool rows16(int64_t ld, int size) { return ld * size % 16 == 0; }

template <typename... P>
bool all16(P... p) {
  return (ptr_aligned(p, 16) && ...);
}

moe_status check_route(const char* fn, int dt, int64_t ld, int T, int E, int k, int score) {
  if (T < 0) return set_last_error(MOE_ERR_INVALID_ARG, "%s: negative size", fn);
  if (E < 1 || E > kMaxE)
    return set_last_error(MOE_ERR_UNSUPPORTED, "%s: E must be in [1, %d]", fn, kMaxE);
  if (k < 1 || k > E || k > kMaxK)
    return set_last_error(MOE_ERR_UNSUPPORTED, "%s: k must be in [1, min(E, %d)]", fn, kMaxK);
  if (!is_dtype(dt)) return set_last_error(MOE_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, dt);
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: unknown score %d", fn, score);
  if (ld < E) return set_last_error(MOE_ERR_INVALID_ARG, "%s: row stride below E", fn);
  return MOE_OK;
}

moe_status check_gate(const char* fn, const void* gate, int kind, int dt, int64_t ld, int H) {
  if (kind < MOE_GATE_NONE || kind > MOE_GATE_ELEMENT)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: unknown gate kind %d", fn, kind);
  if ((kind == MOE_GATE_NONE) != (gate == nullptr))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: gate and gate_kind disagree", fn);
  if (kind != MOE_GATE_NONE && !is_dtype(dt))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: unknown gate dtype %d", fn, dt);
  if (kind == MOE_GATE_ELEMENT && ld < H)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: gate row stride below H", fn);
  return MOE_OK;
}

moe_status check_ws(const char* fn, const void* ws, size_t have, size_t need) {
  if (!ws) return set_last_error(MOE_ERR_INVALID_ARG, "%s: null workspace", fn);
  if (!ptr_aligned(ws, 256))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: ws must be 256-byte aligned", fn);
  if (have < need)
    return set_last_error(MOE_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", fn, have, need);
  return MOE_OK;
}

// A matrix in memory: rows of `width` bytes, `pitch` bytes apart.
struct Region {
  const void* p;
  int64_t rows, width, pitch;
};
Region matrix_at(const void* p, int64_t rows, int64_t cols, int64_t ld, int size) {
  return {p, rows, cols * size, rows > 1 ? ld * size : cols * size};
}
Region vector_at(const void* p, int64_t n, int size) { return {p, 1, n * size, n * size}; }
// Scales of any two positive strides: rows or columns where these lie apart from each other,
// else everything between the first scale and the last.
Region scales_at(const void* p, int64_t rows, int64_t cols, int64_t s_row, int64_t s_col, int size) {
  const int64_t row = (cols - 1) * s_col + 1, col = (rows - 1) * s_row + 1;
  if (rows == 1 || s_row >= row) return matrix_at(p, rows, row, s_row, size);
  if (cols == 1 || s_col >= col) return matrix_at(p, cols, col, s_col, size);
  return vector_at(p, (rows - 1) * s_row + row, size);
}
int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b != 0 && (a < 0) != (b < 0)); }

// Whether two of them have a byte in common; one may lie between the columns of another.
bool overlap(const Region& a, const Region& b) {
  if (!a.p || !b.p || a.rows < 1 || b.rows < 1 || a.width < 1 || b.width < 1) return false;
  const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.p)) -
                    static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.p));
  const int64_t a_end = (a.rows - 1) * a.pitch + a.width, b_end = (b.rows - 1) * b.pitch + b.width;
  if (d >= a_end || d + b_end <= 0) return false;
  if (a.rows == 1 && b.rows == 1) return true;
  // row j of b meets row i of a where -b.width < d + j b.pitch - i a.pitch < a.width
  if (a.rows == 1 || b.rows == 1 || a.pitch == b.pitch) {  // by k = j - i
    const int64_t pitch = a.rows == 1 ? b.pitch : a.pitch;
    const int64_t first = std::max(floor_div(-b.width - d, pitch) + 1, 1 - a.rows);
    const int64_t last = std::min(floor_div(a.width - d - 1, pitch), b.rows - 1);
    return first <= last;
  }
  if (a.rows > b.rows) return overlap(b, a);
  for (int64_t i = 0; i < a.rows; ++i) {
    const int64_t at = d - i * a.pitch;
    const int64_t first = std::max<int64_t>(floor_div(-b.width - at, b.pitch) + 1, 0);
    if (first < b.rows && at + first * b.pitch < a.width) return true;
  }
  return false;
}
// Results share no memory with operands nor with each other.
moe_status check_apart(const char* fn, std::initializer_list<Region> results,
                       std::initializer_list<Region> operands) {
  for (const Region& r : results) {
    bool shared = false;
    for (const Region& o : operands) shared = shared || overlap(r, o);
    for (const Region& o : results) shared = shared || (&o != &r && overlap(r, o));
    if (shared) return set_last_error(MOE_ERR_INVALID_ARG, "%s: results need buffers of their own", fn);
  }
  return MOE_OK;
}

bool is_act(int act) {
  return act == MOE_ACT_NONE || act == MOE_ACT_SILU || act == MOE_ACT_GELU || act == MOE_ACT_RELU;
}

moe_status check_linear(const char* fn, int64_t ld_x, int64_t ld_w, int act, int T, int K, int N) {
  if (T < 0 || N < 0) return set_last_error(MOE_ERR_INVALID_ARG, "%s: negative size", fn);
  if (!is_act(act)) return set_last_error(MOE_ERR_INVALID_ARG, "%s: unknown activation %d", fn, act);
  if (K < 8 || K % 8)
    return set_last_error(MOE_ERR_UNSUPPORTED, "%s: K must be a positive multiple of 8", fn);
  if (ld_x < K || ld_w < K)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: row stride below K", fn);
  if (ld_x % 8 || ld_w % 8)
    return set_last_error(MOE_ERR_UNSUPPORTED, "%s: row strides must be multiples of 8", fn);
  return MOE_OK;
}

// One product D = A B^T.  a_rows, b_rows: rows of D and its columns; an
// MN-major operand lies in memory as [K, rows], the other kind as [rows, K].
moe_status run_linear(const void* a, int64_t ld_a, bool a_mn, const void* b, int64_t ld_b,
                      bool b_mn, const LinearDev& p, cudaStream_t s, const char* what) {
  const int M = p.epi.M, N = p.epi.N, K = p.K;
  const LinearPath path = linear_path(M, N, K, p.epi.out_f32, device_sms());
  const uint32_t lines = path.kind == LinearPath::kTile ? 64 : 128;  // contraction lines of an MN-major box
  CUtensorMap ta, tb;
  moe_status st = a_mn ? make_map_bf16_2d(&ta, a, M, K, ld_a, 64, lines)
                       : make_map_bf16_2d(&ta, a, K, M, ld_a, 64, 128);
  if (st != MOE_OK) return st;
  st = b_mn ? make_map_bf16_2d(&tb, b, N, K, ld_b, 64, lines)
            : make_map_bf16_2d(&tb, b, K, N, ld_b, 64, 128);
  if (st != MOE_OK) return st;
  const cudaError_t e = launch_linear(ta, tb, p, a_mn, b_mn, path, s);
  return e == cudaSuccess ? MOE_OK : cuda_error(e, what);
}

// The gated product x [T, K] by w [2 I, K].
moe_status run_gated(const void* x, int64_t ld_x, const void* w, int64_t ld_w, const LinearDev& p,
                     cudaStream_t s, const char* what) {
  const int T = p.epi.M, I = p.epi.N, K = p.K;
  const LinearPath path = gated_path(T, I, K, device_sms());
  CUtensorMap tx, tw;
  moe_status st = make_map_bf16_2d(&tx, x, K, T, ld_x, 64, 128);
  if (st != MOE_OK) return st;
  st = make_map_bf16_2d(&tw, w, K, 2ull * I, ld_w, 64, path.kind == LinearPath::kTile ? 64 : 128);
  if (st != MOE_OK) return st;
  const cudaError_t e = launch_gated(tx, tw, p, path, s);
  return e == cudaSuccess ? MOE_OK : cuda_error(e, what);
}

struct LinearWs {
  int64_t ld_dz;
  size_t dz, dz_lo, partials, total;
};
// dz is rounded to bf16 for the products of the gradient.  Over many dz that adds
// to the error of a gradient what its own rounding to bf16 does, 1.41 times in
// all.  Of a few dz the roundings do not average out: the squares of n rounding
// errors, of normal gradients times silu's slope, have a mean that varies by 3.4
// / sqrt(n) of itself, so 24 dz leave 1.35 times in the median of draws and 2.1
// in one of a hundred, 256 dz 1.6 and 1024 dz 1.5.  So up to this many dz the rest
// of the rounding is kept too and multiplied first, in two more small products,
// and the gradients are as those of an fp32 dz; beyond, 1.41 within 7 %.
constexpr int64_t kLinearDzSplit = 1024;
LinearWs linear_ws(int T, int N) {
  LinearWs w;
  w.ld_dz = (static_cast<int64_t>(N) + 7) / 8 * 8;
  w.dz = kLinearWsBytes;
  const size_t bytes = static_cast<size_t>(T) * w.ld_dz * 2;
  const bool split = static_cast<int64_t>(T) * N <= kLinearDzSplit;
  w.dz_lo = w.dz + (bytes + 15) / 16 * 16;
  w.partials = (w.dz_lo + (split ? bytes : 0) + 1023) / 1024 * 1024;
  w.total = w.partials + static_cast<size_t>(kLinearDzSlices) * N * 4;
  return w;
}

// The products of a gradient: dx = dz w and dw = dz^T x for dz [T, N] in bf16, dz_lo what
// its rounding left or null.
moe_status gradient_products(const void* dz, const void* dz_lo, int64_t ld_dz, const void* x,
                             int64_t ld_x, const void* w, int64_t ld_w, int T, int K, int N,
                             void* dx, void* dw, uint8_t* wsb, cudaStream_t s, const char* fn) {
  LinearEpi e{};
  e.act = MOE_ACT_NONE;
  e.ld_out = K;
  e.N = K;
  e.vec = true;  // K % 8 == 0
  LinearDev p{};
  p.err = reinterpret_cast<int*>(wsb);
  p.parts = reinterpret_cast<float*>(wsb + 1024);
  e.ld_res = K;
  // dz_lo's product first, then dz's on top of it
  auto product = [&](void* out, int M, int contraction, bool a_mn, const void* b, int64_t ld_b) {
    e.M = M;
    e.out = out;
    p.K = contraction;
    moe_status r = MOE_OK;
    if (dz_lo) {
      e.residual = nullptr;
      p.epi = e;
      r = run_linear(dz_lo, ld_dz, a_mn, b, ld_b, true, p, s, fn);
      if (r != MOE_OK) return r;
    }
    e.residual = dz_lo ? out : nullptr;
    p.epi = e;
    return run_linear(dz, ld_dz, a_mn, b, ld_b, true, p, s, fn);
  };
  moe_status st = MOE_OK;
  if (dx && (st = product(dx, T, N, false, w, ld_w)) != MOE_OK) return st;
  if (dw && (st = product(dw, N, T, true, x, ld_x)) != MOE_OK) return st;
  return MOE_OK;
}

constexpr int kGatedMaxI = (1 << 30) - 1;  // 2 I is an int
moe_status check_gated(const char* fn, int64_t ld_x, int64_t ld_w, int act, int T, int K, int I) {
  if (act == MOE_ACT_NONE)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: a gate has an activation", fn);
  if (I > kGatedMaxI) return set_last_error(MOE_ERR_UNSUPPORTED, "%s: I above 2^30 - 1", fn);
  return check_linear(fn, ld_x, ld_w, act, T, K, I);
}

moe_status check_fp8(const char* fn, int64_t ld_x, int align, int T, int K, int scale_fmt) {
  if (T < 0) return set_last_error(MOE_ERR_INVALID_ARG, "%s: negative size", fn);
  if (K < 128 || K % 128)
    return set_last_error(MOE_ERR_UNSUPPORTED, "%s: K must be a positive multiple of 128", fn);
  if (scale_fmt != MOE_SCALE_F32 && scale_fmt != MOE_SCALE_UE8M0)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: unknown scale format %d", fn, scale_fmt);
  if (ld_x < K) return set_last_error(MOE_ERR_INVALID_ARG, "%s: row stride below K", fn);
  if (ld_x % align)
    return set_last_error(MOE_ERR_UNSUPPORTED, "%s: row strides must be multiples of 16 bytes", fn);
  return MOE_OK;
}

bool scale_aligned(const void* p, int fmt) { return ptr_aligned(p, fmt == MOE_SCALE_F32 ? 4 : 1); }

struct Fp8Ws {
  size_t codes, scales, total;
};
Fp8Ws fp8_ws(int T, int K) {
  Fp8Ws w;
  w.codes = kLinearWsBytes;
  w.scales = w.codes + (static_cast<size_t>(T) * K + 1023) / 1024 * 1024;
  w.total = w.scales + static_cast<size_t>(T) * ((K / 128 + 3) / 4 * 4) * 4;
  return w;
}
// Up to this many tokens the kernel that streams the weights quantises them itself.
constexpr int kFp8QuantiseOnTheWay = 8;

}  // namespace

namespace {

// A call's arguments in 8-byte slots, in the function's order.
struct Packed {
  const unsigned char* block;
  template <typename T>
  T slot(size_t i) const {
    if constexpr (std::is_floating_point_v<T>) {
      double v;
      memcpy(&v, block + 8 * i, 8);
      return static_cast<T>(v);
    } else {
      int64_t v;
      memcpy(&v, block + 8 * i, 8);
      if constexpr (std::is_pointer_v<T>) return reinterpret_cast<T>(static_cast<uintptr_t>(v));
      else return static_cast<T>(v);
    }
  }
  // an int's slot holds a value that an int can
  template <typename T>
  bool fits(size_t i) const {
    return !std::is_same_v<T, int> || slot<int64_t>(i) == slot<int>(i);
  }
  template <typename... A, size_t... I>
  moe_status call(moe_status (*fn)(A...), std::index_sequence<I...>) const {
    if (!(fits<A>(I) && ...))
      return set_last_error(MOE_ERR_UNSUPPORTED, "moe_call_packed: a size above 2^31 - 1");
    return fn(slot<A>(I)...);
  }
  template <typename... A>
  moe_status call(moe_status (*fn)(A...)) const {
    return call(fn, std::index_sequence_for<A...>{});
  }
};

}  // namespace

extern "C" {

moe_status moe_route_scored(const void* logits, moe_dtype dt, int64_t ld_logits, int T, int E,
                            int k, moe_score score, const float* bias, int n_group,
                            int topk_group, int group_top, int renormalise, float scale,
                            int32_t* topk_idx, float* topk_w, void* stream) {
  const char* fn = "moe_route_scored";
  moe_status st = check_route(fn, dt, ld_logits, T, E, k, score);
  if (st != MOE_OK) return st;
  if (n_group < 1 || n_group > 32 || E % n_group)
    return set_last_error(MOE_ERR_UNSUPPORTED, "%s: n_group must be in [1, 32] and divide E", fn);
  if (topk_group < 1 || topk_group > n_group || topk_group * (E / n_group) < k)
    return set_last_error(MOE_ERR_UNSUPPORTED,
                          "%s: topk_group must be in [1, n_group] and its groups hold k experts", fn);
  if (group_top != 1 && group_top != 2)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: group_top must be 1 or 2", fn);
  if (T == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_w)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!all16(logits, bias, topk_idx, topk_w))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: buffers must be 16-byte aligned", fn);
  RouteScoredArgs a;
  a.logits = logits;
  a.ld = ld_logits;
  a.bias = bias;
  a.T = T;
  a.E = E;
  a.k = k;
  a.n_group = n_group;
  a.topk_group = topk_group;
  a.group_top = group_top;
  a.softmax = score == MOE_SCORE_SOFTMAX;
  a.renorm = renormalise != 0;
  a.vec = ld_logits % 4 == 0 && E % 4 == 0;
  a.scale = scale;
  a.idx = topk_idx;
  a.w = topk_w;
  const cudaError_t e =
      launch_route_scored(a, dt == MOE_DT_BF16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_error(e, fn);
}

moe_status moe_route_scored_backward(const void* logits, moe_dtype dt, int64_t ld_logits, int T,
                                     int E, int k, moe_score score, const float* bias,
                                     int renormalise, float scale, const int32_t* topk_idx,
                                     const float* topk_w, const float* grad_w,
                                     void* grad_logits, int64_t ld_grad, void* stream) {
  const char* fn = "moe_route_scored_backward";
  moe_status st = check_route(fn, dt, ld_logits, T, E, k, score);
  if (st != MOE_OK) return st;
  if (ld_grad < E) return set_last_error(MOE_ERR_INVALID_ARG, "%s: row stride below E", fn);
  if (T == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_w || !grad_w || !grad_logits)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!all16(logits, bias, topk_idx, topk_w, grad_w, grad_logits))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: buffers must be 16-byte aligned", fn);
  RouteScoredBwdArgs a;
  a.logits = logits;
  a.ld = ld_logits;
  a.idx = topk_idx;
  a.w = topk_w;
  a.grad_w = grad_w;
  a.bias = bias;
  a.T = T;
  a.E = E;
  a.k = k;
  a.softmax = score == MOE_SCORE_SOFTMAX;
  a.renorm = renormalise != 0;
  const bool whole = E * size_of(dt) % 16 == 0;
  a.vec = ld_logits % 4 == 0 && E % 4 == 0;
  a.vec_out = rows16(ld_grad, size_of(dt)) && whole;
  a.scale = scale;
  a.grad_logits = grad_logits;
  a.ldo = ld_grad;
  const cudaError_t e =
      launch_route_scored_backward(a, dt == MOE_DT_BF16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_error(e, fn);
}

moe_status moe_block_norm(const void* residual, moe_dtype res_dt, int64_t ld_res, const void* y,
                          int64_t ld_y, const void* gate, moe_gate gate_kind, moe_dtype gate_dt,
                          int64_t ld_gate, float scale, int post_norm, const void* post_weight,
                          int pre_norm, const void* pre_weight, moe_dtype weight_dt, float eps,
                          int T, int H, void* residual_out, void* normed, void* stream) {
  const char* fn = "moe_block_norm";
  if (T < 0) return set_last_error(MOE_ERR_INVALID_ARG, "%s: negative size", fn);
  if (H < 1 || H > kNormMaxH)
    return set_last_error(MOE_ERR_UNSUPPORTED, "%s: H must be in [1, %d]", fn, kNormMaxH);
  if (!is_dtype(res_dt) || !is_dtype(weight_dt))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: unknown dtype", fn);
  if (T == 0) return MOE_OK;  // before the pointers: empty buffers may have none
  moe_status st = check_gate(fn, gate, gate_kind, gate_dt, ld_gate, H);
  if (st != MOE_OK) return st;
  if (!y && (gate || post_norm || post_weight))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: a gate or norm of the block needs y", fn);
  if ((!post_norm && post_weight) || (!pre_norm && pre_weight))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: weight of a norm that is off", fn);
  if (!y && !pre_norm) return set_last_error(MOE_ERR_INVALID_ARG, "%s: nothing to compute", fn);
  if (ld_res < H || (y && ld_y < H))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: row stride below H", fn);
  if (!residual || (y && !residual_out) || (pre_norm != 0) != (normed != nullptr))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (residual_out == residual && y && ld_res != H)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: in place only where the row stride is H", fn);
  if (!all16(residual, y, gate, post_weight, pre_weight, residual_out, normed))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: buffers must be 16-byte aligned", fn);
  BlockNormArgs a;
  a.residual = residual;
  a.y = y;
  a.gate = gate;
  a.post_weight = post_weight;
  a.pre_weight = pre_weight;
  a.residual_out = residual_out;
  a.normed = normed;
  a.ld_res = ld_res;
  a.ld_y = ld_y;
  a.ld_gate = ld_gate;
  a.T = T;
  a.H = H;
  a.gate_kind = gate_kind;
  a.gate_bf16 = gate_dt == MOE_DT_BF16;
  a.weight_bf16 = weight_dt == MOE_DT_BF16;
  a.post_norm = post_norm != 0;
  a.pre_norm = pre_norm != 0;
  a.scale = scale;
  a.eps = eps;
  const bool vec = H % 8 == 0 && ld_res % 8 == 0 && (!y || ld_y % 8 == 0) &&
                   (gate_kind != MOE_GATE_ELEMENT || ld_gate % 8 == 0);
  const cudaError_t e =
      launch_block_norm(a, res_dt == MOE_DT_BF16, vec, device_sms(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_error(e, fn);
}

size_t moe_block_norm_backward_workspace_size(int H) {
  return H < 1 ? 0 : 1024 + static_cast<size_t>(kNormBwdBlocks) * 3 * H * 4;
}

moe_status moe_block_norm_backward(const void* grad_residual, int64_t ld_gres,
                                   const void* grad_normed, int64_t ld_gn, const void* residual,
                                   moe_dtype res_dt, int64_t ld_res, const void* y, int64_t ld_y,
                                   const void* gate, moe_gate gate_kind, moe_dtype gate_dt,
                                   int64_t ld_gate, float scale, int post_norm,
                                   const void* post_weight, const void* pre_weight,
                                   moe_dtype weight_dt, float eps, int T, int H,
                                   void* d_residual, void* d_y, void* d_gate,
                                   float* d_post_weight, float* d_pre_weight, void* ws,
                                   size_t ws_bytes, void* stream) {
  const char* fn = "moe_block_norm_backward";
  if (T < 0) return set_last_error(MOE_ERR_INVALID_ARG, "%s: negative size", fn);
  if (H < 1 || H > kNormMaxH)
    return set_last_error(MOE_ERR_UNSUPPORTED, "%s: H must be in [1, %d]", fn, kNormMaxH);
  if (!is_dtype(res_dt) || !is_dtype(weight_dt))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: unknown dtype", fn);
  if (T == 0) {  // before the pointers: empty buffers may have none
    void* sums[3] = {d_post_weight, d_pre_weight, gate_kind == MOE_GATE_CHANNEL ? d_gate : nullptr};
    for (void* p : sums) {
      const cudaError_t e = p ? cudaMemsetAsync(p, 0, static_cast<size_t>(H) * 4,
                                                static_cast<cudaStream_t>(stream))
                              : cudaSuccess;
      if (e != cudaSuccess) return cuda_error(e, fn);
    }
    return MOE_OK;
  }
  moe_status st = check_gate(fn, gate, gate_kind, gate_dt, ld_gate, H);
  if (st != MOE_OK) return st;
  if (!y && (gate || post_norm || post_weight || d_y || d_gate || d_post_weight))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: a gate or norm of the block needs y", fn);
  if (!post_norm && (post_weight || d_post_weight))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: weight of a norm that is off", fn);
  if (!grad_normed && (pre_weight || d_pre_weight))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: pre_weight without grad_normed", fn);
  if (!grad_normed && !grad_residual)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: no gradient given", fn);
  if ((grad_residual && ld_gres < H) || (grad_normed && (ld_gn < H || ld_res < H)) ||
      (y && ld_y < H))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: row stride below H", fn);
  if (d_residual && d_residual == grad_residual && ld_gres != H)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: in place only where the row stride is H", fn);
  if ((st = check_ws(fn, ws, ws_bytes, moe_block_norm_backward_workspace_size(H))) != MOE_OK)
    return st;
  if ((y && !d_y) || (gate && !d_gate) || (grad_normed && !residual))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!all16(grad_residual, grad_normed, residual, y, gate, post_weight, pre_weight, d_residual, d_y,
             d_gate, d_post_weight, d_pre_weight))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: buffers must be 16-byte aligned", fn);
  BlockNormBwdArgs a;
  a.grad_res = grad_residual;
  a.grad_normed = grad_normed;
  a.residual = residual;
  a.y = y;
  a.gate = gate;
  a.post_weight = post_weight;
  a.pre_weight = pre_weight;
  a.d_res = d_residual;
  a.d_y = d_y;
  a.d_gate = d_gate;
  a.d_post = d_post_weight;
  a.d_pre = d_pre_weight;
  a.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 1024);
  a.ld_gres = ld_gres;
  a.ld_gn = ld_gn;
  a.ld_res = ld_res;
  a.ld_y = ld_y;
  a.ld_gate = ld_gate;
  a.T = T;
  a.H = H;
  a.gate_kind = gate_kind;
  a.n_part = (d_pre_weight != nullptr) + (d_post_weight != nullptr) + (gate_kind == MOE_GATE_CHANNEL);
  a.gate_bf16 = gate_dt == MOE_DT_BF16;
  a.weight_bf16 = weight_dt == MOE_DT_BF16;
  a.post_norm = post_norm != 0;
  a.scale = scale;
  a.eps = eps;
  const bool vec = H % 8 == 0 && (!grad_residual || ld_gres % 8 == 0) &&
                   (!grad_normed || (ld_gn % 8 == 0 && ld_res % 8 == 0)) &&
                   (!y || ld_y % 8 == 0) && (gate_kind != MOE_GATE_ELEMENT || ld_gate % 8 == 0);
  const cudaError_t e = launch_block_norm_backward(a, res_dt == MOE_DT_BF16, vec, device_sms(),
                                                   static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_error(e, fn);
}

moe_status moe_linear(const void* x, int64_t ld_x, const void* w, int64_t ld_w, const void* bias,
                      moe_dtype bias_dt, int act, const void* residual, int64_t ld_res, int T,
                      int K, int N, void* out, moe_dtype out_dt, int64_t ld_out, void* preact,
                      void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "moe_linear";
  moe_status st = check_linear(fn, ld_x, ld_w, act, T, K, N);
  if (st != MOE_OK) return st;
  if (!is_dtype(out_dt) || (bias && !is_dtype(bias_dt)))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: unknown dtype", fn);
  if (ld_out < N || (residual && ld_res < N))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: row stride below N", fn);
  if (T == 0 || N == 0) return MOE_OK;
  if (!x || !w || !out) return set_last_error(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (residual == out && ld_res != ld_out)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: in place only with the same row stride", fn);
  if (preact && (preact == out || preact == residual))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: preact needs a buffer of its own", fn);
  if (!all16(x, w, bias, residual, out, preact))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: buffers must be 16-byte aligned", fn);
  if ((st = check_ws(fn, ws, ws_bytes, kLinearWsBytes)) != MOE_OK) return st;
  LinearEpi e;
  e.bias = bias;
  e.residual = residual;
  e.out = out;
  e.preact = preact;
  e.ld_res = ld_res;
  e.ld_out = ld_out;
  e.M = T;
  e.N = N;
  e.act = act;
  e.bias_bf16 = bias_dt == MOE_DT_BF16;
  e.out_f32 = out_dt == MOE_DT_F32;
  e.vec = N % 8 == 0 && rows16(ld_out, size_of(out_dt)) &&
          (!residual || rows16(ld_res, size_of(out_dt)));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (linear_streams(T, N)) {
    LinearStreamArgs g;
    g.x = static_cast<const __nv_bfloat16*>(x);
    g.w = static_cast<const __nv_bfloat16*>(w);
    g.ld_x = ld_x;
    g.ld_w = ld_w;
    g.K = K;
    g.epi = e;
    const cudaError_t r = launch_linear_stream(g, device_sms(), s);
    return r == cudaSuccess ? MOE_OK : cuda_error(r, fn);
  }
  LinearDev p;
  p.epi = e;
  p.K = K;
  p.split = 1;
  p.group = 0;
  p.err = static_cast<int*>(ws);
  p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 1024);
  return run_linear(x, ld_x, false, w, ld_w, false, p, s, fn);
}

size_t moe_linear_workspace_size(void) { return kLinearWsBytes; }

size_t moe_linear_backward_workspace_size(int T, int N) {
  return T < 0 || N < 0 ? 0 : linear_ws(T, N).total;
}

moe_status moe_linear_backward(const void* grad_y, moe_dtype y_dt, int64_t ld_gy, const void* x,
                               int64_t ld_x, const void* w, int64_t ld_w, int act,
                               const void* preact, int64_t ld_z, int T, int K, int N, void* dx,
                               void* dw, float* dbias, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "moe_linear_backward";
  moe_status st = check_linear(fn, ld_x, ld_w, act, T, K, N);
  if (st != MOE_OK) return st;
  if (!is_dtype(y_dt)) return set_last_error(MOE_ERR_INVALID_ARG, "%s: unknown dtype", fn);
  if ((act == MOE_ACT_NONE) != (preact == nullptr) && T > 0 && N > 0)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: an activation and its preact go together", fn);
  if (ld_gy < N || (preact && ld_z < N))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: row stride below N", fn);
  if (N == 0) {
    if (dx && T > 0) {
      const cudaError_t e = cudaMemsetAsync(dx, 0, static_cast<size_t>(T) * K * 2,
                                            static_cast<cudaStream_t>(stream));
      if (e != cudaSuccess) return cuda_error(e, fn);
    }
    return MOE_OK;
  }
  if (!all16(grad_y, x, w, preact, dx, dw, dbias))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: buffers must be 16-byte aligned", fn);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    cudaError_t e = cudaSuccess;
    if (dw) e = cudaMemsetAsync(dw, 0, static_cast<size_t>(N) * K * 2, s);
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, static_cast<size_t>(N) * 4, s);
    return e == cudaSuccess ? MOE_OK : cuda_error(e, fn);
  }
  if (!grad_y || (dx && !w) || (dw && !x))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
  const LinearWs L = linear_ws(T, N);
  if ((st = check_ws(fn, ws, ws_bytes, L.total)) != MOE_OK) return st;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  // dz is grad_y itself where that is bf16 with 16-byte rows and no
  // activation; otherwise it is written, rows padded to 8, by the pass that
  // sums its columns
  const bool direct = act == MOE_ACT_NONE && y_dt == MOE_DT_BF16 && ld_gy % 8 == 0 && N % 8 == 0;
  const bool products = dx || dw;
  // exact in bf16: a bf16 gradient times 0 or 1
  const bool exact = y_dt == MOE_DT_BF16 && (act == MOE_ACT_NONE || act == MOE_ACT_RELU);
  const bool split = products && !exact && static_cast<int64_t>(T) * N <= kLinearDzSplit;
  const void* dz = grad_y;
  const void* dz_lo = nullptr;
  int64_t ld_dz = ld_gy;
  if (!(direct || !products) || dbias) {
    LinearDzArgs a;
    a.dy = grad_y;
    a.preact = preact;
    a.dz = direct || !products ? nullptr : reinterpret_cast<__nv_bfloat16*>(wsb + L.dz);
    a.dz_lo = split ? reinterpret_cast<__nv_bfloat16*>(wsb + L.dz_lo) : nullptr;
    a.ld_dy = ld_gy;
    a.ld_z = ld_z;
    a.ld_dz = L.ld_dz;
    a.T = T;
    a.N = N;
    a.act = act;
    a.f32 = y_dt == MOE_DT_F32;
    a.vec = N % 8 == 0 && rows16(ld_gy, size_of(y_dt)) && (!preact || rows16(ld_z, size_of(y_dt)));
    const int slices = std::min(linear_dz_slices(T, N, device_sms()), kLinearDzSlices);
    a.partials = !dbias ? nullptr : slices == 1 ? dbias : reinterpret_cast<float*>(wsb + L.partials);
    const cudaError_t e = launch_linear_dz(a, slices, dbias, s);
    if (e != cudaSuccess) return cuda_error(e, fn);
    dz_lo = a.dz_lo;
    if (a.dz) {
      dz = a.dz;
      ld_dz = L.ld_dz;
    }
  }
  return gradient_products(dz, dz_lo, ld_dz, x, ld_x, w, ld_w, T, K, N, dx, dw, wsb, s, fn);
}

moe_status moe_gated_linear(const void* x, int64_t ld_x, const void* w, int64_t ld_w,
                            const void* bias, moe_dtype bias_dt, int act, int T, int K, int I,
                            void* out, int64_t ld_out, void* preact, void* ws, size_t ws_bytes,
                            void* stream) {
  const char* fn = "moe_gated_linear";
  moe_status st = check_gated(fn, ld_x, ld_w, act, T, K, I);
  if (st != MOE_OK) return st;
  if (bias && !is_dtype(bias_dt))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: unknown dtype", fn);
  if (ld_out < I) return set_last_error(MOE_ERR_INVALID_ARG, "%s: row stride below I", fn);
  if (T == 0 || I == 0) return MOE_OK;
  if (!x || !w || !out) return set_last_error(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!all16(x, w, bias, out, preact))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: buffers must be 16-byte aligned", fn);
  if ((st = check_ws(fn, ws, ws_bytes, kLinearWsBytes)) != MOE_OK) return st;
  if ((st = check_apart(fn, {matrix_at(out, T, I, ld_out, 2), vector_at(preact, T * 2ll * I, 2)},
                        {matrix_at(x, T, K, ld_x, 2), matrix_at(w, 2ll * I, K, ld_w, 2),
                         vector_at(bias, 2ll * I, size_of(bias_dt))})) != MOE_OK)
    return st;
  LinearEpi e{};
  e.bias = bias;
  e.out = out;
  e.preact = preact;
  e.ld_out = ld_out;
  e.M = T;
  e.N = I;
  e.act = act;
  e.bias_bf16 = bias_dt == MOE_DT_BF16;
  e.vec = I % 8 == 0 && ld_out % 8 == 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (linear_streams(T, 2 * I)) {
    LinearStreamArgs g;
    g.x = static_cast<const __nv_bfloat16*>(x);
    g.w = static_cast<const __nv_bfloat16*>(w);
    g.ld_x = ld_x;
    g.ld_w = ld_w;
    g.K = K;
    g.epi = e;
    const cudaError_t r = launch_gated_stream(g, device_sms(), s);
    return r == cudaSuccess ? MOE_OK : cuda_error(r, fn);
  }
  LinearDev p;
  p.epi = e;
  p.K = K;
  p.split = 1;
  p.group = 0;
  p.err = static_cast<int*>(ws);
  p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 1024);
  return run_gated(x, ld_x, w, ld_w, p, s, fn);
}

size_t moe_gated_linear_backward_workspace_size(int T, int I) {
  return T < 0 || I < 0 || I > kGatedMaxI ? 0 : linear_ws(T, 2 * I).total;
}

moe_status moe_gated_linear_backward(const void* grad_h, int64_t ld_gh, const void* x, int64_t ld_x,
                                     const void* w, int64_t ld_w, int act, const void* preact,
                                     int64_t ld_z, int T, int K, int I, void* dx, void* dw,
                                     float* dbias, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "moe_gated_linear_backward";
  moe_status st = check_gated(fn, ld_x, ld_w, act, T, K, I);
  if (st != MOE_OK) return st;
  if (ld_gh < I || ld_z < 2ll * I)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: row stride too small", fn);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int N = 2 * I;
  if (I == 0 || T == 0) {
    cudaError_t e = cudaSuccess;
    if (dx && T > 0) e = cudaMemsetAsync(dx, 0, static_cast<size_t>(T) * K * 2, s);
    if (e == cudaSuccess && dw && I > 0) e = cudaMemsetAsync(dw, 0, static_cast<size_t>(N) * K * 2, s);
    if (e == cudaSuccess && dbias && I > 0) e = cudaMemsetAsync(dbias, 0, static_cast<size_t>(N) * 4, s);
    return e == cudaSuccess ? MOE_OK : cuda_error(e, fn);
  }
  if (!grad_h || !preact || (dx && !w) || (dw && !x))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!all16(grad_h, x, w, preact, dx, dw, dbias))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: buffers must be 16-byte aligned", fn);
  const LinearWs L = linear_ws(T, N);
  if ((st = check_ws(fn, ws, ws_bytes, L.total)) != MOE_OK) return st;
  if ((st = check_apart(fn, {vector_at(dx, int64_t{T} * K, 2), vector_at(dw, int64_t{N} * K, 2), vector_at(dbias, N, 4)},
                        {matrix_at(grad_h, T, I, ld_gh, 2), matrix_at(x, T, K, ld_x, 2),
                         matrix_at(w, N, K, ld_w, 2), matrix_at(preact, T, N, ld_z, 2)})) != MOE_OK)
    return st;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  const bool products = dx || dw;
  if (!products && !dbias) return MOE_OK;
  LinearDzArgs a;
  a.dy = grad_h;
  a.preact = preact;
  a.dz = products ? reinterpret_cast<__nv_bfloat16*>(wsb + L.dz) : nullptr;
  a.dz_lo = products && static_cast<int64_t>(T) * N <= kLinearDzSplit
                ? reinterpret_cast<__nv_bfloat16*>(wsb + L.dz_lo) : nullptr;
  a.ld_dy = ld_gh;
  a.ld_z = ld_z;
  a.ld_dz = L.ld_dz;
  a.T = T;
  a.N = I;
  a.act = act;
  a.f32 = false;
  a.vec = I % 8 == 0 && ld_gh % 8 == 0 && ld_z % 8 == 0;
  const int slices = std::min(linear_dz_slices(T, I, device_sms()), kLinearDzSlices);
  a.partials = !dbias ? nullptr : slices == 1 ? dbias : reinterpret_cast<float*>(wsb + L.partials);
  const cudaError_t r = launch_gated_dz(a, slices, dbias, s);
  if (r != cudaSuccess) return cuda_error(r, fn);
  if (!products) return MOE_OK;
  return gradient_products(a.dz, a.dz_lo, L.ld_dz, x, ld_x, w, ld_w, T, K, N, dx, dw, wsb, s, fn);
}

moe_status moe_quantize_fp8_rows(const void* x, int64_t ld_x, int T, int K, moe_scale_fmt scale_fmt,
                                 void* q, void* scale, int64_t s_row, int64_t s_kb, void* stream) {
  const char* fn = "moe_quantize_fp8_rows";
  moe_status st = check_fp8(fn, ld_x, 8, T, K, scale_fmt);
  if (st != MOE_OK) return st;
  if (s_row < 1 || s_kb < 1)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: scale strides must be positive", fn);
  if (T == 0) return MOE_OK;
  if (!x || !q || !scale) return set_last_error(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!all16(x, q) || !scale_aligned(scale, scale_fmt))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: x and q must be 16-byte aligned, scales as their type", fn);
  if ((st = check_apart(fn, {vector_at(q, int64_t{T} * K, 1),
                             scales_at(scale, T, K / 128, s_row, s_kb, scale_fmt == MOE_SCALE_F32 ? 4 : 1)},
                        {matrix_at(x, T, K, ld_x, 2)})) != MOE_OK)
    return st;
  const cudaError_t e = launch_fp8_rows({static_cast<const __nv_bfloat16*>(x), static_cast<uint8_t*>(q),
                                         scale, ld_x, s_row, s_kb, T, K / 128,
                                         scale_fmt == MOE_SCALE_UE8M0},
                                        static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_error(e, fn);
}

size_t moe_linear_fp8_workspace_size(int T, int K) { return T < 0 || K < 0 ? 0 : fp8_ws(T, K).total; }

moe_status moe_linear_fp8(const void* x, int64_t ld_x, const void* x_scale, int64_t s_row, int64_t s_kb,
                          const void* w, int64_t ld_w, const void* w_scale,
                          moe_scale_fmt scale_fmt, const void* bias, moe_dtype bias_dt, int act,
                          const void* residual, int64_t ld_res, int T, int K, int N, void* out,
                          moe_dtype out_dt, int64_t ld_out, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "moe_linear_fp8";
  moe_status st = check_fp8(fn, ld_x, x_scale ? 16 : 8, T, K, scale_fmt);
  if (st != MOE_OK) return st;
  if (N < 0) return set_last_error(MOE_ERR_INVALID_ARG, "%s: negative size", fn);
  if (!is_act(act)) return set_last_error(MOE_ERR_INVALID_ARG, "%s: unknown activation %d", fn, act);
  if (!is_dtype(out_dt) || (bias && !is_dtype(bias_dt)))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: unknown dtype", fn);
  if (ld_w < K) return set_last_error(MOE_ERR_INVALID_ARG, "%s: row stride below K", fn);
  if (ld_w % 16)
    return set_last_error(MOE_ERR_UNSUPPORTED, "%s: row strides must be multiples of 16 bytes", fn);
  if (x_scale && (s_row < 1 || s_kb < 1))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: scale strides must be positive", fn);
  if (ld_out < N || (residual && ld_res < N))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: row stride below N", fn);
  if (T == 0 || N == 0) return MOE_OK;
  if (!x || !w || !w_scale || !out) return set_last_error(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (residual == out && ld_res != ld_out)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: in place only with the same row stride", fn);
  if (!all16(x, w, bias, residual, out) || !scale_aligned(x_scale, scale_fmt) ||
      !scale_aligned(w_scale, scale_fmt))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: buffers must be 16-byte aligned, scales as their type", fn);
  const Fp8Ws L = fp8_ws(T, K);
  if ((st = check_ws(fn, ws, ws_bytes, x_scale ? kLinearWsBytes : L.total)) != MOE_OK) return st;
  const int scale_size = scale_fmt == MOE_SCALE_F32 ? 4 : 1;
  if ((st = check_apart(fn, {matrix_at(out, T, N, ld_out, size_of(out_dt))},
                        {matrix_at(x, T, K, ld_x, x_scale ? 1 : 2), matrix_at(w, N, K, ld_w, 1),
                         scales_at(x_scale, T, K / 128, s_row, s_kb, scale_size),
                         vector_at(w_scale, (N + 127ll) / 128 * (K / 128), scale_size),
                         vector_at(bias, N, size_of(bias_dt)),
                         matrix_at(residual == out ? nullptr : residual, T, N, ld_res, size_of(out_dt))})) != MOE_OK)
    return st;
  uint8_t* const wsb = static_cast<uint8_t*>(ws);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  LinearEpi e{};
  e.bias = bias;
  e.residual = residual;
  e.out = out;
  e.ld_res = ld_res;
  e.ld_out = ld_out;
  e.M = T;
  e.N = N;
  e.act = act;
  e.bias_bf16 = bias_dt == MOE_DT_BF16;
  e.out_f32 = out_dt == MOE_DT_F32;
  e.vec = N % 8 == 0 && rows16(ld_out, size_of(out_dt)) &&
          (!residual || rows16(ld_res, size_of(out_dt)));
  Fp8Scales sc{x_scale, w_scale, s_row, s_kb, scale_fmt == MOE_SCALE_UE8M0};
  const int KB = K / 128;
  const bool streams = fp8_streams(T, N);
  if (!x_scale && !(streams && T <= kFp8QuantiseOnTheWay)) {
    // rows of scales padded to 4: a 16-byte load brings those of four K blocks
    const int64_t row = (KB + 3) / 4 * 4;
    const cudaError_t r = launch_fp8_rows({static_cast<const __nv_bfloat16*>(x), wsb + L.codes,
                                           wsb + L.scales, ld_x, row, 1, T, KB, sc.ue8m0 != 0}, s);
    if (r != cudaSuccess) return cuda_error(r, fn);
    x = wsb + L.codes;
    ld_x = K;
    sc.x = wsb + L.scales;
    sc.x_row = row;
    sc.x_kb = 1;
  }
  // rows t0 .. T by the kernel of few tokens
  auto stream_rows = [&](int64_t t0) {
    auto rows = [](const void* p, int64_t bytes) { return static_cast<const uint8_t*>(p) + bytes; };
    Fp8StreamArgs g;
    g.codes = sc.x != nullptr;
    g.x = rows(x, t0 * ld_x * (g.codes ? 1 : 2));
    g.w = static_cast<const uint8_t*>(w);
    g.ld_x = ld_x;
    g.ld_w = ld_w;
    g.sc = sc;
    if (sc.x) g.sc.x = rows(sc.x, t0 * sc.x_row * (sc.ue8m0 ? 1 : 4));
    g.KB = KB;
    g.wpr = g.split = 1;
    g.epi = e;
    g.epi.M = static_cast<int>(T - t0);
    g.epi.out = static_cast<uint8_t*>(out) + t0 * ld_out * size_of(out_dt);
    if (residual) g.epi.residual = rows(residual, t0 * ld_res * size_of(out_dt));
    const cudaError_t r = launch_fp8_stream(g, device_sms(), s);
    return r == cudaSuccess ? MOE_OK : cuda_error(r, fn);
  };
  if (streams) return stream_rows(0);
  const LinearPath path = fp8_path(T, N, K, device_sms());
  CUtensorMap tx, tw;
  if ((st = make_map_u8_2d(&tx, x, K, T, ld_x)) != MOE_OK) return st;
  if ((st = make_map_u8_2d(&tw, w, K, N, ld_w)) != MOE_OK) return st;
  Fp8LinearDev p;
  p.epi = e;
  p.sc = sc;
  p.KB = KB;
  p.split = 1;
  p.group = 0;
  p.parts = reinterpret_cast<float*>(wsb + 1024);
  p.err = static_cast<int*>(ws);
  const int rest = fp8_rest(T, N, K, path, device_sms());
  p.epi.M = T - rest;
  const cudaError_t r = launch_fp8_linear(tx, tw, p, path, s);
  if (r != cudaSuccess) return cuda_error(r, fn);
  return rest ? stream_rows(T - rest) : MOE_OK;
}

moe_status moe_layer_norm(const void* residual, moe_dtype res_dt, int64_t ld_res, const void* y,
                          int64_t ld_y, const void* weight, const void* bias, moe_dtype weight_dt,
                          float eps, int T, int H, void* residual_out, void* normed, void* stream) {
  const char* fn = "moe_layer_norm";
  if (T < 0) return set_last_error(MOE_ERR_INVALID_ARG, "%s: negative size", fn);
  if (H < 1 || H > kNormMaxH)
    return set_last_error(MOE_ERR_UNSUPPORTED, "%s: H must be in [1, %d]", fn, kNormMaxH);
  if (!is_dtype(res_dt) || !is_dtype(weight_dt))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: unknown dtype", fn);
  if (T == 0) return MOE_OK;  // before the pointers: empty buffers may have none
  if (ld_res < H || (y && ld_y < H))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: row stride below H", fn);
  if (!residual || (y && !residual_out) || !normed)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (residual_out == residual && y && ld_res != H)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: in place only where the row stride is H", fn);
  if (!all16(residual, y, weight, bias, residual_out, normed))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: buffers must be 16-byte aligned", fn);
  // in place: the same rows as residual's, which then are a result and no operand
  const Region res = matrix_at(residual, T, H, ld_res, size_of(res_dt));
  const moe_status st = check_apart(
      fn, {vector_at(y ? residual_out : nullptr, int64_t{T} * H, size_of(res_dt)), vector_at(normed, int64_t{T} * H, 2)},
      {y && residual_out == residual ? Region{} : res, matrix_at(y, T, H, ld_y, 2),
       vector_at(weight, H, size_of(weight_dt)), vector_at(bias, H, size_of(weight_dt))});
  if (st != MOE_OK) return st;
  LayerNormArgs a;
  a.residual = residual;
  a.y = y;
  a.weight = weight;
  a.bias = bias;
  a.residual_out = residual_out;
  a.normed = normed;
  a.ld_res = ld_res;
  a.ld_y = ld_y;
  a.T = T;
  a.H = H;
  a.weight_bf16 = weight_dt == MOE_DT_BF16;
  a.eps = eps;
  const bool vec = H % 8 == 0 && ld_res % 8 == 0 && (!y || ld_y % 8 == 0);
  const cudaError_t e =
      launch_layer_norm(a, res_dt == MOE_DT_BF16, vec, device_sms(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_error(e, fn);
}

size_t moe_layer_norm_backward_workspace_size(int H) {
  return H < 1 ? 0 : 1024 + static_cast<size_t>(kNormBwdBlocks) * 2 * H * 4;
}

moe_status moe_layer_norm_backward(const void* grad_residual, int64_t ld_gres, const void* grad_normed,
                                   int64_t ld_gn, const void* residual, moe_dtype res_dt,
                                   int64_t ld_res, const void* weight, moe_dtype weight_dt, float eps,
                                   int T, int H, void* d_residual, void* d_y, float* d_weight,
                                   float* d_bias, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "moe_layer_norm_backward";
  if (T < 0) return set_last_error(MOE_ERR_INVALID_ARG, "%s: negative size", fn);
  if (H < 1 || H > kNormMaxH)
    return set_last_error(MOE_ERR_UNSUPPORTED, "%s: H must be in [1, %d]", fn, kNormMaxH);
  if (!is_dtype(res_dt) || !is_dtype(weight_dt))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: unknown dtype", fn);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {  // before the pointers: empty buffers may have none
    for (float* p : {d_weight, d_bias}) {
      const cudaError_t e = p ? cudaMemsetAsync(p, 0, static_cast<size_t>(H) * 4, s) : cudaSuccess;
      if (e != cudaSuccess) return cuda_error(e, fn);
    }
    return MOE_OK;
  }
  if ((grad_residual && ld_gres < H) || ld_gn < H || ld_res < H)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: row stride below H", fn);
  if (!grad_normed || !residual || !d_residual)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (d_residual == grad_residual && ld_gres != H)
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: in place only where the row stride is H", fn);
  moe_status st = check_ws(fn, ws, ws_bytes, moe_layer_norm_backward_workspace_size(H));
  if (st != MOE_OK) return st;
  if (!all16(grad_residual, grad_normed, residual, weight, d_residual, d_y, d_weight, d_bias))
    return set_last_error(MOE_ERR_INVALID_ARG, "%s: buffers must be 16-byte aligned", fn);
  // in place: as the forward pass; d_weight and d_bias are written after the last read of an operand
  const int64_t n = int64_t{T} * H;
  const int rs = size_of(res_dt);
  st = check_apart(fn, {vector_at(d_residual, n, rs), vector_at(d_y, n, 2)},
                   {d_residual == grad_residual ? Region{} : matrix_at(grad_residual, T, H, ld_gres, rs),
                    matrix_at(grad_normed, T, H, ld_gn, 2), matrix_at(residual, T, H, ld_res, rs),
                    vector_at(weight, H, size_of(weight_dt)), vector_at(d_weight, H, 4), vector_at(d_bias, H, 4)});
  if (st == MOE_OK) st = check_apart(fn, {vector_at(d_weight, H, 4), vector_at(d_bias, H, 4)}, {});
  if (st != MOE_OK) return st;
  LayerNormBwdArgs a;
  a.grad_res = grad_residual;
  a.grad_normed = grad_normed;
  a.residual = residual;
  a.weight = weight;
  a.d_res = d_residual;
  a.d_y = d_y;
  a.d_w = d_weight;
  a.d_b = d_bias;
  a.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 1024);
  a.ld_gres = ld_gres;
  a.ld_gn = ld_gn;
  a.ld_res = ld_res;
  a.T = T;
  a.H = H;
  a.n_part = (d_weight != nullptr) + (d_bias != nullptr);
  a.weight_bf16 = weight_dt == MOE_DT_BF16;
  a.eps = eps;
  const bool vec = H % 8 == 0 && (!grad_residual || ld_gres % 8 == 0) && ld_gn % 8 == 0 && ld_res % 8 == 0;
  const cudaError_t e = launch_layer_norm_backward(a, res_dt == MOE_DT_BF16, vec, device_sms(), s);
  return e == cudaSuccess ? MOE_OK : cuda_error(e, fn);
}

// The Python binding's way in: converting 14 to 29 arguments one by one took longer
// there than launching the kernel.
moe_status moe_call_packed(int call, const void* block) {
  if (block == nullptr)
    return set_last_error(MOE_ERR_INVALID_ARG, "moe_call_packed: null block");
  const Packed a{static_cast<const unsigned char*>(block)};
  switch (call) {
    case 0: return a.call(moe_route_scored);
    case 1: return a.call(moe_route_scored_backward);
    case 2: return a.call(moe_block_norm);
    case 3: return a.call(moe_block_norm_backward);
    case 4: return a.call(moe_linear);
    case 5: return a.call(moe_linear_backward);
    case 7: return a.call(moe_gated_linear);
    case 8: return a.call(moe_gated_linear_backward);
    case 9: return a.call(moe_quantize_fp8_rows);
    case 10: return a.call(moe_linear_fp8);
    case 11: return a.call(moe_layer_norm);
    case 12: return a.call(moe_layer_norm_backward);
  }
  return set_last_error(MOE_ERR_INVALID_ARG, "moe_call_packed: unknown call %d", call);
}

}  // extern "C"
