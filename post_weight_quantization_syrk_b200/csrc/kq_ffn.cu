// The gated feed-forward block in bf16, H = act(X Wg^T) * (X Wu^T)
// (kq_gated_ffn), and its backward pass (kq_gated_ffn_backward):
//   G = X Wg^T, U = X Wu^T (formed again, in fp32),
//   dU = dH act(G), dG = dH U act'(G),
//   dX = dG Wg + dU Wu, dWg = dG^T X, dWu = dU^T X.
// dG and dU are the output gradients of the gate and up linears, H the input of
// the down linear: the tensors whose covariances calibration takes.  Three
// launches of the tile engine (kq_mma.cuh): the gated product with dG, dU (and
// H) in its epilogue; dX with K running over both weights; both weight gradients
// in one grid.  dG and dU are rounded to bf16 once, as outputs, and the products
// take those (each rounding 2^-8 relative at most, as dX's own).
//
// Measured at 4096 x 4096 x 11008: forward 491 to 551 us (1.34 to 1.50 PFLOP/s, with the
// power limit; the tensor pipe is active 93 % of the cycles), backward 1.69 to 1.73 ms
// (1.28 to 1.31).  333 x 1001 x 2730 backward: 41.4 us, its three dependent launches of
// 12 to 15 us each bound by the length of a tile's chain of stages.  8 x 4096 x 11008
// forward: 36 us, the weights at 5.0 TB/s.
#include <algorithm>
#include <initializer_list>

#include "kq_mma.cuh"

namespace {

using namespace kq::mma;

kq_status bf16_map(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t ld, int box_rows) {
  return make_map_2d(m, base, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, cols, rows, ld, 64, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int EPI>
using GatedPair = Cfg<KIND_BF16, 2, 256, false, false, EPI, 6>;
template <int EPI>
using GatedSlim = Cfg<KIND_BF16, 1, 128, false, false, EPI, 6>;
using InputPair = Cfg<KIND_BF16, 2, 256, false, true, EPI_STORE, 6>;
using InputSlim = Cfg<KIND_BF16, 1, 128, false, true, EPI_STORE, 6>;
using WeightPair = Cfg<KIND_BF16, 2, 256, true, true, EPI_STORE, 6>;
using WeightSlim = Cfg<KIND_BF16, 1, 128, true, true, EPI_STORE, 6>;

template <class C>
kq_status go(const char* what, const Maps& m, Params p, int problems, int ks, cudaStream_t st) {
  p.tiles_m = (int)kq::cdiv(p.M, 128 * C::CG);
  p.tiles_n = (int)kq::cdiv(p.N, C::OUTC);
  p.problem_tiles = p.tiles_m * p.tiles_n;
  p.num_tiles = problems * p.problem_tiles;
  p.ks = ks;
  return launch<C>(what, m, p, st);
}

constexpr Cost kGated = {0.46, 0.38, 2.5, 0.5}, kStore = {0.36, 0.33, 2.5, 0.5};

struct Shape {
  int64_t T, d, f;
};

// The gated product: forward, or the backward pass's dG and dU.
template <int EPI>
kq_status gated(const char* what, const Shape& s, const uint16_t* X, int64_t ldx, const uint16_t* Wg, const uint16_t* Wu,
                int64_t ldw, Params p, cudaStream_t st) {
  p.M = s.T;
  p.N = s.f;
  p.kblocks = p.seg_blocks = (int)kq::cdiv(s.d, 64);
  const Plan plan = make_plan(s.T, kq::cdiv(s.T, 128) * kq::cdiv(s.f, 64), kq::cdiv(s.T, 256) * kq::cdiv(s.f, 128), p.kblocks, kGated);
  const bool pair = plan.pair;
  p.a_rows = pair ? 128 : (int)std::min<int64_t>(128, kq::cdiv(s.T, 8) * 8);
  Maps m;
  KQ_TRY(bf16_map(&m.a[0], X, s.d, s.T, ldx, p.a_rows));
  KQ_TRY(bf16_map(&m.b[0], Wg, s.d, s.f, ldw, pair ? 128 : 64));
  KQ_TRY(bf16_map(&m.b[1], Wu, s.d, s.f, ldw, pair ? 128 : 64));
  m.a[1] = m.sfa = m.sfb[0] = m.sfb[1] = m.a[0];
  if (pair) return go<GatedPair<EPI>>(what, m, p, 1, 1, st);
  return go<GatedSlim<EPI>>(what, m, p, 1, plan.ks, st);
}

kq_status check(const char* what, const Shape& s, const uint16_t* X, int64_t ldx, const uint16_t* Wg, const uint16_t* Wu,
                int64_t ldw, int act, const int32_t* info) {
  if (s.T < 0 || s.d < 1 || s.f < 1) return kq::fail(KQ_ERR_INVALID_ARG, "%s: need tokens >= 0, d >= 1, f >= 1", what);
  if (s.T > (1 << 24) || s.d > (1 << 17) || s.f > (1 << 17))
    return kq::fail(KQ_ERR_UNSUPPORTED_SHAPE, "%s: tokens above 2^24, or d or f above 2^17", what);
  if (kq::cdiv(s.T, 128) * kq::cdiv(std::max(s.d, s.f), 64) > (1 << 24))
    return kq::fail(KQ_ERR_UNSUPPORTED_SHAPE, "%s: more than 2^24 tiles of 128 x 64", what);
  if (act != KQ_ACT_SILU && act != KQ_ACT_GELU) return kq::fail(KQ_ERR_INVALID_ARG, "%s: unknown activation", what);
  if ((!X && s.T > 0) || !Wg || !Wu || !info) return kq::fail(KQ_ERR_INVALID_ARG, "%s: NULL pointer", what);
  if (ldx < s.d || ldw < s.d) return kq::fail(KQ_ERR_INVALID_ARG, "%s: leading dimension too small", what);
  if (!kq::aligned(X, 16) || !kq::aligned(Wg, 16) || !kq::aligned(Wu, 16) || (ldx & 7) || (ldw & 7))
    return kq::fail(KQ_ERR_ALIGNMENT, "%s: X and weights 16-byte aligned, leading dimensions %% 8 == 0", what);
  return KQ_OK;
}

// Outputs at the address of an input or of another output (views side by side in one
// tensor are fine).
kq_status distinct(const char* what, std::initializer_list<const void*> outs, std::initializer_list<const void*> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    if (!*o) continue;
    if (std::find(o + 1, outs.end(), *o) != outs.end() || std::find(ins.begin(), ins.end(), *o) != ins.end())
      return kq::fail(KQ_ERR_INVALID_ARG, "%s: an output is another tensor of the call", what);
  }
  return KQ_OK;
}

}  // namespace

extern "C" kq_status kq_gated_ffn(const uint16_t* X, int64_t tokens, int64_t d, int64_t ldx, const uint16_t* W_gate,
                                  const uint16_t* W_up, int64_t f, int64_t ldw, int act, uint16_t* H, int64_t ldh,
                                  int32_t* info, kq_stream_t stream) {
  const char* what = "kq_gated_ffn";
  const Shape s = {tokens, d, f};
  KQ_TRY(check(what, s, X, ldx, W_gate, W_up, ldw, act, info));
  if (tokens == 0) {
    kq::clear_error();
    return KQ_OK;
  }
  if (!H) return kq::fail(KQ_ERR_INVALID_ARG, "%s: NULL pointer", what);
  if (ldh < f) return kq::fail(KQ_ERR_INVALID_ARG, "%s: leading dimension too small", what);
  if (!kq::aligned(H, 2)) return kq::fail(KQ_ERR_ALIGNMENT, "%s: H aligned to its elements", what);
  KQ_TRY(distinct(what, {H}, {X, W_gate, W_up}));
  Params p = {};
  p.act = act;
  p.out[0] = H;
  p.ldo[0] = ldh;
  p.out_vec[0] = kq::aligned(H, 16) && ldh % 8 == 0;
  p.info = info;
  p.wait_ns = kq::wait_limit_ns();
  KQ_TRY(gated<EPI_GATED>(what, s, X, ldx, W_gate, W_up, ldw, p, (cudaStream_t)stream));
  kq::clear_error();
  return KQ_OK;
}

extern "C" kq_status kq_gated_ffn_backward(const uint16_t* X, int64_t tokens, int64_t d, int64_t ldx,
                                           const uint16_t* W_gate, const uint16_t* W_up, int64_t f, int64_t ldw, int act,
                                           const uint16_t* dH, int64_t lddh, uint16_t* dG, uint16_t* dU, int64_t ldg,
                                           uint16_t* H, int64_t ldh, uint16_t* dX, int64_t lddx, uint16_t* dW_gate,
                                           uint16_t* dW_up, int64_t lddw, int32_t* info, kq_stream_t stream) {
  const char* what = "kq_gated_ffn_backward";
  const Shape s = {tokens, d, f};
  KQ_TRY(check(what, s, X, ldx, W_gate, W_up, ldw, act, info));
  if (!dW_gate != !dW_up) return kq::fail(KQ_ERR_INVALID_ARG, "%s: dW_gate and dW_up go together", what);
  // The tensor core truncates as it accumulates, up to 2^-24 of the sum per MMA of 16
  // terms: a sum over 2^18 terms (tokens; or 2 f for dX) loses at most 2^-10, a quarter
  // of what rounding it to bf16 may.
  if (dW_gate && tokens > (1 << 18))
    return kq::fail(KQ_ERR_UNSUPPORTED_SHAPE, "%s: weights' gradients of more than 2^18 tokens (call it per batch and add)", what);
  if (tokens > 0 && (!dH || !dG || !dU)) return kq::fail(KQ_ERR_INVALID_ARG, "%s: NULL pointer", what);
  if (lddh < f || ldg < f || (H && ldh < f) || (dX && lddx < d) || (dW_gate && lddw < d))
    return kq::fail(KQ_ERR_INVALID_ARG, "%s: leading dimension too small", what);
  if (!kq::aligned(dG, 16) || !kq::aligned(dU, 16) || (ldg & 7))
    return kq::fail(KQ_ERR_ALIGNMENT, "%s: dG and dU 16-byte aligned, ldg %% 8 == 0", what);
  if (!kq::aligned(dH, 2) || !kq::aligned(H, 2) || !kq::aligned(dX, 2) || !kq::aligned(dW_gate, 2) || !kq::aligned(dW_up, 2))
    return kq::fail(KQ_ERR_ALIGNMENT, "%s: tensors aligned to their elements", what);
  if (2 * kq::cdiv(f, 128) * kq::cdiv(d, 128) > (1 << 24))
    return kq::fail(KQ_ERR_UNSUPPORTED_SHAPE, "%s: more than 2^24 tiles of 128 x 128", what);
  if (tokens > 0) KQ_TRY(distinct(what, {dG, dU, H, dX, dW_gate, dW_up}, {X, W_gate, W_up, dH}));
  cudaStream_t st = (cudaStream_t)stream;
  if (tokens == 0) {
    for (uint16_t* w : {dW_gate, dW_up})
      if (w) KQ_TRY(kq::cuda_check(cudaMemset2DAsync(w, lddw * 2, 0, d * 2, f, st), what));
    kq::clear_error();
    return KQ_OK;
  }
  {
    Params p = {};
    p.act = act;
    p.out[0] = dG;
    p.out[1] = dU;
    p.ldo[0] = p.ldo[1] = ldg;
    p.out_vec[0] = p.out_vec[1] = 1;
    p.h = reinterpret_cast<__nv_bfloat16*>(H);
    p.ldh = ldh;
    p.h_vec = kq::aligned(H, 16) && ldh % 8 == 0;
    p.dh = reinterpret_cast<const __nv_bfloat16*>(dH);
    p.lddh = lddh;
    p.dh_vec = kq::aligned(dH, 16) && lddh % 8 == 0;
    p.info = info;
    p.wait_ns = kq::wait_limit_ns();
    KQ_TRY(gated<EPI_GATED_BWD>(what, s, X, ldx, W_gate, W_up, ldw, p, st));
  }
  if (dX) {
    // dX [T, d] = [dG dU] [Wg; Wu]: K runs over f twice, the weights MN-major
    Params p = {};
    p.M = tokens;
    p.N = d;
    p.seg_blocks = (int)kq::cdiv(f, 64);
    p.kblocks = 2 * p.seg_blocks;
    p.out[0] = dX;
    p.ldo[0] = lddx;
    p.out_vec[0] = kq::aligned(dX, 16) && lddx % 8 == 0;
    p.info = info;
    p.wait_ns = kq::wait_limit_ns();
    const Plan plan = make_plan(tokens, kq::cdiv(tokens, 128) * kq::cdiv(d, 128), kq::cdiv(tokens, 256) * kq::cdiv(d, 256), p.kblocks, kStore);
    const bool pair = plan.pair;
    p.a_rows = pair ? 128 : (int)std::min<int64_t>(128, kq::cdiv(tokens, 8) * 8);
    Maps m;
    KQ_TRY(bf16_map(&m.a[0], dG, f, tokens, ldg, p.a_rows));
    KQ_TRY(bf16_map(&m.a[1], dU, f, tokens, ldg, p.a_rows));
    KQ_TRY(bf16_map(&m.b[0], W_gate, d, f, ldw, 64));
    KQ_TRY(bf16_map(&m.b[1], W_up, d, f, ldw, 64));
    m.sfa = m.sfb[0] = m.sfb[1] = m.a[0];
    if (pair)
      KQ_TRY(go<InputPair>(what, m, p, 1, 1, st));
    else
      KQ_TRY(go<InputSlim>(what, m, p, 1, plan.ks, st));
  }
  if (dW_gate) {
    // dWg [f, d] = dG^T X and dWu = dU^T X: two problems of one grid, K = tokens
    Params p = {};
    p.M = f;
    p.N = d;
    p.kblocks = p.seg_blocks = (int)kq::cdiv(tokens, 64);
    p.out[0] = dW_gate;
    p.out[1] = dW_up;
    p.ldo[0] = p.ldo[1] = lddw;
    p.out_vec[0] = kq::aligned(dW_gate, 16) && lddw % 8 == 0;
    p.out_vec[1] = kq::aligned(dW_up, 16) && lddw % 8 == 0;
    p.info = info;
    p.wait_ns = kq::wait_limit_ns();
    p.a_rows = 128;
    Maps m;
    KQ_TRY(bf16_map(&m.a[0], dG, f, tokens, ldg, 64));
    KQ_TRY(bf16_map(&m.a[1], dU, f, tokens, ldg, 64));
    KQ_TRY(bf16_map(&m.b[0], X, d, tokens, ldx, 64));
    m.b[1] = m.sfa = m.sfb[0] = m.sfb[1] = m.b[0];
    const Plan plan = make_plan(std::max<int64_t>(f, 65), 2 * kq::cdiv(f, 128) * kq::cdiv(d, 128), 2 * kq::cdiv(f, 256) * kq::cdiv(d, 256), p.kblocks, kStore);
    if (plan.pair)
      KQ_TRY(go<WeightPair>(what, m, p, 2, 1, st));
    else
      KQ_TRY(go<WeightSlim>(what, m, p, 2, plan.ks, st));
  }
  kq::clear_error();
  return KQ_OK;
}
