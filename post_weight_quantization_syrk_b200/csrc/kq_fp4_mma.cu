// kq_fp4_gemm: Y = A B^T of two microscaled 4-bit matrices, and
// kq_fp4_gated_ffn: H = act(X Wg^T) * (X Wu^T) over such operands, on the
// block-scaled tcgen05 kinds (see kq_mma.cuh).  Products and block scales are
// applied in the tensor core, sums are fp32 in TMEM.
//
// Measured (2MNK flops): 8192 x 11008 x 4096 MX 134 us (5.5 PFLOP/s, tensor pipe 71 %
// active), NV 143; x 16384 467 (6.3 PFLOP/s) and 506; gated 8192 x 4096 x 11008 MX 261, NV
// 281.  Back to back on random data the power limit lowers the clock: up to 158, 168, 561,
// 617, 317 and 331.  At long K a stage takes 0.37 us of which the MMAs
// are 0.27 (ring of 5 stages, the loads' latency and the copies of the scales; with 4
// stages 0.39); at K = 4096 a tile's read-out, which no MMA overlaps, adds an eighth.
// 77 x 4096 x 4096 with the quantization of the 77 rows: 11.5 us; 8 x 11008 x 4096 MX 10.2;
// gated 16 x 4096 x 11008: 18.8 us, 2.7 TB/s of weights.
#include "kq_fp4.cuh"
#include "kq_mma.cuh"

namespace {

using namespace kq::mma;

// Tensor maps of the codes (box: 128 bytes x rows) and of the scale tiles
// (rows of 128 words; box: the tiles of one stage).
kq_status codes_map(CUtensorMap* m, const kq_fp4* q, int box_rows) {
  return make_map_2d(m, q->codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, kq::cdiv(q->cols, 32) * 16, q->rows, q->ld, 128, box_rows,
                     CU_TENSOR_MAP_SWIZZLE_128B);
}
kq_status scales_map(CUtensorMap* m, const kq_fp4* q, int atoms) {
  const int64_t tiles = kq::cdiv(q->rows, 128) * kq::fp4::scale_tiles(q->cols, q->format);
  return make_map_2d(m, q->scales, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, 128, tiles, 128, 128, atoms, CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <int KIND, int EPI>
using Pair = Cfg<KIND, 2, 256, false, false, EPI, 5>;
template <int KIND, int EPI>
using Slim = Cfg<KIND, 1, 128, false, false, EPI, 6>;   // 128 columns, or 64 features

template <class C>
kq_status run(const char* what, const kq_fp4* A, const kq_fp4* B0, const kq_fp4* B1, Params p, int ks, cudaStream_t st) {
  Maps m;
  p.a_rows = C::CG == 2 ? 128 : (int)std::min<int64_t>(128, kq::cdiv(p.M, 8) * 8);
  KQ_TRY(codes_map(&m.a[0], A, p.a_rows));
  m.a[1] = m.a[0];
  const int box_b = C::DUAL ? C::BN / 2 : C::BN / C::CG;
  KQ_TRY(codes_map(&m.b[0], B0, box_b));
  KQ_TRY(scales_map(&m.sfa, A, C::ATOMS));
  KQ_TRY(scales_map(&m.sfb[0], B0, C::ATOMS));
  m.b[1] = m.b[0];
  m.sfb[1] = m.sfb[0];
  if (B1) {
    KQ_TRY(codes_map(&m.b[1], B1, box_b));
    KQ_TRY(scales_map(&m.sfb[1], B1, C::ATOMS));
  }
  p.tiles_m = (int)kq::cdiv(p.M, 128 * C::CG);
  p.tiles_n = (int)kq::cdiv(p.N, C::OUTC);
  p.num_tiles = p.problem_tiles = p.tiles_m * p.tiles_n;
  p.steps = (int)kq::cdiv(A->cols, 64);
  p.kblocks = p.seg_blocks = (int)kq::cdiv(A->cols, 256);
  p.kat = (int)kq::fp4::scale_tiles(A->cols, A->format);
  p.ks = ks;
  return launch<C>(what, m, p, st);
}

template <int KIND, int EPI>
kq_status choose(const char* what, const kq_fp4* A, const kq_fp4* B0, const kq_fp4* B1, const Params& p, cudaStream_t st) {
  constexpr bool MX = KIND == KIND_MX;
  constexpr Cost cost = EPI == EPI_STORE ? Cost{0.42, MX ? 0.36 : 0.38, 1.2, 1.2} : Cost{0.54, MX ? 0.35 : 0.37, 1.6, 1.6};
  const Plan plan = make_plan(p.M, kq::cdiv(p.M, 128) * kq::cdiv(p.N, Slim<KIND, EPI>::OUTC),
                              kq::cdiv(p.M, 256) * kq::cdiv(p.N, Pair<KIND, EPI>::OUTC), kq::cdiv(A->cols, 256), cost);
  if (plan.pair) return run<Pair<KIND, EPI>>(what, A, B0, B1, p, 1, st);
  return run<Slim<KIND, EPI>>(what, A, B0, B1, p, plan.ks, st);
}

// Longest K: the tensor core truncates as it accumulates, up to 2^-24 of the sum per
// MMA of 64 columns: over 2^20 columns 2^-10, a quarter of what a rounding to bf16 may lose.
constexpr int64_t kMaxCols = 1 << 20;

}  // namespace

extern "C" kq_status kq_fp4_gemm(const kq_fp4* A, const kq_fp4* B, void* Y, int dtype, int64_t ldy, int32_t* info,
                                 kq_stream_t stream) {
  KQ_TRY(kq::fp4::check(A, "kq_fp4_gemm", "A"));
  KQ_TRY(kq::fp4::check(B, "kq_fp4_gemm", "B"));
  if (A->format != B->format || A->cols != B->cols)
    return kq::fail(KQ_ERR_INVALID_ARG, "kq_fp4_gemm: A and B need the same format and columns");
  if (A->cols > kMaxCols) return kq::fail(KQ_ERR_UNSUPPORTED_SHAPE, "kq_fp4_gemm: more than 2^20 columns");
  if (dtype != KQ_F32 && dtype != KQ_BF16) return kq::fail(KQ_ERR_INVALID_ARG, "kq_fp4_gemm: dtype must be KQ_F32 or KQ_BF16");
  if (!info) return kq::fail(KQ_ERR_INVALID_ARG, "kq_fp4_gemm: NULL pointer");
  if (A->rows == 0 || B->rows == 0) {
    kq::clear_error();
    return KQ_OK;
  }
  if (!Y) return kq::fail(KQ_ERR_INVALID_ARG, "kq_fp4_gemm: NULL pointer");
  if (ldy < B->rows) return kq::fail(KQ_ERR_INVALID_ARG, "kq_fp4_gemm: leading dimension too small");
  const size_t esize = dtype == KQ_F32 ? 4 : 2;
  if (!kq::aligned(Y, esize)) return kq::fail(KQ_ERR_ALIGNMENT, "kq_fp4_gemm: Y aligned to its elements");
  if (kq::cdiv(A->rows, 128) * kq::cdiv(B->rows, 64) > (1 << 24))
    return kq::fail(KQ_ERR_UNSUPPORTED_SHAPE, "kq_fp4_gemm: more than 2^24 tiles of 128 x 64");
  Params p = {};
  p.M = A->rows;
  p.N = B->rows;
  p.out_f32 = dtype == KQ_F32;
  p.out[0] = Y;
  p.ldo[0] = ldy;
  p.out_vec[0] = kq::aligned(Y, 16) && (ldy * (int64_t)esize) % 16 == 0;
  p.ga = A->gscale;
  p.gb[0] = p.gb[1] = B->gscale;
  p.info = info;
  p.wait_ns = kq::wait_limit_ns();
  cudaStream_t st = (cudaStream_t)stream;
  if (A->format == KQ_FP4_MX)
    KQ_TRY((choose<KIND_MX, EPI_STORE>("kq_fp4_gemm", A, B, nullptr, p, st)));
  else
    KQ_TRY((choose<KIND_NV, EPI_STORE>("kq_fp4_gemm", A, B, nullptr, p, st)));
  kq::clear_error();
  return KQ_OK;
}

extern "C" kq_status kq_fp4_gated_ffn(const kq_fp4* X, const kq_fp4* W_gate, const kq_fp4* W_up, int act, uint16_t* H,
                                      int64_t ldh, int32_t* info, kq_stream_t stream) {
  KQ_TRY(kq::fp4::check(X, "kq_fp4_gated_ffn", "X"));
  KQ_TRY(kq::fp4::check(W_gate, "kq_fp4_gated_ffn", "W_gate"));
  KQ_TRY(kq::fp4::check(W_up, "kq_fp4_gated_ffn", "W_up"));
  if (X->format != W_gate->format || X->format != W_up->format || X->cols != W_gate->cols || X->cols != W_up->cols ||
      W_gate->rows != W_up->rows)
    return kq::fail(KQ_ERR_INVALID_ARG, "kq_fp4_gated_ffn: X, W_gate and W_up need the same format and columns, the weights the same rows");
  if (X->cols > kMaxCols) return kq::fail(KQ_ERR_UNSUPPORTED_SHAPE, "kq_fp4_gated_ffn: more than 2^20 columns");
  if (act != KQ_ACT_SILU && act != KQ_ACT_GELU) return kq::fail(KQ_ERR_INVALID_ARG, "kq_fp4_gated_ffn: unknown activation");
  if (!info) return kq::fail(KQ_ERR_INVALID_ARG, "kq_fp4_gated_ffn: NULL pointer");
  if (X->rows == 0 || W_gate->rows == 0) {
    kq::clear_error();
    return KQ_OK;
  }
  if (!H) return kq::fail(KQ_ERR_INVALID_ARG, "kq_fp4_gated_ffn: NULL pointer");
  if (ldh < W_gate->rows) return kq::fail(KQ_ERR_INVALID_ARG, "kq_fp4_gated_ffn: leading dimension too small");
  if (!kq::aligned(H, 2)) return kq::fail(KQ_ERR_ALIGNMENT, "kq_fp4_gated_ffn: H aligned to its elements");
  if (kq::cdiv(X->rows, 128) * kq::cdiv(W_gate->rows, 64) > (1 << 24))
    return kq::fail(KQ_ERR_UNSUPPORTED_SHAPE, "kq_fp4_gated_ffn: more than 2^24 tiles of 128 x 64");
  Params p = {};
  p.M = X->rows;
  p.N = W_gate->rows;
  p.act = act;
  p.out[0] = H;
  p.ldo[0] = ldh;
  p.out_vec[0] = kq::aligned(H, 16) && ldh % 8 == 0;
  p.ga = X->gscale;
  p.gb[0] = W_gate->gscale;
  p.gb[1] = W_up->gscale;
  p.info = info;
  p.wait_ns = kq::wait_limit_ns();
  cudaStream_t st = (cudaStream_t)stream;
  if (X->format == KQ_FP4_MX)
    KQ_TRY((choose<KIND_MX, EPI_GATED>("kq_fp4_gated_ffn", X, W_gate, W_up, p, st)));
  else
    KQ_TRY((choose<KIND_NV, EPI_GATED>("kq_fp4_gated_ffn", X, W_gate, W_up, p, st)));
  kq::clear_error();
  return KQ_OK;
}
