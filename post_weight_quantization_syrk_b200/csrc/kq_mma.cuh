// Tile engine of the 4-bit floating-point product and of the gated
// feed-forward block: D = A B^T on tcgen05 tensor cores with TMA-fed operands,
// fp32 accumulators in TMEM and a fused epilogue (internal).
//
// Operands.  kind::f16 (bf16, K or MN major), or the block-scaled kinds over
// e2m1 codes: kind::mxf4 (one E8M0 scale per 32 codes) and kind::mxf4nvf4 (one
// E4M3 scale per 16).  In all of them a pipeline stage holds 128 bytes of K
// per row (64 bf16 or 256 codes, four MMA steps of 32 bytes) in the 128-byte
// swizzle.  Scale bytes travel as whole 512-byte tiles (128 rows x 4 blocks,
// the layout that tcgen05.cp 32x128b.warpx4 takes), shared memory -> TMEM
// beside the MMAs that use them.
//
// Shapes.  CG = 2: a CTA pair per 256 x 256 tile (cta_group::2), each CTA
// holding 128 rows of A and of B, so an SM fetches 64 bytes per MMA cycle
// instead of the 96 of a single 128 x 256 CTA.  CG = 1: 128 x BN tiles for
// products with few rows, optionally with K split over a cluster of KS CTAs
// whose fp32 partials are summed in rank order through distributed shared
// memory (results do not depend on scheduling).
//
// Gated tiles hold the gate and the up columns of the same features side by
// side: with CG = 2 the pair's first CTA supplies the gate rows of B and the
// second the up rows; with CG = 1 two MMAs per step.  The epilogue then has
// both projections of a feature in one thread.
//
// Warp roles: 0 TMA, 1 TMEM and MMA issue, 2.. epilogue (one lane per row).
// Every mbarrier wait is bounded by a time limit; on expiry the kernel
// records KQ_ERR_TIMEOUT, drains its copies (bounded), frees TMEM and returns.
#pragma once

#include <cuda_bf16.h>

#include "kq_tc.cuh"

namespace kq {
namespace mma {

using namespace kq::tc;

enum { KIND_BF16 = 0, KIND_MX = 1, KIND_NV = 2 };
enum { EPI_STORE = 0, EPI_GATED = 1, EPI_GATED_BWD = 2 };

template <int KIND_, int CG_, int BN_, bool AMN_, bool BMN_, int EPI_, int STAGES_, int EW_>
struct Cfg {
  static constexpr int KIND = KIND_, CG = CG_, BN = BN_, EPI = EPI_, STAGES = STAGES_, EW = EW_;
  static constexpr bool AMN = AMN_, BMN = BMN_, FP4 = KIND != KIND_BF16, DUAL = EPI != EPI_STORE;
  static constexpr int NSUB = (CG == 1 && DUAL) ? 2 : 1;     // MMAs per K step
  static constexpr int MMA_N = BN / NSUB;
  static constexpr int OUTC = DUAL ? BN / 2 : BN;            // output columns of a tile
  static constexpr int A_BYTES = 128 * 128, B_BYTES = BN / CG * 128;
  static constexpr int ATOMS = KIND == KIND_MX ? 2 : (KIND == KIND_NV ? 4 : 0);   // scale tiles per stage and 128 rows
  static constexpr int SFB_TILES = DUAL ? 2 : (BN + 127) / 128;
  static constexpr int SFA_BYTES = ATOMS * 512, SFB_BYTES = SFB_TILES * ATOMS * 512;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
  static constexpr int SF_COLS = ATOMS * 4 * (1 + SFB_TILES);
  // scale buffers in TMEM: one per stage where they fit, else two (the MMA
  // thread then waits for the stage before last)
  static constexpr int NSF = !FP4 ? 0 : (CG == 2 ? STAGES : 2);
  static constexpr int NBUF = (CG == 2 && 2 * BN + NSF * SF_COLS <= 512) ? 2 : 1;  // accumulators
  static constexpr int COLS = NBUF * BN + NSF * SF_COLS;
  static constexpr int TMEM_COLS = COLS <= 64 ? 64 : (COLS <= 128 ? 128 : (COLS <= 256 ? 256 : 512));
  static_assert(COLS <= 512, "TMEM");
  static constexpr int THREADS = 64 + 32 * EW;
  static constexpr int PART_LD = BN + 4;                     // row stride of the split-K partials
  static constexpr int RING = STAGES * STAGE_BYTES;
  static constexpr int SMEM = RING + 1024 + 256;
  static_assert(SMEM <= 232448, "shared memory");
  static_assert(CG == 2 || 128 * PART_LD * 4 <= RING, "split-K partials reuse the ring");
};

struct Maps {
  CUtensorMap a[2], b[2], sfa, sfb[2];
};

struct Params {
  int64_t M, N;          // rows and output columns (features when gated)
  int tiles_m, tiles_n, num_tiles;   // num_tiles counts both problems
  int kblocks;           // stages of K in all
  int seg_blocks;        // stages of the first K segment (== kblocks with one segment)
  int steps;             // MMA steps that hold data (fp4: ceil(K / 64); bf16: 4 * kblocks)
  int problem_tiles;     // tiles of one problem; problem p uses a[p] and out[p]
  int a_rows;            // rows of the A box (CG = 1: no more than M needs)
  int kat;               // scale tiles along K per 128 rows
  int ks;                // CTAs sharing a tile along K (CG = 1)
  int act;
  int out_f32;
  void* out[2];          // store: Y of each problem; gated: H; backward: dG, dU
  int64_t ldo[2];
  int out_vec[2];        // rows can be stored 16 bytes at a time
  __nv_bfloat16* h;      // backward: H (may be NULL)
  int64_t ldh;
  int h_vec;
  const __nv_bfloat16* dh;
  int64_t lddh;
  int dh_vec;
  const float* ga;       // global scales of A and B (NULL: 1)
  const float* gb[2];
  int32_t* info;
  unsigned long long wait_ns;
};

// ------------------------------------------------------------------ PTX

__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// A TMA tile load; with CG = 2 the barrier may be the pair leader's.
template <int CG>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if constexpr (CG == 2) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  } else {
    tma_load_2d(dst, map, x, y, bar);
  }
}

template <int CG, int NCOLS>
__device__ __forceinline__ void alloc_tmem(uint32_t slot) {
  if constexpr (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "n"(NCOLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc<NCOLS>(slot);
  }
}
template <int CG, int NCOLS>
__device__ __forceinline__ void free_tmem(uint32_t taddr) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "n"(NCOLS) : "memory");
  else
    tmem_dealloc<NCOLS>(taddr);
}

// Arrive on `bar` (of both CTAs of a pair) once the MMAs and copies issued so far are done.
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  else
    mma_commit(bar);
}

// The same on this CTA's barrier alone.
template <int CG>
__device__ __forceinline__ void commit_local(uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
  else
    mma_commit(bar);
}

template <int CG>
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

#define KQ_MMA_FP4(CGN, KINDVEC)                                                                                     \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                                      \
               "tcgen05.mma.cta_group::" CGN "." KINDVEC " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),            \
               "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)                                               \
               : "memory")

template <int KIND, int CG>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t acc) {
  if constexpr (KIND == KIND_MX && CG == 1) KQ_MMA_FP4("1", "kind::mxf4.block_scale.scale_vec::2X");
  if constexpr (KIND == KIND_MX && CG == 2) KQ_MMA_FP4("2", "kind::mxf4.block_scale.scale_vec::2X");
  if constexpr (KIND == KIND_NV && CG == 1) KQ_MMA_FP4("1", "kind::mxf4nvf4.block_scale.scale_vec::4X");
  if constexpr (KIND == KIND_NV && CG == 2) KQ_MMA_FP4("2", "kind::mxf4nvf4.block_scale.scale_vec::4X");
}

// One 512-byte scale tile to 4 TMEM columns, repeated in the four lane quarters.
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Instruction descriptor of the block-scaled kinds: scale ids (which half of
// a 4-block word a two-scale step takes), E2M1 operands (1), N >> 3, scale type
// (E8M0: bit 23), M >> 4.
constexpr uint32_t idesc_fp4(bool e8m0, uint32_t M, uint32_t N, uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((e8m0 ? 1u : 0u) << 23) | ((M >> 4) << 24) |
         (sf_id << 29);
}

// 32 lanes x 32 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// ------------------------------------------------------------------ the gate

// p = sigmoid(z): silu z = g; tanh form of gelu z = 2 sqrt(2/pi) (g + 0.044715
// g^3), since (1 + tanh(y)) / 2 = sigmoid(2 y) (no cancellation at either end).
// act(g) = g p, act'(g) = p + g p (1 - p) dz/dg.  Fast exponential and division
// (a few fp32 ulp): the results are rounded to bf16.
struct Gate {
  float p, dz;
};
__device__ __forceinline__ Gate gate_of(float g, int act) {
  constexpr float k2C = 1.5957691216057308f, kA = 0.044715f;
  float z = g, dz = 1.f;
  if (act) {
    const float c = fminf(fmaxf(g, -20.f), 20.f);   // p is 0 or 1 beyond; keeps dz finite
    const float g2 = c * c;
    z = k2C * c * fmaf(kA, g2, 1.f);
    dz = k2C * fmaf(3.f * kA, g2, 1.f);
  }
  return {__fdividef(1.f, 1.f + __expf(-z)), dz};
}

// ------------------------------------------------------------------ stores

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// v[0..n) to bf16 columns c0.. of a row (n a multiple of 8), columns below N only.
template <int n>
__device__ __forceinline__ void store_bf16(__nv_bfloat16* row, int64_t c0, int64_t N, int vec, const float* v) {
  if (vec && c0 + n <= N) {
#pragma unroll
    for (int i = 0; i < n; i += 8)
      *reinterpret_cast<uint4*>(row + c0 + i) = make_uint4(pack_bf16(v[i], v[i + 1]), pack_bf16(v[i + 2], v[i + 3]),
                                                           pack_bf16(v[i + 4], v[i + 5]), pack_bf16(v[i + 6], v[i + 7]));
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i)
      if (c0 + i < N) row[c0 + i] = __float2bfloat16_rn(v[i]);
  }
}

template <int n>
__device__ __forceinline__ void store_f32(float* row, int64_t c0, int64_t N, int vec, const float* v) {
  if (vec && c0 + n <= N) {
#pragma unroll
    for (int i = 0; i < n; i += 4) *reinterpret_cast<float4*>(row + c0 + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i)
      if (c0 + i < N) row[c0 + i] = v[i];
  }
}

template <int n>
__device__ __forceinline__ void load_bf16(const __nv_bfloat16* row, int64_t c0, int64_t N, int vec, float* v) {
  if (vec && c0 + n <= N) {
#pragma unroll
    for (int i = 0; i < n; i += 8) {
      const uint4 q = *reinterpret_cast<const uint4*>(row + c0 + i);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[i + 2 * j] = __uint_as_float(w[j] << 16);
        v[i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = c0 + i < N ? __bfloat162float(row[c0 + i]) : 0.f;
  }
}

// n output columns c0.. of row r from the accumulators (a: the product, or the
// gate projection; u: the up projection), scaled by sa and su.
template <int EPI, int n>
__device__ __forceinline__ void finish(const Params& p, int problem, int64_t r, int64_t c0, float sa, float su, float* a,
                                       float* u) {
  if constexpr (EPI == EPI_STORE) {
#pragma unroll
    for (int i = 0; i < n; ++i) a[i] *= sa;
    if (p.out_f32)
      store_f32<n>(static_cast<float*>(p.out[problem]) + r * p.ldo[problem], c0, p.N, p.out_vec[problem], a);
    else
      store_bf16<n>(static_cast<__nv_bfloat16*>(p.out[problem]) + r * p.ldo[problem], c0, p.N, p.out_vec[problem], a);
  } else if constexpr (EPI == EPI_GATED) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float g = sa * a[i];
      a[i] = g * gate_of(g, p.act).p * (su * u[i]);
    }
    store_bf16<n>(static_cast<__nv_bfloat16*>(p.out[0]) + r * p.ldo[0], c0, p.N, p.out_vec[0], a);
  } else {
    float dh[n];
    load_bf16<n>(p.dh + r * p.lddh, c0, p.N, p.dh_vec, dh);
    if (p.h) {
      float h[n];
#pragma unroll
      for (int i = 0; i < n; ++i) h[i] = a[i] * gate_of(a[i], p.act).p * u[i];
      store_bf16<n>(p.h + r * p.ldh, c0, p.N, p.h_vec, h);
    }
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float g = a[i];
      const Gate q = gate_of(g, p.act);
      // dG = dH u act'(g), dU = dH act(g)
      a[i] = dh[i] * u[i] * fmaf(g * q.p * (1.f - q.p), q.dz, q.p);
      u[i] = dh[i] * (g * q.p);
    }
    store_bf16<n>(static_cast<__nv_bfloat16*>(p.out[0]) + r * p.ldo[0], c0, p.N, p.out_vec[0], a);
    store_bf16<n>(static_cast<__nv_bfloat16*>(p.out[1]) + r * p.ldo[1], c0, p.N, p.out_vec[1], u);
  }
}

// ------------------------------------------------------------------ kernel

// Tile t of a problem -> (row tile, column tile): bands of 8 row tiles are
// walked column by column, so that the tiles in flight share rows and columns
// in L2.
__device__ __forceinline__ void tile_coords(const Params& p, int t, int* tm, int* tn) {
  const int band = 8 * p.tiles_n;
  const int b = t / band, w = min(8, p.tiles_m - 8 * b), r = t - b * band;
  *tm = 8 * b + r % w;
  *tn = r / w;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) tile_kernel(const __grid_constant__ Maps maps, const Params p) {
  constexpr int S = C::STAGES, CG = C::CG;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::RING);
  // bars: full [0, S), empty [S, 2S), acc full [2S, 2S + 2), acc empty [2S + 2, 2S + 4), drained [2S + 4]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + S);
  const uint32_t accfull0 = smem_u32(bars + 2 * S), accempty0 = smem_u32(bars + 2 * S + 2);
  const uint32_t drained = smem_u32(bars + 2 * S + 4);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int ks = CG == 1 ? p.ks : 1;
  const uint32_t crank = (CG == 2 || ks > 1) ? cluster_rank() : 0;
  const uint32_t rank = CG == 2 ? crank : 0;                  // CTA of the pair
  const int unit0 = (int)blockIdx.x / (CG * ks), units = (int)gridDim.x / (CG * ks);
  // this CTA's share of K
  const int kb0 = ks > 1 ? (int)((int64_t)p.kblocks * crank / ks) : 0;
  const int kb1 = ks > 1 ? (int)((int64_t)p.kblocks * (crank + 1) / ks) : p.kblocks;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accfull0 + 8 * b, 1);
      mbar_init(accempty0 + 8 * b, CG * C::EW * 32);
    }
    mbar_init(drained, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) alloc_tmem<CG, C::TMEM_COLS>(smem_u32(tmem_slot));
  fence_before();
  __syncthreads();
  if (CG == 2 || ks > 1) cluster_sync();   // the other CTAs' barriers are ready too
  fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ---------------- TMA producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued_phase[S];
      bool issued[S], ok = true;
      for (int s = 0; s < S; ++s) issued[s] = false;
      const uint32_t stage_tx = (uint32_t)(p.a_rows * 128 + C::B_BYTES + C::SFA_BYTES + C::SFB_BYTES) * CG;
      for (int t = unit0; t < p.num_tiles && ok; t += units) {
        const int problem = t / p.problem_tiles;
        int tm, tn;
        tile_coords(p, t - problem * p.problem_tiles, &tm, &tn);
        const int m0 = tm * 128 * CG + (int)rank * 128, n0 = tn * C::OUTC;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag, p.info, 11, p.wait_ns)) {
            ok = false;
            break;
          }
          uint32_t fb = full0 + 8 * stage;
          if (CG == 1 || rank == 0) mbar_arrive_expect_tx(fb, stage_tx);
          if (CG == 2) fb = mapa(fb, 0);
          const uint32_t sa = smem_u32(smem + stage * C::STAGE_BYTES), sb = sa + C::A_BYTES;
          const int seg = kb >= p.seg_blocks, k = kb - (seg ? p.seg_blocks : 0);
          const CUtensorMap* ma = &maps.a[problem ? 1 : seg];
          const CUtensorMap* mb = &maps.b[seg];
          constexpr int KE = C::FP4 ? 128 : 64;   // map elements per stage along K (bytes of codes, or bf16)
          if constexpr (C::AMN) {
            load_2d<CG>(sa, ma, m0, 64 * k, fb);
            load_2d<CG>(sa + 8192, ma, m0 + 64, 64 * k, fb);
          } else {
            load_2d<CG>(sa, ma, KE * k, m0, fb);
          }
          if constexpr (C::BMN) {
#pragma unroll
            for (int q = 0; q < C::BN / CG / 64; ++q)
              load_2d<CG>(sb + 8192 * q, mb, n0 + (int)rank * (C::BN / CG) + 64 * q, 64 * k, fb);
          } else if constexpr (C::DUAL && CG == 2) {
            load_2d<CG>(sb, &maps.b[rank], KE * k, n0, fb);
          } else if constexpr (C::DUAL) {
            load_2d<CG>(sb, &maps.b[0], KE * k, n0, fb);
            load_2d<CG>(sb + C::MMA_N * 128, &maps.b[1], KE * k, n0, fb);
          } else {
            load_2d<CG>(sb, mb, KE * k, n0 + (int)rank * (C::BN / CG), fb);
          }
          if constexpr (C::FP4) {
            const uint32_t sf = sb + C::B_BYTES;
            load_2d<CG>(sf, &maps.sfa, 0, (m0 / 128) * p.kat + kb * C::ATOMS, fb);
#pragma unroll
            for (int q = 0; q < C::SFB_TILES; ++q)
              load_2d<CG>(sf + C::SFA_BYTES * (1 + q), C::DUAL ? &maps.sfb[q] : &maps.sfb[0], 0,
                          (n0 / 128 + (C::DUAL ? 0 : q)) * p.kat + kb * C::ATOMS, fb);
          }
          issued[stage] = true;
          issued_phase[stage] = phase;
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && rank == 0) {
        // the copies in flight land before the CTA (or pair) can exit
        const unsigned long long t0 = globaltimer();
        for (int s = 0; s < S; ++s)
          while (issued[s] && !mbar_try_wait(full0 + 8 * s, issued_phase[s]) && globaltimer() - t0 < kTimeoutNs) {
          }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (the pair's first CTA)
    if (lane == 0 && rank == 0) {
      int stage = 0, buf = 0;
      uint32_t phase = 0, acc_phase = 0, done = 0;   // done: stages issued so far
      bool ok = true;
      const uint32_t sf0 = tmem + C::NBUF * C::BN;
      for (int t = unit0; t < p.num_tiles && ok; t += units) {
        if (!mbar_wait(accempty0 + 8 * buf, acc_phase ^ 1u, abort_flag, p.info, 12, p.wait_ns)) {
          ok = false;
          break;
        }
        fence_after();
        const uint32_t d = tmem + buf * C::BN;
        // a 64-column MMA in the upper half of a 128-row scale tile takes its columns 2 and 3
        int sfb_shift = 0;
        if constexpr (C::FP4 && C::MMA_N == 64) {
          int tm, tn;
          tile_coords(p, t % p.problem_tiles, &tm, &tn);
          sfb_shift = (tn & 1) ? 2 : 0;
        }
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(full0 + 8 * stage, phase, abort_flag, p.info, 13, p.wait_ns)) {
            ok = false;
            break;
          }
          const uint32_t sa = smem_u32(smem + stage * C::STAGE_BYTES), sb = sa + C::A_BYTES;
          if constexpr (C::FP4) {
            const int slot = C::NSF == S ? stage : (int)(done % C::NSF);
            if (C::NSF < S && done >= (uint32_t)C::NSF) {
              // the MMAs that read this scale buffer last are done
              const uint32_t j = done - C::NSF;
              if (!mbar_wait(empty0 + 8 * (j % S), (j / S) & 1u, abort_flag, p.info, 14, p.wait_ns)) {
                ok = false;
                break;
              }
            }
            fence_after();
            const uint32_t sf = sb + C::B_BYTES;
            const uint32_t ca = sf0 + slot * C::SF_COLS, cb = ca + 4 * C::ATOMS;
#pragma unroll
            for (int q = 0; q < C::ATOMS; ++q) {
              copy_scales<CG>(ca + 4 * q, smem_desc(sf + 512 * q, 128, 128, 0));
#pragma unroll
              for (int b = 0; b < C::SFB_TILES; ++b)   // one K tile's columns side by side
                copy_scales<CG>(cb + 4 * (C::SFB_TILES * q + b),
                                smem_desc(sf + C::SFA_BYTES * (1 + b) + 512 * q, 128, 128, 0));
            }
            const int n = min(4, p.steps - 4 * kb);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (j >= n) break;
              const int atom = C::KIND == KIND_MX ? j / 2 : j;
              const uint32_t id = idesc_fp4(C::KIND == KIND_MX, 128 * CG, C::MMA_N, C::KIND == KIND_MX ? 2 * (j & 1) : 0);
              const uint32_t acc = (kb > kb0 || j > 0) ? 1u : 0u;
#pragma unroll
              for (int s = 0; s < C::NSUB; ++s)
                mma_fp4<C::KIND, CG>(d + s * C::MMA_N, smem_desc(sa + 32 * j, 16, 1024, kSwizzle128),
                                     smem_desc(sb + s * C::MMA_N * 128 + 32 * j, 16, 1024, kSwizzle128), id,
                                     ca + 4 * atom, cb + 4 * (C::SFB_TILES * atom + s) + sfb_shift, acc);
            }
          } else {
            fence_after();
            constexpr uint32_t id = idesc(kFmtBF16, C::AMN, C::BMN, 128 * CG, C::MMA_N);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t acc = (kb > kb0 || j > 0) ? 1u : 0u;
              const uint64_t da = C::AMN ? smem_desc(sa + 2048 * j, 8192, 1024, kSwizzle128)
                                         : smem_desc(sa + 32 * j, 16, 1024, kSwizzle128);
#pragma unroll
              for (int s = 0; s < C::NSUB; ++s) {
                const uint32_t bs = sb + s * C::MMA_N * 128;
                mma_bf16<CG>(d + s * C::MMA_N, da,
                             C::BMN ? smem_desc(bs + 2048 * j, 8192, 1024, kSwizzle128)
                                    : smem_desc(bs + 32 * j, 16, 1024, kSwizzle128),
                             id, acc);
              }
            }
          }
          ++done;
          commit<CG>(empty0 + 8 * stage);   // the stage is free once these MMAs have read it
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        commit<CG>(accfull0 + 8 * buf);
        if (++buf == C::NBUF) {
          buf = 0;
          acc_phase ^= 1u;
        }
      }
      if (done) {
        // every MMA this thread issued has completed before TMEM is released
        commit_local<CG>(drained);
        mbar_drain(drained, 0);
      }
    }
  } else {
    // ---------------- epilogue: lane quarter warp % 4, one row per lane
    const int wq = warp & 3, half = (warp - 2) / 4;
    const int row = 32 * wq + lane;
    int buf = 0;
    uint32_t acc_phase = 0;
    const float sa = (p.ga ? *p.ga : 1.f) * (p.gb[0] ? *p.gb[0] : 1.f);
    const float su = (p.ga ? *p.ga : 1.f) * (p.gb[1] ? *p.gb[1] : 1.f);
    for (int t = unit0; t < p.num_tiles; t += units) {
      const int problem = t / p.problem_tiles;
      int tm, tn;
      tile_coords(p, t - problem * p.problem_tiles, &tm, &tn);
      const int64_t r = (int64_t)tm * 128 * CG + rank * 128 + row, c0 = (int64_t)tn * C::OUTC;
      // one lane waits, the warp follows: every lane leaves together on abort
      bool ready = true;
      if (lane == 0) ready = mbar_wait(accfull0 + 8 * buf, acc_phase, abort_flag, p.info, 15, p.wait_ns);
      if (!__shfl_sync(0xffffffffu, ready ? 1 : 0, 0)) break;
      __syncwarp();
      fence_after();
      const uint32_t d = tmem + ((uint32_t)(32 * wq) << 16) + buf * C::BN;
      constexpr int CW = C::OUTC / (C::EW / 4);   // output columns of this warp
      constexpr int CN = CW < 32 ? CW : 32;
      if (ks > 1) {
        // fp32 partials to this CTA's shared memory, summed below
        float* part = reinterpret_cast<float*>(smem);
#pragma unroll 1
        for (int c = half * (C::BN / (C::EW / 4)); c < (half + 1) * (C::BN / (C::EW / 4)); c += 16) {
          float v[16];
          tmem_ld16(d + c, v);
          if (r < p.M) {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<float4*>(part + row * C::PART_LD + c + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          }
        }
      } else {
        static_assert(CN == 32, "32 output columns at a time");
#pragma unroll 1
        for (int c = half * CW; c < (half + 1) * CW; c += 32) {
          float a[32], u[C::DUAL ? 32 : 1];
          tmem_ld32(d + c, a);
          if constexpr (C::DUAL) tmem_ld32(d + C::BN / 2 + c, u);
          if (r < p.M) finish<C::EPI, 32>(p, problem, r, c0 + c, sa, su, a, u);
        }
      }
      fence_before();
      if (CG == 2)
        mbar_arrive_cluster(mapa(accempty0 + 8 * buf, 0));
      else
        mbar_arrive(accempty0 + 8 * buf);
      if (++buf == C::NBUF) {
        buf = 0;
        acc_phase ^= 1u;
      }
    }
  }

  fence_before();
  __syncthreads();
  if constexpr (CG == 1) {
    if (ks > 1) {
      // sum of the cluster's partials in rank order; each CTA takes a share of the tile's columns
      cluster_sync();
      if (unit0 < p.num_tiles) {
        const int problem = unit0 / p.problem_tiles;
        int tm, tn;
        tile_coords(p, unit0 - problem * p.problem_tiles, &tm, &tn);
        const float sa = (p.ga ? *p.ga : 1.f) * (p.gb[0] ? *p.gb[0] : 1.f);
        const float su = (p.ga ? *p.ga : 1.f) * (p.gb[1] ? *p.gb[1] : 1.f);
        const int rows = (int)min((int64_t)128, p.M - (int64_t)tm * 128);
        const int share = C::OUTC / ks;            // a multiple of 8
        const uint32_t base = smem_u32(smem);
        for (int i = threadIdx.x; i < rows * (share / 8); i += C::THREADS) {
          const int rr = i / (share / 8), c = (int)crank * share + 8 * (i % (share / 8));
          float a[8], u[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) a[e] = u[e] = 0.f;
          for (int q = 0; q < ks; ++q) {
            const uint32_t src = mapa(base + 4u * (uint32_t)(rr * C::PART_LD + c), (uint32_t)q);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              a[e] += ld_cluster(src + 4 * e);
              if constexpr (C::DUAL) u[e] += ld_cluster(src + 2 * C::BN + 4 * e);
            }
          }
          finish<C::EPI, 8>(p, problem, (int64_t)tm * 128 + rr, (int64_t)tn * C::OUTC + c, sa, su, a, u);
        }
      }
      cluster_sync();                              // the partials stay until every CTA has read them
    }
  } else {
    cluster_sync();                                // both CTAs are done with each other's memory
  }
  if (warp == 1) {
    fence_after();
    free_tmem<CG, C::TMEM_COLS>(tmem);
  }
}

// ------------------------------------------------------------------ host

template <class C>
kq_status launch(const char* what, const Maps& maps, const Params& p, int grid, cudaStream_t st) {
  // the attribute belongs to the device: set on every call, as the current device may change
  KQ_TRY(cuda_check(cudaFuncSetAttribute(tile_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM), what));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C::CG == 2 ? 2 : p.ks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (C::CG == 2 || p.ks > 1) ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, tile_kernel<C>, maps, p);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return cuda_check(e, what);
  }
  return launch_check(what);
}

}  // namespace mma
}  // namespace kq
