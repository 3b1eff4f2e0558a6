// Tile engine of the 4-bit floating-point product and of the gated
// feed-forward block: D = A B^T on tcgen05 tensor cores with TMA-fed operands,
// fp32 accumulators in TMEM and a fused epilogue (internal).
//
// Operands.  kind::f16 (bf16, K or MN major), or the block-scaled kinds over
// e2m1 codes: kind::mxf4 (one E8M0 scale per 32 codes) and kind::mxf4nvf4 (one
// E4M3 scale per 16).  In all of them a pipeline stage holds 128 bytes of K
// per row (64 bf16 or 256 codes, four MMA steps of 32 bytes) in the 128-byte
// swizzle.  Scale bytes travel as whole 512-byte tiles (128 rows x 4 blocks) by
// TMA to shared memory and from there to TMEM in one of two ways.  CG = 2: by
// tcgen05.cp, issued by the MMA thread ahead of the step that reads them (6 copies a
// stage with KQ_FP4_MX, 12 with KQ_FP4_NV; 0.37 and 0.385 us a stage of 0.27 us of MMAs
// at 8192 x 11008 x 16384.  From a warp of their own, which the MMA thread then waits
// for: 0.42 and 0.45).  CG = 1: two sets of four warps, one for the ring's even slots and
// one for its odd ones, a warp per lane quarter, with tcgen05.st (the 16 bytes of a tile
// row are a lane's four columns, of which an MMA of half a tile's rows needs two, so that
// TMEM holds a buffer per stage for two CTAs).  Under the pair's dense stream of MMAs
// these stores wait for TMEM (0.87 us a stage).
//
// Shapes.  CG = 2: a CTA pair per 256 x 256 tile (cta_group::2), each CTA
// holding 128 rows of A and of B, so an SM fetches 64 bytes per MMA cycle
// instead of the 96 of a single 128 x 256 CTA.  CG = 1: 128 x BN tiles, one per
// CTA, for products with few rows, optionally with K split over a cluster of KS
// CTAs whose fp32 partials are summed in rank order through distributed shared
// memory (results do not depend on scheduling).
//
// Gated tiles hold the gate and the up columns of the same features side by
// side: with CG = 2 the pair's first CTA supplies the gate rows of B and the
// second the up rows; with CG = 1 two MMAs per step.  The epilogue then has
// both projections of a feature in one thread.
//
// Warp roles: 0 TMA, 1 TMEM and MMA issue, 2-9 the epilogue (one lane per row, two
// warps per lane quarter, output through a swizzled staging buffer so that rows
// leave in full lines).  With CG = 2 bf16 has two accumulators used in turn; beside a
// scale buffer for every stage only one fits, which the epilogue takes into registers
// whole, so that the next tile's MMAs wait for that read only (about 0.9 us a tile of
// 7 us at K = 4096).
// Every mbarrier wait is bounded by a time limit; on expiry the kernel
// records KQ_ERR_TIMEOUT, lets its copies land (bounded), frees TMEM and returns.
#pragma once

#include <cuda_bf16.h>

#include <algorithm>

#include "kq_tc.cuh"

namespace kq {
namespace mma {

using namespace kq::tc;

enum { KIND_BF16 = 0, KIND_MX = 1, KIND_NV = 2 };
enum { EPI_STORE = 0, EPI_GATED = 1, EPI_GATED_BWD = 2 };

template <int KIND_, int CG_, int BN_, bool AMN_, bool BMN_, int EPI_, int STAGES_>
struct Cfg {
  static constexpr int KIND = KIND_, CG = CG_, BN = BN_, EPI = EPI_;
  static constexpr bool AMN = AMN_, BMN = BMN_, FP4 = KIND != KIND_BF16, DUAL = EPI != EPI_STORE;
  static constexpr int NSUB = (CG == 1 && DUAL) ? 2 : 1;     // MMAs per K step
  static constexpr int MMA_N = BN / NSUB;
  static constexpr int OUTC = DUAL ? BN / 2 : BN;            // output columns of a tile
  static constexpr int B_BYTES = BN / CG * 128;
  static constexpr int ATOMS = KIND == KIND_MX ? 2 : (KIND == KIND_NV ? 4 : 0);   // scale tiles per stage and 128 rows
  static constexpr int SFB_TILES = DUAL ? 2 : (BN + 127) / 128;
  static constexpr int SFA_BYTES = ATOMS * 512, SFB_BYTES = SFB_TILES * ATOMS * 512;
  // A comes last in a stage: with few rows its box, and the stage, are shorter
  // (the MMA reads on into what follows: rows past M, whose results are not stored)
  static constexpr int A_OFF = B_BYTES + SFA_BYTES + SFB_BYTES;
  static constexpr int A_BYTES = 128 * 128;
  // TMEM columns of a scale tile of B: a 64-column MMA takes half a tile's rows
  static constexpr int SFB_W = MMA_N == 64 ? 2 : 4;
  static constexpr int SF_COLS = ATOMS * (4 + SFB_W * SFB_TILES);
  static constexpr int NBUF = (CG == 2 && !FP4) ? 2 : 1;     // accumulators
  // TMEM (two 128-row CTAs to an SM): accumulators, then a scale buffer per stage
  static constexpr int TMEM_LIMIT = CG == 2 ? 512 : 256;
  static constexpr int SF_FIT = FP4 ? (TMEM_LIMIT - NBUF * BN) / (FP4 ? SF_COLS : 1) : STAGES_;
  static constexpr int STAGES = SF_FIT < STAGES_ ? SF_FIT : STAGES_;
  static constexpr int COLS = NBUF * BN + STAGES * SF_COLS;
  static constexpr int TMEM_COLS = COLS <= 64 ? 64 : (COLS <= 128 ? 128 : (COLS <= 256 ? 256 : 512));
  static constexpr int EW = 8;                               // epilogue warps
  static constexpr int EW0 = 2;                              // the first of them
  static constexpr int THREADS = 32 * (EW0 + EW);
  static constexpr int PART_LD = BN + 4;                     // row stride of the split-K partials
  static constexpr int RING = STAGES * (A_OFF + A_BYTES);    // at most: stages shrink with A's box, and p.stages may be fewer
  static constexpr int STAGING = EW * 4096;                  // 32 rows x 128 bytes per epilogue warp
  static constexpr int BARS = 1024;                          // barriers, TMEM address, abort flag
  // CG = 1 has one tile per CTA: staging and split-K partials reuse the ring
  static constexpr int MIN_STAGES = 4;
  static constexpr int SMEM = 1024 + BARS + (CG == 2 ? RING + STAGING : MIN_STAGES * (A_OFF + A_BYTES));
  static_assert(SMEM <= 232448, "shared memory");
  static_assert(CG == 2 || (128 * PART_LD * 4 <= MIN_STAGES * (A_OFF + A_BYTES) && STAGING <= MIN_STAGES * A_OFF),
                "the ring holds what reuses it");
  static_assert(STAGES >= MIN_STAGES, "stages");
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
  int stages;            // of the ring in use
  int via_smem;          // CG = 1: the accumulators go through shared memory, spread over all threads
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
// Relaxed: what it hands over is TMEM, which the tcgen05 fences order.  A release at
// cluster scope would wait for the warp's global stores too, some 1000 cycles.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// Counts bytes that no copy will bring as arrived.
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Arrivals come from both CTAs of a pair: acquire at cluster scope.
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// The same without the hardware's own short wait.
__device__ __forceinline__ bool test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait of a whole warp with the contract of mbar_wait (limit 0: give up
// at the first poll that finds the phase incomplete); every lane gets the same
// answer, so the control flow around it stays uniform.  The clock is read only
// after a run of plain polls: reading it costs more than a pipeline stage
// takes, and a wait in a running pipeline ends within a few polls.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int32_t* info, int where,
                                          unsigned long long limit_ns) {
  if (limit_ns == 0) {
    if (__all_sync(0xffffffffu, test_wait(bar, parity))) return true;
    if (threadIdx.x % 32 == 0 && !*abort_flag) {
      *abort_flag = 1;
      report(info, KQ_ERR_TIMEOUT, where);
    }
    return false;
  }
  for (int i = 0; i < 65; ++i)
    if (__all_sync(0xffffffffu, try_wait(bar, parity))) return true;
  bool ok = true;
  if (threadIdx.x % 32 == 0) ok = mbar_wait(bar, parity, abort_flag, info, where, limit_ns);
  ok = __all_sync(0xffffffffu, ok);
  return ok && __all_sync(0xffffffffu, try_wait(bar, parity));   // every lane acquires
}

// The lane of a warp that issues its tcgen05 and TMA instructions (always the same
// one).  The issuing warps run their loops as whole warps and branch on this around
// a stage's instructions: the compiler then knows that one thread is left and
// issues them back to back.  Instructions predicated on a lane number instead cost
// some 80 cycles each (MX pairs, a stage of 4 MMAs and 6 copies: 0.56 us, here 0.37;
// bf16 backward, 333 x 1001 x 2730, single CTAs: 43.4 us, here 41.4).
__device__ __forceinline__ bool elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(r));
  return r != 0;
}

// A TMA tile load; with CG = 2 the barrier may be the pair leader's.
template <int CG>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    tma_load_2d(dst, map, x, y, bar);
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
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// The same on this CTA's barrier alone.
template <int CG>
__device__ __forceinline__ void commit_local(uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
  else
    commit<1>(bar);
}

#define KQ_MMA_BF16(CGN)                                                                                             \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                                                     \
               "tcgen05.mma.cta_group::" CGN ".kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),                        \
               "l"(a), "l"(b), "r"(idesc), "r"(acc)                                                                  \
               : "memory")

template <int CG>
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (CG == 2)
    KQ_MMA_BF16("2");
  else
    KQ_MMA_BF16("1");
}

#define KQ_MMA_FP4(CGN, KINDVEC)                                                                                     \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                                     \
               "tcgen05.mma.cta_group::" CGN "." KINDVEC " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),          \
               "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)                                              \
               : "memory")

template <int KIND, int CG>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t acc) {
  if constexpr (KIND == KIND_MX && CG == 1) KQ_MMA_FP4("1", "kind::mxf4.block_scale.scale_vec::2X");
  if constexpr (KIND == KIND_MX && CG == 2) KQ_MMA_FP4("2", "kind::mxf4.block_scale.scale_vec::2X");
  if constexpr (KIND == KIND_NV && CG == 1) KQ_MMA_FP4("1", "kind::mxf4nvf4.block_scale.scale_vec::4X");
  if constexpr (KIND == KIND_NV && CG == 2) KQ_MMA_FP4("2", "kind::mxf4nvf4.block_scale.scale_vec::4X");
}

// N words per lane to N TMEM columns of the warp's lane quarter.
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t* v) {
  static_assert(N == 8 || N == 16, "8 columns (MX) or 16 (NV)");
  if constexpr (N == 8)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  else
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
        "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// One 512-byte scale tile to 4 TMEM columns, repeated in the four lane quarters
// of both CTAs of a pair.
__device__ __forceinline__ void copy_scales_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Instruction descriptor of the block-scaled kinds: scale ids (which half of
// a 4-block word a two-scale step takes), E2M1 operands (1), N >> 3, scale type
// (E8M0: bit 23), M >> 4.
constexpr uint32_t idesc_fp4(bool e8m0, uint32_t M, uint32_t N, uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((e8m0 ? 1u : 0u) << 23) | ((M >> 4) << 24) |
         (sf_id << 29);
}

// 32 lanes x 32 consecutive 32-bit columns, not waited for: ld_wait comes before
// their use.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
      "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// The wait names the registers, so that nothing that reads them moves above it.
__device__ __forceinline__ void ld_wait32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

// 32 lanes x 32 consecutive 32-bit columns, waited for.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
      "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
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

// ------------------------------------------------------------------ output

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void unpack8(uint4 q, float* v) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}

// 16 bytes of a row from column c, only the elements below N.
template <typename T>
__device__ __forceinline__ void store16(T* row, int64_t c, int64_t N, int vec, uint4 q) {
  constexpr int E = 16 / sizeof(T);
  if (vec && c + E <= N) {
    *reinterpret_cast<uint4*>(row + c) = q;
  } else {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (c + e >= N) break;
      if constexpr (sizeof(T) == 4)
        row[c + e] = __uint_as_float(w[e]);
      else
        row[c + e] = __ushort_as_bfloat16((unsigned short)(w[e / 2] >> (16 * (e & 1))));
    }
  }
}
__device__ __forceinline__ uint4 load16(const __nv_bfloat16* row, int64_t c, int64_t N, int vec) {
  if (vec && c + 8 <= N) return *reinterpret_cast<const uint4*>(row + c);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c + e < N) w[e / 2] |= (uint32_t)__bfloat16_as_ushort(row[c + e]) << (16 * (e & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A warp's staging: 32 rows of 128 bytes; 16-byte piece k of row i lies at
// piece k ^ (i % 8), so that rows and lines are both free of bank conflicts.
__device__ __forceinline__ uint32_t piece(uint32_t stg, int i, int k) { return stg + 128 * i + 16 * (k ^ (i & 7)); }

// The staged rows (row 0 = row r0 of the matrix, columns c0.., P pieces of 16 bytes
// each) to global memory, neighbouring lanes taking neighbouring pieces; or from it.
template <int P, typename T>
__device__ __forceinline__ void rows_out(uint32_t stg, T* base, int64_t ld, int64_t r0, int64_t M, int64_t c0, int64_t N, int vec) {
  const int lane = threadIdx.x % 32, k = lane % P;
  __syncwarp();
#pragma unroll 2
  for (int i = lane / P; i < 32; i += 32 / P)
    if (r0 + i < M) store16(base + (r0 + i) * ld, c0 + k * (16 / (int)sizeof(T)), N, vec, lds128(piece(stg, i, k)));
  __syncwarp();
}
template <int P>
__device__ __forceinline__ void rows_in(uint32_t stg, const __nv_bfloat16* base, int64_t ld, int64_t r0, int64_t M, int64_t c0,
                                        int64_t N, int vec) {
  const int lane = threadIdx.x % 32, k = lane % P;
  __syncwarp();
#pragma unroll 2
  for (int i = lane / P; i < 32; i += 32 / P)
    sts128(piece(stg, i, k), r0 + i < M ? load16(base + (r0 + i) * ld, c0 + 8 * k, N, vec) : make_uint4(0, 0, 0, 0));
  __syncwarp();
}

struct Grads {
  float g, u, h;
};
// dG = dH u act'(g), dU = dH act(g), and H.
__device__ __forceinline__ Grads gate_backward(float g, float u, float dh, int act) {
  const Gate q = gate_of(g, act);
  const float a = g * q.p;
  return {dh * u * fmaf(a * (1.f - q.p), q.dz, q.p), dh * a, a * u};
}

// Eight output columns c.. of row r (the split-K sums).
template <int EPI>
__device__ __forceinline__ void finish8(const Params& p, int problem, int64_t r, int64_t c, float sa, float su, float* a, float* u) {
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out[problem]) + r * p.ldo[problem];
  if constexpr (EPI == EPI_STORE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] *= sa;
    if (p.out_f32) {
      float* f = static_cast<float*>(p.out[problem]) + r * p.ldo[problem];
      const uint32_t* w = reinterpret_cast<const uint32_t*>(a);
      store16(f, c, p.N, p.out_vec[problem], make_uint4(w[0], w[1], w[2], w[3]));
      store16(f, c + 4, p.N, p.out_vec[problem], make_uint4(w[4], w[5], w[6], w[7]));
    } else {
      store16(out, c, p.N, p.out_vec[problem], pack8(a));
    }
  } else if constexpr (EPI == EPI_GATED) {
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = (sa * a[i]) * gate_of(sa * a[i], p.act).p * (su * u[i]);
    store16(out, c, p.N, p.out_vec[0], pack8(a));
  } else {
    float dh[8], h[8];
    unpack8(load16(p.dh + r * p.lddh, c, p.N, p.dh_vec), dh);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const Grads q = gate_backward(a[i], u[i], dh[i], p.act);
      a[i] = q.g;
      u[i] = q.u;
      h[i] = q.h;
    }
    store16(out, c, p.N, p.out_vec[0], pack8(a));
    store16(static_cast<__nv_bfloat16*>(p.out[1]) + r * p.ldo[1], c, p.N, p.out_vec[1], pack8(u));
    if (p.h) store16(p.h + r * p.ldh, c, p.N, p.h_vec, pack8(h));
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

// The scale tiles of a stage from shared memory to this warp's lane quarter of TMEM.
template <class C>
__device__ __forceinline__ void scales_to_tmem(uint32_t sf, uint32_t taddr, int upper_half) {
  const int lane = threadIdx.x % 32;
  uint32_t v[4 * C::ATOMS], w[C::SFB_W * C::SFB_TILES * C::ATOMS];
#pragma unroll
  for (int q = 0; q < C::ATOMS; ++q) {
    const uint4 x = lds128(sf + 512 * q + 16 * lane);
    v[4 * q] = x.x;
    v[4 * q + 1] = x.y;
    v[4 * q + 2] = x.z;
    v[4 * q + 3] = x.w;
#pragma unroll
    for (int b = 0; b < C::SFB_TILES; ++b) {   // one K tile's columns side by side
      const uint4 y = lds128(sf + C::SFA_BYTES + 512 * (C::ATOMS * b + q) + 16 * lane);
      uint32_t* d = w + C::SFB_W * (C::SFB_TILES * q + b);
      if constexpr (C::SFB_W == 4) {
        d[0] = y.x;
        d[1] = y.y;
        d[2] = y.z;
        d[3] = y.w;
      } else {
        d[0] = upper_half ? y.z : y.x;
        d[1] = upper_half ? y.w : y.y;
      }
    }
  }
  tmem_st<4 * C::ATOMS>(taddr, v);
  tmem_st<C::SFB_W * C::SFB_TILES * C::ATOMS>(taddr + 4 * C::ATOMS, w);
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::CG == 1 ? 2 : 1) tile_kernel(const __grid_constant__ Maps maps, const Params p) {
  constexpr int S = C::STAGES, CG = C::CG;
  constexpr bool DRAIN = C::FP4 && CG == 2;   // one accumulator: read out whole before the stores
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem);
  // bars: full [0, S), empty [S, 2S), scales landed [2S, 3S), scales in TMEM
  // [3S, 4S), acc full [4S, 4S + 2), acc empty [4S + 2, 4S + 4), MMAs drained
  // [4S + 4]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 4 * S + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* mate = tmem_slot + 2;   // CG = 2: the other CTA's issued stages, and whether it gave up
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * S, landed0 = full0 + 16 * S, ready0 = full0 + 24 * S;
  const uint32_t accfull0 = full0 + 32 * S, accempty0 = accfull0 + 16, drained = accfull0 + 32;
  const uint32_t ring = full0 + C::BARS;
  const uint32_t stage_bytes = (uint32_t)(C::A_OFF + 128 * p.a_rows);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
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
      mbar_init(landed0 + 8 * s, 1);
      mbar_init(ready0 + 8 * s, 4);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accfull0 + 8 * b, 1);
      mbar_init(accempty0 + 8 * b, CG * C::EW);
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
  // what comes before overlaps the kernel ahead on the stream; no global memory so far
  pdl_wait();
  pdl_trigger();
  const uint32_t sf0 = tmem + C::NBUF * C::BN;

  // CG = 1: the scales of this CTA's stages, by one warp of a set.  A set owns the slots of
  // its parity, so that it waits for every phase of each: a parity wait on a phase whose
  // predecessor another set saw passes too early while that one is still open.
  auto write_scales = [&](int set, int tn) {
    int slot = 0;
    uint32_t phase = 0;
    for (int i = kb0; i < kb1; ++i) {
      if ((slot & 1) == set) {
        if (!warp_wait(landed0 + 8 * slot, phase, abort_flag, p.info, 14, p.wait_ns)) return false;
        // the slot's last MMAs are done: the producer waited for them before this stage's copies
        fence_after();
        if constexpr (C::FP4 && CG == 1)
          scales_to_tmem<C>(ring + slot * stage_bytes + C::B_BYTES,
                            sf0 + slot * C::SF_COLS + ((uint32_t)(32 * (warp & 3)) << 16), tn & 1);
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ready0 + 8 * slot);
      }
      if (++slot == p.stages) {
        slot = 0;
        phase ^= 1u;
      }
    }
    return true;
  };

  uint32_t issued = 0;   // stages whose copies the producer has issued
  constexpr uint32_t cta_tx_fixed = C::B_BYTES + (CG == 2 ? C::SFA_BYTES + C::SFB_BYTES : 0);
  const uint32_t cta_tx = (uint32_t)p.a_rows * 128 + cta_tx_fixed;   // bytes of a stage that a CTA brings
  if (warp == 0) {
    // ---------------- TMA producer
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = unit0; t < p.num_tiles && ok; t += units) {
      const int problem = t / p.problem_tiles;
      int tm, tn;
      tile_coords(p, t - problem * p.problem_tiles, &tm, &tn);
      const int m0 = tm * 128 * CG + (int)rank * 128, n0 = tn * C::OUTC;
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = warp_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag, p.info, 11, p.wait_ns);
        if (!ok) break;
        if (elect()) {
          uint32_t fb = full0 + 8 * stage;
          if (rank == 0) mbar_arrive_expect_tx(fb, cta_tx * CG);
          if (CG == 2) fb = mapa(fb, 0);
          const uint32_t sb = ring + stage * stage_bytes, sa = sb + C::A_OFF;
          const int seg = kb >= p.seg_blocks, k = kb - (seg ? p.seg_blocks : 0);
          const CUtensorMap* ma = &maps.a[problem ? 1 : seg];
          const CUtensorMap* mb = &maps.b[seg];
          constexpr int KE = C::FP4 ? 128 : 64;   // map elements per stage along K (bytes of codes, or bf16)
          if constexpr (C::FP4) {
            const uint32_t sf = sb + C::B_BYTES, lb = CG == 2 ? fb : landed0 + 8 * stage;
            if (CG == 1) mbar_arrive_expect_tx(lb, C::SFA_BYTES + C::SFB_BYTES);
            load_2d<CG>(sf, &maps.sfa, 0, (m0 / 128) * p.kat + kb * C::ATOMS, lb);
#pragma unroll
            for (int q = 0; q < C::SFB_TILES; ++q)
              load_2d<CG>(sf + C::SFA_BYTES * (1 + q), C::DUAL ? &maps.sfb[q] : &maps.sfb[0], 0,
                         (n0 / 128 + (C::DUAL ? 0 : q)) * p.kat + kb * C::ATOMS, lb);
          }
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
        }
        __syncwarp();
        ++issued;
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // the arrivals that free the last stages land before the CTA exits
    for (uint32_t i = issued - min(issued, (uint32_t)p.stages); i < issued && ok; ++i)
      ok = warp_wait(empty0 + 8 * (i % p.stages), i / p.stages & 1u, abort_flag, p.info, 17, p.wait_ns);
  } else if (warp == 1) {
    // ---------------- MMA issuer (the pair's first CTA)
    if (rank == 0) {
      int stage = 0, buf = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true, any = false;
      for (int t = unit0; t < p.num_tiles && ok; t += units) {
        if (!warp_wait(accempty0 + 8 * buf, acc_phase ^ 1u, abort_flag, p.info, 12, p.wait_ns)) break;
        const uint32_t d = tmem + buf * C::BN;
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = warp_wait(full0 + 8 * stage, phase, abort_flag, p.info, 13, p.wait_ns);
          if (C::FP4 && CG == 1 && ok) ok = warp_wait(ready0 + 8 * stage, phase, abort_flag, p.info, 16, p.wait_ns);
          if (!ok) break;
          fence_after();
          const uint32_t sb = ring + stage * stage_bytes, sa = sb + C::A_OFF;
          if (elect()) {
            if constexpr (C::FP4) {
              const uint32_t ca = sf0 + stage * C::SF_COLS, cb = ca + 4 * C::ATOMS;
              const uint64_t da = smem_desc(sa, 16, 1024, kSwizzle128), db = smem_desc(sb, 16, 1024, kSwizzle128);
              const uint64_t sf = smem_desc(sb + C::B_BYTES, 128, 128, 0);   // addresses count 16 bytes
              const int n = min(4, p.steps - 4 * kb);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if (j >= n) break;
                const int atom = C::KIND == KIND_MX ? j / 2 : j;
                if constexpr (CG == 2) {
                  if (C::KIND == KIND_NV || j % 2 == 0) {
                    // the buffer's last MMAs are done: the producer waited for them before it filled the stage again
                    copy_scales_pair(ca + 4 * atom, sf + 32 * atom);
#pragma unroll
                    for (int b = 0; b < C::SFB_TILES; ++b)   // one K tile's columns side by side
                      copy_scales_pair(cb + 4 * (C::SFB_TILES * atom + b), sf + 32 * (C::ATOMS * (1 + b) + atom));
                  }
                }
                const uint32_t id = idesc_fp4(C::KIND == KIND_MX, 128 * CG, C::MMA_N, C::KIND == KIND_MX ? 2 * (j & 1) : 0);
                const uint32_t acc = (kb > kb0 || j > 0) ? 1u : 0u;
#pragma unroll
                for (int s = 0; s < C::NSUB; ++s)
                  mma_fp4<C::KIND, CG>(d + s * C::MMA_N, da + 2 * j, db + s * C::MMA_N * 8 + 2 * j, id, ca + 4 * atom,
                                       cb + C::SFB_W * (C::SFB_TILES * atom + s), acc);
              }
            } else {
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
            commit<CG>(empty0 + 8 * stage);   // the stage is free once these MMAs have read it
          }
          __syncwarp();
          any = true;
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (elect()) commit<CG>(accfull0 + 8 * buf);
        if (++buf == C::NBUF) {
          buf = 0;
          acc_phase ^= 1u;
        }
      }
      if (any) {
        // every MMA this thread issued has completed before TMEM is released
        if (elect()) {
          commit_local<CG>(drained);
          mbar_drain(drained, 0);
        }
        __syncwarp();
      }
    }
  } else {
    // ---------------- epilogue: lane quarter warp % 4, one row per lane
    const int wq = warp & 3, share = (warp - C::EW0) / 4;
    constexpr int CW = C::OUTC / (C::EW / 4);   // output columns of this warp
    constexpr int CH = CW < 64 ? CW : 64;       // taken 64 or 32 at a time
    static_assert(CH == 64 || CH == 32, "64 or 32 output columns at a time");
    const uint32_t stg = (CG == 2 ? ring + C::RING : ring) + 4096 * (warp - C::EW0);
    const float sa = (p.ga ? *p.ga : 1.f) * (p.gb[0] ? *p.gb[0] : 1.f);
    const float su = (p.ga ? *p.ga : 1.f) * (p.gb[1] ? *p.gb[1] : 1.f);
    int buf = 0;
    uint32_t acc_phase = 0;
    for (int t = unit0; t < p.num_tiles; t += units) {
      const int problem = t / p.problem_tiles;
      int tm, tn;
      tile_coords(p, t - problem * p.problem_tiles, &tm, &tn);
      if constexpr (C::FP4 && CG == 1) {
        if (!write_scales(share, tn)) break;
      }
      const int64_t r0 = (int64_t)tm * 128 * CG + rank * 128 + 32 * wq;   // lane 0's row
      const int64_t c0 = (int64_t)tn * C::OUTC + share * CW;
      if (!warp_wait(accfull0 + 8 * buf, acc_phase, abort_flag, p.info, 15, p.wait_ns)) break;
      fence_after();
      const uint32_t d = tmem + ((uint32_t)(32 * wq) << 16) + buf * C::BN + share * CW;
      auto release = [&] {
        fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CG == 2)
            mbar_arrive_cluster(mapa(accempty0 + 8 * buf, 0));
          else
            mbar_arrive(accempty0 + 8 * buf);
        }
      };
      if (CG == 1 && p.via_smem) {
        // fp32 sums (or partial sums) to this CTA's shared memory, finished below
        float* part = reinterpret_cast<float*>(smem + C::BARS);
        if (r0 < p.M) {
#pragma unroll 1
          for (int c = share * (C::BN / 2); c < (share + 1) * (C::BN / 2); c += 16) {
            float v[16];
            tmem_ld16(tmem + ((uint32_t)(32 * wq) << 16) + c, v);
            if (r0 + lane < p.M) {
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4*>(part + (32 * wq + lane) * C::PART_LD + c + i) =
                    make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
          }
        }
        release();
      } else if constexpr (C::EPI == EPI_STORE) {
        if (DRAIN && !p.out_f32) {
          // as they are: packing would keep the accumulator 300 cycles longer
          uint32_t w[CW];
#pragma unroll
          for (int c = 0; c < CW; c += 32) tmem_ld32_async(d + c, w + c);
#pragma unroll
          for (int c = 0; c < CW; c += 32) ld_wait32(w + c);
          release();
#pragma unroll
          for (int c = 0; c < CW; c += CH) {
#pragma unroll
            for (int k = 0; k < CH / 8; ++k) {
              float v[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = sa * __uint_as_float(w[c + 8 * k + i]);
              sts128(piece(stg, lane, k), pack8(v));
            }
            rows_out<CH / 8>(stg, static_cast<__nv_bfloat16*>(p.out[problem]), p.ldo[problem], r0, p.M, c0 + c, p.N,
                             p.out_vec[problem]);
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < CW; c += CH) {
            float v[CH];
#pragma unroll
            for (int h = 0; h < CH; h += 32) tmem_ld32(d + c + h, v + h);
            if (c + CH == CW) release();
#pragma unroll
            for (int i = 0; i < CH; ++i) v[i] *= sa;
            if (p.out_f32) {
#pragma unroll
              for (int h = 0; h < CH; h += 32) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const uint32_t* w = reinterpret_cast<const uint32_t*>(v + h + 4 * k);
                  sts128(piece(stg, lane, k), make_uint4(w[0], w[1], w[2], w[3]));
                }
                rows_out<8>(stg, static_cast<float*>(p.out[problem]), p.ldo[problem], r0, p.M, c0 + c + h, p.N,
                            p.out_vec[problem]);
              }
            } else {
#pragma unroll
              for (int k = 0; k < CH / 8; ++k) sts128(piece(stg, lane, k), pack8(v + 8 * k));
              rows_out<CH / 8>(stg, static_cast<__nv_bfloat16*>(p.out[problem]), p.ldo[problem], r0, p.M, c0 + c, p.N,
                               p.out_vec[problem]);
            }
          }
        }
      } else if constexpr (C::EPI == EPI_GATED) {
        static_assert(CW == CH, "one piece per warp");
        uint32_t wg[CH], wu[CH];
#pragma unroll
        for (int h = 0; h < CH; h += 32) {
          tmem_ld32_async(d + h, wg + h);
          tmem_ld32_async(d + C::BN / 2 + h, wu + h);
        }
#pragma unroll
        for (int h = 0; h < CH; h += 32) {
          ld_wait32(wg + h);
          ld_wait32(wu + h);
        }
        release();
#pragma unroll
        for (int k = 0; k < CH / 8; ++k) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float g = sa * __uint_as_float(wg[8 * k + i]);
            v[i] = g * gate_of(g, p.act).p * (su * __uint_as_float(wu[8 * k + i]));
          }
          sts128(piece(stg, lane, k), pack8(v));
        }
        rows_out<CH / 8>(stg, static_cast<__nv_bfloat16*>(p.out[0]), p.ldo[0], r0, p.M, c0, p.N, p.out_vec[0]);
      } else {
        static_assert(CW == CH, "one piece per warp");
        rows_in<CH / 8>(stg, p.dh, p.lddh, r0, p.M, c0, p.N, p.dh_vec);
        uint4 og[CH / 8], ou[CH / 8], oh[CH / 8];
#pragma unroll
        for (int h = 0; h < CH / 32; ++h) {
          float g[32], u[32];
          tmem_ld32(d + 32 * h, g);
          tmem_ld32(d + C::BN / 2 + 32 * h, u);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float dh[8], vh[8];
            unpack8(lds128(piece(stg, lane, 4 * h + k)), dh);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const Grads q = gate_backward(g[8 * k + i], u[8 * k + i], dh[i], p.act);
              g[8 * k + i] = q.g;
              u[8 * k + i] = q.u;
              vh[i] = q.h;
            }
            og[4 * h + k] = pack8(g + 8 * k);
            ou[4 * h + k] = pack8(u + 8 * k);
            oh[4 * h + k] = pack8(vh);
          }
        }
        release();
        __syncwarp();
#pragma unroll
        for (int k = 0; k < CH / 8; ++k) sts128(piece(stg, lane, k), og[k]);
        rows_out<CH / 8>(stg, static_cast<__nv_bfloat16*>(p.out[0]), p.ldo[0], r0, p.M, c0, p.N, p.out_vec[0]);
#pragma unroll
        for (int k = 0; k < CH / 8; ++k) sts128(piece(stg, lane, k), ou[k]);
        rows_out<CH / 8>(stg, static_cast<__nv_bfloat16*>(p.out[1]), p.ldo[1], r0, p.M, c0, p.N, p.out_vec[1]);
        if (p.h) {
#pragma unroll
          for (int k = 0; k < CH / 8; ++k) sts128(piece(stg, lane, k), oh[k]);
          rows_out<CH / 8>(stg, p.h, p.ldh, r0, p.M, c0, p.N, p.h_vec);
        }
      }
      if (++buf == C::NBUF) {
        buf = 0;
        acc_phase ^= 1u;
      }
    }
  }

  fence_before();
  __syncthreads();
  bool expired = *abort_flag;
  uint32_t mate_issued = issued;
  if constexpr (CG == 2) {
    if (threadIdx.x == 0)
      st_cluster(mapa(smem_u32(const_cast<uint32_t*>(mate)), rank ^ 1u), issued << 1 | (expired ? 1u : 0u));
    __syncwarp();
    cluster_sync();                                // both CTAs are done with each other's memory
    const uint32_t word = *mate;
    expired |= word & 1u;
    mate_issued = word >> 1;
  }
  if (expired) {
    // A wait gave up, so that copies may be in flight that nobody waited for: they land
    // before the CTA (or pair) exits.  The pair's copies all signal the first CTA's
    // barriers, which expect both halves of a stage once that CTA has issued its own; the
    // two may have stopped up to a ring apart.  So the first CTA takes the halves that the
    // second never issued as arrived, announces those that it did not expect, and waits.
    if (warp == 0 && rank == 0) {
      if (CG == 2 && elect()) {
        for (uint32_t i = mate_issued; i < issued; ++i) mbar_complete_tx(full0 + 8 * (i % p.stages), cta_tx);
        for (uint32_t i = issued; i < mate_issued; ++i) mbar_arrive_expect_tx(full0 + 8 * (i % p.stages), cta_tx);
      }
      __syncwarp();
      const unsigned long long t0 = globaltimer();
      const uint32_t n = max(issued, mate_issued);
      for (uint32_t i = n - min(n, (uint32_t)p.stages); i < n; ++i) {
        const uint32_t slot = i % p.stages, ph = i / p.stages & 1u;
        while (!try_wait(full0 + 8 * slot, ph) && globaltimer() - t0 < kTimeoutNs) {
        }
        while (C::FP4 && CG == 1 && !try_wait(landed0 + 8 * slot, ph) && globaltimer() - t0 < kTimeoutNs) {
        }
      }
      __syncwarp();
    }
    if (CG == 2) cluster_sync();
  }
  if constexpr (CG == 1) {
    if (p.via_smem) {
      // sum of the cluster's partials in rank order; the tile's pieces of 8 columns are dealt to its CTAs
      if (ks > 1) cluster_sync();
      const int problem = unit0 / p.problem_tiles;
      int tm, tn;
      tile_coords(p, unit0 - problem * p.problem_tiles, &tm, &tn);
      const float sa = (p.ga ? *p.ga : 1.f) * (p.gb[0] ? *p.gb[0] : 1.f);
      const float su = (p.ga ? *p.ga : 1.f) * (p.gb[1] ? *p.gb[1] : 1.f);
      const int rows = (int)min((int64_t)128, p.M - (int64_t)tm * 128);
      for (int i = threadIdx.x + C::THREADS * (int)crank; i < rows * (C::OUTC / 8); i += C::THREADS * ks) {
        const int rr = i / (C::OUTC / 8), c = 8 * (i % (C::OUTC / 8));
        const uint32_t at = ring + 4u * (uint32_t)(rr * C::PART_LD + c);
        float a[8], u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = u[e] = 0.f;
        // the loads of four CTAs' pieces are in flight together
#pragma unroll 1
        for (int q0 = 0; q0 < ks; q0 += 4) {
          float4 x[4][C::DUAL ? 4 : 2];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (q0 + q < ks) {
              const uint32_t src = ks > 1 ? mapa(at, (uint32_t)(q0 + q)) : at;
              x[q][0] = ld_cluster(src);
              x[q][1] = ld_cluster(src + 16);
              if constexpr (C::DUAL) {
                x[q][2] = ld_cluster(src + 2 * C::BN);
                x[q][3] = ld_cluster(src + 2 * C::BN + 16);
              }
            }
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (q0 + q < ks) {
              const float* f = reinterpret_cast<const float*>(x[q]);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                a[e] += f[e];
                if constexpr (C::DUAL) u[e] += f[8 + e];
              }
            }
          }
        }
        finish8<C::EPI>(p, problem, (int64_t)tm * 128 + rr, (int64_t)tn * C::OUTC + c, sa, su, a, u);
      }
      if (ks > 1) cluster_sync();                  // the partials stay until every CTA has read them
    }
  }
  if (warp == 1) {
    fence_after();
    free_tmem<CG, C::TMEM_COLS>(tmem);
  }
}

// ------------------------------------------------------------------ host

// Which tiles a product runs on: CTA pairs, or 128-row tiles with K over ks CTAs.
struct Plan {
  bool pair;
  int ks;
};

// Microseconds a wave of tiles takes per stage of K, measured (B200, 1.9 GHz): 128-row
// tiles and pairs.  Beside them a wave of 128-row tiles costs about 3 us and one of
// pairs 2, a launch of pairs 4, and a split of K over ks CTAs `split` + `part` ks.
struct Cost {
  double slim, pair, split, part;
};

// M rows, `slim` and `pairs` tiles of either kind, `stages` of K.  Up to 64 rows the
// product streams its weights: K is split until the CTAs, two to an SM, are about as
// many as the SMs (11008 x 4096, 16 rows, MX: 9.9 us with 172 CTAs, 11.4 with 86, 15.4
// with 344; the bound of 176 was not measured between those).  Above, the cheaper by the sums above (MX, 1024 x 4096 x 4096: 11.3 us on
// 64 pairs, 18.7 on 256 tiles; 512 rows: 10.3 on 32 pairs, 9.8 on 128 tiles; gated, 333
// x 1001 x 5460: 13.2 us with K over 2 CTAs, 13.9 without, 15.0 on 16 pairs; bf16 gated
// 128 x 4096 x 11008: 50.6 on pairs, 59.3 on tiles).  Clusters are powers of two: of 5 or
// 6 CTAs fewer fit the GPU at a time (64 x 4096 x 4096: 19.7 us over 5, 11.1 over 4), and
// of 8 no more than a few (64 x 2048 x 5504, 128 CTAs: 17.5 us over 8, 8.5 over 4; 64 x
// 512 x 11008, 32 CTAs: 9.6 over 8, 10.1 over 4).  A CTA is left four stages of K or more
// (64 x 1024 x 4096, 16 stages: 8.8 us over 8, 7.5 over 4).
inline Plan make_plan(int64_t M, int64_t slim, int64_t pairs, int64_t stages, Cost c) {
  constexpr int64_t kSms = 148, kPairs = 74;
  if (M <= 64) {
    int ks = 1;
    while (ks < 8 && slim * ks * 2 <= (ks < 4 ? 176 : 64) && ks * 8 <= stages) ks *= 2;
    return {false, ks};
  }
  Plan best = {true, 1};
  double t = 4 + (2 + c.pair * (double)stages) * (double)cdiv(pairs, kPairs);
  for (int ks = 1; ks <= 8 && ks <= stages && (ks == 1 || slim * ks <= (ks < 8 ? kSms : 64)); ks *= 2) {
    const double u = (3 + c.slim * (double)cdiv(stages, ks)) * (double)cdiv(slim * ks, kSms) + (ks > 1 ? c.split + c.part * ks : 0);
    if (u < t) {
      t = u;
      best = {false, ks};
    }
  }
  return best;
}

// Number of CTAs: a pair's tiles are walked by as many pairs as the GPU holds.
template <class C>
kq_status grid_of(const char* what, const Params& p, int* grid) {
  *grid = p.num_tiles * C::CG * p.ks;
  if (C::CG == 1) return KQ_OK;
  int dev = 0, sms = 0;
  KQ_TRY(cuda_check(cudaGetDevice(&dev), what));
  KQ_TRY(cuda_check(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev), what));
  *grid = std::min(*grid, sms / 2 * 2);
  return KQ_OK;
}

// Bytes of shared memory with `stages` of A boxes of a_rows rows: the last stage's
// MMAs still read 128 rows from its A on.
template <class C>
constexpr int smem_of(int stages, int a_rows) {
  return 1024 + C::BARS + stages * (C::A_OFF + 128 * a_rows) + (128 - a_rows) * 128 + (C::CG == 2 ? C::STAGING : 0);
}

template <class C>
kq_status launch(const char* what, const Maps& maps, Params p, cudaStream_t st) {
  int grid;
  KQ_TRY(grid_of<C>(what, p, &grid));
  // CG = 1: as many stages as leave room for two CTAs to an SM (113 KB each), at least MIN_STAGES
  p.stages = C::STAGES;
  while (C::CG == 1 && p.stages > C::MIN_STAGES && smem_of<C>(p.stages, p.a_rows) > 113 * 1024) --p.stages;
  const int smem = smem_of<C>(p.stages, p.a_rows);
  // few rows: one of the four lane quarters holds them all, so the other warps help through shared memory
  p.via_smem = C::CG == 1 && (p.ks > 1 || p.M <= 32);
  // the attribute belongs to the device: set on every call, as the current device may change
  KQ_TRY(cuda_check(cudaFuncSetAttribute(tile_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         std::max(C::SMEM, 113 * 1024)), what));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C::CG == 2 ? 2 : p.ks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (C::CG == 2 || p.ks > 1) ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, tile_kernel<C>, maps, p);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return cuda_check(e, what);
  }
  return launch_check(what);
}

}  // namespace mma
}  // namespace kq
