// Microscaled 4-bit floating point: quantization to e2m1 codes with block
// scales (kq_fp4_quantize), and the matvec of such a matrix with up to eight
// unquantized vectors (kq_fp4_matvec), the single-token form of the product.
//
// Formats (OCP Microscaling Formats specification, MXFP4; and the two-level
// form with E4M3 scales): a block of 32 columns shares one E8M0 scale
// 2^(floor(log2 amax) - 2), or a block of 16 shares the scale s g, s the E4M3
// value nearest to amax / (6 g) and g one fp32 number per matrix.
#include <cuda_bf16.h>

#include "kq_fp4.cuh"

namespace {

using kq::fp4::block_of;

// ------------------------------------------------------------------ quantize

template <typename T>
__device__ __forceinline__ float as_float(T v);
template <>
__device__ __forceinline__ float as_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float as_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// 32 bytes in one access.
__device__ __forceinline__ void ld32bytes(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}
__device__ __forceinline__ void st32bytes(void* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]),
               "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// How rows can be accessed: 32 bytes at a time, 16, or element by element.
enum { ACCESS_ANY = 0, ACCESS_16 = 1, ACCESS_32 = 2 };
int access_of(const void* p, int64_t ld_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(p) | (uintptr_t)ld_bytes;
  return x % 32 == 0 ? ACCESS_32 : (x % 16 == 0 ? ACCESS_16 : ACCESS_ANY);
}

// Sixteen elements from column c of an aligned row as their bit patterns (W
// words: fp32 one per word, bf16 two), zeros past `cols`.
template <typename T, int W>
__device__ __forceinline__ void load16(const T* row, int c, int cols, int access, uint32_t (&w)[W]) {
  if (c + 16 <= cols) {
    const T* src = row + c;
#pragma unroll
    for (int i = 0; i < W; i += 8) {
      if (access == ACCESS_32) {
        ld32bytes(reinterpret_cast<const uint32_t*>(src) + i, *reinterpret_cast<uint32_t(*)[8]>(w + i));
      } else {
        const uint4 a = reinterpret_cast<const uint4*>(src)[i / 4], b = reinterpret_cast<const uint4*>(src)[i / 4 + 1];
        w[i] = a.x; w[i + 1] = a.y; w[i + 2] = a.z; w[i + 3] = a.w;
        w[i + 4] = b.x; w[i + 5] = b.y; w[i + 6] = b.z; w[i + 7] = b.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (c + i >= cols) continue;
      if constexpr (sizeof(T) == 4)
        w[i] = __float_as_uint(row[c + i]);
      else
        w[i / 2] |= (uint32_t)__bfloat16_as_ushort(row[c + i]) << (16 * (i & 1));
    }
  }
}

// Rows that are not 16-byte aligned go through shared memory: the lanes of a row
// take neighbouring elements of it, so that global accesses stay coalesced, and
// lane l's sixteen words lie 20 l words into the warp's buffer (no bank conflicts
// at 16 bytes per lane).
constexpr int kStageWords = 32 * 20;
__device__ __forceinline__ int stage_at(int first_lane, int e) { return 20 * (first_lane + e / 16) + e % 16; }

// Largest magnitude of the 16, as an fp32 bit pattern: non-negative floats order
// as integers, and NaN and Inf lie on top.
__device__ __forceinline__ uint32_t top_of(const uint32_t (&w)[16]) {
  uint32_t t = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) t = max(t, w[i] & 0x7fffffffu);
  return t;
}
__device__ __forceinline__ uint32_t top_of(const uint32_t (&w)[8]) {
  uint32_t t = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = w[i] & 0x7fff7fffu;
    asm("max.u16x2 %0, %0, %1;" : "+r"(t) : "r"(a));
  }
  return max(t << 16, t & 0xffff0000u);
}
__device__ __forceinline__ float element(const uint32_t (&w)[16], int i) { return __uint_as_float(w[i]); }
__device__ __forceinline__ float element(const uint32_t (&w)[8], int i) {
  return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
}

// Eight values to eight codes: round to nearest even, saturating at 6.
__device__ __forceinline__ uint32_t encode8(const float* q) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return w;
}

// The value of code k of a word.
__device__ __forceinline__ float decode1(uint32_t w, int k) {
  const uint32_t c = w >> (4 * k);
  // e2m1 as the top bits of an fp32 with exponent bias 127 - 126: exact, subnormal included
  return __uint_as_float(((c & 7u) << 22) | ((c & 8u) << 28)) * 0x1p126f;
}

struct QuantParams {
  int64_t rows, ldm, ldc, ldh;
  int cols, kat;        // kat: scale tiles along a row
  const void* M;
  const float* g;
  uint8_t* codes;
  uint8_t* scales;
  float* M_hat;
  int m_access, h_access;
  int32_t* info;
};

// Sixteen columns per lane: a 16-column block is a lane's own, a 32-column one
// two lanes'; four blocks' scale bytes leave as one word.  A warp takes 512
// columns of a row (ROW_LANES 32), or 128 of 4 rows (8) where rows are short,
// two such pieces with their loads in flight together.  The grid covers the scale
// tiles' padding (rows to 128, blocks to 4), whose bytes are zeros.  Bound by
// memory: one read of M, one write of codes and scales (and of M_hat).  4096 x 4096
// fp32 to MX with M_hat: 24.1 us (5.9 TB/s, 91 % of a copy's rate); 2047 x 11008 bf16,
// rows 8 elements apart, to NV with M_hat: 28.7 us (5.1 TB/s, 78 %: a reciprocal per
// block, a product and two FMAs per element and the conversions take 63 % of the issue
// slots, and the loads' latency is a third of a warp's time).
template <typename T, int FMT, int ROW_LANES>
__global__ void __launch_bounds__(256, 4) quantize_kernel(const QuantParams p) {
  constexpr int R = 2;                            // pieces of a warp
  constexpr int LANES = block_of(FMT) / 16;       // lanes per block
  constexpr int W = 16 * sizeof(T) / 4;           // words of 16 elements
  const int lane = threadIdx.x % 32;
  constexpr int per = 32 / ROW_LANES;             // rows of a piece
  const int64_t r0 = ((int64_t)blockIdx.x * 8 + threadIdx.x / 32) * (R * per) + lane / ROW_LANES;
  const int c = ((int)blockIdx.y * ROW_LANES + lane % ROW_LANES) * 16;
  const int padded = (p.cols + 31) / 32 * 32;
  const int kb = c / block_of(FMT);
  kq::pdl_wait();
  kq::pdl_trigger();
  float g = 1.f, g6 = 6.f;
  bool g_ok = true;
  if (FMT == KQ_FP4_NV) {
    g = *p.g;
    g_ok = g > 0.f && isfinite(g);
    g6 = 6.f * g;
  }
  __shared__ __align__(16) uint32_t stage_mem[8][kStageWords];
  uint32_t* stage = stage_mem[threadIdx.x / 32];
  const int row_lane = lane % ROW_LANES, first_lane = lane - row_lane, c_row = c - 16 * row_lane;
  uint32_t v[R][W];
  if (p.m_access == ACCESS_ANY) {
    uint32_t e[R][16];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int64_t r = r0 + k * per;
      const T* row = static_cast<const T*>(p.M) + r * p.ldm + c_row + row_lane;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        e[k][i] = r < p.rows && c_row + row_lane + i * ROW_LANES < p.cols ? __float_as_uint(as_float(row[i * ROW_LANES])) : 0u;
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
#pragma unroll
      for (int i = 0; i < 16; ++i) stage[stage_at(first_lane, i * ROW_LANES + row_lane)] = e[k][i];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(stage + 20 * lane + i);
        if constexpr (W == 16) {
          v[k][i] = x.x; v[k][i + 1] = x.y; v[k][i + 2] = x.z; v[k][i + 3] = x.w;
        } else {
          v[k][i / 2] = __byte_perm(x.x, x.y, 0x7632);
          v[k][i / 2 + 1] = __byte_perm(x.z, x.w, 0x7632);
        }
      }
      __syncwarp();
    }
  } else {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int64_t r = r0 + k * per;
      if (r < p.rows && c < p.cols) {
        load16(static_cast<const T*>(p.M) + r * p.ldm, c, p.cols, p.m_access, v[k]);
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) v[k][i] = 0;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int64_t r = r0 + k * per;
    uint32_t top = top_of(v[k]);
    if (LANES == 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const bool bad = top >= 0x7f800000u || !g_ok;
    uint32_t byte;
    float d, q[16];
    if (FMT == KQ_FP4_MX) {
      // 2^(floor(log2 amax) - 2) from the exponent field; at least 2^-127
      const int field = max((int)(top >> 23) - 2, 0);
      byte = bad ? 0xffu : (uint32_t)field;
      d = field ? __uint_as_float((uint32_t)field << 23) : 0x1p-127f;
      const float inv = __uint_as_float((uint32_t)(254 - field) << 23);   // 1 / d, a power of two
#pragma unroll
      for (int i = 0; i < 16; ++i) q[i] = element(v[k], i) * inv;
    } else {
      const float amax = __uint_as_float(top);
      const float t = fminf(__fdiv_rn(amax, g6), 448.f);
      uint16_t pair;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(pair) : "f"(0.f), "f"(t));
      byte = bad ? 0x7fu : (uint32_t)(pair & 0xff);
      d = kq::fp4::e4m3_value(byte) * g;
      // v / d rounded to fp32.  With the reciprocal r rounded once per block,
      // q0 = v r is within 2 ulp and fma(v - q0 d, r, q0) is the rounded
      // quotient (Markstein's correction step: the residual is exact in an
      // fma); a divide per element would bound the kernel.  Outside the
      // range where the residual is exact, the divide.
      if (d >= 0x1p-90f && d <= 0x1p90f && amax <= 1024.f * d) {
        const float r = __frcp_rn(d);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float x = element(v[k], i), q0 = x * r;
          q[i] = fmaf(fmaf(-q0, d, x), r, q0);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) q[i] = d > 0.f ? __fdiv_rn(element(v[k], i), d) : 0.f;
      }
    }
    uint32_t w0 = bad ? 0u : encode8(q), w1 = bad ? 0u : encode8(q + 8);
    if (bad && r < p.rows && c < p.cols) kq::report(p.info, g_ok ? KQ_ERR_NONFINITE : KQ_ERR_INVALID_ARG, r);
    if (r < p.rows && c < padded) *reinterpret_cast<uint2*>(p.codes + r * p.ldc + c / 2) = make_uint2(w0, w1);
    // four blocks' bytes as one word, written by the first lane of the four
    uint32_t word = byte << (8 * ((lane / LANES) & 3));
#pragma unroll
    for (int o = LANES; o < 4 * LANES; o *= 2) word |= __shfl_xor_sync(0xffffffffu, word, o);
    // a row past the end has zero scales (its values are zeros: MX byte 0 too)
    if (lane % (4 * LANES) == 0 && kb / 4 < p.kat && r < (p.rows + 127) / 128 * 128)
      *reinterpret_cast<uint32_t*>(p.scales + kq::fp4::scale_offset(r, kb, p.kat)) = r < p.rows ? word : 0u;
    if (p.M_hat) {
      if (bad) d = __uint_as_float(0x7fc00000u);
      float h[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[i] = decode1(w0, i) * d;
        h[i + 8] = decode1(w1, i) * d;
      }
      float* row = p.M_hat + r * p.ldh;
      if (p.h_access == ACCESS_ANY) {
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<float4*>(stage + 20 * lane + i) = make_float4(h[i], h[i + 1], h[i + 2], h[i + 3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int e = i * ROW_LANES + row_lane;
          if (r < p.rows && c_row + e < p.cols) row[c_row + e] = __uint_as_float(stage[stage_at(first_lane, e)]);
        }
        __syncwarp();
      } else if (r < p.rows && c + 16 <= p.cols) {
        if (p.h_access == ACCESS_32) {
          st32bytes(row + c, h);
          st32bytes(row + c + 8, h + 8);
        } else {
#pragma unroll
          for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4*>(row + c + i) = make_float4(h[i], h[i + 1], h[i + 2], h[i + 3]);
        }
      } else if (r < p.rows) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (c + i < p.cols) row[c + i] = h[i];
      }
    }
  }
}

// ------------------------------------------------------------------ matvec

// Weights as the 16-row operand of mma.m16n8k16 (bf16, fp32 accumulation), the
// vectors as its 8 columns, so that one decode of a code serves all vectors.
// e2m1 times its scale has at most 6 significant bits: exact in bf16.  bf16
// vectors enter as they are; fp32 vectors as three bf16 parts that sum to them
// (24 bits), one MMA each.
//
// A warp takes 16 rows and goes through its share of K in steps of 128 columns:
// lane (g, t) = (lane / 4, lane % 4) holds 32 consecutive codes of rows g and g +
// 8 and 32 elements of vector g.  A lane's codes and scales arrive by asynchronous
// copies in a ring of its own in shared memory, kDepth steps ahead: a step is 1 KB
// per warp, and an SM needs some 40 KB in flight to draw its share of the memory
// rate (with the next step alone in flight, in registers, a step took the 1 us of
// a load).  The
// K order inside an MMA is free as long as both operands share it: a register
// pairs codes p and p + 4 of a word, which four logic operations bring to bf16
// position, and x is paired alike.  Two arrangements:
//  * bf16 vectors: the 8 warps of a CTA split K of the same 16 rows, each reading
//    the x it needs.
//  * fp32 vectors: splitting x into parts costs as much as decoding the codes of
//    16 rows, and its 4 KB a step (8 vectors) four times their bytes.  So the 8
//    warps of a CTA take 128 rows of the same columns, the parts are formed once
//    per CTA in shared memory, and K is split over a cluster of up to 8 CTAs, whose
//    sums meet in distributed shared memory.
// Sums are added in a fixed order in both.
//
// Measured: 4096 x 4096 MX, one bf16 vector 5.3 us; 11008 x 4096 10.7 us (24 MB, 2.2
// TB/s), eight 12.9; 4096 x 11008 NV, eight fp32 vectors 22.6; 8192 x 28672 NV 144 (0.9
// TB/s), with bf16 vectors 67.  Nothing is saturated.  One bf16 vector, 11008 x 4096: the
// SMs have warps for 70 % of the time and issue in 68 % of that (decoding, 8 codes in some
// 20 instructions, keeps the ALU pipe 63 % busy), DRAM runs at 21 %; a warp has four
// steps, so the rest is the fill and drain of each CTA's ring.  fp32 vectors: 40 % of the
// issue slots, two CTAs to an SM, waits at the barriers around the parts' forming; the
// three MMAs a step use 15 % of the tensor pipe.
constexpr int kWarps = 8;
constexpr int kDepth = 4;         // steps of codes in flight (a power of two)
constexpr int kStageSteps = 12;   // steps of x parts in shared memory at a time (72 KB)

struct MatvecParams {
  const uint8_t* codes;
  const uint8_t* scales;
  const float* g;
  int64_t d_out, d_in, ldc, kat;
  const void* X;
  int64_t ldx;
  int x_vec, batch, ks;   // ks: CTAs along K (fp32)
  void* Y;
  int64_t ldy;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes p and p + 4 of a word as bf16 values times 2^-126.
template <int P>
__device__ __forceinline__ uint32_t spread(uint32_t w) {
  const uint32_t mag = P < 2 ? w << (6 - 4 * P) : w >> (4 * P - 6);
  const uint32_t sgn = w << (12 - 4 * P);
  return (mag & 0x01c001c0u) | (sgn & 0x80008000u);
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// A block's scale as a bf16 pair to multiply spread() with: MX 2^k, or 2^(k + 126)
// where that fits; NV s 2^118 (the missing 2^8 is in the final factor; 448 2^126
// would overflow).
template <int FMT>
__device__ __forceinline__ uint32_t scale_pair(uint32_t byte, bool small) {
  uint32_t h;
  if (FMT == KQ_FP4_MX) {
    h = small ? (byte + 126u) << 7 : (byte == 0xffu ? 0x7fc0u : (byte ? byte << 7 : 0x0040u));
  } else {
    const float s = kq::fp4::e4m3_value(byte) * 0x1p118f;
    h = __float_as_uint(s) >> 16;
  }
  return h | (h << 16);
}

// Spread codes times their scale.  MX: with a scale up to 2 (`small`) its 2^126
// fits in the factor, else 2^126 goes first.
template <int FMT>
__device__ __forceinline__ uint32_t weight(uint32_t spread_pair, uint32_t scale, bool small) {
  if (FMT == KQ_FP4_MX && !small) spread_pair = mul_bf16x2(spread_pair, 0x7e807e80u);
  return mul_bf16x2(spread_pair, scale);
}

// 32 elements of a bf16 vector from column k as 16 words, zeros past d_in.  Plain loads
// here and below: the kernel ahead on the stream may still write x while this one is being
// scheduled, which the read-only path does not allow for.
__device__ __forceinline__ void load_x(const __nv_bfloat16* x, int64_t k, int64_t d_in, bool vec, uint32_t (&w)[16]) {
  if (vec && k + 32 <= d_in) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 q = *reinterpret_cast<const uint4*>(x + k + 8 * i);
      w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (k + i < d_in) w[i / 2] |= (uint32_t)__bfloat16_as_ushort(x[k + i]) << (16 * (i & 1));
  }
}

// Three bf16 parts of an fp32 value in the top halves of three words, by
// truncation, 8 bits each: exact.  A value without a finite remainder (NaN, Inf)
// is its first part alone.
__device__ __forceinline__ void split3(float x, uint32_t (&part)[3]) {
  const uint32_t bits = __float_as_uint(x);
  const bool finite = (bits & 0x7f800000u) != 0x7f800000u;
  // a NaN whose top bits are zero stays one
  part[0] = x != x ? bits | 0x400000u : bits;
  const float r1 = finite ? x - __uint_as_float(bits & 0xffff0000u) : 0.f;
  part[1] = __float_as_uint(r1);
  part[2] = __float_as_uint(r1 - __uint_as_float(part[1] & 0xffff0000u));
}

__device__ __forceinline__ float ld_cluster(const float* mine, uint32_t rank) {
  uint32_t at;
  float v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kWarps * 32, sizeof(T) == 4 ? 3 : 4) matvec_kernel(const MatvecParams p) {
  constexpr bool STAGED = sizeof(T) == 4;
  constexpr int PARTS = STAGED ? 3 : 1;
  constexpr int ROWS = STAGED ? 16 * kWarps : 16;   // rows of a CTA
  constexpr int KW = STAGED ? 1 : kWarps;           // its warps along K
  __shared__ float sums[KW][ROWS][8];
  extern __shared__ uint4 xs[];   // [step][part][lane][4 pieces of 16 bytes], pieces swizzled by lane
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int rank = STAGED ? (int)blockIdx.x % p.ks : 0;
  const int64_t row0 = (int64_t)(STAGED ? blockIdx.x / p.ks : blockIdx.x) * ROWS, r0 = row0 + (STAGED ? 16 * warp : 0);
  // this warp's steps: first, first + KW, ... below last
  const int steps = (int)((p.d_in + 127) / 128), padded = (int)((p.d_in + 31) / 32 * 32);
  const int first = STAGED ? (int)((int64_t)steps * rank / p.ks) : warp;
  const int last = STAGED ? (int)((int64_t)steps * (rank + 1) / p.ks) : steps;
  // the lane's place in its two rows at step `first` (a row past the end reads the last one; never stored)
  const uint8_t* codes[2];
  const uint8_t* scales[2];   // the 4-byte word of four blocks that holds the lane's one (MX) or two (NV)
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t r = min(r0 + g + 8 * h, p.d_out - 1);
    codes[h] = p.codes + r * p.ldc + 16 * t + 64 * (int64_t)first;
    scales[h] = p.scales + kq::fp4::scale_offset(r, FMT == KQ_FP4_MX ? 4 * (int64_t)first : 8 * (int64_t)first + 4 * (t / 2), p.kat);
  }
  __shared__ uint4 code_ring[kDepth][2][kWarps * 32];
  __shared__ uint32_t scale_ring[kDepth][2][kWarps * 32];
  kq::pdl_wait();
  kq::pdl_trigger();

  // the copies of step `first + KW n` into slot n % kDepth; columns past the matrix are zeros
  auto fetch = [&](int n) {
    const int step = first + KW * n, slot = n & (kDepth - 1);
    if (step < last) {
      const int64_t ahead = (int64_t)KW * n;
      const int bytes = 128 * step + 32 * t < padded ? 16 : 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t c = (uint32_t)__cvta_generic_to_shared(&code_ring[slot][h][threadIdx.x]);
        const uint32_t z = (uint32_t)__cvta_generic_to_shared(&scale_ring[slot][h][threadIdx.x]);
        const uint8_t* src = bytes ? codes[h] + 64 * ahead : p.codes;
        const uint8_t* srs = bytes ? scales[h] + (FMT == KQ_FP4_MX ? 512 : 1024) * ahead : p.scales;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(c), "l"(src), "r"(bytes) : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(z), "l"(srs), "r"(bytes / 4) : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  float acc[4] = {0.f, 0.f, 0.f, 0.f};

#pragma unroll
  for (int n = 0; n < kDepth - 1; ++n) fetch(n);
  int piece0 = 0, staged = 0;   // the parts of steps piece0 .. staged - 1 are in shared memory
  if (STAGED) {
    // vectors past the batch: zeros, written once
    for (int i = threadIdx.x; i < min(last - first, kStageSteps) * PARTS * 128; i += kWarps * 32)
      if ((i / 4 % 32) / 4 >= p.batch) xs[i] = make_uint4(0, 0, 0, 0);
    staged = first;
  }
  for (int step = first; step < last; step += KW) {
    if (STAGED && step == staged) {
      // the parts of the next steps' x: a thread takes (step, lane) slots of the batch
      const int n = min(kStageSteps, last - step);
      __syncthreads();
      for (int i = threadIdx.x; i < n * 4 * p.batch; i += kWarps * 32) {
        const int at = i / (4 * p.batch), slot = i % (4 * p.batch);   // slot: the lane it serves
        const float* x = static_cast<const float*>(p.X) + (slot / 4) * p.ldx;
        const int64_t k = 128 * (int64_t)(step + at) + 32 * (slot % 4);
        float v[32];
        if (p.x_vec && k + 32 <= p.d_in) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            asm volatile("ld.global.v4.f32 {%0,%1,%2,%3}, [%4];"
                         : "=f"(v[e]), "=f"(v[e + 1]), "=f"(v[e + 2]), "=f"(v[e + 3])
                         : "l"(x + k + e));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = k + e < p.d_in ? x[k + e] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t b[3][4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t lo[3], hi[3];
            split3(v[8 * j + q], lo);
            split3(v[8 * j + q + 4], hi);
#pragma unroll
            for (int part = 0; part < 3; ++part) b[part][q] = __byte_perm(lo[part], hi[part], 0x7632);
          }
#pragma unroll
          for (int part = 0; part < 3; ++part)
            xs[((at * 3 + part) * 32 + slot) * 4 + (j ^ ((slot >> 1) & 3))] =
                make_uint4(b[part][0], b[part][1], b[part][2], b[part][3]);
        }
      }
      __syncthreads();
      piece0 = step;
      staged += n;
    }
    uint32_t xw[STAGED ? 1 : 16];
    if constexpr (!STAGED) {
#pragma unroll
      for (int i = 0; i < 16; ++i) xw[i] = 0;
      if (g < p.batch) load_x(static_cast<const __nv_bfloat16*>(p.X) + g * p.ldx, 128 * (int64_t)step + 32 * t, p.d_in, p.x_vec, xw);
    }
    const int n = (step - first) / KW, slot = n & (kDepth - 1);
    fetch(n + kDepth - 1);   // into the slot that was read in the last step
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
    const uint4 w[2] = {code_ring[slot][0][threadIdx.x], code_ring[slot][1][threadIdx.x]};
    uint32_t s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t word = scale_ring[slot][h][threadIdx.x];
      s[h] = FMT == KQ_FP4_MX ? word >> (8 * t) & 0xffu : word >> (16 * (t & 1)) & 0xffffu;
    }
    const bool small = FMT == KQ_FP4_MX && !__any_sync(0xffffffffu, max(s[0], s[1]) > 128u);
    uint32_t sc[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      sc[h][0] = scale_pair<FMT>(s[h] & 0xffu, small);
      sc[h][1] = FMT == KQ_FP4_MX ? sc[h][0] : scale_pair<FMT>(s[h] >> 8, small);
    }
    // the tensor core truncates as it accumulates: one chain per 128 columns (and
    // part), the chains summed in rounded fp32, the smallest part first
    float chain[PARTS][4];
#pragma unroll
    for (int c = 0; c < PARTS; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) chain[c][i] = 0.f;
    const uint4* xstep = xs + (STAGED ? step - piece0 : 0) * PARTS * 128 + lane * 4;
    auto products = [&](bool sm) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w0 = j == 0 ? w[0].x : (j == 1 ? w[0].y : (j == 2 ? w[0].z : w[0].w));
        const uint32_t w1 = j == 0 ? w[1].x : (j == 1 ? w[1].y : (j == 2 ? w[1].z : w[1].w));
        const uint32_t c0 = sc[0][j / 2], c1 = sc[1][j / 2];
        const uint32_t a[8] = {weight<FMT>(spread<0>(w0), c0, sm), weight<FMT>(spread<0>(w1), c1, sm),
                               weight<FMT>(spread<1>(w0), c0, sm), weight<FMT>(spread<1>(w1), c1, sm),
                               weight<FMT>(spread<2>(w0), c0, sm), weight<FMT>(spread<2>(w1), c1, sm),
                               weight<FMT>(spread<3>(w0), c0, sm), weight<FMT>(spread<3>(w1), c1, sm)};
#pragma unroll
        for (int part = 0; part < PARTS; ++part) {
          uint4 b;
          if constexpr (STAGED)
            b = xstep[part * 128 + (j ^ ((lane >> 1) & 3))];
          else
            b = make_uint4(__byte_perm(xw[4 * j], xw[4 * j + 2], 0x5410), __byte_perm(xw[4 * j], xw[4 * j + 2], 0x7632),
                           __byte_perm(xw[4 * j + 1], xw[4 * j + 3], 0x5410), __byte_perm(xw[4 * j + 1], xw[4 * j + 3], 0x7632));
          mma16816(chain[part], a[0], a[1], a[2], a[3], b.x, b.y);
          mma16816(chain[part], a[4], a[5], a[6], a[7], b.z, b.w);
        }
      }
    };
    if (FMT == KQ_FP4_NV || small)
      products(true);
    else
      products(false);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float sum = chain[PARTS - 1][i];
#pragma unroll
      for (int c = PARTS - 2; c >= 0; --c) sum += chain[c][i];
      acc[i] += sum;
    }
  }
  float(*mine)[8] = &sums[STAGED ? 0 : warp][STAGED ? 16 * warp : 0];
  mine[g][2 * t] = acc[0];
  mine[g][2 * t + 1] = acc[1];
  mine[g + 8][2 * t] = acc[2];
  mine[g + 8][2 * t + 1] = acc[3];
  auto sync = [&] {
    if (STAGED && p.ks > 1)
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    else
      __syncthreads();
  };
  sync();
  // the row block's outputs, dealt to the cluster's CTAs
  const int ctas = STAGED ? p.ks : 1;
  for (int i = threadIdx.x + kWarps * 32 * rank; i < ROWS * p.batch; i += kWarps * 32 * ctas) {
    const int row = i % ROWS, n = i / ROWS;
    const int64_t r = row0 + row;
    float v[8], y = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if constexpr (STAGED)
        v[q] = q < ctas ? (ctas > 1 ? ld_cluster(&sums[0][row][n], q) : sums[0][row][n]) : 0.f;
      else
        v[q] = sums[q][row][n];
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) y += v[q];
    if (r < p.d_out) {
      if (FMT == KQ_FP4_NV) y *= 256.f * (p.g ? *p.g : 1.f);
      if constexpr (STAGED)
        static_cast<float*>(p.Y)[n * p.ldy + r] = y;
      else
        static_cast<__nv_bfloat16*>(p.Y)[n * p.ldy + r] = __float2bfloat16_rn(y);
    }
  }
  if (STAGED && p.ks > 1) sync();   // the sums stay until every CTA has read them
}

template <typename T, int FMT, int ROW_LANES>
kq_status launch_pieces(const QuantParams& p, cudaStream_t st) {
  const dim3 grid((unsigned)kq::cdiv(kq::cdiv(p.rows, 128) * 128, 8 * 2 * (32 / ROW_LANES)),
                  (unsigned)kq::cdiv((int64_t)p.kat * 4 * block_of(FMT), 16 * ROW_LANES));
  return kq::launch_ex("kq_fp4_quantize", true, quantize_kernel<T, FMT, ROW_LANES>, grid, dim3(256), 0, st, p);
}

template <typename T, int FMT>
kq_status launch_quantize(const QuantParams& p, cudaStream_t st) {
  // up to 384 columns, pieces of 128 leave fewer lanes idle than pieces of 512
  return p.cols <= 384 ? launch_pieces<T, FMT, 8>(p, st) : launch_pieces<T, FMT, 32>(p, st);
}

template <typename T, int FMT>
kq_status launch_matvec(MatvecParams p, cudaStream_t st) {
  const char* what = "kq_fp4_matvec";
  constexpr bool STAGED = sizeof(T) == 4;
  const int64_t steps = kq::cdiv(p.d_in, 128);
  p.ks = !STAGED ? 1 : (steps >= 8 ? 8 : (steps >= 4 ? 4 : (steps >= 2 ? 2 : 1)));
  const int smem = STAGED ? (int)std::min<int64_t>(kStageSteps, kq::cdiv(steps, p.ks)) * 6144 : 0;
  // the attribute belongs to the device: set on every call that needs it, as the current device may change
  if (STAGED)
    KQ_TRY(kq::cuda_check(cudaFuncSetAttribute(matvec_kernel<T, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kStageSteps * 6144), what));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(kq::cdiv(p.d_out, STAGED ? 16 * kWarps : 16) * p.ks));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.ks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.ks > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, matvec_kernel<T, FMT>, p);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return kq::cuda_check(e, what);
  }
  return kq::launch_check(what);
}

}  // namespace

extern "C" size_t kq_fp4_scale_bytes(int64_t rows, int64_t cols, int format) {
  if (rows < 0 || cols < 1 || (format != KQ_FP4_MX && format != KQ_FP4_NV)) return 0;
  return (size_t)kq::cdiv(rows, 128) * (size_t)kq::fp4::scale_tiles(cols, format) * 512;
}

extern "C" kq_status kq_fp4_quantize(const void* M, int dtype, int64_t ldm, const kq_fp4* Q, float* M_hat, int64_t ldh,
                                     int32_t* info, kq_stream_t stream) {
  KQ_TRY(kq::fp4::check(Q, "kq_fp4_quantize", "Q"));
  if (dtype != KQ_F32 && dtype != KQ_BF16) return kq::fail(KQ_ERR_INVALID_ARG, "kq_fp4_quantize: dtype must be KQ_F32 or KQ_BF16");
  if (!info) return kq::fail(KQ_ERR_INVALID_ARG, "kq_fp4_quantize: NULL pointer");
  if (Q->rows == 0) {
    kq::clear_error();
    return KQ_OK;
  }
  if (!M) return kq::fail(KQ_ERR_INVALID_ARG, "kq_fp4_quantize: NULL pointer");
  if (Q->format == KQ_FP4_NV && !Q->gscale) return kq::fail(KQ_ERR_INVALID_ARG, "kq_fp4_quantize: KQ_FP4_NV needs gscale");
  const size_t esize = dtype == KQ_F32 ? 4 : 2;
  if (ldm < Q->cols || (M_hat && ldh < Q->cols)) return kq::fail(KQ_ERR_INVALID_ARG, "kq_fp4_quantize: leading dimension too small");
  if (!kq::aligned(M, esize) || (M_hat && !kq::aligned(M_hat, 4)))
    return kq::fail(KQ_ERR_ALIGNMENT, "kq_fp4_quantize: M and M_hat aligned to their elements");
  if (M_hat == M) return kq::fail(KQ_ERR_INVALID_ARG, "kq_fp4_quantize: M_hat must not overlap M");
  QuantParams p = {};
  p.rows = Q->rows;
  p.cols = (int)Q->cols;
  p.ldm = ldm;
  p.ldc = Q->ld;
  p.ldh = ldh;
  p.kat = (int)kq::fp4::scale_tiles(Q->cols, Q->format);
  p.M = M;
  p.g = Q->gscale;
  p.codes = Q->codes;
  p.scales = Q->scales;
  p.M_hat = M_hat;
  p.m_access = access_of(M, ldm * (int64_t)esize);
  p.h_access = access_of(M_hat, ldh * 4);
  p.info = info;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == KQ_F32)
    KQ_TRY(Q->format == KQ_FP4_MX ? (launch_quantize<float, KQ_FP4_MX>(p, st)) : (launch_quantize<float, KQ_FP4_NV>(p, st)));
  else
    KQ_TRY(Q->format == KQ_FP4_MX ? (launch_quantize<__nv_bfloat16, KQ_FP4_MX>(p, st))
                                  : (launch_quantize<__nv_bfloat16, KQ_FP4_NV>(p, st)));
  kq::clear_error();
  return KQ_OK;
}

extern "C" kq_status kq_fp4_matvec(const kq_fp4* W, const void* X, int dtype, int64_t ldx, int batch, void* Y, int64_t ldy,
                                   kq_stream_t stream) {
  KQ_TRY(kq::fp4::check(W, "kq_fp4_matvec", "W"));
  if (dtype != KQ_F32 && dtype != KQ_BF16) return kq::fail(KQ_ERR_INVALID_ARG, "kq_fp4_matvec: dtype must be KQ_F32 or KQ_BF16");
  if (batch < 1 || batch > 8) return kq::fail(KQ_ERR_UNSUPPORTED_SHAPE, "kq_fp4_matvec: batch outside 1..8");
  if (W->rows == 0) {
    kq::clear_error();
    return KQ_OK;
  }
  if (!X || !Y) return kq::fail(KQ_ERR_INVALID_ARG, "kq_fp4_matvec: NULL pointer");
  if (ldx < W->cols || ldy < W->rows) return kq::fail(KQ_ERR_INVALID_ARG, "kq_fp4_matvec: leading dimension too small");
  const size_t esize = dtype == KQ_F32 ? 4 : 2;
  if (!kq::aligned(X, esize) || !kq::aligned(Y, esize))
    return kq::fail(KQ_ERR_ALIGNMENT, "kq_fp4_matvec: X and Y aligned to their elements");
  MatvecParams p = {};
  p.codes = W->codes;
  p.scales = W->scales;
  p.g = W->gscale;
  p.d_out = W->rows;
  p.d_in = W->cols;
  p.ldc = W->ld;
  p.kat = kq::fp4::scale_tiles(W->cols, W->format);
  p.X = X;
  p.ldx = ldx;
  p.x_vec = kq::aligned(X, 16) && (batch == 1 || (ldx * (int64_t)esize) % 16 == 0);
  p.batch = batch;
  p.Y = Y;
  p.ldy = ldy;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == KQ_F32)
    KQ_TRY(W->format == KQ_FP4_MX ? (launch_matvec<float, KQ_FP4_MX>(p, st)) : (launch_matvec<float, KQ_FP4_NV>(p, st)));
  else
    KQ_TRY(W->format == KQ_FP4_MX ? (launch_matvec<__nv_bfloat16, KQ_FP4_MX>(p, st))
                                  : (launch_matvec<__nv_bfloat16, KQ_FP4_NV>(p, st)));
  kq::clear_error();
  return KQ_OK;
}
