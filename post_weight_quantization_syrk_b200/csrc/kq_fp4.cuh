// Layout helpers of the microscaled 4-bit formats (internal).
#pragma once

#include <algorithm>

#include "kq_internal.cuh"

namespace kq {
namespace fp4 {

__host__ __device__ constexpr int block_of(int format) { return format == KQ_FP4_MX ? 32 : 16; }

// Scale tiles (128 rows x 4 blocks, 512 bytes) along a row.
inline int64_t scale_tiles(int64_t cols, int format) { return cdiv(cdiv(cols, block_of(format)), 4); }

// Byte of row r, block kb, with kat scale tiles along a row.
__device__ __forceinline__ int64_t scale_offset(int64_t r, int64_t kb, int64_t kat) {
  return ((r >> 7) * kat + (kb >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (kb & 3);
}

// Value of an E4M3 byte (NaN for 0x7f).
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  if ((byte & 0x7fu) == 0x7fu) return __uint_as_float(0x7fc00000u);
  // exponent and mantissa on top of an fp32, bias 127 against 7: exact, subnormals included
  const float v = __uint_as_float((byte & 0x7fu) << 20) * 0x1p120f;
  return byte & 0x80u ? -v : v;
}

// Host checks of a matrix description.
inline kq_status check(const kq_fp4* q, const char* what, const char* name) {
  if (!q) return fail(KQ_ERR_INVALID_ARG, "%s: %s is NULL", what, name);
  if (q->format != KQ_FP4_MX && q->format != KQ_FP4_NV)
    return fail(KQ_ERR_INVALID_ARG, "%s: %s has an unknown format", what, name);
  if (q->rows < 0 || q->cols < 1) return fail(KQ_ERR_INVALID_ARG, "%s: %s needs rows >= 0 and cols >= 1", what, name);
  if (q->rows > (1 << 30) || q->cols > (1 << 24))
    return fail(KQ_ERR_UNSUPPORTED_SHAPE, "%s: %s above 2^30 rows or 2^24 columns", what, name);
  if (cdiv(q->rows, 128) * scale_tiles(q->cols, q->format) > 0x7fffffff)   // TMA coordinates are 32 bits
    return fail(KQ_ERR_UNSUPPORTED_SHAPE, "%s: %s has more than 2^31 - 1 scale tiles", what, name);
  if (q->rows > 0 && (!q->codes || !q->scales)) return fail(KQ_ERR_INVALID_ARG, "%s: %s has a NULL pointer", what, name);
  if (q->ld < cdiv(q->cols, 32) * 16) return fail(KQ_ERR_INVALID_ARG, "%s: %s leading dimension too small", what, name);
  if (!aligned(q->codes, 16) || !aligned(q->scales, 16) || (q->ld & 15) || !aligned(q->gscale, 4))
    return fail(KQ_ERR_ALIGNMENT, "%s: %s codes and scales 16-byte aligned, ld %% 16 == 0", what, name);
  if (q->format == KQ_FP4_MX && q->gscale) return fail(KQ_ERR_INVALID_ARG, "%s: %s is KQ_FP4_MX and has a gscale", what, name);
  return KQ_OK;
}

}  // namespace fp4
}  // namespace kq
