// Device-side building blocks shared by the 8-bit operators (gfx950), and the launchers.
#pragma once

#include <hip/hip_runtime.h>

#include "qgemm_w8a8_internal.h"

namespace qgemm {
namespace w8 {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

// Largest magnitude of the 16 lanes of a row (the lanes of one scale block), as the bits of a float:
// compared as whole numbers, a NaN is larger than infinity and infinity larger than any number, so neither
// is lost as it would be by a floating maximum.
__device__ __forceinline__ unsigned max_row16(unsigned m) {
  m = max(m, (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, 0x128, 0xf, 0xf, false));   // row_ror:8
  m = max(m, (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, 0x124, 0xf, 0xf, false));
  m = max(m, (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, 0x122, 0xf, 0xf, false));
  m = max(m, (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, 0x121, 0xf, 0xf, false));
  return m;
}
__device__ __forceinline__ unsigned magnitude(float v) { return __builtin_bit_cast(unsigned, v) & 0x7fffffffu; }

// Scale of a block whose largest |value| is `amax` (bits), and the factor from `unit` times its values to
// codes: values y are held as y = t * r, with t at hand, and amax that of t.  r lies in [1, 2): then t is as large as y, and
// neither factor leaves fp32's range, however small the block.
struct BlockScale { float scale, to_code; };
__device__ __forceinline__ BlockScale block_scale(unsigned amax_bits, float r) {
  constexpr float kLeast = 0x1p-100f;
  const float amax = __builtin_bit_cast(float, amax_bits), y = amax * r;
  BlockScale s;
  if (y < kLeast) {
    s.scale = kLeast / 448.0f;
    s.to_code = r * (448.0f / kLeast);
  } else if (y <= 3.402823466e38f) {
    s.scale = y * (1.0f / 448.0f);
    s.to_code = 448.0f / amax;                       // r cancels in y / scale: one rounding, not three
  } else {
    s.scale = s.to_code = __builtin_nanf("");
  }
  return s;
}
// Sixteen e4m3 codes as two fp16 operands of eight (exact).
//
// The e4m3 MFMA adds the products of eight consecutive k (one lane's eight bytes) after aligning them to the largest
// and cutting them off at 2^-13 of its power of two; only those sums are added in fp32 (measured bit by bit: beside a product of
// 2^16, one of 2^3 counts in the same eight and one of 2^2 does not, in another eight one of 2^-7 does).  That leaves
// a block sum 1.4e-5 of its root mean square off for normal values, 2.4e-5 where some k are ten times as large.  An output
// rounded to 16 bits shows it only where large products cancel; outputs in fp32 and the scales of outputs in 8 bits always do,
// and are made from fp16 operands, whose products and sums are fp32 throughout, at half the MFMA rate.  16-bit outputs are where
// the caller asks for it (QGEMM_W8A8_SUMS_WHOLE).
struct Halves { f16x8 v[2]; };
__device__ __forceinline__ Halves halves(i32x4 codes) {
  Halves h;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned c = (unsigned)codes[i];
    const f16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, false);
    const f16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, true);
    h.v[i >> 1][4 * (i & 1)] = lo[0];
    h.v[i >> 1][4 * (i & 1) + 1] = lo[1];
    h.v[i >> 1][4 * (i & 1) + 2] = hi[0];
    h.v[i >> 1][4 * (i & 1) + 3] = hi[1];
  }
  return h;
}
// Four codes of four values; 448 (1 + 2^-22) still rounds to 448.
__device__ __forceinline__ unsigned codes4(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
}

hipError_t launch_rows(const W8Plan& pl, const W8Args& a, hipStream_t stream);
hipError_t launch_tiles(const W8Plan& pl, const W8Args& a, hipStream_t stream);

}  // namespace w8
}  // namespace qgemm
