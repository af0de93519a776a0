// Device-side building blocks shared by the attention kernels (gfx950), and the launchers.
//
// With value = code * scale + zero, per group g of dims,
//   q . k_t = sum_g ks[t,g] (sum_{d in g} q_d c[t,d]) + kz[t,g] (sum_{d in g} q_d)
//   o_d     = sum_t p_t vs[t,g] (c[t,d] - 8) + sum_t p_t (vz + 8 vs)[t,g]
// so the codes enter the matrix products as the whole numbers they are, and the parameters stay in
// fp32.  A parameter of a token that a query does not see is replaced before it multiplies
// anything, and codes are always finite, so whatever bits lie in unseen slots cannot reach a result.
//
// Codes become fp16 operands with one AND each: a nibble in the low bits of an fp16 pattern is the
// subnormal code * 2^-24 (bits 0..3) or code * 2^-20 (bits 4..7), which the MFMA multiplies exactly;
// the powers of two are taken out of the fp32 result.  Both element types therefore use the fp16
// MFMA (16x16x32).  Each query row is scaled by a power of two, so that its largest finite element lies below
// 2^14 (in [2^13, 2^14) in the rows kernel): bf16 queries fit fp16 exactly down to 2^-27 of that.
//
// The scores are computed transposed, S^T = K Q^T: lane l holds query row l & 15 and tokens
// 4 (l >> 4) .. + 3, which is the operand layout of P^T in O^T = V^T P^T (the contraction runs over
// tokens in that order), so the weights never leave their lane.
#pragma once

#include <hip/hip_runtime.h>

#include "qgemm_attention_geometry.h"
#include "qgemm_attention_internal.h"

namespace qgemm {
namespace attn {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

struct AttnArgs {
  const uint16_t* q;
  const uint8_t* data;
  const int *table, *lens, *starts;
  uint16_t* out;
  long long qs, os;                // token strides in elements
  int total_q, batch, kv_heads, ratio, max_pages, page, num_pages;
  int codes, params, block;        // bytes of one side's codes, of its parameters, of a block
  unsigned page_mul, page_shift;   // t / page = (t * page_mul) >> (32 + page_shift) for t < 2^30
  int max_q, causal, window;
  // rows kernel: while a workgroup's even share is at most piece_share units of 64 tokens, pieces are of
  // twice that share and at least of piece_least units
  int piece_share, piece_least;
  int splits;                      // tiles kernel: workgroups per row tile
  float scale;                     // the caller's scale * log2(e)
  unsigned* tickets;
  float* partials;
};

constexpr unsigned kLow = 0x000F000Fu, kHigh = 0x00F000F0u;
constexpr float kStart = -0x1.fffffep127f;   // running maximum before the first token: no score is below
// Rows kernel: a running maximum is moved when a score exceeds it by kSlack (in bits); weights times scales
// enter the matrix products in units that keep them below kTop, inside fp16.
constexpr float kSlack = 8.0f, kTop = 0x1p15f;

template <bool BF>
__device__ __forceinline__ float from16(unsigned bits) {
  if constexpr (BF) return __builtin_bit_cast(float, bits << 16);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}
// scale (low half) and zero (high half) of a parameter word
template <bool BF>
__device__ __forceinline__ float par_scale(unsigned w) {
  if constexpr (BF) return __builtin_bit_cast(float, w << 16);
  else return (float)__builtin_bit_cast(f16x2, w)[0];
}
template <bool BF>
__device__ __forceinline__ float par_zero(unsigned w) {
  if constexpr (BF) return __builtin_bit_cast(float, w & 0xffff0000u);
  else return (float)__builtin_bit_cast(f16x2, w)[1];
}
template <bool BF>
__device__ __forceinline__ unsigned pack2(float a, float b) {
  if constexpr (BF) return __builtin_bit_cast(unsigned, bf16x2{(__bf16)a, (__bf16)b});
  else return __builtin_bit_cast(unsigned, f16x2{(_Float16)a, (_Float16)b});
}
__device__ __forceinline__ unsigned pack_f16(float a, float b) {
  return __builtin_bit_cast(unsigned, f16x2{(_Float16)a, (_Float16)b});
}

// Eight codes of one dword as fp16 pairs: nibbles (0, 4), (1, 5), (2, 6), (3, 7); the first and third
// pair carry 2^-24, the others 2^-20.
__device__ __forceinline__ u32x4 codes8(unsigned w) {
  const unsigned h = w >> 8;
  return u32x4{w & kLow, w & kHigh, h & kLow, h & kHigh};
}
// The dims, within the dword's eight, of those pairs' slots.
__device__ constexpr int kSlotDim[8] = {0, 4, 1, 5, 2, 6, 3, 7};

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
// A row of 16 lanes turned by DPP control word C (row_ror n: 0x120 + n).
template <int C>
__device__ __forceinline__ unsigned dpp(unsigned x) {
  return (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, C, 0xf, 0xf, false);
}
// Reductions over a wavefront's four rows of 16 lanes, every lane holding the result: a value swapped with
// itself between odd and even rows (then halves) leaves both partners in every lane, in registers, where an
// exchange through LDS would wait for its round trip.
__device__ __forceinline__ float as_float(unsigned x) { return __builtin_bit_cast(float, x); }
template <class F>
__device__ __forceinline__ float over_rows(float x, F f) {
  const unsigned b = __builtin_bit_cast(unsigned, x);
  const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  const unsigned c = __builtin_bit_cast(unsigned, f(as_float(r[0]), as_float(r[1])));
  const auto h = __builtin_amdgcn_permlane32_swap(c, c, false, false);
  return f(as_float(h[0]), as_float(h[1]));
}
__device__ __forceinline__ float sum_rows(float x) {
  return over_rows(x, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float max_rows(float x) {
  return over_rows(x, [](float a, float b) { return __builtin_fmaxf(a, b); });
}
// The exponent of a power of two within the normal range.
__device__ __forceinline__ int exponent_of(float x) { return (int)(__builtin_bit_cast(unsigned, x) >> 23) - 127; }
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// V codes of one 16-token subtile, as loaded (lane r = l & 15, tokens 4 (l >> 4) .. + 3), for tile i:
// the fp16 pairs of tokens (0, 1) and (2, 3) of dim 16 i + r.  Odd i carries 2^-20, even 2^-24.
template <int U>
__device__ __forceinline__ void v_pairs(const unsigned (&w)[U], int i, unsigned& p01, unsigned& p23) {
  unsigned a, b;
  if constexpr (U == 2) {
    a = w[0];
    b = w[1];
  } else {
    constexpr int S = U / 4;                       // dwords per token
    const unsigned sel = (i & 4) ? 0x07060302u : 0x05040100u;
    const int h = S == 2 ? i >> 3 : 0;
    a = __builtin_amdgcn_perm(w[S + h], w[h], sel);
    b = __builtin_amdgcn_perm(w[3 * S + h], w[2 * S + h], sel);
  }
  const unsigned m = (i & 1) ? kHigh : kLow;
  p01 = ((i & 2) ? a >> 8 : a) & m;
  p23 = ((i & 2) ? b >> 8 : b) & m;
}

// The same pair, c 2^-24 (even tile) or c 2^-20, as the whole numbers c - 8.
__device__ __forceinline__ unsigned centre(unsigned pair, bool high) {
  const f16x2 v = __builtin_bit_cast(f16x2, pair | (high ? 0x54005400u : 0x64006400u));      // 64 + c or 1024 + c
  const _Float16 off = high ? (_Float16)72.f : (_Float16)1032.f;
  return __builtin_bit_cast(unsigned, v - f16x2{off, off});
}

// The same as the whole numbers c.
__device__ __forceinline__ f16x2 whole(unsigned pair, bool high) {
  const f16x2 v = __builtin_bit_cast(f16x2, pair | (high ? 0x54005400u : 0x64006400u));
  const _Float16 off = high ? (_Float16)64.f : (_Float16)1024.f;
  return v - f16x2{off, off};
}

__device__ __forceinline__ int page_of(const AttnArgs& a, int t) {
  return (int)(__umulhi((unsigned)t, a.page_mul) >> a.page_shift);
}

// Sum up to and including each lane, by DPP: within rows of 16 lanes, then across them.
template <int C, int ROWS>
__device__ __forceinline__ int dpp_add(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, C, ROWS, 0xf, false);
}
__device__ __forceinline__ int wave_scan(int v) {
  v = dpp_add<0x111, 0xf>(v);                      // row_shr 1, 2, 4, 8
  v = dpp_add<0x112, 0xf>(v);
  v = dpp_add<0x114, 0xf>(v);
  v = dpp_add<0x118, 0xf>(v);
  v = dpp_add<0x142, 0xa>(v);                      // lane 15 of rows 0 and 2 to the next row
  return dpp_add<0x143, 0xc>(v);                   // lane 31 to rows 2 and 3
}
__device__ __forceinline__ int wave_sum(int v) { return __builtin_amdgcn_readlane(wave_scan(v), 63); }

// Sequence b's geometry from device memory.
__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int b) {
  return seq_of(a.starts[b], a.starts[b + 1], a.lens[b], a.total_q, a.max_q, a.max_pages * a.page, a.window);
}

// Device-scope (sc1) accesses for partial results: they pass by the XCD's own L2, so a workgroup on
// another XCD sees them without cache maintenance.
constexpr int kCPolDevice = 16;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(void* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(p, (short)0, bytes, 0x00020000);
}
__device__ __forceinline__ void store4(__amdgpu_buffer_rsrc_t r, int at, f32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, at, 0, kCPolDevice);
}
__device__ __forceinline__ f32x4 load4(__amdgpu_buffer_rsrc_t r, int at) {
  return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, kCPolDevice));
}

// Launchers of one element type and head dim; each kernel source instantiates these per object.
template <bool BF, int D>
hipError_t launch_rows(const AttnPlan& pl, const AttnArgs& a, hipStream_t s);
template <bool BF, int D>
hipError_t launch_tiles(const AttnPlan& pl, const AttnArgs& a, hipStream_t s);

}  // namespace attn
}  // namespace qgemm
