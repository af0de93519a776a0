// qgemm_add_norm: the residual's addition, the RMS norm and the rounding to 16 or 8 bits, in one pass.
//
//   s = x + residual,  y = s / sqrt(mean(s^2) + eps) * w,  16 bits: RNE(y);  8 bits: per block of 128
//   scale = max|y| / 448, code = e4m3(y / scale) = e4m3(s w 448 / max|s w|)
//
// Bound by memory, for few tokens by one trip to it.  A workgroup (or a wavefront) holds a row in registers, C chunks of eight
// values per thread, so it is read once: the sum of squares is reduced over the threads, and a scale block is the sixteen
// lanes of one DPP row.  8192 x 5120: 61.5 us to 16 bits (5.5 TB/s), 58.3 to 8 (5.0 TB/s); 16 x 4096: 2.4 and 2.7 us.
#include "qgemm_w8a8_device.h"

namespace {

using namespace qgemm;
using namespace qgemm::w8;

struct NormArgs {
  const uint16_t *x, *r, *w;
  uint16_t* sum;
  void* y;
  float* ys;
  long long xs, rs, ss;             // token strides in elements
  int tokens, dim, norm;
  float eps;
};

template <bool BF>
__device__ __forceinline__ void unpack8(u32x4 v, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF) {
      f[2 * i] = __builtin_bit_cast(float, v[i] << 16);
      f[2 * i + 1] = __builtin_bit_cast(float, v[i] & 0xffff0000u);
    } else {
      const unsigned two = v[i];                     // __builtin_bit_cast of a vector's element itself takes element 0
      const f16x2 h = __builtin_bit_cast(f16x2, two);
      f[2 * i] = (float)h[0];
      f[2 * i + 1] = (float)h[1];
    }
  }
}
template <bool BF>
__device__ __forceinline__ u32x4 pack8(const float* f) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF) {
      const bf16x2 h = {(__bf16)f[2 * i], (__bf16)f[2 * i + 1]};
      v[i] = __builtin_bit_cast(unsigned, h);
    } else {
      const f16x2 h = {(_Float16)f[2 * i], (_Float16)f[2 * i + 1]};
      v[i] = __builtin_bit_cast(unsigned, h);
    }
  }
  return v;
}

// WAVE: a row to each of a workgroup's four wavefronts; otherwise one to the workgroup.
template <bool BF, bool Q, bool WAVE, int C>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void add_norm(NormArgs a) {
  __shared__ float part[WAVE ? 1 : 16];
  const int T = WAVE ? 64 : blockDim.x, t = WAVE ? threadIdx.x & 63 : threadIdx.x;
  const int row = WAVE ? blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (WAVE && row >= a.tokens) return;
  const uint16_t* x = a.x + row * a.xs;
  const uint16_t* r = a.r ? a.r + row * a.rs : nullptr;
  u32x4 xv[C], rv[C], wv[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int d = 8 * (c * T + t);
    xv[c] = rv[c] = wv[c] = u32x4{};
    if (d < a.dim) {
      xv[c] = *reinterpret_cast<const u32x4*>(x + d);
      if (r) rv[c] = *reinterpret_cast<const u32x4*>(r + d);
      if (a.w) wv[c] = *reinterpret_cast<const u32x4*>(a.w + d);
    }
  }
  float s[C][8], sum = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    unpack8<BF>(xv[c], s[c]);
    if (r) {
      float v[8];
      unpack8<BF>(rv[c], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[c][i] += v[i];
    }
    const int d = 8 * (c * T + t);
    if (a.sum && d < a.dim) *reinterpret_cast<u32x4*>(a.sum + row * a.ss + d) = pack8<BF>(s[c]);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(s[c][i], s[c][i], sum);
  }
  float scale = 1.0f;
  if (a.norm) {
#pragma unroll
    for (int m = 1; m < 64; m *= 2) sum += __shfl_xor(sum, m);
    if constexpr (!WAVE) {
      if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
      __syncthreads();
      sum = 0.f;
      for (int i = 0; i < T / 64; ++i) sum += part[i];
    }
    scale = 1.0f / __builtin_sqrtf(sum / (float)a.dim + a.eps);
  }
  // 8 bits: the root's power of two goes to the values before the weight does, its rest in [1, 2) to the blocks' scales, so that
  // neither a small eps nor a small weight takes s w or a factor out of range.  (Infinite for a row of zeros and eps = 0,
  // whose codes are NaN as 0 / 0 is; 0 where the sum of squares is infinite.)
  const unsigned bits = __builtin_bit_cast(unsigned, scale);
  const float power = __builtin_bit_cast(float, bits & 0x7f800000u), rest = __builtin_bit_cast(float, (bits & 0x007fffffu) | 0x3f800000u);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int d = 8 * (c * T + t);
    float w[8];
    unpack8<BF>(wv[c], w);
    if constexpr (Q) {
      unsigned m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[c][i] *= power;
        if (a.w) s[c][i] *= w[i];
        m = max(m, magnitude(s[c][i]));
      }
      const BlockScale b = block_scale(max_row16(m), rest);   // a block is past the row's end as a whole
      if (d < a.dim) {
        const u32x2 v = {codes4(s[c][0] * b.to_code, s[c][1] * b.to_code, s[c][2] * b.to_code, s[c][3] * b.to_code),
                         codes4(s[c][4] * b.to_code, s[c][5] * b.to_code, s[c][6] * b.to_code, s[c][7] * b.to_code)};
        *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.y) + (size_t)row * a.dim + d) = v;
        if ((threadIdx.x & 15) == 0) a.ys[(size_t)(d / kBlock) * a.tokens + row] = b.scale;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[c][i] = a.w ? s[c][i] * scale * w[i] : s[c][i] * scale;
      if (d < a.dim) *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.y) + (size_t)row * a.dim + d) = pack8<BF>(s[c]);
    }
  }
}

template <bool WAVE, int C>
void launch(bool bf, bool quantized, int threads, hipStream_t s, const NormArgs& a) {
  const dim3 grid((unsigned)(WAVE ? (a.tokens + 3) / 4 : a.tokens)), block(threads);
  if (bf)
    quantized ? add_norm<true, true, WAVE, C><<<grid, block, 0, s>>>(a) : add_norm<true, false, WAVE, C><<<grid, block, 0, s>>>(a);
  else
    quantized ? add_norm<false, true, WAVE, C><<<grid, block, 0, s>>>(a) : add_norm<false, false, WAVE, C><<<grid, block, 0, s>>>(a);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

qgemm_status_t check_rows(const char* name, const void* p, int64_t stride, int dim) {
  if (!aligned(p, 16)) return fail(QGEMM_ERR_MISALIGNED, "%s must be 16-byte aligned", name);
  if (stride < dim || stride % 8 || stride > (int64_t(1) << 31))
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "%s token stride must be a multiple of 8 in [%d, 2^31], got %lld", name, dim,
                (long long)stride);
  return QGEMM_OK;
}

}  // namespace

extern "C" qgemm_status_t qgemm_add_norm(const qgemm_add_norm_t* p, const void* x, int64_t x_stride, const void* residual,
                                         int64_t residual_stride, const void* weight, void* sum_out, int64_t sum_stride,
                                         void* y, float* y_scales, void* stream) {
  clear_error();
  qgemm_status_t st = validate_add_norm(p);
  if (st != QGEMM_OK) return st;
  if (p->tokens == 0) return QGEMM_OK;
  const bool quantized = p->out_dtype == QGEMM_DT_FP8_E4M3;
  if (!x) return fail(QGEMM_ERR_INVALID_ARGUMENT, "x is NULL");
  if (!y) return fail(QGEMM_ERR_INVALID_ARGUMENT, "y is NULL");
  if (quantized && !y_scales) return fail(QGEMM_ERR_INVALID_ARGUMENT, "y_scales is NULL (needed for FP8_E4M3)");
  if (!quantized && y_scales) return fail(QGEMM_ERR_INVALID_ARGUMENT, "y_scales must be NULL for a 16-bit output");
  if ((st = check_rows("x", x, x_stride, p->dim)) != QGEMM_OK) return st;
  if (residual && (st = check_rows("residual", residual, residual_stride, p->dim)) != QGEMM_OK) return st;
  if (sum_out && (st = check_rows("sum_out", sum_out, sum_stride, p->dim)) != QGEMM_OK) return st;
  if (sum_out && ((sum_out == x && sum_stride != x_stride) || (sum_out == residual && sum_stride != residual_stride)))
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "sum_out in place needs its input's own stride, got %lld", (long long)sum_stride);
  if (p->norm && weight && !aligned(weight, 16)) return fail(QGEMM_ERR_MISALIGNED, "weight must be 16-byte aligned");
  if (!aligned(y, 16)) return fail(QGEMM_ERR_MISALIGNED, "y must be 16-byte aligned");
  if (!aligned(y_scales, 4)) return fail(QGEMM_ERR_MISALIGNED, "y_scales must be 4-byte aligned");
  if (y == x || y == residual || y == sum_out)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "y must not overlap x, residual or sum_out");
  NormArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.r = static_cast<const uint16_t*>(residual);
  a.w = p->norm ? static_cast<const uint16_t*>(weight) : nullptr;
  a.sum = static_cast<uint16_t*>(sum_out);
  a.y = y;
  a.ys = y_scales;
  a.xs = x_stride; a.rs = residual_stride; a.ss = sum_stride;
  a.tokens = (int)p->tokens;
  a.dim = p->dim;
  a.norm = p->norm;
  a.eps = p->eps;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool bf = p->dtype == QGEMM_DT_BF16;
  // As many threads as the row has groups of eight values (up to 1024, then two or four groups each): more values per
  // thread wait longer for the first (16 x 4096 to 16 bits: 512 threads 2.36 us, 256 with two groups 2.71; 16 x 8192: 1024
  // 2.94, 256 with four 3.56; 8192 x 8192: 91.9 and 98.1).  Rows up to 512 have one wavefront and no barrier.
  const bool wave = p->dim <= 512;
  const int chunks = wave || p->dim <= 8192 ? 1 : p->dim <= 16384 ? 2 : 4;
  const int threads = wave ? 256 : 64 * ((p->dim + 512 * chunks - 1) / (512 * chunks));
  const int row_threads = wave ? 64 : threads;
  if (p->tokens > 0xffffff00LL / row_threads)
    return fail(QGEMM_ERR_UNSUPPORTED, "%lld rows of %d threads are more than one launch allows", (long long)p->tokens, row_threads);
  if (wave) launch<true, 1>(bf, quantized, threads, s, a);
  else if (chunks == 1) launch<false, 1>(bf, quantized, threads, s, a);
  else if (chunks == 2) launch<false, 2>(bf, quantized, threads, s, a);
  else launch<false, 4>(bf, quantized, threads, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(QGEMM_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  return QGEMM_OK;
}
