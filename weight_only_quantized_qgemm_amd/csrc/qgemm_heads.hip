// qgemm_qk_norm_rope: RMS norm of every query and key head and its rotation, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w,   (y_a, y_b) <- (y_a c - y_b s, y_b c + y_a s)
//
// Bound by memory: 4 bytes per element in and out, about ten operations.  A head is spread over
// D / 8 lanes, eight dims each, laid out so that both dims of every rotated pair sit in one lane:
// with half-split pairs lane j holds dims 4 j .. + 3 and rot / 2 + 4 j .. + 3, with adjacent pairs
// dims 8 j .. + 7, so the rotation needs no exchange between lanes and the sum of squares is the
// only reduction (log2(D / 8) steps).  A wavefront stays on one token, so the token's row of the
// table is loaded once and serves all of the wavefront's heads.  The outputs are stored non-temporally:
// the next reader comes a whole pass later (two runs of heads a wavefront, 8192 tokens of 48 heads:
// 45.9 -> 42.0 us with data past the caches, 38.8 -> 38.2 with data in them).
//
// 8192 tokens of 48 heads of 128, bf16: 38.0 us in a captured graph, 5.35 TB/s; 41.8 us, 4.86 TB/s, when
// nothing lies in the 256 MB cache.  16 tokens of 40 heads: 4 us, a launch.
#include <hip/hip_runtime.h>

#include "qgemm_attention_internal.h"

namespace {

using namespace qgemm;

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct RopeArgs {
  const uint16_t *q, *k, *qw, *kw;
  uint16_t *qo, *ko;
  const int* pos;
  const float* table;
  long long qs, ks, qos, kos;      // token strides in elements
  int q_heads, heads, rot, max_pos, norm;
  int chunks;                      // wavefronts per token
  int tokens;
  float eps;
};

template <bool BF>
__device__ __forceinline__ float from16(unsigned bits) {
  if constexpr (BF) return __builtin_bit_cast(float, bits << 16);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}
template <bool BF>
__device__ __forceinline__ unsigned to16(float v) {
  if constexpr (BF) return __builtin_bit_cast(uint16_t, (__bf16)v);
  else return __builtin_bit_cast(uint16_t, (_Float16)v);
}
template <bool BF>
__device__ __forceinline__ void unpack4(u32x2 v, float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[2 * i] = from16<BF>(v[i] & 0xffffu);
    f[2 * i + 1] = from16<BF>(v[i] >> 16);
  }
}
template <bool BF>
__device__ __forceinline__ u32x2 pack4(const float* f) {
  return u32x2{to16<BF>(f[0]) | to16<BF>(f[1]) << 16, to16<BF>(f[2]) | to16<BF>(f[3]) << 16};
}

template <bool BF, int D, bool IL, int C>
__global__ __launch_bounds__(256) void norm_rope(RopeArgs a) {
  constexpr int L = D / 8, H = 64 / L;               // lanes per head, heads per wavefront
  const int wave = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int token = wave / a.chunks, chunk = wave - token * a.chunks;
  if (token >= a.tokens) return;
  const int j = lane % L;
  // the lane's two runs of four dims; L lanes turn together in the first rot / 8
  const bool turned = 8 * j < a.rot;
  const int d0 = !IL && turned ? 4 * j : 8 * j;
  const int d1 = !IL && turned ? a.rot / 2 + 4 * j : d0 + 4;
  float c[4], s[4];
  if (turned) {
    int p = a.pos[token];
    p = p < 0 ? 0 : p >= a.max_pos ? a.max_pos - 1 : p;
    const float* row = a.table + (size_t)p * a.rot + 4 * j;
    const f32x4 cv = *reinterpret_cast<const f32x4*>(row);
    const f32x4 sv = *reinterpret_cast<const f32x4*>(row + a.rot / 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) { c[i] = cv[i]; s[i] = sv[i]; }
  }
  // heads h, h + chunks * H, ...: loaded at once, then each on its own
  u32x2 in[C][2];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int h = (c * a.chunks + chunk) * H + lane / L;
    if (h >= a.heads) break;
    const uint16_t* x = h >= a.q_heads ? a.k + token * a.ks + (h - a.q_heads) * D : a.q + token * a.qs + h * D;
    in[c][0] = *reinterpret_cast<const u32x2*>(x + d0);
    in[c][1] = *reinterpret_cast<const u32x2*>(x + d1);
  }
#pragma unroll
  for (int n = 0; n < C; ++n) {
    const int h = (n * a.chunks + chunk) * H + lane / L;
    if (h >= a.heads) break;
    const bool isk = h >= a.q_heads;
    uint16_t* o = isk ? a.ko + token * a.kos + (h - a.q_heads) * D : a.qo + token * a.qos + h * D;
    const uint16_t* w = isk ? a.kw : a.qw;
    float y[8];
    unpack4<BF>(in[n][0], y);
    unpack4<BF>(in[n][1], y + 4);
    if (a.norm) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(y[i], y[i], sum);
#pragma unroll
      for (int m = 1; m < L; m *= 2) sum += __shfl_xor(sum, m);
      const float r = 1.0f / __builtin_sqrtf(sum * (1.0f / D) + a.eps);
      float wv[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
      if (w) {
        unpack4<BF>(*reinterpret_cast<const u32x2*>(w + d0), wv);
        unpack4<BF>(*reinterpret_cast<const u32x2*>(w + d1), wv + 4);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = y[i] * r * wv[i];
    }
    if (turned) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        constexpr int kStep = IL ? 2 : 1, kMate = IL ? 1 : 4;
        const float u = y[kStep * i], v = y[kStep * i + kMate];
        y[kStep * i] = u * c[i] - v * s[i];
        y[kStep * i + kMate] = v * c[i] + u * s[i];
      }
    }
    __builtin_nontemporal_store(pack4<BF>(y), reinterpret_cast<u32x2*>(o + d0));
    __builtin_nontemporal_store(pack4<BF>(y + 4), reinterpret_cast<u32x2*>(o + d1));
  }
}

template <int D, int C>
void launch(bool bf, bool interleaved, dim3 grid, hipStream_t s, const RopeArgs& a) {
  const dim3 block(256);
  if (bf) {
    interleaved ? norm_rope<true, D, true, C><<<grid, block, 0, s>>>(a) : norm_rope<true, D, false, C><<<grid, block, 0, s>>>(a);
  } else {
    interleaved ? norm_rope<false, D, true, C><<<grid, block, 0, s>>>(a) : norm_rope<false, D, false, C><<<grid, block, 0, s>>>(a);
  }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

qgemm_status_t check_rows(const char* name, const void* in, int64_t stride, const void* out, int64_t out_stride, int heads,
                          int dim) {
  const long long row = (long long)heads * dim;
  if (!in || !out) return fail(QGEMM_ERR_INVALID_ARGUMENT, "%s or %s_out is NULL (%d heads)", name, name, heads);
  if (!aligned(in, 16) || !aligned(out, 16))
    return fail(QGEMM_ERR_MISALIGNED, "%s and %s_out must be 16-byte aligned", name, name);
  for (int64_t st : {stride, out_stride})
    if (st < row || st % 8 || st > (int64_t(1) << 31))
      return fail(QGEMM_ERR_INVALID_ARGUMENT, "%s token strides must be multiples of 8 in [%lld, 2^31], got %lld", name, row,
                  (long long)st);
  if (in == out && stride != out_stride)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "%s_out in place needs %s's own stride %lld, got %lld", name, name,
                (long long)stride, (long long)out_stride);
  return QGEMM_OK;
}

}  // namespace

extern "C" qgemm_status_t qgemm_qk_norm_rope(const qgemm_norm_rope_t* p, const void* q, int64_t q_stride, const void* k,
                                             int64_t k_stride, const void* q_weight, const void* k_weight,
                                             const int32_t* positions, const float* cos_sin, void* q_out,
                                             int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream) {
  clear_error();
  qgemm_status_t st = validate_norm_rope(p);
  if (st != QGEMM_OK) return st;
  if (p->tokens == 0) return QGEMM_OK;
  if (p->q_heads && (st = check_rows("q", q, q_stride, q_out, q_out_stride, p->q_heads, p->head_dim)) != QGEMM_OK) return st;
  if (p->kv_heads && (st = check_rows("k", k, k_stride, k_out, k_out_stride, p->kv_heads, p->head_dim)) != QGEMM_OK) return st;
  if (p->rot_dim) {
    if (!positions || !cos_sin) return fail(QGEMM_ERR_INVALID_ARGUMENT, "positions or cos_sin is NULL (rot_dim %d)", p->rot_dim);
    if (!aligned(positions, 4)) return fail(QGEMM_ERR_MISALIGNED, "positions must be 4-byte aligned");
    if (!aligned(cos_sin, 16)) return fail(QGEMM_ERR_MISALIGNED, "cos_sin must be 16-byte aligned");
  }
  if (p->norm && ((q_weight && !aligned(q_weight, 16)) || (k_weight && !aligned(k_weight, 16))))
    return fail(QGEMM_ERR_MISALIGNED, "q_weight and k_weight must be 16-byte aligned");
  RopeArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.qw = static_cast<const uint16_t*>(q_weight);
  a.kw = static_cast<const uint16_t*>(k_weight);
  a.qo = static_cast<uint16_t*>(q_out);
  a.ko = static_cast<uint16_t*>(k_out);
  a.pos = positions;
  a.table = cos_sin;
  a.qs = q_stride; a.ks = k_stride; a.qos = q_out_stride; a.kos = k_out_stride;
  a.q_heads = p->q_heads;
  a.heads = p->q_heads + p->kv_heads;
  a.rot = p->rot_dim;
  a.max_pos = p->max_pos;
  a.norm = p->norm;
  a.tokens = (int)p->tokens;
  a.eps = p->eps;
  const int per_wave = 512 / p->head_dim;
  const int runs = (a.heads + per_wave - 1) / per_wave;         // runs of heads that a wavefront holds at once
  // Two runs a wavefront, both loaded before the first is reduced, once every SIMD has several wavefronts
  // (8192 tokens of 48 heads, data past the caches: 50.5 us with one, 42.0 with two); below that the launch is its longest
  // wavefront (one token: 3.3 us against 3.8).
  const bool two = p->tokens * runs > 4096;
  a.chunks = two ? (runs + 1) / 2 : runs;
  const int64_t waves = p->tokens * a.chunks;
  if (!launchable((waves + 3) / 4, 256))
    return fail(QGEMM_ERR_UNSUPPORTED, "tokens * heads needs %lld wavefronts, more than one launch allows", (long long)waves);
  const dim3 grid((unsigned)((waves + 3) / 4));
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool bf = p->dtype == QGEMM_DT_BF16;
  switch (p->head_dim) {
    case 64: two ? launch<64, 2>(bf, p->interleaved, grid, s, a) : launch<64, 1>(bf, p->interleaved, grid, s, a); break;
    case 128: two ? launch<128, 2>(bf, p->interleaved, grid, s, a) : launch<128, 1>(bf, p->interleaved, grid, s, a); break;
    default: two ? launch<256, 2>(bf, p->interleaved, grid, s, a) : launch<256, 1>(bf, p->interleaved, grid, s, a); break;
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(QGEMM_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  return QGEMM_OK;
}
