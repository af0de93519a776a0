// qgemm_cache_write / qgemm_cache_read: the 4-bit paged key/value cache, in and out.
//
// Bound by memory: a 16-bit element in, half a byte and its share of two 16-bit parameters out (and
// the other way round).  A head row of D elements is spread over D / 8 lanes, eight consecutive dims
// (one 16-byte access and one dword of codes) each, so a wavefront holds 512 / D rows; they are
// consecutive tokens of one kv head, and the workgroup's four wavefronts continue them, because their K
// codes, V codes and parameters lie side by side when their slots do (heads side by side instead: read
// 16.3 us against 13.6).  A K dword goes out as it is; V's codes are transposed between the row's lanes
// in registers (through LDS, a nibble at a time: 18.8).  What cache_read writes is not read again by
// it: its stores are non-temporal (17.6 us against 23.8 with data past the caches).
//
// 16383 tokens of 8 heads of 128, fp16, groups of 32, in a captured graph: write 21.9 us, read 13.6 us,
// 5.0 TB/s in both; write 23.0 and read 15.8 us when nothing lies in the 256 MB cache.  Writing is at
// 330 vector instructions a wavefront, about as long as its memory traffic.
#include <hip/hip_runtime.h>

#include "qgemm_attention_internal.h"

namespace {

using namespace qgemm;

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

template <int N>
struct ic { static constexpr int value = N; };

struct CacheArgs {
  const uint16_t *k, *v;           // write: inputs
  uint16_t *ko, *vo;               // read: outputs
  uint8_t* data;
  const long long* slots;
  long long ks, vs;                // token strides in elements
  long long total_slots;
  double per_page;                 // 1 / page
  int tokens, kv_heads, page, codes, params, block;
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

// One row's place: its block, and the token's index in the page.
struct Place {
  uint8_t* block;
  int t;
  bool ok;
};
__device__ __forceinline__ Place place_of(const CacheArgs& a, int token, int head) {
  Place p{nullptr, 0, false};
  if (token >= a.tokens) return p;
  const long long slot = a.slots[token];
  if (slot < 0 || slot >= a.total_slots) return p;
  // slot / page by the reciprocal in fp64, at most one off, instead of a 64-bit division
  long long pg = (long long)((double)slot * a.per_page);
  p.t = (int)(slot - pg * a.page);
  if (p.t < 0) p.t += a.page, --pg;
  if (p.t >= a.page) p.t -= a.page, ++pg;
  p.block = a.data + ((size_t)pg * a.kv_heads + head) * a.block;
  p.ok = true;
  return p;
}

// Lane exchanges inside a row of 16 lanes by DPP: xor 1, xor 2, and the mirrored halves and row, which
// reduce like xor 4 and xor 8 once the quads are equal.
template <int C>
__device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), C, 0xf, 0xf, true));
}
template <int LANES, class F>
__device__ __forceinline__ float reduce(float x, F f) {
  x = f(x, dpp<0xB1>(x));
  x = f(x, dpp<0x4E>(x));
  if constexpr (LANES >= 8) x = f(x, dpp<0x141>(x));
  if constexpr (LANES >= 16) x = f(x, dpp<0x140>(x));
  if constexpr (LANES >= 32) x = f(x, __shfl_xor(x, 16));
  return x;
}

// Quantizes the lane's eight elements within groups of G / 8 lanes: the codes as one dword and the
// group's (scale, zero) as another.  The codes are those of the header's formula in fp32 with IEEE
// division, by Markstein's correction: with y the rounded reciprocal of s, q = d y is within two units
// of d / s in the last place, and q + (d - q s) y, the remainder being exact, is the rounded quotient.
// Three operations an element instead of a division's dozen.  Scales so small that y or the remainder
// leaves the normal range, or that fp16 holds them in fewer bits, divide and clamp.
template <bool BF, int G>
__device__ __forceinline__ void quantize8(u32x4 x, unsigned& codes, unsigned& par) {
  float f[8];
  u16x2 top = {0, 0};                                 // the largest magnitudes' bits: from the exponent's
#pragma unroll                                        // last value on there is an infinity or a NaN
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = from16<BF>(x[i] & 0xffffu);
    f[2 * i + 1] = from16<BF>(x[i] >> 16);
    top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, x[i] & 0x7fff7fffu));
  }
  float lo = f[0], hi = f[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = __builtin_fminf(lo, f[i]);
    hi = __builtin_fmaxf(hi, f[i]);
  }
  if (max(top[0], top[1]) >= (BF ? 0x7f80 : 0x7c00)) hi = __builtin_inff();      // fmin / fmax pass over a NaN
  lo = reduce<G / 8>(lo, [](float a, float b) { return __builtin_fminf(a, b); });
  hi = reduce<G / 8>(hi, [](float a, float b) { return __builtin_fmaxf(a, b); });
  const float span = hi - lo;
  const bool bad = !(span < __builtin_inff());
  // the quotient of 15 by the same correction, from the rounded reciprocal
  constexpr float kY15 = 1.0f / 15.0f;
  const float q15 = span * kY15;
  float s = from16<BF>(to16<BF>(__builtin_fmaf(__builtin_fmaf(-15.f, q15, span), kY15, q15)));
  // A scale of full precision is at most 2^-9 too small: no quotient reaches 15.5, where clamping begins.
  const bool tiny = s < (BF ? 0x1p-60f : 0x1p-14f);
  // A quotient plus 2^23 is 0x4B000000 + code, rounded to even; the constants add up in the
  // packed sum and are taken out at the end.
  constexpr unsigned kBias = 0x4B000000u * 0x11111111u;
  unsigned sum = 0;
  if (__builtin_expect(__any(tiny), 0)) {
    s = from16<BF>(to16<BF>(span / 15.0f));
#pragma unroll
    for (int i = 0; i < 8; ++i)
      sum += __builtin_bit_cast(unsigned, __builtin_amdgcn_fmed3f((f[i] - lo) / s, 0.f, 15.f) + 0x1p23f) << (4 * i);
  } else {
    // one step from the hardware's reciprocal (one unit in the last place) gives the rounded one of a number
    // of so few bits
    const float y0 = __builtin_amdgcn_rcpf(s), y = __builtin_fmaf(__builtin_fmaf(-s, y0, 1.f), y0, y0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = f[i] - lo, q = d * y;
      const float v = __builtin_fmaf(__builtin_fmaf(-q, s, d), y, q);
      sum += __builtin_bit_cast(unsigned, v + 0x1p23f) << (4 * i);
    }
  }
  const bool live = s > 0.f && !bad;
  codes = sum - kBias;                                // not live: nothing of it is used
  if (!live) codes = 0;
  par = bad ? (BF ? 0x7fc07fc0u : 0x7e007e00u) : to16<BF>(s) | to16<BF>(lo) << 16;
}

// V's codes between the lanes of a row.  Lane j has the codes of dims 8 j .. + 7, that is dims 16 i + r with
// i = j / 2 and r = 8 (j % 2) + e for its nibbles e; the layout wants r fixed and i along the nibbles.  So
// lanes of the same parity transpose an 8 x 8 matrix of nibbles (a 4 x 4 one of bytes where D = 64), one
// index bit at a time: the lane that differs in that bit of i hands over the half of its dword where the
// bits of i and e differ.  Each step is its own inverse and the steps commute, so the same call takes the
// stored order back.
template <int M>
__device__ __forceinline__ unsigned from_lane_xor(unsigned x) {
  auto mov = [](unsigned v, auto c) {
    return (unsigned)__builtin_amdgcn_mov_dpp((int)v, decltype(c)::value, 0xf, 0xf, true);
  };
  if constexpr (M == 2) return mov(x, ic<0x4E>{});                          // quad_perm 2 3 0 1
  else if constexpr (M == 4) return mov(mov(x, ic<0x1B>{}), ic<0x141>{});   // reversed quad, reversed eight: xor 3, xor 7
  else return mov(mov(x, ic<0x141>{}), ic<0x140>{});                        // reversed eight, reversed row: xor 7, xor 15
}
template <int D>
__device__ __forceinline__ unsigned transpose(unsigned x, int j) {
  const bool b0 = j & 2, b1 = j & 4, b2 = j & 8;
  // bytes 0..3 are this lane's, 4..7 the other's
  if constexpr (D == 64) {
    x = __builtin_amdgcn_perm(from_lane_xor<2>(x), x, b0 ? 0x03070105u : 0x06020400u);
    return __builtin_amdgcn_perm(from_lane_xor<4>(x), x, b1 ? 0x03020706u : 0x05040100u);
  }
  const unsigned p = from_lane_xor<2>(x), keep = b0 ? 0xf0f0f0f0u : 0x0f0f0f0fu;
  x = (x & keep) | (__builtin_amdgcn_alignbit(p, p, b0 ? 4 : 28) & ~keep);
  x = __builtin_amdgcn_perm(from_lane_xor<4>(x), x, b1 ? 0x03070105u : 0x06020400u);
  return __builtin_amdgcn_perm(from_lane_xor<8>(x), x, b2 ? 0x03020706u : 0x05040100u);
}

template <bool BF, int D, int NG>
__global__ __launch_bounds__(256) void cache_write(CacheArgs a) {
  constexpr int L = D / 8, R = 64 / L, U = D / 32, G = D / NG;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, j = lane % L;
  const int head = blockIdx.x % a.kv_heads;
  const int token = (blockIdx.x / a.kv_heads * 4 + wave) * R + lane / L;
  const Place p = place_of(a, token, head);
  u32x4 kx = {0, 0, 0, 0}, vx = {0, 0, 0, 0};
  if (p.ok) {
    kx = *reinterpret_cast<const u32x4*>(a.k + token * a.ks + head * D + 8 * j);
    vx = *reinterpret_cast<const u32x4*>(a.v + token * a.vs + head * D + 8 * j);
  }
  unsigned kc, kp, vc, vp;
  quantize8<BF, G>(kx, kc, kp);
  quantize8<BF, G>(vx, vc, vp);
  vc = transpose<D>(vc, j);
  if (!p.ok) return;
  *reinterpret_cast<unsigned*>(p.block + p.t * (D / 2) + 4 * (U * (j & 3) + (j >> 2))) = kc;
  uint8_t* vb = p.block + a.codes + (p.t >> 2) * (64 * U) + (p.t & 3) * U;
  const int i = j >> 1 & 7, e = 8 * (j & 1);
  if constexpr (D == 64) {
    // bytes: code of r = e + 2 i low, of the next r high
    unsigned even = vc & 0x0f0f0f0fu, next = vc >> 4 & 0x0f0f0f0fu;
    even = (even | even >> 4) & 0x00ff00ffu;
    next = (next | next >> 4) & 0x00ff00ffu;
    *reinterpret_cast<uint16_t*>(vb + (e + 2 * i) * (4 * U)) = (uint16_t)(even | even >> 8);
    *reinterpret_cast<uint16_t*>(vb + (e + 2 * i + 1) * (4 * U)) = (uint16_t)(next | next >> 8);
  } else {
    *reinterpret_cast<unsigned*>(vb + (e + i) * (4 * U) + (j >> 4) * 4) = vc;
  }
  if (j % (G / 8) == 0) {
    const int at = (j / (G / 8) * a.page + p.t) * 4;
    *reinterpret_cast<unsigned*>(p.block + 2 * a.codes + at) = kp;
    *reinterpret_cast<unsigned*>(p.block + 2 * a.codes + a.params + at) = vp;
  }
}

template <bool BF>
__device__ __forceinline__ u32x4 values8(unsigned codes, unsigned par) {
  const float s = from16<BF>(par & 0xffffu), z = from16<BF>(par >> 16);
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = to16<BF>(__builtin_fmaf((float)(codes >> (8 * i) & 15u), s, z)) |
           to16<BF>(__builtin_fmaf((float)(codes >> (8 * i + 4) & 15u), s, z)) << 16;
  return o;
}

template <bool BF, int D, int NG>
__global__ __launch_bounds__(256) void cache_read(CacheArgs a) {
  constexpr int L = D / 8, R = 64 / L, U = D / 32, G = D / NG;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, j = lane % L;
  const int head = blockIdx.x % a.kv_heads;
  const int token = (blockIdx.x / a.kv_heads * 4 + wave) * R + lane / L;
  const Place p = place_of(a, token, head);
  unsigned kc = 0, vc = 0, kp = 0, vp = 0;
  if (p.ok) {
    kc = *reinterpret_cast<const unsigned*>(p.block + p.t * (D / 2) + 4 * (U * (j & 3) + (j >> 2)));
    const int at = 2 * a.codes + (j / (G / 8) * a.page + p.t) * 4;
    kp = *reinterpret_cast<const unsigned*>(p.block + at);
    vp = *reinterpret_cast<const unsigned*>(p.block + at + a.params);
    const uint8_t* vb = p.block + a.codes + (p.t >> 2) * (64 * U) + (p.t & 3) * U;
    const int i = j >> 1 & 7, e = 8 * (j & 1);
    if constexpr (D == 64) {
      unsigned even = *reinterpret_cast<const uint16_t*>(vb + (e + 2 * i) * (4 * U));
      unsigned next = *reinterpret_cast<const uint16_t*>(vb + (e + 2 * i + 1) * (4 * U));
      even = (even | even << 8) & 0x00ff00ffu;
      next = (next | next << 8) & 0x00ff00ffu;
      vc = ((even | even << 4) & 0x0f0f0f0fu) | ((next | next << 4) & 0x0f0f0f0fu) << 4;
    } else {
      vc = *reinterpret_cast<const unsigned*>(vb + (e + i) * (4 * U) + (j >> 4) * 4);
    }
  }
  vc = transpose<D>(vc, j);
  if (token >= a.tokens) return;
  const size_t at = ((size_t)token * a.kv_heads + head) * D + 8 * j;
  __builtin_nontemporal_store(values8<BF>(kc, kp), reinterpret_cast<u32x4*>(a.ko + at));
  __builtin_nontemporal_store(values8<BF>(vc, vp), reinterpret_cast<u32x4*>(a.vo + at));
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

template <bool BF, int D, int NG>
void launch_one(bool write, dim3 grid, hipStream_t s, const CacheArgs& a) {
  if (write) cache_write<BF, D, NG><<<grid, dim3(256), 0, s>>>(a);
  else cache_read<BF, D, NG><<<grid, dim3(256), 0, s>>>(a);
}
template <bool BF>
void launch_type(int dim, int ng, bool write, dim3 grid, hipStream_t s, const CacheArgs& a) {
  if (dim == 64) ng == 1 ? launch_one<BF, 64, 1>(write, grid, s, a) : launch_one<BF, 64, 2>(write, grid, s, a);
  else if (dim == 128)
    ng == 1 ? launch_one<BF, 128, 1>(write, grid, s, a)
            : ng == 2 ? launch_one<BF, 128, 2>(write, grid, s, a) : launch_one<BF, 128, 4>(write, grid, s, a);
  else
    ng == 1 ? launch_one<BF, 256, 1>(write, grid, s, a)
            : ng == 2 ? launch_one<BF, 256, 2>(write, grid, s, a) : launch_one<BF, 256, 4>(write, grid, s, a);
}

qgemm_status_t enqueue(const qgemm_cache_t* c, bool write, CacheArgs& a, const int64_t* slots, int64_t tokens, void* stream) {
  const BlockGeom g = block_geom(c);
  a.slots = reinterpret_cast<const long long*>(slots);
  a.total_slots = c->num_pages * c->page_size;
  a.tokens = (int)tokens;
  a.kv_heads = c->kv_heads;
  a.page = c->page_size;
  a.per_page = 1.0 / c->page_size;
  a.codes = g.codes;
  a.params = g.params;
  a.block = g.bytes;
  const int rows = 512 / c->head_dim;
  const int64_t groups = (tokens + 4 * rows - 1) / (4 * rows) * c->kv_heads;
  if (!launchable(groups, 256))
    return fail(QGEMM_ERR_UNSUPPORTED, "tokens * kv_heads needs %lld workgroups, more than one launch allows", (long long)groups);
  const dim3 grid((unsigned)groups);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int ng = c->head_dim / c->group_size;
  if (c->dtype == QGEMM_DT_BF16) launch_type<true>(c->head_dim, ng, write, grid, s, a);
  else launch_type<false>(c->head_dim, ng, write, grid, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(QGEMM_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  return QGEMM_OK;
}

qgemm_status_t check_common(const qgemm_cache_t* c, const void* data, const int64_t* slots, int64_t tokens) {
  const qgemm_status_t st = validate_cache(c);
  if (st != QGEMM_OK) return st;
  if (tokens < 0 || tokens > (int64_t(1) << 24))
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "tokens must be in [0, 2^24], got %lld", (long long)tokens);
  if (tokens == 0) return QGEMM_OK;
  if (!data) return fail(QGEMM_ERR_INVALID_ARGUMENT, "data is NULL");
  if (!slots) return fail(QGEMM_ERR_INVALID_ARGUMENT, "slots is NULL");
  if (!aligned(data, 16)) return fail(QGEMM_ERR_MISALIGNED, "data must be 16-byte aligned");
  if (!aligned(slots, 8)) return fail(QGEMM_ERR_MISALIGNED, "slots must be 8-byte aligned");
  return QGEMM_OK;
}

}  // namespace

extern "C" qgemm_status_t qgemm_cache_write(const qgemm_cache_t* c, void* data, const void* k, int64_t k_stride,
                                            const void* v, int64_t v_stride, const int64_t* slots, int64_t tokens,
                                            void* stream) {
  clear_error();
  const qgemm_status_t st = check_common(c, data, slots, tokens);
  if (st != QGEMM_OK || tokens == 0) return st;
  if (!k || !v) return fail(QGEMM_ERR_INVALID_ARGUMENT, "k or v is NULL");
  if (!aligned(k, 16) || !aligned(v, 16)) return fail(QGEMM_ERR_MISALIGNED, "k and v must be 16-byte aligned");
  const int64_t row = (int64_t)c->kv_heads * c->head_dim;
  for (int64_t s : {k_stride, v_stride})
    if (s < row || s % 8 || s > (int64_t(1) << 31))
      return fail(QGEMM_ERR_INVALID_ARGUMENT, "token strides must be multiples of 8 in [%lld, 2^31], got %lld",
                  (long long)row, (long long)s);
  CacheArgs a{};
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.ks = k_stride;
  a.vs = v_stride;
  a.data = static_cast<uint8_t*>(data);
  return enqueue(c, true, a, slots, tokens, stream);
}

extern "C" qgemm_status_t qgemm_cache_read(const qgemm_cache_t* c, const void* data, const int64_t* slots, int64_t tokens,
                                           void* k_out, void* v_out, void* stream) {
  clear_error();
  const qgemm_status_t st = check_common(c, data, slots, tokens);
  if (st != QGEMM_OK || tokens == 0) return st;
  if (!k_out || !v_out) return fail(QGEMM_ERR_INVALID_ARGUMENT, "k_out or v_out is NULL");
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return fail(QGEMM_ERR_MISALIGNED, "k_out and v_out must be 16-byte aligned");
  CacheArgs a{};
  a.ko = static_cast<uint16_t*>(k_out);
  a.vo = static_cast<uint16_t*>(v_out);
  a.data = const_cast<uint8_t*>(static_cast<const uint8_t*>(data));
  return enqueue(c, false, a, slots, tokens, stream);
}
