// What both 8-bit product kernels do with finished fp32 sums (gfx950): the hand-off between workgroups that
// share an output, the gate, and the stores.
#pragma once

#include "qgemm_w8a8_device.h"

namespace qgemm {
namespace w8 {

// Partial sums go between workgroups of different XCDs with device-scope (sc1) stores and loads, which pass by
// the XCDs' own L2 caches; every thread waits for its stores before the barrier that precedes the ticket.
constexpr int kDeviceScope = 16;

__device__ __forceinline__ void store_partial(__amdgpu_buffer_rsrc_t part, int offset, f32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), part, offset, 0, kDeviceScope);
}
__device__ __forceinline__ f32x4 load_partial(__amdgpu_buffer_rsrc_t part, int offset) {
  return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(part, offset, 0, kDeviceScope));
}

// Called by every thread of a workgroup once its partial sums are stored; true in the workgroup that came last
// of `members`.  It leaves the ticket at zero for the next call.
__device__ __forceinline__ bool last_arrival(unsigned* ticket, int members, int* s_last) {
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (threadIdx.x == 0) {
    const unsigned t = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *s_last = t == (unsigned)(members - 1);
    if (*s_last) __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  return *s_last != 0;
}

// act(g) u.  exp2 and the reciprocal are the hardware's (1 ulp each); at large |x| the exponential's argument is
// rounded, which moves an output of e^-|x| by |x| 2^-24 of itself.  tanh(z) = 2 / (1 + exp(-2 z)) - 1 makes both
// gates g / (1 + exp(-p)).
template <int GATE>
__device__ __forceinline__ f32x4 gated(f32x4 g, f32x4 u) {
  if constexpr (GATE == QGEMM_GATE_NONE) return g;
  f32x4 y;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    constexpr float kLog2e = 1.44269504f;
    const float p = GATE == QGEMM_GATE_SILU ? -kLog2e * g[i]
                                            : -2.0f * 0.79788456f * kLog2e * g[i] * __builtin_fmaf(0.044715f, g[i] * g[i], 1.0f);
    y[i] = g[i] * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(p)) * u[i];
  }
  return y;
}

// Four consecutive outputs, each rounded once.
__device__ __forceinline__ void store4(const W8Args& a, size_t at, f32x4 v) {
  if (a.out_dtype == QGEMM_DT_F32) {
    *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at) = v;
  } else if (a.out_dtype == QGEMM_DT_F16) {
    const f16x2 lo = {(_Float16)v[0], (_Float16)v[1]}, hi = {(_Float16)v[2], (_Float16)v[3]};
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at) =
        u32x2{__builtin_bit_cast(unsigned, lo), __builtin_bit_cast(unsigned, hi)};
  } else {
    const bf16x2 lo = {(__bf16)v[0], (__bf16)v[1]}, hi = {(__bf16)v[2], (__bf16)v[3]};
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at) =
        u32x2{__builtin_bit_cast(unsigned, lo), __builtin_bit_cast(unsigned, hi)};
  }
}

}  // namespace w8
}  // namespace qgemm
