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

// Tile of workgroup b.  Workgroups go to the eight XCDs round-robin by number; each XCD takes a contiguous range of
// positions, which walk the tiles in bands of four token rows, so that the tiles an XCD runs at one time share
// tokens and weights in its L2.
__device__ __forceinline__ void tile_of(int b, int tiles, int tiles_n, int& tm, int& tn) {
  constexpr int kBand = 4;
  const int x = b & 7, slot = b >> 3, q = tiles >> 3, r = tiles & 7;
  const int at = x < r ? x * (q + 1) + slot : r * (q + 1) + (x - r) * q + slot;
  const int tiles_m = tiles / tiles_n;
  const int band = at / (kBand * tiles_n), first = band * kBand;
  const int rows = min(kBand, tiles_m - first);
  const int in = at - band * kBand * tiles_n;
  tm = first + in % rows;
  tn = in / rows;
}

// Workgroup barrier without the fence of __syncthreads(), which would wait for every load still in flight.
__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
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

// Four consecutive outputs rounded to 16 bits.
__device__ __forceinline__ u32x2 pack16(const W8Args& a, f32x4 v) {
  if (a.out_dtype == QGEMM_DT_F16) {
    const f16x2 lo = {(_Float16)v[0], (_Float16)v[1]}, hi = {(_Float16)v[2], (_Float16)v[3]};
    return u32x2{__builtin_bit_cast(unsigned, lo), __builtin_bit_cast(unsigned, hi)};
  }
  const bf16x2 lo = {(__bf16)v[0], (__bf16)v[1]}, hi = {(__bf16)v[2], (__bf16)v[3]};
  return u32x2{__builtin_bit_cast(unsigned, lo), __builtin_bit_cast(unsigned, hi)};
}

// Four consecutive outputs, each rounded once.
__device__ __forceinline__ void store4(const W8Args& a, size_t at, f32x4 v) {
  if (a.out_dtype == QGEMM_DT_F32) *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at) = v;
  else *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at) = pack16(a, v);
}

// A wavefront's outputs of 16 tokens on their way to memory: rows of RB bytes in LDS of its own, read back so that each store
// instruction writes whole runs of a row (stored from the MFMA's layout, 32 bytes of sixteen rows at a time, 8192 x 8192 bf16 outputs
// take 24 us).  Chunk c of 16 bytes of row r lies at c ^ r, so that neither side meets itself in the banks.
template <int RB>
struct OutRows {
  static constexpr int CH = RB / 16;
  unsigned char* lds;
  __device__ __forceinline__ unsigned char* at(int row, int byte) const {
    return lds + row * RB + 16 * ((byte >> 4) ^ (row & (CH - 1))) + (byte & 15);
  }
  // out: the first row's first byte; rows and chunks from `rows` and `chunks` on are not stored
  __device__ __forceinline__ void store(unsigned char* out, size_t stride, int rows, int chunks) const {
    asm volatile("" ::: "memory");                   // the wavefront's other lanes wrote what a lane reads here
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int r = 0; r < (16 * CH + 63) / 64; ++r) {
      const int e = 64 * r + lane, row = e / CH, c = e % CH;
      if (16 * CH < 64 && row >= 16) continue;
      const u32x4 v = *reinterpret_cast<const u32x4*>(at(row, 16 * c));
      if (row < rows && c < chunks) *reinterpret_cast<u32x4*>(out + row * stride + 16 * c) = v;
    }
    asm volatile("" ::: "memory");
  }
};

// The end of a workgroup's tile: lane l of a wavefront holds token m0 + 16 (i0 + i) + (l & 15) and weight rows
// 4 (l >> 4) .. + 3 of each block acc[t][i].  `top_lds`, `flag` and out_lds (8 KiB of the wavefront's own) are LDS that
// nothing else uses any more.
//
// Workgroups that share tile `group` of the split ones leave partial tiles in the workspace, and the one that comes last
// sums them in order.
template <int WN, int NW, int GATE, bool Q, bool F32, int TN, int TM>
__device__ __forceinline__ void finish_tile(const W8Args& a, f32x4 (&acc)[TN][TM], unsigned char* top_lds, unsigned char* flag,
                                            unsigned char* out_lds, int group, int splits, int split, int tn, int m0, int i0,
                                            int wn, int c0) {
  constexpr bool G = GATE != QGEMM_GATE_NONE;
  constexpr int BM = 16 * TM * NW / WN;
  const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
  if (splits > 1) {
    constexpr int SLOT = TN * TM * 64 * NW * 16;     // bytes of a partial tile: 16 per thread and block
    const __amdgpu_buffer_rsrc_t part = __builtin_amdgcn_make_buffer_rsrc(
        a.partials + (size_t)group * splits * (SLOT / 4), (short)0, splits * SLOT, 0x00020000);
    const int at = 16 * threadIdx.x;
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
      for (int i = 0; i < TM; ++i) store_partial(part, split * SLOT + (t * TM + i) * (64 * NW * 16) + at, acc[t][i]);
    if (!last_arrival(a.tickets + group, splits, reinterpret_cast<int*>(flag))) return;
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
      for (int i = 0; i < TM; ++i) acc[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < splits; ++s)
#pragma unroll
      for (int t = 0; t < TN; ++t)
#pragma unroll
        for (int i = 0; i < TM; ++i) acc[t][i] += load_partial(part, s * SLOT + (t * TM + i) * (64 * NW * 16) + at);
  }
  constexpr int OT = G ? TN / 2 : TN, ES = Q ? 1 : F32 ? 4 : 2;
  const OutRows<OT * 16 * ES> rows{out_lds};
  const size_t stride = (size_t)a.N * ES;
  const auto store = [&](int i) {
    const int m = m0 + 16 * (i0 + i);
    rows.store(static_cast<unsigned char*>(a.out) + (size_t)m * stride + (size_t)c0 * ES, stride, a.M - m, (a.N - c0) * ES / 16);
  };
  if constexpr (!Q) {
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int t = 0; t < OT; ++t) {
        const f32x4 v = gated<GATE>(acc[t][i], acc[t + TN - OT][i]);
        unsigned char* const to = rows.at(col, (16 * t + 4 * g) * ES);
        if constexpr (F32) *reinterpret_cast<f32x4*>(to) = v;
        else *reinterpret_cast<u32x2*>(to) = pack16(a, v);
      }
      store(i);
    }
  } else {
    auto& top = *reinterpret_cast<unsigned(*)[WN][BM]>(top_lds);   // largest magnitude of a token in each wavefront's columns
    unsigned m[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      m[i] = 0;
#pragma unroll
      for (int t = 0; t < OT; ++t) {
        acc[t][i] = gated<GATE>(acc[t][i], acc[t + OT][i]);
#pragma unroll
        for (int r = 0; r < 4; ++r) m[i] = max(m[i], magnitude(acc[t][i][r]));
      }
      m[i] = max(m[i], (unsigned)__shfl_xor((int)m[i], 16));
      m[i] = max(m[i], (unsigned)__shfl_xor((int)m[i], 32));
      if (g == 0) top[wn][16 * (i0 + i) + col] = m[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int w = 0; w < WN; ++w) m[i] = max(m[i], top[w][16 * (i0 + i) + col]);
      const BlockScale b = block_scale(m[i], 1.0f);
      const int token = m0 + 16 * (i0 + i) + col;
      if (token < a.M && wn == 0 && g == 0) a.os[(size_t)tn * a.M + token] = b.scale;
#pragma unroll
      for (int t = 0; t < OT; ++t) {
        const f32x4 v = acc[t][i];
        *reinterpret_cast<unsigned*>(rows.at(col, 16 * t + 4 * g)) =
            codes4(v[0] * b.to_code, v[1] * b.to_code, v[2] * b.to_code, v[3] * b.to_code);
      }
      store(i);
    }
  }
}

}  // namespace w8
}  // namespace qgemm
