// What both 8-bit product kernels do with finished fp32 sums (gfx950): the hand-off between workgroups that
// share an output, the gate, and the stores.
#pragma once

#include <type_traits>

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
template <int WN, int NW, int GATE, bool Q, bool F32, int TN, int TM>
struct TileEnd {
  static constexpr bool G = GATE != QGEMM_GATE_NONE;
  static constexpr int BM = 16 * TM * NW / WN, OT = G ? TN / 2 : TN, ES = Q ? 1 : F32 ? 4 : 2;
  const W8Args& a;
  unsigned char *top_lds, *flag, *out_lds;
  int tn, m0, i0, wn, c0;

  // Blocks O of the outputs of token block i, from column block o on.
  template <int O>
  __device__ __forceinline__ OutRows<O * 16 * ES> rows() const { return OutRows<O * 16 * ES>{out_lds}; }
  template <int O>
  __device__ __forceinline__ void leave(int i, int o) const {
    const int m = m0 + 16 * (i0 + i), c = c0 + 16 * o;
    const size_t stride = (size_t)a.N * ES;
    rows<O>().store(static_cast<unsigned char*>(a.out) + (size_t)m * stride + (size_t)c * ES, stride, a.M - m, (a.N - c) * ES / 16);
  }
  template <int O>
  __device__ __forceinline__ void put(int t, f32x4 v) const {
    const int lane = threadIdx.x & 63;
    unsigned char* const to = rows<O>().at(lane & 15, (16 * t + 4 * (lane >> 4)) * ES);
    if constexpr (F32) *reinterpret_cast<f32x4*>(to) = v;
    else *reinterpret_cast<u32x2*>(to) = pack16(a, v);
  }
  // e4m3: the largest magnitude of a token in each wavefront's columns
  __device__ __forceinline__ unsigned& top(int w, int i) const {
    return reinterpret_cast<unsigned*>(top_lds)[w * BM + 16 * (i0 + i) + (threadIdx.x & 15)];
  }
  __device__ __forceinline__ void note(int i, const f32x4 (&y)[OT]) const {
    unsigned m = 0;
#pragma unroll
    for (int t = 0; t < OT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) m = max(m, magnitude(y[t][r]));
    m = max(m, (unsigned)__shfl_xor((int)m, 16));
    m = max(m, (unsigned)__shfl_xor((int)m, 32));
    if ((threadIdx.x & 48) == 0) top(wn, i) = m;
  }
  __device__ __forceinline__ void code(int i, const f32x4 (&y)[OT]) const {
    const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15, token = m0 + 16 * (i0 + i) + col;
    unsigned m = 0;
#pragma unroll
    for (int w = 0; w < WN; ++w) m = max(m, top(w, i));
    const BlockScale b = block_scale(m, 1.0f);
    if (token < a.M && wn == 0 && g == 0) a.os[(size_t)tn * a.M + token] = b.scale;
#pragma unroll
    for (int t = 0; t < OT; ++t)
      *reinterpret_cast<unsigned*>(rows<OT>().at(col, 16 * t + 4 * g)) =
          codes4(y[t][0] * b.to_code, y[t][1] * b.to_code, y[t][2] * b.to_code, y[t][3] * b.to_code);
    leave<OT>(i, 0);
  }

  __device__ __forceinline__ void whole(f32x4 (&acc)[TN][TM]) const {
    f32x4 y[TM][OT];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int t = 0; t < OT; ++t) y[i][t] = gated<GATE>(acc[t][i], acc[t + TN - OT][i]);
      if constexpr (Q) {
        note(i, y[i]);
      } else {
#pragma unroll
        for (int t = 0; t < OT; ++t) put<OT>(t, y[i][t]);
        leave<OT>(i, 0);
      }
    }
    if constexpr (Q) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < TM; ++i) code(i, y[i]);
    }
  }

  // Workgroups that share tile `group` of the split ones leave partial tiles in the workspace, in the order of the wavefronts' blocks.
  static constexpr int BLOCK = 64 * NW * 16, SLOT = TN * TM * BLOCK;      // bytes of a block of every wavefront, of a partial tile
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t partials(int group, int splits) const {
    return __builtin_amdgcn_make_buffer_rsrc(a.partials + (size_t)group * splits * (SLOT / 4), (short)0, splits * SLOT, 0x00020000);
  }

  // The one that comes last sums them in order.
  __device__ __forceinline__ void shared_at_once(f32x4 (&acc)[TN][TM], int group, int splits, int split) const {
    const __amdgpu_buffer_rsrc_t part = partials(group, splits);
    const int at = 16 * threadIdx.x;
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
      for (int i = 0; i < TM; ++i) store_partial(part, split * SLOT + (t * TM + i) * BLOCK + at, acc[t][i]);
    if (!last_arrival(a.tickets + (size_t)group * kTileParts, splits, reinterpret_cast<int*>(flag))) return;
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
      for (int i = 0; i < TM; ++i) acc[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < splits; ++s)
#pragma unroll
      for (int t = 0; t < TN; ++t)
#pragma unroll
        for (int i = 0; i < TM; ++i) acc[t][i] += load_partial(part, s * SLOT + (t * TM + i) * BLOCK + at);
    whole(acc);
  }

  // The same part by part (a token block of every wavefront, or half of its columns), with a ticket for each part, and each
  // workgroup starting with another part; whoever comes last to a part sums it in order.  So the parts have different last
  // ones and none reads all partial tiles (300 x 4096 x 4096 by two, 128 tokens: 20.8 us, with one last workgroup 22.0, by four
  // 18.4 and 20.4; 128 x 1024 x 28672, 64 tokens: 21.4 and 25.5.  64 tokens by two or three are too little for four tickets:
  // 300 x 4096 x 4096 by three 18.6 and 16.9).
  __device__ __forceinline__ void shared_in_parts(f32x4 (&acc)[TN][TM], int group, int splits, int split) const {
    constexpr int H = TM == 2 && !Q ? 2 : 1, PARTS = TM * H, PT = TN / H, PO = OT / H;
    static_assert((PARTS == 2 || PARTS == 4) && PARTS <= kTileParts && PARTS * PT <= 63, "tickets of a tile; vmcnt counts at most 63");
    const __amdgpu_buffer_rsrc_t part = partials(group, splits);
    const int at = 16 * threadIdx.x, first = split * PARTS / splits;
    const auto part_at = [&](int x) { return (first + x) % PARTS; };
    const auto hand_over = [&](int which, auto part_q) {
      constexpr int q = decltype(part_q)::value;
      if (which != q) return;
#pragma unroll
      for (int b = 0; b < PT; ++b)
        store_partial(part, split * SLOT + (q * PT + b) * BLOCK + at, acc[b < PO ? q % H * PO + b : OT + q % H * PO + b - PO][q / H]);
      asm volatile("; part %0" ::"i"(q));            // or the compiler makes one store of the four and keeps acc in memory to index it
    };
#pragma unroll
    for (int x = 0; x < PARTS; ++x) {
      hand_over(part_at(x), std::integral_constant<int, 0>{});
      hand_over(part_at(x), std::integral_constant<int, 1>{});
      if constexpr (PARTS > 2) {
        hand_over(part_at(x), std::integral_constant<int, 2>{});
        hand_over(part_at(x), std::integral_constant<int, 3>{});
      }
    }
    unsigned* const tickets = a.tickets + (size_t)group * kTileParts;
    int* const last = reinterpret_cast<int*>(flag);
    unsigned ticket[PARTS];
    const auto arrive = [&](auto at) {
      constexpr int x = decltype(at)::value, pending = (PARTS - 1 - x) * PT;      // stores complete in order
      __builtin_amdgcn_s_waitcnt((pending & 15) | (7 << 4) | (15 << 8) | ((pending >> 4) << 14));
      barrier();
      if (threadIdx.x == 0)
        ticket[x] = __hip_atomic_fetch_add(tickets + part_at(x), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    };
    arrive(std::integral_constant<int, 0>{});
    arrive(std::integral_constant<int, 1>{});
    if constexpr (PARTS > 2) {
      arrive(std::integral_constant<int, 2>{});
      arrive(std::integral_constant<int, 3>{});
    }
    if (threadIdx.x == 0) {
#pragma unroll
      for (int x = 0; x < PARTS; ++x) {
        last[x] = ticket[x] == (unsigned)(splits - 1);
        if (last[x]) __hip_atomic_store(tickets + part_at(x), 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    __syncthreads();
    for (int x = 0; x < PARTS; ++x) {
      if (!last[x]) continue;
      const int q = part_at(x), i = q / H;
      f32x4 v[PT];
#pragma unroll
      for (int b = 0; b < PT; ++b) v[b] = f32x4{0.f, 0.f, 0.f, 0.f};
      int from = 0;
      const auto add = [&](auto ahead) {             // partial tiles whose loads are on their way together
        constexpr int AHEAD = decltype(ahead)::value;
        f32x4 p[AHEAD][PT];
#pragma unroll
        for (int s = 0; s < AHEAD; ++s)
#pragma unroll
          for (int b = 0; b < PT; ++b) p[s][b] = load_partial(part, (from + s) * SLOT + (q * PT + b) * BLOCK + at);
#pragma unroll
        for (int s = 0; s < AHEAD; ++s)
#pragma unroll
          for (int b = 0; b < PT; ++b) v[b] += p[s][b];
        from += AHEAD;
      };
      if constexpr (PT < 8)                          // of eight blocks there are registers for two
        while (from + 4 <= splits) add(std::integral_constant<int, 4>{});
      while (from + 2 <= splits) add(std::integral_constant<int, 2>{});
      if (from < splits) add(std::integral_constant<int, 1>{});
      f32x4 y[PO];
#pragma unroll
      for (int t = 0; t < PO; ++t) y[t] = gated<GATE>(v[t], v[t + PT - PO]);
      if constexpr (Q) {
        note(i, y);
        __syncthreads();
        code(i, y);
      } else {
#pragma unroll
        for (int t = 0; t < PO; ++t) put<PO>(t, y[t]);
        leave<PO>(i, q % H * PO);
      }
    }
  }
};

}  // namespace w8
}  // namespace qgemm
