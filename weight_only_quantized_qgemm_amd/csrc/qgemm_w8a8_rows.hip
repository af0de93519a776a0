// The rows kernel of the 8-bit products: up to 16 tokens, the weights streamed once.
//
//   p_r[m] = sum_b as[b][m] ws[r / 128][b] (sum_{k in block b} a[m][k] w[r][k])
//
// A workgroup owns one 16-row weight block (with a gate that of both projections); its wavefronts take the k
// blocks of 128 in turn, so that together they read 1 KiB of every weight row side by side.  The weights go
// from memory straight into registers, as fp16 into the first operand of v_mfma_f32_16x16x32_f16 and the tokens'
// codes into the second: lane l holds row (token) l & 15 and the 16-byte chunks l >> 4 and 4 + (l >> 4) of the k block,
// the same for both, which is all that a dot product asks of its order.  The result has token l & 15 and weight rows
// 4 (l >> 4) .. + 3 in lane l, so both scales are one factor per lane, applied to the fp32 block sum.
//
// Bound by the weights' way from memory: 4096 x 11008, one token 10.3 us, 4.4 TB/s, 16 tokens 13.1 us; 11008 x 4096 gated
// to 16 bits 17.8 and 19.7 us (5.1 and 4.6 TB/s).  Bringing the tokens into LDS first, for fewer load instructions, delays
// the first product by more than it saves (4096 x 4096, one token: 5.7 us against 5.2).
//
// The wavefronts' sums meet in LDS, in wavefront order.  Where several workgroups make one output (splits along
// K; the eight column blocks of an output scale block) each leaves its fp32 sums in the workspace and takes a
// ticket, and the one that draws the last ticket adds them in order and finishes: no workgroup waits for another.
#include <type_traits>

#include "qgemm_w8a8_fixup.h"

namespace qgemm {
namespace w8 {
namespace {

template <int NW, int GATE, bool Q>
__global__ __launch_bounds__(64 * NW, 4) void rows_kernel(W8Args a) {
  constexpr bool G = GATE != QGEMM_GATE_NONE;
  constexpr int U = G ? 2 : 1;                       // weight blocks: one of either projection
  constexpr int F = Q ? kBlock / 16 : 1;             // workgroups along the columns of one output scale block
  __shared__ f32x4 sums[NW / 2][U][64];
  __shared__ int s_last;
  const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // workgroup = (group, column block in it, split)
  const int members = F * a.splits;
  const int member = blockIdx.x % members, group = blockIdx.x / members;
  const int cb = member / a.splits, split = member - cb * a.splits;
  const int n0 = (group * F + cb) * 16;              // first output column
  const int kb0 = split * a.kb_per_split, kb1 = min(a.KB, kb0 + a.kb_per_split);
  const int token = min(col, a.M - 1);               // tokens past the last repeat it and are not stored

  // (addresses: a uniform base and a 32-bit offset per lane; 16 rows of K <= 2^22 stay below 2^26)
  const uint8_t* wp[U];
  const float* sp[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    wp[u] = a.w + ((size_t)u * a.N + n0) * a.K;
    sp[u] = a.ws + ((size_t)u * a.row_blocks + n0 / kBlock) * a.KB;
  }
  const unsigned woff = col * a.K + 16 * g, aoff = token * a.K + 16 * g;
  f32x4 acc[U];
#pragma unroll
  for (int u = 0; u < U; ++u) acc[u] = f32x4{0.f, 0.f, 0.f, 0.f};

  // two k blocks in flight per wavefront (four leave registers for half as many workgroups: gated 16 x 11008 x 4096 21.9 us
  // against 19.7)
  constexpr int D = 2;
  struct Chunks { i32x4 v[2]; };
  Chunks w[D][U], x[D];
  float sw[D][U], sa[D];
  bool in[D];                                        // whether the block in set d is one of this wavefront's
  const auto chunks = [](const uint8_t* p, unsigned off) {
    return Chunks{{*reinterpret_cast<const i32x4*>(p + off), *reinterpret_cast<const i32x4*>(p + 64 + off)}};
  };
  const auto load = [&](int d, int at) {
    in[d] = at < kb1;
    const int kb = min(at, kb1 - 1);
#pragma unroll
    for (int u = 0; u < U; ++u) w[d][u] = chunks(wp[u] + (size_t)kb * kBlock, woff);
#pragma unroll
    for (int u = 0; u < U; ++u) sw[d][u] = sp[u][kb];
    x[d] = chunks(a.a + (size_t)kb * kBlock, aoff);
    sa[d] = (a.as + (size_t)kb * a.M)[token];
  };
  const auto compute = [&](int d) {
    const Halves x0 = halves(x[d].v[0]), x1 = halves(x[d].v[1]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Halves w0 = halves(w[d][u].v[0]), w1 = halves(w[d][u].v[1]);
      f32x4 p = __builtin_amdgcn_mfma_f32_16x16x32_f16(w0.v[0], x0.v[0], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
      p = __builtin_amdgcn_mfma_f32_16x16x32_f16(w0.v[1], x0.v[1], p, 0, 0, 0);
      p = __builtin_amdgcn_mfma_f32_16x16x32_f16(w1.v[0], x1.v[0], p, 0, 0, 0);
      p = __builtin_amdgcn_mfma_f32_16x16x32_f16(w1.v[1], x1.v[1], p, 0, 0, 0);
      const float s = in[d] ? sa[d] * sw[d][u] : 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[u][r] = __builtin_fmaf(p[r], s, acc[u][r]);
    }
  };
  // The last round is as long as the others: blocks past the end are the last one again, with factor 0 (branches
  // around them would copy the sums from register to register).
  int kb = kb0 + wave;
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, kb + d * NW);
  for (; kb + D * NW < kb1; kb += D * NW) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      compute(d);
      load(d, kb + (D + d) * NW);
    }
  }
#pragma unroll
  for (int d = 0; d < D; ++d) compute(d);

  // the wavefronts' sums: the second half into the first, then those in order
  if (wave >= NW / 2) {
#pragma unroll
    for (int u = 0; u < U; ++u) sums[wave - NW / 2][u][lane] = acc[u];
  }
  __syncthreads();
  if (wave < NW / 2) {
#pragma unroll
    for (int u = 0; u < U; ++u) sums[wave][u][lane] += acc[u];
  }
  __syncthreads();
  const __amdgpu_buffer_rsrc_t part =
      __builtin_amdgcn_make_buffer_rsrc(a.partials + (size_t)group * members * (U * 256), (short)0, members * (U * 1024), 0x00020000);
  const auto slot = [&](int m, int u) { return (m * U + u) * 1024 + 16 * lane; };
  const auto joined = [&](int u) {
    f32x4 v = sums[0][u][lane];
#pragma unroll
    for (int w = 1; w < NW / 2; ++w) v += sums[w][u][lane];
    return v;
  };
  if (members > 1) {
    if (wave < U) store_partial(part, slot(member, wave), joined(wave));
    if (!last_arrival(a.tickets + group, members, &s_last)) return;
  }
  if constexpr (!Q) {
    if (wave > 0) return;
    f32x4 v[2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (members > 1) {
        v[u] = load_partial(part, slot(0, u));
        for (int s = 1; s < a.splits; ++s) v[u] += load_partial(part, slot(s, u));
      } else {
        v[u] = joined(u);
      }
    }
    if (col < a.M) store4(a, (size_t)col * a.N + n0 + 4 * g, gated<GATE>(v[0], v[U - 1]));
  } else {
    // every column block's outputs and largest magnitudes, then the codes
    constexpr int PER = kBlock / 16 / NW > 0 ? kBlock / 16 / NW : 1;     // column blocks of a wavefront
    __shared__ unsigned top[kBlock / 16][16];
    f32x4 y[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int c = wave * PER + j;
      f32x4 v[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
      for (int s = 0; s < a.splits; ++s)
#pragma unroll
        for (int u = 0; u < 2; ++u) v[u] += load_partial(part, slot(c * a.splits + s, u));
      y[j] = gated<GATE>(v[0], v[1]);
      unsigned m = max(max(magnitude(y[j][0]), magnitude(y[j][1])), max(magnitude(y[j][2]), magnitude(y[j][3])));
      m = max(m, (unsigned)__shfl_xor((int)m, 16));
      m = max(m, (unsigned)__shfl_xor((int)m, 32));
      if (g == 0) top[c][col] = m;
    }
    __syncthreads();
    unsigned m = 0;
#pragma unroll
    for (int c = 0; c < kBlock / 16; ++c) m = max(m, top[c][col]);
    const BlockScale b = block_scale(m, 1.0f);
    if (col >= a.M) return;
#pragma unroll
    for (int j = 0; j < PER; ++j)
      *reinterpret_cast<unsigned*>(static_cast<uint8_t*>(a.out) + (size_t)col * a.N + group * kBlock + 16 * (wave * PER + j) + 4 * g) =
          codes4(y[j][0] * b.to_code, y[j][1] * b.to_code, y[j][2] * b.to_code, y[j][3] * b.to_code);
    if (wave == 0 && g == 0) a.os[(size_t)group * a.M + col] = b.scale;
  }
}

template <int NW>
void launch_waves(const W8Plan& pl, const W8Args& a, hipStream_t s) {
  const dim3 grid(pl.grid), block(64 * NW);
  const auto gate = [&](auto g) {
    constexpr int GATE = decltype(g)::value;
    if (a.out_dtype != QGEMM_DT_FP8_E4M3) rows_kernel<NW, GATE, false><<<grid, block, 0, s>>>(a);
    else if constexpr (GATE != QGEMM_GATE_NONE) rows_kernel<NW, GATE, true><<<grid, block, 0, s>>>(a);
  };
  switch (a.gate) {
    case QGEMM_GATE_NONE: gate(std::integral_constant<int, QGEMM_GATE_NONE>{}); break;
    case QGEMM_GATE_SILU: gate(std::integral_constant<int, QGEMM_GATE_SILU>{}); break;
    default: gate(std::integral_constant<int, QGEMM_GATE_GELU_TANH>{}); break;
  }
}

}  // namespace

hipError_t launch_rows(const W8Plan& pl, const W8Args& a, hipStream_t stream) {
  pl.waves == 8 ? launch_waves<8>(pl, a, stream) : launch_waves<4>(pl, a, stream);
  return hipGetLastError();
}

}  // namespace w8
}  // namespace qgemm
