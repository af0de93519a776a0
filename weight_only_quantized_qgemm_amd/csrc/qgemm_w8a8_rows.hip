// The rows kernel of the 8-bit products: a few tokens (M <= 64), the weights streamed once.
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
// The wavefronts' sums meet in LDS, in wavefront order.  Where several workgroups make one output (splits along
// K; the eight column blocks of an output scale block) each leaves its fp32 sums in the workspace and takes a
// ticket, and the one that draws the last ticket adds them in order and finishes: no workgroup waits for another.
#include "qgemm_w8a8_fixup.h"

namespace qgemm {
namespace w8 {
namespace {

template <int MB, int U, int NW, int D, int OCC, int GATE, bool Q>
__global__ __launch_bounds__(64 * NW, OCC) void rows_kernel(W8Args a) {
  constexpr bool G = GATE != QGEMM_GATE_NONE;
  constexpr int CB = G ? U / 2 : U;                  // column blocks of a workgroup
  constexpr int F = Q ? kBlock / 16 / CB : 1;        // workgroups along the columns of one output scale block
  __shared__ f32x4 sums[NW / 2][U][MB][64];
  __shared__ int s_last;
  const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // workgroup = (group, F columns in it, split)
  const int members = F * a.splits;
  const int member = blockIdx.x % members, group = blockIdx.x / members;
  const int cg = member / a.splits, split = member - cg * a.splits;
  const int cb0 = (group * F + cg) * CB;             // first column block
  const int kb0 = split * a.kb_per_split, kb1 = min(a.KB, kb0 + a.kb_per_split);

  // weight block u: column block u % CB of projection u / CB; blocks past the last repeat it and are not stored
  // (addresses: a uniform base and a 32-bit offset per lane; 64 rows of K <= 2^22 stay below 2^28)
  const uint8_t* wp[U];
  const float* sp[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int n = min(cb0 + u % CB, (a.N >> 4) - 1) * 16;
    wp[u] = a.w + ((size_t)(u / CB) * a.N + n) * a.K;
    sp[u] = a.ws + ((size_t)(u / CB) * a.row_blocks + n / kBlock) * a.KB;
  }
  const unsigned woff = col * a.K + 16 * g;
  unsigned token[MB], aoff[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    token[i] = min(16 * i + col, a.M - 1);           // likewise
    aoff[i] = token[i] * a.K + 16 * g;
  }
  f32x4 acc[U][MB];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[u][i] = f32x4{0.f, 0.f, 0.f, 0.f};

  // D k blocks in flight per wavefront, each in registers of its own
  struct Chunks { i32x4 v[2]; };
  Chunks w[D][U], x[D][MB];
  float sw[D][U], sa[D][MB];
  const auto chunks = [](const uint8_t* p, unsigned off) {
    return Chunks{{*reinterpret_cast<const i32x4*>(p + off), *reinterpret_cast<const i32x4*>(p + 64 + off)}};
  };
  bool in[D];                                        // whether the block in set d is one of this wavefront's
  const auto load = [&](int d, int at) {
    in[d] = at < kb1;
    const int kb = min(at, kb1 - 1);
#pragma unroll
    for (int u = 0; u < U; ++u) w[d][u] = chunks(wp[u] + (size_t)kb * kBlock, woff);
#pragma unroll
    for (int i = 0; i < MB; ++i) x[d][i] = chunks(a.a + (size_t)kb * kBlock, aoff[i]);
#pragma unroll
    for (int u = 0; u < U; ++u) sw[d][u] = sp[u][kb];
#pragma unroll
    for (int i = 0; i < MB; ++i) sa[d][i] = (a.as + (size_t)kb * a.M)[token[i]];
  };
  const auto compute = [&](int d) {
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const Halves x0 = halves(x[d][i].v[0]), x1 = halves(x[d][i].v[1]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const Halves w0 = halves(w[d][u].v[0]), w1 = halves(w[d][u].v[1]);
        f32x4 p = __builtin_amdgcn_mfma_f32_16x16x32_f16(w0.v[0], x0.v[0], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
        p = __builtin_amdgcn_mfma_f32_16x16x32_f16(w0.v[1], x0.v[1], p, 0, 0, 0);
        p = __builtin_amdgcn_mfma_f32_16x16x32_f16(w1.v[0], x1.v[0], p, 0, 0, 0);
        p = __builtin_amdgcn_mfma_f32_16x16x32_f16(w1.v[1], x1.v[1], p, 0, 0, 0);
        const float s = in[d] ? sa[d][i] * sw[d][u] : 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[u][i][r] = __builtin_fmaf(p[r], s, acc[u][i][r]);
        if (U * MB > 4) __builtin_amdgcn_sched_barrier(0);   // the weights are converted for each token tile: held, they would not fit
      }
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

  // the wavefronts' sums: 4 .. 7 into 0 .. 3, then those four in order
  if (wave >= NW / 2) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < MB; ++i) sums[wave - NW / 2][u][i][lane] = acc[u][i];
  }
  __syncthreads();
  if (wave < NW / 2) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < MB; ++i) sums[wave][u][i][lane] += acc[u][i];
  }
  __syncthreads();
  const __amdgpu_buffer_rsrc_t part = __builtin_amdgcn_make_buffer_rsrc(
      a.partials + (size_t)group * members * (U * MB * 256), (short)0, members * (U * MB * 1024), 0x00020000);
  const auto slot = [&](int m, int u, int i) { return ((m * U + u) * MB + i) * 1024 + 16 * lane; };
  const auto joined = [&](int u, int i) {
    f32x4 v = sums[0][u][i][lane];
#pragma unroll
    for (int w = 1; w < NW / 2; ++w) v += sums[w][u][i][lane];
    return v;
  };
  if (members > 1) {
    for (int f = wave; f < U * MB; f += NW) store_partial(part, slot(member, f / MB, f % MB), joined(f / MB, f % MB));
    if (!last_arrival(a.tickets + group, members, &s_last)) return;
  }
  if constexpr (!Q) {
    // one (column block, token tile) after the other, by the wavefronts in turn
    for (int f = wave; f < CB * MB; f += NW) {
      const int c = f / MB, i = f % MB;
      f32x4 v[2];
#pragma unroll
      for (int part_of = 0; part_of < (G ? 2 : 1); ++part_of) {
        const int u = part_of * CB + c;
        if (members > 1) {
          v[part_of] = load_partial(part, slot(0, u, i));
          for (int s = 1; s < a.splits; ++s) v[part_of] += load_partial(part, slot(s, u, i));
        } else {
          v[part_of] = joined(u, i);
        }
      }
      const int m = 16 * i + col, n = (cb0 + c) * 16 + 4 * g;
      if (m < a.M && n < a.N) store4(a, (size_t)m * a.N + n, gated<GATE>(v[0], v[G ? 1 : 0]));
    }
  } else {
    // first every column block's outputs and largest magnitudes, then the codes
    constexpr int NB = kBlock / 16;
    __shared__ f32x4 outs[NB * MB][64];
    __shared__ unsigned top[NB * MB][16];
    for (int f = wave; f < NB * MB; f += NW) {
      const int c = f % NB, i = f / NB;
      f32x4 v[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
      for (int s = 0; s < a.splits; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) v[h] += load_partial(part, slot(c / CB * a.splits + s, h * CB + c % CB, i));
      const f32x4 y = gated<GATE>(v[0], v[1]);
      unsigned m = max(max(magnitude(y[0]), magnitude(y[1])), max(magnitude(y[2]), magnitude(y[3])));
      m = max(m, (unsigned)__shfl_xor((int)m, 16));
      m = max(m, (unsigned)__shfl_xor((int)m, 32));
      outs[f][lane] = y;
      if (lane < 16) top[f][lane] = m;
    }
    __syncthreads();
    for (int f = wave; f < NB * MB; f += NW) {
      const int c = f % NB, i = f / NB, t = 16 * i + col;
      unsigned m = 0;
#pragma unroll
      for (int b = 0; b < NB; ++b) m = max(m, top[NB * i + b][col]);
      const BlockScale b = block_scale(m, 1.0f);
      const f32x4 y = outs[f][lane];
      if (t < a.M) {
        *reinterpret_cast<unsigned*>(static_cast<uint8_t*>(a.out) + (size_t)t * a.N + group * kBlock + 16 * c + 4 * g) =
            codes4(y[0] * b.to_code, y[1] * b.to_code, y[2] * b.to_code, y[3] * b.to_code);
        if (c == 0 && g == 0) a.os[(size_t)group * a.M + t] = b.scale;
      }
    }
  }
}

#ifndef R1
#define R1 8, 2, 4
#define R1G 8, 2, 4
#define R2 8, 2, 2
#define R3 8, 2, 2
#define R4 8, 2, 2
#endif
template <int MB, int U, int NW, int D, int OCC>
void launch_mb(const W8Plan& pl, const W8Args& a, hipStream_t s) {
  const dim3 grid(pl.grid), block(64 * NW);
  const bool q = a.out_dtype == QGEMM_DT_FP8_E4M3;
  if (a.gate == QGEMM_GATE_NONE) rows_kernel<MB, U, NW, D, OCC, QGEMM_GATE_NONE, false><<<grid, block, 0, s>>>(a);
  else if constexpr (U > 1) {
  if (a.gate == QGEMM_GATE_SILU)
    q ? rows_kernel<MB, U, NW, D, OCC, QGEMM_GATE_SILU, true><<<grid, block, 0, s>>>(a)
      : rows_kernel<MB, U, NW, D, OCC, QGEMM_GATE_SILU, false><<<grid, block, 0, s>>>(a);
  else
    q ? rows_kernel<MB, U, NW, D, OCC, QGEMM_GATE_GELU_TANH, true><<<grid, block, 0, s>>>(a)
      : rows_kernel<MB, U, NW, D, OCC, QGEMM_GATE_GELU_TANH, false><<<grid, block, 0, s>>>(a);
  }
}

}  // namespace

hipError_t launch_rows(const W8Plan& pl, const W8Args& a, hipStream_t stream) {
  switch (pl.tile) {
    case 16:
      if (pl.blocks == 1) launch_mb<1, 1, R1>(pl, a, stream);
      else launch_mb<1, 2, R1G>(pl, a, stream);
      break;
    case 32: launch_mb<2, rows_blocks(32, false), R2>(pl, a, stream); break;
    case 48: launch_mb<3, rows_blocks(48, false), R3>(pl, a, stream); break;
    default: launch_mb<4, rows_blocks(64, false), R4>(pl, a, stream); break;
  }
  return hipGetLastError();
}

}  // namespace w8
}  // namespace qgemm
