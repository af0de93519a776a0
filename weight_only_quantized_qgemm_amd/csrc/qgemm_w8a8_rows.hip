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

template <int MB, int U, int GATE, bool Q>
__global__ __launch_bounds__(64 * kW8Waves) void rows_kernel(W8Args a) {
  constexpr int NW = kW8Waves, F = Q ? kBlock / 16 : 1;
  __shared__ f32x4 sums[NW][U][MB][64];
  __shared__ int s_last;
  const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // workgroup = (group of F column blocks, column block in it, split)
  const int member = blockIdx.x % (F * a.splits), group = blockIdx.x / (F * a.splits);
  const int cb = member / a.splits, split = member - cb * a.splits;
  const int n0 = (group * F + cb) * 16;              // first output column
  const int kb0 = split * a.kb_per_split, kb1 = min(a.KB, kb0 + a.kb_per_split);

  const uint8_t* wp[U];
  const float* sp[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    wp[u] = a.w + ((size_t)(u * a.N + n0) + col) * a.K + 16 * g;
    sp[u] = a.ws + (size_t)(u * a.row_blocks + n0 / kBlock) * a.KB;
  }
  const uint8_t* ap[MB];
  int token[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    token[i] = min(16 * i + col, a.M - 1);           // rows past the last repeat it and are not stored
    ap[i] = a.a + (size_t)token[i] * a.K + 16 * g;
  }
  f32x4 acc[U][MB];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[u][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Chunks { i32x4 v[2]; };
  const auto chunks = [](const uint8_t* p) {
    return Chunks{{*reinterpret_cast<const i32x4*>(p), *reinterpret_cast<const i32x4*>(p + 64)}};
  };

  for (int kb = kb0 + wave; kb < kb1; kb += NW) {
    Chunks w[U], x[MB];
    float sw[U], sa[MB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      w[u] = chunks(wp[u] + (size_t)kb * kBlock);
      sw[u] = sp[u][kb];
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      x[i] = chunks(ap[i] + (size_t)kb * kBlock);
      sa[i] = a.as[(size_t)kb * a.M + token[i]];
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const Halves x0 = halves(x[i].v[0]), x1 = halves(x[i].v[1]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const Halves w0 = halves(w[u].v[0]), w1 = halves(w[u].v[1]);
        f32x4 p = __builtin_amdgcn_mfma_f32_16x16x32_f16(w0.v[0], x0.v[0], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
        p = __builtin_amdgcn_mfma_f32_16x16x32_f16(w0.v[1], x0.v[1], p, 0, 0, 0);
        p = __builtin_amdgcn_mfma_f32_16x16x32_f16(w1.v[0], x1.v[0], p, 0, 0, 0);
        p = __builtin_amdgcn_mfma_f32_16x16x32_f16(w1.v[1], x1.v[1], p, 0, 0, 0);
        const float s = sa[i] * sw[u];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[u][i][r] = __builtin_fmaf(p[r], s, acc[u][i][r]);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < MB; ++i) sums[wave][u][i][lane] = acc[u][i];
  __syncthreads();
  // wavefront i finishes token tile i
  f32x4 v[U];
  if (wave < MB) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u] = sums[0][u][wave][lane];
#pragma unroll
      for (int w = 1; w < NW; ++w) v[u] += sums[w][u][wave][lane];
    }
  }
  const int members = F * a.splits;
  const __amdgpu_buffer_rsrc_t part = __builtin_amdgcn_make_buffer_rsrc(
      a.partials + (size_t)group * members * (U * MB * 256), (short)0, members * (U * MB * 1024), 0x00020000);
  if (members > 1) {
    if (wave < MB) {
#pragma unroll
      for (int u = 0; u < U; ++u) store_partial(part, ((member * U + u) * MB + wave) * 1024 + 16 * lane, v[u]);
    }
    if (!last_arrival(a.tickets + group, members, &s_last)) return;
  }
  if constexpr (!Q) {
    if (wave >= MB) return;
    if (members > 1) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v[u] = load_partial(part, (u * MB + wave) * 1024 + 16 * lane);
        for (int s = 1; s < a.splits; ++s) v[u] += load_partial(part, ((s * U + u) * MB + wave) * 1024 + 16 * lane);
      }
    }
    const int m = 16 * wave + col;
    if (m < a.M) store4(a, (size_t)m * a.N + n0 + 4 * g, gated<GATE>(v[0], v[U - 1]));
  } else {
    // wavefront w finishes column block w of the scale block, one token tile after the other
    __shared__ unsigned top[NW][16];
    const int n = group * kBlock + 16 * wave + 4 * g;
#pragma unroll
    for (int i = 0; i < MB; ++i) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v[u] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < a.splits; ++s)
          v[u] += load_partial(part, (((wave * a.splits + s) * U + u) * MB + i) * 1024 + 16 * lane);
      }
      const f32x4 y = gated<GATE>(v[0], v[U - 1]);
      unsigned m = max(max(magnitude(y[0]), magnitude(y[1])), max(magnitude(y[2]), magnitude(y[3])));
      m = max(m, (unsigned)__shfl_xor((int)m, 16));
      m = max(m, (unsigned)__shfl_xor((int)m, 32));
      if (i) __syncthreads();
      if (lane < 16) top[wave][lane] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < NW; ++w) m = max(m, top[w][col]);
      const BlockScale b = block_scale(m, 1.0f);
      const int t = 16 * i + col;
      if (t < a.M) {
        *reinterpret_cast<unsigned*>(static_cast<uint8_t*>(a.out) + (size_t)t * a.N + n) =
            codes4(y[0] * b.to_code, y[1] * b.to_code, y[2] * b.to_code, y[3] * b.to_code);
        if (wave == 0 && g == 0) a.os[(size_t)group * a.M + t] = b.scale;
      }
    }
  }
}

template <int MB>
void launch_mb(const W8Plan& pl, const W8Args& a, hipStream_t s) {
  const dim3 grid(pl.grid), block(64 * kW8Waves);
  const bool q = a.out_dtype == QGEMM_DT_FP8_E4M3;
  if (a.gate == QGEMM_GATE_NONE) rows_kernel<MB, 1, QGEMM_GATE_NONE, false><<<grid, block, 0, s>>>(a);
  else if (a.gate == QGEMM_GATE_SILU)
    q ? rows_kernel<MB, 2, QGEMM_GATE_SILU, true><<<grid, block, 0, s>>>(a)
      : rows_kernel<MB, 2, QGEMM_GATE_SILU, false><<<grid, block, 0, s>>>(a);
  else
    q ? rows_kernel<MB, 2, QGEMM_GATE_GELU_TANH, true><<<grid, block, 0, s>>>(a)
      : rows_kernel<MB, 2, QGEMM_GATE_GELU_TANH, false><<<grid, block, 0, s>>>(a);
}

}  // namespace

hipError_t launch_rows(const W8Plan& pl, const W8Args& a, hipStream_t stream) {
  switch (pl.tile) {
    case 16: launch_mb<1>(pl, a, stream); break;
    case 32: launch_mb<2>(pl, a, stream); break;
    case 48: launch_mb<3>(pl, a, stream); break;
    default: launch_mb<4>(pl, a, stream); break;
  }
  return hipGetLastError();
}

}  // namespace w8
}  // namespace qgemm
