// The rows kernel of the 8-bit products: up to 64 tokens, the weights streamed once.
//
//   p_r[m] = sum_b as[b][m] ws[r / 128][b] (sum_{k in block b} a[m][k] w[r][k])
//
// A workgroup owns one 16-row weight block (with a gate that of both projections); its wavefronts take the k
// blocks of 128 in turn, so that together they read 1 KiB of every weight row side by side.  The weights are, as fp16, the
// first operand of v_mfma_f32_16x16x32_f16 and the tokens' codes the second: lane l holds row (token) l & 15 and the
// 16-byte chunks l >> 4 and 4 + (l >> 4) of the k block, the same for both, which is all that a dot product asks of its
// order.  The result has token l & 15 and weight rows 4 (l >> 4) .. + 3 in lane l, so both scales are one factor per lane, applied
// to the fp32 block sum.
//
// Each wavefront brings its k blocks into LDS of its own (buffer loads with the LDS destination, eight rows of 128 bytes
// each, chunk c of row r at c ^ (r & 7)) and reads the operands from there; nothing is shared, so there is no barrier.  Loaded
// straight into the operands' registers, sixteen consecutive lanes address sixteen rows, and the address unit takes them one by
// one: 10240 x 5120, 16 tokens 18.1 us that way and 14.9 this, one token 12.8 and 12.2; 11008 x 4096 gated, 21.8 and 20.2, 19.9 and
// 19.1 (weights from memory).  One token reads at 4.7 TB/s for the latter, at 5.1 for 10240 x 5120 less 2 us for the launch and the
// last block's latency.  With one workgroup a compute unit 4096 x 11008 reads at 3.5 TB/s (12.7 us), with two 8192 x 28672 at 5.1.
//
// The wavefronts' sums meet in LDS, in wavefront order.  Where several workgroups make one output (splits along
// K; the eight column blocks of an output scale block) each leaves its fp32 sums in the workspace and takes a
// ticket, and the one that draws the last ticket adds them in order and finishes: no workgroup waits for another.
#include <type_traits>

#include "qgemm_w8a8_fixup.h"

namespace qgemm {
namespace w8 {
namespace {

// XH: loads of eight tokens each.
template <int NW, int XH, int GATE, bool Q>
__global__ __launch_bounds__(64 * NW) void rows_kernel(W8Args a) {
  constexpr bool G = GATE != QGEMM_GATE_NONE;
  constexpr int U = G ? 2 : 1;                       // weight blocks: one of either projection
  constexpr int F = Q ? kBlock / 16 : 1;             // workgroups along the columns of one output scale block
  // Two stages per wavefront: to 16 tokens 64 KiB for eight, 48 for four with a gate, so that two or three workgroups share a
  // compute unit (one stage more and 11008 x 4096 gated to e4m3 takes 24.7 us instead of 21.6, 4096 x 4096 6.0 instead of 5.4;
  // only 16 x 4096 x 11008 gains, 13.9 and 14.1).
  constexpr int MB = (XH + 1) / 2;                   // token blocks
  constexpr int SLOT = (U + MB) * 16 * kBlock;
  __shared__ __attribute__((aligned(1024))) unsigned char S0[NW * SLOT], S1[NW * SLOT];
  auto& sums = *reinterpret_cast<f32x4(*)[NW / 2][U * MB][64]>(S0);   // after the last k block, as the next two
  int* const s_last = reinterpret_cast<int*>(S1);
  auto& top = *reinterpret_cast<unsigned(*)[kBlock / 16][16 * MB]>(S1 + 16);   // largest magnitude of a token in each column block
  const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // workgroup = (group, column block in it, split)
  const int members = F * a.splits;
  const int member = blockIdx.x % members, group = blockIdx.x / members;
  const int cb = member / a.splits, split = member - cb * a.splits;
  const int n0 = (group * F + cb) * 16;              // first output column
  const int kb0 = split * a.kb_per_split, kb1 = min(a.KB, kb0 + a.kb_per_split);

  // ---- loads; tokens past the last read as zero
  const int drow = lane >> 3, lane_off = drow * a.K + 16 * ((lane & 7) ^ drow);
  const auto rows = [&](const uint8_t* p, int n) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), (short)0, n * a.K, 0x00020000);
  };
  const auto scales = [&](int u) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(a.ws + ((size_t)u * a.row_blocks + n0 / kBlock) * a.KB), (short)0,
                                             a.KB * 4, 0x00020000);
  };
  const __amdgpu_buffer_rsrc_t xr = rows(a.a, a.M), wr0 = rows(a.w + (size_t)n0 * a.K, 16),
                               wr1 = rows(a.w + ((size_t)(U - 1) * a.N + n0) * a.K, 16), sr0 = scales(0), sr1 = scales(U - 1);
  f32x4 acc[U * MB];
#pragma unroll
  for (int u = 0; u < U * MB; ++u) acc[u] = f32x4{0.f, 0.f, 0.f, 0.f};

  float sw[2][U], sa[2][MB];
  bool in[2];                                        // whether the block in stage d is one of this wavefront's
  const auto stage = [&](int d) { return (d ? S1 : S0) + wave * SLOT; };
  const auto as_float = [](unsigned v) { return __builtin_bit_cast(float, v); };
  const auto load = [&](int d, int at) {
    in[d] = at < kb1;
    const int kb = min(at, kb1 - 1);
#pragma unroll
    for (int u = 0; u <= U; ++u)                     // the weights' blocks, then the tokens'
#pragma unroll
      for (int h = 0; h < (u == U ? XH : 2); ++h)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(u == U ? xr : u ? wr1 : wr0, (lds_ptr_t)(stage(d) + (2 * u + h) * 1024), 16,
                                                 lane_off + 8 * h * a.K, kb * kBlock, 0, 0);
#pragma unroll
    for (int u = 0; u < U; ++u) sw[d][u] = as_float(__builtin_amdgcn_raw_buffer_load_b32(u ? sr1 : sr0, 0, 4 * kb, 0));
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(a.as + (size_t)kb * a.M), (short)0, a.M * 4, 0x00020000);
#pragma unroll
    for (int i = 0; i < MB; ++i) sa[d][i] = as_float(__builtin_amdgcn_raw_buffer_load_b32(r, 4 * (16 * i + col), 0, 0));
  };
  constexpr int LOADS = 3 * U + MB + XH;              // vector loads of a stage
  constexpr auto vmcnt = [](int n) { return (n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14); };
  constexpr int lds_read = 15 | (7 << 4) | (3 << 14);       // no LDS read pending
  const int off0 = col * kBlock + 16 * (g ^ (col & 7)), off1 = off0 ^ 64;
  struct Chunks { i32x4 v[2]; };
  Chunks w[U], x[MB];
  float f[U * MB];
  const auto read = [&](int d) {
    __builtin_amdgcn_s_waitcnt(vmcnt(LOADS));        // this stage has landed, the other may be on its way
    // the scales are used from here on: moved up to the other stage's, their product would wait for everything
#pragma unroll
    for (int u = 0; u < U; ++u) asm volatile("" : "+v"(sw[d][u]));
#pragma unroll
    for (int i = 0; i < MB; ++i) asm volatile("" : "+v"(sa[d][i]));
    asm volatile("" ::: "memory");
    const auto chunks = [&](const unsigned char* p) {
      return Chunks{{*reinterpret_cast<const i32x4*>(p + off0), *reinterpret_cast<const i32x4*>(p + off1)}};
    };
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = chunks(stage(d) + u * 2048);
#pragma unroll
    for (int i = 0; i < MB; ++i) x[i] = chunks(stage(d) + (U + i) * 2048);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < MB; ++i) f[u * MB + i] = in[d] ? sa[d][i] * sw[d][u] : 0.f;
    __builtin_amdgcn_s_waitcnt(lds_read);            // before the next load writes the stage
    asm volatile("" ::: "memory");
  };
  const auto compute = [&] {
    Halves wh[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      wh[u][0] = halves(w[u].v[0]);
      wh[u][1] = halves(w[u].v[1]);
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const Halves x0 = halves(x[i].v[0]), x1 = halves(x[i].v[1]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        f32x4 p = __builtin_amdgcn_mfma_f32_16x16x32_f16(wh[u][0].v[0], x0.v[0], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
        p = __builtin_amdgcn_mfma_f32_16x16x32_f16(wh[u][0].v[1], x0.v[1], p, 0, 0, 0);
        p = __builtin_amdgcn_mfma_f32_16x16x32_f16(wh[u][1].v[0], x1.v[0], p, 0, 0, 0);
        p = __builtin_amdgcn_mfma_f32_16x16x32_f16(wh[u][1].v[1], x1.v[1], p, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[u * MB + i][r] = __builtin_fmaf(p[r], f[u * MB + i], acc[u * MB + i][r]);
      }
    }
  };
  // The last round is as long as the others: blocks past the end are the last one again, with factor 0 (branches
  // around them would copy the sums from register to register).
  load(0, kb0 + wave);
  asm volatile("" ::: "memory");                     // the first wait counts the second load
  load(1, kb0 + wave + NW);
  for (int kb = kb0 + wave; kb < kb1; kb += 2 * NW) {
    read(0);
    load(0, kb + 2 * NW);
    compute();
    read(1);
    load(1, kb + 3 * NW);
    compute();
  }
  __builtin_amdgcn_s_waitcnt(0);                     // no load is still writing LDS
  __syncthreads();

  // the wavefronts' sums: the second half into the first, then those in order; block b is token block b % MB of projection b / MB
  constexpr int B = U * MB;
  if (wave >= NW / 2) {
#pragma unroll
    for (int b = 0; b < B; ++b) sums[wave - NW / 2][b][lane] = acc[b];
  }
  __syncthreads();
  if (wave < NW / 2) {
#pragma unroll
    for (int b = 0; b < B; ++b) sums[wave][b][lane] += acc[b];
  }
  __syncthreads();
  const __amdgpu_buffer_rsrc_t part =
      __builtin_amdgcn_make_buffer_rsrc(a.partials + (size_t)group * members * (B * 256), (short)0, members * (B * 1024), 0x00020000);
  const auto slot = [&](int m, int b) { return (m * B + b) * 1024 + 16 * lane; };
  const auto joined = [&](int b) {
    f32x4 v = sums[0][b][lane];
#pragma unroll
    for (int w = 1; w < NW / 2; ++w) v += sums[w][b][lane];
    return v;
  };
  if (members > 1) {
    for (int b = wave; b < B; b += NW) store_partial(part, slot(member, b), joined(b));
    if (!last_arrival(a.tickets + group, members, s_last)) return;
  }
  if constexpr (!Q) {
    const int i = wave;                              // a wavefront finishes a token block
    if (i >= MB) return;
    f32x4 v[2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (members > 1) {
        v[u] = load_partial(part, slot(0, u * MB + i));
        for (int s = 1; s < a.splits; ++s) v[u] += load_partial(part, slot(s, u * MB + i));
      } else {
        v[u] = joined(u * MB + i);
      }
    }
    const int token = 16 * i + col;
    if (token < a.M) store4(a, (size_t)token * a.N + n0 + 4 * g, gated<GATE>(v[0], v[U - 1]));
  } else {
    // every column block's outputs and largest magnitudes, then the codes
    constexpr int PER = kBlock / 16 / NW > 0 ? kBlock / 16 / NW : 1;     // column blocks of a wavefront
    f32x4 y[PER][MB];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int c = wave * PER + j;
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        f32x4 v[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
        for (int s = 0; s < a.splits; ++s)
#pragma unroll
          for (int u = 0; u < 2; ++u) v[u] += load_partial(part, slot(c * a.splits + s, u * MB + i));
        y[j][i] = gated<GATE>(v[0], v[1]);
        unsigned m = max(max(magnitude(y[j][i][0]), magnitude(y[j][i][1])), max(magnitude(y[j][i][2]), magnitude(y[j][i][3])));
        m = max(m, (unsigned)__shfl_xor((int)m, 16));
        m = max(m, (unsigned)__shfl_xor((int)m, 32));
        if (g == 0) top[c][16 * i + col] = m;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int token = 16 * i + col;
      unsigned m = 0;
#pragma unroll
      for (int c = 0; c < kBlock / 16; ++c) m = max(m, top[c][token]);
      const BlockScale b = block_scale(m, 1.0f);
      if (token >= a.M) return;
#pragma unroll
      for (int j = 0; j < PER; ++j)
        *reinterpret_cast<unsigned*>(static_cast<uint8_t*>(a.out) + (size_t)token * a.N + group * kBlock + 16 * (wave * PER + j) + 4 * g) =
            codes4(y[j][i][0] * b.to_code, y[j][i][1] * b.to_code, y[j][i][2] * b.to_code, y[j][i][3] * b.to_code);
      if (wave == 0 && g == 0) a.os[(size_t)group * a.M + token] = b.scale;
    }
  }
}

template <int XH>
void launch_tokens(const W8Plan& pl, const W8Args& a, hipStream_t s) {
  const dim3 grid(pl.grid), block(64 * pl.waves);
  const bool q = a.out_dtype == QGEMM_DT_FP8_E4M3;
  if (a.gate == QGEMM_GATE_NONE)
    pl.waves == 8 ? rows_kernel<XH <= 4 ? 8 : 4, XH, QGEMM_GATE_NONE, false><<<grid, block, 0, s>>>(a)
                  : rows_kernel<4, XH, QGEMM_GATE_NONE, false><<<grid, block, 0, s>>>(a);
  else if (a.gate == QGEMM_GATE_SILU)
    q ? rows_kernel<4, XH, QGEMM_GATE_SILU, true><<<grid, block, 0, s>>>(a)
      : rows_kernel<4, XH, QGEMM_GATE_SILU, false><<<grid, block, 0, s>>>(a);
  else
    q ? rows_kernel<4, XH, QGEMM_GATE_GELU_TANH, true><<<grid, block, 0, s>>>(a)
      : rows_kernel<4, XH, QGEMM_GATE_GELU_TANH, false><<<grid, block, 0, s>>>(a);
}

}  // namespace

hipError_t launch_rows(const W8Plan& pl, const W8Args& a, hipStream_t stream) {
  // up to eight tokens are one load of a k block, not two (10240 x 5120: eight 12.9 us, nine 13.4)
  if (a.M <= 8) launch_tokens<1>(pl, a, stream);
  else if (a.M <= 16) launch_tokens<2>(pl, a, stream);
  else if (a.M <= 32) launch_tokens<4>(pl, a, stream);
  else if (a.M <= 48) launch_tokens<6>(pl, a, stream);
  else launch_tokens<8>(pl, a, stream);
  return hipGetLastError();
}

}  // namespace w8
}  // namespace qgemm
