// The stream kernel of the 8-bit products: tiles of 64 or 128 tokens, where the weights' way into the compute unit
// weighs more than the MFMAs.
//
//   p_r[m] = sum_b as[b][m] ws[r / 128][b] (sum_{k in block b} a[m][k] w[r][k])
//
// Workgroup = eight wavefronts side by side along the weight rows, TN blocks of 16 rows each (with a gate one of either
// projection); all of them take the same 16 TM tokens.  A weight row therefore belongs to one wavefront, which loads it
// straight into registers, ST k blocks ahead: through LDS, as in the tiles kernel, it would be written and read
// there for nothing, and LDS is what such small tiles wait for (a step of 64 tokens x 256 rows reads 96 KB and writes 40;
// here 64 and 8).  The tokens go from memory into LDS (buffer loads with the LDS destination; chunk c of row r at c ^ (r & 7)),
// ST stages deep, and stream past the weights from there.  MFMA operands, scales and precision are those of the tiles kernel.
#include <type_traits>

#include "qgemm_w8a8_fixup.h"

namespace qgemm {
namespace w8 {
namespace {

template <int TM, int TN, int ST, int GATE, bool Q, bool FP16>
__global__ __launch_bounds__(64 * kW8Waves) void stream_kernel(W8Args a) {
  constexpr int NW = kW8Waves, BM = 16 * TM;
  constexpr bool G = GATE != QGEMM_GATE_NONE;
  constexpr int WC = G ? 16 * TN / 2 : 16 * TN, COLS = NW * WC;          // output columns of a wavefront and of the tile
  constexpr int LA = BM / (8 * NW);                  // token loads of a wavefront per step
  static_assert(TM % 4 == 0 && (TN == 2 || (TN == 1 && !G)) && (ST == 3 || ST == 4), "shapes the rings below are made for");
  __shared__ __attribute__((aligned(1024))) unsigned char A0[BM * kBlock], A1[BM * kBlock], A2[BM * kBlock];
  __shared__ __attribute__((aligned(1024))) unsigned char A3[ST > 3 ? BM * kBlock : 16];
  const auto as = [&](int j) -> unsigned char* { return j == 0 ? A0 : j == 1 ? A1 : j == 2 ? A2 : A3; };
  const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles = gridDim.x / a.splits, split = blockIdx.x / tiles, tile = blockIdx.x - split * tiles;
  int tm, tn;
  tile_of(tile, tiles, a.tiles_n, tm, tn);
  const int m0 = tm * BM, n0 = tn * COLS, c0 = n0 + wave * WC;
  const int kb0 = split * a.kb_per_split, kb1 = min(a.KB, kb0 + a.kb_per_split), kl = kb1 - 1;

  // ---- loads: rows past the last read as zero, like the scales of tokens past the last
  const __amdgpu_buffer_rsrc_t ar = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(a.a + (size_t)m0 * a.K), (short)0, min(a.M - m0, BM) * a.K, 0x00020000);
  const int wrows = min(a.N - n0, COLS);
  const auto weights = [&](int part) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.w + ((size_t)part * a.N + n0) * a.K), (short)0, wrows * a.K,
                                             0x00020000);
  };
  const auto scales = [&](int row) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(a.ws + (size_t)row * a.KB), (short)0, a.KB * 4, 0x00020000);
  };
  const __amdgpu_buffer_rsrc_t wr0 = weights(0), wr1 = weights(G ? 1 : 0);
  const int rb = min(c0 / kBlock, a.row_blocks - 1);
  const __amdgpu_buffer_rsrc_t sr0 = scales(rb), sr1 = scales(G ? a.row_blocks + rb : rb);   // 32 rows lie in one block
  const int woff0 = (wave * WC + col) * a.K + 16 * g, woff1 = G ? woff0 : woff0 + 16 * a.K;
  const int arow = 8 * wave + (lane >> 3), aoff = arow * a.K + 16 * ((lane & 7) ^ (lane >> 3));
  const int first_token = 4 * (m0 + col);
  i32x4 w[ST][TN][2];
  float sa[ST][TM], sw[ST][TN];
  const auto load_step = [&](int kb, int j) {
#pragma unroll
    for (int i = 0; i < LA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ar, (lds_ptr_t)(as(j) + 8 * (NW * i + wave) * kBlock), 16, aoff + i * 8 * NW * a.K,
                                               kb * kBlock, 0, 0);
#pragma unroll
    for (int u = 0; u < TN; ++u)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        w[j][u][c] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(u ? wr1 : wr0, (u ? woff1 : woff0) + 64 * c,
                                                                                      kb * kBlock, 0));
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(a.as + (size_t)kb * a.M), (short)0, a.M * 4, 0x00020000);
#pragma unroll
    for (int i = 0; i < TM; ++i)
      sa[j][i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, first_token + 64 * i, 0, 0));
#pragma unroll
    for (int u = 0; u < TN; ++u)
      sw[j][u] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(u ? sr1 : sr0, 0, 4 * kb, 0));
  };
  // The loads of a step stay between two barriers (both are fences to the compiler): the waits count them.
  constexpr int LOADS = LA + 3 * TN + TM;
  static_assert((ST - 1) * LOADS <= 63, "vmcnt counts at most 63");
  constexpr auto vmcnt = [](int n) { return (n & 15) | (7 << 4) | ((n >> 4) << 14); };      // and no LDS read pending

  f32x4 acc[TN][TM];
#pragma unroll
  for (int u = 0; u < TN; ++u)
#pragma unroll
    for (int i = 0; i < TM; ++i) acc[u][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  // block sums that are not yet in acc, with their factors
  f32x4 p[4];
  float s[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    p[f] = f32x4{0.f, 0.f, 0.f, 0.f};
    s[f] = 0.f;
  }
  const auto accumulate = [&](int f, int u, int i) {
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[u][i][r] = __builtin_fmaf(p[f][r], s[f], acc[u][i][r]);
  };

  // tokens: two blocks are read ahead (fp16: one of them is being converted)
  constexpr int RING = FP16 ? 2 : 4;
  struct Chunks { i32x4 v[2]; };
  Chunks x[RING];
  const int off0 = col * kBlock + 16 * (g ^ (col & 7)), off1 = off0 ^ 64;
  const auto read = [&](const unsigned char* As, int i) {
    const unsigned char* q = As + i * 16 * kBlock;
    return Chunks{{*reinterpret_cast<const i32x4*>(q + off0), *reinterpret_cast<const i32x4*>(q + off1)}};
  };
  Halves xh[2][2], wh[TN][2];                        // fp16 operands
  const auto convert = [&](Halves (&to)[2], const Chunks& from, int e) {   // codes 2 e, 2 e + 1
    const unsigned codes = (unsigned)from.v[e >> 3][(e >> 1) & 3];
    const f16x2 v = e & 1 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, 1.0f, true)
                          : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, 1.0f, false);
    to[e >> 3].v[(e >> 2) & 1][2 * (e & 3)] = v[0];
    to[e >> 3].v[(e >> 2) & 1][2 * (e & 3) + 1] = v[1];
  };

  // One k block: its weights are in registers j, its tokens in stage j, the first two token blocks already read.  Once the last
  // token block has been read, one barrier says so and that the next stage has landed.
  const auto step = [&](auto stage, int kb_load) {
    constexpr int J = decltype(stage)::value;
    const unsigned char *const As = as(J), *const An = as((J + 1) % ST);
    if constexpr (FP16) {
#pragma unroll
      for (int u = 0; u < TN; ++u) {
        wh[u][0] = halves(w[J][u][0]);
        wh[u][1] = halves(w[J][u][1]);
      }
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      if (i == TM - 2) {
        __builtin_amdgcn_s_waitcnt(vmcnt((ST - 2) * LOADS));
        barrier();
      }
      const auto ahead = [&] { x[(i + 2) % RING] = i + 2 < TM ? read(As, i + 2) : read(An, i + 2 - TM); };
      if constexpr (FP16) {
#pragma unroll
        for (int e = 0; e < 4 * TN; ++e) {           // (quarter of the k block, weight block)
          const int q = e / TN, u = e % TN, f = (i & 1) * TN + u;
          __builtin_amdgcn_sched_barrier(0);
          if (q == 1) accumulate(TN - f + 2 * u, u, (i + TM - 1) % TM);
          p[f] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wh[u][q >> 1].v[q & 1], xh[i & 1][q >> 1].v[q & 1],
                                                        q ? p[f] : f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
          if (q == 0) s[f] = sa[J][i] * sw[J][u];
          if (e == 0) ahead();
#pragma unroll
          for (int c = 0; c < 4 / TN; ++c) convert(xh[(i + 1) & 1], x[(i + 1) % RING], e * (4 / TN) + c);
        }
      } else {
        const Chunks& xi = x[i % RING];
        const i32x8 x8 = __builtin_shufflevector(xi.v[0], xi.v[1], 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
        for (int u = 0; u < TN; ++u) {
          const int f = i * TN + u, before = (f + TM * TN - 4) % (TM * TN);
          __builtin_amdgcn_sched_barrier(0);
          accumulate(f % 4, before % TN, before / TN);
          const i32x8 w8 = __builtin_shufflevector(w[J][u][0], w[J][u][1], 0, 1, 2, 3, 4, 5, 6, 7);
          p[f % 4] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w8, x8, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
          s[f % 4] = sa[J][i] * sw[J][u];
          if (u == 0) ahead();
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    load_step(kb_load, J);
    __builtin_amdgcn_sched_barrier(0);
  };

#pragma unroll
  for (int j = 0; j < ST; ++j) {
    asm volatile("" ::: "memory");
    load_step(min(kb0 + j, kl), j);
  }
  __builtin_amdgcn_s_waitcnt(vmcnt((ST - 1) * LOADS));
  barrier();
  x[0] = read(A0, 0);
  x[1] = read(A0, 1);
  if constexpr (FP16) {
#pragma unroll
    for (int e = 0; e < 16; ++e) convert(xh[0], x[0], e);
  }
  int kb = kb0;
  const auto next = [&](auto stage) {
    step(stage, min(kb + ST, kl));                   // loads past the end read the last k block again, unused
    ++kb;
  };
  constexpr std::integral_constant<int, 0> S0{};
  constexpr std::integral_constant<int, 1> S1{};
  constexpr std::integral_constant<int, 2> S2{};
  constexpr std::integral_constant<int, (ST > 3 ? 3 : 0)> S3{};
  while (kb + ST <= kb1) {
    next(S0);
    next(S1);
    next(S2);
    if constexpr (ST > 3) next(S3);
  }
  if (kb < kb1) {
    next(S0);
    if (kb < kb1) {
      next(S1);
      if constexpr (ST > 3)
        if (kb < kb1) next(S2);
    }
  }
  if constexpr (FP16) {
#pragma unroll
    for (int u = 0; u < TN; ++u) accumulate(TN + u, u, TM - 1);
  } else {
#pragma unroll
    for (int f = TM * TN - 4; f < TM * TN; ++f) accumulate(f % 4, f % TN, f / TN);
  }
  __builtin_amdgcn_s_waitcnt(0);                     // no load is still writing LDS
  __syncthreads();                                   // and no wavefront reads it: what follows uses it otherwise
  finish_tile<NW, NW, GATE, Q>(a, acc, A0, A1, tile, split, tn, m0, 0, wave, c0);
}

template <int TM, int ST>
void launch_tile(const W8Plan& pl, const W8Args& a, hipStream_t s) {
  const dim3 grid(pl.grid), block(64 * kW8Waves);
  const auto kernel = [&](auto g, auto quantized, auto tn) {
    constexpr int GATE = decltype(g)::value, TN = decltype(tn)::value;
    constexpr bool Q = decltype(quantized)::value;
    if (Q || a.out_dtype == QGEMM_DT_F32) stream_kernel<TM, TN, ST, GATE, Q, true><<<grid, block, 0, s>>>(a);
    else if constexpr (!Q) stream_kernel<TM, TN, ST, GATE, Q, false><<<grid, block, 0, s>>>(a);
  };
  constexpr std::integral_constant<int, QGEMM_GATE_NONE> none{};
  constexpr std::integral_constant<int, QGEMM_GATE_SILU> silu{};
  constexpr std::integral_constant<int, QGEMM_GATE_GELU_TANH> gelu{};
  constexpr std::integral_constant<int, 1> one{};
  constexpr std::integral_constant<int, 2> two{};
  const bool q = a.out_dtype == QGEMM_DT_FP8_E4M3;
  if (a.gate == QGEMM_GATE_NONE) pl.blocks == 1 ? kernel(none, std::false_type{}, one) : kernel(none, std::false_type{}, two);
  else if (a.gate == QGEMM_GATE_SILU) q ? kernel(silu, std::true_type{}, two) : kernel(silu, std::false_type{}, two);
  else q ? kernel(gelu, std::true_type{}, two) : kernel(gelu, std::false_type{}, two);
}

}  // namespace

hipError_t launch_stream(const W8Plan& pl, const W8Args& a, hipStream_t stream) {
  pl.tile == 64 ? launch_tile<4, 4>(pl, a, stream) : launch_tile<8, 3>(pl, a, stream);
  return hipGetLastError();
}

}  // namespace w8
}  // namespace qgemm
