// The tiles kernel of the 8-bit products: any number of tokens.
//
//   p_r[m] = sum_b as[b][m] ws[r / 128][b] (sum_{k in block b} a[m][k] w[r][k])
//
// Workgroup = eight wavefronts, WM along the tokens and WN along the weight rows; each owns TM x TN MFMA blocks of
// 16 tokens x 16 weight rows, the workgroup 16 WM TM tokens x 256 weight rows.  With a gate the first half of a
// wavefront's weight blocks are rows of the gate's projection and the second half the same rows of the other, so that
// both factors of an output meet in one lane.
//
// One step is one k block of 128: tokens and weights go from memory straight into LDS (buffer loads with the LDS
// destination), one stage ahead of the step that computes.  A load writes its 64 lanes' 16 bytes side by side, eight
// rows of 128 bytes; so that the operand reads (16 rows, one chunk each) spread over the banks, chunk c of row r is
// stored at c ^ (r & 7), by the choice of the address that each lane loads.  Rows past the last read as zero.
//
// The weights are the first MFMA operand and the tokens the second: lane l of the result holds token l & 15, so both
// scales of a k block are one factor per lane and MFMA block, and a step costs one fp32 FMA per 128 products beside the
// MFMA (16 issue cycles beside 32 MFMA cycles, or 64 with fp16 operands).
//
// What a step takes (us, 160 tiles at once over 4096 weight rows; its loads and barrier alone, its products and operand reads alone):
//                      e4m3 operands            fp16 operands
//   64 tokens          0.50 (0.39, 0.32)        0.93 (0.39, 0.80)
//   128 tokens         0.70 (0.46, 0.49)        1.45 (0.46, 1.25)
//   256 tokens         1.16 (0.82, 0.99)        2.60 (-, 2.35)
// So neither side bounds the smaller tiles by itself: they overlap in part, and a load's latency and the barrier show.  With fp16
// operands the issue of MFMAs, conversions and FMAs does (8192 x 11008 x 4096 gated to e4m3 1103 us, 1.34 PFLOP/s), with e4m3
// operands and 256 tokens LDS beside the MFMAs (a step reads 192 KiB and receives 64; 8192 x 10240 x 5120 to bf16 374 us, 2.3 PFLOP/s).
// 200 x 10240 x 5120: 26 us with the weights in the 256 MB cache (21 and 18), 35 from memory (34 and 18): the reading, by 160 of 256
// compute units.  Weights straight into registers instead: 50 us, since sixteen lanes would address sixteen rows.  More stages
// hide more of a load's 1.4 us: 64 tokens with two 35.1 us, with four 27.3.
#include <type_traits>

#include "qgemm_w8a8_fixup.h"

namespace qgemm {
namespace w8 {
namespace {

// OUT: outputs in 16 bits, fp32 or e4m3.  FP16: operands converted to fp16, whole sums; fp32 and e4m3 outputs have no other form.
enum Out { OUT_16, OUT_F32, OUT_E4M3 };
template <int WM, int TM, int ST, int GATE, Out OUT, bool FP16>
__global__ __launch_bounds__(64 * kW8Waves) void tiles_kernel(W8Args a) {
  constexpr int NW = kW8Waves, WN = NW / WM, TN = kTileRows / (16 * WN), BM = 16 * WM * TM;
  constexpr bool G = GATE != QGEMM_GATE_NONE, Q = OUT == OUT_E4M3;
  constexpr int COLS = G ? kTileRows / 2 : kTileRows;          // output columns of a tile
  constexpr int LA = BM / (8 * NW), LW = kTileRows / (8 * NW); // loads of a wavefront per step
  static_assert(!G || TN % 2 == 0, "both projections' rows lie in one wavefront");
  // Each stage is arrays of its own, so that the compiler can tell the one that is read from those being filled.
  __shared__ __attribute__((aligned(1024))) unsigned char A0[BM * kBlock], A1[BM * kBlock];
  __shared__ __attribute__((aligned(1024))) unsigned char W0[kTileRows * kBlock], W1[kTileRows * kBlock];
  __shared__ __attribute__((aligned(1024))) unsigned char A2[ST > 2 ? BM * kBlock : 16], W2[ST > 2 ? kTileRows * kBlock : 16];
  __shared__ __attribute__((aligned(1024))) unsigned char A3[ST > 3 ? BM * kBlock : 16], W3[ST > 3 ? kTileRows * kBlock : 16];
  static_assert(ST >= 2 && ST <= 4, "two to four stages");
  const auto as = [&](int j) -> unsigned char* { return j == 0 ? A0 : j == 1 ? A1 : j == 2 ? A2 : A3; };
  const auto ws = [&](int j) -> unsigned char* { return j == 0 ? W0 : j == 1 ? W1 : j == 2 ? W2 : W3; };
  const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  // whole tiles first, then those that are split along K
  const int tail = a.tiles - a.whole, at = blockIdx.x - a.whole;
  const int splits = at < 0 ? 1 : a.splits, split = at < 0 ? 0 : at / tail;
  const int tile = at < 0 ? (int)blockIdx.x : a.whole + at - split * tail;
  int tm, tn;
  tile_of(tile, a.tiles, a.tiles_n, tm, tn);
  const int m0 = tm * BM, n0 = tn * COLS;
  const int kb0 = split * a.kb_per_split, kb1 = splits > 1 ? min(a.KB, kb0 + a.kb_per_split) : a.KB;

  // ---- loads into LDS: 1 KiB each, eight rows
  const int drow = lane >> 3, dchunk = (lane & 7) ^ drow;
  const __amdgpu_buffer_rsrc_t ar = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(a.a + (size_t)m0 * a.K), (short)0, min(a.M - m0, BM) * a.K, 0x00020000);
  const int wrows = min(a.N - n0, COLS);
  const __amdgpu_buffer_rsrc_t wr0 = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(a.w + (size_t)n0 * a.K), (short)0, wrows * a.K, 0x00020000);
  const __amdgpu_buffer_rsrc_t wr1 = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(a.w + (size_t)(G ? a.N + n0 : n0) * a.K), (short)0, wrows * a.K, 0x00020000);
  const auto load = [&](int kb, unsigned char* As, unsigned char* Ws) {
    int lane_off = drow * a.K + 16 * dchunk;
    asm volatile("" : "+v"(lane_off));               // the loads' offsets are added up anew each step, not kept in registers
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const int r = 8 * (NW * i + wave);             // first row of the load
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ar, (lds_ptr_t)(As + r * kBlock), 16, lane_off + r * a.K, kb * kBlock, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < LW; ++i) {
      const int r = 8 * (NW * i + wave);
      if constexpr (G) {
        // row r of the tile: wavefront column r / (16 TN), its block t; blocks past the half are the other projection's
        const int t = (r >> 4) % TN, src = (r >> 4) / TN * (8 * TN) + t % (TN / 2) * 16 + (r & 15);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(t < TN / 2 ? wr0 : wr1, (lds_ptr_t)(Ws + r * kBlock), 16,
                                                 lane_off + src * a.K, kb * kBlock, 0, 0);
      } else {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(wr0, (lds_ptr_t)(Ws + r * kBlock), 16, lane_off + r * a.K, kb * kBlock, 0, 0);
      }
    }
  };

  // ---- scales: one per token block and lane (past the last token: 0); of the weights one per projection (a
  // wavefront's rows of one projection lie in one block of 128)
  const int c0 = n0 + wn * (G ? 8 * TN : 16 * TN);   // the wavefront's first output column
  const int rb = min(c0 / kBlock, a.row_blocks - 1);
  const auto scale_row = [&](int row) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(a.ws + (size_t)row * a.KB), (short)0, a.KB * 4, 0x00020000);
  };
  const __amdgpu_buffer_rsrc_t sr0 = scale_row(rb), sr1 = scale_row((G ? a.row_blocks : 0) + rb);
  const int first_token = 4 * (m0 + 16 * wm * TM + col);
  const auto as_float = [](unsigned v) { return __builtin_bit_cast(float, v); };

  f32x4 acc[TN][TM];
#pragma unroll
  for (int t = 0; t < TN; ++t)
#pragma unroll
    for (int i = 0; i < TM; ++i) acc[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};

  // operand chunks g and 4 + g of row `col` of a block of 16 rows
  const int off0 = col * kBlock + 16 * (g ^ (col & 7)), off1 = off0 ^ 64;
  const auto chunk = [](const unsigned char* p) { return *reinterpret_cast<const i32x4*>(p); };
  const int aoff = 16 * wm * TM * kBlock, woff = 16 * wn * TN * kBlock;
  // chunk c of the weights' blocks: half c & 1 of the operand of block c / 2
  const auto wchunk = [&](const unsigned char* Ws, int c) {
    return chunk(Ws + woff + c / 2 * 16 * kBlock + (c & 1 ? off1 : off0));
  };
  const auto achunk = [&](const unsigned char* As, int i, int c) {
    return chunk(As + aoff + i * 16 * kBlock + (c ? off1 : off0));
  };
  // A step's scales: sa of the tokens, times the weights' of either projection.  With two stages the scales of the next step
  // are loaded as it comes near (the 256-token tile has no registers for two sets), with more together with the step's data:
  // loads return in order, and one waited for late would wait for all.
  constexpr int SETS = ST > 2 ? ST : 1;
  float sa[SETS][TM], sw0[SETS], sw1[SETS], s0[TM], s1[TM];
  const auto load_scales = [&](int kb, int j) {
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(a.as + (size_t)kb * a.M), (short)0, a.M * 4, 0x00020000);
#pragma unroll
    for (int i = 0; i < TM; ++i) sa[j][i] = as_float(__builtin_amdgcn_raw_buffer_load_b32(r, first_token + 64 * i, 0, 0));
    sw0[j] = as_float(__builtin_amdgcn_raw_buffer_load_b32(sr0, 0, 4 * kb, 0));
    sw1[j] = G ? as_float(__builtin_amdgcn_raw_buffer_load_b32(sr1, 0, 4 * kb, 0)) : 0.f;
  };
  // The loads of a step stay between two barriers (both are fences to the compiler): the waits count them.
  constexpr int LOADS = LA + LW + (SETS > 1 ? TM + (G ? 2 : 1) : 0), PEND = (ST - 2) * LOADS;
  static_assert((ST - 1) * LOADS <= 63, "vmcnt counts at most 63");
  constexpr auto vmcnt = [](int n) { return (n & 15) | (7 << 4) | ((n >> 4) << 14); };      // and no LDS read pending
  const auto load_step = [&](int kb, int j) {
    if constexpr (SETS > 1) load_scales(kb, j);
    load(kb, as(j), ws(j));
  };
  f32x4 p[TM];                                       // block sums that are not yet in acc
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    p[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    s0[i] = s1[i] = 0.f;
  }
  const auto accumulate = [&](int t, int i) {
    const float s = G && t >= TN / 2 ? s1[i] : s0[i];
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[t][i][r] = __builtin_fmaf(p[i][r], s, acc[t][i][r]);
  };
  // The scales of a step take effect once the last block of the step before is in acc.
  const auto next_scales = [&](int i, int j) {
    s0[i] = sa[j % SETS][i] * sw0[j % SETS];
    s1[i] = sa[j % SETS][i] * sw1[j % SETS];
  };

  constexpr int RING = FP16 ? 2 : 4;                 // weight chunks in registers
  i32x4 w[RING];
  f16x8 h[2];                                        // fp16: the halves of a chunk; one multiplies while the other is converted
  const auto convert = [&](int c, int b, int e) {    // codes 2 e, 2 e + 1 of half b of chunk c
    const unsigned codes = (unsigned)w[c % RING][2 * b + (e >> 1)];
    const f16x2 v = e & 1 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, 1.0f, true)
                          : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, 1.0f, false);
    h[b][2 * e] = v[0];
    h[b][2 * e + 1] = v[1];
  };
  i32x8 x8[FP16 ? 1 : TM];
  Halves xh[FP16 ? TM : 1][2];
  const auto read_x = [&](const unsigned char* As, int i) {
    const i32x4 lo = achunk(As, i, 0), hi = achunk(As, i, 1);
    if constexpr (FP16) {
      xh[i][0] = halves(lo);
      xh[i][1] = halves(hi);
    } else {
      x8[i] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  };
  const int kl = kb1 - 1;                            // loads past the end read the last k block again, unused
  // One k block: its data lie in stage j, x and the first weight block are in registers.  Block t - 1 enters acc between
  // the MFMAs of block t, so that a wavefront's MFMAs and FMAs overlap (kept apart, the two wavefronts of a SIMD run in step
  // and wait for each other).  Before the last block everything of this step has been read, and the next one's data
  // have landed: one barrier says both, the stage just read receives the step ST further on, and the next step's operands
  // are read while this one finishes.
  const auto step = [&](auto stage, int kb_next, int kb_load) {
    constexpr int J = decltype(stage)::value;
    unsigned char* const Ws = ws(J);
    const unsigned char *const An = as((J + 1) % ST), *const Wn = ws((J + 1) % ST);
#pragma unroll
    for (int t = 0; t < TN; ++t) {
      const bool last = t == TN - 1;
      if (last) {
        __builtin_amdgcn_s_waitcnt(vmcnt(PEND));
        barrier();
        if constexpr (SETS == 1) load_scales(kb_next, 0);
      }
      if constexpr (FP16) {
#pragma unroll
        for (int e = 0; e < 4 * TM; ++e) {           // (half of the block, half of the chunk, token block)
          const int j = e / (2 * TM), b = e / TM % 2, i = e % TM;
          __builtin_amdgcn_sched_barrier(0);
          if (e < TM) accumulate((t + TN - 1) % TN, i);
          if (e < TM && t == 0) next_scales(i, J);
          p[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(h[b], xh[i][j].v[b], e < TM ? f32x4{0.f, 0.f, 0.f, 0.f} : p[i], 0, 0, 0);
          const int c = 2 * t + j;
          if (b == 1 && i == 0) w[c % RING] = last ? wchunk(Wn, j) : wchunk(Ws, c + 2);
#pragma unroll
          for (int f = 0; f < 4 / TM; ++f) convert(c + b, 1 - b, i * (4 / TM) + f);
          if (last && e == 2 * TM - 1) load_step(kb_load, J);
        }
        if (last) {
#pragma unroll
          for (int i = 0; i < TM; ++i) read_x(An, i);
        }
      } else {
        const i32x8 w8 = __builtin_shufflevector(w[2 * t % RING], w[(2 * t + 1) % RING], 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          __builtin_amdgcn_sched_barrier(0);
          accumulate((t + TN - 1) % TN, i);
          if (t == 0) next_scales(i, J);
          p[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w8, x8[i], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
          if (i < 2) w[(2 * t + 2 + i) % RING] = last ? wchunk(Wn, i) : wchunk(Ws, 2 * t + 2 + i);
          if (last) read_x(An, i);
          if (last && i == TM - 1) load_step(kb_load, J);
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  if constexpr (SETS == 1) load_scales(kb0, 0);
#pragma unroll
  for (int j = 0; j < ST; ++j) {
    asm volatile("" ::: "memory");
    load_step(min(kb0 + j, kl), j);
  }
  __builtin_amdgcn_s_waitcnt(vmcnt((ST - 1) * LOADS));
  barrier();
#pragma unroll
  for (int i = 0; i < TM; ++i) read_x(A0, i);
#pragma unroll
  for (int c = 0; c < 2; ++c) w[c] = wchunk(W0, c);
  if constexpr (FP16) {
#pragma unroll
    for (int e = 0; e < 4; ++e) convert(0, 0, e);
  }
  int kb = kb0;
  const auto next = [&](auto stage) {
    step(stage, min(kb + 1, kl), min(kb + ST, kl));
    ++kb;
  };
  constexpr std::integral_constant<int, 0> S0{};
  constexpr std::integral_constant<int, 1> S1{};
  constexpr std::integral_constant<int, (ST > 2 ? 2 : 0)> S2{};
  constexpr std::integral_constant<int, (ST > 3 ? 3 : 0)> S3{};
  while (kb + ST <= kb1) {
    next(S0);
    next(S1);
    if constexpr (ST > 2) next(S2);
    if constexpr (ST > 3) next(S3);
  }
  if (kb < kb1) {
    next(S0);
    if constexpr (ST > 2)
      if (kb < kb1) {
        next(S1);
        if constexpr (ST > 3)
          if (kb < kb1) next(S2);
      }
  }
#pragma unroll
  for (int i = 0; i < TM; ++i) accumulate(TN - 1, i);
  __builtin_amdgcn_s_waitcnt(0);                     // no load is still writing LDS
  __syncthreads();                                   // and no wavefront reads it: what follows uses it otherwise

  const TileEnd<WN, NW, GATE, Q, OUT == OUT_F32, TN, TM> end{a, A0, A1, (wave < 4 ? W0 : W1) + (wave & 3) * 8192, tn, m0, wm * TM, wn, c0};
  if (splits == 1) {
    end.whole(acc);
  } else {
    if constexpr (BM == 64) {
      if (splits < 4) return end.shared_at_once(acc, tile - a.whole, splits, split);
    }
    end.shared_in_parts(acc, tile - a.whole, splits, split);
  }
}

template <int WM, int TM, int ST>
void launch_tile(const W8Plan& pl, const W8Args& a, hipStream_t s) {
  const dim3 grid(pl.grid), block(64 * kW8Waves);
  const auto gate = [&](auto g) {
    constexpr int GATE = decltype(g)::value;
    if (a.out_dtype == QGEMM_DT_F32) tiles_kernel<WM, TM, ST, GATE, OUT_F32, true><<<grid, block, 0, s>>>(a);
    else if (a.out_dtype != QGEMM_DT_FP8_E4M3)
      pl.fp16 ? tiles_kernel<WM, TM, ST, GATE, OUT_16, true><<<grid, block, 0, s>>>(a)
              : tiles_kernel<WM, TM, ST, GATE, OUT_16, false><<<grid, block, 0, s>>>(a);
    else if constexpr (GATE != QGEMM_GATE_NONE) tiles_kernel<WM, TM, ST, GATE, OUT_E4M3, true><<<grid, block, 0, s>>>(a);
  };
  switch (a.gate) {
    case QGEMM_GATE_NONE: gate(std::integral_constant<int, QGEMM_GATE_NONE>{}); break;
    case QGEMM_GATE_SILU: gate(std::integral_constant<int, QGEMM_GATE_SILU>{}); break;
    default: gate(std::integral_constant<int, QGEMM_GATE_GELU_TANH>{}); break;
  }
}

}  // namespace

hipError_t launch_tiles(const W8Plan& pl, const W8Args& a, hipStream_t stream) {
  switch (pl.tile) {
    case 64: launch_tile<2, 2, 4>(pl, a, stream); break;
    case 128: launch_tile<2, 4, 3>(pl, a, stream); break;
    default: launch_tile<4, 4, 2>(pl, a, stream); break;
  }
  return hipGetLastError();
}

}  // namespace w8
}  // namespace qgemm
