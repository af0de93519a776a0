// The tiles kernel of the 8-bit products: any number of tokens.
//
//   p_r[m] = sum_b as[b][m] ws[r / 128][b] (sum_{k in block b} a[m][k] w[r][k])
//
// Workgroup = eight wavefronts, WM along the tokens and WN along the weight rows; each owns TM x TN MFMA tiles of
// 32 tokens x 32 weight rows, the workgroup 32 WM TM tokens x 256 weight rows.  With a gate the first half of a
// wavefront's weight tiles are rows of the gate's projection and the second half the same rows of the other, so that
// both factors of an output meet in one lane.
//
// One step is one k block of 128: tokens and weights go from memory straight into LDS (buffer loads with the LDS
// destination), one stage ahead of the step that computes.  A load writes its 64 lanes' 16 bytes side by side, eight
// rows of 128 bytes; so that the operand reads (32 rows, one chunk each) spread over the banks, chunk c of row r is
// stored at c ^ (r & 7), by the choice of the address that each lane loads.  Rows past the last read as zero.
//
// The weights are the first MFMA operand and the tokens the second: lane l of the result holds token l & 31, so both
// scales of a block are one factor per lane and MFMA tile, and a step costs one fp32 FMA per 128 products beside the
// MFMA (16 of 64 lanes' issue cycles beside 128 MFMA cycles for a 32 x 32 tile).
#include <type_traits>

#include "qgemm_w8a8_fixup.h"

namespace qgemm {
namespace w8 {
namespace {

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

__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int WM, int TM, int GATE, bool Q, bool FP16>
__global__ __launch_bounds__(64 * kW8Waves) void tiles_kernel(W8Args a) {
  constexpr int NW = kW8Waves, WN = NW / WM, TN = kTileRows / (32 * WN), BM = 32 * WM * TM;
  constexpr bool G = GATE != QGEMM_GATE_NONE;
  constexpr int COLS = G ? kTileRows / 2 : kTileRows;          // output columns of a tile
  constexpr int LA = BM / (8 * NW), LW = kTileRows / (8 * NW); // loads of a wavefront per step
  static_assert(!G || TN % 2 == 0, "both projections' rows lie in one wavefront");
  __shared__ __attribute__((aligned(1024))) unsigned char A0[BM * kBlock], A1[BM * kBlock];
  __shared__ __attribute__((aligned(1024))) unsigned char W0[kTileRows * kBlock], W1[kTileRows * kBlock];
  __shared__ int s_last;
  const int lane = threadIdx.x & 63, half = lane >> 5, col = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int tiles = gridDim.x / a.splits, split = blockIdx.x / tiles, tile = blockIdx.x - split * tiles;
  int tm, tn;
  tile_of(tile, tiles, a.tiles_n, tm, tn);
  const int m0 = tm * BM, n0 = tn * COLS;
  const int kb0 = split * a.kb_per_split, kb1 = min(a.KB, kb0 + a.kb_per_split);

  // ---- loads into LDS: 1 KiB each, eight rows
  const int drow = lane >> 3, dchunk = (lane & 7) ^ drow;
  const __amdgpu_buffer_rsrc_t ar = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(a.a + (size_t)m0 * a.K), (short)0, min(a.M - m0, BM) * a.K, 0x00020000);
  const int wrows = min(a.N - n0, COLS);
  const __amdgpu_buffer_rsrc_t wr0 = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(a.w + (size_t)n0 * a.K), (short)0, wrows * a.K, 0x00020000);
  const __amdgpu_buffer_rsrc_t wr1 = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(a.w + (size_t)(G ? a.N + n0 : n0) * a.K), (short)0, wrows * a.K, 0x00020000);
  const int lane_off = drow * a.K + 16 * dchunk;
  const auto load = [&](int kb, unsigned char* As, unsigned char* Ws) {
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const int r = 8 * (NW * i + wave);             // first row of the load
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ar, (lds_ptr_t)(As + r * kBlock), 16, lane_off + r * a.K, kb * kBlock, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < LW; ++i) {
      const int r = 8 * (NW * i + wave);
      if constexpr (G) {
        // row r of the tile: wavefront column r / (32 TN), its tile t; tiles past the half are the other projection's
        const int t = (r >> 5) % TN, src = (r >> 5) / TN * (16 * TN) + t % (TN / 2) * 32 + (r & 31);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(t < TN / 2 ? wr0 : wr1, (lds_ptr_t)(Ws + r * kBlock), 16,
                                                 lane_off + src * a.K, kb * kBlock, 0, 0);
      } else {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(wr0, (lds_ptr_t)(Ws + r * kBlock), 16, lane_off + r * a.K, kb * kBlock, 0, 0);
      }
    }
  };

  // ---- scales: one per token tile and lane; of the weights one per projection (a wavefront's rows of one
  // projection lie in one block of 128)
  const float* sap[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) sap[i] = a.as + min(m0 + 32 * (wm * TM + i) + col, a.M - 1);
  const int c0 = n0 + wn * (G ? 16 * TN : 32 * TN);  // the wavefront's first output column
  const int rb = min(c0 / kBlock, a.row_blocks - 1);
  const float* swp0 = a.ws + (size_t)rb * a.KB;
  const float* swp1 = a.ws + (size_t)((G ? a.row_blocks : 0) + rb) * a.KB;

  f32x16 acc[TN][TM];
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int i = 0; i < TM; ++i) acc[j][i] = f32x16{};

  // chunk 4 j + 2 half + b of a row: the operand of K half j
  int coff[2][2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int b = 0; b < 2; ++b) coff[j][b] = col * kBlock + 16 * ((4 * j + 2 * half + b) ^ (col & 7));
  const auto operand = [&](const unsigned char* p, int j) {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(p + coff[j][0]), hi = *reinterpret_cast<const i32x4*>(p + coff[j][1]);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  const auto accumulate = [&](int t, int i, f32x16 p, float s) {
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[t][i][r] = __builtin_fmaf(p[r], s, acc[t][i][r]);
  };
  // chunk 2 j + half of a row as two fp16 operands of 16 k
  int hoff[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) hoff[j] = col * kBlock + 16 * ((2 * j + half) ^ (col & 7));
  const auto compute16 = [&](const unsigned char* As, const unsigned char* Ws, const float (&sa)[TM], float sw0, float sw1) {
    Halves x[TM][4];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[i][j] = halves(*reinterpret_cast<const i32x4*>(As + 32 * (wm * TM + i) * kBlock + hoff[j]));
#pragma unroll
    for (int t = 0; t < TN; ++t) {
      f32x16 p[TM];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const Halves w = halves(*reinterpret_cast<const i32x4*>(Ws + 32 * (wn * TN + t) * kBlock + hoff[j]));
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < TM; ++i)
            p[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(w.v[b], x[i][j].v[b], j + b ? p[i] : f32x16{}, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < TM; ++i) accumulate(t, i, p[i], sa[i] * (G && t >= TN / 2 ? sw1 : sw0));
    }
  };
  const auto compute8 = [&](const unsigned char* As, const unsigned char* Ws, const float (&sa)[TM], float sw0, float sw1) {
    i32x8 x[TM][2];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) x[i][j] = operand(As + 32 * (wm * TM + i) * kBlock, j);
#pragma unroll
    for (int t = 0; t < TN; ++t) {
      const unsigned char* row = Ws + 32 * (wn * TN + t) * kBlock;
      const i32x8 w0 = operand(row, 0), w1 = operand(row, 1);
      const float sw = G && t >= TN / 2 ? sw1 : sw0;
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        f32x16 p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w0, x[i][0], f32x16{}, 0, 0, 0, 0, 0, 0);
        p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w1, x[i][1], p, 0, 0, 0, 0, 0, 0);
        accumulate(t, i, p, sa[i] * sw);
      }
    }
  };
  const auto compute = [&](const unsigned char* As, const unsigned char* Ws, const float (&sa)[TM], float sw0, float sw1) {
    if constexpr (FP16) compute16(As, Ws, sa, sw0, sw1);
    else compute8(As, Ws, sa, sw0, sw1);
  };

  float sa[2][TM], sw0[2], sw1[2];
  const auto load_scales = [&](int kb, int b) {
#pragma unroll
    for (int i = 0; i < TM; ++i) sa[b][i] = sap[i][(size_t)kb * a.M];
    sw0[b] = swp0[kb];
    sw1[b] = G ? swp1[kb] : 0.f;
  };
  load_scales(kb0, 0);
  load(kb0, A0, W0);
  for (int kb = kb0; kb < kb1; kb += 2) {
    // the step's loads have landed for every wavefront, and every wavefront is done reading the other stage
    __builtin_amdgcn_s_waitcnt(0);
    barrier();
    if (kb + 1 < kb1) {
      load_scales(kb + 1, 1);
      load(kb + 1, A1, W1);
    }
    compute(A0, W0, sa[0], sw0[0], sw1[0]);
    if (kb + 1 >= kb1) break;
    __builtin_amdgcn_s_waitcnt(0);
    barrier();
    if (kb + 2 < kb1) {
      load_scales(kb + 2, 0);
      load(kb + 2, A0, W0);
    }
    compute(A1, W1, sa[1], sw0[1], sw1[1]);
  }

  // ---- splits along K: partial tiles, summed in order by the workgroup that comes last
  if (a.splits > 1) {
    constexpr int SLOT = BM * kTileRows * 4;
    const __amdgpu_buffer_rsrc_t part = __builtin_amdgcn_make_buffer_rsrc(
        a.partials + (size_t)tile * a.splits * (SLOT / 4), (short)0, a.splits * SLOT, 0x00020000);
    const int at = 16 * threadIdx.x;                 // fragment f of a slot: 16 bytes per thread
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          store_partial(part, split * SLOT + ((t * TM + i) * 4 + q) * (64 * NW * 16) + at,
                        f32x4{acc[t][i][4 * q], acc[t][i][4 * q + 1], acc[t][i][4 * q + 2], acc[t][i][4 * q + 3]});
    if (!last_arrival(a.tickets + tile, a.splits, &s_last)) return;
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
      for (int i = 0; i < TM; ++i) acc[t][i] = f32x16{};
    for (int s = 0; s < a.splits; ++s)
#pragma unroll
      for (int t = 0; t < TN; ++t)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x4 v = load_partial(part, s * SLOT + ((t * TM + i) * 4 + q) * (64 * NW * 16) + at);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[t][i][4 * q + r] += v[r];
          }
  }

  // ---- outputs: lane l holds token l & 31 and weight rows 8 q + 4 (l >> 5) .. + 3 of each MFMA tile
  constexpr int OT = G ? TN / 2 : TN;
  const auto four = [&](int t, int i, int q) {
    const f32x4 g = {acc[t][i][4 * q], acc[t][i][4 * q + 1], acc[t][i][4 * q + 2], acc[t][i][4 * q + 3]};
    if constexpr (!G) return g;
    const f32x16& o = acc[t + TN - OT][i];
    return gated<GATE>(g, f32x4{o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]});
  };
  if constexpr (!Q) {
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int m = m0 + 32 * (wm * TM + i) + col;
      if (m >= a.M) continue;
#pragma unroll
      for (int t = 0; t < OT; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = c0 + 32 * t + 8 * q + 4 * half;
          if (n < a.N) store4(a, (size_t)m * a.N + n, four(t, i, q));
        }
    }
  } else {
    __shared__ unsigned top[WN][BM];                 // largest magnitude of a token in each wavefront's columns
    f32x4 y[TM][OT][4];
    unsigned m[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      m[i] = 0;
#pragma unroll
      for (int t = 0; t < OT; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          y[i][t][q] = four(t, i, q);
#pragma unroll
          for (int r = 0; r < 4; ++r) m[i] = max(m[i], magnitude(y[i][t][q][r]));
        }
      m[i] = max(m[i], (unsigned)__shfl_xor((int)m[i], 32));
      if (half == 0) top[wn][32 * (wm * TM + i) + col] = m[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int w = 0; w < WN; ++w) m[i] = max(m[i], top[w][32 * (wm * TM + i) + col]);
      const BlockScale b = block_scale(m[i], 1.0f);
      const int token = m0 + 32 * (wm * TM + i) + col;
      if (token >= a.M) continue;
      if (wn == 0 && half == 0) a.os[(size_t)tn * a.M + token] = b.scale;
#pragma unroll
      for (int t = 0; t < OT; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4 v = y[i][t][q];
          *reinterpret_cast<unsigned*>(static_cast<uint8_t*>(a.out) + (size_t)token * a.N + c0 + 32 * t + 8 * q + 4 * half) =
              codes4(v[0] * b.to_code, v[1] * b.to_code, v[2] * b.to_code, v[3] * b.to_code);
        }
    }
  }
}

template <int WM, int TM>
void launch_tile(const W8Plan& pl, const W8Args& a, hipStream_t s) {
  const dim3 grid(pl.grid), block(64 * kW8Waves);
  const auto gate = [&](auto g) {
    constexpr int GATE = decltype(g)::value;
    if (a.out_dtype == QGEMM_DT_F32) tiles_kernel<WM, TM, GATE, false, true><<<grid, block, 0, s>>>(a);
    else if (a.out_dtype != QGEMM_DT_FP8_E4M3) tiles_kernel<WM, TM, GATE, false, false><<<grid, block, 0, s>>>(a);
    else if constexpr (GATE != QGEMM_GATE_NONE) tiles_kernel<WM, TM, GATE, true, true><<<grid, block, 0, s>>>(a);
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
    case 64: launch_tile<2, 1>(pl, a, stream); break;
    case 128: launch_tile<4, 1>(pl, a, stream); break;
    default: launch_tile<4, 2>(pl, a, stream); break;
  }
  return hipGetLastError();
}

}  // namespace w8
}  // namespace qgemm
