// Host side of the 8-bit operators: descriptor validation, the weights' quantizer and launch planning.
// Nothing in this file touches the GPU.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "qgemm_w8a8_internal.h"

namespace qgemm {

static_assert(sizeof(qgemm_add_norm_t) == 32, "qgemm_add_norm_t layout is part of the ABI");
static_assert(sizeof(qgemm_w8a8_t) == 48, "qgemm_w8a8_t layout is part of the ABI");

static const int kCUs = 256;
static const int kMaxSplits = 32;
static const int64_t kMaxSize = int64_t(1) << 24;
static const int64_t kMaxK = int64_t(1) << 22;

static qgemm_status_t check_dtype(const char* what, int dtype) {
  if (dtype < QGEMM_DT_F16 || dtype > QGEMM_DT_NF4)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "%s value %d is not a qgemm_dtype_t", what, dtype);
  return QGEMM_OK;
}

qgemm_status_t validate_add_norm(const qgemm_add_norm_t* p) {
  if (!p) return fail(QGEMM_ERR_INVALID_ARGUMENT, "problem is NULL");
  qgemm_status_t st = check_dtype("dtype", p->dtype);
  if (st != QGEMM_OK || (st = check_dtype("out_dtype", p->out_dtype)) != QGEMM_OK) return st;
  if (p->dtype != QGEMM_DT_F16 && p->dtype != QGEMM_DT_BF16)
    return fail(QGEMM_ERR_UNSUPPORTED, "dtype must be F16 or BF16, got %d", p->dtype);
  if (p->out_dtype != p->dtype && p->out_dtype != QGEMM_DT_FP8_E4M3)
    return fail(QGEMM_ERR_UNSUPPORTED, "out_dtype must be dtype (%d) or FP8_E4M3, got %d", p->dtype, p->out_dtype);
  if (p->tokens < 0 || p->tokens > kMaxSize)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "tokens must be in [0, %lld], got %lld", (long long)kMaxSize,
                (long long)p->tokens);
  if (p->dim < 8 || p->dim > 32768 || p->dim % 8)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "dim must be a multiple of 8 in [8, 32768], got %d", p->dim);
  if (p->out_dtype == QGEMM_DT_FP8_E4M3 && p->dim % kBlock)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "dim must be a multiple of %d for FP8_E4M3, got %d", kBlock, p->dim);
  if (p->norm != 0 && p->norm != 1) return fail(QGEMM_ERR_INVALID_ARGUMENT, "norm must be 0 or 1, got %d", p->norm);
  if (p->norm && !(p->eps >= 0.0f && std::isfinite(p->eps)))
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0, got %g", (double)p->eps);
  if (p->reserved != 0) return fail(QGEMM_ERR_INVALID_ARGUMENT, "reserved must be 0, got %d", p->reserved);
  return QGEMM_OK;
}

qgemm_status_t validate_w8a8(const qgemm_w8a8_t* p) {
  if (!p) return fail(QGEMM_ERR_INVALID_ARGUMENT, "problem is NULL");
  if (p->M < 0 || p->M > kMaxSize)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "M must be in [0, %lld], got %lld", (long long)kMaxSize, (long long)p->M);
  if (p->N < 16 || p->N > kMaxSize || p->N % 16)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "N must be a multiple of 16 in [16, %lld], got %lld", (long long)kMaxSize,
                (long long)p->N);
  if (p->K < kBlock || p->K > kMaxK || p->K % kBlock)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "K must be a multiple of %d in [%d, %lld], got %lld", kBlock, kBlock,
                (long long)kMaxK, (long long)p->K);
  if (p->gate < QGEMM_GATE_NONE || p->gate > QGEMM_GATE_GELU_TANH)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "gate must be 0, 1 or 2, got %d", p->gate);
  qgemm_status_t st = check_dtype("out_dtype", p->out_dtype);
  if (st != QGEMM_OK) return st;
  if (p->out_dtype == QGEMM_DT_FP8_E4M3) {
    if (p->gate == QGEMM_GATE_NONE)
      return fail(QGEMM_ERR_UNSUPPORTED, "out_dtype FP8_E4M3 needs a gate (without one: F16, BF16 or F32)");
    if (p->N % kBlock)
      return fail(QGEMM_ERR_INVALID_ARGUMENT, "N must be a multiple of %d for out_dtype FP8_E4M3, got %lld", kBlock,
                  (long long)p->N);
  } else if (p->out_dtype > QGEMM_DT_F32) {
    return fail(QGEMM_ERR_UNSUPPORTED, "out_dtype must be F16, BF16, F32 or (with a gate) FP8_E4M3, got %d", p->out_dtype);
  }
  if (p->kernel_hint < QGEMM_W8A8_AUTO || p->kernel_hint > QGEMM_W8A8_TILES)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "kernel_hint must be 0, 1 or 2, got %d", p->kernel_hint);
  if (p->kernel_hint == QGEMM_W8A8_ROWS && p->M > kRowsMaxM)
    return fail(QGEMM_ERR_UNSUPPORTED, "the rows kernel takes M <= %d, got %lld", kRowsMaxM, (long long)p->M);
  if (p->split_hint < 0 || p->split_hint > kMaxSplits)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "split_hint must be in [0, %d], got %d", kMaxSplits, p->split_hint);
  if (p->tile_hint != 0 && p->tile_hint != 64 && p->tile_hint != 128 && p->tile_hint != 256)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "tile_hint must be 0, 64, 128 or 256, got %d", p->tile_hint);
  if (p->sums != QGEMM_W8A8_SUMS_AUTO && p->sums != QGEMM_W8A8_SUMS_WHOLE)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "sums must be 0 or 1 (other values are reserved), got %d", p->sums);
  return QGEMM_OK;
}

// A launch holds less than 2^32 work-items.
static bool launchable(int64_t workgroups) { return workgroups <= 0xffffffffLL / (64 * kW8Waves); }

// `whole` workgroups on their own and `groups` sets of members_n * splits.
static qgemm_status_t finish_plan(W8Plan* pl, int64_t whole, int64_t groups, int members_n, int splits, int KB,
                                  size_t slot_bytes) {
  pl->kb_per_split = (KB + splits - 1) / splits;
  pl->splits = (KB + pl->kb_per_split - 1) / pl->kb_per_split;       // none of them empty
  pl->groups = groups;
  pl->members = members_n * pl->splits;
  const int64_t sets = groups * pl->members, workgroups = whole + sets;
  if (!launchable(workgroups))
    return fail(QGEMM_ERR_UNSUPPORTED, "the problem needs %lld workgroups, more than one launch allows", (long long)workgroups);
  pl->grid = (unsigned)workgroups;
  pl->ws_bytes = pl->members > 1 ? (size_t)kW8Tickets * 4 + (size_t)sets * slot_bytes : 0;
  return QGEMM_OK;
}

// The rows kernel's workgroups along K: as many as give every compute unit one, of four k blocks a wavefront at least, from 17 tokens on
// two: sharing an output takes three dependent trips to memory (unsplit, by two and by four, weights from memory: 4 x 1024 x 2048 3.7, 4.8,
// 6.0 us; 16 x 512 x 4096 5.2, 5.5, 5.6; 4 x 1024 x 8192 6.0, 6.2, 6.9; 16 x 1024 x 8192 7.7, 7.0, 7.2; 40 x 1024 x 8192 10.9, 8.7, 8.0;
// 16 x 1024 x 28672 20.7, 13.6, 10.7).
static int rows_splits(int64_t M, int64_t columns, int KB) {
  const int least = (M <= 16 ? 4 : 2) * kW8Waves;
  return (int)std::min<int64_t>({std::max<int64_t>(1, kCUs / columns), std::max(1, KB / least), kMaxSplits});
}

static qgemm_status_t make_rows_plan(const qgemm_w8a8_t* p, W8Plan* pl) {
  const bool gated = p->gate != QGEMM_GATE_NONE, quantized = p->out_dtype == QGEMM_DT_FP8_E4M3;
  const int KB = (int)(p->K / kBlock);
  const int64_t M = std::max<int64_t>(p->M, 1);
  pl->kind = W8_ROWS;
  const int members = quantized ? kBlock / 16 : 1;
  const int64_t columns = p->N / 16, groups = columns / members;   // workgroups without a split
  int splits = p->split_hint ? std::min(p->split_hint, KB) : rows_splits(M, columns, KB);
  if (groups > kW8Tickets) splits = 1;
  // A wavefront takes its k blocks in pairs; four wavefronts where eight would leave a tenth or more of the pairs' places
  // empty (10240 x 5120, 40 k blocks: one token 12.7 us with eight, 12.2 with four, 16 tokens 16.1 and 14.9; 4096 x 11008, 86: one token
  // 12.7 and 13.2, 16 tokens 14.1 and 13.6), and where the LDS of eight leaves room for one workgroup a compute unit and more are
  // waiting: with a gate (11008 x 4096: 22.8 and 20.0) and from 17 tokens on (17 x 8192 x 4096: 11.2 and 9.9; 17 x 4096 x 4096, one
  // each, 6.05 and 6.05), above 32 always.
  const int per = (KB + splits - 1) / splits;
  const auto places = [&](int waves) { return (per + 2 * waves - 1) / (2 * waves) * 2 * waves; };
  const bool crowded = M > 32 || (M > 16 && columns * splits > kCUs);
  pl->waves = gated || crowded || places(4) * 10 <= places(8) * 9 ? 4 : 8;
  return finish_plan(pl, 0, groups, members, splits, KB, (size_t)(gated ? 2 : 1) * 1024 * ((M + 15) / 16));
}

// Microseconds that a workgroup of the tiles kernel takes for a k block and besides, while every compute unit has one
// (e4m3 and fp16 operands); fitted to one and two rounds of 256 workgroups of each tile at K from 2048 to 11008.
struct TileCost { double step[2], fixed; };
static TileCost tile_cost(int tile) {
  return tile == 256 ? TileCost{{1.57, 2.95}, 9.0} : tile == 128 ? TileCost{{0.93, 1.60}, 5.5} : TileCost{{0.60, 1.0}, 4.5};
}
// That sharing `tiles` tiles between `splits` workgroups each costs: tickets, and the partial tiles' way to memory and back.
static double share_cost(int tile, int64_t tiles, int splits) {
  return splits > 1 ? 3.0 + 0.3 * splits + (double)(tiles * splits) * (tile * kTileRows * 4) * 2 / 10.0e6 : 0.0;
}

// Microseconds of the rows kernel for more than 16 tokens: what a compute unit takes for 16 weight rows' k block, with a gate for
// those of either projection, times its share of them, half of the way from the average to the unit with the most workgroups (they
// overlap).  Fitted to 96 times at 1024 x 28672 to 28672 x 8192, 17 to 64 tokens, with weights from memory: within 7% on average, 28% at
// most (2048 x 8192); the faster kernel is missed by more than 5% on 3 of the 96, by 8% at most.
static double rows_cost(const qgemm_w8a8_t* p) {
  const int KB = (int)(p->K / kBlock), splits = rows_splits(p->M, p->N / 16, KB);
  const int64_t workgroups = p->N / 16 * splits, rounds = (workgroups + kCUs - 1) / kCUs;
  const double blocks = 0.5 * ((double)workgroups / kCUs + (double)rounds) * KB / splits;
  const double one = 0.091 + 0.0018 * (double)p->M;
  if (p->gate == QGEMM_GATE_NONE) return 2.0 + one * blocks;
  if (p->out_dtype != QGEMM_DT_FP8_E4M3) return 2.4 + 1.57 * one * blocks;
  return 6.4 + (p->M > 48 ? 2.16 : 1.65) * one * blocks;            // above 48 tokens a compute unit holds one workgroup, not two
}

qgemm_status_t make_w8a8_plan(const qgemm_w8a8_t* p, W8Plan* pl) {
  *pl = W8Plan{};
  if (p->kernel_hint == QGEMM_W8A8_ROWS || (p->kernel_hint == QGEMM_W8A8_AUTO && p->M <= 16)) return make_rows_plan(p, pl);
  const bool gated = p->gate != QGEMM_GATE_NONE, quantized = p->out_dtype == QGEMM_DT_FP8_E4M3;
  const int KB = (int)(p->K / kBlock);
  const int64_t M = std::max<int64_t>(p->M, 1);
  pl->kind = W8_TILES;
  const int columns = gated ? kTileRows / 2 : kTileRows;
  pl->tiles_n = (int)((p->N + columns - 1) / columns);
  pl->fp16 = quantized || p->out_dtype == QGEMM_DT_F32 || p->sums == QGEMM_W8A8_SUMS_WHOLE;
  // The tiles of whole rounds over the compute units run on their own; those of the last round are split along K as far
  // as that shortens it (all tiles, where there are fewer than compute units).  A split hint takes no part in the choice of tile
  // and kernel, on either side: it splits the launch that is taken without it.
  double best = 0.0;
  int best_splits = 1;
  for (int tile : {64, 128, 256}) {
    if (p->tile_hint && p->tile_hint != tile) continue;
    const int64_t tiles = (M + tile - 1) / tile * pl->tiles_n, tail = tiles % kCUs, rounds = tiles / kCUs;
    const TileCost c = tile_cost(tile);
    for (int s = 1; s <= std::min(kMaxSplits, KB); ++s) {
      const int kb = (KB + s - 1) / s;
      if (s > 1 && (!tail || (KB + kb - 1) / kb != s)) continue;
      const double step = c.step[pl->fp16], tail_rounds = (double)((tail * s + kCUs - 1) / kCUs);
      const double us = (double)rounds * (KB * step + c.fixed) + tail_rounds * (kb * step + c.fixed) + share_cost(tile, tail, s);
      if (pl->tile == 0 || us < best) {
        best = us;
        pl->tile = tile;
        best_splits = s;
      }
    }
  }
  // Up to 64 tokens either kernel may be the faster: the rows kernel reads the tokens again for every 16 weight rows, the tiles
  // kernel has few tiles and joins their splits (4096 x 4096, 17 tokens: 6.1 and 12.2 us, 64 tokens 8.1 and 12.8;
  // 10240 x 5120: 16.2 and 19.3, 28.0 and 20.5; 11008 x 4096 gated to e4m3: 27.0 and 26.5, 46.1 and 27.3; 5632 x 2048, 40 tokens 14.5 and 17.0).
  if (p->kernel_hint == QGEMM_W8A8_AUTO && !p->tile_hint && p->M <= kRowsMaxM) {
    // With so few tokens the weights come from memory: split tiles take about 3 us more than the fit, and no less than that reading.
    const double memory = 3.0 + (double)(p->N * p->K) * (gated ? 2 : 1) / 3.7e6;
    if (rows_cost(p) < std::max(best + (best_splits > 1 ? 3.0 : 0.0), memory)) {
      *pl = W8Plan{};
      return make_rows_plan(p, pl);
    }
  }
  const int64_t tiles = (M + pl->tile - 1) / pl->tile * pl->tiles_n;
  if (!launchable(tiles))
    return fail(QGEMM_ERR_UNSUPPORTED, "the problem needs %lld workgroups, more than one launch allows", (long long)tiles);
  pl->tiles = (int)tiles;
  int splits = p->split_hint ? std::min(p->split_hint, KB) : best_splits;
  int64_t whole = splits == 1 ? tiles : p->split_hint ? 0 : tiles - tiles % kCUs;
  if (tiles - whole > kW8Tickets / kTileParts) whole = tiles;        // a hint, on very many tiles
  if (whole == tiles) splits = 1;
  pl->whole = (int)whole;
  return finish_plan(pl, whole, tiles - whole, 1, splits, KB, (size_t)pl->tile * kTileRows * 4);
}

// RNE to e4m3, |v| <= 448.
static uint8_t e4m3_code(double v) {
  const uint8_t sign = std::signbit(v) ? 0x80 : 0;
  const double a = std::fabs(v);
  int e;
  std::frexp(a, &e);
  e = std::max(e - 1, -6);                                           // exponent of the leading bit
  const int units = (int)std::nearbyint(std::ldexp(a, 3 - e));       // of 2^(e - 3): 0 .. 16
  if (units == 0) return 0;
  // a sum: 16 units of one binade carry into the exponent field, fewer than 8 (e is -6) are a subnormal
  return (uint8_t)(sign | (((e + 7) << 3) + units - 8));
}

}  // namespace qgemm

using namespace qgemm;

extern "C" {

qgemm_status_t qgemm_w8a8_quantize(const qgemm_w8a8_t* p, const float* w, uint8_t* codes, float* scales) {
  clear_error();
  const qgemm_status_t st = validate_w8a8(p);
  if (st != QGEMM_OK) return st;
  if (!w || !codes || !scales) return fail(QGEMM_ERR_INVALID_ARGUMENT, "w, codes and scales must not be NULL");
  const int64_t KB = p->K / kBlock, row_blocks = (p->N + kBlock - 1) / kBlock;
  for (int part = 0; part < (p->gate != QGEMM_GATE_NONE ? 2 : 1); ++part)
    for (int64_t rb = 0; rb < row_blocks; ++rb) {
      const int64_t first = part * p->N + rb * kBlock, rows = std::min<int64_t>(kBlock, p->N - rb * kBlock);
      for (int64_t kb = 0; kb < KB; ++kb) {
        float amax = 0.0f;
        for (int64_t r = first; r < first + rows; ++r)
          for (int64_t k = kb * kBlock; k < (kb + 1) * kBlock; ++k) {
            const float v = std::fabs(w[r * p->K + k]);
            if (!std::isfinite(v)) return fail(QGEMM_ERR_INVALID_ARGUMENT, "w[%lld] is not finite", (long long)(r * p->K + k));
            amax = std::max(amax, v);
          }
        const float scale = amax / 448.0f;
        scales[(part * row_blocks + rb) * KB + kb] = scale;
        for (int64_t r = first; r < first + rows; ++r)
          for (int64_t k = kb * kBlock; k < (kb + 1) * kBlock; ++k) {
            const double x = scale == 0.0f ? 0.0 : (double)w[r * p->K + k] / (double)scale;
            codes[r * p->K + k] = e4m3_code(std::min(std::max(x, -448.0), 448.0));
          }
      }
    }
  return QGEMM_OK;
}

qgemm_status_t qgemm_w8a8_workspace_bytes(const qgemm_w8a8_t* p, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(QGEMM_ERR_INVALID_ARGUMENT, "bytes is NULL");
  qgemm_status_t st = validate_w8a8(p);
  if (st != QGEMM_OK) return st;
  W8Plan pl;
  st = make_w8a8_plan(p, &pl);
  if (st != QGEMM_OK) return st;
  *bytes = p->M ? pl.ws_bytes : 0;
  return QGEMM_OK;
}

qgemm_status_t qgemm_w8a8_describe(const qgemm_w8a8_t* p, char* buf, size_t len) {
  clear_error();
  if (!buf || !len) return fail(QGEMM_ERR_INVALID_ARGUMENT, "buf is NULL or len is 0");
  qgemm_status_t st = validate_w8a8(p);
  if (st != QGEMM_OK) return st;
  W8Plan pl;
  st = make_w8a8_plan(p, &pl);
  if (st != QGEMM_OK) return st;
  const int n = p->M == 0 ? std::snprintf(buf, len, "empty")
                : pl.kind == W8_ROWS ? std::snprintf(buf, len, "rows grid=%u waves=%d splits=%d members=%d", pl.grid, pl.waves, pl.splits, pl.members)
                                     : std::snprintf(buf, len, "tiles grid=%u tokens=%d whole=%d splits=%d operands=%d", pl.grid, pl.tile, pl.whole,
                                                     pl.splits, pl.fp16 ? 16 : 8);
  if (n < 0 || (size_t)n >= len)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "the line needs %d bytes, buf holds %zu", n + 1, len);
  return QGEMM_OK;
}

}  // extern "C"
