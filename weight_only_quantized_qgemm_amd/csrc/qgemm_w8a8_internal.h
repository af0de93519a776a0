// Internal declarations of the 8-bit operators (include/qgemm_w8a8.h): what the host validation and
// the kernel launchers share.
#pragma once

#include "../../include/qgemm_w8a8.h"
#include "qgemm_internal.h"

namespace qgemm {

qgemm_status_t validate_add_norm(const qgemm_add_norm_t* p);
qgemm_status_t validate_w8a8(const qgemm_w8a8_t* p);

// Values of one scale block, along K and along a weight's rows.
constexpr int kBlock = 128;
// Weight rows of a workgroup's tile (tiles kernel); with a gate half of them belong to each projection,
// so that a tile's outputs are one scale block wide.
constexpr int kTileRows = 256;
// The rows kernel takes up to this many tokens.
constexpr int kRowsMaxM = 64;
// Wavefronts of a workgroup (at most: the rows kernel may take 4).
constexpr int kW8Waves = 8;

enum W8Kind : int { W8_ROWS = 1, W8_TILES = 2 };

// Launch plan of qgemm_w8a8_run, a pure function of the descriptor.
struct W8Plan {
  W8Kind kind;
  int tile;            // tiles kernel: tokens of a tile
  bool fp16;           // tiles kernel: operands are converted to fp16, so that sums are whole
  int waves;           // rows kernel: wavefronts of a workgroup
  int tiles, whole, tiles_n;   // tiles kernel: all tiles, those that are not split, those along the weight rows
  int splits;          // workgroups along K
  int kb_per_split;
  int64_t groups;      // tickets: sets of workgroups whose last one finishes the output
  int members;         // workgroups of a set
  unsigned grid;
  size_t ws_bytes;
};
qgemm_status_t make_w8a8_plan(const qgemm_w8a8_t* p, W8Plan* pl);

// The workspace begins with a ticket region of one size, whatever the plan, so that partial results of one
// problem never lie where another counts and one workspace serves them all.
constexpr int64_t kW8Tickets = 1 << 17;
constexpr int kTileParts = 4;          // tickets of a shared tile

namespace w8 {

struct W8Args {
  const uint8_t *a, *w;
  const float *as, *ws;
  void* out;
  float* os;
  unsigned* tickets;
  float* partials;
  int M, N, K, KB;
  int out_dtype, gate;
  int splits, kb_per_split;
  int tiles, whole, tiles_n;        // tiles kernel: all tiles, those that are not split, those along the weight rows
  int row_blocks;                   // scale blocks of one projection's rows
};

}  // namespace w8
}  // namespace qgemm
