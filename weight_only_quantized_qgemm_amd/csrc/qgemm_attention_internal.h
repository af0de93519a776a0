// Internal declarations of the attention operators (include/qgemm_attention.h): what the host
// validation and the kernel launchers share.
#pragma once

#include "../../include/qgemm_attention.h"
#include "qgemm_internal.h"

namespace qgemm {

// Checks of the descriptors; the message names the field.
qgemm_status_t validate_norm_rope(const qgemm_norm_rope_t* p);
qgemm_status_t validate_cache(const qgemm_cache_t* c);
qgemm_status_t validate_attention(const qgemm_attention_t* p);

// A launch holds less than 2^32 work-items.
inline bool launchable(int64_t workgroups, int threads) { return workgroups <= 0xffffffffLL / threads; }

// Byte geometry of one block (one page of one kv head).
struct BlockGeom {
  int codes;      // bytes of one side's codes (= offset of the V codes)
  int params;     // bytes of one side's parameters
  int bytes;      // whole block
};
inline BlockGeom block_geom(const qgemm_cache_t* c) {
  const int ng = c->head_dim / c->group_size;
  BlockGeom g;
  g.codes = c->page_size * c->head_dim / 2;
  g.params = c->page_size * ng * 4;
  g.bytes = 2 * (g.codes + g.params);
  return g;
}

enum AttnKind : int { ATTN_ROWS = 1, ATTN_TILES = 2 };

// Tiles kernel: column tiles of 16 query rows per wavefront and wavefronts per workgroup.
struct TileShape { int cols, waves; };
// Measured at prompts of 4096 (us): D 64 2x8 146, 3x8 233, 4x4 212; D 128 2x8 187, 1x8 277, 2x4 375;
// four groups in bf16 2x8 224, 1x8 388, in fp16 (an accumulator per group) 1x8 397, 2x8 752; D 256 1x8 226,
// 2x4 372, and four groups in bf16 1x8 278, in fp16 1x8 592, 2x4 527.
constexpr TileShape tile_shape(int dim, int groups, bool bf16) {
  if (groups == 4 && !bf16) return dim == 256 ? TileShape{2, 4} : TileShape{1, 8};
  return dim == 256 ? TileShape{1, 8} : TileShape{2, 8};
}
constexpr int tile_rows(TileShape t) { return 16 * t.cols * t.waves; }

// Rows kernel: how short work is cut (see AttnArgs).
struct Pieces { int share, least; };
// One request of 777 / 4000 / 32000 tokens: 10.8 / 11.3 / 17.2 us; least 16 11.5 / 14.2 / 17.4, share 6
// 10.8 / 11.4 / 20.7.
constexpr Pieces kPieces{12, 4};

// Launch plan of qgemm_attention, a pure function of the descriptor.
struct AttnPlan {
  AttnKind kind;
  int groups;          // NG
  int pack;            // rows kernel: subtiles side by side in the 16 columns (F: 1, 2, 4)
  int waves;           // rows kernel: wavefronts per workgroup (1 or 4)
  int tile, splits;    // tiles kernel: query rows per workgroup, workgroups per row tile
  unsigned grid;       // workgroups
  size_t tickets_bytes;
  size_t ws_bytes;
};
qgemm_status_t make_attention_plan(const qgemm_attention_t* p, AttnPlan* pl);

}  // namespace qgemm
