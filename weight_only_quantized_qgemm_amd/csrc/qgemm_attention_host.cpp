// Host side of the attention operators: descriptor validation, cache geometry and launch planning.
// Nothing in this file touches the GPU.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "qgemm_attention_internal.h"

namespace qgemm {

static_assert(sizeof(qgemm_norm_rope_t) == 48, "qgemm_norm_rope_t layout is part of the ABI");
static_assert(sizeof(qgemm_cache_t) == 32, "qgemm_cache_t layout is part of the ABI");
static_assert(sizeof(qgemm_attention_t) == 80, "qgemm_attention_t layout is part of the ABI");

static const int kCUs = 256;
static const int kMaxSplits = 32;           // workgroups per row tile
// The workspace begins with a ticket region of one size, whatever the plan, so that partial results of one
// problem never lie where another counts and one workspace serves them all.
static const int kTickets = 8192;
static const int64_t kMaxTokens = int64_t(1) << 24;

static qgemm_status_t check_dtype_dim(const char* what, int dtype, int head_dim) {
  if (dtype < QGEMM_DT_F16 || dtype > QGEMM_DT_NF4)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "%s dtype value %d is not a qgemm_dtype_t", what, dtype);
  if (dtype != QGEMM_DT_F16 && dtype != QGEMM_DT_BF16)
    return fail(QGEMM_ERR_UNSUPPORTED, "%s dtype must be F16 or BF16, got %d", what, dtype);
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(QGEMM_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256, got %d", head_dim);
  return QGEMM_OK;
}

qgemm_status_t validate_norm_rope(const qgemm_norm_rope_t* p) {
  if (!p) return fail(QGEMM_ERR_INVALID_ARGUMENT, "problem is NULL");
  const qgemm_status_t st = check_dtype_dim("norm_rope", p->dtype, p->head_dim);
  if (st != QGEMM_OK) return st;
  if (p->tokens < 0 || p->tokens > kMaxTokens)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "tokens must be in [0, %lld], got %lld", (long long)kMaxTokens,
                (long long)p->tokens);
  if (p->q_heads < 0 || p->q_heads > 1024 || p->kv_heads < 0 || p->kv_heads > 1024 || p->q_heads + p->kv_heads == 0)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "q_heads and kv_heads must be in [0, 1024] and not both 0, got %d and %d",
                p->q_heads, p->kv_heads);
  if (p->rot_dim < 0 || p->rot_dim > p->head_dim || p->rot_dim % 8)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "rot_dim must be a multiple of 8 in [0, head_dim = %d], got %d", p->head_dim,
                p->rot_dim);
  if (p->rot_dim && (p->max_pos < 1 || p->max_pos > kMaxTokens))
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "max_pos must be in [1, %lld], got %d", (long long)kMaxTokens, p->max_pos);
  if ((p->interleaved | 1) != 1 || (p->norm | 1) != 1)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "interleaved and norm must be 0 or 1, got %d and %d", p->interleaved, p->norm);
  if (p->norm && !(p->eps >= 0.0f && std::isfinite(p->eps)))
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "eps must be finite and at least 0, got %g", (double)p->eps);
  if (p->reserved) return fail(QGEMM_ERR_INVALID_ARGUMENT, "reserved must be 0, got %d", p->reserved);
  return QGEMM_OK;
}

qgemm_status_t validate_cache(const qgemm_cache_t* c) {
  if (!c) return fail(QGEMM_ERR_INVALID_ARGUMENT, "cache is NULL");
  const qgemm_status_t st = check_dtype_dim("cache", c->dtype, c->head_dim);
  if (st != QGEMM_OK) return st;
  if (c->num_pages < 1 || c->num_pages > 0x7fffffffLL)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "num_pages must be in [1, 2^31 - 1], got %lld", (long long)c->num_pages);
  if (c->page_size < 16 || c->page_size > 4096 || c->page_size % 16)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "page_size must be a multiple of 16 in [16, 4096], got %d", c->page_size);
  if (c->kv_heads < 1 || c->kv_heads > 1024)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "kv_heads must be in [1, 1024], got %d", c->kv_heads);
  const int g = c->group_size;
  if (g != c->head_dim && g * 2 != c->head_dim && (g * 4 != c->head_dim || c->head_dim < 128))
    return fail(QGEMM_ERR_UNSUPPORTED, "group_size must be head_dim, head_dim / 2 or (head_dim >= 128) head_dim / 4; got "
                "group_size %d, head_dim %d", g, c->head_dim);
  if (c->reserved) return fail(QGEMM_ERR_INVALID_ARGUMENT, "cache reserved must be 0, got %d", c->reserved);
  return QGEMM_OK;
}

qgemm_status_t validate_attention(const qgemm_attention_t* p) {
  if (!p) return fail(QGEMM_ERR_INVALID_ARGUMENT, "problem is NULL");
  const qgemm_status_t st = validate_cache(&p->cache);
  if (st != QGEMM_OK) return st;
  if (p->total_q < 0 || p->total_q > kMaxTokens)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "total_q must be in [0, %lld], got %lld", (long long)kMaxTokens,
                (long long)p->total_q);
  if (p->batch < 1 || p->batch > 65535)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "batch must be in [1, 65535], got %d", p->batch);
  if (p->q_heads < 1 || p->q_heads > 4096 || p->q_heads % p->cache.kv_heads)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "q_heads must be a positive multiple of kv_heads (%d), at most 4096; got %d",
                p->cache.kv_heads, p->q_heads);
  if (p->total_q && (p->max_q_len < 1 || p->max_q_len > p->total_q))
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "max_q_len must be in [1, total_q = %lld], got %d", (long long)p->total_q,
                p->max_q_len);
  if (p->max_pages < 1 || (int64_t)p->max_pages * p->cache.page_size > (int64_t(1) << 30))
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "max_pages must be positive and max_pages * page_size at most 2^30, got %d "
                "pages of %d", p->max_pages, p->cache.page_size);
  if ((p->causal | 1) != 1) return fail(QGEMM_ERR_INVALID_ARGUMENT, "causal must be 0 or 1, got %d", p->causal);
  if (p->window < 0 || (p->window && !p->causal))
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "window must be 0, or positive with causal = 1; got %d", p->window);
  if (!std::isfinite(p->scale)) return fail(QGEMM_ERR_INVALID_ARGUMENT, "scale must be finite, got %g", (double)p->scale);
  if (p->kernel_hint < QGEMM_ATTENTION_AUTO || p->kernel_hint > QGEMM_ATTENTION_TILES)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "kernel_hint must be 0 to 2, got %d", p->kernel_hint);
  if (p->reserved[0] || p->reserved[1]) return fail(QGEMM_ERR_INVALID_ARGUMENT, "reserved must be 0");
  return QGEMM_OK;
}

qgemm_status_t make_attention_plan(const qgemm_attention_t* p, AttnPlan* pl) {
  std::memset(pl, 0, sizeof(*pl));
  if (p->total_q == 0) return QGEMM_OK;
  pl->groups = p->cache.head_dim / p->cache.group_size;
  const int dim = p->cache.head_dim, ng = pl->groups;
  const int64_t ratio = p->q_heads / p->cache.kv_heads, rows = ratio * p->max_q_len;
  const int64_t tokens = (int64_t)p->max_pages * p->cache.page_size, steps = (tokens + 63) / 64;
  // tiles of `r` query rows over all sequences, each of which may end in a partly filled one
  auto tiles_of = [&](int64_t r) {
    const int64_t by_total = p->batch + ratio * p->total_q / r, by_longest = (rows + r - 1) / r * p->batch;
    return (by_total < by_longest ? by_total : by_longest) * p->cache.kv_heads;
  };

  // ---- rows kernel.  Rows per column group: as few as hold a sequence's rows of a kv head, so that more
  // subtiles lie side by side; 16 rows of D 256 in four groups do not fit the registers.
  pl->pack = rows <= 4 && dim < 256 ? 4 : rows <= 8 || (dim == 256 && ng == 4) ? 2 : 1;
  const int row_tile = 16 / pl->pack;
  const int64_t row_tiles = tiles_of(row_tile);
  // ---- tiles kernel.  A row tile's tokens are split over workgroups (one is resident per compute unit)
  // where a model of the launch, in steps of 64 tokens, says that it is shorter: the longest chain while every
  // workgroup has a compute unit; past that also all workgroups' steps and overheads spread over the chip
  // plus a quarter of a chain for the uneven end.  (6 chunks in a window of 4096, 64 heads: 398 us in one
  // part, 476 in four; 100 queries after 16000 tokens, 32 heads: 740 us in one part, 198 in four, 75 in 16.)
  const TileShape shape = tile_shape(dim, ng, p->cache.dtype == QGEMM_DT_BF16);
  pl->tile = tile_rows(shape);
  const int64_t tiles = tiles_of(pl->tile);
  double best = 0.0;
  pl->splits = 1;
  // the share of the steps that a causal mask leaves: a half where the queries are the whole sequence
  const double left = p->causal && !p->window ? 1.0 - 0.5 * std::min((double)p->max_q_len, (double)tokens) / (double)tokens : 1.0;
  for (int s = 1, levels = 0; s <= kMaxSplits && (s == 1 || ((int64_t)s * 4 <= steps && tiles * s <= kTickets)); ++s) {
    while ((1 << levels) < s) ++levels;
    const double chain = (double)((steps + s - 1) / s), join = levels;
    const double latency = chain + 2.0 + (s > 1 ? 1.0 : 0.0) + join;
    const double spread = left * (double)tiles * s * (chain + 4.0 + (s > 1 ? 4.5 : 0.0)) / kCUs + chain / 4 + join;
    // parts that have work, the last of a tile's being short: do they all start at once?
    const bool at_once = s > 1 && std::min(1.0, left + 0.5 / s) * (double)tiles * s <= kCUs;
    const double cost = at_once || latency > spread ? latency : spread;
    if (s == 1 || cost < best) {
      pl->splits = s;
      best = cost;
    }
  }

  // ---- which: microseconds that a compute unit takes for 64 tokens of 16 rows (rows kernel; of 8 rows for
  // D 256 in four groups) and of a row tile (tiles kernel, fp16 and bf16), for D 64, 128, 256 and NG 1, 2, 4,
  // measured at 32 rows and 8008 tokens x 8, and at a prompt of 4096.
  static const double kRowUnit[3][3] = {{0.31, 0.38, 0.38}, {0.40, 0.50, 0.77}, {1.05, 1.05, 0.90}};
  static const double kTileStep[2][3][3] = {{{2.35, 2.85, 2.85}, {2.95, 4.05, 3.0}, {3.6, 3.9, 8.3}},
                                            {{2.35, 2.4, 2.4}, {2.9, 3.15, 3.5}, {3.6, 3.9, 4.4}}};
  const int di = dim == 64 ? 0 : dim == 128 ? 1 : 2, gi = ng == 1 ? 0 : ng == 2 ? 1 : 2;
  const double rows_us = 10.0 + kRowUnit[di][gi] * (double)row_tiles * (double)steps / kCUs;
  const double tiles_us = 8.0 + kTileStep[p->cache.dtype == QGEMM_DT_BF16][di][gi] * best;
  // the rows kernel numbers the units of all row tiles, as long as the table is wide, in 32 bits
  const bool divides = ((double)steps + 8) * (double)row_tiles <= 2147483647.0;
  const bool use_rows = p->kernel_hint == QGEMM_ATTENTION_ROWS ||
                        (p->kernel_hint == QGEMM_ATTENTION_AUTO && divides && (rows <= row_tile || rows_us <= tiles_us));
  if (use_rows) {
    pl->kind = ATTN_ROWS;
    if (!divides)
      return fail(QGEMM_ERR_UNSUPPORTED, "%lld row tiles of up to %lld tokens are beyond what one launch divides",
                  (long long)row_tiles, (long long)tokens);
    // Many segments (several per resident workgroup of four wavefronts) take a wavefront each: the starts
    // and ends of short ones overlap (500 requests of 200 tokens 64 -> 38 us, 200 of 500 42 -> 30; from
    // 1024 segments of 1500 tokens on four are as good, and better for few long ones).
    pl->waves = row_tiles >= 1536 ? 1 : 4;
    pl->grid = (unsigned)(2 * kCUs * 4 / pl->waves);
    pl->tickets_bytes = (size_t)kTickets * 4;         // one per workgroup, at most 2048
    pl->ws_bytes = pl->tickets_bytes + (size_t)2 * pl->grid * row_tile * (dim + 4) * 4;
    return QGEMM_OK;
  }
  pl->kind = ATTN_TILES;
  if (!launchable(tiles * pl->splits, 64 * shape.waves))
    return fail(QGEMM_ERR_UNSUPPORTED, "the problem needs %lld workgroups, more than one launch allows",
                (long long)(tiles * pl->splits));
  pl->grid = (unsigned)(tiles * pl->splits);
  if (pl->splits > 1) {
    pl->tickets_bytes = (size_t)kTickets * 4;
    pl->ws_bytes = pl->tickets_bytes +
                   (size_t)tiles * pl->splits * ((size_t)pl->tile * dim + (size_t)shape.cols * shape.waves * 256) * 4;
  }
  return QGEMM_OK;
}

}  // namespace qgemm

using namespace qgemm;

extern "C" {

qgemm_status_t qgemm_cache_bytes(const qgemm_cache_t* c, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(QGEMM_ERR_INVALID_ARGUMENT, "bytes is NULL");
  const qgemm_status_t st = validate_cache(c);
  if (st != QGEMM_OK) return st;
  *bytes = (size_t)c->num_pages * c->kv_heads * (size_t)block_geom(c).bytes;
  return QGEMM_OK;
}

qgemm_status_t qgemm_attention_workspace_bytes(const qgemm_attention_t* p, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(QGEMM_ERR_INVALID_ARGUMENT, "bytes is NULL");
  qgemm_status_t st = validate_attention(p);
  if (st != QGEMM_OK) return st;
  AttnPlan pl;
  st = make_attention_plan(p, &pl);
  if (st != QGEMM_OK) return st;
  *bytes = pl.ws_bytes;
  return QGEMM_OK;
}

qgemm_status_t qgemm_attention_describe(const qgemm_attention_t* p, char* buf, size_t len) {
  clear_error();
  if (!buf || !len) return fail(QGEMM_ERR_INVALID_ARGUMENT, "buf is NULL or len is 0");
  qgemm_status_t st = validate_attention(p);
  if (st != QGEMM_OK) return st;
  AttnPlan pl;
  st = make_attention_plan(p, &pl);
  if (st != QGEMM_OK) return st;
  const int n = p->total_q == 0 ? std::snprintf(buf, len, "empty")
                : pl.kind == ATTN_ROWS ? std::snprintf(buf, len, "rows grid=%u groups=%d pack=%d waves=%d", pl.grid, pl.groups,
                                                       pl.pack, pl.waves)
                                       : std::snprintf(buf, len, "tiles grid=%u groups=%d rows=%d splits=%d", pl.grid,
                                                       pl.groups, pl.tile, pl.splits);
  if (n < 0 || (size_t)n >= len)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "the line needs %d bytes, buf holds %zu", n + 1, len);
  return QGEMM_OK;
}

}  // extern "C"
