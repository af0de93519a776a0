// qgemm_attention: argument checks, plan and launch of the rows or tiles kernel.
#include <hip/hip_runtime.h>

#include "qgemm_attention_device.h"

namespace {

using namespace qgemm;

using namespace attn;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

template <bool BF, int D>
hipError_t launch(const AttnPlan& pl, const AttnArgs& a, hipStream_t s) {
  return pl.kind == ATTN_ROWS ? launch_rows<BF, D>(pl, a, s) : launch_tiles<BF, D>(pl, a, s);
}

}  // namespace

extern "C" qgemm_status_t qgemm_attention(const qgemm_attention_t* p, const void* q, int64_t q_stride, const void* data,
                                          const int32_t* page_table, const int32_t* seq_lens, const int32_t* q_start,
                                          void* out, int64_t out_stride, void* workspace, size_t workspace_bytes,
                                          void* stream) {
  clear_error();
  qgemm_status_t st = validate_attention(p);
  if (st != QGEMM_OK) return st;
  if (p->total_q == 0) return QGEMM_OK;
  if (!q || !data || !out) return fail(QGEMM_ERR_INVALID_ARGUMENT, "%s is NULL", !q ? "q" : !data ? "data" : "out");
  if (!page_table || !seq_lens || !q_start)
    return fail(QGEMM_ERR_INVALID_ARGUMENT, "%s is NULL", !page_table ? "page_table" : !seq_lens ? "seq_lens" : "q_start");
  if (!aligned(q, 16) || !aligned(data, 16) || !aligned(out, 16))
    return fail(QGEMM_ERR_MISALIGNED, "q, data and out must be 16-byte aligned");
  if (!aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(q_start, 4))
    return fail(QGEMM_ERR_MISALIGNED, "page_table, seq_lens and q_start must be 4-byte aligned");
  const int64_t row = (int64_t)p->q_heads * p->cache.head_dim;
  for (int64_t s : {q_stride, out_stride})
    if (s < row || s % 8 || s > (int64_t(1) << 31))
      return fail(QGEMM_ERR_INVALID_ARGUMENT, "token strides must be multiples of 8 in [%lld, 2^31], got %lld",
                  (long long)row, (long long)s);
  AttnPlan pl;
  st = make_attention_plan(p, &pl);
  if (st != QGEMM_OK) return st;
  if (pl.ws_bytes) {
    if (!workspace || workspace_bytes < pl.ws_bytes)
      return fail(QGEMM_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes needed, %zu given%s", pl.ws_bytes,
                  workspace ? workspace_bytes : (size_t)0, workspace ? "" : " (NULL)");
    if (!aligned(workspace, 256)) return fail(QGEMM_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  }
  const BlockGeom g = block_geom(&p->cache);
  AttnArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.data = static_cast<const uint8_t*>(data);
  a.table = page_table;
  a.lens = seq_lens;
  a.starts = q_start;
  a.out = static_cast<uint16_t*>(out);
  a.qs = q_stride;
  a.os = out_stride;
  a.total_q = (int)p->total_q;
  a.batch = p->batch;
  a.kv_heads = p->cache.kv_heads;
  a.ratio = p->q_heads / p->cache.kv_heads;
  a.max_pages = p->max_pages;
  a.page = p->cache.page_size;
  // t / page by a multiplication: with 2^s <= page < 2^(s + 1) and mul = floor(2^(31 + s) / page) + 1, the
  // product exceeds t 2^(31 + s) / page by at most t, which is below 2^(31 + s) / page while t < 2^30.
  const unsigned log2_page = 31 - (unsigned)__builtin_clz((unsigned)p->cache.page_size);
  a.page_shift = log2_page - 1;
  a.page_mul = (unsigned)((uint64_t(1) << (31 + log2_page)) / (unsigned)p->cache.page_size + 1);
  a.num_pages = (int)p->cache.num_pages;
  a.codes = g.codes;
  a.params = g.params;
  a.block = g.bytes;
  a.max_q = p->max_q_len;
  a.causal = p->causal;
  a.window = bounded_window(p->window);
  a.scale = p->scale * 1.4426950408889634f;
  hipStream_t s = static_cast<hipStream_t>(stream);
  a.piece_share = kPieces.share;
  a.piece_least = kPieces.least;
  a.splits = pl.splits;
  if (pl.ws_bytes) {
    a.tickets = static_cast<unsigned*>(workspace);
    a.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.tickets_bytes);
  }
  const bool bf = p->cache.dtype == QGEMM_DT_BF16;
  hipError_t e;
  switch (p->cache.head_dim) {
    case 64: e = bf ? launch<true, 64>(pl, a, s) : launch<false, 64>(pl, a, s); break;
    case 128: e = bf ? launch<true, 128>(pl, a, s) : launch<false, 128>(pl, a, s); break;
    default: e = bf ? launch<true, 256>(pl, a, s) : launch<false, 256>(pl, a, s); break;
  }
  if (e != hipSuccess) return fail(QGEMM_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  return QGEMM_OK;
}
