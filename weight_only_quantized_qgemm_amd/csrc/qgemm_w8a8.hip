// qgemm_w8a8_run: checks of the pointers and launch of the planned kernel.
#include "qgemm_w8a8_device.h"

namespace {
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
}  // namespace

extern "C" qgemm_status_t qgemm_w8a8_run(const qgemm_w8a8_t* p, const void* A, const float* a_scales, const void* W,
                                         const float* w_scales, void* out, float* out_scales, void* workspace,
                                         size_t workspace_bytes, void* stream) {
  using namespace qgemm;
  clear_error();
  qgemm_status_t st = validate_w8a8(p);
  if (st != QGEMM_OK) return st;
  if (p->M == 0) return QGEMM_OK;
  const bool quantized = p->out_dtype == QGEMM_DT_FP8_E4M3;
  const struct { const char* name; const void* p; uintptr_t align; } args[] = {
      {"A", A, 16}, {"a_scales", a_scales, 4}, {"W", W, 16}, {"w_scales", w_scales, 4}, {"out", out, 16}};
  for (const auto& x : args) {
    if (!x.p) return fail(QGEMM_ERR_INVALID_ARGUMENT, "%s is NULL", x.name);
    if (!aligned(x.p, x.align)) return fail(QGEMM_ERR_MISALIGNED, "%s must be %d-byte aligned", x.name, (int)x.align);
  }
  if (quantized && !out_scales) return fail(QGEMM_ERR_INVALID_ARGUMENT, "out_scales is NULL (needed for FP8_E4M3)");
  if (!quantized && out_scales) return fail(QGEMM_ERR_INVALID_ARGUMENT, "out_scales must be NULL unless out_dtype is FP8_E4M3");
  if (!aligned(out_scales, 4)) return fail(QGEMM_ERR_MISALIGNED, "out_scales must be 4-byte aligned");
  W8Plan pl;
  st = make_w8a8_plan(p, &pl);
  if (st != QGEMM_OK) return st;
  if (pl.ws_bytes) {
    if (!workspace || workspace_bytes < pl.ws_bytes)
      return fail(QGEMM_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes needed, %zu given%s", pl.ws_bytes,
                  workspace ? workspace_bytes : (size_t)0, workspace ? "" : " (NULL)");
    if (!aligned(workspace, 256)) return fail(QGEMM_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  }
  // What is written must be apart from everything else: other workgroups still read A when the first outputs are stored.
  const uint64_t M = p->M, N = p->N, K = p->K, KB = K / kBlock, parts = p->gate != QGEMM_GATE_NONE ? 2 : 1;
  const struct { const char* name; const void* p; uint64_t bytes; } all[] = {
      {"out", out, M * N * (quantized ? 1 : p->out_dtype == QGEMM_DT_F32 ? 4 : 2)},
      {"out_scales", out_scales, quantized ? M * (N / kBlock) * 4 : 0},
      {"workspace", workspace, pl.ws_bytes},                           // the first three are written
      {"A", A, M * K}, {"a_scales", a_scales, M * KB * 4}, {"W", W, parts * N * K},
      {"w_scales", w_scales, parts * ((N + kBlock - 1) / kBlock) * KB * 4}};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 7; ++j) {
      const uint64_t x = reinterpret_cast<uintptr_t>(all[i].p), y = reinterpret_cast<uintptr_t>(all[j].p);
      if (all[i].bytes && all[j].bytes && x < y + all[j].bytes && y < x + all[i].bytes)
        return fail(QGEMM_ERR_INVALID_ARGUMENT, "%s overlaps %s", all[i].name, all[j].name);
    }
  w8::W8Args a{};
  a.a = static_cast<const uint8_t*>(A);
  a.w = static_cast<const uint8_t*>(W);
  a.as = a_scales;
  a.ws = w_scales;
  a.out = out;
  a.os = out_scales;
  a.tickets = static_cast<unsigned*>(workspace);
  a.partials = pl.ws_bytes ? reinterpret_cast<float*>(static_cast<char*>(workspace) + kW8Tickets * 4) : nullptr;
  a.M = (int)p->M;
  a.N = (int)p->N;
  a.K = (int)p->K;
  a.KB = (int)(p->K / kBlock);
  a.out_dtype = p->out_dtype;
  a.gate = p->gate;
  a.splits = pl.splits;
  a.kb_per_split = pl.kb_per_split;
  a.tiles = pl.tiles;
  a.whole = pl.whole;
  a.tiles_n = pl.tiles_n;
  a.row_blocks = (a.N + kBlock - 1) / kBlock;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = pl.kind == W8_ROWS ? w8::launch_rows(pl, a, s) : w8::launch_tiles(pl, a, s);
  if (e != hipSuccess) return fail(QGEMM_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  return QGEMM_OK;
}
