// The attention kernels' geometry (csrc/qgemm_attention_geometry.h) as C functions, for the CPU tests.
#include "../weight_only_quantized_qgemm_amd/csrc/qgemm_attention_geometry.h"

using namespace qgemm::attn;

extern "C" {

// out: start, n, len, lo, hi of the sequence
void geometry_seq(int s0, int s1, int len, int total_q, int max_q, int tokens, int window, int* out) {
  const Seq s = seq_of(s0, s1, len, total_q, max_q, tokens, bounded_window(window));
  const int v[5] = {s.start, s.n, s.len, s.lo, s.hi};
  for (int i = 0; i < 5; ++i) out[i] = v[i];
}

// the rows that n sequences claim in all, summed in runs of 64
unsigned geometry_claimed(const int* queries, int n) {
  unsigned claimed = 0;
  for (int i = 0; i < n; i += 64) {
    int run = 0;
    for (int j = i; j < n && j < i + 64; ++j) run += queries[j];
    claimed = claim(claimed, run);
  }
  return claimed;
}

// out: lo, hi, per, active, seen of the row tile that begins at row0, of a sequence of n queries and len tokens
void geometry_tile(int n, int len, int row0, int BM, int ratio, int causal, int window, int step, int splits, int* out) {
  Seq s{};
  s.n = n;
  s.len = len;
  const Tile t = tile_of(s, row0, lesser(ratio * n, row0 + BM), BM, ratio, causal, bounded_window(window), step, splits);
  const int v[5] = {t.lo, t.hi, t.per, t.active, t.seen};
  for (int i = 0; i < 5; ++i) out[i] = v[i];
}

}
