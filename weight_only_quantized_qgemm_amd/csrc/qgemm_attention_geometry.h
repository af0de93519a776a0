// Which rows and tokens a workgroup of the attention kernels takes, from the lengths in device memory, in 32-bit
// integers.  Plain constexpr functions: the kernels use them on the device, the CPU tests compile them for the host and hold them
// to the same arithmetic without a limit on its numbers.
//
// No sum here leaves 32 bits: positions are below 2^30, queries are at most 2^24, and the window is
// bounded to 2^30 before a launch.
#pragma once

namespace qgemm {
namespace attn {

constexpr int lesser(int a, int b) { return a < b ? a : b; }
constexpr int greater(int a, int b) { return a < b ? b : a; }

// A window as wide as the longest context hides nothing, and neither does a wider one.
constexpr int kWindowMost = 1 << 30;
constexpr int bounded_window(int window) { return lesser(window, kWindowMost); }

// A sequence's geometry, every value bounded.
struct Seq {
  int start, n, len;               // first query row, queries, tokens
  int lo, hi;                      // tokens any query can see: lo a multiple of 16
};
// From q_start[b], q_start[b + 1] and seq_lens[b]; tokens = max_pages * page_size.
constexpr Seq seq_of(int s0, int s1, int len, int total_q, int max_q, int tokens, int window) {
  Seq s{};
  s.start = lesser(greater(s0, 0), total_q);
  s.n = lesser(greater(lesser(s1, total_q) - s.start, 0), max_q);
  s.len = lesser(greater(len, 0), tokens);
  s.hi = s.len;
  s.lo = window ? greater(s.len - s.n - window + 1, 0) & ~15 : 0;
  if (s.lo > s.hi) s.lo = s.hi & ~15;
  return s;
}

// Launches and workspaces are made for total_q query rows.  Starts that decrease and rise again may claim more,
// and more row tiles than there are workgroups and partial results; no others do.  The claimed rows are summed
// in runs of 64 sequences, whose sum is at most 2^30, and stop there.
constexpr unsigned claim(unsigned claimed, int run) {
  const unsigned sum = claimed + (unsigned)run;
  return sum < 1u << 30 ? sum : 1u << 30;
}

// Tiles kernel: the tokens that rows row0 .. row_end - 1 see, and how a launch of `splits` workgroups per row tile
// of BM rows divides them, in steps of `step` tokens.
struct Tile {
  int lo, hi;                      // tokens: lo a multiple of 16
  int seen;                        // the first that a row sees (or one past all)
  int per, active;                 // steps of a part, parts that have work (the first `active` workgroups)
};
constexpr Tile tile_of(const Seq& s, int row0, int row_end, int BM, int ratio, int causal, int window, int step, int splits) {
  Tile t{};
  const int past = s.len - s.n;    // position of query 0
  t.hi = causal ? lesser(s.len, greater(past + (row_end - 1) / ratio + 1, 0)) : s.len;
  t.seen = window ? greater(past + row0 / ratio - window + 1, 0) : 0;
  t.lo = lesser(t.seen & ~15, t.hi & ~15);
  const int all = (t.hi - t.lo + step - 1) / step;
  // Parts are as long as the sequence's longest row tile needs, tiles that see less have fewer (a prompt of
  // 1500, 32 heads: 83 us with each tile's own length divided, 67; 700 queries after 5000 tokens 150, 128).
  const int longest = window ? lesser(s.len, window + (BM - 1) / ratio + 17) : s.len;
  t.per = greater(1, ((longest + step - 1) / step + splits - 1) / splits);
  t.active = lesser(greater(1, (all + t.per - 1) / t.per), splits);
  return t;
}

}  // namespace attn
}  // namespace qgemm
