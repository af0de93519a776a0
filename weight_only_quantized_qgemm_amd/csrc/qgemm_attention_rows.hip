// Attention with few query rows per kv head (one token, a few drafted ones): the cache is read once,
// tokens spread over wavefronts and workgroups.
//
// Bound by reading the cache: D + 8 NG bytes per token and kv head.  The work is cut into units of 64
// tokens of one (sequence, kv head, row tile), laid end to end, and every workgroup of a fixed grid
// takes an equal run of them, found from the lengths in device memory: the balance does not depend
// on how the lengths differ, and the host needs none of them.  A segment that several workgroups
// share is joined by the last of them to finish, in order (a ticket per segment; nobody waits).
//
// Inside a workgroup the four wavefronts take steps of 16 SUB tokens in turn, each with its own
// running maximum, sum and output, joined through LDS.  The 16 columns of an MFMA are more than
// most calls have query rows, so with F = 2 or 4 each column group of 16 / F holds the same rows for
// another 16-token subtile: the softmax then works on full lanes, and its cost per token falls by F.
//
// 64 requests of up to 8191 tokens, 64 query and 8 kv heads of 128, bf16: 64.2 us, 4.6 TB/s; 4 requests of
// 100000 to 131000 tokens in groups of 64: 105 us, 5.1 TB/s, what a large copy reaches.  One token over 777
// takes 9.9 us: a launch (3.2), three dependent memory trips, one step and one join at about 1.3 us each.
#include <type_traits>

#include "qgemm_attention_device.h"

namespace qgemm {
namespace attn {
namespace {

// What the start and the end of a segment cost, in units of 64 tokens: counted with its tokens when long
// work is divided (64 requests of 0..8191 tokens: 90 us with 0, 70 with 4, 64 with 8, 65 with 12).
constexpr int kOver = 8;

template <int D, int NG, int F>
struct Step {                                       // one step's bytes, in registers
  static constexpr int U = D / 32, SUB = F == 1 ? 2 : F, ST = F == 1 ? 2 : 1;
  // Two steps' registers are held while they fit beside the rest (256 in all, two wavefronts per SIMD);
  // past that the next step is loaded piecewise into the registers that the current one is done with
  // (32 requests of 4000..8190 tokens, D 128: 16 rows and NG 4 116 -> 49 us, 1 row and NG 4 135 -> 110;
  // within the limit two steps are better: 16 rows and NG 2 37.6 -> 35.9, 8 rows and NG 1 44.6 -> 42.2).
  static constexpr bool kTwo = 2 * SUB * U + 8 * ST * NG <= (D == 256 ? 0 : F == 4 ? 40 : 48);
  unsigned k[SUB][U], v[SUB][U];
  u32x4 kp[ST][NG], vp[ST][NG];
};

template <int U>
__device__ __forceinline__ void load_dwords(const uint8_t* p, unsigned (&w)[U]) {
  if constexpr (U == 2) {
    const u32x2 x = *reinterpret_cast<const u32x2*>(p);
    w[0] = x[0];
    w[1] = x[1];
  } else {
#pragma unroll
    for (int j = 0; j < U / 4; ++j) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(p + 16 * j);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[4 * j + i] = x[i];
    }
  }
}

template <bool BF, int D, int NG, int F, int W>
__global__ __launch_bounds__(64 * W, 2) void attention_rows(AttnArgs a) {
  constexpr int U = D / 32, SUB = F == 1 ? 2 : F, ST = F == 1 ? 2 : 1, T = 16 * SUB;
  constexpr int RT = 16 / F;                        // rows per row tile
  constexpr int TILES = D / 16, TG = TILES / NG;    // output tiles, and those of one group
  constexpr int SG = U / NG;                        // k steps of one group
  constexpr int kRowF = D + 4;                      // padded floats of an LDS row
  constexpr int kSlot = RT * (D + 4);               // floats of a partial: rows, then (max, sum) pairs
  typedef Step<D, NG, F> StepT;
  __shared__ __align__(16) float s_o[W * 16 * kRowF];
  __shared__ float s_m[W * 16], s_l[W * 16];
  __shared__ int s_last;

  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  const int fcol = m / RT;                          // the lane's subtile of a step (F > 1)
  const int wg = blockIdx.x;

  // ---- this workgroup's run of units.  Short work is cut coarsely (`piece` units of 64 tokens, so that
  // few segments are split and a workgroup has one piece), long work finely (equal runs).
  auto tiles_of = [&](const Seq& s) { return a.kv_heads * ((a.ratio * s.n + RT - 1) / RT); };
  auto units_of = [&](const Seq& s) { return max(1, (s.hi - s.lo + 63) / 64); };
  Seq mine_seq = lane < a.batch ? load_seq(a, lane) : Seq{0, 0, 0, 0, 0};      // the first 64 stay at hand
  int total = 0;
  unsigned claimed = 0;                             // more query rows than total_q: nothing is computed
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    const Seq x = b0 == 0 ? mine_seq : b0 + lane < a.batch ? load_seq(a, b0 + lane) : Seq{0, 0, 0, 0, 0};
    claimed = claim(claimed, wave_sum(x.n));
    total += wave_sum(tiles_of(x) * units_of(x));
  }
  if (claimed > (unsigned)a.total_q || !total) return;
  const int grid = (int)gridDim.x;
  const int piece = total <= grid * a.piece_share ? max(a.piece_least, (2 * total + grid - 1) / grid) : 1;
  // each segment also counts for kOver units, about what its start and its end cost in long work
  const int over = piece > 1 ? 0 : kOver;
  auto pieces_of = [&](const Seq& s) { return (units_of(s) + piece - 1) / piece + over; };
  {
    total = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
      const Seq x = b0 == 0 ? mine_seq : b0 + lane < a.batch ? load_seq(a, b0 + lane) : Seq{0, 0, 0, 0, 0};
      total += wave_sum(tiles_of(x) * pieces_of(x));
    }
  }
  const int G = min(grid, total);
  if (wg >= G) return;
  const int uq = total / G, ur = total - uq * G;
  int u0 = wg * uq + min(wg, ur);
  const int u1 = u0 + uq + (wg < ur ? 1 : 0);
  auto owner = [&](int u) { return u < ur * (uq + 1) ? u / (uq + 1) : ur + (u - ur * (uq + 1)) / uq; };
  // the sequence that holds piece u0
  int b = 0, before = 0;
  Seq s;
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    const Seq x = b0 == 0 ? mine_seq : b0 + lane < a.batch ? load_seq(a, b0 + lane) : Seq{0, 0, 0, 0, 0};
    const int u = wave_scan(tiles_of(x) * pieces_of(x));
    const unsigned long long past = __ballot(before + u > u0);      // the first lane whose end lies past u0
    if (past) {
      const int l = __builtin_ctzll(past);
      b = b0 + l;
      before += l ? __builtin_amdgcn_readlane(u, l - 1) : 0;
      s.start = __builtin_amdgcn_readlane(x.start, l);
      s.n = __builtin_amdgcn_readlane(x.n, l);
      s.len = __builtin_amdgcn_readlane(x.len, l);
      s.lo = __builtin_amdgcn_readlane(x.lo, l);
      s.hi = __builtin_amdgcn_readlane(x.hi, l);
      break;
    }
    before += __builtin_amdgcn_readlane(u, 63);
  }
  b = __builtin_amdgcn_readfirstlane(b);
  before = __builtin_amdgcn_readfirstlane(before);

  while (u0 < u1) {
    const int nu = pieces_of(s), ub = tiles_of(s) * nu;
    if (u0 >= before + ub) {                        // next sequence (some hold nothing)
      before += ub;
      s = load_seq(a, ++b);
      continue;
    }
    const int seg = (u0 - before) / nu, first = before + seg * nu;   // segment, its first piece
    const int take = min(first + nu - u0, u1 - u0);
    const int rt = seg / a.kv_heads, kvh = seg - rt * a.kv_heads;
    const int at = max(u0 - first - over, 0), cnt = u0 + take - first - over - at;       // pieces of tokens
    if (cnt <= 0) {                                 // the run ends before the segment's first token
      u0 += take;
      continue;
    }
    const int ts = s.lo + 64 * piece * at, te = min(s.hi, ts + 64 * piece * cnt);

    // ---- the wavefront's steps: token ts + T (wave + W j)
    const int steps = te > ts ? (te - ts + T - 1) / T : 0;
    const int mine = steps > wave ? (steps - wave + W - 1) / W : 0;
    constexpr int PER = 64 / SUB;                   // steps whose pages one register holds
    const uint8_t* blk = nullptr;
    int in = 0;
    auto pages = [&](int j0) {                      // lane x: subtile x % SUB of step j0 + x / SUB
      int t = ts + T * (wave + W * (j0 + lane / SUB)) + 16 * (lane % SUB);
      t = min(t, (te - 1) & ~15);                   // past the end: the last subtile again (masked)
      const int p = page_of(a, t);
      int pg = a.table[(long long)b * a.max_pages + p];
      if ((unsigned)pg >= (unsigned)a.num_pages) pg = 0;
      in = t - p * a.page;
      blk = a.data + ((long long)pg * a.kv_heads + kvh) * a.block;
    };
    auto block_at = [&](int x, int& at) {           // subtile x of those at hand (uniform)
      const unsigned long long bits = reinterpret_cast<unsigned long long>(blk);
      const unsigned lo = __builtin_amdgcn_readlane((int)(unsigned)bits, x);
      const unsigned hi = __builtin_amdgcn_readlane((int)(unsigned)(bits >> 32), x);
      at = __builtin_amdgcn_readlane(in, x);
      return reinterpret_cast<const uint8_t*>((unsigned long long)hi << 32 | lo);
    };
    auto params_at = [&](int x) {                   // the lane's tokens' parameters in subtile x (by lane)
      const unsigned long long bits = reinterpret_cast<unsigned long long>(blk);
      const unsigned lo = __shfl((int)(unsigned)bits, x), hi = __shfl((int)(unsigned)(bits >> 32), x);
      return reinterpret_cast<const uint8_t*>((unsigned long long)hi << 32 | lo) + 2 * a.codes + 4 * (__shfl(in, x) + 4 * g);
    };
    auto fetch_k = [&](int j, StepT& st) {
      const int x0 = j % PER * SUB;
#pragma unroll
      for (int f = 0; f < SUB; ++f) {
        int at;
        const uint8_t* p = block_at(x0 + f, at);
        load_dwords<U>(p + (at * (D / 2) + (m * (D / 2) + 4 * U * g)), st.k[f]);
      }
#pragma unroll
      for (int x = 0; x < ST; ++x) {
        const uint8_t* p = params_at(x0 + (F == 1 ? x : fcol));
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) st.kp[x][gr] = *reinterpret_cast<const u32x4*>(p + 4 * gr * a.page);
      }
    };
    auto fetch_v = [&](int j, StepT& st) {
      const int x0 = j % PER * SUB;
#pragma unroll
      for (int f = 0; f < SUB; ++f) {
        int at;
        const uint8_t* p = block_at(x0 + f, at);
        load_dwords<U>(p + a.codes + (at * (D / 2) + lane * (4 * U)), st.v[f]);
      }
#pragma unroll
      for (int x = 0; x < ST; ++x) {
        const uint8_t* p = params_at(x0 + (F == 1 ? x : fcol)) + a.params;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) st.vp[x][gr] = *reinterpret_cast<const u32x4*>(p + 4 * gr * a.page);
      }
    };
    auto fetch = [&](int j, StepT& st) {
      fetch_k(j, st);
      fetch_v(j, st);
    };
    StepT sa;
    // ---- queries: column m holds row rt RT + m % RT, row = query * ratio + head within the group
    const int rows = a.ratio * s.n;
    u32x4 qf[U];
    float qz[NG], kq;
    int see_lo, see_hi;                             // tokens the lane's row sees
    {
      const int row = rt * RT + m % RT;
      const bool on = row < rows;
      const int i = on ? row / a.ratio : 0, h = row - i * a.ratio;
      const int pos = s.len - s.n + i;
      see_hi = a.causal ? min(pos + 1, s.len) : s.len;
      see_lo = a.window ? pos - a.window + 1 : 0;
      const uint16_t* src = a.q + (long long)(s.start + i) * a.qs + (kvh * a.ratio + (on ? h : 0)) * D + 8 * g;
      u32x4 raw[U];
#pragma unroll
      for (int j = 0; j < U; ++j) raw[j] = on ? *reinterpret_cast<const u32x4*>(src + 32 * j) : u32x4{0, 0, 0, 0};
      if (mine) {                                   // the page ids arrive with the queries
        pages(0);
        fetch(0, sa);                               // beside the queries' reduction and conversion
      }
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const float x = __builtin_fabsf(from16<BF>(raw[j][e] >> (16 * o) & 0xffffu));
            top = x < __builtin_inff() ? __builtin_fmaxf(top, x) : top;
          }
      top = max_rows(top);                          // of the lane's row: its result does not depend on its neighbours
      // top = f 2^e, f in [1/2, 1)
      const int e = top > 0.f ? __builtin_amdgcn_frexp_expf(top) : 0;
      kq = __builtin_ldexpf(a.scale, 24 - 14 + e);
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        float sum = 0.f;
#pragma unroll
        for (int j = gr * SG; j < (gr + 1) * SG; ++j) {
          float x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            x[k] = from16<BF>(raw[j][k / 2] >> (16 * (k & 1)) & 0xffffu);
            sum += x[k];
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int sh = 14 - e - ((k & 1) ? 4 : 0);
            qf[j][k] = pack_f16(__builtin_ldexpf(x[kSlotDim[2 * k]], sh), __builtin_ldexpf(x[kSlotDim[2 * k + 1]], sh));
          }
        }
        sum = sum_rows(sum);
        qz[gr] = sum * a.scale;
      }
    }
    // tokens that every row sees
    const int last = min(rows - 1, rt * RT + RT - 1);
    const int all_hi = a.causal ? min(s.len, s.len - s.n + rt * RT / a.ratio + 1) : s.len;
    const int all_lo = a.window ? s.len - s.n + last / a.ratio - a.window + 1 : 0;

    float mx = 0.f, l = 0.f, zs[NG], ps[NG];
    bool fresh = true;                              // the row has seen no token: mx is not set
    f32x4 o[TILES];
    // The row's products of weight and value scale enter the matrix products times inv, a power of two for each
    // group: the largest so far stands between 2^6 and kTop, whatever the scales are, whichever token has
    // the largest score, and however the groups differ.
    float inv[NG];
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      zs[gr] = ps[gr] = 0.f;
      inv[gr] = 0x1p126f;
    }
#pragma unroll
    for (int i = 0; i < TILES; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};

    auto compute = [&](int j, StepT& st, auto scored) {
      const int t0 = ts + T * (wave + W * j);
      // S^T, then scores in bits less the row's running maximum
      float u[ST][4];
#pragma unroll
      for (int x = 0; x < ST; ++x)
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          f32x4 acc;
#pragma unroll
          for (int f = F == 1 ? x : 0; f < (F == 1 ? x + 1 : SUB); ++f) {
            f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = gr * SG; i < (gr + 1) * SG; ++i) c = mfma(codes8(st.k[f][i]), qf[i], c);
            // with F > 1 a lane keeps the subtile of its column group
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[r] = F == 1 || f == 0 || fcol == f ? c[r] : acc[r];
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const unsigned w = st.kp[x][gr][r];
            const float v = __builtin_fmaf(par_zero<BF>(w), qz[gr], gr ? u[x][r] : -mx);
            u[x][r] = __builtin_fmaf(par_scale<BF>(w) * kq, acc[r], v);
          }
        }
      scored();                                     // the keys' registers are free
      if (t0 + T > min(all_hi, te) || t0 < all_lo) {
        // a token that the lane's row does not see: weight 0, and its parameters (any bits) are put away
#pragma unroll
        for (int x = 0; x < ST; ++x)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int t = t0 + 16 * (F == 1 ? x : fcol) + 4 * g + r;
            if (!(t >= see_lo && t < see_hi && t < te)) {
              u[x][r] = -__builtin_inff();
#pragma unroll
              for (int gr = 0; gr < NG; ++gr) st.vp[x][gr][r] = 0u;
            }
          }
      }
      float high = u[0][0];
#pragma unroll
      for (int x = 0; x < ST; ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r) high = __builtin_fmaxf(high, u[x][r]);
      if (__any(high > (fresh ? -__builtin_inff() : kSlack))) {
        // set or move the running maxima that need it, rescale what is summed so far
        const float top = max_rows(high);
        // a row's maximum moves for its own scores only: its result does not depend on its neighbours
        const bool go = top > (fresh ? -__builtin_inff() : kSlack), moved = go && !fresh;
        const float by = go ? top : 0.f, al = moved ? exp2_fast(-by) : 1.f;
        fresh = fresh && !go;
        mx += by;
        l *= al;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          zs[gr] *= al;
          // the products so far became smaller by 2^by: inv takes up the whole powers of two
          const int up = moved ? (int)__builtin_fminf(by, 126.f - (float)exponent_of(inv[gr])) : 0;
          inv[gr] = __builtin_ldexpf(inv[gr], up);
          const float ab = exp2_fast((float)up - (moved ? by : 0.f));
          ps[gr] *= ab;
#pragma unroll
          for (int i = gr * TG; i < (gr + 1) * TG; ++i) o[i] *= ab;
        }
#pragma unroll
        for (int x = 0; x < ST; ++x)
#pragma unroll
          for (int r = 0; r < 4; ++r) u[x][r] -= by;
      }
#pragma unroll
      for (int x = 0; x < ST; ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          u[x][r] = exp2_fast(u[x][r]);
          l += u[x][r];
        }
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        unsigned pk[ST][2];
        float w[ST][4], big = 0.f;
#pragma unroll
        for (int x = 0; x < ST; ++x)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const unsigned v = st.vp[x][gr][r];
            const float sc = par_scale<BF>(v);
            w[x][r] = u[x][r] * sc * inv[gr];
            big = __builtin_fmaxf(big, __builtin_fabsf(w[x][r]));
            zs[gr] = __builtin_fmaf(u[x][r], __builtin_fmaf(sc, 8.f, par_zero<BF>(v)), zs[gr]);
          }
        if (__any(big > kTop)) {                    // set or lower the unit of the rows that need it
          big = 0.f;
#pragma unroll
          for (int x = 0; x < ST; ++x)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              big = __builtin_fmaxf(big, __builtin_fabsf(u[x][r] * par_scale<BF>(st.vp[x][gr][r])));
          big = max_rows(big);
          const int down = big * inv[gr] > kTop ? max(8 - __builtin_amdgcn_frexp_expf(big), -126) - exponent_of(inv[gr]) : 0;
          const float by = __builtin_ldexpf(1.f, down);
          inv[gr] = __builtin_ldexpf(inv[gr], down);
          ps[gr] *= by;
#pragma unroll
          for (int i = gr * TG; i < (gr + 1) * TG; ++i) o[i] *= by;
#pragma unroll
          for (int x = 0; x < ST; ++x)
#pragma unroll
            for (int r = 0; r < 4; ++r) w[x][r] = u[x][r] * par_scale<BF>(st.vp[x][gr][r]) * inv[gr];
        }
#pragma unroll
        for (int x = 0; x < ST; ++x) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // rounded to 11 bits, and summed as rounded: the codes' middle is taken out exactly
            pk[x][h] = pack_f16(w[x][2 * h], w[x][2 * h + 1]);
            ps[gr] = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, pk[x][h]), f16x2{(_Float16)1.f, (_Float16)1.f},
                                            ps[gr], false);
          }
        }
        // O^T += V^T P^T, two subtiles at a time
#pragma unroll
        for (int pr = 0; pr < SUB / 2; ++pr) {
          u32x4 bp;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if constexpr (F == 1) {
              bp[h] = pk[0][h];
              bp[2 + h] = pk[ST - 1][h];
            } else {
              bp[h] = fcol == 2 * pr ? pk[0][h] : 0u;
              bp[2 + h] = fcol == 2 * pr + 1 ? pk[0][h] : 0u;
            }
          }
#pragma unroll
          for (int i = gr * TG; i < (gr + 1) * TG; ++i) {
            unsigned x0, x1, y0, y1;
            v_pairs<U>(st.v[2 * pr], i, x0, x1);
            v_pairs<U>(st.v[2 * pr + 1], i, y0, y1);
            o[i] = mfma(u32x4{x0, x1, y0, y1}, bp, o[i]);
          }
        }
      }
    };
    if constexpr (StepT::kTwo) {
      // two steps' registers: the next step is loaded as a whole before this one is worked on
      StepT sb;
      for (int j = 0; j < mine; j += 2) {
        // PER is even, so only the step after an odd one can need new pages
        if (j + 1 < mine) fetch(j + 1, sb);
        compute(j, sa, [] {});
        if (j + 2 < mine) {
          if ((j + 2) % PER == 0) pages(j + 2);
          fetch(j + 2, sa);
        }
        if (j + 1 < mine) compute(j + 1, sb, [] {});
      }
    } else {
      // one step's: the next keys are loaded once the scores are there, the next values at the end
      for (int j = 0; j < mine; ++j) {
        compute(j, sa, [&] {
          if (j + 1 < mine) {
            if ((j + 1) % PER == 0) pages(j + 1);
            fetch_k(j + 1, sa);
          }
        });
        if (j + 1 < mine) fetch_v(j + 1, sa);
      }
    }

    // ---- join: the wavefront's sums over its lanes, the columns and wavefronts through LDS
    const bool whole = cnt == nu - over;
    // byte offset of a workgroup's partial: 0 for the head of its run, 1 for its tail
    const __amdgpu_buffer_rsrc_t parts = buffer_of(a.partials, 2 * grid * kSlot * 4);
    auto slot_of = [&](int w, int tail) { return (2 * w + tail) * kSlot * 4; };
    const int mydst = slot_of(wg, at ? 0 : 1);
    auto write_out = [&](int row, int d, f32x4 v, float sum) {
      const int gi = rt * RT + row;
      if (gi >= rows) return;
      const int i = gi / a.ratio, h = gi - i * a.ratio;
      const float r = sum == 0.f ? 0.f : 1.0f / sum;                 // 0: nothing was seen, v is 0 as well
      *reinterpret_cast<u32x2*>(a.out + (long long)(s.start + i) * a.os + (kvh * a.ratio + h) * D + d) =
          u32x2{pack2<BF>(v[0] * r, v[1] * r), pack2<BF>(v[2] * r, v[3] * r)};
    };
    l = sum_rows(l);
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      zs[gr] = sum_rows(zs[gr]);
      ps[gr] = sum_rows(ps[gr]);
    }
    __syncthreads();                                // the previous segment is done with LDS
    if (g == 0) {
      s_m[wave * 16 + m] = fresh ? kStart : mx;
      s_l[wave * 16 + m] = l;
    }
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
      const float up = (i & 1) ? 0x1p20f : 0x1p24f;
      f32x4 v;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        v[r] = __builtin_fmaf(__builtin_fmaf(o[i][r], up, -8.f * ps[i / TG]), __builtin_ldexpf(1.f, -exponent_of(inv[i / TG])),
                              zs[i / TG]);
      *reinterpret_cast<f32x4*>(&s_o[(wave * 16 + m) * kRowF + 16 * i + 4 * g]) = v;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < RT * (D / 4); e += 64 * W) {
      const int row = e / (D / 4), d = e % (D / 4) * 4;
      float top = kStart;
#pragma unroll
      for (int w = 0; w < W; ++w)
#pragma unroll
        for (int f = 0; f < F; ++f) top = __builtin_fmaxf(top, s_m[w * 16 + f * RT + row]);
      float sum = 0.f;
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < W; ++w)
#pragma unroll
        for (int f = 0; f < F; ++f) {
          const int c = w * 16 + f * RT + row;
          const float sc = exp2_fast(s_m[c] - top);
          sum = __builtin_fmaf(s_l[c], sc, sum);
          v += *reinterpret_cast<const f32x4*>(&s_o[c * kRowF + d]) * sc;
        }
      if (whole) {
        write_out(row, d, v, sum);
      } else {
        store4(parts, mydst + (row * D + d) * 4, v);
        if (d == 0) store4(parts, mydst + (RT * D + 4 * row) * 4, f32x4{top, sum, 0.f, 0.f});
      }
    }
    if (!whole) {
      const int w0 = owner(first + over), w1 = owner(first + nu - 1);
      __builtin_amdgcn_s_waitcnt(0);                // this thread's partial stores are complete
      __syncthreads();
      if (threadIdx.x == 0)
        s_last = __hip_atomic_fetch_add(a.tickets + w0, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                 (unsigned)(w1 - w0);
      __syncthreads();
      if (s_last) {
        constexpr int kItems = RT * (D / 4), kTeams = kItems < 64 * W ? 64 * W / kItems : 1;
        const int team = threadIdx.x / kItems;      // teams take every kTeams-th piece
        for (int e = threadIdx.x % kItems; e < kItems; e += 64 * W) {
          const int row = e / (D / 4), d = e % (D / 4) * 4;
          float top = kStart, sum = 0.f;
          f32x4 v = {0.f, 0.f, 0.f, 0.f};
          auto add = [&](f32x4 x, float xm, float xs) {
            const float nm = __builtin_fmaxf(top, xm);
            const float old = exp2_fast(top - nm), sc = exp2_fast(xm - nm);
            top = nm;
            sum = sum * old + xs * sc;
            v = v * old + x * sc;
          };
          for (int p0 = w0 + team; p0 <= w1; p0 += 8 * kTeams) {     // eight pieces' loads in flight
            f32x4 ml[8], x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int w = min(p0 + k * kTeams, w1);
              // a segment's first piece is the tail of its workgroup's run, the others are heads of theirs
              const int from = slot_of(w, w == w0);
              ml[k] = load4(parts, from + (RT * D + 4 * row) * 4);
              x[k] = load4(parts, from + (row * D + d) * 4);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (p0 + k * kTeams <= w1) add(x[k], ml[k][0], ml[k][1]);
          }
          if constexpr (kTeams > 1) {
            __syncthreads();
            float* mine_o = s_o + 6 * threadIdx.x;
            mine_o[0] = top;
            mine_o[1] = sum;
#pragma unroll
            for (int r = 0; r < 4; ++r) mine_o[2 + r] = v[r];
            __syncthreads();
            if (team == 0) {
#pragma unroll
              for (int t = 1; t < kTeams; ++t) {
                const float* x = s_o + 6 * (threadIdx.x + t * kItems);
                add(f32x4{x[2], x[3], x[4], x[5]}, x[0], x[1]);
              }
            }
          }
          if (team == 0) write_out(row, d, v, sum);
        }
        if (threadIdx.x == 0) __hip_atomic_store(a.tickets + w0, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      __syncthreads();
    }
    u0 += take;
  }
}

template <bool BF, int D, int NG, int W>
hipError_t launch_waves(const AttnPlan& pl, const AttnArgs& a, hipStream_t s) {
  const dim3 grid(pl.grid), block(64 * W);
  if (pl.pack == 4) {
    if constexpr (D < 256) attention_rows<BF, D, NG, 4, W><<<grid, block, 0, s>>>(a);
  } else if (pl.pack == 2) {
    attention_rows<BF, D, NG, 2, W><<<grid, block, 0, s>>>(a);
  } else {
    if constexpr (D < 256 || NG < 4) attention_rows<BF, D, NG, 1, W><<<grid, block, 0, s>>>(a);
  }
  return hipGetLastError();
}
template <bool BF, int D, int NG>
hipError_t launch_groups(const AttnPlan& pl, const AttnArgs& a, hipStream_t s) {
  return pl.waves == 1 ? launch_waves<BF, D, NG, 1>(pl, a, s) : launch_waves<BF, D, NG, 4>(pl, a, s);
}

}  // namespace

template <bool BF, int D>
hipError_t launch_rows(const AttnPlan& pl, const AttnArgs& a, hipStream_t s) {
  if (pl.groups == 1) return launch_groups<BF, D, 1>(pl, a, s);
  if (pl.groups == 2) return launch_groups<BF, D, 2>(pl, a, s);
  if constexpr (D > 64) return launch_groups<BF, D, 4>(pl, a, s);
  return hipErrorInvalidValue;
}

#ifndef QGEMM_ATTN_UNIT
#error "compiled once per element type and head dim: QGEMM_ATTN_UNIT = 3 * bf16 + (0, 1, 2 for head dim 64, 128, 256)"
#endif
template hipError_t launch_rows<(QGEMM_ATTN_UNIT >= 3), (64 << (QGEMM_ATTN_UNIT % 3))>(const AttnPlan&, const AttnArgs&,
                                                                                    hipStream_t);

}  // namespace attn
}  // namespace qgemm
