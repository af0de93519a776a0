// Attention with many query rows per kv head (prompts, chunks of prompts): query rows over the
// wavefronts, the cache's tokens shared by a workgroup through LDS.
//
// Bound by arithmetic: 4 D operations per visible (row, token) pair on the matrix cores, beside about
// ten vector operations per pair for the softmax, which is what takes longer.  A workgroup holds
// BM = 16 NC NW query rows of one kv head (row = query * ratio + head, so the heads of a group share
// the tokens' codes) and walks 64 tokens at a time.  The wavefronts turn the packed codes of the
// next 64 tokens into MFMA operands once, in LDS, while the
// current ones are read by all (K in two buffers, V in three, one barrier per step).  O^T, the running
// maxima and the sums stay in registers.  The products of the next 32 tokens' keys are issued beside
// the softmax of the current 32, so that the matrix cores and the vector units work at once.
//
// A prompt of 8192 queries of 32 heads of 128, fp16, causal: 679 us, 810 TFLOP/s (plain fp16 products of
// 8192^3 reach 1164 on the same card).  Of its cycles the matrix cores work 32% and the vector units 58%,
// with two wavefronts on a SIMD: what is left to gain is their overlap.
//
// The reference mx of a row bounds score + log2(value scale), in bits, of the tokens it has seen, less kStand:
// w = 2^(score - mx) * scale then fits fp16 whatever the scales are, at no cost per token, and
// 2^-mx drops out with the sum.  mx follows scales down to 2^-60; scales beyond 2^60 (bf16 only) put
// O into units of 2^64, and ones below 2^-60 put it into units of 2^-64.
#include <type_traits>

#include "qgemm_attention_device.h"

namespace qgemm {
namespace attn {
namespace {

// scores may exceed their reference by this many bits less the exponent of the step's largest scale: weights
// stay below 2^15, inside fp16
constexpr int kRoom = 15, kRoomMax = 60;
// Where a reference puts the largest weight of its tokens: 2^6 to 2^7.  Weights down to 2^-20 of that keep 11 bits,
// down to 2^-31 they count, and larger ones have eight bits before the reference moves (with seven, chunks in a window
// take 404 us instead of 398).
constexpr int kStand = 7;
// the largest unit of a token's keys or values, as bits: its reciprocal is a normal number
constexpr unsigned kUnitMost = 0x7e800000u;
// Query rows whose largest lies in [2^-5, 2^6): their elements keep 11 bits down to 2^-13 of the largest and
// are rounded to 2^-24 of it at worst, which is what a 32-bit sum keeps.
constexpr int kQueryExp = 6, kQueryBand = 10;

template <bool BF, int D, int NG, int NC, int NW>
__global__ __launch_bounds__(64 * NW, NW / 4) void attention_tiles(AttnArgs a) {
  constexpr int U = D / 32, TILES = D / 16, TG = TILES / NG, SG = U / NG;
  constexpr int BM = 16 * NC * NW, NT = 64 * NW;
  constexpr int kHalves = D == 256 ? 1 : 2, kStep = 32 * kHalves;  // 32-token halves and tokens of a step
  // One body for both halves where two would spill registers (fp16, D 128 in two groups: a prompt of 4096
  // 300 -> 275 us; elsewhere two are better, D 128 in one group 184 against 205).  With the skew below 236.
  constexpr int kBodies = !BF && D == 128 && NG == 2 ? 1 : kHalves;
  constexpr int SUBS = 2 * kHalves;                 // 16-token subtiles of a step
  constexpr int KB = kStep * D * 2, PB = SUBS * NG * 4 * 16 * 4;   // bytes of K (and of V) operands, of parameters
  constexpr int kSlot = BM * D + NC * NT * 4;       // floats of a partial
  // bf16: fp16 operands hold the values themselves, a power of two per token apart; fp16: the codes
  constexpr bool kDeq = BF;
  // and in several groups K's operands hold (code - 8) * scale, a power of two per token apart: a 3-bit times
  // an 8-bit number fits fp16's 11 bits (down to scales of 2^-25 of the token's largest), so one accumulator
  // serves all groups and twice the rows fit the registers (a prompt of 4096, D 128: four groups 388 -> 234
  // us, D 256: 447 -> 278)
  constexpr bool kDeqK = kDeq && NG > 1;
  constexpr int AG = kDeqK ? 1 : NG;                // accumulators of a score
  __shared__ __align__(16) uint8_t s_k[2][KB], s_v[3][KB];
  // [subtile][group][K scale, K zero, V scale, V middle][16]; kDeq: one V scale per token, in group 0, and
  // in the place of the middle 0, or NaN where the group's parameters are not finite
  __shared__ __align__(16) float s_p[4][PB / 4];
  __shared__ __align__(16) unsigned s_w[2][kDeq ? SUBS * NG * 16 : 4];       // kDeq: V scale, zero as fp16
  __shared__ unsigned s_kw[2][kDeqK ? SUBS * NG * 16 : 4];                   // kDeqK: K scale as fp16, twice
  __shared__ __align__(16) unsigned s_big[4][4];    // per subtile: the largest finite |V scale|, as its bits
  __shared__ int s_odd[4];                          // any V parameter that is not finite
  __shared__ __align__(16) float s_unit[NG];        // a power of two that V values of the group are held times
  __shared__ float s_fit[BM];                       // rows' factors on the products with K
  __shared__ int s_last;

  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;

  // ---- which rows: workgroups with the same kv head sit on the same XCD while heads divide by 8; the
  // row tiles are walked from the last, which sees most
  const int kvh = blockIdx.x % a.kv_heads, rest = blockIdx.x / a.kv_heads;
  const int split = rest % a.splits;
  int entry = rest / a.splits;
  auto queries_in = [&](int b) { return b < a.batch ? load_seq(a, b).n : 0; };
  auto tiles_in = [&](int n) { return (a.ratio * n + BM - 1) / BM; };
  int total = 0;
  unsigned claimed = 0;                             // more than total_q: nothing is computed
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    const int n = queries_in(b0 + lane);
    claimed = claim(claimed, wave_sum(n));
    total += wave_sum(tiles_in(n));
  }
  if (claimed > (unsigned)a.total_q || entry >= total) return;
  entry = total - 1 - entry;
  int b = 0, before = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    const int u = wave_scan(tiles_in(queries_in(b0 + lane)));
    const unsigned long long past = __ballot(before + u > entry);
    if (past) {
      const int l = __builtin_ctzll(past);
      b = b0 + l;
      before += l ? __builtin_amdgcn_readlane(u, l - 1) : 0;
      break;
    }
    before += __builtin_amdgcn_readlane(u, 63);
  }
  b = __builtin_amdgcn_readfirstlane(b);
  before = __builtin_amdgcn_readfirstlane(before);
  const Seq s = load_seq(a, b);
  const int rows = a.ratio * s.n, row0 = (entry - before) * BM;
  const int past = s.len - s.n;                     // position of query 0
  const int row_end = min(rows, row0 + BM);
  const Tile tile = tile_of(s, row0, row_end, BM, a.ratio, a.causal, a.window, kStep, a.splits);
  const int active = tile.active;
  if (split >= active) return;
  const int ts = tile.lo + kStep * tile.per * split, te = min(tile.hi, ts + kStep * tile.per);
  const int steps = te > ts ? (te - ts + kStep - 1) / kStep : 0;

  // ---- filling: wavefront w prepares part w / SUBS of the K and V operands of subtile w % SUBS; two
  // wavefronts also the parameters, a token a lane, a step further ahead (the V operands need them)
  constexpr int PARTS = NW / SUBS, KP = U / PARTS, TP = TILES / PARTS;
  const int fsub = wave % SUBS, part = wave / SUBS;
  const bool fp = wave < 2, fpv = wave == 1;        // K's, V's
  unsigned rk[KP], rv[U == 2 ? 2 : 4], rp[NG];
  bool rp_on = false;
  // Page ids are loaded one step before their blocks' addresses are needed: the subtile's (uniform), and
  // for the parameters the lane's token's.
  const int* row_of = a.table + (long long)b * a.max_pages;
  int pg_sub = 0, pg_tok = 0;
  auto sub_at = [&](int step) {                     // past the end: any subtile, masked
    return __builtin_amdgcn_readfirstlane(min(ts + kStep * step + 16 * fsub, (te - 1) & ~15));
  };
  auto tok_at = [&](int step) { return min(ts + kStep * step + lane % kStep, te - 1); };
  auto block_of = [&](int t, int pg, int& in) {
    in = t - page_of(a, t) * a.page;
    if ((unsigned)pg >= (unsigned)a.num_pages) pg = 0;
    return a.data + ((long long)pg * a.kv_heads + kvh) * a.block;
  };
  auto load_n = [&](const uint8_t* p, unsigned* w, auto n_c) {
    constexpr int n = decltype(n_c)::value;
    if constexpr (n == 1) {
      w[0] = *reinterpret_cast<const unsigned*>(p);
    } else if constexpr (n == 2) {
      const u32x2 x = *reinterpret_cast<const u32x2*>(p);
      w[0] = x[0];
      w[1] = x[1];
    } else {
      const u32x4 x = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = x[i];
    }
  };
  auto fetch_pages = [&](int step) { pg_sub = row_of[page_of(a, sub_at(step))]; };
  auto fetch = [&](int step) {
    int in;
    const uint8_t* blk = block_of(sub_at(step), pg_sub, in);
    load_n(blk + (in * (D / 2) + (m * (D / 2) + 4 * U * g + 4 * KP * part)), rk, std::integral_constant<int, KP>{});
    const uint8_t* vb = blk + a.codes + (in * (D / 2) + lane * (4 * U));
    if constexpr (U <= 4) {
      load_n(vb, rv, std::integral_constant<int, U>{});
    } else {                                        // of each token's two dwords the one that holds the part
#pragma unroll
      for (int t = 0; t < 4; ++t) rv[t] = *reinterpret_cast<const unsigned*>(vb + 8 * t + 4 * (TP == 4 ? part >> 1 : part));
    }
    fetch_pages(step + 1);
  };
  auto fetch_par_pages = [&](int step) {
    if (fp) pg_tok = row_of[page_of(a, tok_at(step))];
  };
  auto fetch_par = [&](int step) {
    if (!fp) return;
    int in;
    const int t = ts + kStep * step + lane % kStep;
    rp_on = t >= tile.seen && t < te;
    const uint8_t* pb = block_of(tok_at(step), pg_tok, in) + 2 * a.codes + (fpv ? a.params : 0);
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) rp[gr] = *reinterpret_cast<const unsigned*>(pb + 4 * (gr * a.page + in));
    fetch_par_pages(step + 1);
  };
  float kq = 0.f;                                   // set below, before the first store
  auto store = [&](int step) {
    const int kb = step & 1, vb = step % 3;
#pragma unroll
    for (int i = 0; i < KP; ++i) {
      u32x4 c = codes8(rk[i]);
      if constexpr (kDeqK) {
        const f16x2 sc = __builtin_bit_cast(f16x2, s_kw[step & 1][(fsub * NG + (part * KP + i) / SG) * 16 + m]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          c[k] = __builtin_bit_cast(unsigned, __builtin_bit_cast(f16x2, centre(c[k], k & 1)) * sc);
      }
      *reinterpret_cast<u32x4*>(&s_k[kb][((fsub * U + part * KP + i) * 64 + lane) * 16]) = c;
    }
    // pairs of tokens (0, 1) and (2, 3): 16 bits each of the part's nibbles
    constexpr int HW = TP == 8 ? 2 : 1;
    unsigned x[HW], y[HW];
    if constexpr (U == 2) {
      x[0] = rv[0] >> (8 * part);
      y[0] = rv[1] >> (8 * part);
    } else {
#pragma unroll
      for (int h = 0; h < HW; ++h) {
        const unsigned sel = (HW == 2 ? h : part & 1) ? 0x07060302u : 0x05040100u;
        x[h] = __builtin_amdgcn_perm(rv[1], rv[0], sel);
        y[h] = __builtin_amdgcn_perm(rv[3], rv[2], sel);
      }
    }
    constexpr int GP = TP <= TG ? 1 : TP / TG;      // groups of a part
    const int gr0 = part * TP / TG;
#pragma unroll
    for (int gg = 0; gg < GP; ++gg) {
      f16x2 s01, s23, z01, z23;
      if constexpr (kDeq) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(&s_w[step & 1][(fsub * NG + gr0 + gg) * 16 + 4 * g]);
        s01 = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(w[1], w[0], 0x05040100u));
        z01 = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(w[1], w[0], 0x07060302u));
        s23 = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(w[3], w[2], 0x05040100u));
        z23 = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(w[3], w[2], 0x07060302u));
      }
#pragma unroll
      for (int ii = gg * (TP / GP); ii < (gg + 1) * (TP / GP); ++ii) {
        const unsigned msk = (ii & 1) ? kHigh : kLow;
        const unsigned px = ((ii & 2) ? x[ii >> 2] >> 8 : x[ii >> 2]) & msk, py = ((ii & 2) ? y[ii >> 2] >> 8 : y[ii >> 2]) & msk;
        u32x2 v;
        if constexpr (kDeq) {
          v = u32x2{__builtin_bit_cast(unsigned, __builtin_elementwise_fma(whole(px, ii & 1), s01, z01)),
                    __builtin_bit_cast(unsigned, __builtin_elementwise_fma(whole(py, ii & 1), s23, z23))};
        } else {
          v = u32x2{centre(px, ii & 1), centre(py, ii & 1)};
        }
        *reinterpret_cast<u32x2*>(&s_v[vb][(((fsub >> 1) * TILES + part * TP + ii) * 64 + lane) * 16 + (fsub & 1) * 8]) = v;
      }
    }
  };
  // Groups of dims whose values differ in size (a few channels far out, in every token) would share one
  // reference, or in bf16 one unit of each token.  Each group's values are divided by a power of two that brings
  // its ordinary scale, the mean exponent over the first step's tokens, down to that of the smallest group; O takes it
  // back at the end.  A token that is far out by itself changes the mean little.
  constexpr int kApart = 40;
  auto set_units = [&] {
    if (NG == 1 || !fpv) return;
    int mean[NG], low = 255;
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      const float sc = __builtin_fabsf(par_scale<BF>(rp[gr])), z = __builtin_fabsf(par_zero<BF>(rp[gr]));
      const unsigned size = __builtin_bit_cast(unsigned, kDeq ? __builtin_fmaxf(z, 16.f * sc) : sc) >> 23;
      const int sum = wave_sum(rp_on && size - 1u < 254u ? (int)size | 1 << 16 : 0);        // exponents, and how many
      mean[gr] = sum ? (int)((float)(sum & 0xffff) / (float)(sum >> 16)) : -1;
      low = min(low, sum ? mean[gr] : 255);
    }
    if (lane == 0)
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) s_unit[gr] = __builtin_ldexpf(1.f, mean[gr] < 0 ? 0 : -min(mean[gr] - low, kApart));
  };
  auto store_par = [&](int step) {
    if (!fp) return;
    const int pb = step & 3;
    float sc[NG], z[NG];
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      sc[gr] = par_scale<BF>(rp[gr]);
      z[gr] = par_zero<BF>(rp[gr]);
    }
    if (!fpv) {
      if constexpr (kDeqK) {
        // the token's unit 2^e, at most its largest scale; that scale becomes 2^11 to 2^12
        unsigned big = 0x00800000u;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          z[gr] = __builtin_fmaf(sc[gr], 8.f, z[gr]);
          if (!(__builtin_fabsf(z[gr]) < __builtin_inff())) {
            sc[gr] = 0.f;
            z[gr] = __builtin_nanf("");
          }
          big = max(big, __builtin_bit_cast(unsigned, __builtin_fabsf(sc[gr])));
        }
        big = min(big & 0x7f800000u, kUnitMost);
        const float back = __builtin_bit_cast(float, 0x7f000000u - big);
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          const float w = sc[gr] * back * 2048.f;
          if (lane < kStep) s_kw[step & 1][((lane >> 4) * NG + gr) * 16 + (lane & 15)] = pack_f16(w, w);
        }
        sc[0] = __builtin_bit_cast(float, big) * kq;
      } else {
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) sc[gr] *= kq;
      }
    } else {
      unsigned big = 0;                             // magnitudes compare as their bits do
      bool odd = false;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        if (!rp_on) sc[gr] = z[gr] = 0.f;           // no token: its bits must not multiply
        const float mid = __builtin_fmaf(sc[gr], 8.f, z[gr]);
        const bool fine = __builtin_fabsf(mid) < __builtin_inff();
        odd |= !fine;
        if constexpr (NG > 1) sc[gr] *= s_unit[gr];
        if constexpr (kDeq) {
          if constexpr (NG > 1) z[gr] *= s_unit[gr];
          sc[gr] = fine ? sc[gr] : 0.f;
          z[gr] = fine ? z[gr] : __builtin_nanf("");
          const float far = __builtin_fmaxf(__builtin_fabsf(z[gr]), 16.f * __builtin_fabsf(sc[gr]));
          big = max(big, fine ? __builtin_bit_cast(unsigned, far) : 0u);
        } else {
          z[gr] = mid;
          big = max(big, fine ? __builtin_bit_cast(unsigned, __builtin_fabsf(sc[gr])) : 0u);
        }
      }
      if constexpr (kDeq) {
        // the token's unit 2^e, at most its largest value's bound; values stay below 8 of it
        big = min(big & 0x7f800000u, kUnitMost);
        const float unit = __builtin_bit_cast(float, big), back = __builtin_bit_cast(float, 0x7f000000u - big);
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          const bool fine = __builtin_fabsf(z[gr]) < __builtin_inff();
          const unsigned w = pack_f16(sc[gr] * back, fine ? z[gr] * back : 0.f);
          if (lane < kStep) s_w[step & 1][((lane >> 4) * NG + gr) * 16 + (lane & 15)] = w;
          z[gr] = fine ? 0.f : __builtin_nanf("");
        }
        sc[0] = unit;
      }
      odd = __any(odd);
      big = max(big, dpp<0x128>(big));              // row_ror 8, 4, 2, 1: over the subtile's 16 lanes
      big = max(big, dpp<0x124>(big));
      big = max(big, dpp<0x122>(big));
      big = max(big, dpp<0x121>(big));
      if ((lane & 15) == 0) s_big[pb][lane >> 4] = big;
      if (lane == 0) s_odd[pb] = odd;
    }
    if (lane < kStep) {
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        float* p = &s_p[pb][(((lane >> 4) * NG + gr) * 4 + (fpv ? 2 : 0)) * 16 + (lane & 15)];
        p[0] = sc[gr];
        p[16] = z[gr];
      }
    }
  };

  // ---- queries
  u32x4 qf[U][NC];
  float qz[NC][NG];
  int see_lo[NC], see_hi[NC];
  // A row's queries enter the products times 2^(14 - e), a rule of the row alone: rows of ordinary size share e =
  // kQueryExp, which is part of the keys' factor; others have their products multiplied by 2^(e - kQueryExp) in a wavefront that
  // holds such a row.
  bool wide = false;
  {
    u32x4 raw[NC][U];
    float top[NC];
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      top[nc] = 0.f;
      const int row = row0 + (wave * NC + nc) * 16 + m;
      const bool on = row < rows;
      const int i = on ? row / a.ratio : 0, h = row - i * a.ratio;
      const int pos = past + i;
      see_hi[nc] = a.causal ? min(pos + 1, s.len) : s.len;
      see_lo[nc] = a.window ? pos - a.window + 1 : 0;
      const uint16_t* src = a.q + (long long)(s.start + i) * a.qs + (kvh * a.ratio + h) * D + 8 * g;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        raw[nc][j] = on ? *reinterpret_cast<const u32x4*>(src + 32 * j) : u32x4{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const float x = __builtin_fabsf(from16<BF>(raw[nc][j][e] >> (16 * o) & 0xffffu));
            top[nc] = x < __builtin_inff() ? __builtin_fmaxf(top[nc], x) : top[nc];
          }
      }
    }
    if (steps) {
      fetch_pages(0);
      fetch_par_pages(0);
      fetch(0);
      fetch_par(0);
    }
    kq = __builtin_ldexpf(a.scale, (kDeqK ? -11 : 24) - 14 + kQueryExp);
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      // the row's largest is f 2^e, f in [1/2, 1)
      top[nc] = max_rows(top[nc]);
      int e = top[nc] > 0.f ? __builtin_amdgcn_frexp_expf(top[nc]) : kQueryExp;
      if (e >= kQueryExp - kQueryBand && e < kQueryExp) e = kQueryExp;
      wide |= e != kQueryExp;
      if (g == 0) s_fit[(wave * NC + nc) * 16 + m] = __builtin_ldexpf(1.f, e - kQueryExp);
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        float sum = 0.f;
#pragma unroll
        for (int j = gr * SG; j < (gr + 1) * SG; ++j) {
          float x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            x[k] = from16<BF>(raw[nc][j][k / 2] >> (16 * (k & 1)) & 0xffffu);
            sum += x[k];
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int sh = 14 - e - (!kDeqK && (k & 1) ? 4 : 0);
            qf[j][nc][k] = pack_f16(__builtin_ldexpf(x[kSlotDim[2 * k]], sh), __builtin_ldexpf(x[kSlotDim[2 * k + 1]], sh));
          }
        }
        sum = sum_rows(sum);
        qz[nc][gr] = sum * a.scale;
      }
    }
  }
  wide = __any(wide);
  // tokens that the wavefront's rows all see
  const int first = row0 + wave * 16 * NC, last = min(rows - 1, first + 16 * NC - 1);
  const bool idle = first >= rows;
  const int all_hi = a.causal ? min(s.len, past + first / a.ratio + 1) : s.len;
  const int all_lo = a.window ? past + last / a.ratio - a.window + 1 : 0;

  // zs: the sums of weight times middle; kDeq: which groups of the row have met a NaN
  constexpr int ZG = kDeq ? 1 : NG;
  float mx[NC], l[NC], zs[NC][ZG];
  unsigned bad[NC];
  bool fresh[NC];                                   // the row has seen no token: mx is not set
  f32x4 o[NC][TILES];
  int tau = -64;                                    // O is in units of 2^tau
#pragma unroll
  for (int nc = 0; nc < NC; ++nc) {
    mx[nc] = l[nc] = 0.f;
    fresh[nc] = true;
    bad[nc] = 0;
#pragma unroll
    for (int gr = 0; gr < ZG; ++gr) zs[nc][gr] = 0.f;
#pragma unroll
    for (int i = 0; i < TILES; ++i) o[nc][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  auto par = [&](int step, int pr, int x, int gr, int c) {
    return *reinterpret_cast<const f32x4*>(&s_p[step & 3][(((2 * pr + x) * NG + gr) * 4 + c) * 16 + 4 * g]);
  };
  typedef f32x4 Acc[2][AG][NC];
  // the products of one half's keys with the rows
  auto products = [&](int step, int pr, Acc& acc) {
    const uint8_t* src = s_k[step & 1];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const u32x4 kf = *reinterpret_cast<const u32x4*>(src + (((2 * pr + x) * U + i) * 64 + lane) * 16);
#pragma unroll
        for (int nc = 0; nc < NC; ++nc) {
          constexpr int AS = U / AG;
          f32x4& c = acc[x][i / AS][nc];
          c = mfma(kf, qf[i][nc], i % AS == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : c);
        }
      }
  };
  float u[NC][2][4];                                // scores in bits less the row's reference, of the half that comes next
  auto score = [&](int step, int pr, const Acc& acc) {
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        const f32x4 sc = par(step, pr, x, kDeqK ? 0 : gr, 0), z = par(step, pr, x, gr, 1);
#pragma unroll
        for (int nc = 0; nc < NC; ++nc)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float v = __builtin_fmaf(z[r], qz[nc][gr], gr ? u[nc][x][r] : -mx[nc]);
            u[nc][x][r] = kDeqK && gr < NG - 1 ? v : __builtin_fmaf(sc[r], acc[x][kDeqK ? 0 : gr][nc][r], v);
          }
      }
  };
  auto fit = [&](Acc& acc) {
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      const float f = s_fit[(wave * NC + nc) * 16 + m];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int gr = 0; gr < AG; ++gr) acc[x][gr][nc] *= f;
    }
  };
  // A half's weights, as B operands, while the next half's products with K run beside them (into
  // buffers that exist even after the last half: its scores are not used).  kMask: a weight of 0 must
  // not meet a parameter that is not finite, or O's unit is not 1, or the products take the rows' factors.
  unsigned seen[NC];
  constexpr int WG = kDeq ? 1 : NG;                 // weights of a token: one, or one per group
  typedef u32x4 Weights[WG][NC];
  auto weights = [&](auto mask_c, int step, int pr, int nstep, int npr, float tf, Acc& acc, Weights& bp) {
    constexpr bool kMask = decltype(mask_c)::value;
    products(nstep, npr, acc);
    if constexpr (kMask) fit(acc);
#pragma unroll
    for (int nc = 0; nc < NC; ++nc)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          u[nc][x][r] = exp2_fast(u[nc][x][r]);
          l[nc] += u[nc][x][r];
        }
#pragma unroll
    for (int gr = 0; gr < WG; ++gr)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        f32x4 sc = par(step, pr, x, gr, 2);
        if constexpr (kMask) sc *= tf;
        if constexpr (!kDeq || kMask) {
#pragma unroll
          for (int g2 = gr; g2 < (kDeq ? NG : gr + 1); ++g2) {
            const f32x4 md = par(step, pr, x, g2, 3);
#pragma unroll
            for (int nc = 0; nc < NC; ++nc)
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const bool on = !kMask || (seen[nc] >> (4 * x + r) & 1);
                if constexpr (kDeq) bad[nc] |= on && md[r] != md[r] ? 1u << g2 : 0u;
                else zs[nc][g2] = __builtin_fmaf(u[nc][x][r], on ? md[r] : 0.f, zs[nc][g2]);
              }
          }
        }
#pragma unroll
        for (int nc = 0; nc < NC; ++nc) {
          float w[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const bool on = !kMask || (seen[nc] >> (4 * x + r) & 1);
            w[r] = on ? u[nc][x][r] * sc[r] : 0.f;
          }
          // rounded to 11 bits
          bp[gr][nc][2 * x] = pack_f16(w[0], w[1]);
          bp[gr][nc][2 * x + 1] = pack_f16(w[2], w[3]);
        }
      }
  };
  // Where the scores' own operations weigh more than the products, the second wavefront of each SIMD passes
  // the step's barrier half a phase earlier in its work than the first, so that one's value products run
  // beside the other's softmax (D 128 in four groups bf16 234 -> 221, fp16 386 -> 379, in two fp16 275 -> 256;
  // in one group 183 -> 188, D 64 144 -> 148).  Every wavefront passes one barrier a step, after what it
  // stores of step j + 1 and after its last products with step j's keys.
  constexpr bool kSkew = D == 128 && NG > 1;
  const bool late = kSkew && __builtin_amdgcn_readfirstlane(wave) >= NW / 2;
  // One half, whose scores u holds.
  auto compute = [&](int step, int pr, int nstep, int npr) {
    const int tp = ts + kStep * step + 32 * pr, vb = step % 3;
    const u32x2 bb = *reinterpret_cast<const u32x2*>(&s_big[step & 3][2 * pr]);
    const unsigned big = __builtin_amdgcn_readfirstlane(max(bb[0], bb[1]));
    const bool odd = __builtin_amdgcn_readfirstlane(s_odd[step & 3]);
    const int e = big ? (int)(big >> 23) - 126 : -kRoomMax;            // scales are below 2^e
    const int unit = e > kRoomMax ? 64 : e < -kRoomMax ? -64 : 0;
    if (unit > tau) {                               // O only ever goes to larger units
      const float f = __builtin_ldexpf(1.f, tau - unit);
#pragma unroll
      for (int nc = 0; nc < NC; ++nc)
#pragma unroll
        for (int i = 0; i < TILES; ++i) o[nc][i] *= f;
      tau = unit;
    }
    const float tf = __builtin_ldexpf(1.f, -tau), room = (float)min(kRoomMax, kRoom - (e - tau));
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) seen[nc] = 255;
    if (tp + 32 > min(all_hi, te) || tp < all_lo || idle) {            // not every row sees every token
#pragma unroll
      for (int nc = 0; nc < NC; ++nc)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int t = tp + 16 * x + 4 * g + r;
            if (!(t >= see_lo[nc] && t < see_hi[nc] && t < te)) {
              seen[nc] &= ~(1u << (4 * x + r));
              u[nc][x][r] = -__builtin_inff();
            }
          }
    }
    bool move = false;
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      float high = u[nc][0][0];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r) high = __builtin_fmaxf(high, u[nc][x][r]);
      move |= high > (fresh[nc] ? -__builtin_inff() : room);
    }
    if (__any(move)) {
      // set or move the references that need it, rescale what is summed so far
#pragma unroll
      for (int nc = 0; nc < NC; ++nc) {
        float top = -__builtin_inff(), want = top;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          f32x4 sm = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int gr = 0; gr < WG; ++gr) {
            const f32x4 v = par(step, pr, x, gr, 2) * tf;
#pragma unroll
            for (int r = 0; r < 4; ++r) sm[r] = __builtin_fmaxf(sm[r], __builtin_fabsf(v[r]));
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float ls = sm[r] > 0.f ? (float)__builtin_amdgcn_frexp_expf(sm[r]) : -(float)kRoomMax;
            top = __builtin_fmaxf(top, u[nc][x][r]);
            want = __builtin_fmaxf(want, u[nc][x][r] + __builtin_fmaxf(ls, -(float)kRoomMax));
          }
        }
        top = max_rows(top);
        want = max_rows(want);
        // a row's reference moves for its own scores only: its result does not depend on its neighbours
        const bool go = top > (fresh[nc] ? -__builtin_inff() : room);
        want -= (float)kStand;
        const float by = go ? (fresh[nc] ? want : __builtin_fmaxf(want, 0.f)) : 0.f;
        const float al = fresh[nc] ? 1.f : exp2_fast(-by);
        fresh[nc] = fresh[nc] && !go;
        mx[nc] += by;
        l[nc] *= al;
#pragma unroll
        for (int gr = 0; gr < ZG; ++gr) zs[nc][gr] *= al;
#pragma unroll
        for (int i = 0; i < TILES; ++i) o[nc][i] *= al;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int r = 0; r < 4; ++r) u[nc][x][r] -= by;
      }
    }
    Acc acc;
    Weights bp;
    if (__builtin_expect(tau || odd || wide, 0)) weights(std::true_type{}, step, pr, nstep, npr, tf, acc, bp);
    else weights(std::false_type{}, step, pr, nstep, npr, tf, acc, bp);
    if (kSkew && pr == 0 && late) __syncthreads();
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
      const u32x4 vf = *reinterpret_cast<const u32x4*>(&s_v[vb][((pr * TILES + i) * 64 + lane) * 16]);
#pragma unroll
      for (int nc = 0; nc < NC; ++nc) o[nc][i] = mfma(vf, bp[kDeq ? 0 : i / TG][nc], o[nc][i]);
    }
    score(nstep, npr, acc);
  };

  // Step j + 1 is stored after every wavefront has passed the barrier of step j, so its K buffer (of step
  // j - 1, whose products were taken before that barrier) and its V buffer (of step j - 2) are free; the
  // parameters are stored a step earlier, into the buffer of step j - 2.
  if (steps) {
    set_units();
    store_par(0);
    if (steps > 1) fetch_par(1);
    __syncthreads();
    store(0);
    if (steps > 1) {
      fetch(1);
      store_par(1);
      if (steps > 2) fetch_par(2);
    }
    __syncthreads();
    {
      Acc acc;
      products(0, 0, acc);
      if (wide) fit(acc);
      score(0, 0, acc);
    }
    for (int j = 0; j < steps; ++j) {
      if (j + 1 < steps) {
        store(j + 1);
        if (j + 2 < steps) {
          fetch(j + 2);
          store_par(j + 2);
          if (j + 3 < steps) fetch_par(j + 3);
        }
      }
#pragma unroll kBodies
      for (int pr = 0; pr < kHalves; ++pr) {
        const bool end = pr == kHalves - 1;
        if (end && !late) __syncthreads();          // step j + 1's operands are in LDS
        compute(j, pr, j + end, end ? 0 : 1);
      }
    }
  }

  // ---- results: lane sums, then out, or a partial for the last split to join
#pragma unroll
  for (int nc = 0; nc < NC; ++nc) {
    l[nc] = sum_rows(l[nc]);
    if constexpr (kDeq) {
      bad[nc] |= __shfl_xor(bad[nc], 16);
      bad[nc] |= __shfl_xor(bad[nc], 32);
    } else {
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        zs[nc][gr] = sum_rows(zs[nc][gr]);
      }
    }
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
      const float back = __builtin_ldexpf(1.f, tau - (NG > 1 && steps ? exponent_of(s_unit[i / TG]) : 0));
      const float z = !kDeq ? zs[nc][kDeq ? 0 : i / TG] : bad[nc] >> (i / TG) & 1 ? __builtin_nanf("") : 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) o[nc][i][r] = __builtin_fmaf(o[nc][i][r], back, z);
    }
  }
#pragma unroll
  for (int nc = 0; nc < NC; ++nc) mx[nc] = fresh[nc] ? kStart : mx[nc];
  // Splits are joined in pairs, pairs of pairs and so on: at each node the second of two to arrive, its
  // part still in registers, adds the first's from the workspace and goes on; the first leaves.  Nobody
  // waits, and a sum of two has the same bits either way round, so the result does not depend on the order.
  if (active > 1) {
    const size_t parts_at = (size_t)(entry * a.kv_heads + kvh) * a.splits;
    unsigned* tickets = a.tickets + parts_at;
    float* base = a.partials + parts_at * kSlot;
    const __amdgpu_buffer_rsrc_t parts = buffer_of(base, a.splits * kSlot * 4);
    for (int i = split, size = 1; size < active; size *= 2, i >>= 1) {
      if ((i ^ 1) * size < active) {                // the node has two children
        const int mydst = i * size * kSlot * 4;
        // a node goes by the first part of its right child: that number's lowest set bit is `size`, so no
        // other node has it, and it is below `splits`
        unsigned* node = tickets + (i | 1) * size;
#pragma unroll
        for (int nc = 0; nc < NC; ++nc) {
#pragma unroll
          for (int x = 0; x < TILES; ++x) store4(parts, mydst + ((nc * TILES + x) * NT + threadIdx.x) * 16, o[nc][x]);
          store4(parts, mydst + (BM * D + (nc * NT + threadIdx.x) * 4) * 4, f32x4{mx[nc], l[nc], 0.f, 0.f});
        }
        __builtin_amdgcn_s_waitcnt(0);              // this thread's stores are complete
        __syncthreads();
        if (threadIdx.x == 0)
          s_last = __hip_atomic_fetch_add(node, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == 1u;
        __syncthreads();
        if (!s_last) return;
        if (threadIdx.x == 0) __hip_atomic_store(node, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const int from = (i ^ 1) * size * kSlot * 4;
#pragma unroll
        for (int nc = 0; nc < NC; ++nc) {
          const f32x4 ml = load4(parts, from + (BM * D + (nc * NT + threadIdx.x) * 4) * 4);
          const float nm = __builtin_fmaxf(mx[nc], ml[0]);
          const float mine = exp2_fast(mx[nc] - nm), other = exp2_fast(ml[0] - nm);
          mx[nc] = nm;
          l[nc] = l[nc] * mine + ml[1] * other;
#pragma unroll
          for (int x = 0; x < TILES; ++x)
            o[nc][x] = o[nc][x] * mine + load4(parts, from + ((nc * TILES + x) * NT + threadIdx.x) * 16) * other;
        }
      }
    }
  }
#pragma unroll
  for (int nc = 0; nc < NC; ++nc) {
    const int row = row0 + (wave * NC + nc) * 16 + m;
    if (row >= rows) continue;
    const int i = row / a.ratio, h = row - i * a.ratio;
    const float r = l[nc] == 0.f ? 0.f : 1.0f / l[nc];
    uint16_t* dst = a.out + (long long)(s.start + i) * a.os + (kvh * a.ratio + h) * D + 4 * g;
#pragma unroll
    for (int x = 0; x < TILES; ++x)
      *reinterpret_cast<u32x2*>(dst + 16 * x) =
          u32x2{pack2<BF>(o[nc][x][0] * r, o[nc][x][1] * r), pack2<BF>(o[nc][x][2] * r, o[nc][x][3] * r)};
  }
}

template <bool BF, int D, int NG>
hipError_t launch_groups(const AttnPlan& pl, const AttnArgs& a, hipStream_t s) {
  constexpr TileShape t = tile_shape(D, NG, BF);
  attention_tiles<BF, D, NG, t.cols, t.waves><<<dim3(pl.grid), dim3(64 * t.waves), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

template <bool BF, int D>
hipError_t launch_tiles(const AttnPlan& pl, const AttnArgs& a, hipStream_t s) {
  if (pl.groups == 1) return launch_groups<BF, D, 1>(pl, a, s);
  if (pl.groups == 2) return launch_groups<BF, D, 2>(pl, a, s);
  if constexpr (D > 64) return launch_groups<BF, D, 4>(pl, a, s);
  return hipErrorInvalidValue;
}

#ifndef QGEMM_ATTN_UNIT
#error "compiled once per element type and head dim: QGEMM_ATTN_UNIT = 3 * bf16 + (0, 1, 2 for head dim 64, 128, 256)"
#endif
template hipError_t launch_tiles<(QGEMM_ATTN_UNIT >= 3), (64 << (QGEMM_ATTN_UNIT % 3))>(const AttnPlan&, const AttnArgs&,
                                                                                     hipStream_t);

}  // namespace attn
}  // namespace qgemm
