// qgemm_attention: softmax(scale q . k^T) v over the 4-bit cache.
//
// With value = code * scale + zero, per group g of dims,
//   q . k_t = sum_g ks[t,g] (sum_{d in g} q_d c[t,d]) + kz[t,g] (sum_{d in g} q_d)
//   o_d     = sum_t p_t vs[t,g(d)] c[t,d] + sum_t p_t vz[t,g(d)]
// so the codes enter the products as the whole numbers they are and the parameters stay in fp32; a
// parameter of a token that a row does not see is never multiplied.
//
// One wavefront per (query token, query head): 64 tokens at a time, one a lane for the scores, the
// running maximum and sum of the softmax, then one dim a lane for the output.
#include <hip/hip_runtime.h>

#include "qgemm_attention_device.h"

namespace {

using namespace qgemm;

using namespace attn;

template <bool BF, int D, int NG>
__global__ __launch_bounds__(64) void attention_row(AttnArgs a) {
  constexpr int U = D / 32, G = D / NG, E = D / 64;
  __shared__ float sq[D], sp[64];
  __shared__ const uint8_t* sb[64];
  __shared__ int st[64];
  const int lane = threadIdx.x;
  const int row = blockIdx.x / a.q_heads, head = blockIdx.x % a.q_heads, kvh = head / a.ratio;
  // the row's sequence
  int b = -1;
  for (int i = 0; i < a.batch; ++i)
    if (row >= a.starts[i] && row < a.starts[i + 1]) { b = i; break; }
  if (b < 0) return;
  const int n = a.starts[b + 1] - a.starts[b];
  int len = a.lens[b];
  len = len < 0 ? 0 : len > a.max_pages * a.page ? a.max_pages * a.page : len;
  const int pos = len - n + (row - a.starts[b]);
  const int end = a.causal ? (pos + 1 < len ? pos + 1 : len) : len;
  const int begin = a.window && pos + 1 > a.window ? pos + 1 - a.window : 0;
  for (int d = lane; d < D; d += 64) sq[d] = from16<BF>(a.q[row * a.qs + head * D + d]);
  __syncthreads();
  float m = -1e30f, l = 0.f, o[E] = {}, zs[E] = {};
  for (int t0 = begin; t0 < end; t0 += 64) {
    const int t = t0 + lane;
    float s = -__builtin_inff();
    if (t < end) {
      int pg = a.table[(size_t)b * a.max_pages + t / a.page];
      if ((unsigned)pg >= (unsigned)a.num_pages) pg = 0;
      const uint8_t* blk = a.data + ((size_t)pg * a.kv_heads + kvh) * a.block;
      const int in = t % a.page;
      sb[lane] = blk;
      st[lane] = in;
      s = 0.f;
      for (int g = 0; g < NG; ++g) {
        float acc = 0.f, qsum = 0.f;
        for (int d = g * G; d < (g + 1) * G; ++d) {
          const int p = U * (d / 8 % 4) + d / 32;
          const unsigned c = blk[in * (D / 2) + 4 * p + d % 8 / 2] >> (4 * (d & 1)) & 15u;
          acc = __builtin_fmaf(sq[d], (float)c, acc);
          qsum += sq[d];
        }
        const unsigned par = *reinterpret_cast<const unsigned*>(blk + 2 * a.codes + (g * a.page + in) * 4);
        s += from16<BF>(par & 0xffffu) * acc + from16<BF>(par >> 16) * qsum;
      }
      s *= a.scale * 0.6931471805599453f;
    }
    float mt = s;
    for (int x = 1; x < 64; x *= 2) mt = __builtin_fmaxf(mt, __shfl_xor(mt, x));
    const float mn = __builtin_fmaxf(m, mt), corr = __expf(m - mn), p = t < end ? __expf(s - mn) : 0.f;
    m = mn;
    sp[lane] = p;
    float ps = p;
    for (int x = 1; x < 64; x *= 2) ps += __shfl_xor(ps, x);
    l = l * corr + ps;
    __syncthreads();
    const int cnt = end - t0 < 64 ? end - t0 : 64;
    for (int e = 0; e < E; ++e) {
      const int d = lane + 64 * e, r = d & 15, i = d >> 4, g = d / G;
      o[e] *= corr;
      zs[e] *= corr;
      for (int x = 0; x < cnt; ++x) {
        const uint8_t* blk = sb[x];
        const int in = st[x];
        const unsigned c = blk[a.codes + ((in >> 2) * 16 + r) * 4 * U + (in & 3) * U + i / 2] >> (4 * (i & 1)) & 15u;
        const unsigned par = *reinterpret_cast<const unsigned*>(blk + 2 * a.codes + a.params + (g * a.page + in) * 4);
        o[e] = __builtin_fmaf(sp[x] * from16<BF>(par & 0xffffu), (float)c, o[e]);
        zs[e] = __builtin_fmaf(sp[x], from16<BF>(par >> 16), zs[e]);
      }
    }
    __syncthreads();
  }
  for (int e = 0; e < E; ++e) {
    const float v = l == 0.f ? 0.f : (o[e] + zs[e]) / l;
    uint16_t bits;
    if constexpr (BF) bits = __builtin_bit_cast(uint16_t, (__bf16)v);
    else bits = __builtin_bit_cast(uint16_t, (_Float16)v);
    a.out[row * a.os + head * D + lane + 64 * e] = bits;
  }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

template <bool BF>
void launch_type(int dim, int ng, dim3 grid, hipStream_t s, const AttnArgs& a) {
  const dim3 b(64);
  if (dim == 64) ng == 1 ? attention_row<BF, 64, 1><<<grid, b, 0, s>>>(a) : attention_row<BF, 64, 2><<<grid, b, 0, s>>>(a);
  else if (dim == 128)
    ng == 1 ? attention_row<BF, 128, 1><<<grid, b, 0, s>>>(a)
            : ng == 2 ? attention_row<BF, 128, 2><<<grid, b, 0, s>>>(a) : attention_row<BF, 128, 4><<<grid, b, 0, s>>>(a);
  else
    ng == 1 ? attention_row<BF, 256, 1><<<grid, b, 0, s>>>(a)
            : ng == 2 ? attention_row<BF, 256, 2><<<grid, b, 0, s>>>(a) : attention_row<BF, 256, 4><<<grid, b, 0, s>>>(a);
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
  a.q_heads = p->q_heads;
  a.kv_heads = p->cache.kv_heads;
  a.ratio = p->q_heads / p->cache.kv_heads;
  a.max_pages = p->max_pages;
  a.page = p->cache.page_size;
  a.num_pages = (int)p->cache.num_pages;
  a.codes = g.codes;
  a.params = g.params;
  a.block = g.bytes;
  a.max_q = p->max_q_len;
  a.causal = p->causal;
  a.window = p->window;
  a.scale = p->scale * 1.4426950408889634f;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  if (pl.kind == ATTN_ROWS) {
    a.units_min = pl.units_min;
    a.tickets = static_cast<unsigned*>(workspace);
    a.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.tickets_bytes);
    switch ((p->cache.dtype == QGEMM_DT_BF16 ? 3 : 0) + (p->cache.head_dim == 64 ? 0 : p->cache.head_dim == 128 ? 1 : 2)) {
      case 0: e = launch_rows<false, 64>(pl, a, s); break;
      case 1: e = launch_rows<false, 128>(pl, a, s); break;
      case 2: e = launch_rows<false, 256>(pl, a, s); break;
      case 3: e = launch_rows<true, 64>(pl, a, s); break;
      case 4: e = launch_rows<true, 128>(pl, a, s); break;
      default: e = launch_rows<true, 256>(pl, a, s); break;
    }
  } else {
    if (p->cache.dtype == QGEMM_DT_BF16) launch_type<true>(p->cache.head_dim, pl.groups, dim3(pl.grid), s, a);
    else launch_type<false>(p->cache.head_dim, pl.groups, dim3(pl.grid), s, a);
    e = hipGetLastError();
  }
  if (e != hipSuccess) return fail(QGEMM_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  return QGEMM_OK;
}
