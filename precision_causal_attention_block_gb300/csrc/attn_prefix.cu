// Attention over the cache where the sequences of a batch share a long prefix: its
// whole 128-key tiles are read once, for the new tokens of all sequences together.
//
//   o = (sum_p 2^(x_p) v_p + sum_r 2^(x_r) v_r) / (sum_p 2^(x_p) + sum_r 2^(x_r))
// over the prefix's keys p and a row's own keys r behind them, so each part can be worked
// out by itself as a mean of values o_i with log2 of its sum of weights, lg_i:
//   lg = log2 sum 2^lg_i,   o = sum 2^(lg_i - lg) o_i.
//
// Three kernels: the attention kernels of attn_cache.cu or attn_cache_rows.cu over the
// prefix, with the tokens of all sequences as the query rows of each K / V head (no masks:
// all of them see all of it), those of attn_cache.cu over what comes behind it, and one
// that joins what they leave: float32 rows of items that were not cut, and the
// parts of those that were (equal runs of key tiles for all CTAs, as there; nothing waits
// for another CTA and no atomics, so results do not depend on timing).
#include "attend.cuh"

namespace flamia {
namespace {

struct JoinArgs {
  AttendArgs prefix, rest;
  int prefix_rows, rest_rows;  // rows an item
  int prefix_ctas, rest_ctas;  // of the launches
};

// Where the parts of an item lie: part 0 in slot 1 of CTA c, the others in slots 0 from
// there on; one part: the item was not cut.
struct Parts {
  int n, c;
  __device__ __forceinline__ size_t slot(int p) const {
    return static_cast<size_t>(p == 0 ? 2 * c + 1 : 2 * (c + p));
  }
};

// Of the item at units at .. at + units - 1, of which the first `cost` have no keys.
__device__ __forceinline__ Parts parts_of(long long total, int grid, int least, long long at,
                                          int units, int cost) {
  const long long ctas = min(static_cast<long long>(grid), div_up(total, least));
  const long long a = div_up((at + cost + 1) * ctas, total) - 1;
  const long long b = div_up((at + units) * ctas, total) - 1;
  return Parts{static_cast<int>(b - a) + 1, static_cast<int>(a)};
}

// A warp a row (token and query head); MANY: the prefix's items have 256 rows.
template <int DIM, bool MANY>
__global__ void __launch_bounds__(256) join_prefix_kernel(const JoinArgs a) {
  constexpr int E = DIM / 32;  // elements a lane
  const AttendArgs& g = a.rest;
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  wait_for_previous();
  const int t = static_cast<int>(row / g.H), h = static_cast<int>(row - static_cast<long long>(t) * g.H);
  if (t >= g.T) return;
  const int b = warp_last_not_above(g.ndocs, t, lane, [&](int i) { return g.cu[i]; });
  const DocRange r = doc_range(g.cu, b, g.T);
  if (t < r.s || t >= r.e) return;
  const int hk = h / g.G, hg = h - hk * g.G;
  const int start = g.starts != nullptr ? g.starts[b] : 0;

  // its parts: of the prefix, then of the rest
  Parts pp{0, 0}, pr{1, 0};
  int rp = 0, rr = 0;  // its row in the item
  if (shares(g, start)) {
    const int n = min(max(g.cu[g.ndocs], 0), g.T);
    const int R = a.prefix_rows, cost = MANY ? kItemCost<256> : kItemCost<8>;
    const int units = a.prefix.shared + cost;
    const long long tiles = (static_cast<long long>(n) * g.G + R - 1) / R;
    const long long at = static_cast<long long>(t) * g.G + hg, rt = at / R;
    rp = static_cast<int>(at - rt * R);
    pp = parts_of(tiles * g.H_kv * units, a.prefix_ctas, cost + 2, (hk * tiles + rt) * units, units,
                  cost);
  }
  if (!g.whole) {
    const int R = a.rest_rows;
    const long long before = g.first[b], total = g.first[g.ndocs];
    const long long tiles = (static_cast<long long>(r.e - r.s) * g.G + R - 1) / R;
    const int units = static_cast<int>((g.first[b + 1] - before) / (tiles * g.H_kv));
    const long long at = static_cast<long long>(t - r.s) * g.G + hg, rt = at / R;
    rr = static_cast<int>(at - rt * R);
    pr = parts_of(total, a.rest_ctas, kItemCost<8> + 2, before + (hk * tiles + rt) * units, units,
                  kItemCost<8>);
  }
  const size_t own = static_cast<size_t>(t) * g.H + h;
  const int parts = pp.n + pr.n;
  auto stat = [&](int p) {
    if (p < pp.n)
      return pp.n == 1 ? a.prefix.row_stats[own] : a.prefix.stats[pp.slot(p) * a.prefix_rows + rp];
    return pr.n == 1 ? g.row_stats[own] : g.stats[pr.slot(p - pp.n) * a.rest_rows + rr];
  };
  auto data = [&](int p) -> const float* {
    if (p < pp.n) {
      if (pp.n == 1) return a.prefix.rows + own * DIM + lane * E;
      const size_t s = pp.slot(p);
      return MANY ? a.prefix.partial + (s * (DIM / 4) + lane * E / 4) * 256 * 4 + rp * 4 + lane * E % 4
                  : a.prefix.partial + (s * a.prefix_rows + rp) * DIM + lane * E;
    }
    return pr.n == 1 ? g.rows + own * DIM + lane * E
                     : g.partial + (pr.slot(p - pp.n) * a.rest_rows + rr) * DIM + lane * E;
  };
  float m = -INFINITY;
  for (int p = lane; p < parts; p += 32) {
    const float x = stat(p);
    m = x > m || x != x ? x : m;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float x = __shfl_xor_sync(0xffffffffu, m, o);
    m = x > m || x != x ? x : m;  // NaN stays
  }
  // (weights in two halves, as a small one may meet large values)
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f, acc[E] = {};
  for (int p0 = 0; p0 < parts; p0 += 32) {
    const float wt = p0 + lane < parts ? exp2f(0.5f * (stat(p0 + lane) - ref)) : 0.f;
    l = fmaf(wt, wt, l);
    const int n = min(32, parts - p0);
#pragma unroll 4
    for (int p = 0; p < n; ++p) {
      const float w = __shfl_sync(0xffffffffu, wt, p);
      const float* x = data(p0 + p);
      if constexpr (E == 4) {
        const float4 v = *reinterpret_cast<const float4*>(x);
        acc[0] = fmaf(w, w * v.x, acc[0]);
        acc[1] = fmaf(w, w * v.y, acc[1]);
        acc[2] = fmaf(w, w * v.z, acc[2]);
        acc[3] = fmaf(w, w * v.w, acc[3]);
      } else {
        const float2 v = *reinterpret_cast<const float2*>(x);
        acc[0] = fmaf(w, w * v.x, acc[0]);
        acc[1] = fmaf(w, w * v.y, acc[1]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (lane == 0 && g.lse != nullptr)
    g.lse[static_cast<size_t>(h) * g.T + t] = (ref + log2f(l)) * kLn2;
  __nv_bfloat162* out = reinterpret_cast<__nv_bfloat162*>(g.o + own * DIM + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2)
    out[e / 2] = __floats2bfloat162_rn(inv == 0.f ? 0.f : acc[e] * inv,
                                       inv == 0.f ? 0.f : acc[e + 1] * inv);
}

// ------------------------------------------------------------------ host

// Rows an item of the two attention kernels, or 0: the call is flamia_attn_cache's.
struct Forms {
  int prefix, rest;
};
Forms forms(int T, int ndocs, int G, int prefix) {
  const int rest = rows_per_item(mean_rows(T, ndocs, G));
  // nothing to share; or every sequence fills a tensor-core operand by itself
  if (ndocs < 2 || prefix < 128 || prefix > kMaxPos || rest == kManyRows) return Forms{0, 0};
  return Forms{rows_per_item(static_cast<long long>(T) * G), rest};
}

// Results of one attention kernel.
size_t results(AttendArgs& g, uint8_t* ws, size_t at, int R, int d) {
  const size_t slots = 2 * static_cast<size_t>(R == kManyRows ? kRowsCtas : kMaxCtas);
  const size_t rows = static_cast<size_t>(g.T) * g.H;
  auto take = [&](size_t n) {
    float* p = reinterpret_cast<float*>(ws + at);
    at += align_up(n * sizeof(float), 256);
    return p;
  };
  g.stats = take(slots * R);
  g.row_stats = take(rows);
  g.partial = take(slots * R * d);
  g.rows = take(rows * d);
  return at;
}

// All of the workspace, from ws on.
size_t layout(AttendArgs& p, AttendArgs& r, void* ws, const Forms& f, int d) {
  uint8_t* base = static_cast<uint8_t*>(ws);
  r.first = reinterpret_cast<long long*>(base);
  size_t at = align_up(sizeof(long long) * (static_cast<size_t>(r.ndocs) + 1), 256);
  at = results(p, base, at, f.prefix, d);
  return results(r, base, at, f.rest, d);
}

template <int DIM>
bool launch_join_prefix(const JoinArgs& a, cudaStream_t s) {
  const long long rows = static_cast<long long>(a.rest.T) * a.rest.H;
  const dim3 grid(static_cast<unsigned>((rows + 7) / 8));
  return a.prefix_rows == kManyRows
             ? launch_after(join_prefix_kernel<DIM, true>, grid, 256, 0, s, a)
             : launch_after(join_prefix_kernel<DIM, false>, grid, 256, 0, s, a);
}

}  // namespace
}  // namespace flamia

using namespace flamia;

extern "C" size_t flamia_attn_cache_prefix_workspace_bytes(int T, int ndocs, int H, int H_kv, int d,
                                                           int prefix) {
  const size_t plain = flamia_attn_cache_workspace_bytes(T, ndocs, H, H_kv, d);
  if (plain == 0 || prefix < 0) return 0;
  const Forms f = forms(T, ndocs, H / H_kv, prefix);
  if (f.rest == 0) return plain;
  AttendArgs p{}, r{};
  p.T = r.T = T;
  p.H = r.H = H;
  p.ndocs = r.ndocs = ndocs;
  return layout(p, r, nullptr, f, d);
}

extern "C" flamia_status flamia_attn_cache_prefix(
    const flamia_kvcache* cache, const void* q_bf16, int64_t q_stride, int T, int H,
    const int32_t* cu_seqlens, int ndocs, const int32_t* starts, const int32_t* page_table,
    int table_stride, int prefix, float softmax_scale, void* o_bf16, float* lse, void* ws,
    size_t ws_bytes, int* dev_status, void* stream) {
  JoinArgs a{};
  const flamia_status st =
      attend_args(a.rest, cache, q_bf16, q_stride, T, H, cu_seqlens, ndocs, starts, page_table,
                  table_stride, softmax_scale, 0, 0, o_bf16, lse, ws, dev_status);
  if (st != FLAMIA_OK) return st;
  if (prefix < 0) return FLAMIA_ERR_INVALID_ARG;
  if (T == 0) return FLAMIA_OK;
  const Forms f = forms(T, ndocs, a.rest.G, prefix);
  if (f.rest == 0)
    return flamia_attn_cache(cache, q_bf16, q_stride, T, H, cu_seqlens, ndocs, starts, page_table,
                             table_stride, softmax_scale, 0, 0, o_bf16, lse, ws, ws_bytes,
                             dev_status, stream);
  AttendArgs &r = a.rest, &p = a.prefix;
  r.prefix = prefix;
  r.shared = prefix / 128;
  p = r;
  if (layout(p, r, ws, f, cache->d) > ws_bytes) return FLAMIA_ERR_WORKSPACE;
  p.whole = 0;
  r.whole = r.cap - 128 * r.shared <= 128 * kWholeTiles;
  a.prefix_rows = f.prefix;
  a.rest_rows = f.rest;
  a.prefix_ctas = f.prefix == kManyRows ? rows_grid() : few_grid(f.prefix);
  a.rest_ctas = few_grid(f.rest);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  flamia_status done = f.prefix == kManyRows ? attend_rows(cache, p, kPrefix, s)
                                             : attend_few(cache, p, f.prefix, kPrefix, s);
  if (done == FLAMIA_OK) done = attend_few(cache, r, f.rest, kRest, s);
  if (done != FLAMIA_OK) return done;
  return (cache->d == 128 ? launch_join_prefix<128>(a, s) : launch_join_prefix<64>(a, s))
             ? FLAMIA_OK
             : FLAMIA_ERR_CUDA;
}
