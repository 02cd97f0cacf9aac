// Attention over the cache where the sequences of a batch share a long prefix: its
// whole 128-key tiles are read once, for the new tokens of all sequences together.
//
//   o = (sum_p 2^(x_p) v_p + sum_r 2^(x_r) v_r) / (sum_p 2^(x_p) + sum_r 2^(x_r))
// over the prefix's keys p and a row's own keys r behind them, so each part can be worked
// out by itself as a mean of values o_i with log2 of its sum of weights, lg_i:
//   lg = log2 sum 2^lg_i,   o = sum 2^(lg_i - lg) o_i.
//
// Few query rows of a K / V head in the whole batch: one launch of attn_cache.cu's
// kernels over items of both kinds.  Many: the kernel of attn_prefix_rows.cu over the prefix
// (no masks: all rows see all of it), then attn_cache.cu's over what comes behind it.
// In both cases a last kernel joins what they leave: float32 rows of items that
// were not cut and the parts of those that were (equal runs of key tiles for all CTAs, as
// there; nothing waits for another CTA and there are no atomics on results, so these do not
// depend on timing).  Each row's record of where its parts lie (RowParts) is written with
// them, so that the join has no search and no plan before its first loads.
//
// Floor: K and V of the prefix once (2 H_kv (d + 1) bytes a token) and of each own tail.
// Measured, the whole call (us; plain: flamia_attn_cache on the same batch): 8 tokens over
// 2,048, 16 heads of 128, 16.7 (floor 1.4, plain 22.0: latency); 89 of 96 sequences over
// 16,421, 32 / 8 heads of 128, 83 (12.7, 255: 43 over the prefix, 29 the tails, 11 the join);
// 24 over 131,072, 32 heads of 64, 216 (84, 1,735: the softmax of 24 rows a tile); 128 x 4
// drafted tokens over 8,191, 16 / 4 heads of 128, 85 (17.9, 161: as the batch).
#include "attend.cuh"

namespace flamia {
namespace {

// Results of one kind of items.
struct Side {
  const RowParts* where;
  const float *row_stats, *rows, *stats, *partial;
  int R;  // rows an item
};

struct JoinArgs {
  Side prefix, rest;
  const int32_t* cu;
  __nv_bfloat16* o;
  float* lse;
  int ndocs, T, H, G;
};

// A row's parts.  (Records out of range come from malformed offsets, for which none was
// written.)
struct Parts {
  int n, cta, row;
  __device__ __forceinline__ Parts(RowParts w, bool any, int R) {
    n = any ? w.n & ~kShares : 0;
    cta = w.at & 0xFFFF;
    row = (w.at >> 16) & (R - 1);
    const int ctas = R == kManyRows ? kRowsCtas : kMaxCtas;
    if (cta >= ctas || n < 0 || n > ctas - cta) n = 0;
  }
  __device__ __forceinline__ size_t slot(int p) const {
    return static_cast<size_t>(p == 0 ? 2 * cta + 1 : 2 * (cta + p));
  }
  __device__ __forceinline__ float stat(const Side& s, int p, int own) const {
    return n > 1 ? s.stats[slot(p) * s.R + row] : s.row_stats[own];
  }
  // Its values in [slot][row][d], or the whole row.
  __device__ __forceinline__ const float* data(const Side& s, int p, int own, int d) const {
    return n > 1 ? s.partial + (slot(p) * s.R + row) * d : s.rows + static_cast<size_t>(own) * d;
  }
};

__device__ __forceinline__ float max_or_nan(float m, float x) {
  return x > m || x != x ? x : m;  // NaN stays
}
// Weights of parts are taken in two halves, as a small one may meet large values.
__device__ __forceinline__ float half_weight(float stat, float ref) {
  return exp2f(0.5f * (stat - ref));
}
// What is summed so far, when the reference goes from m to m1 (of nothing: nothing).
__device__ __forceinline__ float rescale(float m, float m1) {
  return m == -INFINITY ? 0.f : half_weight(m, m1);
}
__device__ __forceinline__ void add4(float (&acc)[4], float w, const float4& v) {
  acc[0] = fmaf(w, w * v.x, acc[0]);
  acc[1] = fmaf(w, w * v.y, acc[1]);
  acc[2] = fmaf(w, w * v.z, acc[2]);
  acc[3] = fmaf(w, w * v.w, acc[3]);
}
__device__ __forceinline__ uint2 mean4(const float (&acc)[4], float inv) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(inv == 0.f ? 0.f : acc[0] * inv,
                                                 inv == 0.f ? 0.f : acc[1] * inv);
  const __nv_bfloat162 b = __floats2bfloat162_rn(inv == 0.f ? 0.f : acc[2] * inv,
                                                 inv == 0.f ? 0.f : acc[3] * inv);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// Both joins wait for memory: the values of 32 (8) parts are loaded beside their statistics,
// before the weights are known, and the reference moves from batch to batch.
//
// One launch: four warps a row (token and query head), four elements a lane, parts by turns
// (d = 64: two of a warp's side by side).  5 rows of 8 heads over 16,384 keys: the call takes
// 26.5 us, and 35 with one warp a row and values loaded behind the weights.
constexpr int kJoinWarps = 4;
template <int DIM>
__global__ void __launch_bounds__(32 * kJoinWarps) join_few_kernel(const JoinArgs g) {
  constexpr int kLanes = DIM / 4, kTurns = 32 / kLanes * kJoinWarps;
  __shared__ float4 s_acc[kTurns][kLanes];
  const int lane = threadIdx.x & 31, own = blockIdx.x;
  const int turn = threadIdx.x / kLanes, e = lane % kLanes;
  wait_for_previous();
  const int t = own / g.H, h = own - t * g.H;
  const int end = g.cu[g.ndocs];
  const RowParts wr = g.rest.where[own], wp = g.prefix.where[own];
  if (t >= end) return;
  const Parts pr(wr, true, g.rest.R), pp(wp, (wr.n & kShares) != 0, g.prefix.R);
  const int parts = pp.n + pr.n;
  float m = -INFINITY, l = 0.f, acc[4] = {};
  for (int p0 = 0; p0 < parts; p0 += 32) {
    float4 v[32 / kTurns];
#pragma unroll
    for (int j = 0; j < 32 / kTurns; ++j) {
      const int q = p0 + j * kTurns + turn;
      v[j] = q >= parts ? make_float4(0.f, 0.f, 0.f, 0.f)
                        : reinterpret_cast<const float4*>(
                              q < pp.n ? pp.data(g.prefix, q, own, DIM)
                                       : pr.data(g.rest, q - pp.n, own, DIM))[e];
    }
    const int p = p0 + lane;
    const float x = p >= parts ? -INFINITY
                               : p < pp.n ? pp.stat(g.prefix, p, own) : pr.stat(g.rest, p - pp.n, own);
    float m1 = max_or_nan(m, x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m1 = max_or_nan(m1, __shfl_xor_sync(0xffffffffu, m1, o));
    const float ref = m1 == -INFINITY ? 0.f : m1, f = rescale(m, ref);
    const float wt = half_weight(x, ref);  // (behind the last part: 0)
    l = fmaf(wt, wt, f * f * l);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = f * (f * acc[i]);
#pragma unroll
    for (int j = 0; j < 32 / kTurns; ++j)
      add4(acc, __shfl_sync(0xffffffffu, wt, j * kTurns + turn), v[j]);
    m = m1;
  }
  s_acc[turn][e] = make_float4(acc[0], acc[1], acc[2], acc[3]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  __syncthreads();
  if (threadIdx.x >= kLanes) return;
  float sum[4] = {};
#pragma unroll
  for (int j = 0; j < kTurns; ++j) add4(sum, 1.f, s_acc[j][e]);
  if (threadIdx.x == 0 && g.lse != nullptr)
    g.lse[static_cast<size_t>(h) * g.T + t] = ((m == -INFINITY ? 0.f : m) + log2f(l)) * kLn2;
  *reinterpret_cast<uint2*>(g.o + static_cast<size_t>(own) * DIM + e * 4) =
      mean4(sum, l == 0.f ? 0.f : 1.f / l);
}

// Two launches: a thread a row and 4 elements, the rows those of an item over the prefix,
// as its parts lie [slot][d / 4][256 rows][4].  (8 elements and the maxima first: 83.3 us for
// the batch of 96, 81.1 so.)
template <int DIM>
__global__ void __launch_bounds__(256) join_many_kernel(const JoinArgs g, int row_tiles) {
  constexpr int kBatch = 8;
  const int hk = blockIdx.x / row_tiles;
  const int row = (blockIdx.x - hk * row_tiles) * 256 + threadIdx.x;
  const int t = row / g.G, h = hk * g.G + row - t * g.G;
  const int c = blockIdx.y;
  wait_for_previous();
  if (t >= g.T) return;
  const int own = t * g.H + h;
  const int end = g.cu[g.ndocs];
  const RowParts wr = g.rest.where[own], wp = g.prefix.where[own];
  if (t >= end) return;
  const Parts pr(wr, true, g.rest.R), pp(wp, (wr.n & kShares) != 0, 256);
  const int parts = pp.n + pr.n;
  float m = -INFINITY, l = 0.f, acc[4] = {};
#pragma unroll 1
  for (int p = 0; p < parts; p += kBatch) {
    float x[kBatch], m1 = m;
    float4 v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int q = p + i;
      x[i] = -INFINITY;
      v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (q < pp.n) {
        x[i] = pp.stat(g.prefix, q, own);
        v[i] = reinterpret_cast<const float4*>(
            pp.n > 1 ? g.prefix.partial + (pp.slot(q) * (DIM / 4) + c) * 1024 + pp.row * 4
                     : g.prefix.rows + static_cast<size_t>(own) * DIM + c * 4)[0];
      } else if (q < parts) {
        x[i] = pr.stat(g.rest, q - pp.n, own);
        v[i] = reinterpret_cast<const float4*>(pr.data(g.rest, q - pp.n, own, DIM))[c];
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) m1 = max_or_nan(m1, x[i]);
    const float ref = m1 == -INFINITY ? 0.f : m1, f = rescale(m, ref);
    l *= f * f;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = f * (f * acc[e]);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float w = half_weight(x[i], ref);  // (behind the last part: 0)
      l = fmaf(w, w, l);
      add4(acc, w, v[i]);
    }
    m = m1;
  }
  if (c == 0 && g.lse != nullptr)
    g.lse[static_cast<size_t>(h) * g.T + t] = ((m == -INFINITY ? 0.f : m) + log2f(l)) * kLn2;
  *reinterpret_cast<uint2*>(g.o + static_cast<size_t>(own) * DIM + c * 4) =
      mean4(acc, l == 0.f ? 0.f : 1.f / l);
}

// ------------------------------------------------------------------ host

// Rows an item over the prefix and over the rest, or 0: the call is flamia_attn_cache's.
struct Forms {
  int prefix, rest;
};
// Beyond 32 rows in the batch 256 an item, with 8 an item over the rest, or 32 in both where
// there is little to do: up to 64 rows, counted in key tiles (two for what is a sequence's own).
// 32 against 256 an item, us, heads of 128, 16,384 shared: 4 of them, 40 rows 26.5 and 39.4;
// 8, 36 rows 35.8 and 41.6, 64 rows 40.5 and 40.8; 16, 40 rows 71 and 70, 64 rows 93 and 83.
// 2,048 shared: 16 heads, 64 rows 52.8 and 54.6; 32 heads of 64, 40 rows 63 and 55.
// What sharing saves is the reading of the prefix by every sequence but one, at some 10 TB/s,
// as the L2 cache serves most of that; what it costs is the join and, with 256 rows, a
// launch and the larger items.  So it is done from so many bytes on.  Shared against plain,
// us, below and above: 8 rows 16.6 and 16.6 at 7.5 MB, 17.0 and 18.1 at 14.8; 16 rows 19.3 and
// 19.0 at 16 MB, 17.9 and 19.0 at 23; 32 rows 30.8 and 29.9 at 65 MB, 33.5 and 35.5 at
// 131; 256 rows 50.9 and 45.5 at 266 MB, 55.4 and 61.4 at 401.
Forms forms(int T, int ndocs, int G, int H_kv, int d, int prefix, int flags) {
  const int rest = rows_per_item(mean_rows(T, ndocs, G));
  // nothing to share; or every sequence fills a tensor-core operand by itself
  if (ndocs < 2 || prefix < 128 || prefix > kMaxPos || rest == kManyRows) return Forms{0, 0};
  const long long rows = static_cast<long long>(T) * G;
  const bool little = rows <= 64 && H_kv * (2ll * (prefix / 128) + 2ll * ndocs) <= 2560;
  const int all = rows <= 32 ? rows_per_item(rows) : little ? 32 : kManyRows;
  const double saved = (ndocs - 1.) * (prefix / 128 * 128) * H_kv * 2. * (d + 1);
  const double least = all == 8 ? 10e6 : all == 16 ? 20e6 : all == 32 ? 100e6 : 300e6;
  if (saved < least && !(flags & FLAMIA_FLAG_PREFIX_ALWAYS)) return Forms{0, 0};
  return Forms{all, all == kManyRows ? rest : all};
}

// The workspace, from ws on.
struct Layout {
  RowParts* where[2];
  float *row_stats[2], *rows[2], *stats[2], *partial[2];
  size_t total;
};
Layout layout(void* ws, const Forms& f, int T, int H, int d) {
  Layout w{};
  uint8_t* base = static_cast<uint8_t*>(ws);
  const size_t rows = static_cast<size_t>(T) * H;
  auto take = [&](size_t n) {
    uint8_t* p = base + w.total;
    w.total += align_up(n, 256);
    return p;
  };
  const bool two = f.prefix == kManyRows;
  for (int i = 0; i < 2; ++i) {
    w.where[i] = reinterpret_cast<RowParts*>(take(sizeof(RowParts) * rows));
    w.row_stats[i] = reinterpret_cast<float*>(take(sizeof(float) * rows));
    w.rows[i] = reinterpret_cast<float*>(take(sizeof(float) * rows * d));
    if (i == 0 && !two) continue;  // (one launch: in the same slots)
    const int R = i == 0 ? f.prefix : f.rest;
    const size_t slots = 2 * static_cast<size_t>(R == kManyRows ? kRowsCtas : kMaxCtas);
    w.stats[i] = reinterpret_cast<float*>(take(sizeof(float) * slots * R));
    w.partial[i] = reinterpret_cast<float*>(take(sizeof(float) * slots * R * d));
  }
  if (!two) {
    w.stats[0] = w.stats[1];
    w.partial[0] = w.partial[1];
  }
  return w;
}

template <int DIM>
bool launch_join_prefix(const JoinArgs& a, int H_kv, cudaStream_t s) {
  if (a.prefix.R != kManyRows)
    return launch_after(join_few_kernel<DIM>, dim3(a.T * a.H), 32 * kJoinWarps, 0, s, a);
  const int row_tiles = static_cast<int>((static_cast<long long>(a.T) * a.G + 255) / 256);
  return launch_after(join_many_kernel<DIM>, dim3(row_tiles * H_kv, DIM / 4), 256, 0, s, a,
                      row_tiles);
}

}  // namespace
}  // namespace flamia

using namespace flamia;

extern "C" size_t flamia_attn_cache_prefix_workspace_bytes(int T, int ndocs, int H, int H_kv, int d,
                                                           int prefix, int flags) {
  const size_t plain = flamia_attn_cache_workspace_bytes(T, ndocs, H, H_kv, d);
  if (plain == 0 || prefix < 0 || (flags & ~FLAMIA_FLAG_PREFIX_ALWAYS)) return 0;
  const Forms f = forms(T, ndocs, H / H_kv, H_kv, d, prefix, flags);
  return f.rest == 0 ? plain : layout(nullptr, f, T, H, d).total;
}

extern "C" flamia_status flamia_attn_cache_prefix(
    const flamia_kvcache* cache, const void* q_bf16, int64_t q_stride, int T, int H,
    const int32_t* cu_seqlens, int ndocs, const int32_t* starts, const int32_t* page_table,
    int table_stride, int prefix, float softmax_scale, int flags, void* o_bf16, float* lse, void* ws,
    size_t ws_bytes, int* dev_status, void* stream) {
  AttendArgs g{};
  const flamia_status st =
      attend_args(g, cache, q_bf16, q_stride, T, H, cu_seqlens, ndocs, starts, page_table,
                  table_stride, softmax_scale, 0, 0, o_bf16, lse, ws, dev_status);
  if (st != FLAMIA_OK) return st;
  if (flags & ~FLAMIA_FLAG_PREFIX_ALWAYS) return FLAMIA_ERR_UNSUPPORTED;
  if (prefix < 0) return FLAMIA_ERR_INVALID_ARG;
  if (T == 0) return FLAMIA_OK;
  const Forms f = forms(T, ndocs, g.G, g.H_kv, cache->d, prefix, flags);
  if (f.rest == 0)
    return flamia_attn_cache(cache, q_bf16, q_stride, T, H, cu_seqlens, ndocs, starts, page_table,
                             table_stride, softmax_scale, 0, 0, o_bf16, lse, ws, ws_bytes,
                             dev_status, stream);
  const Layout w = layout(ws, f, T, H, cache->d);
  if (w.total > ws_bytes) return FLAMIA_ERR_WORKSPACE;
  JoinArgs a{};
  for (int i = 0; i < 2; ++i) {
    g.where[i] = w.where[i];
    g.row_stats[i] = w.row_stats[i];
    g.rows[i] = w.rows[i];
    (i == 0 ? a.prefix : a.rest) = Side{w.where[i], w.row_stats[i], w.rows[i], w.stats[i],
                                        w.partial[i], i == 0 ? f.prefix : f.rest};
  }
  a.cu = cu_seqlens;
  a.o = g.o;
  a.lse = lse;
  a.ndocs = ndocs;
  a.T = T;
  a.H = H;
  a.G = g.G;
  g.prefix = prefix;
  g.shared = prefix / 128;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  flamia_status done = FLAMIA_OK;
  if (f.prefix == kManyRows) {
    AttendArgs p = g;
    p.whole = 0;
    p.stats = w.stats[0];
    p.partial = w.partial[0];
    done = attend_prefix_rows(cache, p, s);
  }
  // items over the rest stay whole as flamia_attn_cache's do, but not beside items over the
  // prefix, with which they have to be counted alike
  g.whole = f.prefix == kManyRows && g.cap - 128 * g.shared <= 128 * kWholeTiles;
  g.stats = w.stats[1];
  g.partial = w.partial[1];
  if (done == FLAMIA_OK)
    done = attend_few(cache, g, f.rest, f.prefix == kManyRows ? kRest : kBoth, s);
  if (done != FLAMIA_OK) return done;
  return (cache->d == 128 ? launch_join_prefix<128>(a, cache->H_kv, s)
                          : launch_join_prefix<64>(a, cache->H_kv, s))
             ? FLAMIA_OK
             : FLAMIA_ERR_CUDA;
}
