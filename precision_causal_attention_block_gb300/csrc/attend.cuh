// Shared by the kernels of attention over the paged cache: the arguments, the
// cutting of all items' key tiles into equal runs, and the joining of the parts
// of an item.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "paged.cuh"

namespace flamia {

constexpr int kMaxCtas = 512;   // runs of a launch (the workspace is sized for it)
constexpr int kSlots = 2 * kMaxCtas;  // partial results
constexpr int kRowsCtas = 160;        // the same with 256 rows an item
constexpr int kSegSlots = 4;
constexpr int kMaxPos = 1 << 30;
// An item's own steps (queries, first references, output) in tiles.  2 .. 6 are
// within 3% of one another on the ragged and the windowed batch; with 256 rows an
// item, 505 tokens over 7,866: 116, 113, 112, 113, 113 us with 1, 3, 5, 7, 9; 4,096
// tokens over none: 198, 198, 201, 203, 208.
template <int R>
constexpr int kItemCost = R == 256 ? 5 : 3;
// Items of at most so many tiles (as the page table's width bounds them) stay whole: 64
// sequences over 512 tokens 19.9 us whole, 23.7 cut and joined; over 1,024 tokens 38.9
// against 37.9.
constexpr int kWholeTiles = 4;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kHigh = 30;       // eV may exceed E0 by this before E0 moves
constexpr int kLow = 60;        // keys whose eV lies further below E0 are summed apart

struct AttendArgs {
  const uint8_t *k_scales, *v_scales;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  const int32_t *cu, *starts, *table;
  int4* joins;       // [kMaxCtas][2]: items to join
  float* stats;      // [kSlots][R] log2 sum 2^x
  float* partial;    // o: [kSlots][R][d]; 256 rows: [slots][d / 4][R][4]
  int* status;
  long long q_stride;
  int T, H, H_kv, G, ndocs, table_stride, num_pages, page_size, window, sinks;
  int cap;           // positions that the page table has room for
  int whole;         // items stay whole
  float scale_log2;
};

// Two bounded waits of a converged warp whose latencies overlap: a wait for a
// phase that is long complete still takes some 150 cycles.  (From 16 rows on;
// with 8, where HBM sets the pace, it measured slower: 99 us against 97 on 96
// ragged contexts.)
__device__ __forceinline__ bool wait_both(uint32_t bar0, uint32_t parity0, uint32_t bar1,
                                          uint32_t parity1, const volatile int* abort) {
  const bool a = mbar_try_wait(bar0, parity0);
  const bool b = mbar_try_wait(bar1, parity1);
  if (__all_sync(0xffffffffu, a && b)) return true;
  return mbar_wait_w_ab(bar0, parity0, abort) && mbar_wait_w_ab(bar1, parity1, abort);
}

// A pair of floats rounded to FP16.
__device__ __forceinline__ uint32_t half2_of(float2 a) {
  const __half2 h = __floats2half2_rn(a.x, a.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// A sum m 2^e of softmax weights 2^(x - ref) with an exponent of its own (a whole
// number; it moves with the reference), for what a row's running sum cannot hold; m =
// 0: nothing.  NaN stays.
struct Sum {
  float m, e;
  __device__ __forceinline__ void add(float qm, float qe) {
    if (qm == 0.f) return;
    if (m == 0.f) {
      m = qm;
      e = qe;
      return;
    }
    const float top = fmaxf(e, qe);
    auto scaled = [&](float x, float ex) {
      return ldexpf(x, max(static_cast<int>(ex - top), -400));
    };
    m = scaled(m, e) + scaled(qm, qe);
    e = top;
  }
};
constexpr float kNoExponent = -1e30f;

// References beyond kLarge, where float32 begins to lose fractions of the scores: a
// reference set from a row's largest score could leave that one above it by many units
// (weights past their range) or below it (none at all).  So it is set some steps of
// float32 too low, what exceeds it by no more than room(-ref) does not move it, and
// weights above the largest are cut to that (scores that close count as equal).
constexpr float kLarge = 65536.f;
__device__ __forceinline__ float lowered(float nref) {
  return fabsf(nref) > kLarge ? nref + ceilf(fabsf(nref) * 0x1p-21f) : nref;
}
__device__ __forceinline__ float room(float nref) {
  return fabsf(nref) > kLarge ? fabsf(nref) * 0x1p-19f : 0.f;
}
__device__ __forceinline__ float cut(float y, float most) {  // (NaN stays)
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(y), "f"(most));
  return r;
}
// 2^k, k cut to the exponents of normal floats.
__device__ __forceinline__ float pow2_within(int k) { return exp2i(min(max(k, -126), 127)); }
__device__ __forceinline__ float pow2_byte(int byte) {
  return byte > 0 ? __uint_as_float(static_cast<uint32_t>(byte) << 23) : 0x1p-127f;
}

// ------------------------------------------------------------------ work

// Sequence b's share of the work: row tiles x K / V heads items of `tiles` key
// tiles (an upper bound over its row tiles, the last one's: a segment that runs past
// its item's last tile is cut there.  So the first row tiles of a prompt count for more
// than they have: 4,096 tokens over none take 197 us, at 349 TFLOP/s, where 505 over
// 7,361 run at 563).  An item is `units` long: kItemCost, then a unit
// for each tile; one unit if items stay whole.
struct SeqWork {
  int s, n, start;     // packed rows [s, s + n) at positions start ..
  int row_tiles, tiles, units;
  __device__ __forceinline__ long long total(int H_kv) const {
    return static_cast<long long>(row_tiles) * H_kv * units;
  }
};

template <int R>
__device__ __forceinline__ SeqWork seq_work(const AttendArgs& g, int b) {
  SeqWork w;
  const DocRange r = doc_range(g.cu, b, g.T);
  w.s = r.s;
  w.n = r.e - r.s;
  w.start = g.starts != nullptr ? g.starts[b] : 0;
  if (w.start > kMaxPos - w.n) w.start = -w.n;  // reported by the producer
  w.start = max(w.start, -kMaxPos);
  w.row_tiles = static_cast<int>((static_cast<long long>(w.n) * g.G + R - 1) / R);
  // (no further than the page table: a wild first position costs no endless walk)
  const int end = min(max(w.start + w.n, 0), g.cap);
  int tiles = (end + 127) >> 7;
  if (g.window > 0)
    tiles = min(tiles, ((min(g.sinks, end) + 127) >> 7) +
                           ((min(g.window, end) + R / g.G + 1 + 127) >> 7) + 1);
  w.tiles = max(tiles, 1);
  w.units = g.whole ? 1 : w.tiles + kItemCost<R>;
  return w;
}

// A run of one item's key tiles, handed from the producer to the other roles.
struct Segment {
  int s, n, start;  // as SeqWork; s < 0: no more work
  int hk, row0;     // K / V head; first row (token-major, then query head)
  int i0, i1;       // its key tiles: list positions i0 .. i1 - 1
  int ns, wt;       // list position i is key tile i (i < ns) or i - ns + wt
  int slot;         // partial result slot, or -1: the whole item
};

__device__ __forceinline__ int tile_of(const Segment& g, int i) {
  return i < g.ns ? i : i - g.ns + g.wt;
}

// The piece of a tile (a page of less than 128 rows, or the whole tile) that
// holds one of its keys.
__device__ __forceinline__ int piece_of(int key_in, int page_size) {
  return page_size == 32 ? key_in >> 5 : page_size == 64 ? key_in >> 6 : 0;
}

// a * b / c and a / c for a, b, c >= 0, in 32 bits where they suffice (a 64-bit
// division takes some hundred cycles, and the first copies wait for it).
__device__ __forceinline__ long long mul_div(long long a, long long b, long long c) {
  const long long ab = a * b;
  if (((ab | c) >> 32) == 0)
    return static_cast<uint32_t>(ab) / static_cast<uint32_t>(c);
  return ab / c;
}
__device__ __forceinline__ long long div_up(long long a, long long c) {
  return mul_div(a + c - 1, 1, c);
}

// CTAs that get a run: at least two tiles each, as far as there are any.
template <int R>
__device__ __forceinline__ long long active_ctas(const AttendArgs& g, long long total) {
  const int least = g.whole ? 1 : kItemCost<R> + 2;
  return min(static_cast<long long>(gridDim.x), div_up(total, least));
}

// Total units, and this CTA's run of them: [u0, u1), starting at unit `off` of
// sequence b.  Every thread sums a stretch of sequences; the one whose stretch
// holds u0 walks it.
template <int R, int kThreads, class Sm>
__device__ __forceinline__ void make_plan(const AttendArgs& g, Sm& sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = (g.ndocs + kThreads - 1) / kThreads;
  const int b0 = min(tid * each, g.ndocs), b1 = min(b0 + each, g.ndocs);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) sum += seq_work<R>(g, b).total(g.H_kv);
  long long inc = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += y;
  }
  if (lane == 31) sm.scan[warp] = inc;
  if (tid == 0) sm.plan_b = g.ndocs;
  __syncthreads();
  long long before = inc - sum, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sm.scan[w];
    total += sm.scan[w];
  }
  const long long ctas = active_ctas<R>(g, total);
  const long long c = blockIdx.x;
  const long long u0 = c < ctas ? mul_div(total, c, ctas) : total;
  const long long u1 = c < ctas ? mul_div(total, c + 1, ctas) : total;
  if (tid == 0) {
    sm.plan_u0 = u0;
    sm.plan_u1 = u1;
    sm.plan_total = total;
  }
  if (u0 < u1 && before <= u0 && u0 < before + sum) {
    long long off = u0 - before;
    int b = b0;
    SeqWork w = seq_work<R>(g, b);
    while (b < b1 - 1 && off >= w.total(g.H_kv)) {
      off -= w.total(g.H_kv);
      w = seq_work<R>(g, ++b);
    }
    sm.plan_b = b;
    sm.plan_seq = w;
    sm.plan_off = off;
  }
  __syncthreads();
}

// Joins the parts of an item that several CTAs shared (part 0 in slot 1 of the
// CTA before, the others in slots 0 from this CTA on): o = sum 2^(lg_p - lg) o_p, the
// weights in two halves, as a small one may meet large values (2^-150 x 2^100).
// One warp a row, without shared memory, so that blocks fit beside the first
// kernel's CTAs and are there when it ends.
template <int DIM, int R>
__global__ void __launch_bounds__(256) join_kernel(const AttendArgs g) {
  constexpr int E = DIM / 32;  // elements a lane
  constexpr bool ROWS = R == 256;  // written by threads that own rows
  const int lane = threadIdx.x & 31, r = blockIdx.y * 8 + (threadIdx.x >> 5);
  // (no start_next here: the next call's CTAs, let in among these, made that
  // call slower by up to 20%)
  wait_for_previous();
  const int4 j0 = g.joins[2 * blockIdx.x], j1 = g.joins[2 * blockIdx.x + 1];
  const int parts = j0.x;
  if (parts <= 0 || r >= static_cast<long long>(j0.z) * g.G - j1.x) return;
  const int c0 = blockIdx.x;
  auto slot = [&](int p) { return static_cast<size_t>(p == 0 ? 2 * (c0 - 1) + 1 : 2 * (c0 + p - 1)); };
  auto at = [&](int p) { return slot(p) * R + r; };  // the part's row
  float m = -INFINITY;
  for (int p = lane; p < parts; p += 32) {
    const float x = g.stats[at(p)];
    m = x > m || x != x ? x : m;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float x = __shfl_xor_sync(0xffffffffu, m, o);
    m = x > m || x != x ? x : m;  // NaN stays
  }
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f, acc[E] = {};
  for (int p0 = 0; p0 < parts; p0 += 32) {
    const float wt = p0 + lane < parts ? exp2f(0.5f * (g.stats[at(p0 + lane)] - ref)) : 0.f;
    l = fmaf(wt, wt, l);
    const int n = min(32, parts - p0);
#pragma unroll 8
    for (int p = 0; p < n; ++p) {
      const float w = __shfl_sync(0xffffffffu, wt, p);
      const float* x = g.partial + (ROWS ? (slot(p0 + p) * (DIM / 4) + lane * E / 4) * R * 4 +
                                               r * 4 + lane * E % 4
                                         : at(p0 + p) * DIM + lane * E);
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
  const int i = (j1.x + r) / g.G, hq = j0.w * g.G + (j1.x + r) % g.G;
  if (lane == 0 && g.lse != nullptr)
    g.lse[static_cast<size_t>(hq) * g.T + j0.y + i] = (ref + log2f(l)) * kLn2;
  __nv_bfloat162* out = reinterpret_cast<__nv_bfloat162*>(
      g.o + (static_cast<size_t>(j0.y + i) * g.H + hq) * DIM + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2)
    out[e / 2] = __floats2bfloat162_rn(inv == 0.f ? 0.f : acc[e] * inv,
                                       inv == 0.f ? 0.f : acc[e + 1] * inv);
}

template <int DIM, int R>
inline bool launch_join(int grid, cudaStream_t s, const AttendArgs& g) {
  return launch_after(join_kernel<DIM, R>, dim3(grid, R / 8), 256, 0, s, g);
}

// launch_after for a kernel whose shared-memory limit has to be raised: once on a
// device, and again if a launch fails (a new context does not have it).
template <class... P, class... A>
inline bool launch_large(void (*kern)(P...), std::atomic<unsigned long long>& raised, dim3 grid,
                         int threads, size_t smem, cudaStream_t s, const A&... args) {
  auto raise = [&]() {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(smem)) == cudaSuccess;
  };
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(raised.load(std::memory_order_relaxed) & bit)) {
    if (!raise()) return false;
    raised.fetch_or(bit, std::memory_order_relaxed);
  }
  return launch_after(kern, grid, threads, smem, s, args...) ||
         (raise() && launch_after(kern, grid, threads, smem, s, args...));
}

// The kernel for many query rows (256 an item).
flamia_status attend_rows(const flamia_kvcache* c, const AttendArgs& g, cudaStream_t s);

}  // namespace flamia
