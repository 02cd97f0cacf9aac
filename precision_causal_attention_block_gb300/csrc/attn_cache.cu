// Attention of new tokens over the paged MXFP8 cache.
//
// The product is turned around so that the cache fills the tensor core's M:
// per 128-key tile S^T = K Q^T (M = 128 keys) and O^T += V^T P^T (M = d), with
// the few query rows of one K / V head (group x new tokens, R of them) as N.  K
// and V go from HBM to the tensor core by TMA as the E4M3 codes that the cache
// holds, V read MN-major, so nothing converts or transposes them; BF16 queries
// and float32 weights become sums of E4M3 terms instead, side by side in N:
//   q 2^-e = h + 2^-4 l              (e per row; exact for the elements above
//                                     2^-13 of the row's largest),
//   w      = h + 2^-5 m + 2^-10 l    (relative error at most 2^-14, floor 2^-23
//                                     of the largest weight; with 16 and 32 rows of
//                                     w rounded to FP16, 2^-11),
// which costs N = 2 R and 3 R columns of a product that reads M = 128 rows of
// shared memory in any case.
//
// The key factor 2^eK multiplies the score x (in log2 units); V's 2^eV goes into
// the weight, as the thread that owns a key adds eV to its score:
//   w = 2^(x + eV - ref + kShift),   l = sum w 2^(E0 - eV),
//   o = O^T 2^E0 / l,   log2 sum 2^x = ref - kShift - E0 + log2 l,
// with one integer reference a row (a running maximum of x + eV) and one
// integer E0 (a running maximum of eV) for all rows.  What float32 cannot hold beside
// the rest of l goes to a sum with an exponent of its own, kept a row in shared memory
// (Sum): l itself whenever E0 rises (lifted to the new E0 it could leave float32, and
// a reference that moved along would push the next weights, which count as much, under
// their range), and the keys whose values are more than 2^kLow below E0 (zero values
// under a heavy first token; or rows that do not see the large value beside them).
// References move only when a tile exceeds them by more than kSlack, which the one
// barrier of a tile votes on; O^T is then rescaled in tensor memory.
//
// Work: the key tiles of all (sequence, K / V head, row tile) items are laid end
// to end, with kItemCost tiles' worth for each item's own steps, and cut into
// equal runs, one for each resident CTA, so that a batch of ragged lengths keeps
// every SM reading until the end (single and drafted tokens, chunks of a long
// prompt; the early row tiles of a prompt end before their share, see seq_work).  A
// CTA finishes the items that lie whole inside its run; of the (at most two) it shares
// it leaves o and log2 sum 2^x in the workspace, and a second small kernel, launched
// with programmatic dependent launch, joins them in order of position (no atomics:
// results do not depend on timing).  Where the page table is too narrow for more than
// kWholeTiles tiles an item, items stay whole and the second kernel is not
// launched.
//
// Warps 0-3 (16 and 32 rows: 0-7, two halves of the rows): softmax (thread = key =
// TMEM lane); then one TMA producer warp and one MMA issuer warp.
//
// (More query rows than 96 a K / V head: attn_cache_rows.cu.)
//
// Measured: 96 sequences with one new token over 16 .. 16,384 cached (32 / 8 heads
// of 128) 100 us, 5.75 TB/s of codes and scales; one token over 131,072 (32 heads of
// 64) 100 us, 5.45 TB/s; 48 sequences with 4 drafted tokens, a window of 4,096 (16 /
// 4 heads of 128) 54 us, 3.7 TB/s.  HBM bounds the first two, the softmax warps'
// work and waits for a tile (some 2,500 cycles with 8 or 16 rows, 4,000 with 32,
// two or three tiles at a time on an SM) the last.
#include <cuda_bf16.h>

#include <cmath>

#include "attend.cuh"

namespace flamia {
namespace {

constexpr float kUnset = 1e30f; // -reference of a row that has seen no key yet
constexpr int kUnseen = -200;   // eV of a key that no row sees
constexpr int kWhole = 1 << 8;  // every row sees every key of a tile

// ------------------------------------------------------------------ PTX

// 16-byte multiples from global to shared memory; completes on an mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// Barrier of the N threads of the softmax warps that also ORs a predicate over
// them.
template <int N>
__device__ __forceinline__ bool softmax_vote(bool p) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<int>(p)), "n"(N)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void sts64(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// Four FP16 weights (two pairs): their E4M3 codes in one word, and 32 (w - code)
// in place of the weights (exact).
__device__ __forceinline__ uint32_t take_term(uint32_t& a, uint32_t& b) {
  uint32_t w;
  const uint32_t p32 = 0x50005000u, n32 = 0xD000D000u;  // 32, -32
  asm("{\n\t.reg .b16 ca, cb;\n\t.reg .b32 ha, hb, ta, tb;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 ca, %0;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 cb, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 ha, ca;\n\t"
      "cvt.rn.f16x2.e4m3x2 hb, cb;\n\t"
      "mul.rn.f16x2 ta, %0, %3;\n\t"
      "mul.rn.f16x2 tb, %1, %3;\n\t"
      "fma.rn.f16x2 %0, ha, %4, ta;\n\t"
      "fma.rn.f16x2 %1, hb, %4, tb;\n\t"
      "mov.b32 %2, {ca, cb};\n\t}"
      : "+r"(a), "+r"(b), "=r"(w)
      : "r"(p32), "r"(n32));
  return w;
}
// Four FP16 values as E4M3 codes.
__device__ __forceinline__ uint32_t e4m3x4_of_half(uint32_t a, uint32_t b) {
  uint32_t w;
  asm("{\n\t.reg .b16 ca, cb;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 ca, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 cb, %2;\n\t"
      "mov.b32 %0, {ca, cb};\n\t}"
      : "=r"(w)
      : "r"(a), "r"(b));
  return w;
}
// The same with float32 weights.
__device__ __forceinline__ uint32_t take_term(float2& a, float2& b) {
  uint32_t w, ha, hb;
  asm("{\n\t.reg .b16 ca, cb;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 ca, %4, %3;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 cb, %6, %5;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, ca;\n\t"
      "cvt.rn.f16x2.e4m3x2 %2, cb;\n\t"
      "mov.b32 %0, {ca, cb};\n\t}"
      : "=r"(w), "=r"(ha), "=r"(hb)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  const float2 n32 = make_float2(-32.f, -32.f), p32 = make_float2(32.f, 32.f);
  a = __ffma2_rn(__half22float2(*reinterpret_cast<const __half2*>(&ha)), n32, __fmul2_rn(a, p32));
  b = __ffma2_rn(__half22float2(*reinterpret_cast<const __half2*>(&hb)), n32, __fmul2_rn(b, p32));
  return w;
}

__device__ __forceinline__ float2 as_f2(uint32_t a, uint32_t b) {
  return make_float2(__uint_as_float(a), __uint_as_float(b));
}

// ------------------------------------------------------------------ kernel

template <int DIM, int R>
struct Cfg {
  static constexpr int kHalves = R == 8 ? 1 : 2;     // softmax warpgroups
  static constexpr int kRows = R / kHalves;         // rows of a softmax thread
  static constexpr int kSoftmax = 128 * kHalves;    // softmax threads
  static constexpr int kThreads = kSoftmax + 64;
  static constexpr int kCtas = R == 8 ? 3 : 2;      // resident CTAs per SM
  // Stages.  32 rows: K is read once its scores are there and V a softmax later,
  // so each has a ring of its own, and the scale bytes (and which pieces were
  // loaded) one that is at least two longer, as the softmax of a tile is done two
  // score products later (a chunk of 512 tokens over 8,192: 284 -> 257 us).  With
  // fewer rows, where HBM sets the pace, K, V and scales of a tile share a stage
  // and a barrier (96 ragged contexts: 102 us against 128).
  static constexpr bool kSplit = R == 32;
  static constexpr int kKS = (R == 8 ? 2 : 3) * (128 / DIM);
  static constexpr int kVS = (R == 16 ? 3 : 2) * (128 / DIM);
  static constexpr int kSS = kSplit ? 8 : kKS;
  static_assert(kSplit ? kSS >= kKS + 2 : kKS == kVS, "rings");
  static constexpr int kTileBytes = 128 * DIM;
  // 16 and 32 rows are bound by the softmax warps: their weights go through FP16
  // (relative error 2^-11)
  static constexpr bool kHalfWeights = R >= 16;
  // The last term ends 2^-20 below 1 (half of E4M3's smallest step, twice 2^-5 down),
  // and the largest weight is between 2^(kShift - 1) and 2^(kShift + kSlack)
  static constexpr float kShift = 4.f;           // log2 of a weight at the reference
  static constexpr float kSlack = 8.f - kShift;  // weights <= 2^8 < 448
  static constexpr int kNS = 2 * R;                 // columns of S^T
  static constexpr int kNO = R == 8 ? 32 : 3 * R;   // columns of O^T
  static constexpr int kAtoms = (kNO + 31) / 32;    // P^T: 32 columns x 128 keys each
  static constexpr uint32_t kColO = 2 * kNS;
  static constexpr uint32_t kCols = R == 8 ? 64 : R == 16 ? 128 : 256;
  static_assert(kColO + kNO <= kCols, "tensor memory");
};

template <int DIM, int R>
struct Smem {
  using C = Cfg<DIM, R>;
  alignas(1024) uint8_t v[C::kVS][C::kTileBytes];
  alignas(1024) uint8_t k[C::kKS][C::kTileBytes];
  alignas(1024) uint8_t p[C::kAtoms * 4096];
  alignas(1024) uint8_t q[2 * R * DIM];
  alignas(128) uint8_t ks[C::kSS][128];
  alignas(128) uint8_t vs[C::kSS][128];
  alignas(16) float qf[R];      // 2^e of a row x softmax scale x log2 e
  alignas(16) float nref[R];    // kShift - reference
  alignas(16) float fac[R];     // change of scale of O^T and l
  float ve[R];                  // for o
  Sum past[R];                  // sum 2^(x + nref) of what is not in l
  float far[4][R], fare[4][R];  // a tile's share of it, by warp
  int has[R];                   // the row has a reference
  int large;                    // some row's is beyond kLarge
  bool nan[2][128];  // a half-seen key's value holds a NaN (by tile parity)
  alignas(16) int pos[R];       // position of a row's token, -1: no such row
  alignas(16) int orow[R];      // its row of o, -1: none
  float red[4][R];
  int2 rede[C::kSoftmax / 32];
  uint64_t k_full[C::kKS], k_empty[C::kKS], v_full[C::kVS], v_empty[C::kVS];
  uint64_t sc_full[C::kSS];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t q_full, o_empty, drained;
  uint64_t seg_full[kSegSlots], seg_empty[kSegSlots];
  Segment seg[kSegSlots];
  int2 tile[C::kSS];            // first key; pieces that were loaded, kWhole
  int plan_b, sharer;
  SeqWork plan_seq;
  long long plan_off, plan_u0, plan_u1, plan_total;
  long long scan[C::kThreads / 32];
  uint32_t tmem_base;
  volatile int abort;
};

// The queries of a segment held by one softmax thread: 16-byte chunks of rows
// r0 + tid / (d / 8), r0 = 0, kPer, 2 kPer, ...
template <int DIM, int R>
struct Queries {
  using C = Cfg<DIM, R>;
  static constexpr int kLanes = DIM / 8, kPer = C::kSoftmax / kLanes;
  static constexpr int kIters = (R + kPer - 1) / kPer;
  uint4 w[kIters];

  __device__ __forceinline__ void load(const AttendArgs& g, const Segment& sg, int tid) {
#pragma unroll
    for (int it = 0; it < kIters; ++it) {
      const int r = it * kPer + tid / kLanes;
      const int row = sg.row0 + r;
      w[it] = make_uint4(0, 0, 0, 0);
      if (r < R && row < static_cast<long long>(sg.n) * g.G) {
        const int i = row / g.G, hq = sg.hk * g.G + row - i * g.G;
        w[it] = *reinterpret_cast<const uint4*>(g.q + (sg.s + i) * g.q_stride +
                                                static_cast<long long>(hq) * DIM +
                                                tid % kLanes * 8);
      }
    }
  }

  // Two E4M3 terms a row into shared memory (K-major rows of DIM bytes, 16-byte
  // chunks swizzled as TMA does), and the row factors.
  __device__ __forceinline__ void split(uint8_t* q, float* qf, float scale_log2, int tid) const {
    const int ch = tid % kLanes;
#pragma unroll
    for (int it = 0; it < kIters; ++it) {
      const int r = it * kPer + tid / kLanes;
      float x[8];
      const uint32_t ww[4] = {w[it].x, w[it].y, w[it].z, w[it].w};
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(ww[j] << 16);
        x[2 * j + 1] = __uint_as_float(ww[j] & 0xFFFF0000u);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!(fabsf(x[j]) < INFINITY)) x[j] = __uint_as_float(0x7FC00000u);
        amax = fmaxf(amax, fabsf(x[j]));  // of the finite ones
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const int e = roundup_exponent(amax);
      const float inv = exp2i(-e);
      uint32_t hc[4], lc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = x[2 * j] * inv, c = x[2 * j + 1] * inv;
        hc[j] = cvt_e4m3x2(a, c);
        const float2 h = e4m3x2_to_float2(hc[j]);
        lc[j] = cvt_e4m3x2((a - h.x) * 16.f, (c - h.y) * 16.f);
      }
      if (r < R) {
        auto at = [&](int n) {
          const int c16 = ch >> 1;
          const int sw = DIM == 128 ? (c16 ^ (n & 7)) : (c16 ^ ((n >> 1) & 3));
          return reinterpret_cast<uint2*>(q + n * DIM + sw * 16 + (ch & 1) * 8);
        };
        *at(r) = make_uint2(hc[0] | (hc[1] << 16), hc[2] | (hc[3] << 16));
        *at(R + r) = make_uint2(lc[0] | (lc[1] << 16), lc[2] | (lc[3] << 16));
        if (ch == 0) qf[r] = scale_log2 * (e < -126 ? 0x1p-127f : exp2i(e));
      }
    }
  }
};

template <int DIM, int R, int KEYS>
__global__ void __launch_bounds__(Cfg<DIM, R>::kThreads, Cfg<DIM, R>::kCtas)
    attend_kernel(const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const AttendArgs g) {
  using C = Cfg<DIM, R>;
  constexpr int kProducer = C::kSoftmax / 32, kIssuer = kProducer + 1;
  extern __shared__ uint8_t smem_raw[];
  Smem<DIM, R>& sm = *reinterpret_cast<Smem<DIM, R>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < C::kKS; ++i) {
      mbar_init(smem_u32(&sm.k_full[i]), 1);
      mbar_init(smem_u32(&sm.k_empty[i]), 1);
    }
    for (int i = 0; i < C::kSS; ++i) mbar_init(smem_u32(&sm.sc_full[i]), 1);
    for (int i = 0; i < C::kVS; ++i) {
      mbar_init(smem_u32(&sm.v_full[i]), 1);
      mbar_init(smem_u32(&sm.v_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.s_full[i]), 1);
      mbar_init(smem_u32(&sm.p_full[i]), C::kSoftmax / 32);
      mbar_init(smem_u32(&sm.pv_done[i]), 1);
    }
    mbar_init(smem_u32(&sm.q_full), C::kSoftmax / 32);
    mbar_init(smem_u32(&sm.o_empty), C::kSoftmax / 32);
    mbar_init(smem_u32(&sm.drained), 1);
    for (int i = 0; i < kSegSlots; ++i) {
      mbar_init(smem_u32(&sm.seg_full[i]), 1);
      mbar_init(smem_u32(&sm.seg_empty[i]), kProducer + 1);  // softmax warps, MMA issuer
    }
    sm.abort = 0;
    fence_barrier_init();
  }
  if (warp == kIssuer) {
    tmem_alloc(smem_u32(&sm.tmem_base), C::kCols);
    tmem_relinquish();
    // (only now: the next kernel's CTAs, which wait for this one's end, must not hold
    // tensor memory that a CTA of this one still asks for)
    start_next();
  }
  wait_for_previous();
  check_offsets(g.cu, g.ndocs, g.T, static_cast<long long>(blockIdx.x) * C::kThreads + tid,
                static_cast<long long>(gridDim.x) * C::kThreads, g.status);
  tc_fence_before();
  make_plan<R, KEYS, C::kThreads>(g, sm);
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  if (warp == kProducer) {
    // ------------------------------------------------------------ producer
    const long long u0 = sm.plan_u0, u1 = sm.plan_u1, total = sm.plan_total;
    const int pieces = g.page_size >= 128 ? 1 : 128 / g.page_size;
    const int piece = 128 / pieces;  // keys
    if (lane == 0) {
      prefetch_tensormap(&map_k);
      prefetch_tensormap(&map_v);
    }
    int b = sm.plan_b, tc = 0, kc = 0, vc = 0, nseg = 0;  // kc, vc: tiles of K and V issued
    long long u = u0;
    bool ok = true, first = true;
    int4 join0 = make_int4(0, 0, 0, 0), join1 = make_int4(0, 0, 0, 0);
    // place inside sequence b: item (hk, rt), unit o of it
    SeqWork w{};
    int hk = 0, rt = 0, o = 0;
    if (u < u1) {
      w = sm.plan_seq;
      const long long item = mul_div(sm.plan_off, 1, w.units);
      o = static_cast<int>(sm.plan_off - item * w.units);
      hk = static_cast<int>(mul_div(item, 1, w.row_tiles));
      rt = static_cast<int>(item - static_cast<long long>(hk) * w.row_tiles);
    }
    while (ok) {
      Segment sg{};
      int hi = 0, wlo = 0, pf = 0, pl = 0;  // pf, pl: positions of the first and last row
      if (u >= u1) {
        sg.s = -1;
      } else {
        const int take = static_cast<int>(min(u1 - u, static_cast<long long>(w.units - o)));
        const bool over = of_prefix<KEYS>(b), cut = !g.whole;
        const int cost = cut ? kItemCost<R> : 0;
        const int i0 = max(o - cost, 0);
        const int i1 = cut ? max(o + take - cost, 0) : w.tiles;
        sg.s = w.s;
        sg.n = w.n;
        sg.start = w.start;
        sg.hk = hk;
        sg.row0 = rt * R;
        pf = w.start + sg.row0 / g.G;
        // (rows of a call are below 2^31)
        const unsigned last = min(static_cast<unsigned>(w.n) * g.G, static_cast<unsigned>(sg.row0 + R)) - 1;
        pl = w.start + static_cast<int>(last / g.G);
        hi = over ? g.shared * 128 : max(pl + 1, 0);
        wlo = g.window > 0 ? max(pf - g.window + 1, 0) : 0;
        const bool sharing = KEYS != kAll && !over && shares(g, w.start, w.n);
        sg.wt = sharing ? g.shared : wlo >> 7;
        sg.ns = KEYS == kAll ? min((g.sinks + 127) >> 7, sg.wt) : 0;
        const int list = sg.ns + max(((hi + 127) >> 7) - sg.wt, 0);
        sg.i0 = min(i0, list);
        sg.i1 = min(i1, list);
        sg.slot = -1;
        if (i0 > 0)
          sg.slot = 2 * blockIdx.x;
        else if (i1 < w.tiles)
          sg.slot = 2 * blockIdx.x + 1;
        if (KEYS != kAll && i0 == 0 && i1 > 0)
          sg.parts = (cut ? parts_from_here<R>(g, u - o, w.units, total) : 1) |
                     (over ? kOver : 0) | (sharing ? kShares : 0);
        if (KEYS == kAll && first && i0 > 0) {
          // the second CTA of an item has it joined: parts are the CTA before
          // this one (slot 1) and slots 0 from here on
          const long long ctas = active_ctas<R>(g, total), c = blockIdx.x, ui = u0 - o;
          if (c > 0 && mul_div(total, c - 1, ctas) <= ui + kItemCost<R>) {
            const long long last = div_up((ui + w.units) * ctas, total) - 1;
            join0 = make_int4(static_cast<int>(last - c + 2), w.s, w.n, hk);
            join1 = make_int4(sg.row0, 0, 0, 0);
          }
        }
        if (!over && lane == 0 && hk == 0 && rt == 0 && i0 == 0) {
          const int raw = g.starts != nullptr ? g.starts[seq_of<KEYS>(b)] : 0;
          if (raw > g.cap - w.n) report(g.status, FLAMIA_DEV_BAD_PAGE);
        }
        first = false;
        u += take;
        if (i1 <= i0) continue;  // the run ends before the item's first tile
      }
      // hand it on
      const int sl = nseg % kSegSlots;
      if (nseg >= kSegSlots)
        ok = mbar_wait_w_ab(smem_u32(&sm.seg_empty[sl]), ((nseg / kSegSlots) - 1) & 1, &sm.abort);
      if (!ok) break;
      if (lane == 0) {
        sm.seg[sl] = sg;
        mbar_arrive(smem_u32(&sm.seg_full[sl]));
      }
      __syncwarp();
      ++nseg;
      if (sg.s < 0) break;
      // its key tiles; the page-table entries of a tile are read one tile ahead
      const int seq = of_prefix<KEYS>(b) ? sm.sharer : seq_of<KEYS>(b);
      const int32_t* row = g.table + static_cast<long long>(seq) * g.table_stride;
      auto entry = [&](int i, bool& need, int& in_page) {
        const int kp = tile_of(sg, i) * 128 + lane * piece;
        need = lane < pieces && kp < hi &&
               (g.window == 0 || kp + piece > wlo || kp < g.sinks);
        const int slot = kp / g.page_size;
        in_page = kp - slot * g.page_size;
        return need && slot < g.table_stride ? row[slot] : -1;
      };
      bool need;
      int in_page;
      int page = sg.i0 < sg.i1 ? entry(sg.i0, need, in_page) : -1;
      // the next item meanwhile
      o = 0;
      if (u < u1 && ++rt == w.row_tiles) {
        rt = 0;
        if (++hk == g.H_kv) {
          hk = 0;
          do {
            w = seq_work<R, KEYS>(g, ++b, 0);  // there is one: u < u1
          } while (w.row_tiles == 0 && seq_of<KEYS>(b) + 1 < g.ndocs);
        }
      }
      for (int i = sg.i0; i < sg.i1; ++i, ++tc) {
        const int pg = page, ip = in_page;
        const bool nd = need, good = nd && pg >= 0 && pg < g.num_pages;
        if (i + 1 < sg.i1) page = entry(i + 1, need, in_page);
        if (nd && !good) report(g.status, FLAMIA_DEV_BAD_PAGE);
        const unsigned mask = __ballot_sync(0xffffffffu, good);
        const int n = __popc(mask), pr = lane * piece;  // first key of the piece in the tile
        const int prow = pg * g.H_kv + sg.hk;
        const long long sc = static_cast<long long>(prow) * g.page_size + ip;
        const int kt = tc % C::kKS, vt = tc % C::kVS, ss = tc % C::kSS;
        const int k0 = tile_of(sg, i) * 128;
        const bool whole = n == pieces && k0 + 127 <= pf &&
                           (g.window == 0 || k0 > pl - g.window || k0 + 127 < g.sinks);
        const int2 info = make_int2(k0, static_cast<int>(mask) | (whole ? kWhole : 0));
        auto wait_v_slot = [&]() {
          return tc < C::kVS ||
                 mbar_wait_w_ab(smem_u32(&sm.v_empty[vt]), ((tc / C::kVS) - 1) & 1, &sm.abort);
        };
        auto load_k = [&](uint32_t bar, uint32_t sc_bar) {
          tma_load_3d(smem_u32(sm.k[kt]) + pr * DIM, &map_k, bar, 0, ip, prow);
          bulk_load(smem_u32(sm.ks[ss]) + pr, g.k_scales + sc, piece, sc_bar);
          bulk_load(smem_u32(sm.vs[ss]) + pr, g.v_scales + sc, piece, sc_bar);
        };
        auto load_v = [&](uint32_t bar) {
          tma_load_3d(smem_u32(sm.v[vt]) + pr * DIM, &map_v, bar, 0, ip, prow);
        };
        const uint32_t kbar = smem_u32(&sm.k_full[kt]);
        if constexpr (C::kSplit) {
          if (tc >= C::kKS)
            ok = mbar_wait_w_ab(smem_u32(&sm.k_empty[kt]), ((tc / C::kKS) - 1) & 1, &sm.abort);
          if (!ok) break;
          const uint32_t sbar = smem_u32(&sm.sc_full[ss]), vbar = smem_u32(&sm.v_full[vt]);
          if (lane == 0) {
            sm.tile[ss] = info;
            mbar_arrive_expect_tx(sbar, n * 2 * piece);
            mbar_arrive_expect_tx(kbar, n * piece * DIM);
          }
          __syncwarp();
          if (good) load_k(kbar, sbar);
          ++kc;
          ok = wait_v_slot();
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(vbar, n * piece * DIM);
          __syncwarp();
          if (good) load_v(vbar);
          ++vc;
        } else {
          ok = wait_v_slot();
          if (!ok) break;
          if (lane == 0) {
            sm.tile[ss] = info;
            mbar_arrive_expect_tx(kbar, n * (2 * piece * DIM + 2 * piece));
          }
          __syncwarp();
          if (good) {
            load_k(kbar, kbar);
            load_v(kbar);
          }
          ++kc;
        }
        __syncwarp();
      }
    }
    // what the second kernel has to join for this CTA's first item
    if (KEYS == kAll && lane == 0 && !g.whole) {
      g.joins[2 * blockIdx.x] = join0;
      g.joins[2 * blockIdx.x + 1] = join1;
    }
    // every issued copy has landed before the CTA can exit
    for (int j = max(0, kc - C::kKS); j < kc; ++j)
      ok &= mbar_wait_w(smem_u32(&sm.k_full[j % C::kKS]), (j / C::kKS) & 1) &&
            (!C::kSplit || mbar_wait_w(smem_u32(&sm.sc_full[j % C::kSS]), (j / C::kSS) & 1));
    for (int j = max(0, vc - C::kVS); j < vc; ++j)
      ok &= mbar_wait_w(smem_u32(&sm.v_full[j % C::kVS]), (j / C::kVS) & 1);
    if (!ok) sm.abort = 1;
  } else if (warp == kIssuer) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t lay = DIM == 128 ? kLayoutSW128 : kLayoutSW64;
    constexpr uint32_t sbo = 8 * DIM;
    const uint32_t id_s = idesc_f8(128, C::kNS, 0, 0);
    const uint32_t id_o = idesc_f8(128, C::kNO, 1, 1);
    const uint64_t dk0 = smem_desc(smem_u32(sm.k[0]), 0, sbo, lay);
    const uint64_t dq = smem_desc(smem_u32(sm.q), 0, sbo, lay);
    // head dim 64: M = 128 takes a second 64-row atom; it reads the bytes one
    // tile on (V's next stage or K's first), into lanes 64 .. 127 of O^T, which
    // nobody reads
    const uint64_t dv0 =
        smem_desc(smem_u32(sm.v[0]), DIM == 64 ? C::kTileBytes : 0, sbo, lay);
    // P^T: MN-major, atoms of 32 columns x 8 keys, 4,096 bytes from one set of
    // 32 columns to the next
    const uint64_t dp0 = smem_desc(smem_u32(sm.p), 4096, 256, kLayoutSW32);
    constexpr uint32_t kStep = C::kTileBytes / 16;
    int tc = 0, nlive = 0;
    bool ok = true;
    for (int ns = 0; ok; ++ns) {
      const int sl = ns % kSegSlots;
      ok = mbar_wait_w_ab(smem_u32(&sm.seg_full[sl]), (ns / kSegSlots) & 1, &sm.abort);
      if (!ok) break;
      const int s = sm.seg[sl].s, nt = sm.seg[sl].i1 - sm.seg[sl].i0;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.seg_empty[sl]));
      if (s < 0) break;
      if (nt <= 0) continue;
      // S^T of tile t of the segment
      auto issue_s = [&](int t) {
        const int x = tc + t, st = x % C::kKS, sb = x & 1;
        if (lane == 0) {
#pragma unroll
          for (int ks = 0; ks < DIM / 32; ++ks)
            mma_f8(tmem + sb * C::kNS, dk0 + st * kStep + 2 * ks, dq + 2 * ks, id_s, ks > 0);
          tc_commit(smem_u32(&sm.s_full[sb]));
          if (C::kSplit) tc_commit(smem_u32(&sm.k_empty[st]));
        }
        __syncwarp();
      };
      auto wait_k = [&](int t) {
        const int x = tc + t;
        return mbar_wait_w_ab(smem_u32(&sm.k_full[x % C::kKS]), (x / C::kKS) & 1, &sm.abort);
      };
      ok = mbar_wait_w_ab(smem_u32(&sm.q_full), nlive & 1, &sm.abort) && wait_k(0);
      if (!ok) break;
      tc_fence_after();
      issue_s(0);
      for (int t = 0; t < nt && ok; ++t) {
        // the next scores first, if their keys come before this tile's weights
        const int x = tc + t, st = x % C::kVS;
        bool ahead = false;
        if (t + 1 < nt) {
          const int y = x + 1;
          const uint64_t t0 = globaltimer_ns();
          for (int spin = 0;; ++spin) {
            if (__all_sync(0xffffffffu,
                           mbar_test(smem_u32(&sm.k_full[y % C::kKS]), (y / C::kKS) & 1))) {
              tc_fence_after();
              issue_s(t + 1);
              ahead = true;
              break;
            }
            if (__all_sync(0xffffffffu, mbar_test(smem_u32(&sm.p_full[x & 1]), (x >> 1) & 1)))
              break;
            // (bounded: the wait below reports)
            if ((spin & 63) == 63 && __any_sync(0xffffffffu, sm.abort || globaltimer_ns() - t0 >
                                                                             kWaitTimeoutNs))
              break;
          }
        }
        ok = mbar_wait_w_ab(smem_u32(&sm.p_full[x & 1]), (x >> 1) & 1, &sm.abort);
        if (C::kSplit && ok)
          ok = mbar_wait_w_ab(smem_u32(&sm.v_full[st]), (x / C::kVS) & 1, &sm.abort);
        // O^T of the segment before has been read
        if (ok && t == 0 && nlive > 0)
          ok = mbar_wait_w_ab(smem_u32(&sm.o_empty), (nlive - 1) & 1, &sm.abort);
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint64_t dv = dv0 + st * kStep + ks * (32 * DIM / 16);
            mma_f8(tmem + C::kColO, dv, dp0 + ks * (1024 / 16), id_o, t > 0 || ks > 0);
          }
          tc_commit(smem_u32(&sm.pv_done[x & 1]));
          tc_commit(smem_u32(&sm.v_empty[st]));
        }
        __syncwarp();
        if (t + 1 < nt && !ahead) {
          ok = wait_k(t + 1);
          if (!ok) break;
          tc_fence_after();
          issue_s(t + 1);
        }
      }
      tc += nt;
      ++nlive;
    }
    if (!ok) {
      sm.abort = 1;
      // what was issued ends before shared memory and tensor memory go
      if (lane == 0) tc_commit(smem_u32(&sm.drained));
      __syncwarp();
      mbar_wait_w(smem_u32(&sm.drained), 0);
    }
  } else {
    // ------------------------------------------------------------ softmax
    constexpr int RW = C::kRows;
    // This thread's rows: eight from r0 on, and with 32 an item eight from r0 + 16 on if it
    // has any there.  (A row is a column of the products, and nothing else depends on what stays
    // in one without a row.  131,072 keys shared by 24 rows of 32 heads of 64: 265 -> 221
    // us; 16,384 by 32 rows of 16 heads of 128: 61.7 -> 62.6.  Plain calls, 16 sequences over
    // 4,096: 24 rows of 16 heads of 64 77.8 -> 71.6, 25 77.8 -> 75.8, 17 of 8 heads of 128 58.3
    // -> 56.3; 32 rows, 8 over 8,192, 32 heads of 64 124.9 -> 122.9, 8 of 128 59.4 and 60.4 ->
    // 58.4 and 59.4; one over 16,384 41.0 in both.  The same for the first eight costs 16 rows
    // an item 55 -> 58 us.)
    constexpr int kNext = 8 * C::kHalves;
    const int half = C::kHalves == 1 ? 0 : warp >> 2, r0 = half * 8;
    const int key_in = tid & 127;                   // its key inside a tile
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    auto vote = [&](bool p) { return softmax_vote<C::kSoftmax>(p); };
    auto sync = [&]() { named_barrier_sync(1, C::kSoftmax); };
    int tc = 0, ss = 0, sph = 0;  // tiles so far; their place and phase in the ring of scales
    bool ok = true, late = false;  // late: a wait ran out where the warps cannot part
    auto fail = [&]() {
      late = true;
      sm.abort = 1;
    };
    // a segment's queries are loaded while the one before ends; its ring slot is
    // free again when the segment is done
    Queries<DIM, R> queries;
    auto await = [&](int n) {
      const bool got = mbar_wait_w_ab(smem_u32(&sm.seg_full[n % kSegSlots]),
                                      (n / kSegSlots) & 1, &sm.abort);
      if (got) {
        const Segment& x = sm.seg[n % kSegSlots];
        if (x.s >= 0 && x.i1 > x.i0) queries.load(g, x, tid);
      }
      return got;
    };
    ok = await(0);
    for (int ns = 0;; ++ns) {
      // (also: everybody is done with the row tables of the segment before)
      if (vote(!ok || late)) {
        ok = false;
        break;
      }
      const Segment& sg = sm.seg[ns % kSegSlots];
      if (sg.s < 0) break;
      const int nt = sg.i1 - sg.i0;
      const int rows = static_cast<int>(
          min(static_cast<long long>(R), static_cast<long long>(sg.n) * g.G - sg.row0));
      if (tid < R) {
        const int i = (sg.row0 + tid) / g.G, hq = sg.hk * g.G + (sg.row0 + tid) % g.G;
        const bool live = tid < rows;
        sm.pos[tid] = live ? sg.start + i : -1;
        sm.orow[tid] = live ? (sg.s + i) * g.H + hq : -1;
        sm.nref[tid] = C::kShift;
        sm.has[tid] = 0;
        sm.past[tid] = Sum{0.f, kNoExponent};
      }
      if (tid == 0) sm.large = 0;
      if (nt > 0) {
        queries.split(sm.q, sm.qf, g.scale_log2, tid);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.q_full));
      }
      sync();  // row tables
      auto has_rows = [&](int c) { return c == 0 || r0 + c < rows; };
      float2 l[RW / 2];
#pragma unroll
      for (int r = 0; r < RW / 2; ++r) l[r] = make_float2(0.f, 0.f);
      // l of a row over the keys (threads); the caller's barrier, then sum_of(row)
      auto sum_keys = [&]() {
#pragma unroll
        for (int r = 0; r < RW; ++r) {
          float s = r & 1 ? l[r / 2].y : l[r / 2].x;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          if (lane == 0) sm.red[warp & 3][r0 + r / 8 * kNext + r % 8] = s;
        }
      };
      auto sum_of = [&](int r) {
        return (sm.red[0][r] + sm.red[1][r]) + (sm.red[2][r] + sm.red[3][r]);
      };
      int e0 = -127;
      bool large = false;
#pragma unroll 1
      for (int t = 0; t < nt; ++t, ++tc) {
        const int buf = tc & 1;
        // the scores and the scale bytes (a split ring's K barrier may be two phases
        // on by now).  A wait that runs out ends the other roles' waits and this
        // role at the next segment: until then all softmax warps keep step.
        const uint32_t sbar = smem_u32(&sm.s_full[buf]);
        const uint32_t cbar = smem_u32(C::kSplit ? &sm.sc_full[ss] : &sm.k_full[ss]);
        if (R == 8 ? !mbar_wait_w_ab(sbar, (tc >> 1) & 1, &sm.abort) ||
                         !mbar_wait_w_ab(cbar, sph, &sm.abort)
                   : !wait_both(sbar, (tc >> 1) & 1, cbar, sph, &sm.abort))
          fail();
        tc_fence_after();
        int ev = sm.vs[ss][key_in] - 127;  // V's exponent; kUnseen
        const float kf = pow2_byte(sm.ks[ss][key_in]);
        const bool whole = (sm.tile[ss].y & kWhole) != 0;
        if (!whole) {  // some rows do not see some keys
          const int2 info = sm.tile[ss];
          const int st = tc % C::kVS, key = info.x + key_in;
          if (C::kSplit &&
              !mbar_wait_w_ab(smem_u32(&sm.v_full[st]), (tc / C::kVS) & 1, &sm.abort))
            fail();
          const int pf = sg.start + sg.row0 / g.G;               // positions of the first
          const int pl = sg.start + (sg.row0 + rows - 1) / g.G;  // and the last row
          const bool here = (info.y >> piece_of(key_in, g.page_size)) & 1;
          const bool first = g.window == 0 || key < g.sinks;
          const bool any = here && key <= pl && (first || key > pf - g.window);
          const bool every = here && key <= pf && (first || key > pl - g.window);
          if (!any) ev = kUnseen;
          // A value that some rows see and others do not must not reach the
          // others: 0 x NaN is NaN.  Unseen rows of V are cleared, and half-seen
          // ones that hold a NaN, which moves into the weights of the rows that
          // see them.  (The first half looks; the vote orders the second.)
          if (half == 0) {
            // (each thread starts at another 16 bytes of its row: no bank conflicts)
            uint4* vr = reinterpret_cast<uint4*>(sm.v[st] + key_in * DIM);
            constexpr int kChunks = DIM / 16;
            const int turn = key_in / (128 / DIM);
            bool nan = false;
            if (any && !every) {
#pragma unroll 4
              for (int i = 0; i < kChunks; ++i) {
                const uint4 a = vr[(i + turn) % kChunks];
                const uint32_t aa[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  nan |= ((((aa[j] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0);
              }
            }
            sm.nan[buf][key_in] = nan;
            if (!any || nan) {
#pragma unroll 4
              for (int i = 0; i < kChunks; ++i) vr[(i + turn) % kChunks] = make_uint4(0, 0, 0, 0);
            }
          }
        }
        // x + eV - ref + kShift of rows r0 + c .. + 7.  They are taken anew from
        // tensor memory where they are needed (for the vote, the references, the
        // weights): held in registers over the vote they cost more, in spills.
        auto scores = [&](const int c, float2 (&y)[4]) {
          const float2 kf2 = make_float2(kf, kf);
          const float evf = static_cast<float>(ev);
          const float2 ev2 = make_float2(evf, evf), lo2 = make_float2(0.0625f, 0.0625f);
          uint32_t h[8], lo[8];
          tmem_ld8(tmem + lanes + buf * C::kNS + r0 + c, h);
          tmem_ld8(tmem + lanes + buf * C::kNS + R + r0 + c, lo);
          tmem_ld_wait();
#pragma unroll
          for (int r = 0; r < 8; r += 4) {
            const float4 qf = *reinterpret_cast<const float4*>(sm.qf + r0 + c + r);
            const float4 nr = *reinterpret_cast<const float4*>(sm.nref + r0 + c + r);
            const float2 a = __ffma2_rn(as_f2(lo[r], lo[r + 1]), lo2, as_f2(h[r], h[r + 1]));
            const float2 b =
                __ffma2_rn(as_f2(lo[r + 2], lo[r + 3]), lo2, as_f2(h[r + 2], h[r + 3]));
            y[r / 2] = __ffma2_rn(a, __fmul2_rn(kf2, make_float2(qf.x, qf.y)),
                                  __fadd2_rn(ev2, make_float2(nr.x, nr.y)));
            y[r / 2 + 1] = __ffma2_rn(b, __fmul2_rn(kf2, make_float2(qf.z, qf.w)),
                                      __fadd2_rn(ev2, make_float2(nr.z, nr.w)));
          }
          if (!whole) {
            const int2 info = sm.tile[ss];
            const int key = info.x + key_in;
            const bool here = (info.y >> piece_of(key_in, g.page_size)) & 1;
            const bool first = g.window == 0 || key < g.sinks;
#pragma unroll
            for (int r = 0; r < 8; ++r) {
              const int p = sm.pos[r0 + c + r];
              if (!(here && key <= p && (first || key > p - g.window)))
                (r & 1 ? y[r / 2].y : y[r / 2].x) = -INFINITY;
            }
          }
        };
        // Do the references hold?  On an item's first tile there are none.
        bool move = true;
        if (t > 0) {
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < R; c += kNext) {
            if (!has_rows(c)) break;
            float2 y[4];
            scores(c, y);
#pragma unroll
            for (int r = 0; r < 4; ++r) mx = fmax3(mx, y[r].x, y[r].y);
          }
          move = mx > C::kShift + C::kSlack || ev > e0 + kHigh ||
                 (ev < e0 - kLow && ev != kUnseen);
        }
        move = vote(move);
        if (move) {  // E0, then the rows' references
          const int em = __reduce_max_sync(0xffffffffu, ev);
          const int el = __reduce_min_sync(0xffffffffu, ev == kUnseen ? 127 : ev);
          if (lane == 0) sm.rede[warp] = make_int2(em, el);
          // rows without a reference are measured from 0
          if (tid < R && sm.nref[tid] == kUnset) sm.nref[tid] = C::kShift;
          sync();
          int top = -127, low = 127;
#pragma unroll
          for (int w = 0; w < C::kSoftmax / 32; ++w) {
            top = max(top, sm.rede[w].x);
            low = min(low, sm.rede[w].y);
          }
          if (t == 0) {
            e0 = top;
          } else if (top > e0 + kHigh) {  // (the same in all warps)
            sum_keys();
            sync();
            if (tid < R) sm.past[tid].add(sum_of(tid), -static_cast<float>(e0));
            sync();
#pragma unroll
            for (int r = 0; r < RW / 2; ++r) l[r] = make_float2(0.f, 0.f);
            e0 = top;
          }
          const bool apart = low < e0 - kLow;
#pragma unroll 1
          for (int c = 0; c < R; c += kNext) {
            if (!has_rows(c)) break;
            float2 y[4];
            scores(c, y);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
              const float a = warp_max(r & 1 ? y[r / 2].y : y[r / 2].x);
              if (lane == 0) sm.red[warp & 3][r0 + c + r] = a;
            }
            if (apart) {  // keys that l does not hold
#pragma unroll
              for (int r = 0; r < 8; ++r) {
                float x = (r & 1 ? y[r / 2].y : y[r / 2].x) - static_cast<float>(ev);
                if (ev >= e0 - kLow) x = -INFINITY;
                const float m = ceilf(fmaxf(warp_max(x), kNoExponent));
                float s = ex2_approx(x - m);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                if (lane == 0) {
                  sm.far[warp & 3][r0 + c + r] = s;
                  sm.fare[warp & 3][r0 + c + r] = m;
                }
              }
            }
          }
          sync();
          if (tid < R) {
            const float a = fmaxf(fmaxf(sm.red[0][tid], sm.red[1][tid]),
                                  fmaxf(sm.red[2][tid], sm.red[3][tid]));
            // A row keeps its reference while it holds; one that has seen
            // nothing (or nothing but NaN) has none.
            const float n0 = sm.nref[tid];
            float n1 = n0, f = 1.f;
            if (apart)
              for (int w = 0; w < 4; ++w) sm.past[tid].add(sm.far[w][tid], sm.fare[w][tid]);
            if (tid >= rows) {
              n1 = -kUnset;
            } else if (!sm.has[tid]) {
              const bool now = a > -INFINITY;
              n1 = now ? lowered(n0 - ceilf(a - C::kShift)) : kUnset;
              if (now) sm.past[tid].e += n1 - n0;
              sm.has[tid] = now;
            } else if (a > C::kShift + C::kSlack + room(n0)) {
              n1 = lowered(n0 - ceilf(a - C::kShift));
              f = ex2_approx(n1 - n0);
              sm.past[tid].e += n1 - n0;
            }
            if (tid < rows && n1 != kUnset && fabsf(n1) > kLarge) sm.large = 1;
            sm.nref[tid] = n1;
            sm.fac[tid] = f;
          }
          sync();
          large = sm.large;
#pragma unroll
          for (int r = 0; r < RW; r += 4) {
            const float4 f = *reinterpret_cast<const float4*>(sm.fac + r0 + r / 8 * kNext + r % 8);
            l[r / 2] = __fmul2_rn(l[r / 2], make_float2(f.x, f.y));
            l[r / 2 + 1] = __fmul2_rn(l[r / 2 + 1], make_float2(f.z, f.w));
          }
          if (t > 0) {  // O^T, once the product before has added to it
            if (!mbar_wait_w_ab(smem_u32(&sm.pv_done[buf ^ 1]), ((tc - 1) >> 1) & 1, &sm.abort))
              fail();
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 3 * R; c += kNext) {
              const int in = r0 + c % R, col = c + r0;
              if (R == 32 && in >= rows) continue;
              uint32_t a[8];
              tmem_ld8(tmem + lanes + C::kColO + col, a);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 8; ++i)
                a[i] = __float_as_uint(__uint_as_float(a[i]) * sm.fac[in + i]);
              tmem_st8(tmem + lanes + C::kColO + col, a);
            }
            tmem_st_wait();
          }
        }
        // (whether the product before has read P^T is asked here and looked at
        // when the first weights are there)
        const bool p_free =
            tc == 0 || mbar_test(smem_u32(&sm.pv_done[buf ^ 1]), ((tc - 1) >> 1) & 1);
        // weights and their 8-bit terms
        const float gl = ev < e0 - kLow ? 0.f : exp2i(e0 - ev);
        const float2 g2 = make_float2(gl, gl);
#pragma unroll
        for (int c = 0; c < R; c += kNext) {
          if (!has_rows(c)) break;
          const int at8 = c / kNext * 4;  // in l
          float2 y[4];
          scores(c, y);
          if (!whole && sm.nan[buf][key_in]) {
            const float nv = __uint_as_float(0x7FC00000u);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              if (y[r].x != -INFINITY) y[r].x = nv;
              if (y[r].y != -INFINITY) y[r].y = nv;
            }
          }
          if (large) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              y[r] = make_float2(cut(y[r].x, C::kShift + C::kSlack),
                                 cut(y[r].y, C::kShift + C::kSlack));
          }
          uint32_t tw[3][2];
#pragma unroll
          for (int r = 0; r < 8; r += 4) {
            float2 a = make_float2(ex2_approx(y[r / 2].x), ex2_approx(y[r / 2].y));
            float2 b = make_float2(ex2_approx(y[r / 2 + 1].x), ex2_approx(y[r / 2 + 1].y));
            l[at8 + r / 2] = __ffma2_rn(a, g2, l[at8 + r / 2]);
            l[at8 + r / 2 + 1] = __ffma2_rn(b, g2, l[at8 + r / 2 + 1]);
            if constexpr (C::kHalfWeights) {
              uint32_t ha = half2_of(a), hb = half2_of(b);
              tw[0][r / 4] = take_term(ha, hb);
              tw[1][r / 4] = take_term(ha, hb);
              tw[2][r / 4] = e4m3x4_of_half(ha, hb);
            } else {
              tw[0][r / 4] = take_term(a, b);
              tw[1][r / 4] = take_term(a, b);
              tw[2][r / 4] = cvt_e4m3x4(a.x, a.y, b.x, b.y);
            }
          }
          if (c == 0 && !__all_sync(0xffffffffu, p_free) &&
              !mbar_wait_w_ab(smem_u32(&sm.pv_done[buf ^ 1]), ((tc - 1) >> 1) & 1, &sm.abort))
            fail();
          // P^T: key rows of 32 columns (32 bytes), 16-byte chunks swizzled
#pragma unroll
          for (int term = 0; term < 3; ++term) {
            const int n = term * R + c, col = n + r0;  // column of the first row
            const uint32_t at = smem_u32(sm.p) + (R == 32 ? term : n / 32) * 4096 + key_in * 32 +
                                ((((key_in >> 2) & 1) * 16) ^ (col & 16)) + (col & 8);
            sts64(at, tw[term][0], tw[term][1]);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[buf]));
        if (++ss == C::kSS) {
          ss = 0;
          sph ^= 1;
        }
      }

      // the next segment's queries come while this one's last product runs
      ok = await(ns + 1);
      // ---------------------------------------------------------- epilogue
      if (nt > 0) {
        const int x = tc - 1;
        if (!mbar_wait_w_ab(smem_u32(&sm.pv_done[x & 1]), (x >> 1) & 1, &sm.abort)) fail();
        tc_fence_after();
      }
      const int slot = sg.slot;
      const int rest = sg.parts & kOver ? 0 : 1;  // (of an item that was not cut)
      sum_keys();
      sync();
      if (tid < rows) {
        Sum all = sm.past[tid];
        all.add(sum_of(tid), -static_cast<float>(e0));
        const float lg = all.m == 0.f ? -INFINITY : log2f(all.m) + all.e - sm.nref[tid];
        // o = O^T 2^(ref - kShift) / sum, the power of two in two halves
        const int k = static_cast<int>(-all.e);
        sm.fac[tid] = all.m == 0.f ? 0.f : pow2_within(k / 2) / all.m;  // (0: nothing seen)
        sm.ve[tid] = pow2_within(k - k / 2);
        const int orow = sm.orow[tid];
        if (slot >= 0)
          g.stats[static_cast<size_t>(slot) * R + tid] = lg;
        else if (KEYS != kAll)
          g.row_stats[rest][orow] = lg;
        else if (g.lse != nullptr)
          g.lse[static_cast<size_t>(orow % g.H) * g.T + orow / g.H] = lg * kLn2;
        if (KEYS != kAll && sg.parts != 0)
          g.where[rest][orow] =
              RowParts{static_cast<int>(blockIdx.x) | (tid << 16), sg.parts & ~kOver};
      }
      sync();
      const bool active = DIM == 128 || key_in < DIM;
#pragma unroll
      for (int c = 0; c < R; c += kNext) {
        if (!has_rows(c)) break;
        uint32_t h[8], m[8], lo[8];
        if (nt > 0) {
          const uint32_t at = tmem + lanes + C::kColO + r0 + c;
          tmem_ld8(at, h);
          tmem_ld8(at + R, m);
          tmem_ld8(at + 2 * R, lo);
          tmem_ld_wait();
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = r0 + c + i;
          if (r < rows && active) {
            const float f = sm.fac[r];
            float v = 0.f;
            if (nt > 0 && f != 0.f)
              v = fmaf(fmaf(__uint_as_float(lo[i]), 0x1p-5f, __uint_as_float(m[i])), 0x1p-5f,
                       __uint_as_float(h[i])) * f * sm.ve[r];
            if (slot >= 0)
              g.partial[(static_cast<size_t>(slot) * R + r) * DIM + key_in] = v;
            else if (KEYS != kAll)
              g.rows[rest][static_cast<size_t>(sm.orow[r]) * DIM + key_in] = v;
            else
              g.o[static_cast<size_t>(sm.orow[r]) * DIM + key_in] = __float2bfloat16(v);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (nt > 0) mbar_arrive(smem_u32(&sm.o_empty));
        mbar_arrive(smem_u32(&sm.seg_empty[ns % kSegSlots]));
      }
    }
    if (!ok) sm.abort = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && sm.abort) report(g.status, FLAMIA_DEV_TIMEOUT);
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

// ------------------------------------------------------------------ host

struct Workspace {
  size_t joins, stats, partial, total;
};
Workspace layout(int R, int d) {
  Workspace w;
  const size_t slots = R == kManyRows ? 2 * kRowsCtas : kSlots;
  w.joins = 0;
  w.stats = align_up(sizeof(int4) * 2 * kMaxCtas, 256);
  w.partial = w.stats + align_up(sizeof(float) * slots * R, 256);
  w.total = w.partial + sizeof(float) * slots * R * d;
  return w;
}

// The pages' rows seen as (byte of a row, row of a page, page x head).
bool make_page_map(CUtensorMap* map, const uint8_t* codes, const flamia_kvcache* c) {
  EncodeTiledFn enc = get_encode_tiled();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(c->d), static_cast<cuuint64_t>(c->page_size),
                        static_cast<cuuint64_t>(c->num_pages) * c->H_kv};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(c->d),
                           static_cast<cuuint64_t>(c->d) * c->page_size};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(c->d),
                       static_cast<cuuint32_t>(c->page_size < 128 ? c->page_size : 128), 1u};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(codes), dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle_for_row_bytes(c->d),
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DIM, int R, int KEYS>
flamia_status launch(const flamia_kvcache* c, const AttendArgs& g, cudaStream_t s) {
  CUtensorMap mk, mv;
  if (!make_page_map(&mk, c->k_codes, c) || !make_page_map(&mv, c->v_codes, c))
    return FLAMIA_ERR_CUDA;
  constexpr int smem = static_cast<int>(sizeof(Smem<DIM, R>)) + 1024;
  static_assert(Cfg<DIM, R>::kCtas * (smem + 1024) <= 228 * 1024, "shared memory");
  const int grid = min(kMaxCtas, num_sms() * Cfg<DIM, R>::kCtas);
  static std::atomic<unsigned long long> raised{0};
  return launch_large(attend_kernel<DIM, R, KEYS>, raised, dim3(grid), Cfg<DIM, R>::kThreads, smem, s, mk,
                      mv, g) &&
                 (KEYS != kAll || g.whole || launch_join<DIM, R>(grid, s, g))
             ? FLAMIA_OK
             : FLAMIA_ERR_CUDA;
}

template <int KEYS>
flamia_status launch_few(const flamia_kvcache* c, const AttendArgs& g, int R, cudaStream_t s) {
  if (c->d == 128)
    return R == 8 ? launch<128, 8, KEYS>(c, g, s)
                  : R == 16 ? launch<128, 16, KEYS>(c, g, s) : launch<128, 32, KEYS>(c, g, s);
  return R == 8 ? launch<64, 8, KEYS>(c, g, s)
                : R == 16 ? launch<64, 16, KEYS>(c, g, s) : launch<64, 32, KEYS>(c, g, s);
}

}  // namespace

flamia_status attend_few(const flamia_kvcache* c, const AttendArgs& g, int R, Keys keys,
                         cudaStream_t s) {
  return keys == kAll ? launch_few<kAll>(c, g, R, s)
                      : keys == kBoth ? launch_few<kBoth>(c, g, R, s)
                                      : launch_few<kRest>(c, g, R, s);
}

// Query rows side by side in one item: those of a K / V head's mean number of
// new tokens, up to 32, or 256 (attn_cache_rows.cu).  More rows than there are cost
// softmax time and resident CTAs (4 rows a head: 101, 109, 161 us with 8, 16, 32; one
// row: 98, 127, 196), fewer read K and V again for each item (16 rows a head: 74,
// 56, 80 us).  32 against 256 (heads of 128): 8 sequences over 2,048, 64 rows 55 and
// 58 us, 96 rows 72 and 60, 128 rows 90 and 63; one sequence over 4,096, 64 rows 28
// and 35, 128 rows 33 and 36; 64 sequences over 100, 400 rows 73 and 40; 505 rows over
// 7,300 206 and 105.  The mean is of the whole call: prompts beside single tokens
// give both the same rows (2,048 tokens over none and 63 single ones over 8,192, 32 /
// 8 heads of 128: 613 us, apart 120 and 169).
int rows_per_item(long long rows) {
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 96 ? 32 : kManyRows;
}

}  // namespace flamia

using namespace flamia;

extern "C" size_t flamia_attn_cache_workspace_bytes(int T, int ndocs, int H, int H_kv, int d) {
  if (!supported_dim(d) || !valid_batch(T, ndocs) || H <= 0 || H > 4096 || H_kv <= 0 ||
      H % H_kv != 0)
    return 0;
  return layout(rows_per_item(mean_rows(T, ndocs, H / H_kv)), d).total;
}

namespace flamia {

flamia_status attend_args(AttendArgs& g, const flamia_kvcache* cache, const void* q_bf16,
                          int64_t q_stride, int T, int H, const int32_t* cu_seqlens, int ndocs,
                          const int32_t* starts, const int32_t* page_table, int table_stride,
                          float softmax_scale, int window, int sinks, void* o_bf16, float* lse,
                          const void* ws, int* dev_status) {
  const flamia_status st = check_cache(cache);
  if (st != FLAMIA_OK) return st;
  if (!valid_batch(T, ndocs) || table_stride <= 0 || H <= 0 || H > 4096 || H % cache->H_kv != 0 ||
      !(softmax_scale > 0.f) || std::isinf(softmax_scale) || window < 0 || sinks < 0 ||
      (sinks > 0 && window == 0) || static_cast<long long>(T) * H >= (1ll << 31) - 64)
    return FLAMIA_ERR_INVALID_ARG;
  if (T == 0) return FLAMIA_OK;
  if (!valid_rows(q_bf16, q_stride) || o_bf16 == nullptr || !aligned(o_bf16, 16) ||
      cu_seqlens == nullptr || page_table == nullptr || ws == nullptr || !aligned(ws, 256) ||
      !aligned(lse, 4))
    return FLAMIA_ERR_INVALID_ARG;
  g.k_scales = cache->k_scales;
  g.v_scales = cache->v_scales;
  g.q = static_cast<const __nv_bfloat16*>(q_bf16);
  g.o = static_cast<__nv_bfloat16*>(o_bf16);
  g.lse = lse;
  g.cu = cu_seqlens;
  g.starts = starts;
  g.table = page_table;
  g.status = dev_status;
  g.q_stride = q_stride;
  g.T = T;
  g.H = H;
  g.H_kv = cache->H_kv;
  g.G = H / cache->H_kv;
  g.ndocs = ndocs;
  g.table_stride = table_stride;
  g.num_pages = cache->num_pages;
  g.page_size = cache->page_size;
  // positions stay below 2^30: larger windows and first tokens see the same
  g.window = window < kMaxPos ? window : kMaxPos;
  g.sinks = sinks < kMaxPos ? sinks : kMaxPos;
  const long long cap = static_cast<long long>(table_stride) * cache->page_size;
  g.cap = static_cast<int>(cap < kMaxPos ? cap : kMaxPos);
  g.whole = cap <= 128 * kWholeTiles;
  g.scale_log2 = softmax_scale * 1.44269504088896340736f;
  return FLAMIA_OK;
}

}  // namespace flamia

extern "C" flamia_status flamia_attn_cache(const flamia_kvcache* cache, const void* q_bf16,
                                           int64_t q_stride, int T, int H,
                                           const int32_t* cu_seqlens, int ndocs,
                                           const int32_t* starts, const int32_t* page_table,
                                           int table_stride, float softmax_scale, int window,
                                           int sinks, void* o_bf16, float* lse, void* ws,
                                           size_t ws_bytes, int* dev_status, void* stream) {
  AttendArgs g{};
  const flamia_status st =
      attend_args(g, cache, q_bf16, q_stride, T, H, cu_seqlens, ndocs, starts, page_table,
                  table_stride, softmax_scale, window, sinks, o_bf16, lse, ws, dev_status);
  if (st != FLAMIA_OK || T == 0) return st;
  const int R = rows_per_item(mean_rows(T, ndocs, g.G));
  const Workspace w = layout(R, cache->d);
  if (ws_bytes < w.total) return FLAMIA_ERR_WORKSPACE;
  g.joins = reinterpret_cast<int4*>(static_cast<uint8_t*>(ws) + w.joins);
  g.stats = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + w.stats);
  g.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + w.partial);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return R == kManyRows ? attend_rows(cache, g, s) : attend_few(cache, g, R, kAll, s);
}
