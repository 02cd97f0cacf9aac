// Attention over the paged MXFP8 cache for many query rows (a prompt, or the
// next chunk of one): 256 rows of a K / V head, two tiles of 128, are the
// tensor core's M, and every key tile that is read serves them all.
//
// Per 128-key tile and row tile S = Q K^T (M = 128 rows, N = 128 keys) and
// O += P V (P from tensor memory), both with FP16 operands: cached codes are
// FP16 numbers exactly, queries times 2^-e are down to 2^-24 of the row's
// largest element, and weights round to 2^-11 of themselves (or to 2^-24 of the
// largest).  One product each instead of a product for each of several 8-bit
// terms; the codes are converted once for 256 rows.  The exponents of K and V
// enter the scores of a key, as in attn_cache.cu:
//   w = 2^(x + eV - ref),  l = sum w 2^(E0 - eV),
//   o = O 2^E0 / l,        log2 sum 2^x = ref - E0 + log2 l,
// and a Sum for what l cannot hold, as there; but a thread owns a row here, so maxima
// and sums need no other thread.  A row's reference is an integer that moves when a tile
// exceeds it by more than kSlack;
// where 32 keys have one K and one V exponent (always, with exponents of 32-token
// blocks) their largest score comes with a load from tensor memory.
//
// Warps 0-3 and 4-7: softmax of the two row tiles (thread = row = TMEM lane);
// 8-11: converters, a 32-key block each (codes from global memory through
// registers into swizzled shared memory, K's and V's in turn, one loaded while the
// other is converted); 12: MMA issuer; 13: walks the CTA's run.  While one row
// tile's softmax runs the tensor core works for the other.  Runs of key tiles, parts
// and joins are those of attend.cuh.
//
// Measured: 505 tokens over 7,866 (16 heads of 128, two sequences) 112 us, 560
// TFLOP/s; 512 over 8,000 (32 / 8 heads, four sequences) 332 us (32 rows an item: 824).
// With an exponent a token every tile takes the slow body: 505 over 7,361 246 us
// against 112.  Clock stamps, when the first of these took 118 us: a key tile takes
// some 5,000 cycles where the tensor core is busy for 2,300, as the softmax of a row
// tile (2,800) and its two products follow one another and the other row tile fills
// the gaps only in part; a CTA's first scores come 16,000 cycles after its start (plan,
// queries), its output takes 5,000.  Scores of 64 keys in two buffers, so that the
// softmax does not wait for them, took longer (146 us against 122 then: twice the
// products to issue); K and V loaded and converted side by side, 139 registers
// and more code, too (181: spills, and misses in the instruction cache).
#include <cmath>

#include "attend.cuh"

namespace flamia {
namespace {

constexpr float kSlack = 8.f;
// Columns 32 c .. 32 c + 31 of a tile: flags.
constexpr int kUniform = 1;   // one K and one V exponent
constexpr int kEvery = 2;     // every row sees every key
constexpr int kHere = 4;      // there is a page
constexpr int kLowShift = 8;  // from here on: the byte of the smallest eV that a row sees

// A row of 32 keys' exponents.
struct alignas(16) Keys32 {
  float kf;     // 2^eK  (kUniform)
  int ev;       // eV    (kUniform)
  int top;      // the largest eV that a row sees; -127: none
  int flags;
};

template <int DIM>
struct Cfg {
  static constexpr int kRows = 256;
  static constexpr int kThreads = 512;  // (14 and 15 idle: registers move by four warps)
  static constexpr int kBlock = 128 * 128;            // 64 columns of 128 rows, bytes
  static constexpr int kTileBytes = DIM / 64 * kBlock;
  static constexpr uint32_t kColO = 256;
};

// A segment with what the converters need: its keys' end hi, the first key wlo of
// its window, positions pf and pl of its first and last row, its sequence.
struct RowSegment : Segment {
  int hi, wlo, pf, pl, seq;
};

template <int DIM>
struct Smem {
  using C = Cfg<DIM>;
  alignas(1024) uint8_t q[2][C::kTileBytes];
  alignas(1024) uint8_t k[2][C::kTileBytes];
  alignas(1024) uint8_t v[2][C::kTileBytes];
  alignas(16) float kf[4][128];   // 2^eK, eV of each key: a ring of four tiles, as
  alignas(16) int ev[4][128];     // the softmax is done two score products later
  Keys32 col[4][4];
  uint32_t nan[4][4];             // half-seen keys whose value holds a NaN
  Sum past[C::kRows];             // sum 2^(x + nref) of what is not in a row's l
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], sc_full[4];
  uint64_t s_full[2], p_full[2], pv_done[2];  // by row tile
  uint64_t q_full[2], drained;
  uint64_t seg_full[kSegSlots], seg_empty[kSegSlots];
  RowSegment seg[kSegSlots];
  int plan_b;
  SeqWork plan_seq;
  long long plan_off, plan_u0, plan_u1, plan_total;
  long long scan[C::kThreads / 32];
  uint32_t tmem_base;
  volatile int abort;
};

// ------------------------------------------------------------------ PTX

// Barrier of a softmax warpgroup that also ORs a predicate over it.
__device__ __forceinline__ bool group_vote(int id, bool p) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<int>(p)), "r"(id)
      : "memory");
  return r != 0;
}

// D (+)= A * B, FP16 x FP16 -> F32: A and B in shared memory, or A in tensor
// memory (two elements a 32-bit column).  idesc_f8's fields serve: the operand
// formats are 0 for FP16, too.  Descriptors come as their low words (the address)
// and one high word.  Issued by one elected thread of a converged warp: under a
// branch for one lane the eight products of a tile took 850 cycles to issue
// (505 tokens over 7,866: 137 us against 122).
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t hi,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 da, {%1, %3};\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b,
                                           uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// A warpgroup's registers a thread from here on.  The kernel starts with 128 each;
// 2 x 168 + 112 + 64 is what four warpgroups then had.
template <bool MORE, int N>
__device__ __forceinline__ void set_registers() {
  if (MORE)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void sts128(uint32_t addr, const uint4& w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w.x), "r"(w.y),
               "r"(w.z), "r"(w.w)
               : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 w;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
               : "r"(addr)
               : "memory");
  return w;
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t w;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(addr) : "memory");
  return w;
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t w) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(w) : "memory");
}

// 16 bytes from global to shared memory, of which the first n are read (0 or 16;
// the others become zeros), and the wait for all of the thread's.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Two E4M3 codes as FP16 (exact; NaN stays).
__device__ __forceinline__ uint32_t half2_of_codes(uint32_t codes) {
  uint32_t h;
  asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}"
      : "=r"(h)
      : "r"(codes));
  return h;
}

// Byte offset of 16-byte chunk j of a row in an FP16 operand tile: blocks of 64
// columns, rows of 128 bytes, chunks swizzled as the 128-byte mode does.
template <int DIM>
__device__ __forceinline__ uint32_t tile_at(int row, int j) {
  return (j >> 3) * Cfg<DIM>::kBlock + row * 128 + (((j & 7) ^ (row & 7)) << 4);
}

// ------------------------------------------------------------------ work

// The segments of a CTA's run, in order.
template <int R>
struct Walk {
  SeqWork w;
  long long u0, u, u1, total;
  int b, hk = 0, rt = 0, o = 0;
  bool first = true;
  int4 join0 = make_int4(0, 0, 0, 0), join1 = make_int4(0, 0, 0, 0);

  template <class Sm>
  __device__ __forceinline__ explicit Walk(const Sm& sm)
      : w{}, u0(sm.plan_u0), u(sm.plan_u0), u1(sm.plan_u1), total(sm.plan_total), b(sm.plan_b) {
    if (u < u1) {
      w = sm.plan_seq;
      const long long item = mul_div(sm.plan_off, 1, w.units);
      o = static_cast<int>(sm.plan_off - item * w.units);
      hk = static_cast<int>(mul_div(item, 1, w.row_tiles));
      rt = static_cast<int>(item - static_cast<long long>(hk) * w.row_tiles);
    }
  }

  // The next segment (s < 0: none).
  __device__ __forceinline__ RowSegment next(const AttendArgs& g, bool reports) {
    RowSegment sg{};
    while (u < u1) {
      const int take = static_cast<int>(min(u1 - u, static_cast<long long>(w.units - o)));
      const int cost = g.whole ? 0 : kItemCost<R>;
      const int i0 = max(o - cost, 0);
      const int i1 = g.whole ? w.tiles : max(o + take - cost, 0);
      sg.seq = b;
      sg.s = w.s;
      sg.n = w.n;
      sg.start = w.start;
      sg.hk = hk;
      sg.row0 = rt * R;
      sg.pf = w.start + sg.row0 / g.G;
      sg.pl = w.start + static_cast<int>(min(static_cast<long long>(w.n) * g.G - 1,
                                          static_cast<long long>(sg.row0) + R - 1) /
                                      g.G);
      sg.hi = max(sg.pl + 1, 0);
      sg.wlo = g.window > 0 ? max(sg.pf - g.window + 1, 0) : 0;
      sg.wt = sg.wlo >> 7;
      sg.ns = min((g.sinks + 127) >> 7, sg.wt);
      const int list = sg.ns + max(((sg.hi + 127) >> 7) - sg.wt, 0);
      sg.i0 = min(i0, list);
      sg.i1 = min(i1, list);
      sg.slot = -1;
      if (i0 > 0)
        sg.slot = 2 * blockIdx.x;
      else if (i1 < w.tiles)
        sg.slot = 2 * blockIdx.x + 1;
      if (first && i0 > 0) {
        // the second CTA of an item has it joined: parts are the CTA before this
        // one (slot 1) and slots 0 from here on
        const long long ctas = active_ctas<R>(g, total), c = blockIdx.x, ui = u0 - o;
        if (c > 0 && mul_div(total, c - 1, ctas) <= ui + kItemCost<R>) {
          const long long last = div_up((ui + w.units) * ctas, total) - 1;
          join0 = make_int4(static_cast<int>(last - c + 2), w.s, w.n, hk);
          join1 = make_int4(sg.row0, 0, 0, 0);
        }
      }
      if (reports && hk == 0 && rt == 0 && i0 == 0) {
        const int raw = g.starts != nullptr ? g.starts[b] : 0;
        if (raw > g.cap - w.n) report(g.status, FLAMIA_DEV_BAD_PAGE);
      }
      first = false;
      u += take;
      o = 0;
      if (u < u1 && ++rt == w.row_tiles) {
        rt = 0;
        if (++hk == g.H_kv) {
          hk = 0;
          do {
            w = seq_work<R>(g, ++b);  // there is one: u < u1
          } while (w.row_tiles == 0 && b + 1 < g.ndocs);
        }
      }
      if (i1 > i0) return sg;  // (else the run ends before the item's first tile)
    }
    sg.s = -1;
    return sg;
  }
};

// A converter warp's 32 keys of a tile, on their way from the cache.
template <int DIM>
struct Block32 {
  static constexpr int kLanes = DIM / 16;       // lanes a row: 16 codes each
  static constexpr int kPer = 32 / kLanes;      // rows side by side
  static constexpr int kIters = 32 / kPer;
  unsigned seen;   // its keys that some row of the item sees
  uint4 w[kIters]; // K's codes, or V's

  // Codes of the keys that some row of the item sees, zeros for the others (their
  // weights are 0, and 0 x NaN would not be).
  __device__ __forceinline__ void load(const uint8_t* src, int lane) {
    src += lane * 16;
#pragma unroll
    for (int it = 0; it < kIters; ++it) {
      w[it] = make_uint4(0, 0, 0, 0);
      if ((seen >> (it * kPer + lane / kLanes)) & 1)
        w[it] = *reinterpret_cast<const uint4*>(src + it * kPer * DIM);
    }
  }
  // As FP16 into rows row0 .. of an operand tile.
  __device__ __forceinline__ void store(uint32_t tile, int row0, int lane) const {
    const int c = lane % kLanes;
#pragma unroll
    for (int it = 0; it < kIters; ++it) {
      const int r = row0 + it * kPer + lane / kLanes;
      const uint32_t x[4] = {w[it].x, w[it].y, w[it].z, w[it].w};
      uint32_t h[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[2 * j] = half2_of_codes(x[j] & 0xFFFFu);
        h[2 * j + 1] = half2_of_codes(x[j] >> 16);
      }
      // (the lanes of a row's second half store the other chunk first: no bank
      // conflicts)
      const uint4 a = make_uint4(h[0], h[1], h[2], h[3]), b = make_uint4(h[4], h[5], h[6], h[7]);
      const bool turn = c >= 4;
      sts128(tile + tile_at<DIM>(r, 2 * c + turn), turn ? b : a);
      sts128(tile + tile_at<DIM>(r, 2 * c + !turn), turn ? a : b);
    }
  }
};

// Adds 2^(x + nref) of a tile's keys whose eV lies below floor_ev to a row's sum.  (Not inlined:
// rare, and inside the tile's code it made a prompt chunk 139 us against 119.)
__device__ __noinline__ void sum_apart(Sum& past, const float* kf, const int* ev,
                                       const Keys32* col, const uint32_t* nan, uint32_t t_s,
                                       float qf, float nref, int floor_ev, int k0, int pos,
                                       int window, int sinks) {
  float top = kNoExponent, sum = 0.f;
#pragma unroll 1
  for (int i = 0; i < 32; ++i) {  // the largest, then the sum
    const int at = (i & 15) * 8, flags = col[at / 32].flags;
    uint32_t s[8];
    tmem_ld8(t_s + at, s);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int key = k0 + at + j;
      const bool seen =
          (flags & kEvery) ||
          ((flags & kHere) && key <= pos && (window == 0 || key < sinks || key > pos - window));
      float x = fmaf(__uint_as_float(s[j]), kf[at + j] * qf, nref);
      if (!(flags & kEvery) && (nan[at / 32] >> ((at + j) & 31)) & 1)
        x = __uint_as_float(0x7FC00000u);
      if (!seen || ev[at + j] >= floor_ev) x = -INFINITY;
      if (i < 16)
        top = fmaxf(top, x);
      else
        sum += ex2_approx(x - top);
    }
    if (i == 15) top = ceilf(top);
  }
  past.add(sum, top);
}

template <int DIM>
__global__ void __launch_bounds__(Cfg<DIM>::kThreads, 1) attend_rows_kernel(const AttendArgs g,
                                                                           const uint8_t* k_codes,
                                                                           const uint8_t* v_codes) {
  using C = Cfg<DIM>;
  constexpr int R = C::kRows;
  extern __shared__ uint8_t smem_raw[];
  Smem<DIM>& sm = *reinterpret_cast<Smem<DIM>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.k_full[i]), 4);
      mbar_init(smem_u32(&sm.v_full[i]), 4);
      mbar_init(smem_u32(&sm.k_empty[i]), 1);
      mbar_init(smem_u32(&sm.v_empty[i]), 1);
      mbar_init(smem_u32(&sm.q_full[i]), 4);
      mbar_init(smem_u32(&sm.s_full[i]), 1);
      mbar_init(smem_u32(&sm.p_full[i]), 4);
      mbar_init(smem_u32(&sm.pv_done[i]), 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&sm.sc_full[i]), 4);
    mbar_init(smem_u32(&sm.drained), 1);
    for (int i = 0; i < kSegSlots; ++i) {
      mbar_init(smem_u32(&sm.seg_full[i]), 1);
      mbar_init(smem_u32(&sm.seg_empty[i]), 13);  // softmax, converters, MMA issuer
    }
    sm.abort = 0;
    fence_barrier_init();
  }
  // All of the SM's tensor memory is taken here, which may wait for CTAs of the
  // kernel before.  So it comes after that kernel's end, and the next kernel is
  // let in when every CTA of this one has its share: neither can hold what the
  // other waits for.
  wait_for_previous();
  if (warp == 12) {
    tmem_alloc(smem_u32(&sm.tmem_base), 512);
    tmem_relinquish();
  }
  check_offsets(g.cu, g.ndocs, g.T, static_cast<long long>(blockIdx.x) * C::kThreads + tid,
                static_cast<long long>(gridDim.x) * C::kThreads, g.status);
  tc_fence_before();
  make_plan<R, C::kThreads>(g, sm);
  tc_fence_after();
  start_next();
  const uint32_t tmem = sm.tmem_base;

  if (warp >= 8 && warp < 12) {
    // ---------------------------------------------------------- converters
    set_registers<false, 112>();
    const int cw = warp - 8;
    int tc = 0;
    bool ok = true;
    for (int ns = 0; ok; ++ns) {
      const int sl = ns % kSegSlots;
      ok = mbar_wait_w_ab(smem_u32(&sm.seg_full[sl]), (ns / kSegSlots) & 1, &sm.abort);
      if (!ok) break;
      const RowSegment sg = sm.seg[sl];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.seg_empty[sl]));
      if (sg.s < 0) break;
      const int hi = sg.hi, wlo = sg.wlo, pf = sg.pf, pl = sg.pl;
      const int32_t* table = g.table + static_cast<long long>(sg.seq) * g.table_stride;
      auto any = [&](int key) {
        return key <= pl && (g.window == 0 || key < g.sinks || key > pf - g.window);
      };
      auto every = [&](int key) {
        return key <= pf && (g.window == 0 || key < g.sinks || key > pl - g.window);
      };
      // K's codes, then V's, of one tile after another; what is next is loaded before
      // what is there is converted (one body for both: the code has to fit the
      // instruction cache together with the softmax's).
      Block32<DIM> next, cur;
      int row = 0, kbyte = 0, vbyte = 0, kbyte1 = 0, vbyte1 = 0;
      bool good = false;
      // First rows of the block at the next 32 list positions (a lane each), in units of
      // 32 rows of the codes; -1: no page.
      int rows32 = -1;
      auto look_up = [&](int i) {
        const int key0 = tile_of(sg, i) * 128 + cw * 32, slot = key0 / g.page_size;
        const bool need = i < sg.i1 && key0 < hi &&
                          (g.window == 0 || key0 + 32 > wlo || key0 < g.sinks);
        const int page = need && slot < g.table_stride ? table[slot] : -1;
        const bool there = page >= 0 && page < g.num_pages;
        if (need && !there) report(g.status, FLAMIA_DEV_BAD_PAGE);
        // (a cache that fits the memory has fewer than 2^31 of them)
        rows32 = there ? (page * g.H_kv + sg.hk) * (g.page_size / 32) +
                             (key0 - slot * g.page_size) / 32
                       : -1;
      };
      auto load_k = [&](int i) {
        if (((i - sg.i0) & 31) == 0) look_up(i + lane);
        row = __shfl_sync(0xffffffffu, rows32, (i - sg.i0) & 31);
        next.seen = __ballot_sync(0xffffffffu,
                                  row >= 0 && any(tile_of(sg, i) * 128 + cw * 32 + lane));
        const long long at = static_cast<long long>(max(row, 0)) * 32 + lane;
        kbyte1 = g.k_scales[at];
        vbyte1 = g.v_scales[at];
      };
      auto load_codes = [&](const uint8_t* codes) {
        next.load(codes + static_cast<long long>(max(row, 0)) * 32 * DIM, lane);
      };
      if (sg.i0 < sg.i1) {
        load_k(sg.i0);
        load_codes(k_codes);
      }
#pragma unroll 1
      for (int j = 2 * sg.i0; j < 2 * sg.i1; ++j) {
        const int i = j >> 1, st = tc & 1, ss = tc & 3;
        const bool is_v = j & 1;
        cur = next;
        if (!is_v) {
          good = row >= 0;
          kbyte = kbyte1;
          vbyte = vbyte1;
        } else if (i + 1 < sg.i1) {
          load_k(i + 1);
        }
        if (j + 1 < 2 * sg.i1) load_codes(is_v ? k_codes : v_codes);
        if (tc >= 2)  // (the use before)
          ok = mbar_wait_w_ab(smem_u32(is_v ? &sm.v_empty[st] : &sm.k_empty[st]),
                              ((tc >> 1) & 1) ^ 1, &sm.abort);
        if (!ok) break;
        const int key = tile_of(sg, i) * 128 + cw * 32 + lane;
        const bool half = !__all_sync(0xffffffffu, good && every(key));
        if (!is_v) {  // exponents; keys that no row sees take those of one that is seen
          const unsigned live = cur.seen;
          const bool seen = (live >> lane) & 1;
          const int one = live ? __ffs(live) - 1 : 0;
          const int kb0 = live ? __shfl_sync(0xffffffffu, kbyte, one) : 0;
          const int vb0 = live ? __shfl_sync(0xffffffffu, vbyte, one) : 0;
          const int kx = seen ? kbyte : kb0, vx = seen ? vbyte : vb0;
          const bool uniform = __all_sync(0xffffffffu, kx == kb0 && vx == vb0);
          const int top = __reduce_max_sync(0xffffffffu, vx);
          const int low = live ? __reduce_min_sync(0xffffffffu, vx) : 255;
          sm.kf[ss][cw * 32 + lane] = pow2_byte(kx);
          sm.ev[ss][cw * 32 + lane] = vx - 127;
          if (lane == 0)
            sm.col[ss][cw] = Keys32{pow2_byte(kb0), vb0 - 127, live ? top - 127 : -127,
                                    (uniform ? kUniform : 0) | (half ? 0 : kEvery) |
                                        (good ? kHere : 0) | (low << kLowShift)};
        } else if (half) {
          // A value that some rows see and others do not must not reach the others:
          // one that holds a NaN is cleared, and the NaN moves into the weights of
          // the rows that see it.
          uint32_t flags = 0;
#pragma unroll
          for (int it = 0; it < cur.kIters; ++it) {
            const uint32_t x[4] = {cur.w[it].x, cur.w[it].y, cur.w[it].z, cur.w[it].w};
            bool nan = false;
#pragma unroll
            for (int m = 0; m < 4; ++m)
              nan |= (((x[m] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
            const unsigned lanes = __ballot_sync(0xffffffffu, nan);
#pragma unroll
            for (int m = 0; m < cur.kPer; ++m) {
              if ((lanes >> (m * cur.kLanes)) & ((1u << cur.kLanes) - 1)) {
                flags |= 1u << (it * cur.kPer + m);
                if (lane / cur.kLanes == m) cur.w[it] = make_uint4(0, 0, 0, 0);
              }
            }
          }
          if (lane == 0) sm.nan[ss][cw] = flags;
        }
        cur.store(smem_u32(is_v ? sm.v[st] : sm.k[st]), cw * 32, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(is_v ? &sm.v_full[st] : &sm.k_full[st]));
          if (!is_v) mbar_arrive(smem_u32(&sm.sc_full[ss]));
        }
        tc += is_v;
      }
    }
    if (!ok) sm.abort = 1;
  } else if (warp < 8) {
    set_registers<true, 168>();
    // ------------------------------------------------------------- softmax
    const int wg = warp >> 2, r = tid;   // row tile, row of the item
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + wg * 128, t_o = tmem + lanes + C::kColO + wg * DIM;
    const uint32_t sbar = smem_u32(&sm.s_full[wg]), pbar = smem_u32(&sm.p_full[wg]),
                   obar = smem_u32(&sm.pv_done[wg]);
    int tc = 0, x = 0;  // key tiles of the CTA; of this row tile
    bool late = false;  // a wait ran out: all warps go on to the next vote
    auto fail = [&]() {
      late = true;
      sm.abort = 1;
    };
    for (int ns = 0;; ++ns) {
      const int sl = ns % kSegSlots;
      if (!late &&
          !mbar_wait_w_ab(smem_u32(&sm.seg_full[sl]), (ns / kSegSlots) & 1, &sm.abort))
        fail();
      if (group_vote(1 + wg, late)) break;
      const RowSegment& sg = sm.seg[sl];
      if (sg.s < 0) break;
      const int nt = sg.i1 - sg.i0;
      const long long all = static_cast<long long>(sg.n) * g.G - sg.row0;
      const int rows = static_cast<int>(min(static_cast<long long>(R), all));
      const bool active = wg == 0 || rows > 128;
      const int pos = r < rows ? max(sg.start + (sg.row0 + r) / g.G, -1) : -1;
      float qf = 0.f;
      if (nt > 0 && active) {
        // This warp's 32 rows: copied to their place by 16-byte chunks, four lanes a
        // row, then each lane converts its own row there.
        const uint32_t qs = smem_u32(sm.q[wg]);
        const int w0 = (warp & 3) * 32;
#pragma unroll 1
        for (int it = 0; it < 4; ++it) {
          const int rr = w0 + it * 8 + (lane >> 2), row = sg.row0 + wg * 128 + rr;
          const bool there = wg * 128 + rr < rows;
          const int i = there ? row / g.G : 0, h = there ? sg.hk * g.G + row - i * g.G : 0;
          const __nv_bfloat16* src =
              g.q + (sg.s + i) * g.q_stride + static_cast<long long>(h) * DIM;
#pragma unroll
          for (int c = 0; c < DIM / 8; c += 4)
            copy16(qs + tile_at<DIM>(rr, c + (lane & 3)), src + (c + (lane & 3)) * 8,
                   there ? 16 : 0);
        }
        copies_wait();
        __syncwarp();
        const int rr = w0 + lane;
        // magnitudes as integers; 0x7F80 and above: infinities and NaN, which become
        // NaN and stay out of the maximum
        uint32_t a = 0;
#pragma unroll 4
        for (int c = 0; c < DIM / 8; ++c) {
          const uint4 w = lds128(qs + tile_at<DIM>(rr, c));
          a = __vmaxu2(a, __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                   __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu)));
        }
        a = max(a & 0xFFFFu, a >> 16);
        if (a >= 0x7F80u) {
          a = 0;
#pragma unroll 1
          for (int e = 0; e < DIM / 2; ++e) {
            const uint32_t at = qs + tile_at<DIM>(rr, e >> 2) + (e & 3) * 4;
            uint32_t w = lds32(at);
            if ((w & 0x7F80u) == 0x7F80u)
              w = (w & 0xFFFF0000u) | 0x7FC0u;
            else
              a = max(a, w & 0x7FFFu);
            if ((w & 0x7F800000u) == 0x7F800000u)
              w = (w & 0xFFFFu) | 0x7FC00000u;
            else
              a = max(a, (w >> 16) & 0x7FFFu);
            sts32(at, w);
          }
        }
        const int ex = roundup_exponent(__uint_as_float(a << 16));
        const float2 inv = make_float2(exp2i(-ex), exp2i(-ex));
        qf = g.scale_log2 * (ex < -126 ? 0x1p-127f : exp2i(ex));
#pragma unroll 4
        for (int c = 0; c < DIM / 8; ++c) {
          const uint32_t at = qs + tile_at<DIM>(rr, c);
          const uint4 w = lds128(at);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
          uint32_t h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            h[j] = half2_of(__fmul2_rn(
                make_float2(__uint_as_float(ww[j] << 16), __uint_as_float(ww[j] & 0xFFFF0000u)),
                inv));
          sts128(at, make_uint4(h[0], h[1], h[2], h[3]));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.q_full[wg]));
      }

      float l = 0.f, nref = 0.f;  // nref: -reference
      bool has = false;           // the row has a reference
      bool large = false;         // some row's of the warp is beyond kLarge
      sm.past[r] = Sum{0.f, kNoExponent};
      int e0 = -127;
#pragma unroll 1
      for (int t = 0; t < (active ? nt : 0); ++t, ++x) {
        const int ss = (tc + t) & 3;
        // (the scores first: a row tile that sat out an item is ahead of the ring of
        // exponents, whose phase says nothing until then)
        if (!wait_both(sbar, x & 1, smem_u32(&sm.sc_full[ss]), ((tc + t) >> 2) & 1, &sm.abort))
          fail();
        tc_fence_after();
        const int top = max(max(sm.col[ss][0].top, sm.col[ss][1].top),
                            max(sm.col[ss][2].top, sm.col[ss][3].top));
        if (t == 0) {
          e0 = top;
        } else if (top > e0 + kHigh) {  // (as in attn_cache.cu)
          sm.past[r].add(l, -static_cast<float>(e0));
          l = 0.f;
          e0 = top;
        }
        const int k0 = tile_of(sg, sg.i0 + t) * 128;
        const int floor_ev = e0 - kLow;
        // 32 keys with one K and one V exponent: y = x kq + (eV + nref)
        float kq[4], evf[4];
        int flags = kUniform | kEvery, low = 127;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const Keys32 kc = sm.col[ss][c];
          kq[c] = kc.kf * qf;
          evf[c] = static_cast<float>(kc.ev);
          flags &= kc.flags;
          low = min(low, (kc.flags >> kLowShift) - 127);
        }
        const bool apart = low < floor_ev;  // some keys are not in l
        const bool plain = flags == (kUniform | kEvery) && !apart;
        if (!(flags & kEvery) &&  // half-seen keys: V has been searched for NaN
            !mbar_wait_w_ab(smem_u32(&sm.v_full[(tc + t) & 1]), ((tc + t) >> 1) & 1, &sm.abort))
          fail();
        // Any 32 keys: their y, masked.
        auto scores = [&](int c, float (&y)[32]) {
          uint32_t s[32];
          tmem_ld32(t_s + c * 32, s);
          const int flags = sm.col[ss][c].flags;
          uint32_t m = 0xFFFFFFFFu, nan = 0;
          if (!(flags & kEvery)) {
            const int k = k0 + c * 32;
            auto below = [](int n) {  // bits 0 .. n - 1
              return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
            };
            m = flags & kHere ? below(pos - k + 1) : 0u;
            if (g.window > 0) m &= ~below(pos - g.window - k + 1) | below(g.sinks - k);
            nan = sm.nan[ss][c];
          }
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 kf = *reinterpret_cast<const float4*>(&sm.kf[ss][c * 32 + j]);
            const int4 ev = *reinterpret_cast<const int4*>(&sm.ev[ss][c * 32 + j]);
            const float kk[4] = {kf.x, kf.y, kf.z, kf.w};
            const int ee[4] = {ev.x, ev.y, ev.z, ev.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float v = fmaf(__uint_as_float(s[j + i]), kk[i] * qf,
                             static_cast<float>(ee[i]) + nref);
              if ((nan >> (j + i)) & 1) v = __uint_as_float(0x7FC00000u);
              y[j + i] = (m >> (j + i)) & 1 ? v : -INFINITY;
            }
          }
        };
        // Does the reference hold?  (The largest score comes with the load.)
        float mx = -INFINITY;
        uint32_t s0[32], s1[32];
        if (plain) {
          float m0, m1;
          tmem_ld32_max(t_s + 64, s0, m0);
          tmem_ld32_max(t_s + 96, s1, m1);
          tmem_ld_wait();
          mx = fmaxf(fmaf(m0, kq[2], evf[2] + nref), fmaf(m1, kq[3], evf[3] + nref));
          tmem_ld32_max(t_s, s0, m0);
          tmem_ld32_max(t_s + 32, s1, m1);
          tmem_ld_wait();
          mx = fmax3(mx, fmaf(m0, kq[0], evf[0] + nref), fmaf(m1, kq[1], evf[1] + nref));
        } else {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float y[32];
            scores(c, y);
#pragma unroll
            for (int j = 0; j < 32; j += 2) mx = fmax3(mx, y[j], y[j + 1]);
          }
        }
        // Where it does not, or there is none yet, it moves.
        const bool need = has ? mx > kSlack + room(nref) : mx > -INFINITY;
        if (__any_sync(0xffffffffu, need)) {
          float f = 1.f;
          if (need) {
            const float by = lowered(nref - ceilf(mx)) - nref;
            if (has) {
              f = ex2_approx(by);
              l *= f;
            }
            nref += by;
            sm.past[r].e += by;
            has = true;
          }
          large = __any_sync(0xffffffffu, fabsf(nref) > kLarge);
          if (t > 0) {  // O, once the product before has added to it
            if (!mbar_wait_w_ab(obar, (x - 1) & 1, &sm.abort)) fail();
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < DIM; c += 8) {
              uint32_t a[8];
              tmem_ld8(t_o + c, a);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 8; ++i) a[i] = __float_as_uint(__uint_as_float(a[i]) * f);
              tmem_st8(t_o + c, a);
            }
            tmem_st_wait();
          }
        }
        // Weights.  Those of 32 keys take half of the scores' columns, and none whose
        // scores are still to be read.
        if (plain && !large) {
          auto weights = [&](int c, const uint32_t (&s)[32]) {
            const Keys32 kc = sm.col[ss][c];
            const float kq = kc.kf * qf, add = static_cast<float>(kc.ev) + nref;
            const float2 kq2 = make_float2(kq, kq), add2 = make_float2(add, add);
            float2 y[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              y[j] = __ffma2_rn(
                  make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), kq2, add2);
              y[j] = make_float2(ex2_approx(y[j].x), ex2_approx(y[j].y));
            }
            float2 a = y[0], b = y[1];
#pragma unroll
            for (int j = 2; j < 16; j += 2) {
              a = __fadd2_rn(a, y[j]);
              b = __fadd2_rn(b, y[j + 1]);
            }
            a = __fadd2_rn(a, b);
            l = fmaf(a.x + a.y, exp2i(e0 - kc.ev), l);
            uint32_t p[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) p[j] = half2_of(y[j]);
            tmem_st16(t_s + c * 16, p);
          };
#pragma unroll 1
          for (int c = 0; c < 4; c += 2) {
            weights(c, s0);
            if (c == 0) tmem_ld32(t_s + 64, s0);
            weights(c + 1, s1);
            if (c == 0) tmem_ld32(t_s + 96, s1);
            tmem_ld_wait();
          }
        } else {
          if (apart)
            sum_apart(sm.past[r], sm.kf[ss], sm.ev[ss], sm.col[ss], sm.nan[ss], t_s, qf, nref,
                      floor_ev, k0, pos, g.window, g.sinks);
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float y[32];
            scores(c, y);
            uint32_t p[16];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const int ev = sm.ev[ss][c * 32 + j];
              y[j] = ex2_approx(cut(y[j], kSlack));
              l = fmaf(y[j], ev < floor_ev ? 0.f : exp2i(e0 - ev), l);
              if (j & 1) p[j / 2] = half2_of(make_float2(y[j - 1], y[j]));
            }
            tmem_st16(t_s + c * 16, p);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pbar);
      }
      // ------------------------------------------------------------ epilogue
      if (active) {
        const int slot = sg.slot;
        const int tok = (sg.row0 + r) / g.G, hq = sg.hk * g.G + (sg.row0 + r) - tok * g.G;
        const bool live = r < static_cast<long long>(sg.n) * g.G - sg.row0;
        if (nt > 0) {
          if (!mbar_wait_w_ab(obar, (x - 1) & 1, &sm.abort)) fail();
          tc_fence_after();
        }
        Sum past = sm.past[r];
        past.add(l, -static_cast<float>(e0));
        const float lg = past.m == 0.f ? -INFINITY : log2f(past.m) + past.e - nref;
        const int k = static_cast<int>(-past.e);  // (as in attn_cache.cu)
        const float inv = past.m == 0.f ? 0.f : pow2_within(k / 2) / past.m;
        const float ve = pow2_within(k - k / 2);
        const size_t out = static_cast<size_t>(sg.s + tok) * g.H + hq;
        if (live) {
          if (slot >= 0)
            g.stats[static_cast<size_t>(slot) * R + r] = lg;
          else if (g.lse != nullptr)
            g.lse[static_cast<size_t>(hq) * g.T + sg.s + tok] = lg * kLn2;
        }
#pragma unroll
        for (int c = 0; c < DIM; c += 32) {
          uint32_t a[32] = {};
          if (nt > 0) {
            tmem_ld32(t_o + c, a);
            tmem_ld_wait();
          }
#pragma unroll
          for (int j = 0; j < 32; ++j)
            a[j] = inv == 0.f ? 0u : __float_as_uint(__uint_as_float(a[j]) * inv * ve);
          if (live) {
            if (slot >= 0) {
              uint4* p = reinterpret_cast<uint4*>(g.partial) +
                         (static_cast<size_t>(slot) * (DIM / 4) + c / 4) * R + r;
#pragma unroll
              for (int j = 0; j < 8; ++j)
                p[j * R] = make_uint4(a[4 * j], a[4 * j + 1], a[4 * j + 2], a[4 * j + 3]);
            } else {
              uint4* p = reinterpret_cast<uint4*>(g.o + out * DIM + c);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const __nv_bfloat162 b = __floats2bfloat162_rn(
                      __uint_as_float(a[8 * j + 2 * i]), __uint_as_float(a[8 * j + 2 * i + 1]));
                  h[i] = *reinterpret_cast<const uint32_t*>(&b);
                }
                p[j] = make_uint4(h[0], h[1], h[2], h[3]);
              }
            }
          }
        }
        tc_fence_before();
      }
      tc += max(nt, 0);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.seg_empty[sl]));
    }
  } else {
    set_registers<false, 64>();  // (all four warps at once)
    if (warp == 13) {
      // ------------------------------------------------------------ walker
      Walk<R> walk(sm);
      bool ok = true;
      for (int ns = 0; ok; ++ns) {
        const RowSegment sg = walk.next(g, lane == 0);
        const int sl = ns % kSegSlots;
        if (ns >= kSegSlots)
          ok = mbar_wait_w_ab(smem_u32(&sm.seg_empty[sl]), ((ns / kSegSlots) - 1) & 1, &sm.abort);
        if (!ok) break;
        if (lane == 0) {
          sm.seg[sl] = sg;
          mbar_arrive(smem_u32(&sm.seg_full[sl]));
        }
        __syncwarp();
        if (sg.s < 0) break;
      }
      // what the second kernel has to join for this CTA's first item
      if (lane == 0 && !g.whole) {
        g.joins[2 * blockIdx.x] = walk.join0;
        g.joins[2 * blockIdx.x + 1] = walk.join1;
      }
      if (!ok) sm.abort = 1;
    } else if (warp == 12) {
      // ---------------------------------------------------------- MMA issuer
      const uint32_t id_s = idesc_f8(128, 128, 0, 0), id_o = idesc_f8(128, DIM, 0, 1);
      const uint64_t dq = smem_desc(smem_u32(sm.q[0]), 0, 1024, kLayoutSW128);
      const uint32_t q0 = static_cast<uint32_t>(dq), hi = static_cast<uint32_t>(dq >> 32);
      const uint32_t k0 =
          static_cast<uint32_t>(smem_desc(smem_u32(sm.k[0]), 0, 1024, kLayoutSW128));
      const uint32_t v0 =
          static_cast<uint32_t>(smem_desc(smem_u32(sm.v[0]), C::kBlock, 1024, kLayoutSW128));
      constexpr uint32_t kStep = C::kTileBytes / 16;
      int tc = 0, x[2] = {0, 0}, nq[2] = {0, 0};  // tiles and items of each row tile
      bool ok = true;
      for (int ns = 0; ok; ++ns) {
        const int sl = ns % kSegSlots;
        ok = mbar_wait_w_ab(smem_u32(&sm.seg_full[sl]), (ns / kSegSlots) & 1, &sm.abort);
        if (!ok) break;
        const int s = sm.seg[sl].s, nt = sm.seg[sl].i1 - sm.seg[sl].i0;
        const int tiles =
            static_cast<long long>(sm.seg[sl].n) * g.G - sm.seg[sl].row0 > 128 ? 2 : 1;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.seg_empty[sl]));
        if (s < 0) break;
        if (nt <= 0) continue;
        auto issue_s = [&](int y, int w) {  // scores of row tile w and key tile y
          const uint32_t a = q0 + w * kStep, b = k0 + (y & 1) * kStep;
          __syncwarp();
#pragma unroll
          for (int ks = 0; ks < DIM / 16; ++ks) {
            const uint32_t at = (ks >> 2) * (C::kBlock / 16) + (ks & 3) * 2;
            mma_f16(tmem + w * 128, a + at, b + at, hi, id_s, ks > 0);
          }
          tc_commit_w(smem_u32(&sm.s_full[w]));
          if (w == tiles - 1) tc_commit_w(smem_u32(&sm.k_empty[y & 1]));
          __syncwarp();
        };
        auto wait_k = [&](int y) {
          return mbar_wait_w_ab(smem_u32(&sm.k_full[y & 1]), (y >> 1) & 1, &sm.abort);
        };
        ok = wait_k(tc);
        for (int w = 0; w < tiles && ok; ++w) {
          ok = mbar_wait_w_ab(smem_u32(&sm.q_full[w]), nq[w]++ & 1, &sm.abort);
          if (!ok) break;
          tc_fence_after();
          issue_s(tc, w);
        }
        for (int t = 0; t < nt && ok; ++t) {
          const int y = tc + t;
          for (int w = 0; w < tiles && ok; ++w) {
            // (the keys and values first: they are there long before the weights, and a
            // wait costs some 200 cycles even so)
            if (w == 0)
              ok = mbar_wait_w_ab(smem_u32(&sm.v_full[y & 1]), (y >> 1) & 1, &sm.abort) &&
                   (t + 1 == nt || wait_k(y + 1));
            if (ok) ok = mbar_wait_w_ab(smem_u32(&sm.p_full[w]), x[w] & 1, &sm.abort);
            if (!ok) break;
            ++x[w];
            tc_fence_after();
            __syncwarp();
            const uint32_t a = tmem + w * 128, b = v0 + (y & 1) * kStep;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              mma_f16_ts(tmem + C::kColO + w * DIM, a + ks * 8, b + ks * (2048 / 16), hi, id_o,
                         t > 0 || ks > 0);
            tc_commit_w(smem_u32(&sm.pv_done[w]));
            if (w == tiles - 1) tc_commit_w(smem_u32(&sm.v_empty[y & 1]));
            __syncwarp();
            if (t + 1 < nt) issue_s(y + 1, w);
          }
        }
        tc += nt;
      }
      if (!ok) {
        sm.abort = 1;
        // what was issued ends before shared memory and tensor memory go
        __syncwarp();
        tc_commit_w(smem_u32(&sm.drained));
        mbar_wait_w(smem_u32(&sm.drained), 0);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && sm.abort) report(g.status, FLAMIA_DEV_TIMEOUT);
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int DIM>
bool launch(const flamia_kvcache* c, const AttendArgs& g, cudaStream_t s) {
  constexpr int smem = static_cast<int>(sizeof(Smem<DIM>)) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory");
  const int grid = min(kRowsCtas, num_sms());
  static std::atomic<unsigned long long> raised{0};
  return launch_large(attend_rows_kernel<DIM>, raised, dim3(grid), Cfg<DIM>::kThreads, smem, s, g,
                      static_cast<const uint8_t*>(c->k_codes),
                      static_cast<const uint8_t*>(c->v_codes)) &&
         (g.whole || launch_join<DIM, 256>(grid, s, g));
}

}  // namespace

flamia_status attend_rows(const flamia_kvcache* c, const AttendArgs& g, cudaStream_t s) {
  return (c->d == 128 ? launch<128>(c, g, s) : launch<64>(c, g, s)) ? FLAMIA_OK : FLAMIA_ERR_CUDA;
}

}  // namespace flamia
