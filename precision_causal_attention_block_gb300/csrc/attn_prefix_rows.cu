// Attention of many query rows over a shared prefix: its whole 128-key tiles, with the
// tokens of all sequences as the rows of each K / V head, 256 an item.
//
// The products and numerics are those of attn_cache_rows.cu (S = Q K^T and O += P V in FP16,
// the weights in tensor memory, w = 2^(x + eV - ref), l = sum w 2^(E0 - eV)), without masks:
// every row sees every key.  What differs is the order of work.  Scores come 64 keys at a
// time, in the two halves of a row tile's 128 columns; while the softmax takes one half, the
// tensor core adds the weights of the other to O and works out the scores that follow them,
// and each row tile has an issuing warp of its own.  So the softmax warps wait only where the
// products are behind.  All roles walk the CTA's run by themselves (its items are alike), which
// saves the hand-over of segments before the first loads.
//
// Measured: 89 tokens of 32 query and 8 K / V heads of 128 (356 rows a head) over 16,384 keys,
// 41 to 45 us with the launch and the set-up; the bytes alone (34 MB) take 5, the products 13 at
// the burst rate.  The tensor pipe is busy 30% of the time and the schedulers issue in 46% of
// the cycles.  Clock stamps: a half of a row tile takes its softmax warps 2,150 cycles (scores
// 350, weights 500, their stores 390, waits 250), a block of K or V its converters 2,050 (1,090
// of them to convert and store it, 700 until it is there), whatever the rows: the two chains
// are equally long.  One row tile's keys shared between both softmax warpgroups was slower
// (batch of 96 81.7 -> 86.7 us: the converters, and twice the parts to join).
//
// Warps 0-3 and 4-7: softmax of the two row tiles (thread = row = TMEM lane); 8-11:
// converters, a 32-key block each; 12 and 13: MMA issuers of the row tiles.
#include <climits>

#include "attend_rows.cuh"

namespace flamia {
namespace {

template <int DIM>
using Cfg = RowsCfg<DIM>;
constexpr int kR = 256;
constexpr int kCost = kItemCost<kR>;

template <int DIM>
struct Smem {
  using C = Cfg<DIM>;
  alignas(1024) uint8_t q[2][C::kTileBytes];
  alignas(1024) uint8_t k[2][C::kTileBytes];
  alignas(1024) uint8_t v[2][C::kTileBytes];
  alignas(16) float kf[4][128];   // 2^eK, eV of each key: a ring of four tiles, as
  alignas(16) int ev[4][128];     // the softmax is done two score products later
  Keys32 col[4][4];
  Sum past[kR];                   // sum 2^(x + nref) of what is not in a row's l
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], sc_full[4];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // by row tile and half
  uint64_t q_full[2], drained[2];
  int sharer;
  uint32_t tmem_base;
  volatile int abort;
};

// ------------------------------------------------------------------ work

// An item's key tiles i0 .. i1 - 1 in this CTA's run.
struct Piece {
  int hk, rt;   // K / V head, row tile of 256
  int i0, i1;
  long long at;  // the item's first unit
};

// The run: every role walks it for itself.
struct Run {
  long long u, u1, total;
  int units, hk, rt, o, row_tiles, tiles;

  __device__ __forceinline__ Run(const AttendArgs& g, int sharer) {
    const int n = min(max(g.cu[g.ndocs], 0), g.T);
    row_tiles = sharer < g.ndocs
                    ? static_cast<int>((static_cast<long long>(n) * g.G + kR - 1) / kR)
                    : 0;
    tiles = g.shared;
    units = tiles + kCost;
    total = static_cast<long long>(row_tiles) * g.H_kv * units;
    const long long ctas = active_ctas<kR>(g, total), c = blockIdx.x;
    u = c < ctas ? mul_div(total, c, ctas) : total;
    u1 = c < ctas ? mul_div(total, c + 1, ctas) : total;
    hk = rt = o = 0;
    if (u < u1) {
      const long long item = mul_div(u, 1, units);
      o = static_cast<int>(u - item * units);
      hk = static_cast<int>(mul_div(item, 1, row_tiles));
      rt = static_cast<int>(item - static_cast<long long>(hk) * row_tiles);
    }
  }
  __device__ __forceinline__ bool next(Piece& p) {
    while (u < u1) {
      const int take = static_cast<int>(min(u1 - u, static_cast<long long>(units - o)));
      p = Piece{hk, rt, max(o - kCost, 0), max(o + take - kCost, 0), u - o};
      u += take;
      o = 0;
      if (++rt == row_tiles) {
        rt = 0;
        ++hk;
      }
      if (p.i1 > p.i0) return true;  // (else the run ends before the item's first tile)
    }
    return false;
  }
};

// Adds 2^(x + nref) of 64 keys whose eV lies below floor_ev to a row's sum.  (Not inlined:
// rare.)
__device__ __noinline__ void sum_apart(Sum& past, const float* kf, const int* ev,
                                       const Keys32* col, uint32_t t_s, float qf, float nref,
                                       int floor_ev) {
  float top = kNoExponent, sum = 0.f;
#pragma unroll 1
  for (int i = 0; i < 16; ++i) {  // the largest, then the sum
    const int at = (i & 7) * 8;
    const bool here = col[at / 32].flags & kHere;
    uint32_t s[8];
    tmem_ld8(t_s + at, s);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float x = fmaf(__uint_as_float(s[j]), kf[at + j] * qf, nref);
      if (!here || ev[at + j] >= floor_ev) x = -INFINITY;
      if (i < 8)
        top = fmaxf(top, x);
      else
        sum += ex2_approx(x - top);
    }
    if (i == 7) top = ceilf(top);
  }
  past.add(sum, top);
}

// The products of one half: N of them, operands kStep apart, issued by one elected thread that
// is elected once.  (mma_f16's descriptors, as their low words and one high word.)
template <int DIM>
__device__ __forceinline__ void mma_scores(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t hi,
                                           uint32_t idesc) {
  static_assert(RowsCfg<DIM>::kBlock / 16 == 1024, "blocks of 64 columns");
  if constexpr (DIM == 128) {
    asm volatile(
        "{\n\t.reg .pred e, t, f;\n\t.reg .b32 x, y;\n\t.reg .b64 da, db;\n\t"
        "setp.eq.b32 t, 0, 0;\n\tsetp.ne.b32 f, 0, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
#define FLAMIA_MMA(off, p)                                                  \
  "add.u32 x, %1, " off ";\n\tadd.u32 y, %2, " off ";\n\t"                 \
  "mov.b64 da, {x, %3};\n\tmov.b64 db, {y, %3};\n\t"                       \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, " p ";\n\t"
        FLAMIA_MMA("0", "f") FLAMIA_MMA("2", "t") FLAMIA_MMA("4", "t") FLAMIA_MMA("6", "t")
        FLAMIA_MMA("1024", "t") FLAMIA_MMA("1026", "t") FLAMIA_MMA("1028", "t")
        FLAMIA_MMA("1030", "t") "}" ::"r"(d_tmem),
        "r"(a), "r"(b), "r"(hi), "r"(idesc)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred e, t, f;\n\t.reg .b32 x, y;\n\t.reg .b64 da, db;\n\t"
        "setp.eq.b32 t, 0, 0;\n\tsetp.ne.b32 f, 0, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t" FLAMIA_MMA("0", "f") FLAMIA_MMA("2", "t")
            FLAMIA_MMA("4", "t") FLAMIA_MMA("6", "t") "}" ::"r"(d_tmem),
        "r"(a), "r"(b), "r"(hi), "r"(idesc)
        : "memory");
#undef FLAMIA_MMA
  }
}
__device__ __forceinline__ void mma_values(uint32_t d_tmem, uint32_t a_tmem, uint32_t b,
                                           uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, t, p;\n\t.reg .b32 x, y;\n\t.reg .b64 db;\n\t"
      "setp.eq.b32 t, 0, 0;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
#define FLAMIA_MMA(aoff, boff, p)                                           \
  "add.u32 x, %1, " aoff ";\n\tadd.u32 y, %2, " boff ";\n\t"               \
  "mov.b64 db, {y, %3};\n\t"                                               \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %4, " p ";\n\t"
      FLAMIA_MMA("0", "0", "p") FLAMIA_MMA("8", "128", "t") FLAMIA_MMA("16", "256", "t")
      FLAMIA_MMA("24", "384", "t") "}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
#undef FLAMIA_MMA
}

// This warp's 32 query rows as FP16 numbers x 2^-e into rows row0 .. of an operand tile: copied
// to their place by 16-byte chunks, d / 8 lanes a row, then each lane converts its own row
// there.  Returns the lane's row's factor.  (Instructions set the pace: with rows worked
// out anew in every step and maxima across lanes an item's queries took 11,000 cycles.)
template <int DIM>
__device__ __forceinline__ float load_queries(const AttendArgs& g, int hk, int first, int rows,
                                              int row0, uint32_t tile, int lane) {
  constexpr int kLanes = DIM / 8, kPer = 32 / kLanes;
  const int sub = lane / kLanes, c = lane % kLanes, in = row0 & 127;
  const int i = (first + row0 + sub) / g.G;
  int h = first + row0 + sub - i * g.G;
  const __nv_bfloat16* src =
      g.q + i * g.q_stride + static_cast<long long>(hk * g.G + h) * DIM + c * 8;
  const long long step = g.q_stride - static_cast<long long>(g.G) * DIM;  // to the next token
#pragma unroll 2
  for (int r = sub; r < 32; r += kPer) {
    const bool there = row0 + r < rows;
    copy16(tile + tile_at<DIM>(in + r, c), there ? src : g.q, there ? 16 : 0);
    src += kPer * DIM;
    h += kPer;
    while (h >= g.G) {
      h -= g.G;
      src += step;
    }
  }
  copies_wait();
  __syncwarp();
  // magnitudes as integers; 0x7F80 and above: infinities and NaN, which become NaN and stay
  // out of the maximum
  const int r = in + lane;
  uint32_t a = 0;
#pragma unroll 4
  for (int c = 0; c < DIM / 8; ++c) {
    const uint4 w = lds128(tile + tile_at<DIM>(r, c));
    a = __vmaxu2(a, __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                             __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu)));
  }
  a = max(a & 0xFFFFu, a >> 16);
  if (a >= 0x7F80u) {
    a = 0;
#pragma unroll 1
    for (int e = 0; e < DIM / 2; ++e) {
      const uint32_t at = tile + tile_at<DIM>(r, e >> 2) + (e & 3) * 4;
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
#pragma unroll 4
  for (int c = 0; c < DIM / 8; ++c) {
    const uint32_t at = tile + tile_at<DIM>(r, c);
    const uint4 w = lds128(at);
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
    uint32_t y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      y[j] = half2_of(__fmul2_rn(
          make_float2(__uint_as_float(ww[j] << 16), __uint_as_float(ww[j] & 0xFFFF0000u)), inv));
    sts128(at, make_uint4(y[0], y[1], y[2], y[3]));
  }
  return g.scale_log2 * (ex < -126 ? 0x1p-127f : exp2i(ex));
}

template <int DIM>
__global__ void __launch_bounds__(Cfg<DIM>::kThreads, 1)
    attend_prefix_rows_kernel(const AttendArgs g, const uint8_t* k_codes, const uint8_t* v_codes) {
  using C = Cfg<DIM>;
  extern __shared__ uint8_t smem_raw[];
  Smem<DIM>& sm = *reinterpret_cast<Smem<DIM>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.k_full[i]), 4);
      mbar_init(smem_u32(&sm.v_full[i]), 4);
      mbar_init(smem_u32(&sm.k_empty[i]), 2);  // issuers
      mbar_init(smem_u32(&sm.v_empty[i]), 2);
      mbar_init(smem_u32(&sm.q_full[i]), 4);
      mbar_init(smem_u32(&sm.drained[i]), 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(smem_u32(&sm.s_full[i][h]), 1);
        mbar_init(smem_u32(&sm.p_full[i][h]), 4);
        mbar_init(smem_u32(&sm.pv_done[i][h]), 1);
      }
    }
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&sm.sc_full[i]), 4);
    sm.abort = 0;
    sm.sharer = g.ndocs;
    fence_barrier_init();
  }
  __syncthreads();
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
  // the first sequence that shares the prefix: its pages are read
  for (int b = tid; b < g.ndocs; b += C::kThreads) {
    if (reads_for_all(g, b)) {
      atomicMin(&sm.sharer, b);
      break;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  start_next();
  const uint32_t tmem = sm.tmem_base;
  const int sharer = sm.sharer;
  Run run(g, sharer);
  const int n_rows = static_cast<int>(
      min(static_cast<long long>(min(max(g.cu[g.ndocs], 0), g.T)) * g.G, (1ll << 31) - 1));
  Piece pc;

  if (warp >= 8 && warp < 12) {
    // ---------------------------------------------------------- converters
    set_registers<false, 112>();
    const int cw = warp - 8;
    int tc = 0;
    bool ok = true;
    const int32_t* table = g.table + static_cast<long long>(sharer) * g.table_stride;
    while (ok && run.next(pc)) {
      // K's codes, then V's, of one tile after another; what is next is loaded before
      // what is there is converted (one body for both, for the instruction cache).
      Block32<DIM> next, cur;
      int row = 0, kbyte = 0, vbyte = 0, kbyte1 = 0, vbyte1 = 0;
      bool good = false;
      // First rows of the block at the next 32 tiles (a lane each), in units of 32 rows
      // of the codes; -1: no page.
      int rows32 = -1;
      auto look_up = [&](int i) {
        const int key0 = i * 128 + cw * 32, slot = key0 / g.page_size;
        const bool need = i < pc.i1;
        const int page = need && slot < g.table_stride ? table[slot] : -1;
        const bool there = page >= 0 && page < g.num_pages;
        if (need && !there) report(g.status, FLAMIA_DEV_BAD_PAGE);
        rows32 = there ? (page * g.H_kv + pc.hk) * (g.page_size / 32) +
                             (key0 - slot * g.page_size) / 32
                       : -1;
      };
      auto load_k = [&](int i) {
        if (((i - pc.i0) & 31) == 0) look_up(i + lane);
        row = __shfl_sync(0xffffffffu, rows32, (i - pc.i0) & 31);
        next.seen = row >= 0 ? 0xffffffffu : 0u;
        const long long at = static_cast<long long>(max(row, 0)) * 32 + lane;
        kbyte1 = g.k_scales[at];
        vbyte1 = g.v_scales[at];
      };
      auto load_codes = [&](const uint8_t* codes) {
        next.load(codes + static_cast<long long>(max(row, 0)) * 32 * DIM, lane);
      };
      load_k(pc.i0);
      load_codes(k_codes);
#pragma unroll 1
      for (int j = 2 * pc.i0; j < 2 * pc.i1; ++j) {
        const int i = j >> 1, st = tc & 1, ss = tc & 3;
        const bool is_v = j & 1;
        cur = next;
        if (!is_v) {
          good = row >= 0;
          kbyte = kbyte1;
          vbyte = vbyte1;
        } else if (i + 1 < pc.i1) {
          load_k(i + 1);
        }
        if (j + 1 < 2 * pc.i1) load_codes(is_v ? k_codes : v_codes);
        if (tc >= 2)  // (the use before)
          ok = mbar_wait_w_ab(smem_u32(is_v ? &sm.v_empty[st] : &sm.k_empty[st]),
                              ((tc >> 1) & 1) ^ 1, &sm.abort);
        if (!ok) break;
        if (!is_v) {
          const int kx = good ? kbyte : 0, vx = good ? vbyte : 0;
          const int kb0 = __shfl_sync(0xffffffffu, kx, 0), vb0 = __shfl_sync(0xffffffffu, vx, 0);
          const bool uniform = __all_sync(0xffffffffu, kx == kb0 && vx == vb0);
          const int top = __reduce_max_sync(0xffffffffu, vx);
          const int low = good ? __reduce_min_sync(0xffffffffu, vx) : 255;
          sm.kf[ss][cw * 32 + lane] = pow2_byte(kx);
          sm.ev[ss][cw * 32 + lane] = vx - 127;
          if (lane == 0)
            sm.col[ss][cw] = Keys32{pow2_byte(kb0), vb0 - 127, good ? top - 127 : -127,
                                    (uniform ? kUniform : 0) | (good ? kEvery | kHere : 0) |
                                        (low << kLowShift)};
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
    // The product of half y has ended.  (A barrier for each half: the one before it on the
    // same barrier has, as later scores came behind it, and the next one cannot have.)
    auto wait_pv = [&](int y) {
      return mbar_wait_w_ab(smem_u32(&sm.pv_done[wg][y & 1]), (y >> 1) & 1, &sm.abort);
    };
    int tc = 0, x = 0;  // key tiles of the CTA; halves of this row tile
    bool ok = true;     // (a wait that ran out: the warp leaves, and the others' waits end)
    while (ok && run.next(pc)) {
      const int nt = pc.i1 - pc.i0, first = pc.rt * kR;
      const int rows = min(kR, n_rows - first);
      const bool active = wg == 0 || rows > 128;
      float qf = 0.f;  // the row's 2^e x softmax scale x log2 e
      if (active) {
        qf = load_queries<DIM>(g, pc.hk, first, rows, warp * 32, smem_u32(sm.q[wg]), lane);
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
      for (int j = 0; j < (active ? 2 * nt : 0); ++j, ++x) {
        const int half = j & 1, ss = (tc + (j >> 1)) & 3;
        ok = mbar_wait_w_ab(smem_u32(&sm.s_full[wg][half]), (x >> 1) & 1, &sm.abort);
        if (ok && half == 0)
          ok = mbar_wait_w_ab(smem_u32(&sm.sc_full[ss]), ((tc + (j >> 1)) >> 2) & 1, &sm.abort);
        if (!ok) break;
        tc_fence_after();
        const Keys32* col = sm.col[ss] + 2 * half;
        const Keys32 k0 = col[0], k1 = col[1];
        const int top = max(k0.top, k1.top);
        if (j == 0) {
          e0 = top;
        } else if (top > e0 + kHigh) {  // (as in attn_cache.cu)
          sm.past[r].add(l, -static_cast<float>(e0));
          l = 0.f;
          e0 = top;
        }
        const int floor_ev = e0 - kLow;
        // 32 keys with one K and one V exponent: y = x kq + (eV + nref)
        const float kq0 = k0.kf * qf, kq1 = k1.kf * qf;
        const int flags = k0.flags & k1.flags & (kUniform | kEvery);
        const int low = min(k0.flags >> kLowShift, k1.flags >> kLowShift) - 127;
        const bool apart = low < floor_ev;  // some keys are not in l
        const bool plain = flags == (kUniform | kEvery) && !apart;
        const uint32_t t_h = t_s + half * 64;
        // Any 32 keys: their y, masked where there is no page.
        auto scores = [&](int c, float (&y)[32]) {
          uint32_t s[32];
          tmem_ld32(t_h + c * 32, s);
          const bool here = col[c].flags & kHere;
          const float* kfs = sm.kf[ss] + half * 64 + c * 32;
          const int* evs = sm.ev[ss] + half * 64 + c * 32;
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 kf = *reinterpret_cast<const float4*>(kfs + i);
            const int4 ev = *reinterpret_cast<const int4*>(evs + i);
            const float kk[4] = {kf.x, kf.y, kf.z, kf.w};
            const int ee[4] = {ev.x, ev.y, ev.z, ev.w};
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const float v = fmaf(__uint_as_float(s[i + m]), kk[m] * qf,
                                   static_cast<float>(ee[m]) + nref);
              y[i + m] = here ? v : -INFINITY;
            }
          }
        };
        // Does the reference hold?  (The largest score comes with the load.)
        float mx = -INFINITY;
        uint32_t s0[32], s1[32];
        if (plain) {
          float m0, m1;
          tmem_ld32_max(t_h, s0, m0);
          tmem_ld32_max(t_h + 32, s1, m1);
          tmem_ld_wait();
          mx = fmaxf(fmaf(m0, kq0, static_cast<float>(k0.ev) + nref),
                     fmaf(m1, kq1, static_cast<float>(k1.ev) + nref));
        } else {
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            float y[32];
            scores(c, y);
#pragma unroll
            for (int i = 0; i < 32; i += 2) mx = fmax3(mx, y[i], y[i + 1]);
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
          if (j > 0) {  // O, once the product before has added to it
            ok = wait_pv(x - 1);
            if (!ok) break;
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
        // Weights, in the first half of the scores' columns.
        if (plain && !large) {
          auto weights = [&](int c, const uint32_t (&s)[32], float kq, int kev) {
            const float add = static_cast<float>(kev) + nref;
            const float2 kq2 = make_float2(kq, kq), add2 = make_float2(add, add);
            float2 y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              y[i] = __ffma2_rn(
                  make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), kq2, add2);
              y[i] = make_float2(ex2_approx(y[i].x), ex2_approx(y[i].y));
            }
            float2 a = y[0], b = y[1];
#pragma unroll
            for (int i = 2; i < 16; i += 2) {
              a = __fadd2_rn(a, y[i]);
              b = __fadd2_rn(b, y[i + 1]);
            }
            a = __fadd2_rn(a, b);
            l = fmaf(a.x + a.y, exp2i(e0 - kev), l);
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) p[i] = half2_of(y[i]);
            tmem_st16(t_h + c * 16, p);
          };
          weights(0, s0, kq0, k0.ev);
          weights(1, s1, kq1, k1.ev);
        } else {
          if (apart)
            sum_apart(sm.past[r], sm.kf[ss] + half * 64, sm.ev[ss] + half * 64, col, t_h, qf, nref,
                      floor_ev);
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            float y[32];
            scores(c, y);
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int ev = sm.ev[ss][half * 64 + c * 32 + i];
              y[i] = ex2_approx(cut(y[i], kSlack));
              l = fmaf(y[i], ev < floor_ev ? 0.f : exp2i(e0 - ev), l);
              if (i & 1) p[i / 2] = half2_of(make_float2(y[i - 1], y[i]));
            }
            tmem_st16(t_h + c * 16, p);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[wg][half]));
      }
      // ------------------------------------------------------------ epilogue
      if (ok && active) {
        ok = wait_pv(x - 1);
        if (!ok) break;
        tc_fence_after();
        const bool cut = pc.i0 > 0 || pc.i1 < run.tiles;
        const int slot = 2 * blockIdx.x + (pc.i0 == 0);
        const int tok = (first + r) / g.G, hq = pc.hk * g.G + (first + r) - tok * g.G;
        const bool live = r < rows;
        Sum past = sm.past[r];
        past.add(l, -static_cast<float>(e0));
        const float lg = past.m == 0.f ? -INFINITY : log2f(past.m) + past.e - nref;
        const int k = static_cast<int>(-past.e);  // (as in attn_cache.cu)
        const float inv = past.m == 0.f ? 0.f : pow2_within(k / 2) / past.m;
        const float ve = pow2_within(k - k / 2);
        const size_t out = static_cast<size_t>(tok) * g.H + hq;
        if (live) {
          if (cut)
            g.stats[static_cast<size_t>(slot) * kR + r] = lg;
          else
            g.row_stats[0][out] = lg;
          if (pc.i0 == 0)
            g.where[0][out] = RowParts{static_cast<int>(blockIdx.x) | (r << 16),
                                       parts_from_here<kR>(g, pc.at, run.units, run.total)};
        }
#pragma unroll
        for (int c = 0; c < DIM; c += 32) {
          uint32_t a[32];
          tmem_ld32(t_o + c, a);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j)
            a[j] = inv == 0.f ? 0u : __float_as_uint(__uint_as_float(a[j]) * inv * ve);
          if (live) {
            uint4* p = cut ? reinterpret_cast<uint4*>(g.partial) +
                                 (static_cast<size_t>(slot) * (DIM / 4) + c / 4) * kR + r
                           : reinterpret_cast<uint4*>(g.rows[0] + out * DIM + c);
            const int step = cut ? kR : 1;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              p[j * step] = make_uint4(a[4 * j], a[4 * j + 1], a[4 * j + 2], a[4 * j + 3]);
          }
        }
        tc_fence_before();
        __syncwarp();
      }
      tc += nt;
    }
    if (!ok) sm.abort = 1;
  } else {
    set_registers<false, 64>();  // (all four warps at once)
    if (warp < 14) {
      // -------------------------------------------------------- MMA issuers
      const int w = warp - 12;
      const uint32_t id_s = idesc_f8(128, 64, 0, 0), id_o = idesc_f8(128, DIM, 0, 1);
      const uint64_t dq = smem_desc(smem_u32(sm.q[w]), 0, 1024, kLayoutSW128);
      const uint32_t q0 = static_cast<uint32_t>(dq), hi = static_cast<uint32_t>(dq >> 32);
      const uint32_t k0 =
          static_cast<uint32_t>(smem_desc(smem_u32(sm.k[0]), 0, 1024, kLayoutSW128));
      const uint32_t v0 =
          static_cast<uint32_t>(smem_desc(smem_u32(sm.v[0]), C::kBlock, 1024, kLayoutSW128));
      constexpr uint32_t kStep = C::kTileBytes / 16;
      const uint32_t t_s = tmem + w * 128, t_o = tmem + C::kColO + w * DIM;
      int tc = 0, x = 0, nq = 0;  // tiles of the CTA; halves and items of this row tile
      bool ok = true;
      auto wait_k = [&](int y) {
        return mbar_wait_w_ab(smem_u32(&sm.k_full[y & 1]), (y >> 1) & 1, &sm.abort);
      };
      auto wait_v = [&](int y) {
        return mbar_wait_w_ab(smem_u32(&sm.v_full[y & 1]), (y >> 1) & 1, &sm.abort);
      };
      // scores of half h of tile y
      auto issue_s = [&](int y, int h) {
        const uint32_t b = k0 + (y & 1) * kStep + h * (8192 / 16);
        __syncwarp();
        mma_scores<DIM>(t_s + h * 64, q0, b, hi, id_s);
        tc_commit_w(smem_u32(&sm.s_full[w][h]));
        if (h == 1) tc_commit_w(smem_u32(&sm.k_empty[y & 1]));
        __syncwarp();
      };
      while (ok && run.next(pc)) {
        const int nt = pc.i1 - pc.i0;
        if (w == 1 && n_rows - pc.rt * kR <= 128) {
          // (no rows here: K and V are free as soon as they are there)
          for (int t = 0; t < nt && ok; ++t) {
            ok = wait_k(tc + t);
            if (ok && lane == 0) mbar_arrive(smem_u32(&sm.k_empty[(tc + t) & 1]));
            ok = ok && wait_v(tc + t);
            if (ok && lane == 0) mbar_arrive(smem_u32(&sm.v_empty[(tc + t) & 1]));
            __syncwarp();
          }
          tc += nt;
          continue;
        }
        ok = wait_k(tc) && mbar_wait_w_ab(smem_u32(&sm.q_full[w]), nq++ & 1, &sm.abort);
        if (!ok) break;
        tc_fence_after();
        issue_s(tc, 0);
        issue_s(tc, 1);
        for (int j = 0; j < 2 * nt && ok; ++j, ++x) {
          const int y = tc + (j >> 1), h = j & 1;
          // (the keys and values first: they are there long before the weights)
          if (h == 0) ok = wait_v(y) && (j + 2 >= 2 * nt || wait_k(y + 1));
          ok = ok && mbar_wait_w_ab(smem_u32(&sm.p_full[w][h]), (x >> 1) & 1, &sm.abort);
          if (!ok) break;
          tc_fence_after();
          __syncwarp();
          const uint32_t b = v0 + (y & 1) * kStep + h * (8192 / 16);
          mma_values(t_o, t_s + h * 64, b, hi, id_o, j > 0);
          tc_commit_w(smem_u32(&sm.pv_done[w][h]));
          if (h == 1) tc_commit_w(smem_u32(&sm.v_empty[y & 1]));
          __syncwarp();
          if (j + 2 < 2 * nt) issue_s(y + 1, h);
        }
        tc += nt;
      }
      if (!ok) {
        sm.abort = 1;
        // what was issued ends before shared memory and tensor memory go
        __syncwarp();
        tc_commit_w(smem_u32(&sm.drained[w]));
        mbar_wait_w(smem_u32(&sm.drained[w]), 0);
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
  static std::atomic<unsigned long long> raised{0};
  return launch_large(attend_prefix_rows_kernel<DIM>, raised, dim3(min(kRowsCtas, num_sms())),
                      Cfg<DIM>::kThreads, smem, s, g, static_cast<const uint8_t*>(c->k_codes),
                      static_cast<const uint8_t*>(c->v_codes));
}

}  // namespace

flamia_status attend_prefix_rows(const flamia_kvcache* c, const AttendArgs& g, cudaStream_t s) {
  return (c->d == 128 ? launch<128>(c, g, s) : launch<64>(c, g, s)) ? FLAMIA_OK : FLAMIA_ERR_CUDA;
}

}  // namespace flamia
