// Attention of few query rows of a K / V head over the cache, for calls whose sequences
// share a prefix: up to 96 rows of the whole batch over the prefix, and every sequence's
// rows over what comes behind it.
//
// Here HBM or latency sets the pace, not the tensor core: a 128-key tile's codes take some
// 1,400 cycles of an SM's share of HBM (heads of 128), the products of 16 rows with it a few
// hundred.  So each warp works for itself, on 32 keys at a time, with warp-level products
// (m16n8k16, FP16 with float32 sums) whose operands are registers: no barriers, no tensor
// memory to hand out, and short chains from the codes to the result, where a tcgen05 kernel's
// tile goes through four roles.
//
//   S = Q K^T:  the cached codes are FP16 numbers exactly; the lane that holds key j of the
//     B fragment reads d / 4 bytes of it side by side, as the order of the dims inside the
//     sum is free (Q's fragments take the same).
//   O += P V:  P's fragments are S's.  A lane reads d / 8 dims of four keys; pairs of keys
//     are brought together byte by byte before they are converted, and the order of the
//     output's columns is free again: a lane ends with d / 4 dims side by side of two rows.
// Numerics as in attn_cache_rows.cu: queries times 2^-e, w = 2^(x + eV - ref) rounded to FP16,
// l = sum w 2^(E0 - eV), references that move when a block exceeds them by more than
// kSlack (a vote of the warp), a Sum for what l cannot hold, masks with NaN.
//
// A CTA's four warps take every fourth 32-key block of its run of key tiles and are joined in
// shared memory; parts of an item in several CTAs by attn_prefix.cu's last kernel.  Codes go
// through a ring of each warp's own (cp.async; every lane reads back what it asked for).
#include "attend_rows.cuh"

namespace flamia {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

template <int DIM, int MT>  // MT x 16 rows an item
struct Few {
  static constexpr int kRows = 16 * MT;
  static constexpr int kKSteps = DIM / 16;
  static constexpr int kOut = DIM / 8;              // column tiles of O
  static constexpr int kStages = DIM == 128 ? 2 : 4;
  static constexpr int kKBytes = 32 * DIM;          // K's codes of 32 keys
  static constexpr int kStage = 2 * kKBytes + 80;   // and V's, their scale bytes, a flag
  static constexpr int kRing = (kStages * kStage + 127) / 128 * 128;
  static constexpr int kCtas = 3;
  static_assert(kRows * DIM * 4 <= kRing, "a warp's O takes the place of its ring");
};

// What the warps of a CTA work on: an item's keys k_lo .. k_hi - 1.
struct Piece {
  int s;                // its first packed row; -1: the run has ended
  int rows;             // of the item
  int start, row0, hk, seq;
  int k_lo, k_hi;
  int every;            // keys before this one are seen by all rows
  int slot;             // partial result slot, or -1: the whole item
  int side;             // 0: over the prefix, 1: not
  int parts;            // RowParts::n if it holds the item's first tile, or 0
};

template <int DIM, int MT>
struct Smem {
  using C = Few<DIM, MT>;
  alignas(128) uint8_t ring[kWarps][C::kRing];
  uint4 q[MT][C::kKSteps][32];     // A fragments of the queries, by lane
  float qf[C::kRows];              // 2^e x softmax scale x log2 e
  int pos[C::kRows];               // -1: no such row
  Sum past[kWarps][2 * MT][32];    // sum 2^(x + nref) of what is not in a lane's l
  float lg[kWarps][C::kRows];
  Piece piece[2];
  int plan_b, sharer;
  SeqWork plan_seq;
  long long plan_off, plan_u0, plan_u1, plan_total;
  long long scan[kWarps];
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four E4M3 codes as FP16 pairs (exact; NaN stays).
__device__ __forceinline__ void halves_of_codes(uint32_t codes, uint32_t& a, uint32_t& b) {
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(codes));
}

// N bytes (8 or 16) from global to shared memory; zeros if there is nothing to read.
template <int N>
__device__ __forceinline__ void fetch(uint32_t dst, const void* src, bool there = true) {
  if (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src),
                 "r"(there ? 8 : 0)
                 : "memory");
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void fetch_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ bool holds_nan(uint32_t codes) {
  return (((codes & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
}

// The CTA's run, cut into pieces by one thread (its state stays in shared memory: sm.plan_*).
template <int R, int KEYS, class Sm>
__device__ __noinline__ void next_piece(const AttendArgs& g, Sm& sm, Piece& out) {
  constexpr int kCost = kItemCost<R, KEYS>;
  // plan_off: the unit inside sequence plan_b at which the run goes on
  SeqWork w = sm.plan_seq;
  long long u = sm.plan_u0;
  const long long u1 = sm.plan_u1, total = sm.plan_total;
  Piece p{};
  p.s = -1;
  while (u < u1) {
    const long long item = mul_div(sm.plan_off, 1, w.units);
    const int o = static_cast<int>(sm.plan_off - item * w.units);
    const int hk = static_cast<int>(mul_div(item, 1, w.row_tiles));
    const int rt = static_cast<int>(item - static_cast<long long>(hk) * w.row_tiles);
    const int take = static_cast<int>(min(u1 - u, static_cast<long long>(w.units - o)));
    const int i0 = g.whole ? 0 : max(o - kCost, 0);
    const int i1 = g.whole ? w.tiles : max(o + take - kCost, 0);
    const int v = sm.plan_b;
    const bool over = of_prefix<KEYS>(v), sharing = !over && shares(g, w.start);
    const int seq = over ? sm.sharer : seq_of<KEYS>(v);
    if (!over && hk == 0 && rt == 0 && i0 == 0) {
      const int raw = g.starts != nullptr ? g.starts[seq] : 0;
      if (raw > g.cap - w.n) report(g.status, FLAMIA_DEV_BAD_PAGE);
    }
    if (i1 > i0) {  // (else the run ends before the item's first tile)
      const int wt = sharing ? g.shared : 0;
      const bool cut = i0 > 0 || i1 < w.tiles;
      p.s = w.s;
      p.row0 = rt * R;
      p.rows = static_cast<int>(
          min(static_cast<long long>(R), static_cast<long long>(w.n) * g.G - p.row0));
      p.start = w.start;
      p.hk = hk;
      p.seq = seq;
      p.k_lo = (i0 + wt) * 128;
      // behind the last key that its last row sees
      const int hi = over ? g.shared * 128 : max(w.start + (p.row0 + p.rows - 1) / g.G + 1, 0);
      p.k_hi = min((i1 + wt) * 128, hi);
      p.every = over ? hi : w.start + p.row0 / g.G + 1;
      p.slot = cut ? 2 * static_cast<int>(blockIdx.x) + (i0 == 0) : -1;
      p.side = over ? 0 : 1;
      p.parts = i0 > 0 ? 0
                       : (cut ? parts_from_here<R, KEYS>(g, u - o, w.units, total) : 1) |
                             (sharing ? kShares : 0);
    }
    u += take;
    sm.plan_off += take;
    if (sm.plan_off == w.total(g.H_kv) && u < u1) {
      int b = v;
      do {
        w = seq_work<R, KEYS>(g, ++b, sm.sharer);  // there is one: u < u1
      } while (w.row_tiles == 0 && seq_of<KEYS>(b) + 1 < g.ndocs);
      sm.plan_b = b;
      sm.plan_seq = w;
      sm.plan_off = 0;
    }
    if (p.s >= 0) break;
  }
  sm.plan_u0 = u;
  out = p;
}

template <int DIM, int MT, int KEYS>
__global__ void __launch_bounds__(kThreads, Few<DIM, MT>::kCtas)
    attend_prefix_few_kernel(const AttendArgs g, const uint8_t* k_codes, const uint8_t* v_codes) {
  using C = Few<DIM, MT>;
  constexpr int R = C::kRows, KS = C::kKSteps;
  extern __shared__ uint8_t smem_raw[];
  Smem<DIM, MT>& sm = *reinterpret_cast<Smem<DIM, MT>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gr = lane >> 2, t = lane & 3;  // fragments: row (or key, or column), quarter
  start_next();
  wait_for_previous();
  check_offsets(g.cu, g.ndocs, g.T, static_cast<long long>(blockIdx.x) * kThreads + tid,
                static_cast<long long>(gridDim.x) * kThreads, g.status);
  make_plan<R, KEYS, kThreads>(g, sm);
  if (tid == 0) next_piece<R, KEYS>(g, sm, sm.piece[0]);
  __syncthreads();
  const uint32_t ring = smem_u32(sm.ring[warp]);

#pragma unroll 1
  for (int np = 0;; ++np) {
    const Piece& pc = sm.piece[np & 1];
    if (pc.s < 0) break;
    // ------------------------------------------------------------- keys
    const int k_lo = pc.k_lo, k_hi = pc.k_hi;
    // this warp's 32-key blocks (0 or less: none)
    const int mine = ((max(k_hi - k_lo, 0) + 31) / 32 - warp + kWarps - 1) / kWarps;
    int rows32 = -1;  // first rows of its next 32 blocks (a lane each) / 32; -1: no page
    auto key_of = [&](int m) { return k_lo + (warp + m * kWarps) * 32; };
    auto issue = [&](int m) {
      if (m < mine) {
        if ((m & 31) == 0) {
          const int key0 = key_of(m + lane), slot = key0 / g.page_size;
          const bool need = m + lane < mine;
          const int page = need && slot < g.table_stride
                               ? g.table[static_cast<long long>(pc.seq) * g.table_stride + slot]
                               : -1;
          const bool there = page >= 0 && page < g.num_pages;
          if (need && !there) report(g.status, FLAMIA_DEV_BAD_PAGE);
          rows32 = there ? (page * g.H_kv + pc.hk) * (g.page_size / 32) +
                               (key0 - slot * g.page_size) / 32
                         : -1;
        }
        const int row = __shfl_sync(0xffffffffu, rows32, m & 31);
        const long long base = static_cast<long long>(max(row, 0)) * 32;
        const int n = row < 0 ? 0 : k_hi - key_of(m);  // keys that are there (32 or more: all)
        const uint32_t at = (m % C::kStages) * C::kStage;
        const uint32_t kd = ring + at + lane * 16, vd = ring + at + C::kKBytes + lane * (DIM / 8);
        const uint8_t* kc = k_codes + base * DIM + gr * DIM + t * (DIM / 4);
        const uint8_t* vc = v_codes + base * DIM + 2 * t * DIM + gr * (DIM / 8);
        auto all = [&](auto there) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int p = 0; p < DIM / 64; ++p)
              fetch<16>(kd + (j * (DIM / 64) + p) * 512, kc + j * 8 * DIM + p * 16,
                        there(j * 8 + gr));
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int key = (j >> 2) * 16 + ((j >> 1) & 1) * 8 + (j & 1);
            fetch<DIM / 8>(vd + j * (4 * DIM), vc + key * DIM, there(key + 2 * t));
          }
        };
        if (n >= 32)
          all([](int) { return true; });
        else
          all([&](int key) { return key < n; });
        if (lane == 0)
          *reinterpret_cast<int*>(sm.ring[warp] + at + 2 * C::kKBytes + 64) = row >= 0;
        if (lane < 4)
          fetch<16>(ring + at + 2 * C::kKBytes + lane * 16,
                    (lane < 2 ? g.k_scales : g.v_scales) + base + (lane & 1) * 16, n > 0);
      }
      fetch_commit();
    };
#pragma unroll 1
    for (int m = 0; m < C::kStages; ++m) issue(m);

    // ------------------------------------------------------------- queries
    // DIM / 8 lanes a row; their numbers go to the lanes whose fragments hold them.
    {
      constexpr int kLanes = DIM / 8, kPer = kThreads / kLanes;
      const int c = tid % kLanes;
#pragma unroll 1
      for (int r = tid / kLanes; r < R; r += kPer) {
        const int i = (pc.row0 + r) / g.G, h = pc.hk * g.G + pc.row0 + r - i * g.G;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (r < pc.rows)
          w = *reinterpret_cast<const uint4*>(g.q + (pc.s + i) * g.q_stride +
                                              static_cast<long long>(h) * DIM + c * 8);
        uint32_t x[4] = {w.x, w.y, w.z, w.w};
        // magnitudes as integers; 0x7F80 and above: infinities and NaN, which become NaN
        // and stay out of the maximum
        uint32_t a = __vmaxu2(__vmaxu2(x[0] & 0x7FFF7FFFu, x[1] & 0x7FFF7FFFu),
                              __vmaxu2(x[2] & 0x7FFF7FFFu, x[3] & 0x7FFF7FFFu));
        a = max(a & 0xFFFFu, a >> 16);
        if (a >= 0x7F80u) {
          a = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if ((x[e] & 0x7F80u) == 0x7F80u)
              x[e] = (x[e] & 0xFFFF0000u) | 0x7FC0u;
            else
              a = max(a, x[e] & 0x7FFFu);
            if ((x[e] & 0x7F800000u) == 0x7F800000u)
              x[e] = (x[e] & 0xFFFFu) | 0x7FC00000u;
            else
              a = max(a, (x[e] >> 16) & 0x7FFFu);
          }
        }
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1)
          a = max(a, __shfl_xor_sync(0xffffffffu, a, off));
        const int ex = roundup_exponent(__uint_as_float(a << 16));
        const float2 inv = make_float2(exp2i(-ex), exp2i(-ex));
        const int dd = c * 8 % (DIM / 4), to = (r & 7) * 4 + c * 8 / (DIM / 4), half = (r >> 3) & 1;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          (&sm.q[r >> 4][dd / 4 + e / 2][to].x)[(e & 1) * 2 + half] = half2_of(__fmul2_rn(
              make_float2(__uint_as_float(x[e] << 16), __uint_as_float(x[e] & 0xFFFF0000u)), inv));
        if (c == 0) {
          sm.qf[r] = g.scale_log2 * (ex < -126 ? 0x1p-127f : exp2i(ex));
          sm.pos[r] = r < pc.rows ? max(pc.start + i, -1) : -1;
        }
      }
    }
    __syncthreads();
    if (warp == kWarps - 1 && lane == 0)  // (it has the fewest blocks)
      next_piece<R, KEYS>(g, sm, sm.piece[(np + 1) & 1]);
    __syncwarp();

    float o[MT][C::kOut][4];
    float l[2 * MT], nref[2 * MT];  // by row: 16 (i / 2) + 8 (i % 2) + lane / 4
    uint32_t has = 0;               // rows with a reference
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < C::kOut; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][i][e] = 0.f;
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) {
      l[i] = nref[i] = 0.f;
      sm.past[warp][i][lane] = Sum{0.f, kNoExponent};
    }
    int e0 = -127;
    bool large = false;

    // ------------------------------------------------------------- blocks
#pragma unroll 1
    for (int m = 0; m < mine; ++m) {
      fetch_wait<C::kStages - 1>();
      __syncwarp();
      const uint8_t* st = sm.ring[warp] + (m % C::kStages) * C::kStage;
      const int key0 = key_of(m);
      // scores
      float s[MT][4][4];
      {
        uint32_t kw[4][KS];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int p = 0; p < DIM / 64; ++p) {
            const uint4 x =
                *reinterpret_cast<const uint4*>(st + (j * (DIM / 64) + p) * 512 + lane * 16);
            kw[j][4 * p] = x.x, kw[j][4 * p + 1] = x.y, kw[j][4 * p + 2] = x.z,
            kw[j][4 * p + 3] = x.w;
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][j][e] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t a[MT][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const uint4 x = sm.q[mt][k][lane];
            a[mt][0] = x.x, a[mt][1] = x.y, a[mt][2] = x.z, a[mt][3] = x.w;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t b0, b1;
            halves_of_codes(kw[j][k], b0, b1);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) mma16816(s[mt][j], a[mt], b0, b1);
          }
        }
      }
      // exponents: one of K and one of V for all 32 keys, or each key's
      const uint8_t* ksc = st + 2 * C::kKBytes;
      const uint8_t* vsc = ksc + 32;
      const bool there = *reinterpret_cast<const int*>(ksc + 64) != 0;
      const bool all = there && key0 + 32 <= k_hi;          // every key is there
      const bool every = all && key0 + 32 <= pc.every;      // and every row sees it
      const int kb0 = ksc[0], vb0 = vsc[0];
      const bool uniform =
          __all_sync(0xffffffffu, ksc[lane] == kb0 && vsc[lane] == vb0) && all;
      uint32_t nan = 0;  // of this lane's keys: half seen, with a NaN in V
      int top = vb0 - 127, low = top;  // the largest and the smallest eV of keys that are there
      if (!every) {
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(st + C::kKBytes + j * (4 * DIM) +
                                                                lane * (DIM / 8));
          bool bad = false;
#pragma unroll
          for (int i = 0; i < DIM / 32; ++i) bad |= holds_nan(w[i]);
          nan |= static_cast<uint32_t>(bad) << j;
        }
        nan |= __shfl_xor_sync(0xffffffffu, nan, 4);
        nan |= __shfl_xor_sync(0xffffffffu, nan, 8);
        nan |= __shfl_xor_sync(0xffffffffu, nan, 16);
      }
      if (!uniform) {
        const bool live = there && key0 + lane < k_hi;
        const int v = vsc[lane] - 127;
        top = __reduce_max_sync(0xffffffffu, live ? v : -127);
        low = __reduce_min_sync(0xffffffffu, live ? v : 128);
      }
      if (m == 0) {
        e0 = top;
      } else if (top > e0 + kHigh) {  // (as in attn_cache.cu)
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
          sm.past[warp][i][lane].add(l[i], -static_cast<float>(e0));
          l[i] = 0.f;
        }
        e0 = top;
      }
      const bool apart = low < e0 - kLow;  // some keys are not in l
      // y = x + eV - ref
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) {
        const float qf = sm.qf[(i >> 1) * 16 + (i & 1) * 8 + gr];
        float* y0 = &s[i >> 1][0][0] + 2 * (i & 1);
        if (uniform) {
          const float f = pow2_byte(kb0) * qf, a = static_cast<float>(vb0 - 127) + nref[i];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            y0[4 * j] = fmaf(y0[4 * j], f, a);
            y0[4 * j + 1] = fmaf(y0[4 * j + 1], f, a);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = j * 8 + 2 * t + e;
              y0[4 * j + e] = fmaf(y0[4 * j + e], pow2_byte(ksc[key]) * qf,
                                   static_cast<float>(vsc[key] - 127) + nref[i]);
            }
        }
        if (!every) {
          // (key j * 8 + 2 t + e is V's number 2 j + e of this lane)
          const int pos = pc.side == 0 ? k_hi : sm.pos[(i >> 1) * 16 + (i & 1) * 8 + gr];
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = key0 + j * 8 + 2 * t + e;
              float& y = y0[4 * j + e];
              if ((nan >> (j * 2 + e)) & 1) y = __uint_as_float(0x7FC00000u);
              if (!(there && key < k_hi && key <= pos)) y = -INFINITY;
            }
        }
      }
      // Do the references hold?
      bool need = false;
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) {
        const float* y = &s[i >> 1][0][0] + 2 * (i & 1);
        const float mx = fmaxf(fmax3(fmax3(y[0], y[1], y[4]), y[5], y[8]), fmax3(y[9], y[12], y[13]));
        need |= (has >> i) & 1 ? mx > kSlack + room(nref[i]) : mx > -INFINITY;
      }
      if (__any_sync(0xffffffffu, need)) {
        large = false;
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
          float* y = &s[i >> 1][0][0] + 2 * (i & 1);
          float x = fmaxf(fmax3(fmax3(y[0], y[1], y[4]), y[5], y[8]), fmax3(y[9], y[12], y[13]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));  // the row's, over its four lanes
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          const bool had = (has >> i) & 1;
          if (had ? x > kSlack + room(nref[i]) : x > -INFINITY) {
            const float by = lowered(nref[i] - ceilf(x)) - nref[i];
            const float f = had ? ex2_approx(by) : 1.f;
            l[i] *= f;
            nref[i] += by;
            sm.past[warp][i][lane].e += by;
            has |= 1u << i;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              y[4 * j] += by;
              y[4 * j + 1] += by;
            }
#pragma unroll
            for (int n = 0; n < C::kOut; ++n) {
              o[i >> 1][n][2 * (i & 1)] *= f;
              o[i >> 1][n][2 * (i & 1) + 1] *= f;
            }
          }
          large |= fabsf(nref[i]) > kLarge;
        }
        large = __any_sync(0xffffffffu, large);
      }
      if (apart) {  // keys that l does not hold: sum 2^(x + nref)
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
          const float* y = &s[i >> 1][0][0] + 2 * (i & 1);
          float x[8], most = kNoExponent, sum = 0.f;
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const int v = vsc[(n >> 1) * 8 + 2 * t + (n & 1)] - 127;
            x[n] = v < e0 - kLow ? y[4 * (n >> 1) + (n & 1)] - static_cast<float>(v) : -INFINITY;
            most = fmaxf(most, x[n]);
          }
          most = ceilf(most);
#pragma unroll
          for (int n = 0; n < 8; ++n) sum += ex2_approx(x[n] - most);
          sm.past[warp][i][lane].add(sum, most);
        }
      }
      // weights
      uint32_t p[MT][2][4];
      if (large) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][j][e] = cut(s[mt][j][e], kSlack);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][j][e] = ex2_approx(s[mt][j][e]);
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) {
        const float* y = &s[i >> 1][0][0] + 2 * (i & 1);
        if (uniform) {
          const float a = ((y[0] + y[1]) + (y[4] + y[5])) + ((y[8] + y[9]) + (y[12] + y[13]));
          l[i] = fmaf(a, apart ? 0.f : exp2i(e0 - (vb0 - 127)), l[i]);
        } else {
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const int v = vsc[(n >> 1) * 8 + 2 * t + (n & 1)] - 127;
            if (v >= e0 - kLow && v <= e0 + kHigh)  // (else not there, or apart)
              l[i] = fmaf(y[4 * (n >> 1) + (n & 1)], exp2i(e0 - v), l[i]);
          }
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float* y = &s[mt][2 * kk + (e >> 1)][2 * (e & 1)];
            p[mt][kk][e] = half2_of(make_float2(y[0], y[1]));
          }
      // O += P V
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        uint32_t v[4][DIM / 32];  // four keys, DIM / 8 dims each
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint8_t* at = st + C::kKBytes + (kk * 4 + j) * (4 * DIM) + lane * (DIM / 8);
          if constexpr (DIM == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(at);
            v[j][0] = x.x, v[j][1] = x.y, v[j][2] = x.z, v[j][3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(at);
            v[j][0] = x.x, v[j][1] = x.y;
          }
        }
        if (nan != 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if ((nan >> (kk * 4 + j)) & 1) {
#pragma unroll
              for (int w = 0; w < DIM / 32; ++w) v[j][w] = 0;
            }
        }
#pragma unroll
        for (int w = 0; w < DIM / 32; ++w) {
          uint32_t b[4][2];
          halves_of_codes(__byte_perm(v[0][w], v[1][w], 0x5140), b[0][0], b[1][0]);
          halves_of_codes(__byte_perm(v[0][w], v[1][w], 0x7362), b[2][0], b[3][0]);
          halves_of_codes(__byte_perm(v[2][w], v[3][w], 0x5140), b[0][1], b[1][1]);
          halves_of_codes(__byte_perm(v[2][w], v[3][w], 0x7362), b[2][1], b[3][1]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) mma16816(o[mt][4 * w + i], p[mt][kk], b[i][0], b[i][1]);
        }
      }
      __syncwarp();
      issue(m + C::kStages);
    }
    fetch_wait<0>();
    __syncwarp();

    // ------------------------------------------------------------- results
    // The warp's rows as means of values (as in attn_cache.cu) over its ring, 16-byte chunks
    // swizzled by the row.
    float* out = reinterpret_cast<float*>(sm.ring[warp]);
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) {
      Sum all = sm.past[warp][i][lane];
      all.add(l[i], -static_cast<float>(e0));
#pragma unroll
      for (int off = 1; off < 4; off <<= 1) {
        const float a = __shfl_xor_sync(0xffffffffu, all.m, off);
        const float b = __shfl_xor_sync(0xffffffffu, all.e, off);
        all.add(a, b);
      }
      const int r = (i >> 1) * 16 + (i & 1) * 8 + gr;
      const float lg = all.m == 0.f ? -INFINITY : log2f(all.m) + all.e - nref[i];
      const int k = static_cast<int>(-all.e);
      const float inv = all.m == 0.f ? 0.f : pow2_within(k / 2) / all.m;
      const float ve = pow2_within(k - k / 2);
      if (t == 0) sm.lg[warp][r] = lg;
      // dims t (d / 4) + n, then + d / 8: column tile n's two columns of this lane
#pragma unroll
      for (int n = 0; n < C::kOut; n += 4)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = 2 * (i & 1) + e;
          float4 x = make_float4(o[i >> 1][n][c] * inv * ve, o[i >> 1][n + 1][c] * inv * ve,
                                 o[i >> 1][n + 2][c] * inv * ve, o[i >> 1][n + 3][c] * inv * ve);
          if (inv == 0.f) x = make_float4(0.f, 0.f, 0.f, 0.f);
          const int chunk = (t * (DIM / 4) + e * (DIM / 8) + n) / 4;
          *reinterpret_cast<float4*>(out + r * DIM + (chunk ^ (r & 7)) * 4) = x;
        }
    }
    __syncthreads();
    // the four warps' joined: kThreads / R threads a row
    constexpr int kPer = kThreads / R, kMine = DIM / kPer;  // threads a row, dims a thread
    const int r = tid / kPer, d0 = tid % kPer * kMine;
    if (r < pc.rows) {
      float lg[kWarps], ref = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        lg[w] = sm.lg[w][r];
        ref = lg[w] > ref || lg[w] != lg[w] ? lg[w] : ref;  // NaN stays
      }
      const float base = ref == -INFINITY ? 0.f : ref;
      float sum = 0.f, acc[kMine] = {};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float wt = exp2f(0.5f * (lg[w] - base));  // (in two halves)
        sum = fmaf(wt, wt, sum);
        const float* x = reinterpret_cast<const float*>(sm.ring[w]) + r * DIM;
#pragma unroll
        for (int i = 0; i < kMine; i += 4) {
          const float4 v = *reinterpret_cast<const float4*>(x + (((d0 + i) / 4) ^ (r & 7)) * 4);
          acc[i] = fmaf(wt, wt * v.x, acc[i]);
          acc[i + 1] = fmaf(wt, wt * v.y, acc[i + 1]);
          acc[i + 2] = fmaf(wt, wt * v.z, acc[i + 2]);
          acc[i + 3] = fmaf(wt, wt * v.w, acc[i + 3]);
        }
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const int i = (pc.row0 + r) / g.G, hq = pc.hk * g.G + pc.row0 + r - i * g.G;
      const size_t own = static_cast<size_t>(pc.s + i) * g.H + hq;
      float* dst = (pc.slot >= 0 ? g.partial + (static_cast<size_t>(pc.slot) * R + r) * DIM
                                 : g.rows[pc.side] + own * DIM) + d0;
#pragma unroll
      for (int e = 0; e < kMine; e += 4) {
        float4 v = make_float4(acc[e] * inv, acc[e + 1] * inv, acc[e + 2] * inv, acc[e + 3] * inv);
        if (inv == 0.f) v = make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(dst + e) = v;
      }
      if (d0 == 0) {
        const float st = base + log2f(sum);
        if (pc.slot >= 0)
          g.stats[static_cast<size_t>(pc.slot) * R + r] = st;
        else
          g.row_stats[pc.side][own] = st;
        if (pc.parts != 0)
          g.where[pc.side][own] = RowParts{static_cast<int>(blockIdx.x) | (r << 16), pc.parts};
      }
    }
    __syncthreads();
  }
}

template <int DIM, int MT, int KEYS>
bool launch(const flamia_kvcache* c, const AttendArgs& g, cudaStream_t s) {
  constexpr int smem = static_cast<int>(sizeof(Smem<DIM, MT>)) + 128;
  static_assert(Few<DIM, MT>::kCtas * (smem + 1024) <= 228 * 1024, "shared memory");
  static std::atomic<unsigned long long> raised{0};
  return launch_large(attend_prefix_few_kernel<DIM, MT, KEYS>, raised,
                      dim3(min(kMaxCtas, num_sms() * Few<DIM, MT>::kCtas)), kThreads, smem, s, g,
                      static_cast<const uint8_t*>(c->k_codes),
                      static_cast<const uint8_t*>(c->v_codes));
}

template <int KEYS>
bool launch(const flamia_kvcache* c, const AttendArgs& g, int R, cudaStream_t s) {
  if (c->d == 128) return launch<128, 1, KEYS>(c, g, s);
  return R == 16 ? launch<64, 1, KEYS>(c, g, s) : launch<64, 2, KEYS>(c, g, s);
}

}  // namespace

flamia_status attend_prefix_few(const flamia_kvcache* c, const AttendArgs& g, int R, Keys keys,
                                cudaStream_t s) {
  return (keys == kBoth ? launch<kBoth>(c, g, R, s) : launch<kRest>(c, g, R, s)) ? FLAMIA_OK
                                                                                : FLAMIA_ERR_CUDA;
}

}  // namespace flamia
