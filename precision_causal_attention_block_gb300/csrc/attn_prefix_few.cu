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

template <int DIM, int MT>
struct Smem {
  using C = Few<DIM, MT>;
  alignas(128) uint8_t ring[kWarps][C::kRing];
  float lg[kWarps][C::kRows];
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

// N bytes (8 or 16) from global to shared memory; zeros if there is nothing to read.
template <int N>
__device__ __forceinline__ void fetch(uint32_t dst, const void* src, bool there) {
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

// What the warps of a CTA work on: an item's key tiles i0 .. i1 - 1 (list positions; key tile
// i + wt), of keys below hi.
struct Piece {
  int s, n, start, hk, row0, i0, i1, wt, hi, seq;
  bool over, sharing, cut;  // of the prefix; its sequence shares it; parts elsewhere
  long long at;             // the item's first unit
};

// The CTA's run, walked by all warps alike.
template <int R, int KEYS>
struct Run {
  SeqWork w;
  long long u, u1, total;
  int v, hk = 0, rt = 0, o = 0, sharer;

  template <class Sm>
  __device__ __forceinline__ explicit Run(const Sm& sm)
      : w{}, u(sm.plan_u0), u1(sm.plan_u1), total(sm.plan_total), v(sm.plan_b), sharer(sm.sharer) {
    if (u < u1) {
      w = sm.plan_seq;
      const long long item = mul_div(sm.plan_off, 1, w.units);
      o = static_cast<int>(sm.plan_off - item * w.units);
      hk = static_cast<int>(mul_div(item, 1, w.row_tiles));
      rt = static_cast<int>(item - static_cast<long long>(hk) * w.row_tiles);
    }
  }
  __device__ __forceinline__ bool next(const AttendArgs& g, Piece& p) {
    while (u < u1) {
      constexpr int kCost = kItemCost<R, KEYS>;
      const int take = static_cast<int>(min(u1 - u, static_cast<long long>(w.units - o)));
      const int i0 = g.whole ? 0 : max(o - kCost, 0);
      const int i1 = g.whole ? w.tiles : max(o + take - kCost, 0);
      p.s = w.s;
      p.n = w.n;
      p.start = w.start;
      p.hk = hk;
      p.row0 = rt * R;
      p.over = of_prefix<KEYS>(v);
      p.sharing = !p.over && shares(g, w.start);
      p.seq = p.over ? sharer : seq_of<KEYS>(v);
      p.wt = p.sharing ? g.shared : 0;
      // behind the last key that its last row sees
      const int rows = static_cast<int>(min(static_cast<long long>(w.n) * g.G - p.row0,
                                            static_cast<long long>(R)));
      p.hi = p.over ? g.shared * 128
                    : max(w.start + static_cast<int>(static_cast<unsigned>(p.row0 + rows - 1) /
                                                     static_cast<unsigned>(g.G)) + 1, 0);
      p.i0 = i0;
      p.i1 = i1;
      p.cut = i0 > 0 || i1 < w.tiles;
      p.at = u - o;
      if (!p.over && hk == 0 && rt == 0 && i0 == 0 && threadIdx.x == 0) {
        const int raw = g.starts != nullptr ? g.starts[p.seq] : 0;
        if (raw > g.cap - w.n) report(g.status, FLAMIA_DEV_BAD_PAGE);
      }
      const int units = w.units;
      u += take;
      o = 0;
      parts = 1;
      if (p.cut && i0 == 0) parts = parts_from_here<R, KEYS>(g, p.at, units, total);
      if (u < u1 && ++rt == w.row_tiles) {
        rt = 0;
        if (++hk == g.H_kv) {
          hk = 0;
          do {
            w = seq_work<R, KEYS>(g, ++v, sharer);  // there is one: u < u1
          } while (w.row_tiles == 0 && seq_of<KEYS>(v) + 1 < g.ndocs);
        }
      }
      if (i1 > i0) return true;  // (else the run ends before the item's first tile)
    }
    return false;
  }
  int parts = 1;  // of the last piece's item, if it holds the first
};

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
  Run<R, KEYS> run(sm);
  Piece pc;
  const uint32_t ring = smem_u32(sm.ring[warp]);

  while (run.next(g, pc)) {
    // ------------------------------------------------------------- keys
    const int k_lo = (pc.i0 + pc.wt) * 128, k_hi = min((pc.i1 + pc.wt) * 128, pc.hi);
    const int blocks = (max(k_hi - k_lo, 0) + 31) / 32;
    const int mine = (blocks - warp + kWarps - 1) / kWarps;  // this warp's (0 or less: none)
    const int32_t* table = g.table + static_cast<long long>(pc.seq) * g.table_stride;
    int rows32 = -1;  // first rows of its next 32 blocks (a lane each) / 32; -1: no page
    auto key_of = [&](int m) { return k_lo + (warp + m * kWarps) * 32; };
    auto issue = [&](int m) {
      if (m < mine) {
        if ((m & 31) == 0) {
          const int key0 = key_of(m + lane), slot = key0 / g.page_size;
          const bool need = m + lane < mine;
          const int page = need && slot < g.table_stride ? table[slot] : -1;
          const bool there = page >= 0 && page < g.num_pages;
          if (need && !there) report(g.status, FLAMIA_DEV_BAD_PAGE);
          rows32 = there ? (page * g.H_kv + pc.hk) * (g.page_size / 32) +
                               (key0 - slot * g.page_size) / 32
                         : -1;
        }
        const int row = __shfl_sync(0xffffffffu, rows32, m & 31);
        const long long base = static_cast<long long>(max(row, 0)) * 32;
        const int n = row < 0 ? 0 : k_hi - key_of(m);  // keys that are there (32 or more: all)
        const uint32_t st = ring + (m % C::kStages) * C::kStage;
        const uint8_t* kc = k_codes + base * DIM + t * (DIM / 4);
        const uint8_t* vc = v_codes + base * DIM + gr * (DIM / 8);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int p = 0; p < DIM / 64; ++p)
            fetch<16>(st + (j * (DIM / 64) + p) * 512 + lane * 16, kc + (j * 8 + gr) * DIM + p * 16,
                      j * 8 + gr < n);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int key = (j >> 2) * 16 + ((j >> 1) & 1) * 8 + 2 * t + (j & 1);
          fetch<DIM / 8>(st + C::kKBytes + j * (4 * DIM) + lane * (DIM / 8), vc + key * DIM, key < n);
        }
        if (lane == 0)
          *reinterpret_cast<int*>(sm.ring[warp] + (m % C::kStages) * C::kStage + 2 * C::kKBytes + 64) =
              row >= 0;
        if (lane < 4)
          fetch<16>(st + 2 * C::kKBytes + lane * 16,
                    (lane < 2 ? g.k_scales : g.v_scales) + base + (lane & 1) * 16, n > 0);
      }
      fetch_commit();
    };
#pragma unroll
    for (int m = 0; m < C::kStages; ++m) issue(m);

    // ------------------------------------------------------------- queries
    const int rows =
        static_cast<int>(min(static_cast<long long>(R), static_cast<long long>(pc.n) * g.G - pc.row0));
    uint32_t q[MT][KS][4];
    float qf[MT][2];
    int pos[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = mt * 16 + half * 8 + gr;
        const int i = (pc.row0 + r) / g.G, h = pc.hk * g.G + pc.row0 + r - i * g.G;
        pos[mt][half] = r < rows ? max(pc.start + i, -1) : -1;
        const __nv_bfloat16* src =
            g.q + (pc.s + i) * g.q_stride + static_cast<long long>(h) * DIM + t * (DIM / 4);
        uint4 x[DIM / 32];
        uint32_t a = 0;
#pragma unroll
        for (int p = 0; p < DIM / 32; ++p) {
          x[p] = make_uint4(0, 0, 0, 0);
          if (r < rows) x[p] = reinterpret_cast<const uint4*>(src)[p];
        }
        // magnitudes as integers; 0x7F80 and above: infinities and NaN, which become NaN
        // and stay out of the maximum
#pragma unroll
        for (int p = 0; p < DIM / 32; ++p)
          a = __vmaxu2(a, __vmaxu2(__vmaxu2(x[p].x & 0x7FFF7FFFu, x[p].y & 0x7FFF7FFFu),
                                   __vmaxu2(x[p].z & 0x7FFF7FFFu, x[p].w & 0x7FFF7FFFu)));
        a = max(a & 0xFFFFu, a >> 16);
        if (a >= 0x7F80u) {
          a = 0;
#pragma unroll
          for (int p = 0; p < DIM / 32; ++p) {
            uint32_t* w = &x[p].x;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t y = e == 0 ? x[p].x : e == 1 ? x[p].y : e == 2 ? x[p].z : x[p].w;
              if ((y & 0x7F80u) == 0x7F80u)
                y = (y & 0xFFFF0000u) | 0x7FC0u;
              else
                a = max(a, y & 0x7FFFu);
              if ((y & 0x7F800000u) == 0x7F800000u)
                y = (y & 0xFFFFu) | 0x7FC00000u;
              else
                a = max(a, (y >> 16) & 0x7FFFu);
              w[e] = y;
            }
          }
        }
        a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
        a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
        const int ex = roundup_exponent(__uint_as_float(a << 16));
        const float2 inv = make_float2(exp2i(-ex), exp2i(-ex));
        qf[mt][half] = g.scale_log2 * (ex < -126 ? 0x1p-127f : exp2i(ex));
        auto half2 = [&](uint32_t w) {
          return half2_of(__fmul2_rn(
              make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)), inv));
        };
#pragma unroll
        for (int p = 0; p < DIM / 32; ++p) {
          q[mt][2 * p][half] = half2(x[p].x);
          q[mt][2 * p][2 + half] = half2(x[p].y);
          q[mt][2 * p + 1][half] = half2(x[p].z);
          q[mt][2 * p + 1][2 + half] = half2(x[p].w);
        }
      }
    }
    // the first row's position: blocks up to it are seen by all rows
    const int pf = pc.start + static_cast<int>(static_cast<unsigned>(pc.row0) /
                                               static_cast<unsigned>(g.G));

    float o[MT][C::kOut][4];
    float l[MT][2], nref[MT][2];
    Sum past[MT][2];
    bool has[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int i = 0; i < C::kOut; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][i][e] = 0.f;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        l[mt][half] = nref[mt][half] = 0.f;
        past[mt][half] = Sum{0.f, kNoExponent};
        has[mt][half] = false;
      }
    }
    int e0 = -127;
    bool large = false, begun = false;

    // ------------------------------------------------------------- blocks
#pragma unroll 1
    for (int m = 0; m < mine; ++m) {
      fetch_wait<C::kStages - 1>();
      __syncwarp();
      const uint8_t* st = sm.ring[warp] + (m % C::kStages) * C::kStage;
      const int key0 = key_of(m);
      const bool there = *reinterpret_cast<const int*>(st + 2 * C::kKBytes + 64) != 0;
      // scores
      float s[MT][4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t kw[KS];
#pragma unroll
        for (int p = 0; p < DIM / 64; ++p) {
          const uint4 x =
              *reinterpret_cast<const uint4*>(st + (j * (DIM / 64) + p) * 512 + lane * 16);
          kw[4 * p] = x.x, kw[4 * p + 1] = x.y, kw[4 * p + 2] = x.z, kw[4 * p + 3] = x.w;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][j][e] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const uint32_t b0 = half2_of_codes(kw[k] & 0xFFFFu), b1 = half2_of_codes(kw[k] >> 16);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) mma16816(s[mt][j], q[mt][k], b0, b1);
        }
      }
      // exponents: one of K and one of V for all 32 keys, or each key's
      const uint8_t* ksc = st + 2 * C::kKBytes;
      const uint8_t* vsc = ksc + 32;
      const bool all = there && key0 + 32 <= k_hi;         // every key is there
      const bool every = all && (pc.over || key0 + 31 <= pf);  // and every row sees it
      const int kb = ksc[lane], vb = vsc[lane];
      const int kb0 = __shfl_sync(0xffffffffu, kb, 0), vb0 = __shfl_sync(0xffffffffu, vb, 0);
      const bool uniform = __all_sync(0xffffffffu, kb == kb0 && vb == vb0) && all;
      uint32_t nan = 0;  // of this lane's keys: half seen, with a NaN in V
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
      // Of keys that some row sees: the largest and the smallest eV.
      int top = vb0 - 127, low = vb0 - 127;
      if (!uniform) {
        const bool live = there && key0 + lane < k_hi;
        top = __reduce_max_sync(0xffffffffu, live ? vb - 127 : -127);
        low = __reduce_min_sync(0xffffffffu, live ? vb - 127 : 128);
      }
      if (!begun) {
        e0 = top;
        begun = true;
      } else if (top > e0 + kHigh) {  // (as in attn_cache.cu)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            past[mt][half].add(l[mt][half], -static_cast<float>(e0));
            l[mt][half] = 0.f;
          }
        e0 = top;
      }
      const bool apart = low < e0 - kLow;  // some keys are not in l
      // y = x + eV - ref
      int ev[4][2];
      if (uniform) {
        const float kf = pow2_byte(kb0), evf = static_cast<float>(vb0 - 127);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const float f0 = kf * qf[mt][0], f1 = kf * qf[mt][1];
          const float a0 = evf + nref[mt][0], a1 = evf + nref[mt][1];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[mt][j][0] = fmaf(s[mt][j][0], f0, a0);
            s[mt][j][1] = fmaf(s[mt][j][1], f0, a0);
            s[mt][j][2] = fmaf(s[mt][j][2], f1, a1);
            s[mt][j][3] = fmaf(s[mt][j][3], f1, a1);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = j * 8 + 2 * t + e;
            const float kf = pow2_byte(ksc[key]);
            ev[j][e] = vsc[key] - 127;
            const float evf = static_cast<float>(ev[j][e]);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                float& y = s[mt][j][2 * half + e];
                y = fmaf(y, kf * qf[mt][half], evf + nref[mt][half]);
              }
          }
      }
      if (!every) {
        // (key j * 8 + 2 t + e is V's number (j >> 1) * 4 + (j & 1) * 2 + e of this lane)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = key0 + j * 8 + 2 * t + e;
            const bool bad = (nan >> (j * 2 + e)) & 1;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                float& y = s[mt][j][2 * half + e];
                const bool seen = there && key < k_hi && (pc.over || key <= pos[mt][half]);
                y = !seen ? -INFINITY : bad ? __uint_as_float(0x7FC00000u) : y;
              }
          }
      }
      // Do the references hold?
      bool need = false;
      float mx[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int c = 2 * half;
          mx[mt][half] =
              fmaxf(fmax3(fmax3(s[mt][0][c], s[mt][0][c + 1], s[mt][1][c]), s[mt][1][c + 1],
                          s[mt][2][c]),
                    fmax3(s[mt][2][c + 1], s[mt][3][c], s[mt][3][c + 1]));
          need |= has[mt][half] ? mx[mt][half] > kSlack + room(nref[mt][half])
                                : mx[mt][half] > -INFINITY;
        }
      if (__any_sync(0xffffffffu, need)) {
        large = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float x = mx[mt][half];  // the row's, over its four lanes
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            float& ref = nref[mt][half];
            const bool moves = has[mt][half] ? x > kSlack + room(ref) : x > -INFINITY;
            if (moves) {
              const float by = lowered(ref - ceilf(x)) - ref;
              const float f = has[mt][half] ? ex2_approx(by) : 1.f;
              l[mt][half] *= f;
              ref += by;
              past[mt][half].e += by;
              has[mt][half] = true;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                s[mt][j][2 * half] += by;
                s[mt][j][2 * half + 1] += by;
              }
#pragma unroll
              for (int i = 0; i < C::kOut; ++i) {
                o[mt][i][2 * half] *= f;
                o[mt][i][2 * half + 1] *= f;
              }
            }
            large |= fabsf(ref) > kLarge;
          }
        large = __any_sync(0xffffffffu, large);
      }
      if (apart) {  // keys that l does not hold: sum 2^(x + nref)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float x[8], most = kNoExponent, sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int v = uniform ? vb0 - 127 : ev[i / 2][i & 1];
              x[i] = v < e0 - kLow ? s[mt][i / 2][2 * half + (i & 1)] - static_cast<float>(v)
                                   : -INFINITY;
              most = fmaxf(most, x[i]);
            }
            most = ceilf(most);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += ex2_approx(x[i] - most);
            past[mt][half].add(sum, most);
          }
      }
      // weights
      uint32_t p[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if (large) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][j][e] = cut(s[mt][j][e], kSlack);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][j][e] = ex2_approx(s[mt][j][e]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int c = 2 * half;
          if (uniform) {
            const float a = ((s[mt][0][c] + s[mt][0][c + 1]) + (s[mt][1][c] + s[mt][1][c + 1])) +
                            ((s[mt][2][c] + s[mt][2][c + 1]) + (s[mt][3][c] + s[mt][3][c + 1]));
            l[mt][half] = fmaf(a, apart ? 0.f : exp2i(e0 - (vb0 - 127)), l[mt][half]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (ev[j][e] >= e0 - kLow && ev[j][e] <= e0 + kHigh)  // (else unseen, or apart)
                  l[mt][half] = fmaf(s[mt][j][c + e], exp2i(e0 - ev[j][e]), l[mt][half]);
          }
        }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          p[mt][kk][0] = half2_of(make_float2(s[mt][2 * kk][0], s[mt][2 * kk][1]));
          p[mt][kk][1] = half2_of(make_float2(s[mt][2 * kk][2], s[mt][2 * kk][3]));
          p[mt][kk][2] = half2_of(make_float2(s[mt][2 * kk + 1][0], s[mt][2 * kk + 1][1]));
          p[mt][kk][3] = half2_of(make_float2(s[mt][2 * kk + 1][2], s[mt][2 * kk + 1][3]));
        }
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
          if ((nan >> (kk * 4 + j)) & 1) {
#pragma unroll
            for (int w = 0; w < DIM / 32; ++w) v[j][w] = 0;
          }
        }
#pragma unroll
        for (int w = 0; w < DIM / 32; ++w) {
          const uint32_t a0 = __byte_perm(v[0][w], v[1][w], 0x5140);
          const uint32_t a1 = __byte_perm(v[0][w], v[1][w], 0x7362);
          const uint32_t c0 = __byte_perm(v[2][w], v[3][w], 0x5140);
          const uint32_t c1 = __byte_perm(v[2][w], v[3][w], 0x7362);
          const uint32_t b[4][2] = {
              {half2_of_codes(a0 & 0xFFFFu), half2_of_codes(c0 & 0xFFFFu)},
              {half2_of_codes(a0 >> 16), half2_of_codes(c0 >> 16)},
              {half2_of_codes(a1 & 0xFFFFu), half2_of_codes(c1 & 0xFFFFu)},
              {half2_of_codes(a1 >> 16), half2_of_codes(c1 >> 16)}};
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
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        Sum all = past[mt][half];
        all.add(l[mt][half], -static_cast<float>(e0));
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
          const float a = __shfl_xor_sync(0xffffffffu, all.m, off);
          const float b = __shfl_xor_sync(0xffffffffu, all.e, off);
          all.add(a, b);
        }
        const int r = mt * 16 + half * 8 + gr;
        const float lg = all.m == 0.f ? -INFINITY : log2f(all.m) + all.e - nref[mt][half];
        const int k = static_cast<int>(-all.e);
        const float inv = all.m == 0.f ? 0.f : pow2_within(k / 2) / all.m;
        const float ve = pow2_within(k - k / 2);
        if (t == 0) sm.lg[warp][r] = lg;
        // dims t (d / 4) + i, then + d / 8: column tile i's two columns of this lane
#pragma unroll
        for (int i = 0; i < C::kOut; i += 4)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float4 x;
            x.x = o[mt][i][2 * half + e] * inv * ve;
            x.y = o[mt][i + 1][2 * half + e] * inv * ve;
            x.z = o[mt][i + 2][2 * half + e] * inv * ve;
            x.w = o[mt][i + 3][2 * half + e] * inv * ve;
            if (inv == 0.f) x = make_float4(0.f, 0.f, 0.f, 0.f);
            const int chunk = (t * (DIM / 4) + e * (DIM / 8) + i) / 4;
            *reinterpret_cast<float4*>(out + r * DIM + (chunk ^ (r & 7)) * 4) = x;
          }
      }
    __syncthreads();
    // the four warps' joined: kThreads / R threads a row
    constexpr int kPer = kThreads / R, kMine = DIM / kPer;  // threads a row, dims a thread
    const int r = tid / kPer, d0 = tid % kPer * kMine;
    if (r < rows) {
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
      const int side = pc.over ? 0 : 1, slot = 2 * blockIdx.x + (pc.i0 == 0);
      float* dst = (pc.cut ? g.partial + (static_cast<size_t>(slot) * R + r) * DIM
                           : g.rows[side] + own * DIM) + d0;
#pragma unroll
      for (int e = 0; e < kMine; e += 4) {
        float4 v = make_float4(acc[e] * inv, acc[e + 1] * inv, acc[e + 2] * inv, acc[e + 3] * inv);
        if (inv == 0.f) v = make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(dst + e) = v;
      }
      if (d0 == 0) {
        const float st = base + log2f(sum);
        if (pc.cut)
          g.stats[static_cast<size_t>(slot) * R + r] = st;
        else
          g.row_stats[side][own] = st;
        if (pc.i0 == 0)
          g.where[side][own] = RowParts{static_cast<int>(blockIdx.x) | (r << 16),
                                        run.parts | (pc.sharing ? kShares : 0)};
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
