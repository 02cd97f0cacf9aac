// Attention of new tokens over the paged MXFP8 cache.
//
// The product is turned around so that the cache fills the tensor core's M:
// per 128-key tile S^T = K Q^T (M = 128 keys) and O^T += V^T P^T (M = d), with
// the few query rows of one K / V head (group x new tokens, R of them) as N.  K
// and V go from HBM to the tensor core by TMA as the E4M3 codes that the cache
// holds, V read MN-major, so nothing converts or transposes them; BF16 queries
// and float32 weights become sums of E4M3 terms instead, side by side in N:
//   q 2^-e = h + 2^-4 l            (e per row; exact for the elements above
//                                   2^-14 of the row's largest),
//   w = 2^-4 (h + 2^-5 m + 2^-10 l)  (relative error 2^-14, floor 2^-24 of the
//                                   largest weight),
// which costs N = 2 R and 3 R columns of a product that reads M = 128 rows of
// shared memory in any case.
//
// The key factor 2^eK multiplies the score, V's 2^eV goes into the weight: the
// thread that owns a key adds eV to its score.  The softmax keeps two running
// references a row, of the scores (for the sum l) and of score + eV (for the
// weights), so that values of very different exponents, and zero values under
// a heavy first token, keep their precision.  References move only when a tile
// exceeds them by more than their slack (kSlackW, kSlackM), which the one
// barrier of a tile votes on; then O^T is rescaled in tensor memory.
//
// Work: all (sequence, K / V head, row tile) items' key tiles are laid end to
// end and cut into equal runs, one for each resident CTA, so that a batch of
// ragged lengths keeps every SM reading until the end.  A CTA finishes the
// items that lie whole inside its run; of the (at most two) it shares it
// leaves (m, l, O) in the workspace, and a second small kernel, launched
// with programmatic dependent launch, joins them in order of position (no
// atomics: results do not depend on timing).
//
// Warps 0-3: softmax (thread = key = TMEM lane); 4: TMA producer; 5: MMA issuer.
#include <cuda_bf16.h>

#include <cmath>

#include "paged.cuh"

namespace flamia {
namespace {

constexpr int kThreads = 192;
constexpr int kMaxCtas = 512;   // runs of a launch (the workspace is sized for it)
constexpr int kSegSlots = 4;
constexpr int kMaxPos = 1 << 30;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kUnset = -1e30f;   // reference of a row that has seen no key
constexpr float kSlackM = 60.f;    // l <= 2^60 x keys: far inside float32
constexpr float kSlackW = 4.f;     // weights <= 2^(kShiftW + 4) = 256 < 448
constexpr float kShiftW = 4.f;
// parameters of the partial results: [slot][R] {m, l, w, -}, then [slot][R][d]
constexpr int kSlots = 2 * kMaxCtas;

struct AttendArgs {
  const uint8_t *k_scales, *v_scales;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  const int32_t *cu, *starts, *table;
  int4* joins;       // [kMaxCtas][2]: items to join
  float4* stats;     // [kSlots][R]
  float* partial;    // [kSlots][R][d]
  int* status;
  long long q_stride;
  int T, H, H_kv, G, ndocs, table_stride, num_pages, page_size, window, sinks;
  float scale_log2;
};

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

// Barrier of the softmax warps that also ORs a predicate over them.
__device__ __forceinline__ bool softmax_vote(bool p) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<int>(p))
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void softmax_sync() { named_barrier_sync(1, 128); }

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void sts8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ float pow2_byte(int byte) {
  return byte > 0 ? __uint_as_float(static_cast<uint32_t>(byte) << 23) : 0x1p-127f;
}

// ------------------------------------------------------------------ work

// Sequence b's share of the work: row tiles x K / V heads x key tiles (an upper
// bound of the tiles of its row tiles: a segment that runs past its item's last
// tile is cut there).
struct SeqWork {
  int s, n, start;     // packed rows [s, s + n) at positions start ..
  int row_tiles, tiles;
  __device__ __forceinline__ long long units(int H_kv) const {
    return static_cast<long long>(row_tiles) * tiles * H_kv;
  }
};

template <int R>
__device__ __forceinline__ SeqWork seq_work(const AttendArgs& g, int b) {
  SeqWork w;
  const DocRange r = doc_range(g.cu, b, g.T);
  w.s = r.s;
  w.n = r.e - r.s;
  w.start = g.starts != nullptr ? __ldg(g.starts + b) : 0;
  if (w.start > kMaxPos - w.n) w.start = -w.n;  // reported by the producer
  w.start = max(w.start, -kMaxPos);
  w.row_tiles = static_cast<int>((static_cast<long long>(w.n) * g.G + R - 1) / R);
  const int end = max(w.start + w.n, 0);
  int tiles = (end + 127) >> 7;
  if (g.window > 0)
    tiles = min(tiles, ((min(g.sinks, end) + 127) >> 7) +
                           ((min(g.window, end) + R / g.G + 1 + 127) >> 7) + 1);
  w.tiles = max(tiles, 1);
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

// ------------------------------------------------------------------ kernel

template <int DIM, int R>
struct Cfg {
  static constexpr int kCtas = R == 8 ? 3 : 2;  // resident CTAs per SM
  static constexpr int kStages = (R == 16 ? 3 : 2) * (128 / DIM);
  static constexpr int kTileBytes = 128 * DIM;
  static constexpr int kNS = 2 * R;                 // columns of S^T
  static constexpr int kNO = (3 * R + 15) / 16 * 16;  // columns of O^T
  static constexpr uint32_t kColO = 2 * kNS;
  static constexpr uint32_t kCols = R == 8 ? 64 : R == 16 ? 128 : 256;
  static_assert(kColO + kNO <= kCols, "tensor memory");
};

template <int DIM, int R>
struct Smem {
  using C = Cfg<DIM, R>;
  // The last P^T rows of a product with R = 8 (columns 24 .. 31, ignored) read
  // on into the bytes behind p.
  alignas(1024) uint8_t v[C::kStages][C::kTileBytes];
  alignas(1024) uint8_t k[C::kStages][C::kTileBytes];
  alignas(1024) uint8_t p[2][3 * R * 128];
  alignas(1024) uint8_t q[2 * R * DIM];
  alignas(128) uint8_t ks[C::kStages][128];
  alignas(128) uint8_t vs[C::kStages][128];
  alignas(16) float qf[R];      // 2^e of a row x softmax scale x log2 e
  alignas(16) float ref_m[R], ref_w[R], f_m[R], f_w[R];
  alignas(16) int pos[R];       // position of a row's token, -1: no such row
  alignas(16) int orow[R];      // its row of o, -1: none
  float red[4][R][2];
  uint64_t full[C::kStages], empty[C::kStages];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t q_full, o_empty;
  uint64_t seg_full[kSegSlots], seg_empty[kSegSlots];
  Segment seg[kSegSlots];
  int loaded[C::kStages];       // pieces of the tile that were loaded
  int plan_b;
  long long plan_off, plan_u0, plan_u1, plan_total;
  long long scan[kThreads / 32];
  uint32_t tmem_base;
  int stop[2];                  // softmax warps: a wait ran out (by tile parity)
  volatile int abort;
};

// CTAs that get a run: at least two tiles each, as far as there are any.
__device__ __forceinline__ long long active_ctas(long long total) {
  return min(static_cast<long long>(gridDim.x), (total + 1) / 2);
}

// Total units, and this CTA's run of them: [u0, u1), starting at unit `off` of
// sequence b.  Every thread sums a stretch of sequences; the one whose stretch
// holds u0 walks it.
template <int R, class Sm>
__device__ __forceinline__ void make_plan(const AttendArgs& g, Sm& sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = (g.ndocs + kThreads - 1) / kThreads;
  const int b0 = min(tid * each, g.ndocs), b1 = min(b0 + each, g.ndocs);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) sum += seq_work<R>(g, b).units(g.H_kv);
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
  const long long ctas = active_ctas(total);
  const long long c = blockIdx.x;
  const long long u0 = c < ctas ? total * c / ctas : total;
  const long long u1 = c < ctas ? total * (c + 1) / ctas : total;
  if (tid == 0) {
    sm.plan_u0 = u0;
    sm.plan_u1 = u1;
    sm.plan_total = total;
  }
  if (u0 < u1 && before <= u0 && u0 < before + sum) {
    long long off = u0 - before;
    int b = b0;
    for (; b < b1 - 1; ++b) {
      const long long u = seq_work<R>(g, b).units(g.H_kv);
      if (off < u) break;
      off -= u;
    }
    sm.plan_b = b;
    sm.plan_off = off;
  }
  __syncthreads();
}

template <int DIM, int R>
__global__ void __launch_bounds__(kThreads, Cfg<DIM, R>::kCtas)
    attend_kernel(const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const AttendArgs g) {
  using C = Cfg<DIM, R>;
  extern __shared__ uint8_t smem_raw[];
  Smem<DIM, R>& sm = *reinterpret_cast<Smem<DIM, R>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(smem_u32(&sm.full[i]), 1);
      mbar_init(smem_u32(&sm.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.s_full[i]), 1);
      mbar_init(smem_u32(&sm.p_full[i]), 128);
      mbar_init(smem_u32(&sm.pv_done[i]), 1);
      sm.stop[i] = 0;
    }
    mbar_init(smem_u32(&sm.q_full), 128);
    mbar_init(smem_u32(&sm.o_empty), 128);
    for (int i = 0; i < kSegSlots; ++i) {
      mbar_init(smem_u32(&sm.seg_full[i]), 1);
      mbar_init(smem_u32(&sm.seg_empty[i]), 5);  // four softmax warps, the MMA issuer
    }
    sm.abort = 0;
    fence_barrier_init();
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(&sm.tmem_base), C::kCols);
    tmem_relinquish();
  }
  check_offsets(g.cu, g.ndocs, g.T, static_cast<long long>(blockIdx.x) * kThreads + tid,
                static_cast<long long>(gridDim.x) * kThreads, g.status);
  tc_fence_before();
  make_plan<R>(g, sm);
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  if (warp == 4) {
    // ------------------------------------------------------------ producer
    const long long u0 = sm.plan_u0, u1 = sm.plan_u1, total = sm.plan_total;
    const int pieces = g.page_size >= 128 ? 1 : 128 / g.page_size;
    const int piece = 128 / pieces;  // keys
    if (lane == 0) {
      prefetch_tensormap(&map_k);
      prefetch_tensormap(&map_v);
    }
    int b = sm.plan_b, tc = 0, nseg = 0;
    long long off = sm.plan_off, u = u0;
    bool ok = true, first = true;
    int4 join0 = make_int4(0, 0, 0, 0), join1 = make_int4(0, 0, 0, 0);
    while (ok) {
      Segment sg{};
      int hi = 0, wlo = 0;
      if (u >= u1 || b >= g.ndocs) {
        sg.s = -1;
      } else {
        const SeqWork w = seq_work<R>(g, b);
        if (off >= w.units(g.H_kv)) {  // the next sequence
          off = 0;
          ++b;
          continue;
        }
        const int i = static_cast<int>(off % w.tiles);
        const long long item = off / w.tiles;
        sg.s = w.s;
        sg.n = w.n;
        sg.start = w.start;
        sg.hk = static_cast<int>(item / w.row_tiles);
        sg.row0 = static_cast<int>(item % w.row_tiles) * R;
        const long long left = u1 - u;
        const int take = static_cast<int>(min(left, static_cast<long long>(w.tiles - i)));
        // positions of the row tile's first and last token
        const int pf = w.start + sg.row0 / g.G;
        const int pl = w.start + static_cast<int>(min(static_cast<long long>(w.n) * g.G - 1,
                                                      static_cast<long long>(sg.row0) + R - 1) /
                                                  g.G);
        hi = max(pl + 1, 0);
        wlo = g.window > 0 ? max(pf - g.window + 1, 0) : 0;
        sg.wt = wlo >> 7;
        sg.ns = min((g.sinks + 127) >> 7, sg.wt);
        const int list = sg.ns + max(((hi + 127) >> 7) - sg.wt, 0);
        sg.i0 = min(i, list);
        sg.i1 = min(i + take, list);
        sg.slot = -1;
        if (i > 0)
          sg.slot = 2 * blockIdx.x;
        else if (take < w.tiles)
          sg.slot = 2 * blockIdx.x + 1;
        if (first && i > 0) {
          // the second CTA of an item's run has it joined: parts are the
          // CTA before this one (slot 1) and slots 0 from here on
          const long long ctas = active_ctas(total);
          const long long c = blockIdx.x, ui = u0 - i;
          if (c > 0 && total * (c - 1) / ctas <= ui) {
            const long long last = ((ui + w.tiles) * ctas + total - 1) / total - 1;
            join0 = make_int4(static_cast<int>(last - c + 2), w.s, w.n, sg.hk);
            join1 = make_int4(sg.row0, 0, 0, 0);
          }
        }
        first = false;
        if (lane == 0 && i == 0 && sg.hk == 0 && sg.row0 == 0) {
          const int raw = g.starts != nullptr ? __ldg(g.starts + b) : 0;
          if (raw > kMaxPos - w.n) report(g.status, FLAMIA_DEV_BAD_PAGE);
        }
        off += take;
        u += take;
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
      const int32_t* row = g.table + static_cast<long long>(b) * g.table_stride;
      auto entry = [&](int i, bool& need, int& in_page) {
        const int kp = tile_of(sg, i) * 128 + lane * piece;
        need = lane < pieces && kp < hi &&
               (g.window == 0 || kp + piece > wlo || kp < g.sinks);
        const int slot = kp / g.page_size;
        in_page = kp - slot * g.page_size;
        return need && slot < g.table_stride ? __ldg(row + slot) : -1;
      };
      bool need;
      int in_page;
      int page = sg.i0 < sg.i1 ? entry(sg.i0, need, in_page) : -1;
      for (int i = sg.i0; i < sg.i1; ++i, ++tc) {
        const int pg = page, ip = in_page;
        const bool nd = need, good = nd && pg >= 0 && pg < g.num_pages;
        if (i + 1 < sg.i1) page = entry(i + 1, need, in_page);
        if (nd && !good) report(g.status, FLAMIA_DEV_BAD_PAGE);
        const unsigned mask = __ballot_sync(0xffffffffu, good);
        const int st = tc % C::kStages;
        if (tc >= C::kStages)
          ok = mbar_wait_w_ab(smem_u32(&sm.empty[st]), ((tc / C::kStages) - 1) & 1, &sm.abort);
        if (!ok) break;
        const uint32_t bar = smem_u32(&sm.full[st]);
        if (lane == 0) {
          sm.loaded[st] = static_cast<int>(mask);
          mbar_arrive_expect_tx(bar, __popc(mask) * (2 * piece * DIM + 2 * piece));
        }
        __syncwarp();
        if (good) {
          const int pr = lane * piece;  // first key of the piece inside the tile
          const int prow = pg * g.H_kv + sg.hk;
          const long long sc = static_cast<long long>(prow) * g.page_size + ip;
          tma_load_3d(smem_u32(sm.k[st]) + pr * DIM, &map_k, bar, 0, ip, prow);
          bulk_load(smem_u32(sm.ks[st]) + pr, g.k_scales + sc, piece, bar);
          tma_load_3d(smem_u32(sm.v[st]) + pr * DIM, &map_v, bar, 0, ip, prow);
          bulk_load(smem_u32(sm.vs[st]) + pr, g.v_scales + sc, piece, bar);
        }
        __syncwarp();
      }
    }
    // what the second kernel has to join for this CTA's first item
    if (lane == 0) {
      g.joins[2 * blockIdx.x] = join0;
      g.joins[2 * blockIdx.x + 1] = join1;
    }
    // every issued copy has landed before the CTA can exit
    for (int j = max(0, tc - C::kStages); j < tc; ++j)
      ok &= mbar_wait_w(smem_u32(&sm.full[j % C::kStages]), (j / C::kStages) & 1);
    if (!ok) sm.abort = 1;
  } else if (warp == 5) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t lay = DIM == 128 ? kLayoutSW128 : kLayoutSW64;
    constexpr uint32_t sbo = 8 * DIM;
    const uint32_t id_s = idesc_f8(128, C::kNS, 0, 0);
    const uint32_t id_o = idesc_f8(128, C::kNO, 1, 0);
    const uint64_t dk0 = smem_desc(smem_u32(sm.k[0]), 0, sbo, lay);
    const uint64_t dq = smem_desc(smem_u32(sm.q), 0, sbo, lay);
    // head dim 64: M = 128 takes a second 64-row atom; it reads the tile of K
    // that lies behind V's, into lanes 64 .. 127 of O^T, which nobody reads
    const uint64_t dv0 = smem_desc(
        smem_u32(sm.v[0]), DIM == 64 ? smem_u32(sm.k[0]) - smem_u32(sm.v[0]) : 0, sbo, lay);
    const uint64_t dp0 = smem_desc(smem_u32(sm.p[0]), 0, 1024, kLayoutSW128);
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
        const int st = (tc + t) % C::kStages, sb = (tc + t) & 1;
#pragma unroll
        for (int ks = 0; ks < DIM / 32; ++ks)
          mma_f8_w(tmem + sb * C::kNS, dk0 + st * kStep + 2 * ks, dq + 2 * ks, id_s, ks > 0);
        tc_commit_w(smem_u32(&sm.s_full[sb]));
      };
      auto wait_full = [&](int t) {
        const int x = tc + t;
        return mbar_wait_w_ab(smem_u32(&sm.full[x % C::kStages]), (x / C::kStages) & 1,
                              &sm.abort);
      };
      ok = mbar_wait_w_ab(smem_u32(&sm.q_full), nlive & 1, &sm.abort) && wait_full(0);
      if (!ok) break;
      tc_fence_after();
      issue_s(0);
      for (int t = 0; t < nt && ok; ++t) {
        // the next scores first, if their keys are here already
        bool ahead = false;
        if (t + 1 < nt) {
          const int x = tc + t + 1;
          ahead = __all_sync(0xffffffffu, mbar_test(smem_u32(&sm.full[x % C::kStages]),
                                                    (x / C::kStages) & 1));
          if (ahead) {
            tc_fence_after();
            issue_s(t + 1);
          }
        }
        const int x = tc + t, pb = x & 1;
        ok = mbar_wait_w_ab(smem_u32(&sm.p_full[pb]), (x >> 1) & 1, &sm.abort);
        // O^T of the segment before has been read
        if (ok && t == 0 && nlive > 0)
          ok = mbar_wait_w_ab(smem_u32(&sm.o_empty), (nlive - 1) & 1, &sm.abort);
        if (!ok) break;
        tc_fence_after();
        const int st = x % C::kStages;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_f8_w(tmem + C::kColO, dv0 + st * kStep + ks * (32 * DIM / 16),
                   dp0 + pb * (3 * R * 128 / 16) + 2 * ks, id_o, t > 0 || ks > 0);
        tc_commit_w(smem_u32(&sm.empty[st]));
        tc_commit_w(smem_u32(&sm.pv_done[pb]));
        if (t + 1 < nt && !ahead) {
          ok = wait_full(t + 1);
          if (!ok) break;
          tc_fence_after();
          issue_s(t + 1);
        }
      }
      tc += nt;
      ++nlive;
    }
    if (!ok) sm.abort = 1;
  } else {
    // ------------------------------------------------------------ softmax
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    int tc = 0;
    bool ok = true, late = false;  // late: a wait ran out where the warps cannot part
    for (int ns = 0;; ++ns) {
      const int sl = ns % kSegSlots;
      ok = mbar_wait_w_ab(smem_u32(&sm.seg_full[sl]), (ns / kSegSlots) & 1, &sm.abort);
      if (!ok) sm.stop[0] = sm.stop[1] = 1;
      Segment sg{};
      if (ok) sg = sm.seg[sl];
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(smem_u32(&sm.seg_empty[sl]));
      // (also: everybody is done with the row tables of the segment before)
      if (softmax_vote(!ok)) {
        ok = false;
        break;
      }
      if (sg.s < 0) break;
      const int nt = sg.i1 - sg.i0;
      const int rows = static_cast<int>(
          min(static_cast<long long>(R), static_cast<long long>(sg.n) * g.G - sg.row0));
      // row tables, and the queries as two E4M3 terms
      if (tid < R) {
        const int i = (sg.row0 + tid) / g.G, hq = sg.hk * g.G + (sg.row0 + tid) % g.G;
        const bool live = tid < rows;
        sm.pos[tid] = live ? sg.start + i : -1;
        sm.orow[tid] = live ? (sg.s + i) * g.H + hq : -1;
        sm.ref_m[tid] = sm.ref_w[tid] = kUnset;
      }
      if (nt > 0) {
        constexpr int LPR = DIM / 8, PER = 128 / LPR;
#pragma unroll 1
        for (int r0 = 0; r0 < R; r0 += PER) {
          const int r = r0 + tid / LPR, ch = tid % LPR;
          uint4 w = make_uint4(0, 0, 0, 0);
          if (r < rows) {
            const int i = (sg.row0 + r) / g.G, hq = sg.hk * g.G + (sg.row0 + r) % g.G;
            w = __ldg(reinterpret_cast<const uint4*>(
                g.q + (sg.s + i) * g.q_stride + static_cast<long long>(hq) * DIM + ch * 8));
          }
          float x[8];
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
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
          for (int o = LPR / 2; o > 0; o >>= 1)
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
            // K-major rows of DIM bytes, 16-byte chunks swizzled as TMA does
            auto at = [&](int n) {
              const int c16 = ch >> 1;
              const int sw = DIM == 128 ? (c16 ^ (n & 7)) : (c16 ^ ((n >> 1) & 3));
              return reinterpret_cast<uint2*>(sm.q + n * DIM + sw * 16 + (ch & 1) * 8);
            };
            *at(r) = make_uint2(hc[0] | (hc[1] << 16), hc[2] | (hc[3] << 16));
            *at(R + r) = make_uint2(lc[0] | (lc[1] << 16), lc[2] | (lc[3] << 16));
            if (ch == 0) sm.qf[r] = g.scale_log2 * (e < -126 ? 0x1p-127f : exp2i(e));
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(smem_u32(&sm.q_full));
      }
      softmax_sync();  // row tables
      float l[R];
#pragma unroll
      for (int r = 0; r < R; ++r) l[r] = 0.f;
      // every row sees the keys below pf + 1 (and, windowed, from wlast on)
      const int pf = sg.start + sg.row0 / g.G;
      const int pl = sg.start + (sg.row0 + rows - 1) / g.G;
      const int wlast = g.window > 0 ? pl - g.window + 1 : 0;
      const int all_pieces = g.page_size >= 128 ? 1 : (1 << (128 / g.page_size)) - 1;

      for (int t = 0; t < nt; ++t, ++tc) {
        const int st = tc % C::kStages, buf = tc & 1;
        const int k0 = tile_of(sg, sg.i0 + t) * 128, key = k0 + tid;
        ok = mbar_wait_w_ab(smem_u32(&sm.s_full[buf]), (tc >> 1) & 1, &sm.abort);
        // the scale bytes: landed before the scores could be computed
        ok = ok && mbar_wait_w_ab(smem_u32(&sm.full[st]), (tc / C::kStages) & 1, &sm.abort);
        // the product two tiles back has read this buffer of P^T
        if (tc >= 2)
          ok = ok && mbar_wait_w_ab(smem_u32(&sm.pv_done[buf]), ((tc - 2) >> 1) & 1, &sm.abort);
        if (!ok) sm.stop[tc & 1] = 1;
        tc_fence_after();
        float x[R];
        const int eb = sm.vs[st][tid];
        const float kf = pow2_byte(sm.ks[st][tid]), ev = static_cast<float>(eb - 127);
        if (ok) {
#pragma unroll
          for (int c = 0; c < R; c += 8) {
            uint32_t h[8], lo[8];
            tmem_ld8(tmem + lanes + buf * C::kNS + c, h);
            tmem_ld8(tmem + lanes + buf * C::kNS + R + c, lo);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 8; ++i)
              x[c + i] = fmaf(__uint_as_float(lo[i]), 0.0625f, __uint_as_float(h[i])) *
                         (kf * sm.qf[c + i]);
          }
        } else {
#pragma unroll
          for (int r = 0; r < R; ++r) x[r] = 0.f;
        }
        // keys that not every row sees
        const int loaded = sm.loaded[st];
        const bool whole = loaded == all_pieces && k0 + 127 <= pf &&
                           (g.window == 0 || k0 >= wlast || k0 + 127 < g.sinks);
        if (!whole) {
          const int piece = g.page_size >= 128 ? 0 : tid / g.page_size;
          const bool here = (loaded >> piece) & 1;
          bool any = false, every = true;
          uint32_t seen[(R + 31) / 32] = {};
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const int p = sm.pos[r];
            const bool s = here && key <= p &&
                           (g.window == 0 || key > p - g.window || key < g.sinks);
            if (s) seen[r / 32] |= 1u << (r % 32);
            else x[r] = -INFINITY;
            any |= s;
            every &= s || r >= rows;
          }
          // A value that some rows see and others do not must not reach the
          // others: 0 x NaN is NaN.  Unseen rows of V are cleared; a NaN in a
          // half-seen one moves into the weights of those that see it.
          if (!every) {
            uint4* vr = reinterpret_cast<uint4*>(sm.v[st] + tid * DIM);
            bool nan = false;
            if (any) {
              for (int i = 0; i < DIM / 16; ++i) {
                const uint4 a = vr[i];
                const uint32_t aa[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  nan |= ((((aa[j] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0);
              }
            }
            if (!any || nan)
              for (int i = 0; i < DIM / 16; ++i) vr[i] = make_uint4(0, 0, 0, 0);
            if (nan) {
#pragma unroll
              for (int r = 0; r < R; ++r)
                if ((seen[r / 32] >> (r % 32)) & 1) x[r] = __uint_as_float(0x7FC00000u);
            }
          }
        }
        // do the references hold?
        bool over = false;
#pragma unroll
        for (int r = 0; r < R; ++r)
          over |= x[r] > sm.ref_m[r] + kSlackM || x[r] + ev > sm.ref_w[r] + kSlackW;
        const bool move = softmax_vote(over);
        if (sm.stop[tc & 1]) {  // the same for all: written before the barrier
          ok = false;
          break;
        }
        if (move) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float a = warp_max(x[r]), c = warp_max(x[r] + ev);
            if (lane == 0) {
              sm.red[warp][r][0] = a;
              sm.red[warp][r][1] = c;
            }
          }
          softmax_sync();
          if (tid < R) {
            float a = -INFINITY, c = -INFINITY;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              a = fmaxf(a, sm.red[w][tid][0]);
              c = fmaxf(c, sm.red[w][tid][1]);
            }
            const float m0 = sm.ref_m[tid], w0 = sm.ref_w[tid];
            const float m1 = a > m0 + kSlackM ? ceilf(a) : m0;
            const float w1 = c > w0 + kSlackW ? ceilf(c) : w0;
            sm.ref_m[tid] = m1;
            sm.ref_w[tid] = w1;
            sm.f_m[tid] = ex2_approx(m0 - m1);
            sm.f_w[tid] = ex2_approx(w0 - w1);
          }
          softmax_sync();
#pragma unroll
          for (int r = 0; r < R; ++r) l[r] *= sm.f_m[r];
          if (t > 0) {  // O^T, once the product before has added to it
            if (!mbar_wait_w_ab(smem_u32(&sm.pv_done[buf ^ 1]), ((tc - 1) >> 1) & 1, &sm.abort)) {
              late = true;
              sm.stop[(tc + 1) & 1] = 1;
            }
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 3 * R; c += 8) {
              uint32_t a[8];
              tmem_ld8(tmem + lanes + C::kColO + c, a);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 8; ++i)
                a[i] = __float_as_uint(__uint_as_float(a[i]) * sm.f_w[(c + i) % R]);
              tmem_st8(tmem + lanes + C::kColO + c, a);
            }
            tmem_st_wait();
          }
        }
        // weights: P^T as rows of 128 bytes (one a query row and term), keys
        // along them, 16-byte chunks swizzled
        const uint32_t pbase = smem_u32(sm.p[buf]) + (tid & 15);
#pragma unroll
        for (int r = 0; r < R; r += 2) {
          l[r] += ex2_approx(x[r] - sm.ref_m[r]);
          l[r + 1] += ex2_approx(x[r + 1] - sm.ref_m[r + 1]);
          float a = ex2_approx(x[r] + (ev - sm.ref_w[r] + kShiftW));
          float b = ex2_approx(x[r + 1] + (ev - sm.ref_w[r + 1] + kShiftW));
#pragma unroll
          for (int term = 0; term < 3; ++term) {
            const uint32_t c = cvt_e4m3x2(a, b);
            const int n0 = term * R + r, n1 = n0 + 1;
            sts8(pbase + n0 * 128 + (((tid >> 4) ^ (n0 & 7)) << 4), c);
            sts8(pbase + n1 * 128 + (((tid >> 4) ^ (n1 & 7)) << 4), c >> 8);
            if (term < 2) {
              const float2 h = e4m3x2_to_float2(c);
              a = (a - h.x) * 32.f;
              b = (b - h.y) * 32.f;
            }
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(smem_u32(&sm.p_full[buf]));
      }
      if (!ok) break;

      // ---------------------------------------------------------- epilogue
      if (nt > 0) {
        const int x = tc - 1;
        ok = mbar_wait_w_ab(smem_u32(&sm.pv_done[x & 1]), (x >> 1) & 1, &sm.abort);
        tc_fence_after();
      }
      // l over the keys (threads)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float s = l[r];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) sm.red[warp][r][0] = s;
      }
      if (softmax_vote(!ok || late)) {
        ok = false;
        break;
      }
      if (tid < rows) {
        const float s = (sm.red[0][tid][0] + sm.red[1][tid][0]) +
                        (sm.red[2][tid][0] + sm.red[3][tid][0]);
        const float m = sm.ref_m[tid], w = sm.ref_w[tid];
        if (sg.slot >= 0) {
          g.stats[static_cast<size_t>(sg.slot) * R + tid] = make_float4(m, s, w, 0.f);
        } else {
          // o = O^T 2^(w - shift - m) / l; nothing seen: l = 0
          sm.f_m[tid] = s == 0.f ? 0.f : 1.f / s;
          sm.f_w[tid] = s == 0.f ? 0.f : exp2f(w - kShiftW - m);
          const int orow = sm.orow[tid];
          if (g.lse != nullptr)
            g.lse[static_cast<size_t>(orow % g.H) * g.T + orow / g.H] = (m + log2f(s)) * kLn2;
        }
      }
      softmax_sync();
      const bool active = DIM == 128 || tid < DIM;
#pragma unroll
      for (int c = 0; c < R; c += 8) {
        uint32_t h[8], m[8], lo[8];
        if (nt > 0) {
          tmem_ld8(tmem + lanes + C::kColO + c, h);
          tmem_ld8(tmem + lanes + C::kColO + R + c, m);
          tmem_ld8(tmem + lanes + C::kColO + 2 * R + c, lo);
          tmem_ld_wait();
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = c + i;
          if (r < rows && active) {
            const float v =
                nt > 0 ? fmaf(fmaf(__uint_as_float(lo[i]), 0x1p-5f, __uint_as_float(m[i])), 0x1p-5f,
                              __uint_as_float(h[i]))
                       : 0.f;
            if (sg.slot >= 0)
              g.partial[(static_cast<size_t>(sg.slot) * R + r) * DIM + tid] = v;
            else
              g.o[static_cast<size_t>(sm.orow[r]) * DIM + tid] =
                  __float2bfloat16(sm.f_m[r] == 0.f ? 0.f : v * sm.f_m[r] * sm.f_w[r]);
          }
        }
      }
      if (nt > 0) {
        tc_fence_before();
        mbar_arrive(smem_u32(&sm.o_empty));
      }
    }
    if (!ok) sm.abort = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && sm.abort) report(g.status, FLAMIA_DEV_TIMEOUT);
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

// Joins the parts of an item that several CTAs shared: part 0 in slot 1 of the
// CTA before, the others in slots 0 from this CTA on.
template <int DIM, int R>
__global__ void __launch_bounds__(8 * DIM) join_kernel(const AttendArgs g) {
  __shared__ float s_wt[8][kMaxCtas];
  __shared__ float s_tot[8][2];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 j0 = g.joins[2 * blockIdx.x], j1 = g.joins[2 * blockIdx.x + 1];
  const int parts = j0.x;
  if (parts <= 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = blockIdx.x, first = blockIdx.y * 8;
  auto slot = [&](int p) { return p == 0 ? 2 * (c0 - 1) + 1 : 2 * (c0 + p - 1); };
  const int rows = static_cast<int>(
      min(static_cast<long long>(R), static_cast<long long>(j0.z) * g.G - j1.x));
  if (warp < 8 && first + warp < rows) {
    const int r = first + warp;
    float m = kUnset, w = kUnset;
    for (int p = lane; p < parts; p += 32) {
      const float4 s = g.stats[static_cast<size_t>(slot(p)) * R + r];
      m = fmaxf(m, s.x);
      w = fmaxf(w, s.z);
    }
    m = warp_max(m);
    w = warp_max(w);
    float l = 0.f;
    for (int p = lane; p < parts; p += 32) {
      const float4 s = g.stats[static_cast<size_t>(slot(p)) * R + r];
      l += s.y * ex2_approx(s.x - m);
      s_wt[warp][p] = ex2_approx(s.z - w);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) {
      s_tot[warp][0] = l == 0.f ? 0.f : 1.f / l;
      s_tot[warp][1] = exp2f(w - kShiftW - m);
      if (g.lse != nullptr) {
        const int i = (j1.x + r) / g.G, hq = j0.w * g.G + (j1.x + r) % g.G;
        g.lse[static_cast<size_t>(hq) * g.T + j0.y + i] = (m + log2f(l)) * kLn2;
      }
    }
  }
  __syncthreads();
  const int rl = threadIdx.x / DIM, dd = threadIdx.x % DIM, r = first + rl;
  if (r >= rows) return;
  float acc = 0.f;
#pragma unroll 8
  for (int p = 0; p < parts; ++p)
    acc += s_wt[rl][p] * g.partial[(static_cast<size_t>(slot(p)) * R + r) * DIM + dd];
  const int i = (j1.x + r) / g.G, hq = j0.w * g.G + (j1.x + r) % g.G;
  g.o[(static_cast<size_t>(j0.y + i) * g.H + hq) * DIM + dd] =
      __float2bfloat16(s_tot[rl][0] == 0.f ? 0.f : acc * s_tot[rl][0] * s_tot[rl][1]);
}

// ------------------------------------------------------------------ host

// Query rows side by side in one item: those of a K / V head's mean number of
// new tokens, up to 32 (more rows reuse a K / V tile more often, but each costs
// its share of the softmax warps' time).
int rows_per_item(int T, int ndocs, int G) {
  const long long rows = ((static_cast<long long>(T) + ndocs - 1) / ndocs) * G;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
}

struct Workspace {
  size_t joins, stats, partial, total;
};
Workspace layout(int R, int d) {
  Workspace w;
  w.joins = 0;
  w.stats = align_up(sizeof(int4) * 2 * kMaxCtas, 256);
  w.partial = w.stats + align_up(sizeof(float4) * static_cast<size_t>(kSlots) * R, 256);
  w.total = w.partial + sizeof(float) * static_cast<size_t>(kSlots) * R * d;
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

template <int DIM, int R>
flamia_status launch(const flamia_kvcache* c, const AttendArgs& g, cudaStream_t s) {
  CUtensorMap mk, mv;
  if (!make_page_map(&mk, c->k_codes, c) || !make_page_map(&mv, c->v_codes, c))
    return FLAMIA_ERR_CUDA;
  constexpr int smem = static_cast<int>(sizeof(Smem<DIM, R>)) + 1024;
  if (cudaFuncSetAttribute(attend_kernel<DIM, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           smem) != cudaSuccess)
    return FLAMIA_ERR_CUDA;
  const int grid = min(kMaxCtas, num_sms() * Cfg<DIM, R>::kCtas);
  attend_kernel<DIM, R><<<grid, kThreads, smem, s>>>(mk, mv, g);
  if (cudaGetLastError() != cudaSuccess) return FLAMIA_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, R / 8);
  cfg.blockDim = dim3(8 * DIM);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, join_kernel<DIM, R>, g) != cudaSuccess) return FLAMIA_ERR_CUDA;
  count_launches(2);
  return FLAMIA_OK;
}

}  // namespace
}  // namespace flamia

using namespace flamia;

extern "C" size_t flamia_attn_cache_workspace_bytes(int T, int ndocs, int H, int H_kv, int d) {
  if (!supported_dim(d) || !valid_batch(T, ndocs) || H <= 0 || H > 4096 || H_kv <= 0 ||
      H % H_kv != 0)
    return 0;
  return layout(rows_per_item(T, ndocs, H / H_kv), d).total;
}

extern "C" flamia_status flamia_attn_cache(const flamia_kvcache* cache, const void* q_bf16,
                                           int64_t q_stride, int T, int H,
                                           const int32_t* cu_seqlens, int ndocs,
                                           const int32_t* starts, const int32_t* page_table,
                                           int table_stride, float softmax_scale, int window,
                                           int sinks, void* o_bf16, float* lse, void* ws,
                                           size_t ws_bytes, int* dev_status, void* stream) {
  const flamia_status st = check_cache(cache);
  if (st != FLAMIA_OK) return st;
  if (!valid_batch(T, ndocs) || table_stride <= 0 || H <= 0 || H > 4096 || H % cache->H_kv != 0 ||
      !(softmax_scale > 0.f) || std::isinf(softmax_scale) || window < 0 || sinks < 0 ||
      (sinks > 0 && window == 0) || static_cast<long long>(T) * H >= (1ll << 31))
    return FLAMIA_ERR_INVALID_ARG;
  if (T == 0) return FLAMIA_OK;
  if (!valid_rows(q_bf16, q_stride) || o_bf16 == nullptr || !aligned(o_bf16, 16) ||
      cu_seqlens == nullptr || page_table == nullptr || ws == nullptr || !aligned(ws, 256) ||
      !aligned(lse, 4))
    return FLAMIA_ERR_INVALID_ARG;
  const int G = H / cache->H_kv, d = cache->d;
  const int R = rows_per_item(T, ndocs, G);
  const Workspace w = layout(R, d);
  if (ws_bytes < w.total) return FLAMIA_ERR_WORKSPACE;
  AttendArgs g{};
  g.k_scales = cache->k_scales;
  g.v_scales = cache->v_scales;
  g.q = static_cast<const __nv_bfloat16*>(q_bf16);
  g.o = static_cast<__nv_bfloat16*>(o_bf16);
  g.lse = lse;
  g.cu = cu_seqlens;
  g.starts = starts;
  g.table = page_table;
  g.joins = reinterpret_cast<int4*>(static_cast<uint8_t*>(ws) + w.joins);
  g.stats = reinterpret_cast<float4*>(static_cast<uint8_t*>(ws) + w.stats);
  g.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + w.partial);
  g.status = dev_status;
  g.q_stride = q_stride;
  g.T = T;
  g.H = H;
  g.H_kv = cache->H_kv;
  g.G = G;
  g.ndocs = ndocs;
  g.table_stride = table_stride;
  g.num_pages = cache->num_pages;
  g.page_size = cache->page_size;
  // positions stay below 2^30: larger windows and first tokens see the same
  g.window = window < kMaxPos ? window : kMaxPos;
  g.sinks = sinks < kMaxPos ? sinks : kMaxPos;
  g.scale_log2 = softmax_scale * 1.44269504088896340736f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 128)
    return R == 8 ? launch<128, 8>(cache, g, s)
                  : R == 16 ? launch<128, 16>(cache, g, s) : launch<128, 32>(cache, g, s);
  return R == 8 ? launch<64, 8>(cache, g, s)
                : R == 16 ? launch<64, 16>(cache, g, s) : launch<64, 32>(cache, g, s);
}
