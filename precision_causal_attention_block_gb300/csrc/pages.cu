// Pages of the cache: copying them, sharing them between sequences that continue one
// another (fork, with counts of a page's users), handing out pages for new tokens
// (reserve, with a copy of a page that others use as well) and moving the used ones to
// the front of the pool (compact).
//
// The books (page table, counts) are kept on the device, so that a captured step can
// hand out its own pages.  Their results do not depend on timing: free pages are taken
// in ascending order by (sequence, slot), counts are sums, and of the users of a page
// that all want to write it the last in order keeps it.  Books are small (4 bytes a page
// and a table entry), so one CTA works them out between barriers of its own; what it
// decides is left as a list of copies for a second kernel on the whole GPU, or, if these are
// few, copied by itself.
//
// Copies are HBM-bound: a warp takes up to 64 rows of one head of K or V (8 or 4 KB),
// all its loads before its stores.  4,099 pages of 64 tokens, 8 heads of 128 (1.08 GB both
// ways): 160 us, 6.8 TB/s; 7 small pages: 2.1 us on the device, 10 with the host's call.
//
// The books are chains of dependent loads between a CTA's barriers: fork of 8 rows of 9 slots
// with the pages of their next tokens 13 us on the device (two kernels) and 20 with the host's
// calls, of 192 rows of 128 slots 5 + 4 us and 10 for the pages; compact of 5,451 pages, half
// of them in use, 8 us beside 52 for its copies.
#include "paged.cuh"

namespace flamia {
namespace {

constexpr int kMaxPoolSeqs = 1 << 16;
constexpr int kPlan = 1024;       // threads of the CTA that keeps the books
constexpr int kCopyThreads = 256;
constexpr int kCopyRows = 64;     // rows a warp copies

// ------------------------------------------------------------------ copies

struct CopyArgs {
  const uint8_t* from[4];  // K codes, V codes, K scales, V scales
  uint8_t* to[4];
  const int32_t *src, *dst;  // pairs of whole pages, or
  const int4* list;          // (source, target, rows, -): see reserve and compact
  const int* count;          // entries on the device, or NULL: n of them
  int* status;
  // compact: page numbers behind `live` in the page table take their new ones
  const int32_t* moved;
  const int* live;
  int32_t* table;
  long long entries;
  int n, H_kv, page_size, from_pages, to_pages;
};

// Table entries of moved pages, by the warp's lanes.
__device__ __forceinline__ void renumber(const CopyArgs& g, int live, long long warp0,
                                         long long warps) {
  const int lane = threadIdx.x & 31;
  for (long long i = warp0 * 32 + lane; i < g.entries; i += warps * 32) {
    const int p = g.table[i];
    if (p >= live && p < g.from_pages) g.table[i] = g.moved[p];
  }
}

// n entries, units of ROWS rows of a page's head (K or V) by warps in turn.
template <int DIM, int ROWS>
__device__ __forceinline__ void copy_units(const CopyArgs& g, int n, long long warp0,
                                           long long warps) {
  constexpr int kPer = ROWS * DIM / 16 / 32;  // 16-byte pieces a lane
  const int lane = threadIdx.x & 31;
  const int blocks = (g.page_size + ROWS - 1) / ROWS;
  const int per = 2 * g.H_kv * blocks;  // units of a page: K / V, head, block of rows
  const long long units = static_cast<long long>(n) * per;
  for (long long u = warp0; u < units; u += warps) {
    const int i = static_cast<int>(u / per);
    int at = static_cast<int>(u - static_cast<long long>(i) * per);
    const int4 e = g.list != nullptr ? g.list[i] : make_int4(g.src[i], g.dst[i], g.page_size, 0);
    if (e.x < 0 || e.y < 0) continue;
    if (e.x >= g.from_pages || e.y >= g.to_pages) {
      if (lane == 0) report(g.status, FLAMIA_DEV_BAD_PAGE);
      continue;
    }
    const int kv = at >= g.H_kv * blocks;
    at -= kv * g.H_kv * blocks;
    const int h = at / blocks, r0 = (at - h * blocks) * ROWS;
    const int rows = min(min(e.z, g.page_size) - r0, ROWS);
    if (rows <= 0) continue;
    const long long from = (static_cast<long long>(e.x) * g.H_kv + h) * g.page_size + r0;
    const long long to = (static_cast<long long>(e.y) * g.H_kv + h) * g.page_size + r0;
    const uint4* s = reinterpret_cast<const uint4*>((kv ? g.from[1] : g.from[0]) + from * DIM);
    uint4* d = reinterpret_cast<uint4*>((kv ? g.to[1] : g.to[0]) + to * DIM);
    const uint8_t* ss = (kv ? g.from[3] : g.from[2]) + from;
    uint8_t* ds = (kv ? g.to[3] : g.to[2]) + to;
    const int pieces = rows * (DIM / 16);
    uint4 x[kPer];
    uint32_t sc = 0;
    const int b = 2 * lane;
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (j * 32 + lane < pieces) x[j] = s[j * 32 + lane];
    if (b + 1 < rows)
      sc = *reinterpret_cast<const uint16_t*>(ss + b);
    else if (b < rows)
      sc = ss[b];
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (j * 32 + lane < pieces) d[j * 32 + lane] = x[j];
    if (b + 1 < rows)
      *reinterpret_cast<uint16_t*>(ds + b) = static_cast<uint16_t>(sc);
    else if (b < rows)
      ds[b] = static_cast<uint8_t>(sc);
  }
}

template <int DIM>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const CopyArgs g) {
  const long long warps = static_cast<long long>(gridDim.x) * (kCopyThreads / 32);
  const long long warp0 =
      static_cast<long long>(blockIdx.x) * (kCopyThreads / 32) + (threadIdx.x >> 5);
  start_next();
  wait_for_previous();
  if (g.moved != nullptr) renumber(g, *g.live, warp0, warps);
  copy_units<DIM, kCopyRows>(g, g.count != nullptr ? *g.count : g.n, warp0, warps);
}

// All of the arguments but the entries.
void copy_args(CopyArgs& g, const flamia_kvcache* from, const flamia_kvcache* to) {
  g.from[0] = from->k_codes;
  g.from[1] = from->v_codes;
  g.from[2] = from->k_scales;
  g.from[3] = from->v_scales;
  g.to[0] = to->k_codes;
  g.to[1] = to->v_codes;
  g.to[2] = to->k_scales;
  g.to[3] = to->v_scales;
  g.H_kv = from->H_kv;
  g.page_size = from->page_size;
  g.from_pages = from->num_pages;
  g.to_pages = to->num_pages;
}

// `most`: as many entries as there can be.
flamia_status launch_copy(const CopyArgs& g, int d, long long most, cudaStream_t s) {
  // (2 x 4096 x 2^14 blocks at most: an int)
  const long long units = most * (2ll * g.H_kv * ((g.page_size + kCopyRows - 1) / kCopyRows));
  long long ctas = units / (kCopyThreads / 32) + 1;
  const long long remap = (g.entries + kCopyThreads - 1) / kCopyThreads;
  if (ctas < remap) ctas = remap;
  const long long cap = 16ll * num_sms();
  if (ctas > cap) ctas = cap;
  return launch_after(d == 128 ? copy_kernel<128> : copy_kernel<64>,
                      dim3(static_cast<unsigned>(ctas < 1 ? 1 : ctas)), kCopyThreads, 0, s, g)
             ? FLAMIA_OK
             : FLAMIA_ERR_CUDA;
}

// ------------------------------------------------------------------ fork

struct ForkArgs {
  int32_t *refs, *table, *lens;
  const int32_t *parents, *children;
  int32_t* rows;  // [n][stride]: what the children's rows become
  int32_t* held;  // [n]: their lengths; -1: the entry does nothing
  int* status;
  int n, nseq, stride, num_pages, page_size;
};

constexpr int kForkThreads = 256;

// Entry i (a CTA each): its parent's row and length are put by and all counts set, so
// that the second kernel can write rows that are other entries' parents.
__global__ void __launch_bounds__(kForkThreads) fork_read_kernel(const ForkArgs g) {
  const int i = blockIdx.x, tid = threadIdx.x;
  start_next();
  wait_for_previous();
  const int child = g.children[i];
  const int parent = g.parents != nullptr ? g.parents[i] : -1;
  bool again = false;  // a later entry names the same child, and counts instead
  for (int j = i + 1 + tid; j < g.n; j += kForkThreads) again |= g.children[j] == child;
  again = __syncthreads_or(again);
  const bool bad = child >= g.nseq || parent >= g.nseq;
  if (bad && tid == 0) report(g.status, FLAMIA_DEV_BAD_PAGE);
  if (bad || again || child < 0) {
    if (tid == 0) g.held[i] = -1;
    return;
  }
  const int len = parent >= 0 ? max(g.lens[parent], 0) : 0;
  const int32_t* from = g.table + static_cast<long long>(max(parent, 0)) * g.stride;
  const int32_t* old = g.table + static_cast<long long>(child) * g.stride;
  int32_t* row = g.rows + static_cast<long long>(i) * g.stride;
  const int need = len / g.page_size + (len % g.page_size > 0);
  if (need > g.stride && tid == 0) report(g.status, FLAMIA_DEV_BAD_PAGE);
  for (int j = tid; j < g.stride; j += kForkThreads) {
    const int was = old[j];
    int now = j < need ? from[j] : -1;
    if (j < need && (now < 0 || now >= g.num_pages)) {
      report(g.status, FLAMIA_DEV_BAD_PAGE);
      now = -1;
    }
    if (was >= 0 && was < g.num_pages && was != now) atomicSub(&g.refs[was], 1);
    if (now >= 0 && was != now) atomicAdd(&g.refs[now], 1);
    row[j] = now;
  }
  if (tid == 0) g.held[i] = len;
}

__global__ void __launch_bounds__(kForkThreads) fork_write_kernel(const ForkArgs g) {
  const int i = blockIdx.x, tid = threadIdx.x;
  start_next();
  wait_for_previous();
  const int len = g.held[i];
  if (len < 0) return;
  const int child = g.children[i];
  const int32_t* row = g.rows + static_cast<long long>(i) * g.stride;
  int32_t* to = g.table + static_cast<long long>(child) * g.stride;
  for (int j = tid; j < g.stride; j += kForkThreads) to[j] = row[j];
  if (tid == 0) g.lens[child] = len;
}

// The same by one CTA, without a second launch or a workspace.
constexpr int kSmallForks = 128;    // entries, and
constexpr int kSmallSlots = 4096;   // slots of their rows
constexpr int kSmallThreads = 512;

__global__ void __launch_bounds__(kSmallThreads) fork_small_kernel(const ForkArgs g) {
  constexpr int kEach = kSmallSlots / kSmallThreads;
  __shared__ int s_child[kSmallForks], s_parent[kSmallForks], s_len[kSmallForks];
  const int tid = threadIdx.x;
  start_next();
  wait_for_previous();
  if (tid < g.n) {
    s_child[tid] = g.children[tid];
    s_parent[tid] = g.parents != nullptr ? g.parents[tid] : -1;
  }
  __syncthreads();
  if (tid < g.n) {
    const int child = s_child[tid], parent = s_parent[tid];
    bool does = child >= 0 && child < g.nseq && parent < g.nseq;
    if (child >= g.nseq || parent >= g.nseq) report(g.status, FLAMIA_DEV_BAD_PAGE);
    for (int j = tid + 1; j < g.n; ++j) does &= s_child[j] != child;
    const int len = does && parent >= 0 ? max(g.lens[parent], 0) : 0;
    if (does && (len - 1) / g.page_size >= g.stride) report(g.status, FLAMIA_DEV_BAD_PAGE);
    s_len[tid] = does ? len : -1;
  }
  __syncthreads();
  const int slots = g.n * g.stride;
  int row[kEach];  // what the slots become
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int at = k * kSmallThreads + tid;
    row[k] = -1;
    if (at >= slots) continue;
    const int i = at / g.stride, j = at - i * g.stride, len = s_len[i];
    if (len < 0) continue;
    const int was = g.table[static_cast<long long>(s_child[i]) * g.stride + j];
    if (j < len / g.page_size + (len % g.page_size > 0)) {
      row[k] = g.table[static_cast<long long>(s_parent[i]) * g.stride + j];
      if (row[k] < 0 || row[k] >= g.num_pages) {
        report(g.status, FLAMIA_DEV_BAD_PAGE);
        row[k] = -1;
      }
    }
    if (was != row[k]) {
      if (was >= 0 && was < g.num_pages) atomicSub(&g.refs[was], 1);
      if (row[k] >= 0) atomicAdd(&g.refs[row[k]], 1);
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int at = k * kSmallThreads + tid;
    if (at >= slots) continue;
    const int i = at / g.stride, j = at - i * g.stride;
    if (s_len[i] >= 0) g.table[static_cast<long long>(s_child[i]) * g.stride + j] = row[k];
  }
  if (tid < g.n && s_len[tid] >= 0) g.lens[s_child[tid]] = s_len[tid];
}

// ------------------------------------------------------------------ books

// The CTA that keeps the books makes their copies itself if these can be no more than so many
// bytes.  That saves a launch: reserve of a step that copies nothing, as most do, 5.7 us and not
// 7.5, captured 3.7 and not 4.9.  But copies by one CTA take longer: with fork, 4 of at most
// 162 KB 19.1 us and not 21.8, captured 11.9 and not 11.0; 8 of 292 KB 19.1 and 21.8, 13.8
// and 11.1; 16 of 552 KB 19.9 and 21.9, 17.2 and 10.9; 32 of 1,072 KB 26.2 and 21.4, 24.7
// and 11.5; compact of at most 471 KB 18.7 and 20.7, 12.5 and 8.8.
constexpr long long kOwnBytes = 512 << 10;
constexpr long long kOwnEntries = 1 << 15;  // of the page table, that compact numbers anew
constexpr int kOwnRows = 32;  // rows a warp copies then (1,024 threads: 64 registers)
bool makes_copies(const flamia_kvcache* c, long long most) {
  return most * 2 * c->H_kv * c->page_size * (c->d + 1) <= kOwnBytes;
}

// Exclusive prefix of x over the CTA's threads, and their sum.  (Two barriers; scratch
// may be used again at once.)
__device__ __forceinline__ int cta_prefix(int x, int* scratch, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += y;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  const int sum = scratch[lane];  // 32 warps
  int before = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, before, off);
    if (lane >= off) before += y;
  }
  total = __shfl_sync(0xffffffffu, before, 31);
  return __shfl_sync(0xffffffffu, before - sum, warp) + inc - x;
}

// Counts of pages p .. p + 7 (0x7fffffff behind the last), as the atomics left them.
__device__ __forceinline__ void eight_counts(const int32_t* refs, int p, int pages, int (&r)[8]) {
  if (p + 8 <= pages && (reinterpret_cast<uintptr_t>(refs) & 15) == 0) {
    const int4 a = __ldcg(reinterpret_cast<const int4*>(refs + p));
    const int4 b = __ldcg(reinterpret_cast<const int4*>(refs + p) + 1);
    r[0] = a.x, r[1] = a.y, r[2] = a.z, r[3] = a.w;
    r[4] = b.x, r[5] = b.y, r[6] = b.z, r[7] = b.w;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = p + k < pages ? __ldcg(refs + p + k) : 0x7fffffff;
  }
}

// A slot of a sequence that new tokens touch.
struct Slot {
  int32_t seq, slot, page, users;  // its page and that page's count, if it has one
};

struct ReserveArgs {
  int32_t *refs, *table;
  const int32_t *cu, *starts;
  int32_t* granted;  // [nseq + 1]
  Slot* slots;     // [cap]
  int32_t* rank;   // [cap]: which of the new pages a slot takes, -1: none
  int32_t* fresh;  // [cap]: the new pages
  int4* list;      // [nseq]: copies
  int* count;      // their number
  int* status;
  int T, nseq, stride, num_pages, page_size, cap;
};

template <int DIM>  // 0: the copies are left to a second kernel
__global__ void __launch_bounds__(kPlan) reserve_kernel(const ReserveArgs g, const CopyArgs c) {
  __shared__ int scratch[32];
  __shared__ int s_copies;
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) s_copies = 0;
  start_next();
  wait_for_previous();
  // Malformed offsets: ranges that overlap touch more slots than there is room for, and a page
  // that a slot did not get may be another sequence's as well.  So nobody gets any.
  bool malformed = tid == 0 && (g.cu[0] != 0 || g.cu[g.nseq] > g.T);
  for (int i = tid; i < g.nseq; i += kPlan) malformed |= g.cu[i] > g.cu[i + 1];
  if (malformed) report(g.status, FLAMIA_DEV_BAD_SEQLENS);
  // the slots, in order of sequence and position (a sequence's first two by its own
  // thread; those of longer ones by the whole warp)
  int n = 0;
  bool outside = false;  // some sequence's positions are, of its row
  auto put = [&](int b, int slot, int at) {
    if (at >= g.cap) return;  // (malformed offsets only: see reserve_slots)
    const int page = g.table[static_cast<long long>(b) * g.stride + slot];
    Slot s{b, slot, page, 0};
    if (page >= g.num_pages) {
      report(g.status, FLAMIA_DEV_BAD_PAGE);
      s.users = 1;  // left as it is
    } else if (page >= 0) {
      s.users = __ldcg(g.refs + page);
    }
    g.slots[at] = s;
  };
  for (int b0 = 0; b0 < g.nseq; b0 += kPlan) {
    const int b = b0 + tid;
    int first = 0, cnt = 0;
    if (b < g.nseq) {
      const DocRange r = doc_range(g.cu, b, g.T);
      const int start = g.starts != nullptr ? g.starts[b] : 0;
      if (r.e > r.s) {
        const long long last = (static_cast<long long>(start) + (r.e - r.s) - 1) / g.page_size;
        if (start < 0 || last >= g.stride) {
          report(g.status, FLAMIA_DEV_BAD_PAGE);  // (none of the sequence's)
          outside = true;
        } else {
          first = start / g.page_size;
          cnt = static_cast<int>(last) - first + 1;
        }
      }
    }
    int total;
    const int at = n + cta_prefix(cnt, scratch, total);
    if (cnt > 0) put(b, first, at);
    if (cnt > 1) put(b, first + 1, at + 1);
    unsigned more = __ballot_sync(0xffffffffu, cnt > 2);
    while (more) {
      const int l = __ffs(more) - 1;
      more &= more - 1;
      const int c = __shfl_sync(0xffffffffu, cnt, l), a = __shfl_sync(0xffffffffu, at, l);
      const int f = __shfl_sync(0xffffffffu, first, l);
      for (int k = 2 + lane; k < c; k += 32) put(b - lane + l, f + k, a + k);
    }
    n += total;
  }
  malformed = __syncthreads_or(malformed);
  if (malformed) n = 0;
  // A page with other users: every slot here that holds it gives it up; if nobody is
  // left, the last of them keeps it.
  bool shared = false;
  for (int c = tid; c < n; c += kPlan) {
    const Slot s = g.slots[c];
    if (s.page >= 0 && s.users > 1) {
      atomicSub(g.refs + s.page, 1);
      shared = true;
    }
  }
  shared = __syncthreads_or(shared);
  if (shared) {
    for (int c = tid; c < n; c += kPlan) {
      const Slot s = g.slots[c];
      if (s.page >= 0 && s.users > 1 && __ldcg(g.refs + s.page) <= 0)
        atomicMin(g.refs + s.page, -(c + 1));
    }
    __syncthreads();
  }
  // which slots take a new page
  int need = 0;
  for (int c0 = 0; c0 < n; c0 += kPlan) {
    const int c = c0 + tid;
    bool takes = false;
    if (c < n) {
      const Slot s = g.slots[c];
      takes = s.page < 0 || (s.users > 1 && __ldcg(g.refs + s.page) != -(c + 1));
    }
    int total;
    const int at = need + cta_prefix(takes, scratch, total);
    if (c < n) g.rank[c] = takes ? at : -1;
    need += total;
  }
  // the first free pages
  int found = 0;
  for (long long p0 = 0; p0 < g.num_pages && found < need; p0 += 8 * kPlan) {
    const long long p = p0 + 8 * tid;
    int r[8], mine = 0, total;
    if (p < g.num_pages) {
      eight_counts(g.refs, static_cast<int>(p), g.num_pages, r);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) r[k] = 0x7fffffff;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) mine += r[k] == 0;
    int at = found + cta_prefix(mine, scratch, total);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (r[k] == 0) {
        if (at < need) g.fresh[at] = static_cast<int>(p) + k;
        ++at;
      }
    }
    found += total;
  }
  __syncthreads();
  const bool enough = found >= need;
  if (!enough && tid == 0) report(g.status, FLAMIA_DEV_CAPACITY);
  for (int c = tid; c < n; c += kPlan) {
    const Slot s = g.slots[c];
    const int k = g.rank[c];
    if (!enough) {  // all as it was
      if (s.page >= 0 && s.users > 1) g.refs[s.page] = s.users;
    } else if (k >= 0) {
      const int page = g.fresh[k];
      g.table[static_cast<long long>(s.seq) * g.stride + s.slot] = page;
      g.refs[page] = 1;
      const int start = g.starts != nullptr ? g.starts[s.seq] : 0;
      const int rows = start - s.slot * g.page_size;  // that the sequence holds in it
      if (s.page >= 0 && rows > 0)
        g.list[atomicAdd(&s_copies, 1)] = make_int4(s.page, page, rows, 0);
    } else if (s.page >= 0 && s.users > 1) {
      g.refs[s.page] = 1;  // kept
    }
  }
  outside = __syncthreads_or(outside);
  if (tid == 0) *g.count = s_copies;
  if (g.granted != nullptr)
    for (int i = tid; i <= g.nseq; i += kPlan) g.granted[i] = enough && !outside && !malformed ? g.cu[i] : 0;
  if constexpr (DIM > 0) copy_units<DIM, kOwnRows>(c, s_copies, tid >> 5, kPlan / 32);
}

struct CompactArgs {
  int32_t* refs;
  int32_t *src, *dst;  // [num_pages / 2 + 1]
  int32_t* moved;      // [num_pages]: new numbers of pages behind the live ones
  int4* list;
  int *count, *live, *live_out;
  int num_pages, page_size;
};

template <int DIM>  // (as above)
__global__ void __launch_bounds__(kPlan) compact_kernel(const CompactArgs g, const CopyArgs c) {
  __shared__ int scratch[32];
  const int tid = threadIdx.x;
  start_next();
  wait_for_previous();
  auto counts = [&](long long p, int (&r)[8]) {
    if (p < g.num_pages) {
      eight_counts(g.refs, static_cast<int>(p), g.num_pages, r);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) r[k] = 0x7fffffff;
    }
  };
  int mine = 0, live;
#pragma unroll 4
  for (long long p = 8 * tid; p < g.num_pages; p += 8 * kPlan) {
    int r[8];
    counts(p, r);
#pragma unroll
    for (int k = 0; k < 8; ++k) mine += r[k] > 0 && p + k < g.num_pages;
  }
  cta_prefix(mine, scratch, live);
  // free pages among the first `live`, used ones behind them: as many of each
  int holes = 0, movers = 0;
  for (long long p0 = 0; p0 < g.num_pages; p0 += 8 * kPlan) {
    const long long p = p0 + 8 * tid;
    int r[8], h = 0, m = 0, total;
    counts(p, r);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const bool there = p + k < g.num_pages;
      h += there && r[k] <= 0 && p + k < live;
      m += there && r[k] > 0 && p + k >= live;
    }
    // (16 bits each: at most 8,192 a round)
    const int at = cta_prefix(h | (m << 16), scratch, total);
    int ah = holes + (at & 0xFFFF), am = movers + (at >> 16);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (p + k >= g.num_pages) continue;
      const int page = static_cast<int>(p) + k;
      if (page < live) {
        if (r[k] <= 0) g.dst[ah++] = page;
      } else if (r[k] > 0) {
        g.src[am++] = page;
      } else {
        g.moved[page] = -1;
      }
    }
    holes += total & 0xFFFF;
    movers += total >> 16;
  }
  __syncthreads();
  for (int k = tid; k < movers; k += kPlan) {
    const int a = g.src[k], b = g.dst[k];
    g.moved[a] = b;
    g.refs[b] = __ldcg(g.refs + a);
    g.refs[a] = 0;
    g.list[k] = make_int4(a, b, g.page_size, 0);
  }
  if (tid == 0) {
    *g.count = movers;
    *g.live = live;
    if (g.live_out != nullptr) *g.live_out = live;
  }
  if constexpr (DIM > 0) {
    __syncthreads();
    renumber(c, live, tid >> 5, kPlan / 32);
    copy_units<DIM, kOwnRows>(c, movers, tid >> 5, kPlan / 32);
  }
}

// ------------------------------------------------------------------ host

// Slots that the new tokens of a call can touch: T tokens fill T / page_size pages and
// begin and end inside two more a sequence (if no two sequences have the same tokens).
long long reserve_slots(int T, int nseq, int stride, int page_size) {
  const long long by_tokens = T / page_size + 2ll * nseq, all = static_cast<long long>(nseq) * stride;
  return by_tokens < all ? by_tokens : all;
}

bool valid_pool(int num_pages, int page_size, int nseq, int stride) {
  return num_pages > 0 && page_size > 0 && nseq > 0 && nseq <= kMaxPoolSeqs && stride > 0 &&
         static_cast<long long>(nseq) * stride < (1ll << 31);
}

bool valid_books(const int32_t* refs, const int32_t* table) {
  return refs != nullptr && table != nullptr && aligned(refs, 4) && aligned(table, 4);
}

// Parts of the workspace, in turn.
struct Parts {
  uint8_t* base;
  size_t used = 0;
  template <class X>
  X* take(long long n) {
    X* p = reinterpret_cast<X*>(base + used);
    used += align_up(sizeof(X) * static_cast<size_t>(n), 256);
    return p;
  }
};

size_t reserve_parts(ReserveArgs& g, void* ws) {
  Parts w{static_cast<uint8_t*>(ws)};
  g.count = w.take<int>(1);
  g.slots = w.take<Slot>(g.cap);
  g.rank = w.take<int32_t>(g.cap);
  g.fresh = w.take<int32_t>(g.cap);
  g.list = w.take<int4>(g.nseq);
  return w.used;
}

size_t compact_parts(CompactArgs& g, void* ws) {
  Parts w{static_cast<uint8_t*>(ws)};
  int* head = w.take<int>(2);
  g.count = head;
  g.live = head + 1;
  g.src = w.take<int32_t>(g.num_pages / 2 + 1);
  g.dst = w.take<int32_t>(g.num_pages / 2 + 1);
  g.moved = w.take<int32_t>(g.num_pages);
  g.list = w.take<int4>(g.num_pages / 2 + 1);
  return w.used;
}

size_t fork_parts(ForkArgs& g, void* ws) {
  Parts w{static_cast<uint8_t*>(ws)};
  g.held = w.take<int32_t>(g.n);
  g.rows = w.take<int32_t>(static_cast<long long>(g.n) * g.stride);
  return w.used;
}

}  // namespace
}  // namespace flamia

using namespace flamia;

extern "C" flamia_status flamia_pages_copy(const flamia_kvcache* from, const flamia_kvcache* to,
                                           const int32_t* src, const int32_t* dst, int n,
                                           int* dev_status, void* stream) {
  flamia_status st = check_cache(from);
  if (st == FLAMIA_OK) st = check_cache(to);
  if (st != FLAMIA_OK) return st;
  if (from->page_size != to->page_size || from->H_kv != to->H_kv || from->d != to->d || n < 0)
    return FLAMIA_ERR_INVALID_ARG;
  if (n == 0) return FLAMIA_OK;
  if (src == nullptr || dst == nullptr || !aligned(src, 4) || !aligned(dst, 4))
    return FLAMIA_ERR_INVALID_ARG;
  CopyArgs g{};
  g.src = src;
  g.dst = dst;
  g.n = n;
  g.status = dev_status;
  copy_args(g, from, to);
  return launch_copy(g, from->d, n, static_cast<cudaStream_t>(stream));
}

extern "C" size_t flamia_pages_fork_workspace_bytes(int n, int table_stride) {
  if (!valid_pool(1, 1, n, table_stride)) return 0;
  ForkArgs g{};
  g.n = n;
  g.stride = table_stride;
  return fork_parts(g, nullptr);
}

extern "C" flamia_status flamia_pages_fork(int32_t* refs, int num_pages, int32_t* page_table,
                                           int table_stride, int nseq, int page_size,
                                           const int32_t* parents, const int32_t* children, int n,
                                           int32_t* lens, void* ws, size_t ws_bytes,
                                           int* dev_status, void* stream) {
  if (!valid_pool(num_pages, page_size, nseq, table_stride) || n < 0 || n > nseq)
    return FLAMIA_ERR_INVALID_ARG;
  if (n == 0) return FLAMIA_OK;
  if (!valid_books(refs, page_table) || children == nullptr || !aligned(children, 4) ||
      !aligned(parents, 4) || lens == nullptr || !aligned(lens, 4) || ws == nullptr ||
      !aligned(ws, 256))
    return FLAMIA_ERR_INVALID_ARG;
  ForkArgs g{};
  g.n = n;
  g.stride = table_stride;
  if (fork_parts(g, ws) > ws_bytes) return FLAMIA_ERR_WORKSPACE;
  g.refs = refs;
  g.table = page_table;
  g.lens = lens;
  g.parents = parents;
  g.children = children;
  g.status = dev_status;
  g.nseq = nseq;
  g.num_pages = num_pages;
  g.page_size = page_size;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // (8 rows of 9 slots with the pages of their next tokens 22 us on the host against 37 with two
  // launches and a workspace of the call; 10.5 against 15.7 on the device, reserve as two kernels)
  if (n <= kSmallForks && static_cast<long long>(n) * table_stride <= kSmallSlots)
    return launch_after(fork_small_kernel, dim3(1), kSmallThreads, 0, s, g) ? FLAMIA_OK
                                                                            : FLAMIA_ERR_CUDA;
  return launch_after(fork_read_kernel, dim3(n), kForkThreads, 0, s, g) &&
                 launch_after(fork_write_kernel, dim3(n), kForkThreads, 0, s, g)
             ? FLAMIA_OK
             : FLAMIA_ERR_CUDA;
}

extern "C" size_t flamia_pages_reserve_workspace_bytes(int T, int nseq, int table_stride,
                                                       int page_size) {
  if (!valid_pool(1, page_size, nseq, table_stride) || !valid_batch(T, nseq)) return 0;
  ReserveArgs g{};
  g.nseq = nseq;
  g.cap = static_cast<int>(reserve_slots(T, nseq, table_stride, page_size));
  return reserve_parts(g, nullptr);
}

extern "C" flamia_status flamia_pages_reserve(const flamia_kvcache* cache, int32_t* refs,
                                              int32_t* page_table, int table_stride, int nseq,
                                              int T, const int32_t* cu_seqlens,
                                              const int32_t* starts, int32_t* granted, void* ws,
                                              size_t ws_bytes, int* dev_status, void* stream) {
  const flamia_status st = check_cache(cache);
  if (st != FLAMIA_OK) return st;
  if (!valid_pool(cache->num_pages, cache->page_size, nseq, table_stride) || !valid_batch(T, nseq))
    return FLAMIA_ERR_INVALID_ARG;
  if (T == 0) return FLAMIA_OK;
  if (!valid_books(refs, page_table) || cu_seqlens == nullptr || ws == nullptr ||
      !aligned(ws, 256) || !aligned(granted, 4) || granted == cu_seqlens)
    return FLAMIA_ERR_INVALID_ARG;
  ReserveArgs g{};
  g.nseq = nseq;
  g.cap = static_cast<int>(reserve_slots(T, nseq, table_stride, cache->page_size));
  if (reserve_parts(g, ws) > ws_bytes) return FLAMIA_ERR_WORKSPACE;
  g.refs = refs;
  g.table = page_table;
  g.cu = cu_seqlens;
  g.starts = starts;
  g.granted = granted;
  g.status = dev_status;
  g.T = T;
  g.stride = table_stride;
  g.num_pages = cache->num_pages;
  g.page_size = cache->page_size;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CopyArgs c{};
  c.list = g.list;
  c.count = g.count;
  c.status = dev_status;
  copy_args(c, cache, cache);
  const bool own = makes_copies(cache, nseq);
  const auto kern = !own ? reserve_kernel<0> : cache->d == 128 ? reserve_kernel<128> : reserve_kernel<64>;
  if (!launch_after(kern, dim3(1), kPlan, 0, s, g, c)) return FLAMIA_ERR_CUDA;
  return own ? FLAMIA_OK : launch_copy(c, cache->d, nseq, s);
}

extern "C" size_t flamia_pages_compact_workspace_bytes(int num_pages) {
  if (num_pages <= 0) return 0;
  CompactArgs g{};
  g.num_pages = num_pages;
  return compact_parts(g, nullptr);
}

extern "C" flamia_status flamia_pages_compact(const flamia_kvcache* cache, int32_t* refs,
                                              int32_t* page_table, int table_stride, int nseq,
                                              int32_t* live, void* ws, size_t ws_bytes,
                                              int* dev_status, void* stream) {
  const flamia_status st = check_cache(cache);
  if (st != FLAMIA_OK) return st;
  if (!valid_pool(cache->num_pages, cache->page_size, nseq, table_stride) ||
      !valid_books(refs, page_table) || !aligned(live, 4) || ws == nullptr || !aligned(ws, 256))
    return FLAMIA_ERR_INVALID_ARG;
  CompactArgs g{};
  g.num_pages = cache->num_pages;
  if (compact_parts(g, ws) > ws_bytes) return FLAMIA_ERR_WORKSPACE;
  g.refs = refs;
  g.page_size = cache->page_size;
  g.live_out = live;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CopyArgs c{};
  c.list = g.list;
  c.count = g.count;
  c.status = dev_status;
  c.moved = g.moved;
  c.live = g.live;
  c.table = page_table;
  c.entries = static_cast<long long>(nseq) * table_stride;
  copy_args(c, cache, cache);
  const long long most = cache->num_pages / 2;
  const bool own = makes_copies(cache, most) && c.entries <= kOwnEntries;
  const auto kern = !own ? compact_kernel<0> : cache->d == 128 ? compact_kernel<128> : compact_kernel<64>;
  if (!launch_after(kern, dim3(1), kPlan, 0, s, g, c)) return FLAMIA_ERR_CUDA;
  return own ? FLAMIA_OK : launch_copy(c, cache->d, most, s);
}
