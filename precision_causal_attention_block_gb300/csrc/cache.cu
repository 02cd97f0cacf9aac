// Paged key-value cache in the quantiser's format: write (quantise BF16 K and
// V rows into it) and read back.
//
// One warp owns one 32-token block of one head of K or V: the block's rows
// (32 x d BF16, 8 or 4 KB) stay in its registers between the maximum and the
// codes, so each element is read once, and no shared memory or block-wide
// barrier is needed.  Blocks are found without a prefix sum over the
// sequences: sequence b owns the block numbers from cu[b] / 32 + 2 b on, which
// leaves room for its ragged first and last block whatever its start.
// HBM-bound: 2 bytes on the BF16 side, 1 code byte and d^-1 scale bytes on the
// other.
#include <cuda_bf16.h>

#include "paged.cuh"

namespace flamia {
namespace {

constexpr int kCacheThreads = 128;

struct CacheArgs {
  uint8_t* codes[2];   // K, V
  uint8_t* scales[2];
  __nv_bfloat16* rows[2];
  long long stride[2];
  const int32_t* cu;
  const int32_t* starts;
  const int32_t* table;
  int* status;
  int T, H_kv, ndocs, table_stride, num_pages, page_size;
  long long units;  // warps of the launch: blocks x heads x {K, V}
};

// The block of one warp: positions [p0, p0 + 32) of a sequence, of which the
// call's tokens are [lo, hi) (as offsets into the block).
struct Block {
  int lo, hi;
  int h, kv;          // head, 0 = K / 1 = V
  int page, in_page;  // its page (-1: none) and first row in it
  long long token;    // packed row of offset 0 (may lie before the document)
  // first row in the codes / scales arrays
  __device__ __forceinline__ long long row(const CacheArgs& g) const {
    return (static_cast<long long>(page) * g.H_kv + h) * g.page_size + in_page;
  }
};

// The page is looked up but not checked: a caller can have the rows' loads
// under way before it looks (valid_page).
__device__ __forceinline__ bool find_block(const CacheArgs& g, long long unit, int lane,
                                           Block& blk) {
  const int per = 2 * g.H_kv;
  const int vb = static_cast<int>(unit / per);
  const int hk = static_cast<int>(unit - static_cast<long long>(vb) * per);
  blk.kv = hk >= g.H_kv;
  blk.h = hk - blk.kv * g.H_kv;
  const int b = warp_last_not_above(
      g.ndocs, vb, lane, [&](int i) { return (g.cu[i] >> 5) + 2 * i; });
  const int start = g.starts != nullptr ? g.starts[b] : 0;
  const DocRange r = doc_range(g.cu, b, g.T);
  if (r.e <= r.s) return false;
  if (start < 0) {
    if (lane == 0) report(g.status, FLAMIA_DEV_BAD_PAGE);
    return false;
  }
  const int j = vb - ((r.s >> 5) + 2 * b);  // block of the sequence's new tokens
  const int lead = start & 31, n = r.e - r.s;
  if (j < 0 || 32ll * j >= static_cast<long long>(lead) + n) return false;
  const long long p0 = static_cast<long long>(start - lead) + 32ll * j;
  blk.lo = j == 0 ? lead : 0;
  blk.hi = static_cast<int>(min(32ll, static_cast<long long>(start) + n - p0));
  const long long slot = p0 / g.page_size;
  blk.page = -1;
  if (slot < g.table_stride)
    blk.page = g.table[static_cast<long long>(b) * g.table_stride + slot];
  blk.in_page = static_cast<int>(p0 - slot * g.page_size);
  blk.token = r.s + p0 - start;
  return true;
}

__device__ __forceinline__ bool valid_page(const CacheArgs& g, const Block& blk, int lane) {
  const bool ok = blk.page >= 0 && blk.page < g.num_pages;
  if (!ok && lane == 0) report(g.status, FLAMIA_DEV_BAD_PAGE);
  return ok;
}

// Magnitudes of a BF16 pair as two 16-bit integers (their order is the
// values'); 0x7F80 and above are infinities and NaN.
__device__ __forceinline__ uint32_t mag(uint32_t w) { return w & 0x7FFF7FFFu; }
__device__ __forceinline__ uint32_t mag(const uint4& x) {
  return __vmaxu2(__vmaxu2(mag(x.x), mag(x.y)), __vmaxu2(mag(x.z), mag(x.w)));
}
// Non-finite elements of a BF16 pair become NaN (their codes then, too); clear:
// become 0 (for the maximum).
__device__ __forceinline__ uint32_t mark(uint32_t w, bool clear) {
  const uint32_t n = clear ? 0u : 0x7FC0u;
  if ((w & 0x7F80u) == 0x7F80u) w = (w & 0xFFFF0000u) | n;
  if ((w & 0x7F800000u) == 0x7F800000u) w = (w & 0x0000FFFFu) | (n << 16);
  return w;
}
__device__ __forceinline__ uint4 mark(const uint4& x, bool clear) {
  return make_uint4(mark(x.x, clear), mark(x.y, clear), mark(x.z, clear), mark(x.w, clear));
}

// 8 BF16 elements times inv, as E4M3 codes.
__device__ __forceinline__ uint2 encode(const uint4& x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  const float2 f = make_float2(inv, inv);
  float2 v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = __fmul2_rn(make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u)), f);
  return make_uint2(cvt_e4m3x4(v[0].x, v[0].y, v[1].x, v[1].y),
                    cvt_e4m3x4(v[2].x, v[2].y, v[3].x, v[3].y));
}

// Instructions, not HBM, would set the pace of a plain loop here: maxima run on
// packed 16-bit integers, products on float pairs, and infinities and NaN are
// looked for once a block (a maximum of 0x7F80 or more) instead of at each
// element.  58,918 tokens x 16 heads x 128: 103 us, 7.0 TB/s (510 us with a check
// at each element and 178 registers, 199 with 96 registers).  With an exponent a
// token, 3 or 4 shuffles an access come on top: 142 us.
template <int DIM, bool TOK>
__global__ void __launch_bounds__(kCacheThreads, 5) cache_write_kernel(const CacheArgs g) {
  constexpr int LPR = DIM / 8;   // lanes per row: 8 elements each
  constexpr int RPI = 32 / LPR;  // rows per warp-wide access
  constexpr int NLD = 32 / RPI;  // accesses per block
  const int lane = threadIdx.x & 31;
  const long long unit =
      static_cast<long long>(blockIdx.x) * (kCacheThreads / 32) + (threadIdx.x >> 5);
  start_next();
  wait_for_previous();
  check_offsets(g.cu, g.ndocs, g.T,
                static_cast<long long>(blockIdx.x) * kCacheThreads + threadIdx.x,
                static_cast<long long>(gridDim.x) * kCacheThreads, g.status);
  Block blk;
  if (unit >= g.units || !find_block(g, unit, lane, blk)) return;
  const int sub = lane / LPR, chunk = lane % LPR;
  const long long stride = blk.kv ? g.stride[1] : g.stride[0];
  const __nv_bfloat16* src =
      (blk.kv ? g.rows[1] : g.rows[0]) + (blk.token + sub) * stride + blk.h * DIM + chunk * 8;
  const bool full = blk.lo == 0 && blk.hi == 32;

  uint4 x[NLD];
  if (full) {
#pragma unroll
    for (int i = 0; i < NLD; ++i)
      x[i] = *reinterpret_cast<const uint4*>(src + i * RPI * stride);
  } else {
#pragma unroll
    for (int i = 0; i < NLD; ++i) {
      const int r = i * RPI + sub;
      x[i] = make_uint4(0, 0, 0, 0);
      if (r >= blk.lo && r < blk.hi)
        x[i] = *reinterpret_cast<const uint4*>(src + i * RPI * stride);
    }
  }
  if (!valid_page(g, blk, lane)) return;
  const long long row = blk.row(g);
  uint8_t* codes = (blk.kv ? g.codes[1] : g.codes[0]) + row * DIM;
  uint8_t* scales = (blk.kv ? g.scales[1] : g.scales[0]) + row;
  // what the block holds before the call (a lane's row) keeps its exponent, or a larger
  // one; rows that were written again may have exponents of their own
  int held = -127;
  if (!TOK && lane < blk.lo) held = static_cast<int>(scales[lane]) - 127;

  uint32_t all = 0;
#pragma unroll
  for (int i = 0; i < NLD; ++i) all = __vmaxu2(all, mag(x[i]));
  all = __reduce_max_sync(0xffffffffu, max(all & 0xFFFFu, all >> 16));
  if (all >= 0x7F80u) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < NLD; ++i) {
      a = __vmaxu2(a, mag(mark(x[i], true)));
      x[i] = mark(x[i], false);
    }
    all = __reduce_max_sync(0xffffffffu, max(a & 0xFFFFu, a >> 16));
  }
  uint2* out = reinterpret_cast<uint2*>(codes + sub * DIM) + chunk;
  if constexpr (TOK) {
#pragma unroll
    for (int i = 0; i < NLD; ++i) {
      const int r = i * RPI + sub;
      uint32_t m = mag(mark(x[i], true));
      m = max(m & 0xFFFFu, m >> 16);
#pragma unroll
      for (int off = LPR / 2; off > 0; off >>= 1)
        m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
      const int e = roundup_exponent(__uint_as_float(m << 16));
      if (r >= blk.lo && r < blk.hi) {
        out[i * RPI * (DIM / 8)] = encode(x[i], exp2i(-e));
        if (chunk == 0) scales[r] = static_cast<uint8_t>(e + 127);
      }
    }
  } else {
    int e = roundup_exponent(__uint_as_float(all << 16));
    if (blk.lo > 0) e = max(e, __reduce_max_sync(0xffffffffu, held));
    const float inv = exp2i(-e);  // e in [-127, 120]: 2^-e is a normal float
    if (full) {
#pragma unroll
      for (int i = 0; i < NLD; ++i) out[i * RPI * (DIM / 8)] = encode(x[i], inv);
      scales[lane] = static_cast<uint8_t>(e + 127);
    } else {
#pragma unroll
      for (int i = 0; i < NLD; ++i) {
        const int r = i * RPI + sub;
        if (r >= blk.lo && r < blk.hi) out[i * RPI * (DIM / 8)] = encode(x[i], inv);
      }
      const bool grew = lane < blk.lo && e > held;
      if (lane < blk.hi && (lane >= blk.lo || grew)) scales[lane] = static_cast<uint8_t>(e + 127);
      const unsigned again = __ballot_sync(0xffffffffu, grew);
      if (again) {
        // held codes are rounded again under a larger exponent
#pragma unroll 1
        for (int r0 = 0; r0 < blk.lo; r0 += RPI) {
          const int r = r0 + sub;  // (below 32)
          const int by = __shfl_sync(0xffffffffu, held, r) - e;
          if ((again >> r) & 1) {
            const float f = by < -126 ? 0.f : exp2i(by);
            uint2* at = reinterpret_cast<uint2*>(codes + r * DIM) + chunk;
            uint2 c = *at;
            const float2 v0 = e4m3x2_to_float2(c.x & 0xFFFFu), v1 = e4m3x2_to_float2(c.x >> 16);
            const float2 v2 = e4m3x2_to_float2(c.y & 0xFFFFu), v3 = e4m3x2_to_float2(c.y >> 16);
            c.x = cvt_e4m3x4(v0.x * f, v0.y * f, v1.x * f, v1.y * f);
            c.y = cvt_e4m3x4(v2.x * f, v2.y * f, v3.x * f, v3.y * f);
            *at = c;
          }
        }
      }
    }
  }
}

// 79,477 tokens x 16 heads x 128: 144 us, 6.8 TB/s.
template <int DIM>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const CacheArgs g) {
  constexpr int LPR = DIM / 8;
  constexpr int RPI = 32 / LPR;
  constexpr int NLD = 32 / RPI;
  const int lane = threadIdx.x & 31;
  const long long unit =
      static_cast<long long>(blockIdx.x) * (kCacheThreads / 32) + (threadIdx.x >> 5);
  start_next();
  wait_for_previous();
  check_offsets(g.cu, g.ndocs, g.T,
                static_cast<long long>(blockIdx.x) * kCacheThreads + threadIdx.x,
                static_cast<long long>(gridDim.x) * kCacheThreads, g.status);
  Block blk;
  if (unit >= g.units || !find_block(g, unit, lane, blk) || !valid_page(g, blk, lane)) return;
  const int sub = lane / LPR, chunk = lane % LPR;
  __nv_bfloat16* rows = blk.kv ? g.rows[1] : g.rows[0];
  const long long stride = blk.kv ? g.stride[1] : g.stride[0];
  const long long row = blk.row(g);
  const uint8_t* codes = (blk.kv ? g.codes[1] : g.codes[0]) + row * DIM;
  const uint8_t* scales = (blk.kv ? g.scales[1] : g.scales[0]) + row;
  uint2 x[NLD];
#pragma unroll
  for (int i = 0; i < NLD; ++i) {
    const int r = i * RPI + sub;
    x[i] = make_uint2(0, 0);
    if (r >= blk.lo && r < blk.hi) x[i] = reinterpret_cast<const uint2*>(codes + r * DIM)[chunk];
  }
  const int sc = scales[lane];
#pragma unroll
  for (int i = 0; i < NLD; ++i) {
    const int r = i * RPI + sub;
    const int byte = __shfl_sync(0xffffffffu, sc, r);
    const float f = byte > 0 ? __uint_as_float(static_cast<uint32_t>(byte) << 23) : 0x1p-127f;
    if (r >= blk.lo && r < blk.hi) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = e4m3x2_to_float2(((j < 2 ? x[i].x : x[i].y) >> (16 * (j & 1))) & 0xFFFFu);
        const __nv_bfloat162 p = __floats2bfloat162_rn(v.x * f, v.y * f);
        w[j] = *reinterpret_cast<const uint32_t*>(&p);
      }
      *reinterpret_cast<uint4*>(rows + (blk.token + r) * stride + blk.h * DIM + chunk * 8) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

flamia_status fill_args(CacheArgs& g, const flamia_kvcache* cache, const void* k, int64_t k_stride,
                        const void* v, int64_t v_stride, int T, const int32_t* cu, int ndocs,
                        const int32_t* starts, const int32_t* table, int table_stride,
                        int* status) {
  const flamia_status st = check_cache(cache);
  if (st != FLAMIA_OK) return st;
  if (!valid_batch(T, ndocs) || table_stride <= 0) return FLAMIA_ERR_INVALID_ARG;
  if (T == 0) return FLAMIA_OK;
  if (!valid_rows(k, k_stride) || !valid_rows(v, v_stride) || cu == nullptr || table == nullptr)
    return FLAMIA_ERR_INVALID_ARG;
  g.codes[0] = cache->k_codes;
  g.codes[1] = cache->v_codes;
  g.scales[0] = cache->k_scales;
  g.scales[1] = cache->v_scales;
  g.rows[0] = static_cast<__nv_bfloat16*>(const_cast<void*>(k));
  g.rows[1] = static_cast<__nv_bfloat16*>(const_cast<void*>(v));
  g.stride[0] = k_stride;
  g.stride[1] = v_stride;
  g.cu = cu;
  g.starts = starts;
  g.table = table;
  g.status = status;
  g.T = T;
  g.H_kv = cache->H_kv;
  g.ndocs = ndocs;
  g.table_stride = table_stride;
  g.num_pages = cache->num_pages;
  g.page_size = cache->page_size;
  // block numbers run to cu[ndocs] / 32 + 2 ndocs
  g.units = (static_cast<long long>(T) / 32 + 2ll * ndocs) * 2 * g.H_kv;
  return FLAMIA_OK;
}

flamia_status launch(void (*kern)(const CacheArgs), const CacheArgs& g, cudaStream_t s) {
  const long long blocks = (g.units * 32 + kCacheThreads - 1) / kCacheThreads;
  if (blocks >= (1ll << 31)) return FLAMIA_ERR_INVALID_ARG;
  return launch_after(kern, dim3(static_cast<unsigned>(blocks)), kCacheThreads, 0, s, g)
             ? FLAMIA_OK
             : FLAMIA_ERR_CUDA;
}

}  // namespace
}  // namespace flamia

using namespace flamia;

extern "C" flamia_status flamia_cache_write(const flamia_kvcache* cache, const void* k_bf16,
                                            int64_t k_stride, const void* v_bf16,
                                            int64_t v_stride, int T, const int32_t* cu_seqlens,
                                            int ndocs, const int32_t* starts,
                                            const int32_t* page_table, int table_stride,
                                            int format, int* dev_status, void* stream) {
  if (format != FLAMIA_FORMAT_MXFP8 && format != FLAMIA_FORMAT_TOKEN_SCALES)
    return FLAMIA_ERR_UNSUPPORTED;
  CacheArgs g{};
  const flamia_status st = fill_args(g, cache, k_bf16, k_stride, v_bf16, v_stride, T, cu_seqlens,
                                     ndocs, starts, page_table, table_stride, dev_status);
  if (st != FLAMIA_OK || T == 0) return st;
  const bool tok = format == FLAMIA_FORMAT_TOKEN_SCALES;
  return launch(cache->d == 128
                    ? (tok ? cache_write_kernel<128, true> : cache_write_kernel<128, false>)
                    : (tok ? cache_write_kernel<64, true> : cache_write_kernel<64, false>),
                g, static_cast<cudaStream_t>(stream));
}

extern "C" flamia_status flamia_cache_read(const flamia_kvcache* cache, void* k_bf16,
                                           int64_t k_stride, void* v_bf16, int64_t v_stride,
                                           int T, const int32_t* cu_seqlens, int ndocs,
                                           const int32_t* starts, const int32_t* page_table,
                                           int table_stride, int* dev_status, void* stream) {
  CacheArgs g{};
  const flamia_status st = fill_args(g, cache, k_bf16, k_stride, v_bf16, v_stride, T, cu_seqlens,
                                     ndocs, starts, page_table, table_stride, dev_status);
  if (st != FLAMIA_OK || T == 0) return st;
  const int64_t row = static_cast<int64_t>(cache->H_kv) * cache->d;
  if (T > 1 && (k_stride < row || v_stride < row)) return FLAMIA_ERR_INVALID_ARG;
  return launch(cache->d == 128 ? cache_read_kernel<128> : cache_read_kernel<64>, g,
                static_cast<cudaStream_t>(stream));
}
