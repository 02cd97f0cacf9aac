// Attention of new tokens over the paged MXFP8 cache.
//
// First form: one warp per (token, head).  32 keys at a time: each lane takes
// one key's score, the warp folds the running maximum and sum of the softmax
// into its float32 output row (d / 32 elements a lane).
#include <cuda_bf16.h>

#include <cmath>

#include "paged.cuh"

namespace flamia {
namespace {

constexpr int kThreads = 128;
constexpr float kLn2 = 0.69314718055994530942f;

struct AttendArgs {
  const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  const int32_t *cu, *starts, *table;
  int* status;
  long long q_stride;
  int T, H, H_kv, ndocs, table_stride, num_pages, page_size, window, sinks;
  float scale_log2;
};

__device__ __forceinline__ float pow2_byte(int byte) {
  return byte > 0 ? __uint_as_float(static_cast<uint32_t>(byte) << 23) : 0x1p-127f;
}

template <int DIM>
__global__ void __launch_bounds__(kThreads) attend_kernel(const AttendArgs g) {
  constexpr int EPL = DIM / 32;
  __shared__ float s_q[kThreads / 32][DIM];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long unit = static_cast<long long>(blockIdx.x) * (kThreads / 32) + warp;
  check_offsets(g.cu, g.ndocs, g.T, static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x,
                static_cast<long long>(gridDim.x) * kThreads, g.status);
  const int t = static_cast<int>(unit / g.H), h = static_cast<int>(unit % g.H);
  if (t >= g.T) return;
  const int b = warp_last_not_above(g.ndocs, t, lane, [&](int i) { return __ldg(g.cu + i); });
  const DocRange r = doc_range(g.cu, b, g.T);
  if (t < r.s || t >= r.e) return;
  const int hk = h / (g.H / g.H_kv);
  const long long pos =
      (g.starts != nullptr ? static_cast<long long>(__ldg(g.starts + b)) : 0) + (t - r.s);
  const __nv_bfloat16* q = g.q + t * g.q_stride + h * DIM;
  for (int i = lane; i < DIM; i += 32) s_q[warp][i] = __bfloat162float(q[i]);
  __syncwarp();
  float m = -INFINITY, l = 0.f, acc[EPL] = {};
  const long long wlo = g.window > 0 ? max(0ll, pos - g.window + 1) : 0;
  for (long long k0 = 0; k0 <= pos; k0 += 32) {
    if (k0 + 31 < wlo && k0 >= g.sinks) continue;
    const long long slot = k0 / g.page_size;
    const int page = slot < g.table_stride
                         ? __ldg(g.table + static_cast<long long>(b) * g.table_stride + slot)
                         : -1;
    if (page < 0 || page >= g.num_pages) {
      if (lane == 0) report(g.status, FLAMIA_DEV_BAD_PAGE);
      continue;
    }
    const long long row = (static_cast<long long>(page) * g.H_kv + hk) * g.page_size +
                          (k0 - slot * g.page_size);
    const long long key = k0 + lane;
    const bool seen = key <= pos && (key >= wlo || key < g.sinks);
    float s = -INFINITY;
    if (seen) {
      float a = 0.f;
      const uint4* kc = reinterpret_cast<const uint4*>(g.k_codes + (row + lane) * DIM);
      for (int i = 0; i < DIM / 16; ++i) {
        const uint4 w = kc[i];
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 u = e4m3x2_to_float2(x[j] & 0xFFFFu), v = e4m3x2_to_float2(x[j] >> 16);
          const float* qq = &s_q[warp][i * 16 + j * 4];
          a += u.x * qq[0] + u.y * qq[1] + v.x * qq[2] + v.y * qq[3];
        }
      }
      s = a * pow2_byte(g.k_scales[row + lane]) * g.scale_log2;
    }
    float mx = s;
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    const float mn = fmaxf(m, mx);
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float f = exp2f(m - ref);
    const float p = seen ? exp2f(s - ref) : 0.f;
    float ps = p;
    for (int off = 16; off > 0; off >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, off);
    l = l * f + ps;
    m = mn;
    const float pv = seen ? p * pow2_byte(g.v_scales[row + lane]) : 0.f;
    const unsigned any = __ballot_sync(0xffffffffu, seen);
#pragma unroll
    for (int i = 0; i < EPL; ++i) acc[i] *= f;
    for (int k = 0; k < 32; ++k) {
      const float w = __shfl_sync(0xffffffffu, pv, k);
      if (!((any >> k) & 1)) continue;
      const uint8_t* vc = g.v_codes + (row + k) * DIM;
#pragma unroll
      for (int i = 0; i < EPL; ++i) acc[i] += w * e4m3x2_to_float2(vc[lane + 32 * i]).x;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    g.o[(static_cast<long long>(t) * g.H + h) * DIM + lane + 32 * i] = __float2bfloat16(acc[i] * inv);
  if (g.lse != nullptr && lane == 0)
    g.lse[static_cast<long long>(h) * g.T + t] = (m + log2f(l)) * kLn2;
}

}  // namespace
}  // namespace flamia

using namespace flamia;

extern "C" size_t flamia_attn_cache_workspace_bytes(int T, int ndocs, int H, int H_kv, int d) {
  if (!supported_dim(d) || !valid_batch(T, ndocs) || H <= 0 || H > 4096 || H_kv <= 0 ||
      H % H_kv != 0)
    return 0;
  return 256;
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
      !(softmax_scale > 0.f) || std::isinf(softmax_scale) || window < 0 || sinks < 0 || (sinks > 0 && window == 0) ||
      static_cast<long long>(T) * H >= (1ll << 31))
    return FLAMIA_ERR_INVALID_ARG;
  if (T == 0) return FLAMIA_OK;
  if (!valid_rows(q_bf16, q_stride) || o_bf16 == nullptr || !aligned(o_bf16, 16) ||
      cu_seqlens == nullptr || page_table == nullptr || ws == nullptr ||
      !aligned(ws, 256) || !aligned(lse, 4))
    return FLAMIA_ERR_INVALID_ARG;
  if (ws_bytes < flamia_attn_cache_workspace_bytes(T, ndocs, H, cache->H_kv, cache->d))
    return FLAMIA_ERR_WORKSPACE;
  AttendArgs g{};
  g.k_codes = cache->k_codes;
  g.k_scales = cache->k_scales;
  g.v_codes = cache->v_codes;
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
  g.ndocs = ndocs;
  g.table_stride = table_stride;
  g.num_pages = cache->num_pages;
  g.page_size = cache->page_size;
  g.window = window;
  g.sinks = sinks;
  g.scale_log2 = softmax_scale * 1.44269504088896340736f;
  const long long units = static_cast<long long>(T) * H;
  const unsigned blocks = static_cast<unsigned>((units * 32 + kThreads - 1) / kThreads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cache->d == 128)
    attend_kernel<128><<<blocks, kThreads, 0, s>>>(g);
  else
    attend_kernel<64><<<blocks, kThreads, 0, s>>>(g);
  count_launches(1);
  return cudaGetLastError() == cudaSuccess ? FLAMIA_OK : FLAMIA_ERR_CUDA;
}
