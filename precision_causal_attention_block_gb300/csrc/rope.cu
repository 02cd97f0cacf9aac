// Rotary positions of Q and K, and of dQ and dK (the transpose).
//
// Pair i of a row at position p turns by p * turns[i] / 2^64 of a circle.  The
// product is taken modulo 2^64, so whole turns drop out exactly at any
// position.  The top 32 bits of what is left are the angle, rounded to float32 for
// sine and cosine (an error of 2^-26 turns): no float64 (this GPU runs it at a small
// fraction of its float32 rate) and no table of cosines to read.
//
// A CTA takes kTok tokens: its threads work out the tokens' cosines and sines
// once, pass them through shared memory, and each keeps those of one 16-element
// unit of the row (8 pairs) in registers while it walks the heads of Q and K.
// HBM-bound: 2 bytes read and 2 written per element.  131,072 tokens x 64 heads of
// 64: 300 us, 7.1 TB/s of reads and writes.
//
// With several axes (time, height, width of a picture's patches) each pair takes the
// position of its own axis, and the caller gives the positions of every token: no
// document has to be looked for, and the rest is the same (131,072 tokens, 32 + 32 heads
// of 64, three axes, interleaved, transposed: 306 us, 7.0 TB/s).
#include <cuda_bf16.h>

#include <climits>
#include <cmath>

#include "paged.cuh"

namespace flamia {
namespace {

constexpr int kRopeThreads = 256;

struct RopeArgs {
  const __nv_bfloat16* q_in;
  __nv_bfloat16* q_out;
  const __nv_bfloat16* k_in;
  __nv_bfloat16* k_out;
  long long q_in_stride, q_out_stride, k_in_stride, k_out_stride;
  const unsigned long long* turns;
  const int32_t* cu;
  const int32_t* starts;
  const uint8_t* axes;       // of each pair, with positions [naxes][pos_stride]
  const int32_t* positions;
  long long pos_stride;
  int* status;
  int T, H, H_kv, ndocs, rot, naxes;
  float mscale, sign;
};

__device__ __forceinline__ void unpack(const uint4& w, float (&v)[8]) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(x[i] << 16);
    v[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack(const float (&v)[8]) {
  uint32_t x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    x[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

template <int DIM, int kTok, bool INTER, bool AXES>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs g) {
  constexpr int kUnits = DIM / 16;                       // 16-element units of a row
  constexpr int kLanes = kRopeThreads / kUnits / kTok;   // heads walked side by side
  __shared__ float2 s_trig[kTok][DIM / 2];
  __shared__ int s_pos[kTok];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t0 = blockIdx.x * kTok;
  const int unit = tid % kUnits, hl = (tid / kUnits) % kLanes, tk = tid / (kUnits * kLanes);
  const int t = t0 + tk;
  const bool turn = unit * 16 < g.rot;
  const int half = g.rot / 2;
  // the unit's two 8-element chunks: both halves of its pairs, or 16
  // neighbouring elements (interleaved pairs, or the part that is copied)
  const int c0 = (INTER || !turn) ? unit * 16 : unit * 8;
  const int c1 = (INTER || !turn) ? c0 + 8 : c0 + half;
  const int heads = g.H + g.H_kv;
  // kBatch heads at a time: all their loads before the first store (the
  // compiler cannot move loads over stores that may alias them).  With one
  // token a CTA, where latency counts, those of the first batch come before the
  // positions and angles are worked out (a decode step of 16 tokens: 3.0 -> 2.7
  // us; with four, other CTAs fill the wait, and registers count: 16,384 tokens
  // x 32 heads 45.5 us without, 47.3 with it).
  constexpr int kBatch = 4;
  uint4 w0[kBatch], w1[kBatch];
  auto load = [&](int h0) {
    const __nv_bfloat16* qi = g.q_in + t * g.q_in_stride;
    const __nv_bfloat16* ki = g.k_in + t * g.k_in_stride;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int h = h0 + j * kLanes;
      if (h < heads) {
        const __nv_bfloat16* in = h < g.H ? qi + h * DIM : ki + (h - g.H) * DIM;
        w0[j] = *reinterpret_cast<const uint4*>(in + c0);
        w1[j] = *reinterpret_cast<const uint4*>(in + c1);
      }
    }
  };
  start_next();
  wait_for_previous();
  if (kTok == 1 && t < g.T) load(hl);

  check_offsets(g.cu, g.ndocs, g.T, static_cast<long long>(blockIdx.x) * kRopeThreads + tid,
                static_cast<long long>(gridDim.x) * kRopeThreads, g.status);
  // position of each token (INT_MIN: in no document; with axes 0 stands for its own)
  if (warp < kTok) {
    const int t = t0 + warp;
    int pos = INT_MIN;
    if (AXES) {
      if (t < min(g.cu[g.ndocs], g.T)) pos = 0;
    } else if (t < g.T) {
      const int b = warp_last_not_above(g.ndocs, t, lane, [&](int i) { return g.cu[i]; });
      const DocRange r = doc_range(g.cu, b, g.T);
      if (t >= r.s && t < r.e) pos = (g.starts != nullptr ? g.starts[b] : 0) + t - r.s;
    }
    if (lane == 0) s_pos[warp] = pos;
  }
  __syncthreads();
  for (int i = tid; i < kTok * half; i += kRopeThreads) {
    const int tk = i / half, pair = i - tk * half;
    int pos = s_pos[tk];
    if (AXES && pos != INT_MIN)
      pos = g.positions[min(static_cast<int>(g.axes[pair]), g.naxes - 1) * g.pos_stride + t0 + tk];
    const unsigned long long ph =
        static_cast<unsigned long long>(static_cast<long long>(pos)) * g.turns[pair];
    float sn, cs;
    sincospif(static_cast<float>(static_cast<int>(ph >> 32)) * 0x1p-31f, &sn, &cs);
    s_trig[tk][pair] = make_float2(cs * g.mscale, sn * g.mscale * g.sign);
  }
  __syncthreads();

  if (s_pos[tk] == INT_MIN) return;
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 w = turn ? s_trig[tk][unit * 8 + i] : make_float2(1.f, 0.f);
    cs[i] = w.x;
    sn[i] = w.y;
  }
  __nv_bfloat16* qo = g.q_out + t * g.q_out_stride;
  __nv_bfloat16* ko = g.k_out + t * g.k_out_stride;
  for (int h0 = hl; h0 < heads; h0 += kBatch * kLanes) {
    if (kTok != 1 || h0 != hl) load(h0);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int h = h0 + j * kLanes;
      if (h >= heads) break;
      __nv_bfloat16* out = h < g.H ? qo + h * DIM : ko + (h - g.H) * DIM;
      if (turn) {
        float x[8], y[8], u[8], v[8];
        unpack(w0[j], x);
        unpack(w1[j], y);
        if (INTER) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            u[2 * i] = x[2 * i] * cs[i] - x[2 * i + 1] * sn[i];
            u[2 * i + 1] = x[2 * i] * sn[i] + x[2 * i + 1] * cs[i];
            v[2 * i] = y[2 * i] * cs[4 + i] - y[2 * i + 1] * sn[4 + i];
            v[2 * i + 1] = y[2 * i] * sn[4 + i] + y[2 * i + 1] * cs[4 + i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            u[i] = x[i] * cs[i] - y[i] * sn[i];
            v[i] = x[i] * sn[i] + y[i] * cs[i];
          }
        }
        w0[j] = pack(u);
        w1[j] = pack(v);
      }
      *reinterpret_cast<uint4*>(out + c0) = w0[j];
      *reinterpret_cast<uint4*>(out + c1) = w1[j];
    }
  }
}

template <int DIM, bool AXES>
bool launch(const RopeArgs& g, bool inter, cudaStream_t s) {
  // Four tokens a CTA share its set-up; with few tokens one each, so that a
  // decode step's heads spread over the GPU (40 heads of 128, one against four:
  // 300 tokens 2.9 us against 3.4, 600 tokens 3.8 against 3.6, 4,800 tokens 21.4
  // against 15.8).
  const bool few = g.T < 3 * 152;
  const int tok = few ? 1 : 4;
  const int grid = (g.T + tok - 1) / tok;
  auto kern = few ? (inter ? rope_kernel<DIM, 1, true, AXES> : rope_kernel<DIM, 1, false, AXES>)
                  : (inter ? rope_kernel<DIM, 4, true, AXES> : rope_kernel<DIM, 4, false, AXES>);
  return launch_after(kern, dim3(grid), kRopeThreads, 0, s, g);
}

// Both entry points: `g` holds the positions (or starts) already.
template <bool AXES>
flamia_status rope(RopeArgs g, const void* q_in, void* q_out, int64_t q_in_stride,
                   int64_t q_out_stride, const void* k_in, void* k_out, int64_t k_in_stride,
                   int64_t k_out_stride, int T, int H, int H_kv, int d, const uint64_t* turns,
                   int rot_dim, float mscale, int flags, const int32_t* cu_seqlens, int ndocs,
                   int* dev_status, void* stream) {
  if (!supported_dim(d)) return FLAMIA_ERR_UNSUPPORTED;
  if (flags & ~(FLAMIA_FLAG_ROPE_INTERLEAVED | FLAMIA_FLAG_ROPE_INVERSE))
    return FLAMIA_ERR_UNSUPPORTED;
  if (rot_dim < 16 || rot_dim > d || rot_dim % 16 != 0) return FLAMIA_ERR_UNSUPPORTED;
  if (!valid_batch(T, ndocs) || H <= 0 || H > 4096 || H_kv < 0 || H_kv > 4096 ||
      !std::isfinite(mscale))
    return FLAMIA_ERR_INVALID_ARG;
  if (AXES && (g.naxes < 1 || g.naxes > rot_dim / 2 || g.pos_stride < 0 ||
               g.pos_stride >= (1ll << 40)))
    return FLAMIA_ERR_INVALID_ARG;
  if (T == 0) return FLAMIA_OK;
  if (turns == nullptr || cu_seqlens == nullptr || !aligned(turns, 8))
    return FLAMIA_ERR_INVALID_ARG;
  if (AXES && (g.axes == nullptr || g.positions == nullptr || !aligned(g.positions, 4)))
    return FLAMIA_ERR_INVALID_ARG;
  if (!valid_rows(q_in, q_in_stride) || !valid_rows(q_out, q_out_stride) ||
      (T > 1 && q_out_stride < static_cast<int64_t>(H) * d) ||
      (q_in == q_out && q_in_stride != q_out_stride))
    return FLAMIA_ERR_INVALID_ARG;
  if (H_kv > 0 && (!valid_rows(k_in, k_in_stride) || !valid_rows(k_out, k_out_stride) ||
                   (T > 1 && k_out_stride < static_cast<int64_t>(H_kv) * d) ||
                   (k_in == k_out && k_in_stride != k_out_stride)))
    return FLAMIA_ERR_INVALID_ARG;
  g.q_in = static_cast<const __nv_bfloat16*>(q_in);
  g.q_out = static_cast<__nv_bfloat16*>(q_out);
  g.k_in = static_cast<const __nv_bfloat16*>(k_in);
  g.k_out = static_cast<__nv_bfloat16*>(k_out);
  g.q_in_stride = q_in_stride;
  g.q_out_stride = q_out_stride;
  g.k_in_stride = k_in_stride;
  g.k_out_stride = k_out_stride;
  g.turns = reinterpret_cast<const unsigned long long*>(turns);
  g.cu = cu_seqlens;
  g.status = dev_status;
  g.T = T;
  g.H = H;
  g.H_kv = H_kv;
  g.ndocs = ndocs;
  g.rot = rot_dim;
  g.mscale = mscale;
  g.sign = (flags & FLAMIA_FLAG_ROPE_INVERSE) ? -1.f : 1.f;
  const bool inter = (flags & FLAMIA_FLAG_ROPE_INTERLEAVED) != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return (d == 128 ? launch<128, AXES>(g, inter, s) : launch<64, AXES>(g, inter, s))
             ? FLAMIA_OK
             : FLAMIA_ERR_CUDA;
}

}  // namespace
}  // namespace flamia

using namespace flamia;

extern "C" flamia_status flamia_rope(const void* q_in, void* q_out, int64_t q_in_stride,
                                     int64_t q_out_stride, const void* k_in, void* k_out,
                                     int64_t k_in_stride, int64_t k_out_stride, int T, int H,
                                     int H_kv, int d, const uint64_t* turns, int rot_dim,
                                     float mscale, int flags, const int32_t* cu_seqlens,
                                     int ndocs, const int32_t* starts, int* dev_status,
                                     void* stream) {
  RopeArgs g{};
  g.starts = starts;
  return rope<false>(g, q_in, q_out, q_in_stride, q_out_stride, k_in, k_out, k_in_stride,
                     k_out_stride, T, H, H_kv, d, turns, rot_dim, mscale, flags, cu_seqlens, ndocs,
                     dev_status, stream);
}

extern "C" flamia_status flamia_rope_axes(const void* q_in, void* q_out, int64_t q_in_stride,
                                          int64_t q_out_stride, const void* k_in, void* k_out,
                                          int64_t k_in_stride, int64_t k_out_stride, int T, int H,
                                          int H_kv, int d, const uint64_t* turns,
                                          const uint8_t* axes, int rot_dim, float mscale, int flags,
                                          const int32_t* positions, int64_t pos_stride, int naxes,
                                          const int32_t* cu_seqlens, int ndocs, int* dev_status,
                                          void* stream) {
  RopeArgs g{};
  g.axes = axes;
  g.positions = positions;
  g.pos_stride = pos_stride;
  g.naxes = naxes;
  return rope<true>(g, q_in, q_out, q_in_stride, q_out_stride, k_in, k_out, k_in_stride,
                    k_out_stride, T, H, H_kv, d, turns, rot_dim, mscale, flags, cu_seqlens, ndocs,
                    dev_status, stream);
}
