// Shared by the rotary kernel and the paged-cache kernels: packed documents
// that may end before the last row, page lookup, host argument checks.
#pragma once

#include "common.cuh"
#include "ptx.cuh"

namespace flamia {

// Largest number of sequences of a rotary or cache call.
constexpr int kMaxSeqs = 1 << 20;

// A document's token range [s, e) clamped to [0, T] (malformed offsets give
// an empty or shortened one; check_offsets reports them).
struct DocRange {
  int s, e;
};
__device__ __forceinline__ DocRange doc_range(const int32_t* cu, int b, int T) {
  DocRange r;
  r.s = min(max(cu[b], 0), T);
  r.e = min(max(cu[b + 1], r.s), T);
  return r;
}

// Largest b in [0, n) with key(b) <= x for non-decreasing key with key(0) <=
// x, found by a whole converged warp: every step 32 probes inside (lo, hi), so
// up to 33 sequences cost one dependent load and 1,000 two.  Every step
// shrinks the interval, so it ends on any input; the caller checks what it gets.
template <class Key>
__device__ __forceinline__ int warp_last_not_above(int n, int x, int lane, Key key) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int span = hi - lo;
    const int p = span <= 33 ? min(lo + 1 + lane, hi - 1)
                             : lo + static_cast<int>((static_cast<long long>(lane + 1) * span) / 33);
    const unsigned below = __ballot_sync(0xffffffffu, key(p) <= x);
    const int k = __ffs(~below) - 1;  // leading lanes whose probe is not above x (-1: all)
    const int last = __shfl_sync(0xffffffffu, p, k < 0 ? 31 : max(k - 1, 0));
    const int next = __shfl_sync(0xffffffffu, p, max(k, 0));
    if (k != 0) lo = last;
    if (k >= 0) hi = next;
    if (span <= 33) break;  // every inner point was probed
  }
  return lo;
}

// Light validation of cu_seqlens, spread over a grid's threads.
__device__ __forceinline__ void check_offsets(const int32_t* cu, int ndocs, int T,
                                              long long thread, long long nthreads, int* status) {
  for (long long i = thread; i < ndocs; i += nthreads)
    if (cu[i] > cu[i + 1]) report(status, FLAMIA_DEV_BAD_SEQLENS);
  if (thread == 0 && (cu[0] != 0 || cu[ndocs] > T))
    report(status, FLAMIA_DEV_BAD_SEQLENS);
}

// Programmatic dependent launch: the serving kernels follow one another closely
// (rotary, cache write, attention, join), so each is launched with
// launch_after, which lets its CTAs start while the kernel before it in the
// stream drains, and begins with wait_for_previous: nothing is read or written
// before that kernel has completed.  start_next lets the kernel behind it do the
// same.  A kernel's lifetime then begins before the end of the one that writes its
// inputs, so all of them (rows, codes, scales, offsets, positions, page tables) are
// read by ordinary loads behind the wait and through pointers without __restrict__,
// never as read-only data (__ldg), which neither the wait nor its clobber binds.
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void start_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <class... P, class... A>
inline bool launch_after(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                         const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) {
    cudaGetLastError();  // (not left behind for the caller's next check)
    return false;
  }
  count_launches(1);
  return true;
}

// Host checks shared by the cache calls.
inline flamia_status check_cache(const flamia_kvcache* c) {
  if (c == nullptr || c->k_codes == nullptr || c->k_scales == nullptr || c->v_codes == nullptr ||
      c->v_scales == nullptr)
    return FLAMIA_ERR_INVALID_ARG;
  if (!supported_dim(c->d)) return FLAMIA_ERR_UNSUPPORTED;
  if (c->page_size <= 0 || c->page_size > (1 << 20) ||
      !(c->page_size == 32 || c->page_size == 64 || c->page_size % 128 == 0))
    return FLAMIA_ERR_UNSUPPORTED;
  if (c->num_pages <= 0 || c->H_kv <= 0 || c->H_kv > 4096 ||
      static_cast<long long>(c->num_pages) * c->H_kv >= (1ll << 31))
    return FLAMIA_ERR_INVALID_ARG;
  if (!aligned(c->k_codes, 128) || !aligned(c->v_codes, 128) || !aligned(c->k_scales, 32) ||
      !aligned(c->v_scales, 32))
    return FLAMIA_ERR_INVALID_ARG;
  return FLAMIA_OK;
}

// A strided BF16 row tensor [T][heads][d]: 16-byte aligned rows.
inline bool valid_rows(const void* x, int64_t stride) {
  return x != nullptr && aligned(x, 16) && stride >= 0 && stride % 8 == 0 &&
         stride < (1ll << 40);
}

inline bool valid_batch(int T, int ndocs) {
  return T >= 0 && T <= kMaxTokens && ndocs >= 1 && ndocs <= kMaxSeqs;
}

}  // namespace flamia
