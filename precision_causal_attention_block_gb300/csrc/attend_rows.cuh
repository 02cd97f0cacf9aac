// Shared by the kernels that take 256 query rows of a K / V head as the tensor core's M
// (attn_cache_rows.cu, attn_prefix_rows.cu): FP16 products, operand tiles, and codes on
// their way from the cache into them.
#pragma once

#include "attend.cuh"

namespace flamia {

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

// Operand tiles of FP16 numbers.
template <int DIM>
struct RowsCfg {
  static constexpr int kRows = 256;
  static constexpr int kThreads = 512;  // (14 and 15 idle: registers move by four warps)
  static constexpr int kBlock = 128 * 128;            // 64 columns of 128 rows, bytes
  static constexpr int kTileBytes = DIM / 64 * kBlock;
  static constexpr uint32_t kColO = 256;
};

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

// Four E4M3 codes as FP16 pairs (exact; NaN stays).
__device__ __forceinline__ void halves_of_codes(uint32_t codes, uint32_t& a, uint32_t& b) {
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(codes));
}

// Byte offset of 16-byte chunk j of a row in an FP16 operand tile: blocks of 64
// columns, rows of 128 bytes, chunks swizzled as the 128-byte mode does.
template <int DIM>
__device__ __forceinline__ uint32_t tile_at(int row, int j) {
  return (j >> 3) * RowsCfg<DIM>::kBlock + row * 128 + (((j & 7) ^ (row & 7)) << 4);
}

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
      for (int j = 0; j < 4; ++j) halves_of_codes(x[j], h[2 * j], h[2 * j + 1]);
      // (the lanes of a row's second half store the other chunk first: no bank
      // conflicts)
      const uint4 a = make_uint4(h[0], h[1], h[2], h[3]), b = make_uint4(h[4], h[5], h[6], h[7]);
      const bool turn = c >= 4;
      sts128(tile + tile_at<DIM>(r, 2 * c + turn), turn ? b : a);
      sts128(tile + tile_at<DIM>(r, 2 * c + !turn), turn ? a : b);
    }
  }
};

}  // namespace flamia
