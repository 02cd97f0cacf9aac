/*
 * flamia.h -- C ABI of the token-block microscaled (MXFP8) causal flash
 * attention hot path for one GB300 (sm_103a) GPU.
 *
 * The method is the one described in "FLAMIA: FLAsh MIcroscaling Attention
 * for Fast and Causally Safe Training on Blackwell" (review page
 * jaehun.me/en/posts/paper-2611-03344v1, sections cited per entry point; and
 * the summary page agihunt.info/en/papers/2611.03344).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Packed layout.  Documents are concatenated along the token axis.  A tensor
 *   "[T, H, d]" is row-major (token, head, dim) with no padding.
 *   cu_seqlens is int32[ndocs + 1] in DEVICE memory: document b is tokens
 *   [cu_seqlens[b], cu_seqlens[b+1]); cu_seqlens[0] == 0, cu_seqlens[ndocs]
 *   == T, non-decreasing (empty documents are allowed).
 * - Ownership.  Every pointer argument is a DEVICE pointer owned by the caller
 *   unless stated otherwise.  The library never allocates, frees or
 *   synchronises, and never reads device data on the host.  All work is
 *   enqueued on `stream` (a cudaStream_t, NULL = legacy default stream).
 * - Errors.  Argument errors found on the host return a flamia_status and
 *   enqueue nothing.  Errors found on the device (malformed cu_seqlens,
 *   capacity overflow, a bounded wait that timed out) are OR-ed into the
 *   int at `dev_status` (device memory, may be NULL to ignore) as
 *   FLAMIA_DEV_* bits; read it after synchronising the stream.  No kernel
 *   traps or spins without bound.
 * - Support.  head_dim d in {64, 128}; 1 <= H <= 4096; T <= 2^20 tokens,
 *   T * H < 2^31, T * H * d < 2^40; multi-head attention, and grouped K / V
 *   heads through the _gqa entry points; causal masking, or none with
 *   FLAMIA_FLAG_NONCAUSAL.  Larger sizes return FLAMIA_ERR_INVALID_ARG.
 * - Formats.  E4M3 = OCP FP8 E4M3FN (bias 7, max 448, subnormals kept).
 *   E8M0 = 2^(byte - 127).  E2M1 = {0, .5, 1, 1.5, 2, 3, 4, 6} with sign,
 *   two codes per byte, element 2i in the low nibble.
 */
#ifndef FLAMIA_H
#define FLAMIA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FLAMIA_OK = 0,
  FLAMIA_ERR_INVALID_ARG = 1,   /* null pointer, bad size, misaligned buffer      */
  FLAMIA_ERR_UNSUPPORTED = 2,   /* d not in {64,128}, unknown format or flag      */
  FLAMIA_ERR_WORKSPACE = 3,     /* workspace / work-list buffer too small         */
  FLAMIA_ERR_CUDA = 4           /* a CUDA runtime call failed (launch, memset)    */
} flamia_status;

/* Bits OR-ed into *dev_status by the kernels. */
#define FLAMIA_DEV_BAD_SEQLENS 0x1  /* cu_seqlens not monotone or not ending at T */
#define FLAMIA_DEV_CAPACITY    0x2  /* more work items than the buffer holds, or
                                       more pages asked for than are free        */
#define FLAMIA_DEV_TIMEOUT     0x4  /* a bounded wait gave up; outputs invalid    */
#define FLAMIA_DEV_RANGE       0x8  /* a scale exponent left the E8M0 range a mode
                                       supports (per-token operand scales with
                                       |V| near 2^96 or beyond); outputs invalid */
#define FLAMIA_DEV_BAD_PAGE    0x10 /* a page-table entry that a call needs lies outside
                                       [0, num_pages), or a sequence's positions
                                       outside its table, or a sequence outside the
                                       page table; that page is neither read nor
                                       written                                   */

/* Quantiser output formats. */
#define FLAMIA_FORMAT_MXFP8       0 /* E4M3 codes + per-token E8M0 scales          */
#define FLAMIA_FORMAT_MXFP8_NVFP4 1 /* the above plus NVFP4 codes and scales       */
#define FLAMIA_FORMAT_HADAMARD 0x10 /* OR-ed into FLAMIA_FORMAT_MXFP8: rotate each
                                       (token, head) row by H_d before the block
                                       statistics (for Q and K; see below)       */
#define FLAMIA_FORMAT_TOKEN_SCALES 0x20 /* OR-ed into FLAMIA_FORMAT_MXFP8 (with or
                                       without FLAMIA_FORMAT_HADAMARD): one
                                       exponent per (token, head) instead of per
                                       32-token block (per-token operand scales,
                                       see FLAMIA_FLAG_TOKEN_SCALES)             */

/* Attention flags. */
#define FLAMIA_FLAG_NVFP4_QK 0x1    /* score product QK^T (fwd and bwd recompute)
                                       from the NVFP4 copy of Q and K (d == 64)   */
#define FLAMIA_FLAG_NONCAUSAL 0x4   /* every query sees every key of its own
                                       document (no causal mask)                 */
#define FLAMIA_FLAG_HADAMARD 0x2    /* q and k were quantised with
                                       FLAMIA_FORMAT_HADAMARD: scores use
                                       softmax_scale / d; the backward returns
                                       dQ and dK rotated back by H_d            */
#define FLAMIA_FLAG_DETERMINISTIC_DQ 0x8 /* backward only: the float32 dQ
                                       partials of a query tile are added in
                                       a fixed key-tile order, so dQ is the
                                       same bit for bit on every run            */
#define FLAMIA_FLAG_DQ_FP16 0x10    /* backward only: dQ partials reduce-added
                                       in FP16 behind a power-of-two prescale
                                       from sequence-wide maxima                */
#define FLAMIA_FLAG_DQ_CAUSAL_SCALE 0x20 /* with FLAMIA_FLAG_DQ_FP16: the prescale
                                       of a query row from the keys it sees     */
#define FLAMIA_FLAG_SCHEDULE_STATIC 0x40 /* forward / backward: the persistent CTAs
                                       take their work items in a static snake
                                       over the cost-sorted list instead of
                                       claiming the next unclaimed item        */
#define FLAMIA_FLAG_DS_ROW_EXPONENTS 0x100 /* backward only: dQ's dS
                                       operand rounded with one exponent per
                                       (query row, 32-key block) instead of per
                                       32 x 32 block (dK keeps the block ones) */
#define FLAMIA_FLAG_TOKEN_SCALES 0x200 /* forward / backward: q, k, v and dout were
                                       quantised with FLAMIA_FORMAT_TOKEN_SCALES
                                       (one exponent per token); the per-token
                                       factors along each contraction are folded
                                       into the opposite operand before its E4M3
                                       rounding (see the forward and backward);
                                       the backward implies
                                       FLAMIA_FLAG_DS_ROW_EXPONENTS.  Not with
                                       FLAMIA_FLAG_NVFP4_QK                      */
#define FLAMIA_FLAG_DS_ZERO_COUNT 0x400 /* backward only: count, over every pair
                                       a query sees, the dS entries that are
                                       nonzero and, of those, the ones whose
                                       E4M3 code under the 32 x 32 block exponent
                                       is zero (rounded to zero), into two uint64
                                       at flamia_bwd_ds_counts_offset of the
                                       workspace (cleared by the call); not with
                                       FLAMIA_FLAG_DETERMINISTIC_DQ or
                                       FLAMIA_FLAG_DQ_FP16                       */
#define FLAMIA_FLAG_SCHEDULE_RULE 0x80 /* forward / backward: the pages' rule,
                                       dynamic claims for causal calls and, for
                                       non-causal ones, only when the longest
                                       document is at least 4x the average
                                       (static snake otherwise).  Default, no
                                       flag: dynamic claims (measured fastest
                                       on every workload here)                 */
#define FLAMIA_FLAG_BWD_CTA_PAIR 0x800 /* backward only, head dim 128: the
                                       2-CTA mode (review page sec. 3.4
                                       "Backward pass"): clusters of two CTAs,
                                       each pair splitting 256 keys and running
                                       its products together; FLAMIA_ERR_
                                       UNSUPPORTED with the NVFP4 path,
                                       FLAMIA_FLAG_DETERMINISTIC_DQ,
                                       FLAMIA_FLAG_DQ_FP16, query-row dS
                                       exponents, per-token scales, the dS
                                       diagnostic or a static schedule          */
#define FLAMIA_FLAG_BWD_ONE_CTA 0x1000 /* backward only: one CTA per 128-key
                                       tile.  With neither flag the backward
                                       takes the measured rule, which picks
                                       one-CTA items on every shape (the pair
                                       measured about 1.5x slower on the
                                       packed 4 x 4096 and variable-length
                                       workloads)                              */

/* Rotary flags. */
#define FLAMIA_FLAG_ROPE_INTERLEAVED 0x2000 /* pair i of a row is elements (2i, 2i + 1);
                                       default: (i, i + rot_dim / 2)              */
#define FLAMIA_FLAG_ROPE_INVERSE 0x4000 /* the transposed rotation: gradients of the
                                       rotated rows -> gradients of the rows      */

/* Shared-prefix flag. */
#define FLAMIA_FLAG_PREFIX_ALWAYS 0x8000 /* flamia_attn_cache_prefix: the prefix is read once
                                       for all sequences whatever the sizes (default: where
                                       that was measured faster)                  */

/*
 * One quantised operand, all device pointers owned by the caller.
 *  codes        u8  [T, H, d]     E4M3 codes.
 *  scales       u8  [H, T]        E8M0 byte of each token's 32-token block
 *                                 (dense: one entry per token and head).
 *  nvfp4_codes  u8  [T, H, d/2]   packed E2M1 (NULL unless NVFP4 requested).
 *  nvfp4_scales u8  [T, H, d/16]  E4M3 scale of each 16-element group (NULL
 *                                 unless NVFP4 requested).
 * codes and nvfp4_codes must be 16-byte aligned.
 */
typedef struct {
  uint8_t* codes;
  uint8_t* scales;
  uint8_t* nvfp4_codes;
  uint8_t* nvfp4_scales;
} flamia_qtensor;

/*
 * Fused token-block quantiser.
 * Source: review page sec. 3.1 (one power-of-two exponent per 32 consecutive
 * tokens x the full head dimension, E4M3 codes; the scale is constant along
 * the head dimension, so the payload serves K-major and MN-major products),
 * sec. 3.2 (exponent rounded up: the scaled block maximum never exceeds 448),
 * sec. 3.4 "Quantization fusion" (statistics, codes and scales in one launch)
 * and "Packed documents" (blocks never cross a document; dense per-token
 * scale table).  Blocks of document [s, e) are [s + 32i, min(s + 32i + 32, e)).
 * Exponent: smallest e with amax <= 448 * 2^e, clamped to [-127, 127]
 * (amax == 0 -> -127); codes = RNE_E4M3(x * 2^-e); scale byte = e + 127.
 * With format FLAMIA_FORMAT_MXFP8_NVFP4 the same pass also writes the NVFP4
 * copy (sec. 3.1 mixed path): per token and 16-element group, scale = the
 * smallest E4M3 value >= amax / 6, codes = RNE_E2M1(x / scale).
 * With FLAMIA_FORMAT_HADAMARD (sec. 3.4 "Hadamard rotation": the head-dim
 * channels of Q and K are mixed by an orthogonal transform inside the
 * quantiser) each row x is first replaced by x H_d, H_d the unnormalised
 * Sylvester-Hadamard matrix (entries +-1, H_d H_d = d I), computed in float32
 * by butterflies of stride 1, 2, .., d/2 in that order; the statistics and
 * codes are those of the rotated rows.  Not combinable with the NVFP4 copy
 * (FLAMIA_ERR_UNSUPPORTED) nor with o_bf16 / D.
 *
 *  x_bf16     [T, H, d] BF16 input (finite values).
 *  o_bf16, D  optional (both NULL or both set): the forward output O [T, H, d]
 *             BF16 and D float [H, T] = sum_k dequant(x)[t,h,k] * O[t,h,k]
 *             (review sec. 3.3: D from the same quantised dO used for dP).
 *  out        host pointer to a flamia_qtensor naming the caller's buffers.
 */
flamia_status flamia_quantize_tokenblock(const void* x_bf16, int T, int H, int d,
                                         const int32_t* cu_seqlens, int ndocs, int format,
                                         const void* o_bf16, float* D,
                                         const flamia_qtensor* out, int* dev_status,
                                         void* stream);

/*
 * Q, K and V of one call quantised by one launch (review page, sec. 3.4
 * "Quantization fusion": one pass per operand; one launch for the three
 * fills the GPU for longer and pays one tail).  The results are bit for bit
 * those of flamia_quantize_tokenblock on q with format_qk (H heads), on k
 * with format_qk (H_kv heads) and on v with FLAMIA_FORMAT_MXFP8 (H_kv heads).
 * format_qk: FLAMIA_FORMAT_MXFP8, FLAMIA_FORMAT_MXFP8_NVFP4 or
 * FLAMIA_FORMAT_MXFP8 | FLAMIA_FORMAT_HADAMARD (then V, never rotated, takes
 * a second launch).  q_bf16 [T, H, d], k_bf16 and v_bf16 [T, H_kv, d];
 * H_kv divides H.  Errors as for flamia_quantize_tokenblock.
 */
flamia_status flamia_quantize_qkv(const void* q_bf16, const void* k_bf16, const void* v_bf16,
                                  int T, int H, int H_kv, int d, const int32_t* cu_seqlens,
                                  int ndocs, int format_qk, const flamia_qtensor* q,
                                  const flamia_qtensor* k, const flamia_qtensor* v,
                                  int* dev_status, void* stream);

/*
 * Work list.  Source: review page sec. 3.4 "Work scheduling": a forward item
 * is 256 consecutive queries of one document (two 128-query tiles), its cost
 * the number of 128-key blocks it visits; items are sorted by descending
 * cost, built on the GPU once per micro-batch without a host sync.  The
 * backward items are 128-key tiles costed by the 128-query tiles that see
 * them.  Ties keep generation order (document, then position).
 *
 * Buffer layout (device, caller-owned, flamia_worklist_bytes(T, ndocs) bytes,
 * 256-byte aligned):
 *   int32 header[16]: [0] n_fwd, [1] n_bwd, [2] cap_fwd, [3] cap_bwd,
 *                     [4] max cost, [5] n_tile_fwd, [6] n_tile_bwd;
 *                     [7], [8] used by the builder; [9] .. [12] item claim
 *                     counters of the attention kernels (zero between
 *                     calls); the rest reserved.
 *   int32x4 fwd_items[cap_fwd] at byte 64: {doc, q_start, q_end, cost}
 *   int32x4 bwd_items[cap_bwd] after it:    {doc, k_start, k_end, cost}
 *   int32x4 tile_fwd[cap_fwd], tile_bwd[cap_bwd] after them: the same two
 *     lists without the items of documents of at most 32 tokens (n_tile_*
 *     entries each); the tensor-core kernels walk these, while documents of
 *     one 32-token block run on a CUDA-core kernel that needs no list.
 *   followed by the builder's scratch.
 * Each array starts on a 256-byte boundary.
 * cap_fwd = T/256 + ndocs + 1, cap_bwd = T/128 + ndocs + 1 (upper bounds).
 */
size_t flamia_worklist_bytes(int T, int ndocs);
flamia_status flamia_build_worklist(const int32_t* cu_seqlens, int ndocs, int T,
                                    void* wl, size_t wl_bytes, int* dev_status,
                                    void* stream);

/*
 * Work list without any device allocation, for callers that cannot allocate:
 * a framework whose caching allocator owns the device memory and hands the
 * library only its output tensors, a plugin host that gives the library no
 * allocator, or a latency-critical loop that cannot afford the implicit device
 * synchronisation of cudaMalloc / cudaFree.  The paper has no counterpart:
 * it is a convenience of this library's interface.
 *
 * Same inputs and the same output as flamia_build_worklist, but `wl` only
 * needs the header and the four item arrays (the layout above up to the end
 * of tile_bwd; a flamia_worklist_bytes-sized buffer always suffices).  The
 * builder's scratch lives in an 8 MiB array in the library's own device
 * memory, allocated on every GPU that loads the library and held until the
 * process exits.  The scratch grows mainly with the number of documents: any
 * document mix of up to 131,072 tokens fits, and at the 1,048,576-token
 * maximum up to 65,536 documents do; a layout whose scratch would exceed
 * 8 MiB returns FLAMIA_ERR_WORKSPACE without launching.
 * No cudaMalloc / cudaFree is called.  The first call in a CUDA context (with
 * its device current) looks up the array's device address and caches it under
 * the context's unique ID; make that first call before any stream capture.  A
 * context created later (after cudaDeviceReset, say) looks it up again.  All calls share the one array:
 * calls whose kernels overlap on the GPU (different streams, or different
 * host threads without ordering) race and produce garbage; serialise them.
 * Nothing left in the array by an earlier call is read by a later one.
 */
flamia_status flamia_build_worklist_static(const int32_t* cu_seqlens, int ndocs, int T,
                                           void* wl, size_t wl_bytes, int* dev_status,
                                           void* stream);

/*
 * Causal forward.  Source: review page sec. 1.2 (S = QK^T scale, P =
 * softmax(S), O = PV, row statistics saved), sec. 3.1 (unscaled E4M3 product
 * for QK^T with the query factor folded into the softmax scale and the key
 * factor applied separately; E4M3 probability operand; BF16 output), sec. 3.4
 * "Packed documents" (outputs written in place to the packed buffer).
 * Numerics: s_ij = scale * log2(e) * 2^eQ(i) * 2^eK(j) * <q_i, k_j> (codes),
 * running integer row maximum m_i = ceil(max_j s_ij), P~ = exp2(s - m),
 * l = sum P~, operand P^ = RNE_E4M3(2^8 P~), O = 2^-8 sum_j P^ V^_j / l,
 * LSE = (m + log2 l) ln 2.
 * FLAMIA_FLAG_HADAMARD: q and k hold Q H_d and K H_d, so the call uses
 * softmax_scale / d for the scores (the same S exactly, d a power of two).
 * Not combinable with FLAMIA_FLAG_NVFP4_QK.
 * FLAMIA_FLAG_NONCAUSAL (review page sec. 4.8, the non-causal packed call):
 * every query sees every key of its own document; the same numerics, the
 * same work list (its costs are the causal ones: only the order of the items
 * follows from them).
 *
 *  q, k, v      host pointers to quantised operands (E4M3 + scales; with
 *               FLAMIA_FLAG_NVFP4_QK also the NVFP4 copies of q and k).
 *  wl           a work list built for the same cu_seqlens / T.  Items are
 *               claimed dynamically in list order (longest first, sec. 3.4:
 *               the paper's dynamic assignment for causal calls) through a
 *               counter in the list's header, which the call updates and
 *               resets before it ends; calls that share one work list must
 *               not run at the same time (a forward and a backward may).
 *  o_bf16       [T, H, d] BF16 output.   lse  float [H, T] (natural log).
 * Only tokens inside documents are written.
 */
flamia_status flamia_attn_fwd(const flamia_qtensor* q, const flamia_qtensor* k,
                              const flamia_qtensor* v, const int32_t* cu_seqlens, int ndocs,
                              int T, int H, int d, float softmax_scale, int flags,
                              void* wl, void* o_bf16, float* lse, int* dev_status,
                              void* stream);

/*
 * Grouped-query attention: k and v carry H_kv heads (H_kv divides H); query
 * head h reads K / V head h / (H / H_kv).  k, v codes [T, H_kv, d], scales
 * [H_kv, T]; q, o [T, H, d]; lse [H, T].  flamia_attn_fwd is this call with
 * H_kv = H.  FLAMIA_ERR_INVALID_ARG if H_kv does not divide H.
 */
flamia_status flamia_attn_fwd_gqa(const flamia_qtensor* q, const flamia_qtensor* k,
                                  const flamia_qtensor* v, const int32_t* cu_seqlens, int ndocs,
                                  int T, int H, int H_kv, int d, float softmax_scale, int flags,
                                  void* wl, void* o_bf16, float* lse, int* dev_status,
                                  void* stream);

/*
 * Workspace of the forward: 0 bytes for every size (the review page, sec.
 * 3.4, keeps the forward's running statistics and P^ on chip; O and LSE are
 * its outputs).  Kept so that a caller sizes both calls the same way;
 * returns 0 also for unsupported sizes.
 */
size_t flamia_fwd_workspace_bytes(int T, int H, int d);

/*
 * Workspace of the backward, each part padded to 256 bytes: a float32
 * [T, H, d] dQ accumulator (FLAMIA_FLAG_DQ_FP16 uses its first half as an
 * FP16 [T, H, d] one), an int32 [T, H] array of turn counters
 * (FLAMIA_FLAG_DETERMINISTIC_DQ), the int8 [H, T] prescale exponents of the
 * FP16 accumulator, 3 H ints of scratch and the two dS counters
 * (FLAMIA_FLAG_DS_ZERO_COUNT).  The caller allocates it; the
 * backward clears what it uses itself.
 */
size_t flamia_bwd_workspace_bytes(int T, int H, int d);

/*
 * Byte offset, inside the backward workspace, of the two uint64 counters that
 * FLAMIA_FLAG_DS_ZERO_COUNT fills: [0] nonzero dS entries among the pairs the
 * queries see, [1] those of them whose E4M3 code in the 32 x 32 block payload
 * is zero.  The review page (sec. 3.3, and the dS-scale ablation of sec. 4)
 * takes this fraction as the sign of a badly set dS scale.  Read it after the
 * backward has completed.  0 for unsupported sizes.
 */
size_t flamia_bwd_ds_counts_offset(int T, int H, int d);

/*
 * Causal backward.  Source: review page sec. 1.2 (recompute P; dV = P^T dO,
 * dP = dO V^T, dS = P o (dP - D), dQ = dS K, dK = dS^T Q), sec. 3.3 (the
 * recompute uses the forward's quantised Q, K, tiling, masks and exp; D from
 * the same quantised dO), sec. 3.1 (dS to E4M3 with one scale per 32x32 block
 * so one payload feeds dQ and dK), sec. 3.4 "Backward pass".
 * Numerics: P = exp2(s - LSE log2 e); dV operand RNE_E4M3(2^8 P); dS in float
 * from the unquantised P; dS exponent = round-up rule on each document-aligned
 * 32x32 block maximum; dQ and dK scaled by softmax_scale after the products;
 * dQ partial sums are added in float32 (no prescale), then converted to BF16.
 * FLAMIA_FLAG_NONCAUSAL: as for the forward; dS is masked only at the
 * document ends.
 * FLAMIA_FLAG_HADAMARD: as for the forward, with softmax_scale / d, and the
 * gradients of the rotated operands are rotated back before the BF16
 * conversion: dQ = dQ_r H_d, dK = dK_r H_d (float32 butterflies as in the
 * quantiser).
 * FLAMIA_FLAG_DETERMINISTIC_DQ: by default the key tiles' dQ partials reach
 * the float32 accumulator in whatever order the CTAs finish (the sum varies
 * in its last bits from run to run).  With the flag, the 128-key tiles of a
 * document add their partials to a query tile in descending order (a turn
 * counter per query tile, bounded waits; each head's work items are claimed
 * shortest first, so a key tile never waits for one claimed after it), and
 * O, dQ, dK and dV are bitwise reproducible.  A wait that times out (2 s)
 * sets FLAMIA_DEV_TIMEOUT.
 * FLAMIA_FLAG_DS_ROW_EXPONENTS (review page, sec. 3.2: the query-row-wise dS
 * exponents that remove the leakage inside blocks): a 32 x 32 dS block
 * shares one exponent across 32 query rows, so a later row's gradient moves
 * the rounding of an earlier row's dQ; with the flag the dQ product takes dS
 * rounded per (query row, 32-key block), carried as its block scales, while
 * dK keeps the shared exponents (dK of a key sums every later query anyway).
 * FLAMIA_FLAG_DQ_FP16 (review page, sec. 3.2 "accumulator leakage", sec.
 * 3.5.3: the FP16 dQ reduce that halves the reduction traffic): each key
 * tile's float32 dQ partial of query row i is multiplied by 2^p(i), rounded
 * to FP16 and reduce-added into an FP16 accumulator; dQ = softmax_scale *
 * 2^-p(i) * acc.  p(i) = 15 - ceil(log2(16 d 448^3)) - (e_dO(i) + max e_V +
 * max e_K), e the E8M0 block exponents (every element |x| <= 448 2^e), which
 * bounds |2^p acc| by 2^15; clamped to [-126, 126].  The maxima run over
 * the head's whole sequence, so a later token changes the rounding of
 * earlier rows; with FLAMIA_FLAG_DQ_CAUSAL_SCALE they run over the keys the
 * row sees (its document up to the row; the whole document in a non-causal
 * call), which removes that dependence.  Combinable with every other flag.
 *
 *  dout         host pointer to the quantised dO (from the quantiser run with
 *               o_bf16 = the forward output, which also produced D).
 *  D, lse       float [H, T] from the quantiser and the forward.
 *  dq, dk, dv   [T, H, d] BF16 outputs (only tokens inside documents written).
 *  ws           flamia_bwd_workspace_bytes(T, H, d) bytes, 256-byte aligned.
 *  wl           as for the forward (its own claim counter).
 */
flamia_status flamia_attn_bwd(const flamia_qtensor* q, const flamia_qtensor* k,
                              const flamia_qtensor* v, const flamia_qtensor* dout,
                              const float* D, const float* lse,
                              const int32_t* cu_seqlens, int ndocs, int T, int H, int d,
                              float softmax_scale, int flags, void* wl,
                              void* dq_bf16, void* dk_bf16, void* dv_bf16,
                              void* ws, size_t ws_bytes, int* dev_status, void* stream);

/*
 * Grouped-query backward: as flamia_attn_bwd with K / V heads shared as in
 * flamia_attn_fwd_gqa; dq [T, H, d], dk and dv [T, H_kv, d] (the gradient of
 * a K / V head sums over its H / H_kv query heads); dout, D, lse per query
 * head.  The workspace is flamia_bwd_workspace_bytes(T, H, d).
 */
flamia_status flamia_attn_bwd_gqa(const flamia_qtensor* q, const flamia_qtensor* k,
                                  const flamia_qtensor* v, const flamia_qtensor* dout,
                                  const float* D, const float* lse, const int32_t* cu_seqlens,
                                  int ndocs, int T, int H, int H_kv, int d, float softmax_scale,
                                  int flags, void* wl, void* dq_bf16, void* dk_bf16,
                                  void* dv_bf16, void* ws, size_t ws_bytes, int* dev_status,
                                  void* stream);

/*
 * Rotary positions of Q and K (and, inverted, of dQ and dK).  The paper has no
 * counterpart: it is what a model applies to Q and K before the quantiser, and
 * to dQ and dK after the backward.
 *
 * Token t of document b stands at position p = starts[b] + t - cu_seqlens[b]
 * (starts NULL: 0; p is an int32).  Pair i < rot_dim / 2 of every head's row is turned by the
 * angle 2 pi frac(p * turns[i] / 2^64) and multiplied by mscale:
 *   (x, y) -> mscale (x cos - y sin, x sin + y cos);
 * FLAMIA_FLAG_ROPE_INVERSE turns the other way (the transpose, mscale kept).
 * Elements rot_dim .. d - 1 of a row are copied.  turns[i] is the step of one
 * position in 2^-64 turns, round(2^64 w_i / (2 pi)) for an angle of p w_i: the
 * product with p wraps at whole turns, so far positions lose nothing.
 *
 *  q_in, q_out  BF16 rows [T][H][d]: head h of token t at t * stride + h * d
 *               (strides in elements, multiples of 8, >= H * d; rows 16-byte
 *               aligned, so a slice of a packed QKV tensor will do).  q_out
 *               may be q_in with the same stride (in place); otherwise the
 *               two must not overlap.  k_in, k_out the same with H_kv heads
 *               (H_kv 0: no K; otherwise it need not divide H).
 *  turns        device uint64[rot_dim / 2].  rot_dim: a multiple of 16, 16 .. d.
 *  starts       device int32[ndocs] or NULL.
 *  cu_seqlens   as elsewhere, but it may end before T (a padded batch): rows
 *               behind the last document are not written.
 *  flags        FLAMIA_FLAG_ROPE_INTERLEAVED | FLAMIA_FLAG_ROPE_INVERSE.
 * T == 0 enqueues nothing.  ndocs <= 2^20.
 */
flamia_status flamia_rope(const void* q_in, void* q_out, int64_t q_in_stride,
                          int64_t q_out_stride, const void* k_in, void* k_out,
                          int64_t k_in_stride, int64_t k_out_stride, int T, int H, int H_kv,
                          int d, const uint64_t* turns, int rot_dim, float mscale, int flags,
                          const int32_t* cu_seqlens, int ndocs, const int32_t* starts,
                          int* dev_status, void* stream);

/*
 * Rotary positions with several axes (time, height and width of the patches of an
 * image or a video; text moves along all of them together): flamia_rope with the
 * position of pair i of token t taken from positions[axes[i] * pos_stride + t].
 * The caller gives all positions, so there are no starts; a position may be negative.
 *
 *  axes       device uint8[rot_dim / 2]: the axis of each pair (naxes - 1 at most;
 *             larger entries count as that).
 *  positions  device int32, naxes rows of T entries, pos_stride entries apart.
 *  naxes      1 .. rot_dim / 2.
 * Everything else as for flamia_rope (tokens behind the last document are not
 * written; FLAMIA_FLAG_ROPE_INVERSE turns gradients back).
 */
flamia_status flamia_rope_axes(const void* q_in, void* q_out, int64_t q_in_stride,
                               int64_t q_out_stride, const void* k_in, void* k_out,
                               int64_t k_in_stride, int64_t k_out_stride, int T, int H, int H_kv,
                               int d, const uint64_t* turns, const uint8_t* axes, int rot_dim,
                               float mscale, int flags, const int32_t* positions,
                               int64_t pos_stride, int naxes, const int32_t* cu_seqlens,
                               int ndocs, int* dev_status, void* stream);

/*
 * Paged key-value cache: the K and V of running sequences in the quantiser's
 * format, for the calls below.  All device pointers, owned by the caller.
 *  k_codes, v_codes    u8 [num_pages][H_kv][page_size][d]  E4M3 codes.
 *  k_scales, v_scales  u8 [num_pages][H_kv][page_size]     E8M0 byte per token.
 * codes 128-byte aligned, scales 32-byte aligned.  page_size: 32, 64 or a
 * multiple of 128 up to 2^20; num_pages * H_kv < 2^31; 1 <= H_kv <= 4096.
 * Position p of sequence b is row p % page_size of page
 * page_table[b * table_stride + p / page_size] (device int32, entries of pages
 * that no call needs are not read; table_stride entries per sequence).  Two
 * sequences may share pages that are only read.
 */
typedef struct {
  uint8_t* k_codes;
  uint8_t* k_scales;
  uint8_t* v_codes;
  uint8_t* v_scales;
  int32_t num_pages;
  int32_t page_size;
  int32_t H_kv;
  int32_t d;
} flamia_kvcache;

/*
 * Quantises new tokens into the cache.  Token t of document b goes to position
 * starts[b] + t - cu_seqlens[b] of sequence b (starts NULL: 0).
 * format FLAMIA_FORMAT_MXFP8: one exponent per 32-token block (positions 32 i ..
 * 32 i + 31) and head, the rule of flamia_quantize_tokenblock over the new
 * tokens of the block; where the block already holds tokens (starts[b] inside
 * it) the exponent is the larger of that and the largest held one, and the codes c
 * of held tokens with a smaller one become RNE_E4M3(c 2^(e_old - e)).  So a prompt
 * written at starts 0 gets the codes and scale bytes that flamia_quantize_tokenblock
 * gives it, bit for bit, and a call repeated at once on the same tokens changes
 * nothing.
 * FLAMIA_FORMAT_TOKEN_SCALES OR-ed in: one exponent per token and head.
 * A sequence is written in one of the two formats throughout (what is held is
 * taken as the same one); readers take either.
 * Infinities and NaN become NaN codes and do not enter the block maximum.
 * Positions behind the last new token keep what they held.
 *
 *  k_bf16, v_bf16  BF16 rows [T][H_kv][d], token strides in elements (multiples
 *                  of 8), rows 16-byte aligned.
 * cu_seqlens may end before T; documents may be empty (idle sequences).  No
 * two documents of a call may write the same page.  T == 0 enqueues nothing.
 */
flamia_status flamia_cache_write(const flamia_kvcache* cache, const void* k_bf16,
                                 int64_t k_stride, const void* v_bf16, int64_t v_stride, int T,
                                 const int32_t* cu_seqlens, int ndocs, const int32_t* starts,
                                 const int32_t* page_table, int table_stride, int format,
                                 int* dev_status, void* stream);

/*
 * Reads cached tokens back: positions starts[b] .. of sequence b into packed
 * tokens [cu_seqlens[b], cu_seqlens[b + 1]) as BF16 (code * 2^e, rounded to
 * nearest even where BF16 cannot hold it: only below its normal range).
 * Arguments as for flamia_cache_write, k_bf16 / v_bf16 the outputs (strides
 * >= H_kv * d); rows without a cached token or a valid page keep what they held.
 */
flamia_status flamia_cache_read(const flamia_kvcache* cache, void* k_bf16, int64_t k_stride,
                                void* v_bf16, int64_t v_stride, int T, const int32_t* cu_seqlens,
                                int ndocs, const int32_t* starts, const int32_t* page_table,
                                int table_stride, int* dev_status, void* stream);

/*
 * Pages of the cache: the books that say who uses which, kept on the device so that a
 * captured step can hand out its own pages.
 *  page_table  device int32 [nseq][table_stride], as above: a row a sequence, -1
 *              where it has no page.  1 <= nseq <= 65,536, nseq * table_stride < 2^31.
 *  refs        device int32 [num_pages]: how many slots of the page table hold each
 *              page; 0: free.  A fresh pool has zeros here and -1 in the table; the
 *              calls keep the two in line, and both are the caller's to read.
 * Calls on one pool must not overlap one another, nor calls that use its pages.
 * What they decide does not depend on timing.  A sequence outside the table or a page
 * outside the pool sets FLAMIA_DEV_BAD_PAGE and is left alone.
 */

/*
 * Copies pages: page dst[i] of `to` becomes page src[i] of `from` (K and V, codes and
 * scale bytes).  The two caches have the same page_size, H_kv and d, and may be one;
 * no page may then be both source and target, and in any case none a target twice.
 * Pairs with a negative entry are left out.  The page table and refs are not touched.
 *  src, dst   device int32[n].   n == 0 enqueues nothing.
 */
flamia_status flamia_pages_copy(const flamia_kvcache* from, const flamia_kvcache* to,
                                const int32_t* src, const int32_t* dst, int n, int* dev_status,
                                void* stream);

/*
 * Sequence children[i] goes on from where parents[i] stands: it gives its pages back,
 * takes those that hold the first lens[parents[i]] tokens of the parent, shared with it
 * (refs counted), and that length.  parents[i] < 0, or parents NULL: it only gives
 * its pages back and has length 0 then.  All parents are read before any child is
 * written, so children may be parents (beams put in a new order); a sequence that is
 * its own parent gives back the pages behind its length.  children[i] < 0: nothing.  Of
 * entries with the same child the last one counts.  No page is copied: see
 * flamia_pages_reserve.
 *  parents, children  device int32[n], n <= nseq.   n == 0 enqueues nothing.
 *  lens       device int32 [nseq]: tokens that each sequence holds (its next starts).
 *  ws         flamia_pages_fork_workspace_bytes(n, table_stride) bytes, 256-byte aligned.
 */
size_t flamia_pages_fork_workspace_bytes(int n, int table_stride);
flamia_status flamia_pages_fork(int32_t* refs, int num_pages, int32_t* page_table,
                                int table_stride, int nseq, int page_size,
                                const int32_t* parents, const int32_t* children, int n,
                                int32_t* lens, void* ws, size_t ws_bytes, int* dev_status,
                                void* stream);

/*
 * Pages for the new tokens of a call: afterwards every slot that positions starts[b] ..
 * starts[b] + n_b - 1 of sequence b fall into (n_b = cu_seqlens[b + 1] - cu_seqlens[b])
 * holds a page that no other slot holds.  In order of sequence and slot: one without a page takes
 * the lowest free one; one whose page has other users takes the lowest free one, to which
 * the rows of positions below starts[b] are copied, and leaves the old one; if all the
 * users of a page are among the call's slots, the last of them keeps it.  If there are not
 * as many free pages, nothing is changed and FLAMIA_DEV_CAPACITY is set; nor is it where
 * cu_seqlens is malformed (it falls, does not begin with 0 or ends behind T:
 * FLAMIA_DEV_BAD_SEQLENS).  A sequence whose positions lie outside its row gets none.
 * cu_seqlens and starts as for flamia_cache_write (cu_seqlens may end before T).
 * T == 0 enqueues nothing (granted stays as it was).
 *  granted    device int32[nseq + 1], not cu_seqlens, or NULL: the offsets for the step's
 *             other calls.  cu_seqlens, or zeros if there were not as many pages, cu_seqlens
 *             is malformed or a sequence's positions lie outside its row: with those the calls
 *             do nothing, where with cu_seqlens they would write into pages that other
 *             sequences hold as well.
 *  ws         flamia_pages_reserve_workspace_bytes(T, nseq, table_stride, page_size)
 *             bytes, 256-byte aligned.
 */
size_t flamia_pages_reserve_workspace_bytes(int T, int nseq, int table_stride, int page_size);
flamia_status flamia_pages_reserve(const flamia_kvcache* cache, int32_t* refs,
                                   int32_t* page_table, int table_stride, int nseq, int T,
                                   const int32_t* cu_seqlens, const int32_t* starts,
                                   int32_t* granted, void* ws, size_t ws_bytes, int* dev_status,
                                   void* stream);

/*
 * Moves the pages in use to the front of the pool: with `live` of them, the k-th used
 * page from page `live` on is copied to the k-th free one before it, and the page table
 * and refs follow.  Other records of page numbers are the caller's to change.
 *  live       device int32[1], or NULL: the number of pages in use.
 *  ws         flamia_pages_compact_workspace_bytes(num_pages) bytes, 256-byte aligned.
 */
size_t flamia_pages_compact_workspace_bytes(int num_pages);
flamia_status flamia_pages_compact(const flamia_kvcache* cache, int32_t* refs,
                                   int32_t* page_table, int table_stride, int nseq, int32_t* live,
                                   void* ws, size_t ws_bytes, int* dev_status, void* stream);

/*
 * Attention of new tokens over the cache (single tokens, drafted tokens or
 * the next chunk of a prompt, mixed freely in one call), after they were
 * written to it with the same cu_seqlens, starts and page_table.  Query i of
 * sequence b stands at position p = starts[b] + i (starts NULL: 0).  It sees
 * key j iff 0 <= j <= p and, with window > 0, j > p - window or j < sinks.
 *   o = softmax(softmax_scale q K^T) V over the seen keys, K and V the cached
 *   values code * 2^e; lse = log sum exp of the scaled scores (natural log).
 * A query that sees no key (p < 0) gets o = 0 and lse = -inf.  A NaN key or
 * value that a query sees makes its output NaN; one that it does not see, and
 * whatever lies behind a sequence's last token, changes nothing.  Queries enter
 * exactly but for elements below 2^-13 of their row's largest, which are rounded to
 * 2^-21 of that.  Scores and sums are float32; a softmax weight is rounded to 2^-14
 * of itself (to FP16, 2^-11, with more than 8 query rows a sequence and K / V head
 * on average) or 2^-23 of the row's largest weight times value scale, whichever is
 * more; scores beyond 2^16 within 2^-19 of one another may count as equal.  Positions
 * stay below 2^30.
 * Query head h reads K / V head h / (H / H_kv).
 *
 *  q_bf16     BF16 rows [T][H][d], token stride in elements (multiple of 8).
 *  o_bf16     [T, H, d] BF16.   lse  float [H, T], or NULL.
 *  window     0: every earlier key.   sinks  >= 0; needs window > 0 if > 0.
 *  ws         flamia_attn_cache_workspace_bytes bytes, 256-byte aligned; calls
 *             that may overlap (on two streams, in two graphs, from two threads on
 *             one stream: a call is two kernels) need one each.  Nothing is kept in it.
 * cu_seqlens may end before T: rows behind the last sequence are not written
 * (lse columns neither).  T == 0 enqueues nothing.
 */
size_t flamia_attn_cache_workspace_bytes(int T, int ndocs, int H, int H_kv, int d);
flamia_status flamia_attn_cache(const flamia_kvcache* cache, const void* q_bf16, int64_t q_stride,
                                int T, int H, const int32_t* cu_seqlens, int ndocs,
                                const int32_t* starts, const int32_t* page_table,
                                int table_stride, float softmax_scale, int window, int sinks,
                                void* o_bf16, float* lse, void* ws, size_t ws_bytes,
                                int* dev_status, void* stream);

/*
 * flamia_attn_cache (without a window) for a batch whose sequences begin with the same
 * `prefix` tokens: a prompt that was forked, a system prompt, a document that all ask
 * about.  A sequence whose new tokens all stand at prefix - 1 or behind (starts[b] >=
 * prefix - 1), and inside its table row, shares it: its first `prefix` positions hold what
 * those of the other sharing sequences hold, as a rule in the same pages, and those of the
 * first such sequence with new tokens are read for all of them.  Nothing checks this: a
 * sequence as long as that which begins with something else goes into another call.  The
 * others, and calls that gain nothing by it (one sequence, a prefix below 128, more than 96
 * query rows a sequence and K / V head on average; without FLAMIA_FLAG_PREFIX_ALWAYS those
 * that save too few bytes) are flamia_attn_cache's.  The results are what that call gives, in
 * other roundings: with more than 8 query rows of a K / V head in the batch (T * H / H_kv) a
 * weight is rounded to 2^-11 of itself.
 *
 *  flags      0 or FLAMIA_FLAG_PREFIX_ALWAYS.
 *  ws         flamia_attn_cache_prefix_workspace_bytes bytes, 256-byte aligned, as for
 *             flamia_attn_cache (a call is two or three kernels).
 */
size_t flamia_attn_cache_prefix_workspace_bytes(int T, int ndocs, int H, int H_kv, int d,
                                                int prefix, int flags);
flamia_status flamia_attn_cache_prefix(const flamia_kvcache* cache, const void* q_bf16,
                                       int64_t q_stride, int T, int H, const int32_t* cu_seqlens,
                                       int ndocs, const int32_t* starts, const int32_t* page_table,
                                       int table_stride, int prefix, float softmax_scale,
                                       int flags, void* o_bf16, float* lse, void* ws,
                                       size_t ws_bytes, int* dev_status, void* stream);

/* Static description of a status code (never NULL). */
const char* flamia_status_str(flamia_status s);

#ifdef __cplusplus
}
#endif

#endif /* FLAMIA_H */
