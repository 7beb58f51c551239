/*
 * w4a16.h -- C ABI of the GB300 (sm_103a) group-quantized INT4-weight x
 * bf16-activation matmul library.
 *
 *   y[M, N] = x[M, K] . dequant(W)[N, K]^T,   w[n][k] = (q[n][k] - z[n][k/G]) * scale[n][k/G]
 *
 * The dequantisation is the exact "(q - z) * scale" of the INT4 kernels in the
 * GRIMOIRE v1.7 release notes ("What changed"): q a 4-bit code, one bf16 scale
 * per (output row, K-group) with group G = 64 or 128, and z = 8 for the
 * symmetric GPTQ-Int4 checkpoints or a packed 4-bit zero point for the
 * asymmetric AutoRound W4A16 ones (same page, measurement table). The regimes
 * are those the same pages measure: one-row decode, 2-16 rows of batched
 * decode and speculative verify, the output-vocabulary head over all verify
 * rows in one pass, and 4,096-row prompts with the feed-forward gate fused in
 * (GRIMOIRE v1.8 release notes, "INT4 verify faster" and "INT4 prompt
 * processing").
 *
 * A third weight form, affine, rebuilds w[n][k] = scale[n][k/G] * q[n][k] +
 * bias[n][k/G] with a bf16 bias per group in place of the zero point: the MLX
 * affine 4-bit checkpoints that TensorFold PR #859 runs ("What this changes":
 * every code keeps its value, scale and bias; groups of 64). Its calls carry
 * "affine" in their names; the others take zero-point forms only.
 *
 * Canonical (input) layout, row-major, little-endian:
 *   qweight int32  [N][K/8]            nibble j (bits 4j..4j+3) of word c holds k = 8c + j
 *   scales  bf16   [N][K/G]            bf16 values passed as uint16_t bit patterns
 *   zeros   int32  [N][ceil(K/G/8)]    nibble j of word c holds the zero of group 8c + j
 *                                      (asymmetric only; unused nibbles ignored)
 *   biases  bf16   [N][K/G]            affine form only
 *
 * Conventions for every call:
 *   - Pointers named x, y, h, qweight, scales, zeros, packed, w_out are DEVICE
 *     pointers owned by the caller; the library allocates no device memory
 *     and keeps no pointer after a call returns.
 *   - Every compute call is asynchronous on `stream` (NULL = legacy default
 *     stream) and launches kernels on the calling thread's current device.
 *   - Return value: W4A16_OK (0) or a negative W4A16_ERR_* code. On any error
 *     detected before launch nothing is launched and no memory is written.
 *     W4A16_ERR_CUDA means a CUDA call failed; w4a16_last_cuda_error() gives
 *     its cudaError_t value (thread-local).
 *   - bf16 values are IEEE bfloat16 bit patterns in uint16_t; outputs are
 *     rounded to nearest-even from float32.
 *   - `sym` names the weight form: 0 = packed zero points, 1 = symmetric
 *     (z = 8; `zeros` is ignored and may be NULL), W4A16_AFFINE (2) =
 *     scale * q + bias, accepted only where a comment says so. Any other
 *     value is W4A16_ERR_INVALID_ARG (size queries return 0).
 *   - Supported sizes: 1 <= M, 1 <= N, 64 <= K, K % G == 0, G in {64, 128},
 *     M, N, K below 2^31 / 16.
 *   - Alignment: x, y, h 16 bytes; packed 256 bytes (cudaMalloc gives both).
 */
#ifndef W4A16_H_
#define W4A16_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* cudaStream_t without the CUDA headers (same type as the runtime's). */
typedef struct CUstream_st *w4a16_stream_t;

#define W4A16_OK 0
#define W4A16_ERR_INVALID_ARG (-1)  /* size, group, null pointer or reserved argument */
#define W4A16_ERR_MISALIGNED (-2)   /* a pointer breaks the alignment rules above */
#define W4A16_ERR_UNSUPPORTED (-3)  /* the current device is not an sm_103 GPU */
#define W4A16_ERR_CUDA (-4)         /* a CUDA call failed; see w4a16_last_cuda_error() */
#define W4A16_ERR_TIMEOUT (-5)      /* a bounded wait inside a kernel gave up */
#define W4A16_ERR_INDEX (-6)        /* a kernel met an index outside its buffers and skipped it */

/* Weight forms (the `sym` argument). */
#define W4A16_ZERO_POINTS 0
#define W4A16_SYMMETRIC 1
#define W4A16_AFFINE 2

/*
 * Size in bytes of the repacked weight that w4a16_repack (sym 0 or 1) or
 * w4a16_repack_affine (sym = W4A16_AFFINE) writes for an N x K weight (codes,
 * scales, and the zero points (sym = 0) or the biases (affine), each section
 * 256-byte aligned; rows padded to a multiple of 16). Returns 0 when the
 * sizes or the form are not supported.
 */
size_t w4a16_repacked_bytes(int N, int K, int group, int sym);

/*
 * Offline repack of one canonical weight (qweight, scales, zeros as above)
 * into the library's tiled layout in `packed` (w4a16_repacked_bytes bytes,
 * caller-allocated device memory). Pure bit moves: no value is rounded, so
 * every dequantised weight stays exactly (q - z) * scale. Rows are tiled 16 at
 * a time; within a tile and a 64-wide K chunk each of 32 lanes owns one
 * 16-byte run of codes for two rows and 16 consecutive k, the order in which
 * the kernels consume them. Scales (and zeros) sit per tile in blocks of four
 * groups. Padding rows get code 0, scale 0 and zero 0. Not timed on the hot
 * path; asynchronous on `stream`.
 */
int w4a16_repack(const int32_t *qweight, const uint16_t *scales, const int32_t *zeros,
                 int N, int K, int group, int sym, void *packed, w4a16_stream_t stream);

/* Size of the repacked gate/up pair of w4a16_repack_gateup or, for sym =
 * W4A16_AFFINE, w4a16_repack_affine_gateup (N_each rows each). */
size_t w4a16_gateup_repacked_bytes(int N_each, int K, int group, int sym);

/*
 * Offline repack of the feed-forward gate and up weights (two canonical
 * weights of N_each rows each) into one buffer whose 16-row tiles alternate
 * gate, up, gate, up, ... (N_each padded to a multiple of 128), so that one
 * tile of the prompt GEMM holds 128 gate rows and the 128 matching up rows.
 * The result is also a valid w4a16_repack buffer of 2 * round_up(N_each, 128)
 * rows in that interleaved order.
 */
int w4a16_repack_gateup(const int32_t *qw_gate, const uint16_t *sc_gate, const int32_t *z_gate,
                        const int32_t *qw_up, const uint16_t *sc_up, const int32_t *z_up,
                        int N_each, int K, int group, int sym, void *packed,
                        w4a16_stream_t stream);

/*
 * y[M][N] (bf16, row-major) = x[M][K] (bf16, row-major) . dequant(W)^T, with
 * W given as the output of w4a16_repack for the same (N, K, group, sym).
 * float32 accumulation; each group's partial sum is scaled in float32.
 * `scales` and `zeros` are reserved: scales and zero points travel inside
 * `packed`, and both must be NULL (else W4A16_ERR_INVALID_ARG).
 * Kernel choice: M <= 32 -> a decode kernel (each weight read and unpacked
 * once for all rows, multiply-adds on the tensor core): the one that stages x
 * once per CTA when M <= 8 and its grid fills the GPU, or for 9-16 rows of a
 * zero-point weight whose grid spans 1.5 CTAs per SM, else the one with a
 * weight ring per warp; M > 32 -> the tcgen05 GEMM. A CUDA-core one-row GEMV
 * is selectable (w4a16_set_kernel_override).
 * Results are bitwise reproducible run to run (no atomics in any sum).
 */
int w4a16_gemm(const uint16_t *x, const void *packed, const uint16_t *scales,
               const int32_t *zeros, int M, int N, int K, int group, int sym, uint16_t *y,
               w4a16_stream_t stream);

/*
 * Greedy pick over the output columns: argmax[m] = the first n at which the
 * bf16 output y[m][n] of w4a16_gemm (same x, packed, sizes) is largest, as
 * torch.argmax over a bf16 row returns it: among equal values the lowest n;
 * -0 equals +0; a NaN counts as the maximum. For the output-vocabulary head
 * this replaces reading back M x N logits with M indices (the GPU argmax
 * after the tall head in lucebox PR #823; one pass over all verify rows as in
 * the GRIMOIRE v1.8 release notes, "INT4 verify faster").
 *
 *   argmax  int64 [M], device, 8-byte aligned; written by this call
 *   y       bf16 [M][N] or NULL. M <= 32: the decode kernel forms the argmax
 *           in its epilogue and stores y only when y is not NULL (the logits
 *           need not exist). M > 32: required; the tcgen05 GEMM writes y and
 *           a second kernel reads it back.
 *
 * Launches three kernels on `stream` (zero the keys, the GEMM, turn keys
 * into indices), all taking part in programmatic overlap when it is on; the
 * result is ready when the stream reaches the end of the call. Errors as
 * w4a16_gemm.
 */
int w4a16_gemm_argmax(const uint16_t *x, const void *packed, int M, int N, int K, int group, int sym,
                      uint16_t *y, int64_t *argmax, w4a16_stream_t stream);

/*
 * Top-k of bf16 rows: the greedy pick on the GPU (lucebox PR #823,
 * description) widened to the k largest entries of each row of the logits
 * y [M][N], with the argmax's rules: largest value first; equal values
 * lowest column first (-0 equals +0); a NaN ranks above +inf (NaNs among
 * themselves by column). k = 1 gives w4a16_gemm_argmax's index.
 *
 *   y     bf16 [M][N], device, 2-byte aligned (16-byte aligned rows with N a
 *         multiple of 8 take 16-byte loads); read only
 *   k     1 <= k <= min(N, 1024)
 *   idx   int64 [M][k], device, 8-byte aligned: the columns, best first
 *   vals  bf16 [M][k], device, or NULL: y at those columns (bit patterns)
 *
 * One kernel on `stream`: per row, one cluster of up to 16 CTAs (two radix
 * passes of 8 bits over the order-preserving 16-bit codes of the values,
 * histograms summed over distributed shared memory, then a sort of the k
 * picks); it allocates nothing and takes part in programmatic overlap when
 * that is on. Errors: W4A16_ERR_INVALID_ARG (null y or idx, M or N out of
 * range, k out of range), W4A16_ERR_MISALIGNED, as w4a16_gemm otherwise.
 */
int w4a16_topk(const uint16_t *y, int M, int N, int k, int64_t *idx, uint16_t *vals, w4a16_stream_t stream);

/*
 * w4a16_gemm into y (required: the logits the selection reads), then
 * w4a16_topk of y. Every argument is checked before the first launch.
 */
int w4a16_gemm_topk(const uint16_t *x, const void *packed, int M, int N, int K, int group, int sym, int k,
                    uint16_t *y, int64_t *idx, uint16_t *vals, w4a16_stream_t stream);

/*
 * Fused feed-forward gate (GRIMOIRE v1.8, "INT4 prompt processing"):
 *   h[M][N_each] = SiLU(x Wg^T) * (x Wu^T),  SiLU(v) = v / (1 + e^-v),
 * with both products accumulated in float32 and never rounded before the
 * SiLU and the product; h is rounded once to bf16. `packed_gateup` comes from
 * w4a16_repack_gateup. Any M >= 1.
 */
int w4a16_gateup_silu(const uint16_t *x, const void *packed_gateup, int M, int N_each, int K,
                      int group, int sym, uint16_t *h, w4a16_stream_t stream);

/*
 * Test export: w_out[N][K] (float32, row-major) = (q - z) * scale read back
 * from a repacked buffer through the kernels' own unpack (exact), or, for
 * sym = W4A16_AFFINE, scale * q + bias rounded once to float32.
 */
int w4a16_dequantize(const void *packed, int N, int K, int group, int sym, float *w_out,
                     w4a16_stream_t stream);

/* ------------------------------------------------------------------------
 * Affine form: w[n][k] = scale[n][k/G] * q[n][k] + bias[n][k/G]
 * (TensorFold PR #859, "What this changes" and the AffineN notes). Every
 * code is used exactly; the products x * q are summed per group on the
 * tensor cores in float32 and each group adds scale * sum + bias * X[g][m],
 * X[g][m] = sum over the group of x[m][k]. Sizes, alignment, streams and
 * errors as for the calls above.
 * ------------------------------------------------------------------------ */

/*
 * Offline repack of an affine weight: qweight as above, scales and biases
 * bf16 [N][K/G]. The biases sit in the scales' tiled layout, and once more as
 * the tcgen05 GEMM's bias operand: bf16 [rows][kb3] with each bias at three
 * consecutive columns (against the three parts of the x group sums). Writes
 * w4a16_repacked_bytes(N, K, group, W4A16_AFFINE) bytes; padding rows get
 * code 0, scale 0 and bias 0.
 */
int w4a16_repack_affine(const int32_t *qweight, const uint16_t *scales, const uint16_t *biases, int N, int K,
                        int group, void *packed, w4a16_stream_t stream);

/* The gate/up pair of w4a16_repack_gateup in the affine form. */
int w4a16_repack_affine_gateup(const int32_t *qw_gate, const uint16_t *sc_gate, const uint16_t *b_gate,
                               const int32_t *qw_up, const uint16_t *sc_up, const uint16_t *b_up, int N_each,
                               int K, int group, void *packed, w4a16_stream_t stream);

/*
 * Group sums of the activations, X[m][g] = sum_{k in group g} x[m][k] summed
 * in float32, each stored as three bf16 parts that add up to it exactly
 * (hi = bf16(X), mid = bf16(X - hi), lo = X - hi - mid): bf16 [M][kb3],
 * kb3 = 3 * K/G rounded up to 64, the parts of X[m][g] at columns 3g .. 3g+2,
 * zeros beyond 3 * K/G. The tcgen05 GEMM multiplies them by the weight's
 * biases on the tensor cores (exact bf16 products, float32 sums). They depend
 * on x alone, so one table serves every affine weight that reads the same x
 * with the same group size. `xsum` is caller-owned device memory of
 * w4a16_xsum_bytes(M, K, group) bytes, 16-byte aligned; w4a16_xsum_bytes
 * returns 0 for unsupported sizes.
 */
size_t w4a16_xsum_bytes(int M, int K, int group);
int w4a16_xsum(const uint16_t *x, int M, int K, int group, uint16_t *xsum, w4a16_stream_t stream);

/*
 * y[M][N] (bf16) = x . (scale * q + bias)^T, W from w4a16_repack_affine.
 * `xsum` (w4a16_xsum of the same x, K and group, complete when the stream
 * reaches this call) is read by the tcgen05 GEMM (M > 32); it may be NULL
 * when M <= 32, where the decode kernel forms the group sums itself with one
 * more tensor-core product per 16 k (then it is not read).
 */
int w4a16_gemm_affine(const uint16_t *x, const uint16_t *xsum, const void *packed, int M, int N, int K, int group,
                      uint16_t *y, w4a16_stream_t stream);

/*
 * w4a16_gemm_affine without the caller's group-sum table: this library's own
 * addition, with no counterpart on the pages the method comes from. For
 * M > 32 the group sums go to a fixed 4 MiB device array inside the library's
 * module image (one per device, found once with cudaGetSymbolAddress), so the
 * call allocates nothing and needs no workspace argument; sizes whose table
 * (w4a16_xsum_bytes) exceeds 4 MiB are W4A16_ERR_INVALID_ARG (at K = 5120 and
 * group 64, M up to 8,192). Every entry the GEMM reads, the zero padding
 * included, is written by the call itself before the GEMM reads it, so
 * nothing has to start at zero. The array is shared: calls in flight at the
 * same time on one device (other streams, other host threads) race on it and
 * may compute wrong results; calls in order on one stream are safe. M <= 32
 * uses no table and behaves exactly as w4a16_gemm_affine.
 */
int w4a16_gemm_affine_noalloc(const uint16_t *x, const void *packed, int M, int N, int K, int group, uint16_t *y,
                              w4a16_stream_t stream);

/* h = SiLU(x Wg^T) * (x Wu^T) as w4a16_gateup_silu, affine weights from
 * w4a16_repack_affine_gateup; `xsum` as for w4a16_gemm_affine. */
int w4a16_gateup_silu_affine(const uint16_t *x, const uint16_t *xsum, const void *packed_gateup, int M, int N_each,
                             int K, int group, uint16_t *h, w4a16_stream_t stream);

/* ------------------------------------------------------------------------
 * Affine form at other code widths: modules of 2 to 8 bits, every code
 * keeping its value, scale and bias (TensorFold PR #859, "What this changes"
 * and the native 2, 3, 5 and 6-bit tiles note): w = scale * q + bias with q in
 * 0 .. 2^bits - 1.
 *
 * Canonical qweight: uint32 [N][ceil(K * bits / 32)], one little-endian bit
 * stream per row, code k at bits [bits * k, bits * k + bits) of the row's
 * stream (running into the next word where it does not fit); at 4 bits this
 * is the nibble packing above. scales, biases: bf16 [N][K/G].
 *
 * The repacked weight reuses the 4-bit affine kernels exactly: 2- and 3-bit
 * codes are widened into the 4-bit tiles (4 bits of memory per code); 5- to
 * 8-bit codes q = 16 qh + ql become two nibble planes over K' = 2K, group g's
 * high plane (codes qh, scale 16 * scale, the bias) followed by its low plane
 * (codes ql, the scale, bias 0), multiplied by x's group g twice (8 bits of
 * memory per code). 16 * scale is exact in bf16 for |scale| < 2^123.
 * ------------------------------------------------------------------------ */

/* Bytes of the repacked b-bit weight (0 for bits outside 2..8 or unsupported sizes). */
size_t w4a16_affine_bits_repacked_bytes(int N, int K, int group, int bits);

/* Offline repack of a b-bit affine weight; packed 256-byte aligned. */
int w4a16_repack_affine_bits(const uint32_t *qweight, const uint16_t *scales, const uint16_t *biases, int N, int K,
                             int group, int bits, void *packed, w4a16_stream_t stream);

/*
 * Bytes of the caller-owned scratch a w4a16_gemm_affine_bits call needs
 * (never 0 for supported sizes; 0 means unsupported): for 5-8 bits x with
 * each group written twice, bf16 [M][2K] (256-byte aligned), then the table of
 * x group sums of w4a16_xsum for the widened K (written when M > 32).
 */
size_t w4a16_affine_bits_scratch_bytes(int M, int K, int group, int bits);

/*
 * y[M][N] (bf16) = x . (scale * q + bias)^T for a weight from
 * w4a16_repack_affine_bits. `scratch`: w4a16_affine_bits_scratch_bytes(M, K,
 * group, bits) bytes of device memory, 256-byte aligned, used only by this
 * call while it runs on `stream` (calls in flight at once need their own).
 * Launches: the widened x (5-8 bits), the group sums (M > 32), the affine
 * GEMM. The output meets the same bound as the 4-bit form.
 */
int w4a16_gemm_affine_bits(const uint16_t *x, void *scratch, const void *packed, int M, int N, int K, int group,
                           int bits, uint16_t *y, w4a16_stream_t stream);

/* Test export: w_out[N][K] (float32) = scale * q + bias of the repacked b-bit
 * weight, rounded once to float32, q read back from its nibble planes. */
int w4a16_dequantize_affine_bits(const void *packed, int N, int K, int group, int bits, float *w_out,
                                 w4a16_stream_t stream);

/* ------------------------------------------------------------------------
 * Attention of drafted tokens over a paged key/value cache, and the cache
 * itself. These calls are the rest of a speculative verify step around the
 * products above (2-16 drafted rows checked at once: GRIMOIRE v1.8 release
 * notes, "INT4 verify faster"; the greedy pick on the GPU: lucebox PR #823).
 *
 * One step: w4a16_kv_reserve gives every sequence room, w4a16_kv_append
 * writes the drafted tokens' keys and values behind each context (per layer),
 * w4a16_tree_attention attends (per layer), the head's w4a16_gemm_argmax
 * picks a token for every node, w4a16_tree_accept walks down the tree, and
 * w4a16_kv_compact moves the accepted rows together and advances the lengths.
 *
 * Arrays, all device memory:
 *   page_table  int32 [rows][max_pages]  page ids of row b's context in order;
 *               entries past the pages a row holds are -1
 *   lengths     int32 [rows]             cached tokens of each row
 *   starts      int32 [rows + 1]         tokens starts[b] .. starts[b+1] - 1 are
 *               row b's new tokens; starts[0] = 0, ascending. Tokens at
 *               starts[rows] and above are padding: not read, not written
 *   mask        int64 [tokens]           bit j of a token's word: it attends to
 *               new token j of its row (itself included: its own bit). Bits at
 *               the row's number of new tokens and above are ignored
 *   refs        int32 [pages]            how many rows hold each page; 0 = free
 * New token i of row b has position lengths[b] + i; position p is row
 * p % page_rows of page page_table[b][p / page_rows]. rows, tokens and n are
 * at least 1: a caller with nothing to do makes no call.
 *
 * What only the device can see is checked there: a page id outside the
 * cache, a position past the table, starts that descend or exceed max_tree,
 * a row index outside the table. Nothing outside a buffer is touched; the
 * offending key, row or sequence is skipped and w4a16_kernel_status()
 * returns W4A16_ERR_INDEX.
 * ------------------------------------------------------------------------ */

/* Element types of a cache. */
#define W4A16_KV_BF16 0
#define W4A16_KV_E4M3 1 /* value = code * scale[kv head] */

/*
 * A paged cache. Element (layer, page, head, row, d) of the keys sits at
 * k + layer * k_layer + page * k_page + head * k_head + row * k_row + d, in
 * elements; the values likewise. Every stride and both bases are multiples
 * of 16 bytes. dim 64, 128 or 256; page_rows 16, 32, 64, 128 or 256. Calls on
 * one layer (append, attention) take layers = 1. Pages and layers must not
 * overlap.
 */
typedef struct w4a16_kv_cache {
  void *k, *v;
  const float *k_scale, *v_scale; /* W4A16_KV_E4M3: float32 [kv_heads], positive; else NULL (calls that only move rows: not read) */
  int64_t k_layer, k_page, k_head, k_row;
  int64_t v_layer, v_page, v_head, v_row;
  int32_t layers, pages, kv_heads, page_rows, dim, type;
} w4a16_kv_cache;

/* Most new tokens of a sequence in one attention or acceptance call (bits of
 * a mask word), and most rows one fork, free or reserve call may name. */
#define W4A16_MAX_TREE 64
#define W4A16_MAX_ROWS 4096
#define W4A16_MAX_SEQUENCES 65535 /* rows of one append, attention, acceptance or compaction */

/*
 * Writes the new tokens' keys and values (bf16 [tokens][kv_heads][dim];
 * element (t, h, d) at t * k_token + h * k_head_stride + d, strides multiples
 * of 8 elements, bases 16-byte aligned) into their pages. bf16 caches: moved
 * bit by bit. E4M3 caches: x / scale[head] in float32, rounded to the nearest
 * code (ties to even) and saturated at +-448; NaN stays NaN. Any number of
 * new tokens per row, so prompts too.
 */
int w4a16_kv_append(const uint16_t *k, const uint16_t *v, int64_t k_token, int64_t k_head_stride, int64_t v_token,
                    int64_t v_head_stride, const w4a16_kv_cache *cache, const int32_t *page_table, int max_pages,
                    const int32_t *lengths, const int32_t *starts, int rows, int tokens, w4a16_stream_t stream);

/*
 * out[t][h] (bf16 [tokens][heads][dim], row-major) = softmax(q . K^T * scale) . V
 * over the positions token t sees: all lengths[b] cached ones, and new token
 * j where bit j of mask[t] is set (mask NULL: the new tokens up to and
 * including t). Query head h reads kv head h / (heads / kv_heads). A token
 * that sees nothing gets 0. Keys and values at positions a token does not see
 * do not touch its result, whatever they hold. The new tokens' keys and
 * values are read from the cache (w4a16_kv_append first).
 *
 *   q          element (t, h, d) at t * q_token + h * q_head + d, strides
 *              multiples of 8 elements, base 16-byte aligned
 *   max_tree   1 .. W4A16_MAX_TREE, at least every row's number of new tokens
 *   workspace  w4a16_tree_attention_workspace_bytes(heads, kv_heads, dim,
 *              max_tree) bytes, 256-byte aligned, used only while the call
 *              runs on `stream`; no content is kept or expected. A call makes
 *              up to two launches that share it: host threads that call at the
 *              same time need one each, also on one stream
 *
 * Scores, softmax statistics and sums are float32; a weight e^(s - max) is
 * rounded once, to 2^-8 of itself or better. Over an E4M3 cache that holds for
 * weights down to 2^-26 of the row's largest; below, a weight is off by up to
 * 2^-37 of the largest. Results are bitwise reproducible run to run on one
 * device.
 */
size_t w4a16_tree_attention_workspace_bytes(int heads, int kv_heads, int dim, int max_tree);
int w4a16_tree_attention(const uint16_t *q, int64_t q_token, int64_t q_head, const w4a16_kv_cache *cache,
                         const int32_t *page_table, int max_pages, const int32_t *lengths, const int32_t *starts,
                         const int64_t *mask, int rows, int tokens, int heads, int max_tree, float scale,
                         uint16_t *out, void *workspace, w4a16_stream_t stream);

/*
 * Greedy acceptance. target[t] is the model's pick after token t
 * (w4a16_gemm_argmax), draft[t] the drafted token at node t, mask as above
 * with ancestors at lower indices: a node's parent is its highest set bit
 * below its own. From node 0 (always accepted: the step's last committed
 * token) the walk goes to the lowest child whose draft equals the target of
 * the node it stands on, until there is none.
 *   path   int32 [rows][max_tree]  accepted nodes in order, then -1
 *   count  int32 [rows]            how many (0 for a row without new tokens)
 *   token  int64 [rows]            the target of the last one (-1 without)
 * mask NULL: one chain, node i's parent is i - 1.
 */
int w4a16_tree_accept(const int64_t *target, const int64_t *draft, const int64_t *mask, const int32_t *starts,
                      int rows, int tokens, int max_tree, int32_t *path, int32_t *count, int64_t *token,
                      w4a16_stream_t stream);

/*
 * Probabilities of the head's logits: out[t][j] (float32 [tokens][vocab],
 * row-major) = e^(l_j / T) / sum_i e^(l_i / T), over the logits of row t that are
 * not below its floor; the others get 0.
 *
 *   logits       bf16, element (t, j) at t * logits_row + j
 *   temperature  float32 [tokens], or NULL: 1. A row with T <= 0 (or NaN) is
 *                greedy: 1 at the first maximum, as w4a16_gemm_argmax, else 0
 *   floor        float32 [tokens] (the last of the row's top-k values, w4a16_topk;
 *                or its maximum + T * log(share)), or NULL: none
 *
 * A row with nothing above -inf gets 0 throughout; a NaN (or +inf) that is kept
 * makes the row's kept probabilities NaN. A probability is off by less than 2^-17 +
 * 2^-22 (max - l_j) / T of itself; below 2^-126 it may be 0. A T between 0 and 2^-127
 * counts as 2^-127. out must not overlap what is read.
 */
int w4a16_probabilities(const uint16_t *logits, int64_t logits_row, const float *temperature, const float *floor,
                        int tokens, int vocab, float *out, w4a16_stream_t stream);

/*
 * Sampled acceptance: w4a16_tree_accept for a target that samples. p and q are
 * the target's and the drafter's probabilities after each token (float32,
 * element (t, j) at t * p_row + j; 0 <= p, q <= 1, a row's sum below 2). The
 * children of a node were drawn from q at it, each on its own; q NULL: they were
 * picked without chance (the likeliest tokens, a lookup). From node 0 (always
 * accepted) the walk asks the children of the node it stands on, lowest first:
 *
 *   child x is accepted where u[x] * q(x) * S < max(p(x) - c * q(x), 0); the walk
 *   goes on from there. c = 0 and S = 1 for the first child; a refusal makes
 *   c += S, S = sum_j max(p_j - c * q_j, 0)
 *   (q NULL: q is 1 at the child alone. A refused child's probability is taken
 *   out of p, S is the sum of the rest, and the same token again is refused.)
 *
 * At the end the token is drawn from what is left there, w_j = max(p_j - c *
 * q_j, 0): the first j with w_0 + ... + w_j > u[root] * sum w. Where that leaves
 * nothing p itself is w; a row of p without probability gives token -1. So
 * accepted tokens and the drawn one are distributed as if sampled from p one by
 * one.
 *
 *   draft, mask, starts, max_tree, path, count as in w4a16_tree_accept
 *   u      float32 [tokens], in [0, 1): each node's own number, the root's for
 *          the token
 *   token  int64 [rows]  the token drawn (-1 for a row without new tokens)
 *
 * A NaN or negative probability counts as 0, one above 1 as 1; a drafted token
 * outside the vocabulary is passed over (W4A16_ERR_INDEX). A walk that meets a sum
 * of 64 or a c of 128 ends there with token -1 (W4A16_ERR_INDEX too; rows that sum
 * to less than 2 have neither). Probabilities (and what
 * refusals leave of each) are rounded to multiples of 2^-46 and summed exactly,
 * tests are double: results do not depend on any order.
 */
int w4a16_tree_sample(const float *p, int64_t p_row, const float *q, int64_t q_row, int vocab, const int64_t *draft,
                      const int64_t *mask, const int32_t *starts, const float *u, int rows, int tokens, int max_tree,
                      int32_t *path, int32_t *count, int64_t *token, w4a16_stream_t stream);

/*
 * Keeps the accepted rows: in every layer and head, position lengths[b] +
 * path[b][i] moves to lengths[b] + i for i < count[b], and lengths_out[b] =
 * lengths[b] + count[b]. path[b] ascends (as w4a16_tree_accept gives it).
 * lengths_out must not overlap lengths.
 */
int w4a16_kv_compact(const w4a16_kv_cache *cache, const int32_t *page_table, int max_pages, const int32_t *lengths,
                     const int32_t *path, const int32_t *count, int rows, int max_tree, int32_t *lengths_out,
                     w4a16_stream_t stream);

/*
 * Drops the `n` table rows rows[0 .. n-1] (distinct): one reference of every
 * page they hold, their table entries become -1 and their lengths 0.
 */
int w4a16_kv_free(int32_t *page_table, int max_pages, int table_rows, int32_t *lengths, int32_t *refs, int pages,
                  const int32_t *rows, int n, w4a16_stream_t stream);

/*
 * Branches: for each j < n, the empty table row dst[j] becomes a copy of row
 * src[j]. Whole pages are shared (one more reference); a part-filled last
 * page is copied, in every layer, into a free page of its own (only the rows
 * in use). dst are distinct and empty (freed, or never used); a src may be named many times. Free
 * pages are taken lowest id first, in the order of j. All or nothing: ok[0] =
 * 1, or 0 and nothing changed when the free pages do not suffice (or an index
 * is bad: then W4A16_ERR_INDEX too). Pages that a src holds past its length
 * (w4a16_kv_reserve) are not shared.
 */
int w4a16_kv_fork(const w4a16_kv_cache *cache, int32_t *page_table, int max_pages, int table_rows, int32_t *lengths,
                  int32_t *refs, const int32_t *src, const int32_t *dst, int n, int32_t *ok, w4a16_stream_t stream);

/*
 * Room to grow: row rows[j] (distinct) gets free pages, lowest id first in
 * the order of j, until it holds want[j] tokens. All or nothing, as above.
 */
int w4a16_kv_reserve(int32_t *page_table, int max_pages, int table_rows, int32_t *refs, int pages, int page_rows,
                     const int32_t *rows, const int32_t *want, int n, int32_t *ok, w4a16_stream_t stream);

/* ------------------------------------------------------------------------
 * Low-rank adapters of many requests beside one product:
 *
 *   out[t] = y[t] + scale[e] * (x[t] . A[e]^T) . B[e]^T,  e = adapter[b]
 *
 * for the tokens t of row b (starts[b] .. starts[b + 1] - 1, as above; starts
 * NULL: rows = tokens and each token is a row). y is what a w4a16 product gave
 * for the same x. A row with adapter -1 gets y, bit by bit.
 *
 *   y, out     bf16 [tokens][outer], element (t, n) at t * row stride + n (row
 *              strides of y, out and x below 2^30 elements). out
 *              may be y (then rows without an adapter are not touched); it must
 *              not overlap y otherwise (other columns of the same wider rows
 *              are apart), nor x, a or b
 *   x          bf16 [tokens][inner], x_row a multiple of 8, base 16-byte aligned
 *   a          bf16 [adapters][rank][inner], b bf16 [adapters][outer][rank]:
 *              strides multiples of 8, bases 16-byte aligned
 *   scale      float32 [adapters], or NULL: 1
 *   adapter    int32 [rows]
 *   adapters   1 .. W4A16_MAX_ADAPTERS; rank a multiple of 8 up to
 *              W4A16_MAX_RANK (smaller adapters padded with zeros); inner a
 *              multiple of 8; outer any
 *   workspace  w4a16_lora_workspace_bytes(tokens, rank, inner) bytes, 256-byte
 *              aligned, used only while the call runs on `stream`. A call makes
 *              two launches that share it. (The size grows with each argument:
 *              one for the largest call is enough for smaller ones)
 *
 * Sums are float32; x A^T goes into the second product whole, or (above rank 32, in
 * the kernels for prompts, so never up to 128 tokens) with 16 bits of mantissa; out is
 * rounded once. Results are bitwise reproducible, and a token's does not depend on
 * what the tokens beside it hold (on how many there are by the order of its sums, and
 * those 16 bits). What is not finite stays with its token, or with its adapter and
 * column, and is what the formula says (an infinite weight times values of x A^T from
 * 2^-95 on). Tokens at starts[rows] and above are not read and not written. An adapter
 * outside -1 .. adapters - 1 counts as -1, a row whose offsets cannot be is left
 * out, and where offsets descend, tokens of a row that lie before the end of an earlier
 * one are that one's, or nobody's (then they are not written);
 * w4a16_kernel_status() then returns W4A16_ERR_INDEX.
 * ------------------------------------------------------------------------ */
#define W4A16_MAX_ADAPTERS 4096
#define W4A16_MAX_RANK 128
size_t w4a16_lora_workspace_bytes(int tokens, int rank, int inner);
int w4a16_lora_add(const uint16_t *y, int64_t y_row, const uint16_t *x, int64_t x_row, const uint16_t *a,
                   int64_t a_adapter, int64_t a_row, const uint16_t *b, int64_t b_adapter, int64_t b_row,
                   const float *scale, const int32_t *adapter, const int32_t *starts, int rows, int tokens,
                   int adapters, int rank, int inner, int outer, uint16_t *out, int64_t out_row, void *workspace,
                   w4a16_stream_t stream);

/*
 * Waits for all work on the current device, then reads and clears the
 * device error word that a kernel sets when one of its bounded waits gave up
 * (W4A16_ERR_TIMEOUT; the kernel's outputs are then undefined) or when one
 * of the cache calls skipped an index outside its buffers (W4A16_ERR_INDEX).
 * W4A16_OK when neither happened since the last call.
 */
int w4a16_kernel_status(void);

/* Static string for a status code. */
const char *w4a16_strerror(int status);

/* cudaError_t of the last W4A16_ERR_CUDA on this thread (0 if none). */
int w4a16_last_cuda_error(void);

/*
 * Kernel selection override for A/B measurement: 0 = automatic (default),
 * 1 = force the CUDA-core one-row GEMV for M = 1 (zero-point forms), 2 = force
 * the small-M tensor-core kernel with per-warp weight rings for M <= 32, 3 =
 * force the tcgen05 GEMM for any M, 4 = force the small-M kernel that stages x
 * once per CTA for M <= 16 (automatic choice: M <= 8 calls whose grid of
 * 128-row CTAs fills the GPU, e.g. the output-vocabulary head), 5 = force the
 * tcgen05 decode kernel (weights dequantised into tensor memory) for plain
 * zero-point and symmetric w4a16_gemm calls with M <= 32.
 * Returns the previous value. Process-wide; not thread-safe against
 * concurrent calls.
 */
int w4a16_set_kernel_override(int which);

/*
 * Programmatic overlap of consecutive decode calls (M <= 32), off by default.
 * When on, the M <= 32 kernels are launched with programmatic stream
 * serialization: a call may start while the previous kernel on its stream is
 * still running, begin streaming its packed weights (and scales and zeros)
 * at once, and wait for that kernel to finish (and its writes to become
 * visible) before it reads x or writes y / h. This hides each call's launch
 * and weight-fetch ramp behind the tail of the call before it, the common
 * case of decode layers run back to back (also inside CUDA graphs).
 * Turn it on only while the packed buffers are read-only: written once (at
 * load time, e.g. by w4a16_repack), then made complete by a synchronization
 * (cudaStreamSynchronize or an event the stream waits on) before the first
 * call that uses them, because the weight reads of a call are not ordered
 * after kernels still in flight on its stream. Process-wide; the setting is
 * read when a call is launched. Returns the previous setting (0 or 1), or -1
 * for a value other than 0 or 1.
 */
int w4a16_set_programmatic_overlap(int on);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_H_ */
