/*
 * bitlinear.h -- C ABI of the B200 (sm_100a) BitLinear library.
 *
 * The library computes the forward pass of a BitNet a4.8 BitLinear layer:
 * ternary {-1, 0, +1} weights stored at 2 bits, multiplied by per-token
 * quantised activations. Sources (web pages on the method):
 *   [R] "BitNet a4.8: 4-bit Activations for 1-bit LLMs", Telegram review
 *       (t.center/ru/toshoseti/992), sections "Метод" and "Эксперименты".
 *   [A] "BitNet a4.8: 4-bit Activations for 1-bit LLMs", arXiv 2411.04965
 *       summary page, section "摘要（原文）" (English abstract).
 *
 * Conventions (all entry points):
 *   - Return value: BITLINEAR_OK (0) or a negative BITLINEAR_ERR_* code.
 *     bitlinear_last_error() gives a message for the calling thread.
 *   - Argument errors are found on the host and returned before any launch.
 *   - "device" pointers are CUDA global memory owned by the caller; the
 *     library never allocates, frees or keeps them. Work is asynchronous on
 *     the given stream (NULL = legacy default stream).
 *   - bf16 values are passed as their 16-bit patterns (uint16_t).
 *   - Matrices are row-major. X is M x K (one row per token); weights are
 *     described as W [K x N] (in x out) and stored transposed and packed.
 *   - M == 0 is a valid empty call: nothing is launched.
 *   - Device pointers to TMA-read operands must be 16-byte aligned.
 *   - Launches go to the device current on the calling thread. Each kernel's
 *     shared-memory limit is raised once per device (thread-safe), so one
 *     process may drive several GPUs.
 *   - dev_status (nullable, device int): a kernel that gives up a bounded
 *     wait ORs BITLINEAR_STATUS_TIMEOUT into it and returns early; the
 *     output is then undefined. The paged-cache calls also report indexes
 *     that lie outside their tensors (BITLINEAR_STATUS_BAD_INDEX) and a pool
 *     without enough free pages (BITLINEAR_STATUS_NO_PAGES). The caller
 *     zeroes it; read it with bitlinear_check_status().
 */
#ifndef BITLINEAR_H
#define BITLINEAR_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* bitlinear_stream_t; /* same type as cudaStream_t */

enum {
  BITLINEAR_OK = 0,
  BITLINEAR_ERR_INVALID_ARG = -1,
  BITLINEAR_ERR_ALIGNMENT = -2,
  BITLINEAR_ERR_UNSUPPORTED = -3,
  BITLINEAR_ERR_CUDA = -4,
  BITLINEAR_ERR_TIMEOUT = -5,
  BITLINEAR_ERR_INDEX = -6,   /* a kernel met an index outside its tensors */
  BITLINEAR_ERR_NO_PAGES = -7 /* fewer free pages than wanted */
};

enum { BITLINEAR_MODE_INT8 = 0, BITLINEAR_MODE_INT4 = 1, BITLINEAR_MODE_FP4 = 2 };

enum { BITLINEAR_STATUS_TIMEOUT = 1, BITLINEAR_STATUS_BAD_INDEX = 2, BITLINEAR_STATUS_NO_PAGES = 4 };

/* Message for the last error returned on this thread ("" if none). */
const char* bitlinear_last_error(void);

/* Library ABI version (major * 100 + minor). */
int bitlinear_version(void);

/*
 * Offline weight preparation (HOST memory, synchronous, no GPU needed).
 * Ternary weights: [R] "Метод". The pages give no scale or rounding rule;
 * this library uses absmean per column group g:
 *   gamma_g = max((float)(sum |W[k,n]| over the group, fp64, row-major order
 *             / count), 1e-5f)
 *   W_t[k,n] = clamp(round_half_even(W[k,n] / gamma_g), -1, 1)   (fp32 divide)
 * and packs code c = W_t + 1 in {0,1,2} at 2 bits: row n of Wp holds K/4
 * bytes; the little-endian 32-bit word j covers k = 16j .. 16j+15 and holds
 * element 16j + 8h + i (h in {0,1}, i in 0..7) in bits [4i+2h, 4i+2h+2).
 *   W          fp32 [K x N] row-major (host)
 *   group_ends G increasing column ends, group_ends[G-1] == N (host); G in 1..8
 *   Wp         uint8 [N x K/4] (host, written)
 *   gamma      fp32 [G] (host, written)
 * Requires K % 16 == 0, N >= 1.
 */
int bitlinear_ternarize_pack(const float* W, int64_t K, int64_t N, const int64_t* group_ends,
                             int G, uint8_t* Wp, float* gamma);

/*
 * Per-token activation quantiser ([A] abstract: 4-bit activations on the
 * inputs of attention and FFN; [R] "Метод": INT4 or FP4, absmax INT8).
 * Per row m, in fp32: a' = max(max_k |h[m,k]|, 1e-5f), then
 *   INT8 / INT4 (Q = 127 / 7): q = clamp(rne(h * (Q / a')), -Q-1, Q) as int8
 *   FP4: v = h * (6 / a') rounded to e2m1 (nearest, ties to even, saturating
 *        at 6, sign of v kept), two per byte, even k in the low nibble
 *   xs[m] = a' / Q   (Q = 6 for FP4): the dequantisation multiplier.
 * h = x, or when up != NULL the ReLU^2-gated product ([R] "Метод": ReLU^2 in
 * the FFN gate) h = (r * r) * up with r = (x > 0 ? x : 0), all in fp32.
 *   x, up   device bf16 [M x ldx] (row stride ldx elements); up nullable
 *   q_out   device int8 [M x K] for INT8/INT4, uint8 [M x K/2] for FP4
 *   xs_out  device fp32 [M]
 * Requires K % 16 == 0, K <= 49152, ldx >= K, ldx % 8 == 0.
 */
int bitlinear_quant_act(const uint16_t* x, const uint16_t* up, int64_t M, int64_t K, int64_t ldx,
                        int mode, void* q_out, float* xs_out, bitlinear_stream_t stream);

/*
 * Top-k sparsification then INT8 ([R] "Метод": top-k with 50% sparsity on
 * the out_proj input; [A] abstract: sparsified intermediate states then
 * 8-bit quantisation). Per row: keep the k largest |x| (compared as bf16
 * magnitude bits; equal magnitudes kept lowest column first), zero the rest,
 * then the INT8 quantiser above on the sparsified row.
 *   k        0 selects ceil(K/2); values above K keep the whole row
 *   q_out    device int8 [M x K]; xs_out device fp32 [M]
 *   mask_out nullable device uint8 [M x K/8]: bit (k % 8) of byte k/8 = kept
 * Requires K % 16 == 0, K <= 16384, ldx >= K, ldx % 8 == 0.
 */
int bitlinear_topk_sparsify_i8(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, int64_t k,
                               int8_t* q_out, float* xs_out, uint8_t* mask_out,
                               bitlinear_stream_t stream);

/*
 * BitLinear GEMM, ternary weights x 8-bit integer activation codes
 * ([A] abstract; [R] "Метод"), on tcgen05 tensor cores:
 *   acc[m,n] = sum_k xq[m,k] * W_t[k,n]                (exact int32)
 *   y[m,n]   = bf16_rne((float)acc * (xs[m] * gamma[g(n)]))  (fp32 multiplies)
 *   xq         device int8 [M x K], row stride K
 *   xs         device fp32 [M]
 *   Wp         device uint8 [N x K/4] from bitlinear_ternarize_pack
 *   gamma      device fp32 [G];  group_ends HOST int64 [G] (as for the pack)
 *   y          device bf16 [M x ldy]
 * Requires K % 64 == 0, K <= 32768 (|acc| < 2^22, converted exactly to fp32),
 * N % 16 == 0, ldy >= N, ldy % 8 == 0, G in 1..8.
 * The w2a4 entry point takes INT4 codes ([-8, 7]) in int8 containers: sm_100
 * tensor cores have no 4-bit integer kind, so both run the s8 MMA.
 */
int bitlinear_gemm_w2a8(const int8_t* xq, const float* xs, const uint8_t* Wp, const float* gamma,
                        const int64_t* group_ends, int G, int64_t M, int64_t N, int64_t K,
                        uint16_t* y, int64_t ldy, int* dev_status, bitlinear_stream_t stream);
int bitlinear_gemm_w2a4(const int8_t* xq, const float* xs, const uint8_t* Wp, const float* gamma,
                        const int64_t* group_ends, int G, int64_t M, int64_t N, int64_t K,
                        uint16_t* y, int64_t ldy, int* dev_status, bitlinear_stream_t stream);

/*
 * BitLinear GEMM, ternary weights x FP4 (e2m1) activations ([R] "Метод":
 * FP4 variant; [A] abstract: INT4/FP4 kernels). acc = sum of e2m1 values x
 * W_t in fp32 (exact: multiples of 0.5 below 2^24), same epilogue as above.
 *   xf4  device uint8 [M x K/2] packed e2m1 from bitlinear_quant_act(FP4)
 * Requires K % 128 == 0 and the w2a8 requirements.
 */
int bitlinear_gemm_w2fp4(const uint8_t* xf4, const float* xs, const uint8_t* Wp,
                         const float* gamma, const int64_t* group_ends, int G, int64_t M,
                         int64_t N, int64_t K, uint16_t* y, int64_t ldy, int* dev_status,
                         bitlinear_stream_t stream);

/* The same GEMMs writing the raw accumulators instead of bf16 (for checking
 * the contraction alone): acc device int32 / fp32 [M x N], row stride N. */
int bitlinear_gemm_w2a8_acc(const int8_t* xq, const uint8_t* Wp, int64_t M, int64_t N, int64_t K,
                            int32_t* acc, int* dev_status, bitlinear_stream_t stream);
int bitlinear_gemm_w2fp4_acc(const uint8_t* xf4, const uint8_t* Wp, int64_t M, int64_t N,
                             int64_t K, float* acc, int* dev_status, bitlinear_stream_t stream);

/*
 * Decode-time BitLinear (few tokens): same inputs and result as
 * bitlinear_gemm_w2a8 for 1 <= M <= 64, with weights streamed once from HBM.
 * Requires K % 128 == 0, N % 128 == 0 and the w2a8 requirements.
 */
int bitlinear_gemv_w2(const int8_t* xq, const float* xs, const uint8_t* Wp, const float* gamma,
                      const int64_t* group_ends, int G, int64_t M, int64_t N, int64_t K,
                      uint16_t* y, int64_t ldy, int* dev_status, bitlinear_stream_t stream);

/*
 * Decode-time BitLinear with the activation quantiser fused in: the same
 * result, bit for bit, as bitlinear_quant_act(x, up, M, K, ldx, mode) followed
 * by bitlinear_gemv_w2 on its codes ([R] "Метод": INT4 codes on the q/k/v and
 * gate/up inputs, ReLU^2 gate then INT8 on the down_proj input; [A] abstract:
 * 4-bit activations), without the codes ever reaching HBM: every CTA
 * quantises the few token rows itself.
 *   x, up   device bf16 [M x ldx]; up nullable (ReLU^2 gate when given)
 *   mode    BITLINEAR_MODE_INT8 or BITLINEAR_MODE_INT4
 *   other arguments as bitlinear_gemv_w2
 * Requires 1 <= M <= 8 (BITLINEAR_ERR_UNSUPPORTED above), ldx >= K,
 * ldx % 8 == 0, x and up 16-byte aligned, and the bitlinear_gemv_w2
 * requirements.
 */
int bitlinear_gemv_w2_quant(const uint16_t* x, const uint16_t* up, int64_t ldx, int mode,
                            const uint8_t* Wp, const float* gamma, const int64_t* group_ends, int G,
                            int64_t M, int64_t N, int64_t K, uint16_t* y, int64_t ldy,
                            int* dev_status, bitlinear_stream_t stream);

/*
 * KV-cache quantiser ([R] "Эксперименты": 3-bit KV cache, the <bos> and
 * <eos> tokens kept at 4 bits). Per (token t, head h) over the head dim:
 *   a' = max(max_d |x|, 1e-5f); tokens listed in keep4_pos: Q = 7, codes in
 *   [-8, 7]; others: Q = 3, codes in [-4, 3]; code = clamp(rne(x * (Q / a')))
 *   scale[t,h] = a' / Q
 * Storage: codes3 row (t,h) = 3D/8 bytes, code + 4 as a little-endian 3-bit
 * stream (code d in bits [3d, 3d+3)); all zero for 4-bit tokens.
 * codes4 row (j,h) for the j-th listed token = D/2 bytes, code + 8, low
 * nibble first.
 *   kv         device bf16 [T x H x D]
 *   keep4_pos  device int32 [n_keep4], strictly increasing positions < T
 *              (nullable iff n_keep4 == 0)
 *   codes3     device uint8 [T x H x 3D/8]
 *   codes4     device uint8 [n_keep4 x H x D/2] (nullable iff n_keep4 == 0)
 *   scale      device fp32 [T x H]
 * Requires D in {64, 128, 256}.
 */
int kv_quant_3bit(const uint16_t* kv, int64_t T, int64_t H, int64_t D, const int32_t* keep4_pos,
                  int64_t n_keep4, uint8_t* codes3, uint8_t* codes4, float* scale,
                  bitlinear_stream_t stream);

/*
 * The same quantiser ([R] "Эксперименты") applied to the K and the V cache
 * of a layer in one launch: k_* are written exactly as kv_quant_3bit(k, ...)
 * would write them, v_* as kv_quant_3bit(v, ...), with one keep4_pos list
 * for both. Saves the second launch's ramp when both are quantised
 * together, as in a decoder layer. Same requirements, per tensor, as
 * kv_quant_3bit; the two tensors may not overlap their outputs.
 */
int kv_quant_3bit_kv(const uint16_t* k, const uint16_t* v, int64_t T, int64_t H, int64_t D,
                     const int32_t* keep4_pos, int64_t n_keep4, uint8_t* k_codes3, uint8_t* k_codes4,
                     float* k_scale, uint8_t* v_codes3, uint8_t* v_codes4, float* v_scale,
                     bitlinear_stream_t stream);

/*
 * The positions kept at 4 bits, from the token ids ([R] "Эксперименты": the
 * <bos> and <eos> tokens stay at 4 bits): every t < T whose token_ids[t]
 * equals one of special_ids, in increasing order; the list kv_quant_3bit and
 * kv_attention_3bit take.
 *   token_ids    device int32 [T]
 *   special_ids  host int32 [n_special], 1 <= n_special <= 8 (e.g. the bos
 *                and eos ids)
 *   pos_out      device int32 [T]; the first *count_out entries are written
 *   count_out    device int32 [1]
 * Runs as one block on the stream (the count is device memory: read it back
 * to size the list on the host).
 */
int kv_keep4_positions(const int32_t* token_ids, int64_t T, const int32_t* special_ids,
                       int n_special, int32_t* pos_out, int32_t* count_out,
                       bitlinear_stream_t stream);

/*
 * Decode attention over that cache ([R] "Эксперименты": the 3-bit KV cache
 * with <bos>/<eos> at 4 bits is what attention reads at inference). For
 * every query (b, h) and every cached token t < T of head h:
 *   s_t = (q[b,h] . k[t,h]) / sqrt(D),  p = softmax_t(s),
 *   out[b,h] = bf16_rne(sum_t p_t v[t,h])
 * with k, v dequantised from the kv_quant_3bit storage ((code) * scale), in
 * fp32 with an online softmax. Agrees with the fp64 result within one bf16
 * ulp plus 2^-16 (sum_t p_t |v_t| + |out|) per element (fp32 rounding of
 * the D-term scores and of the weighted sums).
 *   q          device bf16 [B x H x D]
 *   k_*, v_*   codes3 / codes4 / scale of K and V as written by kv_quant_3bit
 *              with the same keep4_pos list (codes4 nullable iff n_keep4 == 0)
 *   keep4_pos  device int32 [n_keep4], strictly increasing, n_keep4 <= 1024
 *   out        device bf16 [B x H x D]
 *   dev_status as for the GEMMs (bounded waits on the cache tiles)
 * Requires D in {128, 256}, H % 4 == 0, T >= 1, every pointer but keep4_pos
 * 16-byte aligned (codes4 only when n_keep4 > 0); B == 0 launches nothing.
 */
int kv_attention_3bit(const uint16_t* q, int64_t B, int64_t H, int64_t D, int64_t T,
                      const uint8_t* k_codes3, const uint8_t* k_codes4, const float* k_scale,
                      const uint8_t* v_codes3, const uint8_t* v_codes4, const float* v_scale,
                      const int32_t* keep4_pos, int64_t n_keep4, uint16_t* out, int* dev_status,
                      bitlinear_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * The paged 3-bit KV cache: the kv_quant_3bit storage ([R] "Эксперименты":
 * 3-bit KV cache, <bos> and <eos> kept at 4 bits) in pages of
 * BITLINEAR_PAGE_TOKENS tokens, for batches of sequences that grow, fork and
 * end, and that may share the pages of a common prefix.
 *
 * Pool of one layer: `pages`, device uint8 [n_pages x H x block] with
 * block = kv_page_block_bytes(D); the block of a (page, head) holds, with
 * RB = 3D/8,
 *   bytes [0, 64 RB)        K codes: row o (the page's token o) at o RB, the
 *                           little-endian 3-bit stream of kv_quant_3bit
 *   bytes [64 RB, 128 RB)   V codes: byte i of token o's row at
 *                           64 RB + (o / 4) 4 RB + 4 i + o % 4
 *   fp32 [64], fp32 [64]    K scales, V scales
 * A token kept at 4 bits has its K scale stored negated, zero bytes for its
 * 3-bit rows but for byte 0 of the K row, which is j, and its 4-bit rows in
 * row j of `codes4`, device uint8 [n_pages x H x C4 x D]: K's D/2 bytes, then
 * V's (code + 8, low nibble first). C4 (0..64, 0: no codes4) is the pool's
 * number of 4-bit rows a page.
 * A pool of L layers holds the layers' pools one behind the other:
 * [L x n_pages x H x block]; page p means page p of every layer.
 *
 * Sequences: row r of `tables`, device int32 [R x W] with rows ldt apart,
 * lists the pages of sequence r: its token t lies in page tables[r][t / 64].
 * lens[r] is its number of tokens (0: none); the entries behind its last page
 * say nothing. refs[p] is how many table entries name page p; a page is free
 * exactly when refs[p] == 0.
 *
 * Indexes in device memory cannot be checked on the host: an entry that lies
 * outside its tensor is left out (never accessed) and reported in dev_status.
 * Calls that share a pool or its tables are ordered by their stream, or by
 * the caller.
 * ---------------------------------------------------------------------------
 */
#define BITLINEAR_PAGE_TOKENS 64

/* Bytes of the block of a (page, head): 64 (3D/4 + 8); 0 if D is none of
 * 64, 128, 256. */
int64_t kv_page_block_bytes(int64_t D);

/*
 * Quantise new tokens into a pool: token i of k and v is written to slot
 * slots[i] = page * 64 + place in the page, exactly as kv_quant_3bit
 * quantises it (4 bits where row4[i] >= 0).
 *   k, v     device bf16 [n x H x D], tokens ldk / ldv elements apart (slices
 *            of a fused projection's output will do)
 *   slots    device int32 [n]; negative: the token is left out. Slots that
 *            are not negative are distinct
 *   row4     device int32 [n], nullable: the 4-bit row of the token's page
 *            that takes token i, 0 .. C4 - 1, or negative: 3 bits. Tokens of
 *            one page have distinct rows
 *   pages, codes4   one layer's pool, written; codes4 nullable iff C4 == 0
 * Requires D in {64, 128, 256}, ldk, ldv >= H D and multiples of 8, k, v,
 * pages, codes4 16-byte aligned, finite values (a row with others is stored
 * as some row).
 */
int kv_append_3bit(const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv, int64_t n,
                   int64_t H, int64_t D, const int32_t* slots, const int32_t* row4, uint8_t* pages,
                   int64_t n_pages, uint8_t* codes4, int64_t C4, int* dev_status,
                   bitlinear_stream_t stream);

/*
 * Copy page src[i] onto page dst[i], in all L layers.
 *   pages    device uint8 [L x n_pages x page_bytes], page_bytes = H * block
 *   codes4   device uint8 [L x n_pages x page_bytes4], page_bytes4 = H C4 D;
 *            nullable iff page_bytes4 == 0
 *   src, dst device int32 [n]; a pair of two negative pages is left out. No
 *            page is the destination of two pairs, or source and destination
 * Requires page_bytes, page_bytes4 multiples of 16 and 16-byte aligned pools.
 */
int kv_pages_copy(uint8_t* pages, int64_t page_bytes, uint8_t* codes4, int64_t page_bytes4,
                  int64_t L, int64_t n_pages, const int32_t* src, const int32_t* dst, int64_t n,
                  int* dev_status, bitlinear_stream_t stream);

/*
 * Fork sequences: row children[i] becomes the sequence of row parents[i],
 * on the same pages (their reference counts rise by one).
 *   parents, children  device int32 [n], n <= 65535
 * A child holds no tokens before, and no entry's parent is among the
 * children: entries that break this are left out and reported. Of the entries
 * that name one child the first counts, the others are left out and reported.
 */
int kv_pages_fork(int32_t* tables, int64_t R, int64_t W, int64_t ldt, int32_t* lens, int32_t* refs,
                  int64_t n_pages, const int32_t* parents, const int32_t* children, int64_t n,
                  int* dev_status, bitlinear_stream_t stream);

/*
 * Make room for n_new[i] more tokens of row rows[i], and list their slots.
 * The entries are served as if one after the other: a partly filled last
 * page with another reference is left to the others and copied to a new page
 * (in all L layers); further pages follow as the tokens need them. New pages
 * are the lowest free ones. If the pool has fewer free pages than all entries
 * need, none is served (BITLINEAR_STATUS_NO_PAGES): lengths, references and
 * the tables' entries of the sequences stay, and all slots are negative.
 *   pages, codes4, L, page_bytes, page_bytes4   as for kv_pages_copy
 *   rows     device int32 [n], n <= 1024, distinct: a row named again is left
 *            out and reported
 *   n_new    device int32 [n], each 0 .. max_new
 *   slots    device int32 [n x max_new], written: the slots of row rows[i]'s
 *            new tokens, then -1: what kv_append_3bit takes
 *   work     device int32 [2 n], written
 * Rows whose tokens would not fit into W pages are left out and reported.
 */
int kv_pages_grow(uint8_t* pages, int64_t page_bytes, uint8_t* codes4, int64_t page_bytes4,
                  int64_t L, int64_t n_pages, int32_t* tables, int64_t R, int64_t W, int64_t ldt,
                  int32_t* lens, int32_t* refs, const int32_t* rows, const int32_t* n_new,
                  int64_t n, int64_t max_new, int32_t* slots, int32_t* work, int* dev_status,
                  bitlinear_stream_t stream);

/*
 * End sequences, or take back their last tokens: row rows[i] keeps its first
 * keep[i] tokens (0 where keep is NULL; all where it has no more), and the
 * pages behind them lose its reference. A row named again counts once.
 *   rows, keep  device int32 [n], n <= 65535; keep nullable, not negative
 */
int kv_pages_free(int32_t* tables, int64_t R, int64_t W, int64_t ldt, int32_t* lens, int32_t* refs,
                  int64_t n_pages, const int32_t* rows, const int32_t* keep, int64_t n,
                  int* dev_status, bitlinear_stream_t stream);

/*
 * Move the n_live pages in use to the front of the pool: the k-th free page
 * below n_live takes the k-th page in use at or above it (in all L layers),
 * and the tables of all R rows follow.
 * Page ids that are kept elsewhere do not: after the call, take the list of a
 * shared prefix (kv_attention_3bit_paged's `shared`) again from the table of a
 * row that holds it. The old list names other pages, and no call can tell.
 *   n_live   device int32 [1], written: the pages from n_live on are free
 *   work     device int32 [2 n_pages + 3], written
 */
int kv_pages_compact(uint8_t* pages, int64_t page_bytes, uint8_t* codes4, int64_t page_bytes4,
                     int64_t L, int64_t n_pages, int32_t* tables, int64_t R, int64_t W, int64_t ldt,
                     int32_t* lens, int32_t* refs, int32_t* n_live, int32_t* work, int* dev_status,
                     bitlinear_stream_t stream);

/*
 * Decode attention over a paged cache, the pages of a shared prefix read once
 * for the whole batch. Sequence b has lens[b] tokens, of which the last Sq are
 * its queries' own (already appended): token t lies in page shared[t / 64]
 * while t < 64 n_shared, and in page tables[b][t / 64 - n_shared] after that.
 * Query i of sequence b sees the tokens t < lens[b] - Sq + 1 + i; query head
 * hq reads cache head hq / (Hq / H):
 *   s_t = (q . k_t) / sqrt(D),  p = softmax_t(s),
 *   out[b,i,hq] = bf16_rne(sum_t p_t v_t), zero where no token is seen
 * with k, v dequantised from the pages (code * scale), sums in 32 bits. A
 * token's weight p_t x (V scale) enters the products as a whole number (up to
 * 2 rows of a head) or as two 16-bit floats: 2^-22 of it or 2^-30 of the row's
 * largest weight, whichever is more, may be lost.
 *   q        device bf16 [B x Sq x Hq x D], tokens (b, i) ldq elements apart
 *   pages, codes4   one layer's pool
 *   shared   device int32 [n_shared], nullable iff n_shared == 0
 *   tables   device int32 [B x W], rows ldt apart, nullable iff W == 0: the
 *            pages behind the shared ones (columns n_shared and up of the
 *            kv_pages_* tables of sequences forked from one prefix)
 *   lens     device int32 [B]
 *   out      device bf16 [B x Sq x Hq x D]
 *   work     device memory of at least kv_attention_3bit_paged_workspace()
 *            bytes, 16-byte aligned, for this call alone until it has run
 *            (nullable iff that is 0)
 * Requires D in {64, 128, 256}, Hq a multiple of H, Sq <= 128, B <= 65535,
 * ldq >= Hq D and a multiple of 8, q, pages, codes4, out 16-byte aligned, and
 * finite q and scales.
 */
int64_t kv_attention_3bit_paged_workspace(int64_t B, int64_t Sq, int64_t Hq, int64_t H, int64_t D,
                                          int64_t n_shared, int64_t W);
int kv_attention_3bit_paged(const uint16_t* q, int64_t ldq, int64_t B, int64_t Sq, int64_t Hq,
                            int64_t H, int64_t D, const uint8_t* pages, int64_t n_pages,
                            const uint8_t* codes4, int64_t C4, const int32_t* shared,
                            int64_t n_shared, const int32_t* tables, int64_t W, int64_t ldt,
                            const int32_t* lens, uint16_t* out, void* work, int64_t work_bytes,
                            int* dev_status, bitlinear_stream_t stream);

/*
 * Measurement helper (not part of the method): the dense tensor-pipe rate of
 * this GPU in the MMA shapes the GEMMs issue, for roofline denominators.
 * Launches one CTA pair per two SMs (kind 0, 1) or one CTA per SM (kind 2);
 * each issues 4 * iters back-to-back tcgen05 MMAs on operands resident in
 * shared memory (no unpack, no global reads) and writes the device time of
 * its stream, in ns, to ns_out[unit].
 *   kind 0: kind::i8, CTA pair, M = 256, N = 256, K = 32 (2 M N K ops each)
 *   kind 1: kind::mxf4, CTA pair, M = 256, N = 256, K = 64, unit scales
 *   kind 2: kind::i8, one CTA, M = 128, N = 256, K = 32
 *   ns_out     device uint64 [SM count] (the first *units_out entries written)
 *   units_out  host int: CTA pairs (kind 0, 1) or CTAs (kind 2) launched
 * Rate = units * 4 * iters * 2 M N K / max(ns_out).
 */
int bitlinear_tensor_peak(int kind, int iters, uint64_t* ns_out, int* units_out, int* dev_status,
                          bitlinear_stream_t stream);

/* Synchronise the stream and read *dev_status: BITLINEAR_OK,
 * BITLINEAR_ERR_TIMEOUT if a kernel gave up a bounded wait,
 * BITLINEAR_ERR_INDEX if one met an index outside its tensors, or
 * BITLINEAR_ERR_NO_PAGES. */
int bitlinear_check_status(const int* dev_status, bitlinear_stream_t stream);

/*
 * Launch overlap (programmatic dependent launch), process-wide, default off.
 * When enabled, later launches may start while the previous kernel in the
 * same stream is still running: each kernel first does the work that needs
 * only the weights (Wp, gamma: loads into shared memory, barrier and tensor
 * memory set-up) and waits for that previous kernel to complete before it
 * reads activation codes, inputs or scales, or writes any output. Enable it
 * only when no call's Wp or gamma is written by the kernel just before it in
 * its stream. A CUDA graph keeps the setting in force when it was captured.
 */
int bitlinear_set_launch_overlap(int enable);

/* Limit (ns) on every in-kernel wait of later launches; default 2e9. */
int bitlinear_set_wait_timeout_ns(int64_t ns);

/* Launch one block that waits on an mbarrier nothing arrives on, bounded by
 * timeout_ns, then reports BITLINEAR_STATUS_TIMEOUT into dev_status: checks
 * the bounded-wait path without any real fault. */
int bitlinear_debug_wait_timeout(int* dev_status, int64_t timeout_ns, bitlinear_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* BITLINEAR_H */
