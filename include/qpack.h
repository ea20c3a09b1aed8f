/*
 * qpack.h — C ABI of libqpack: group-quantized low-bit weights with dequantization fused into the
 * decode-phase matrix-vector product (and the small-batch and prefill matrix products), for one NVIDIA
 * GB300 (sm_103a).
 *
 * Sources. P1 = the 2/3/5/6-bit quantization article (lpnh.cn/news/2857666); P2 = the DBHOO-CIM INT4 CPU
 * inference article (pwwt.cn/news/4452170). Where the pages leave a bit order open, fields are little-endian
 * with weight i at the lowest free bit.
 *
 * Conventions shared by every entry point:
 *  - W is row-major [N, K]: N output features (rows), K input features. Groups and super-blocks run along K.
 *  - All data pointers are DEVICE pointers owned by the caller; the library never allocates device memory
 *    and never frees caller memory. Calls are asynchronous on `stream` (NULL = the legacy default stream).
 *  - fp16 and bf16 data are passed as their 16-bit patterns (uint16_t).
 *  - Argument errors are detected on the host before anything is launched and returned as a negative
 *    qpack_status; a failed launch returns QPACK_ERR_CUDA. Data-dependent conditions are reported through a
 *    device status word (qpack_quantize*) and never trap.
 *  - N == 0 (or M == 0) is accepted and launches nothing.
 */
#ifndef QPACK_H_
#define QPACK_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *qpack_stream_t; /* identical to cudaStream_t */

/* Weight formats. Q4G32: INT4 symmetric, group 32, fp32 group scales (P2 §3.1–§3.2, §4.1).
 * Q2S/Q3S/Q5S/Q6S: 256-weight super-blocks of 84/110/176/210 bytes (P1 §2.3 byte table).
 * Q4G32H: the INT4 codes of Q4G32 with fp16 group scales, used rounded (4.5 bpw, P1 §2.1).
 * Q4G16: the INT4 rule of Q4G32 with groups of 16 weights, fp32 scales (6 bpw, P2 §5.1); K a
 * multiple of 32.
 * Q4G32A: INT4 asymmetric, group 32 (P2 §5.1; P1 §2.1's zero-point form w' = s*(q - z)): unsigned codes 0..15,
 * one fp32 pair (s, z) per group with z an integer value 0..15 (6 bpw): lo = min(0, min w), hi = max(0, max w),
 * s = max((hi - lo) / 15, 1e-12), z = clamp(rint(-lo / s), 0, 15), q = clamp(rint(w / s) + z, 0, 15). */
typedef enum {
    QPACK_Q4G32 = 0,
    QPACK_Q2S = 1,
    QPACK_Q3S = 2,
    QPACK_Q5S = 3,
    QPACK_Q6S = 4,
    QPACK_Q4G32H = 5,
    QPACK_Q4G16 = 6,
    QPACK_Q4G32A = 7
} qpack_format;

typedef enum { QPACK_F32 = 0, QPACK_F16 = 1, QPACK_BF16 = 2 } qpack_dtype;

typedef enum {
    QPACK_OK = 0,
    QPACK_ERR_ARG = -1,        /* null pointer where one is required, bad enum, negative size */
    QPACK_ERR_SHAPE = -2,      /* K not a multiple of the format's group (32) or super-block (256), M out of range */
    QPACK_ERR_ALIGN = -3,      /* a pointer or leading dimension breaks the stated alignment */
    QPACK_ERR_RANGE = -4,      /* reserved: data-dependent range failure reported synchronously */
    QPACK_ERR_CUDA = -5,       /* a CUDA runtime call or kernel launch failed */
    QPACK_ERR_UNSUPPORTED = -6 /* format / path combination not provided */
} qpack_status;

/* Bit OR-ed into the device status word when a super-block's fp16 d or dmin, or a Q4G32H fp16 group scale,
 * overflows to infinity (P1 §2.3 warns about fp16 super-scale overflow). */
#define QPACK_FLAG_RANGE 1

/* Sizes of the packed representation (host-only, no GPU work).
 *  row_stride    bytes between consecutive packed rows (super-block formats: rows padded to 16 B, P1 §3.3)
 *  packed_bytes  N * row_stride
 *  scale_stride  INT4 formats: elements between consecutive rows of the separate group-scale array (fp32 for
 *                Q4G32 / Q4G16 / Q4G32A, fp16 for Q4G32H; K/32 (K/16 for Q4G16 and for Q4G32A's (s, z) pairs)
 *                rounded up so that rows are 16 bytes, P2 §4.1); 0 otherwise
 *  scale_bytes   INT4 formats: N * scale_stride * (4 or 2); 0 otherwise
 *  block_bytes   bytes per 256-weight super-block (84/110/176/210, P1 §2.3); 0 for the INT4 formats
 *  nsub          sub-blocks per super-block (16, or 8 for Q5S); for the INT4 formats the groups per row
 *  weight_bytes  packed_bytes + scale_bytes: the bytes one product call streams from memory
 * Returns QPACK_OK, QPACK_ERR_ARG (bad format, negative size, null out) or QPACK_ERR_SHAPE. */
typedef struct {
    int64_t row_stride;
    int64_t packed_bytes;
    int64_t scale_stride;
    int64_t scale_bytes;
    int64_t block_bytes;
    int64_t nsub;
    int64_t weight_bytes;
} qpack_layout_t;
int qpack_layout(int fmt, int64_t N, int64_t K, qpack_layout_t *out);

/* Quantize W into unpacked parts (P2 §3.1 for Q4G32; two-level round-to-nearest for the super-block formats,
 * following P1 §2.1's fp16 super-scale -> sub-block scale -> weight structure: each sub-block's own scale, fp16 d
 * (and dmin) used rounded, integer sub-block scales against it, codes against the rounded sub-block scale).
 *  W          [N, K] of dtype wdt (F32, F16 or BF16), 16-byte aligned
 *  codes      [N, K] int8: the integer q (Q4G32/Q4G32H/Q4G16 -8..7, Q4G32A 0..15, Q3S -4..3, Q6S -32..31,
 *             Q2S 0..3, Q5S 0..31)
 *  gscale     Q4G32: [N, K/32], Q4G16: [N, K/16] fp32 group scales; Q4G32A: [N, K/16] fp32, the pair (s, z) of
 *             group g at 2g, 2g + 1; NULL for other formats
 *  sub_scale  super-block formats: [N, K/256 * nsub] uint8 sub-block scale integers L_j; NULL for the INT4 formats
 *  sub_min    Q2S/Q5S: [N, K/256 * nsub] uint8 sub-block minimum integers M_j; NULL otherwise
 *  d, dmin    super-block formats: [N, K/256] fp16 bits of d; dmin for Q2S/Q5S only (NULL otherwise).
 *             Q4G32H: d holds the [N, K/32] fp16 group scales (2-byte aligned), dmin NULL
 *  status     device int32 (may be NULL): QPACK_FLAG_RANGE is OR-ed in; the caller clears it.
 * The results are bit-identical to the IEEE fp32 definition (round to nearest even, true division, no FMA). */
int qpack_quantize(int fmt, const void *W, int wdt, int64_t N, int64_t K, int8_t *codes, float *gscale,
                   uint8_t *sub_scale, uint8_t *sub_min, uint16_t *d, uint16_t *dmin, int32_t *status,
                   qpack_stream_t stream);

/* Pack unpacked parts (layouts as produced by qpack_quantize) into the format's bytes: P2 §3.2 nibble
 * packing (low nibble = even index) for Q4G32; P1 §2.2 cross-byte packing and §2.3 bit planes for the
 * super-block formats (little-endian fields, weight i at the lowest free bit).
 *  packed        [N, row_stride] bytes, 16-byte aligned; padding bytes are written as zero
 *  group_scales  Q4G32, Q4G16, Q4G32A: [N, scale_stride] fp32, Q4G32H: [N, scale_stride] fp16; 16-byte aligned,
 *                padding written as zero; NULL for the super-block formats. Q4G32A pairs are copied bit for bit;
 *                the products and qpack_dequant read z as an integer 0..15 */
int qpack_pack(int fmt, int64_t N, int64_t K, const int8_t *codes, const float *gscale, const uint8_t *sub_scale,
               const uint8_t *sub_min, const uint16_t *d, const uint16_t *dmin, uint8_t *packed,
               void *group_scales, qpack_stream_t stream);

/* Fused quantize + pack: W straight to packed bytes (and INT4 group scales) in one pass over W.
 * Arguments as qpack_quantize (W, wdt, status) and qpack_pack (packed, group_scales). */
int qpack_quantize_pack(int fmt, const void *W, int wdt, int64_t N, int64_t K, uint8_t *packed,
                        void *group_scales, int32_t *status, qpack_stream_t stream);

/* Inverse of qpack_pack: packed bytes back to unpacked parts (same pointer conventions). */
int qpack_unpack(int fmt, int64_t N, int64_t K, const uint8_t *packed, const void *group_scales, int8_t *codes,
                 float *gscale, uint8_t *sub_scale, uint8_t *sub_min, uint16_t *d, uint16_t *dmin,
                 qpack_stream_t stream);

/* Dequantize a packed matrix to fp32 out [N, K] (the page's self-check path, P1 §3.4): Q4G32 w' = s*q,
 * Q4G32H w' = fp32(s16)*q; Q4G32A w' = s*(q - z);
 * symmetric super-blocks w' = (d*L_j)*q; asymmetric w' = (d*L_j)*q - (dmin*M_j), each step an fp32 rounding,
 * no FMA. out must be 16-byte aligned. */
int qpack_dequant(int fmt, int64_t N, int64_t K, const uint8_t *packed, const void *group_scales, float *out,
                  qpack_stream_t stream);

/* Fused dequant-GEMV (decode, batch 1; P1 §1.2 and §3.3, P2 §3.3 "fused dequantization"):
 *   y[r] = sum_k w'[r,k] * x[k],  r < N
 * packed weights are read exactly once and unpacked in registers. x is rounded once to 16-bit integers per
 * 16-element half of each 32-element unit: step sigma = m / 32767 (m = the half's largest |x|), so every staged
 * value is within m / 65000 of x and the half's largest element is exact to 2.4e-7 relative; code x activation sums
 * are exact int32 within a half, fp32 across halves. Worst case over all finite fp16 x, the staging moves y[r] by at
 * most sqrt(15) / 65000 * ||w'_r||_2 * ||x||_2 = 6.0e-5 * ||w'_r||_2 * ||x||_2.
 *  packed, group_scales  as produced by qpack_pack (group_scales NULL except the INT4 formats), 16-byte aligned
 *  x                     [K] fp16, 16-byte aligned
 *  y                     [N] fp32, 4-byte aligned
 *  K                     any multiple of the format's group (rows longer than one SM's shared memory can stage go
 *                        in K splits whose products are added to y in split order)
 * Parity bound against an fp64 sum: |y[r] - y_ref[r]| <= 1e-4 * ||w'_r||_2 * ||x||_2 for every finite x.
 * Non-finite activations: if x holds an inf or a nan, every y[r] is nan and QPACK_FAULT_NONFINITE_X is set in the
 * fault word (qpack_fetch_fault_flags); the IEEE sum would be nan or +-inf, and the call refuses to pick one. */
int qgemv(int fmt, const uint8_t *packed, const void *group_scales, int64_t N, int64_t K, const uint16_t *x,
          float *y, qpack_stream_t stream);

/* Small-batch decode GEMM (P2 §5.2 decode vs prefill; batch up to 16):
 *   Y[m, r] = sum_k w'[r,k] * X[m,k],  m < M, r < N,  1 <= M <= 16
 * each packed weight is read once and reused across the M activation rows; activations and sums as in qgemv
 * (a non-finite activation makes every output of its row nan and sets QPACK_FAULT_NONFINITE_X).
 *  X  [M, ldx] fp16, 16-byte aligned, ldx >= K and ldx a multiple of 8
 *  Y  [M, ldy] fp32, ldy >= N
 * Same parity bound as qgemv, per element. */
int qgemm_small(int fmt, const uint8_t *packed, const void *group_scales, int64_t N, int64_t K, int M,
                const uint16_t *X, int64_t ldx, float *Y, int64_t ldy, qpack_stream_t stream);

/* Prefill dequant GEMM on the tensor cores (P1 §1.2: prefill is a dense [tokens, hidden] x [hidden, hidden]
 * contraction):
 *   Y[m, n] = sum_k bf16(X[m,k]) * bf16(w'[n,k]),  fp32 accumulation, Y rounded to bf16
 * Weight tiles are dequantized to bf16 in shared memory and fed to tcgen05 MMA with TMEM accumulators; by
 * default two CTAs on two SMs share each MMA (see QPACK_OPT_PREFILL_TILE_ROWS).
 *  formats  the INT4 formats (K a multiple of 64) and the super-block formats (K a multiple of 256)
 *  X        [M, ldx] bf16, 16-byte aligned, ldx >= K, ldx a multiple of 8
 *  Y        [M, ldy] bf16, 2-byte aligned, ldy >= N (16-byte aligned rows with ldy % 8 == 0 store fastest)
 * Parity bound: ||Y - Y_ref||_2 / ||Y_ref||_2 <= 2e-2 with Y_ref in fp64.
 * No workspace argument: accumulators live in TMEM and tiles in shared memory, and Y is written directly. */
int qgemm_prefill(int fmt, const uint8_t *packed, const void *group_scales, int64_t N, int64_t K, int64_t M,
                  const uint16_t *X, int64_t ldx, uint16_t *Y, int64_t ldy, qpack_stream_t stream);

/* 8-bit KV cache (2/3/5/6-bit article §4.1: the KV cache in 8 bits with one fp16 scale per 32 elements, about
 * 1.06 bytes per element instead of 2). Groups are 32 consecutive elements of the flat array.
 *   d = fp16_rn(max|v| / 127) (fp32 division; the rounded d is the one used), q = clamp(rint(v / d), -127, 127),
 *   q = 0 when d == 0.
 *  v       [n] fp16 keys or values, 16-byte aligned; finite (non-finite inputs give unspecified codes, no fault)
 *  codes   [n] int8 out, 8-byte aligned
 *  scales  [n / 32] fp16 out, 2-byte aligned
 *  n       a multiple of 32 (QPACK_ERR_SHAPE otherwise); 0 launches nothing
 * Codes and scales are bit-identical to the oracle's. The caller owns every buffer. */
int qpack_kv_quantize(const uint16_t *v, int64_t n, int8_t *codes, uint16_t *scales, qpack_stream_t stream);

/* Inverse of qpack_kv_quantize (the Mix-Quant article §2.3: the int8 cache dequantized to fp16 in bulk):
 *   out[i] = fp16_rn(d_g * q_i), g = i / 32 (the product is exact in fp32).
 *  codes 8-byte aligned, scales 2-byte aligned, out [n] fp16 16-byte aligned; n a multiple of 32. */
int qpack_kv_dequant(const int8_t *codes, const uint16_t *scales, int64_t n, uint16_t *out, qpack_stream_t stream);

/* ---------------------------------------------------------------------------------------------------------------
 * Paged KV cache: the cache of many sequences in pages, the operators that write, read and attend to it, and the page
 * operators that share, release, extend and compact it.
 *
 * A pool holds `layers` x `pages` pages of `page_tokens` tokens: per layer and page, keys and values
 * [heads][page_tokens][dim] without gaps, in 8 bits (QPACK_KV_I8: int8 codes and one fp16 scale per 32 elements, the
 * rule of qpack_kv_quantize; scales [heads][page_tokens][dim / 32]) or in 16 bits (fp16, bf16; scales NULL). Element
 * (layer, page, head, slot, i) of k and v is at layer * layer_stride + page * page_stride
 * + (head * page_tokens + slot) * dim + i, its scale at layer * scale_layer_stride + page * scale_page_stride
 * + (head * page_tokens + slot) * (dim / 32) + i / 32 (offsets are 64-bit). An 8-bit element stands for
 * v' = fp16_rn(scale * code), as qpack_kv_dequant gives it.
 *  heads        key/value heads;  dim  64, 128 or 256;  page_tokens  a power of two, 1 to 1024
 *  k, v         16-byte aligned, layer_stride and page_stride multiples of 16 elements
 *  k_scales, v_scales  16-byte aligned, their strides multiples of dim / 32 elements
 *
 * Sequences are rows of a page table on the device: token t of sequence s is in page
 * tables[s * stride + t / page_tokens], slot t % page_tokens. lens[s] counts its tokens, refs[p] the sequences that
 * hold page p (0: free). Entries that hold no page are -1. Append, read and attend need no refs (may be NULL).
 *
 * Device data that is out of range (a page number outside the pool, a position outside the table, a length longer than
 * the table or negative, a sequence number outside the table) never reaches memory outside the buffers: the access is
 * left out and QPACK_FAULT_PAGE is set in the fault word (qpack_fetch_fault_flags). */
typedef enum { QPACK_KV_I8 = 0, QPACK_KV_F16 = 1, QPACK_KV_BF16 = 2 } qpack_kv_type;

typedef struct {
    void *k, *v;
    uint16_t *k_scales, *v_scales;
    int64_t layer_stride, page_stride;
    int64_t scale_layer_stride, scale_page_stride;
    int64_t pages;          /* 1 to 2^31 - 1 */
    int32_t layers, heads, page_tokens, dim;
    int32_t type;           /* qpack_kv_type */
    int32_t reserved;       /* 0 */
} qpack_kv_pool_t;

typedef struct {
    int32_t *tables;        /* [seqs, stride], the first max_pages entries of each row used */
    int32_t *lens;          /* [seqs] */
    int32_t *refs;          /* [pages], or NULL where the call does not use it */
    int64_t stride;
    int64_t pages;          /* entries of refs */
    int32_t seqs, max_pages;
} qpack_kv_tables_t;

#define QPACK_FAULT_PAGE 32     /* device data out of range: a page, position, length or sequence number */
#define QPACK_FAULT_NO_PAGES 64 /* a request of qpack_kv_reserve / qpack_kv_fork was refused: no free page, or its
                                   row of the table is full (fork: the child is not empty) */

/* Append n tokens to a layer of the cache: token i goes to position pos[i] of sequence seqs[i].
 *  k, v       [n, ld] rows of heads * dim elements of dtype dt (QPACK_F32, F16 or BF16; a product's fp32 output goes in
 *             as it is), 16-byte aligned, ldk and ldv >= heads * dim and multiples of 8
 *  seqs       [n] int32, or NULL: token i belongs to sequence i
 *  pos        [n] int32, or NULL: the sequence's last token, lens[seq] - 1. A negative position skips the token.
 *             lens is not changed (qpack_kv_reserve extends a sequence). No two tokens may name the same place.
 *  rope       NULL, or [rope_rows, dim] fp32, 16-byte aligned: row p holds cos (dim / 2) and sin (dim / 2) of position
 *             p, and keys are rotated before they are stored: (x_i, x_{i + dim/2}) ->
 *             (x_i c_i - x_{i + dim/2} s_i, x_{i + dim/2} c_i + x_i s_i), every operation rounded to fp32. Keys of
 *             positions behind the table are stored as they are, and QPACK_FAULT_PAGE is set.
 * 8-bit pools: per 32 elements d = fp16_rn(max|x| / 127) (at most 65504), q = clamp(rint(x / d), -127, 127), 0 where d
 * is 0, in fp32 with IEEE division; 16-bit pools: rounded to nearest even. Non-finite inputs give unspecified codes. */
int qpack_kv_append(const qpack_kv_pool_t *pool, int layer, const qpack_kv_tables_t *t, const int32_t *seqs,
                    const int32_t *pos, int64_t n, const void *k, const void *v, int dt, int64_t ldk, int64_t ldv,
                    const float *rope, int64_t rope_rows, qpack_stream_t stream);

/* The inverse: rows of the cache, token i from position pos[i] of sequence seqs[i] (NULL as above), as dt (QPACK_F32,
 * F16 or BF16) into k, v [n, ld] (16-byte aligned, ld >= heads * dim and a multiple of 8). Either of k and v may be
 * NULL. Tokens with a negative position, or out of range, are written as zero. */
int qpack_kv_read(const qpack_kv_pool_t *pool, int layer, const qpack_kv_tables_t *t, const int32_t *seqs,
                  const int32_t *pos, int64_t n, void *k, void *v, int dt, int64_t ldk, int64_t ldv,
                  qpack_stream_t stream);

/* Attention of one new token a sequence over its cache (grouped queries: query heads h * q_heads / heads ... share
 * key/value head h). Row b takes sequence s = seqs[b] (NULL: b), L = lens[s] and, with window > 0, its last `window`
 * tokens only (0: all): lo = max(0, L - window).
 *   x_t = scale * <q~_b, k'_t>, lo <= t < L
 *   out_b = sum_t e^{x_t - m} v'_t / sum_t e^{x_t - m},  lse_b = ln sum_t e^{x_t}
 * Sums, softmax statistics and accumulators are fp32; queries and probabilities enter the tensor cores as two 16-bit
 * terms each (22 bits) where the pool is 8-bit or fp16; where it is bf16, queries as three (24), probabilities as three where
 * the output is fp32, else as two (16). An empty range gives out = 0 and lse = -inf.
 * The formula is for finite keys and values (a value above 65504 in an fp16 pool, or a scale times a code, is infinite).
 * A key that is not may make the heads of its key/value head NaN in its row, even where the formula gives it no weight; a
 * value that is not makes its element of their outputs infinite or NaN. Nothing else changes. Slots that hold no token
 * of the range may hold anything. A query that is not finite makes its own head NaN.
 *  q     [B, ldq] of dtype qdt, q_heads * dim elements a row, 16-byte aligned, ldq a multiple of 8; q_heads a multiple
 *        of the pool's heads, at most 65536
 *  rope  as in qpack_kv_append, applied to q at position L - 1 (NULL: q as it is)
 *  out   [B, ldo] of dtype odt, 16-byte aligned, ldo >= q_heads * dim and a multiple of 8
 *  lse   [B, q_heads] fp32, or NULL
 *  ws    workspace of at least the bytes that qpack_kv_attend_workspace gives on this device, 16-byte aligned, its
 *        first QPACK_KV_ATTEND_ZEROED bytes zeroed once before its first use. Each call leaves it ready for the next, of
 *        any shape that it is large enough for; calls that may run at the same time need a workspace each.
 *  B     at most 4096. Results do not depend on the order in which blocks run.
 * QPACK_ERR_UNSUPPORTED: one row of the table could hold more than 2^31 tiles over all heads. */
#define QPACK_KV_ATTEND_ZEROED (1 << 20)
int qpack_kv_attend(const qpack_kv_pool_t *pool, int layer, const qpack_kv_tables_t *t, const int32_t *seqs, int B,
                    const void *q, int qdt, int64_t ldq, int q_heads, float scale, int64_t window, const float *rope,
                    int64_t rope_rows, void *out, int odt, int64_t ldo, float *lse, void *ws, int64_t ws_bytes,
                    qpack_stream_t stream);
int qpack_kv_attend_workspace(const qpack_kv_pool_t *pool, int B, int q_heads, int64_t *bytes);

/* Attention of one new token a row, as qpack_kv_attend without a window, for batches in which groups of rows share a prefix
 * (samples forked from one prompt): a prefix is read once a group.
 * Rows first[g] .. first[g + 1] - 1 are group g; they share the first prefix[g] tokens, which are read from the pages of the
 * group's first row. Of a row's sequence (seqs as above, L = lens) the tokens t < min(L, prefix[g]) are those, and the tokens
 * prefix[g] <= t < L are its own. Rows of no group have no prefix. With sequences that share their prefixes by
 * qpack_kv_fork (full pages are the same, a last page that is not full is a copy) the result is qpack_kv_attend's but for
 * the terms below and the order of sums.
 * It pays where many rows share many tokens (us in a graph, qpack_kv_attend / this call, 8 bits, 32 query heads over 8 of 128,
 * rows of one group, prefix: 64 rows 300 tokens 19 / 29, 1000 31 / 30, 10000 200 / 54; 16 rows 1000 13 / 22, 3000 24 / 24, 10000
 * 57 / 37; 8 rows 10000 33 / 35, 60000 151 / 81; up to 4 rows never by much): rows times prefix above some 50000 tokens in that
 * shape, rows 8 or more. Below, a call costs its three launches, some 20 us, where qpack_kv_attend takes 6 to 20. fp16 queries
 * (qpack_qk_norm_rope's output, say) without rope halve the product with the keys against fp32 ones, and let long prefixes be taken
 * by 256 queries at a time instead of 128 (32 rows of 10000: 43 us against 46).
 *  first   [groups + 1] int32, rising from 0 or more to at most B (equal neighbours: a group without rows); anything else sets
 *          QPACK_FAULT_PAGE, and all rows go without a prefix. May be NULL where groups is 0.
 *  prefix  [groups] int32, 0 to the length of the group's first row; others are cut to that and set QPACK_FAULT_PAGE
 *  groups  at most 512
 * Scores, maxima, sums and accumulators are fp32. Over the prefix, queries and probabilities enter the tensor cores as two 16-bit
 * terms each (22 bits where the pool is 8-bit or fp16, 16 where it is bf16; a query is one term where that holds it whole: fp16,
 * or bf16 over a bf16 pool, without rope). Own tokens are attended to as by qpack_kv_attend.
 * A prefix's key that is not finite may make the heads of its group that see it NaN, a value that is not makes its own element
 * infinite or NaN (NaN, perhaps, in rows that end before it too); everything else keeps its bits. A query that is not finite
 * makes its own head NaN.
 * The other arguments, limits and errors are qpack_kv_attend's; QPACK_ERR_UNSUPPORTED also where a row of the table could hold
 * more than 2^31 - 256 tokens, or its tiles of 64 tokens for all queries in blocks of 128 (one more a group) come to 2^30.
 *  ws      at least qpack_kv_shared_workspace bytes for this B or more, 16-byte aligned, the first QPACK_KV_ATTEND_ZEROED of
 *          them zeroed once; as qpack_kv_attend's otherwise, and good for its calls too. */
int qpack_kv_attend_shared(const qpack_kv_pool_t *pool, int layer, const qpack_kv_tables_t *t, const int32_t *seqs, int B,
                           const int32_t *first, const int32_t *prefix, int groups, const void *q, int qdt, int64_t ldq,
                           int q_heads, float scale, const float *rope, int64_t rope_rows, void *out, int odt, int64_t ldo,
                           float *lse, void *ws, int64_t ws_bytes, qpack_stream_t stream);
int qpack_kv_shared_workspace(const qpack_kv_pool_t *pool, int B, int q_heads, int64_t *bytes);

/* Page operators. All work on the device alone and are deterministic: new pages are the lowest-numbered free ones, in
 * the order of the requests. n <= 4096 sequences a call, each listed once.
 *
 * reserve: extend sequence seqs[i] by add[i] >= 0 tokens. Request i needs the pages between its old and new length, and
 * is granted (pages entered in the table, refs 1, lens raised) when the pages that it and all requests before it need
 * are free and its row holds them; otherwise it is left as it was and QPACK_FAULT_NO_PAGES is set. A negative seqs[i]
 * is skipped. */
int qpack_kv_reserve(const qpack_kv_pool_t *pool, const qpack_kv_tables_t *t, const int32_t *seqs, const int32_t *add,
                     int64_t n, qpack_stream_t stream);

/* fork: make the empty sequence dst[i] a copy of src[i] (one src may be forked many times; no dst may be a src). Full
 * pages are shared (refs + 1); a last page that is not full is copied into a fresh page, over all layers, the filled
 * tokens only. Refused as in reserve, and where dst[i] is not empty; the page that a refused request of a known sequence would
 * have got is passed over. ws: qpack_kv_page_workspace bytes, 16-byte aligned, no initial value needed. */
int qpack_kv_fork(const qpack_kv_pool_t *pool, const qpack_kv_tables_t *t, const int32_t *src, const int32_t *dst,
                  int64_t n, void *ws, int64_t ws_bytes, qpack_stream_t stream);

/* free: take one reference from every page of sequence seqs[i], clear its row (-1) and its length. A negative seqs[i] is
 * skipped. */
int qpack_kv_free(const qpack_kv_tables_t *t, const int32_t *seqs, int64_t n, qpack_stream_t stream);

/* compact: move live pages (refs > 0) so that they are the lowest-numbered ones. With n live pages, the i-th live page
 * numbered n or more moves to the i-th free page below n, over all layers; every table entry and reference count
 * follows. The results go to tables_out (rows of `stride`) and refs_out, which may be t->tables and t->refs.
 *  moved  device int32, or NULL: the number of pages moved */
int qpack_kv_compact(const qpack_kv_pool_t *pool, const qpack_kv_tables_t *t, int32_t *tables_out, int32_t *refs_out,
                     int32_t *moved, void *ws, int64_t ws_bytes, qpack_stream_t stream);

/* Copy the contents of page src[i] to page dst[i] over all layers, n pages (device int32 arrays). No dst may be listed
 * twice or be a src. */
int qpack_kv_copy_pages(const qpack_kv_pool_t *pool, const int32_t *src, const int32_t *dst, int64_t n,
                        qpack_stream_t stream);
int qpack_kv_page_workspace(const qpack_kv_pool_t *pool, const qpack_kv_tables_t *t, int64_t *bytes);

/* ---------------------------------------------------------------------------------------------------------------
 * What a decode step does to query and key heads between their product and the cache: the root-mean-square norm of each
 * head and the position rotation, in one pass over queries and keys.
 *   y = x / sqrt(mean(x^2) + eps) * weight      (weight NULL: y = x)
 *   (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s)  for the pairs of the first rope_dim elements, the rest stays y
 * in fp32, products and sums rounded each by itself (without a weight rotated keys are those that qpack_kv_append would
 * store), the result rounded once to odt. Heads that are rotated here go to qpack_kv_append and the attention calls without
 * their `rope`.
 *  q, k        either may be NULL, or have 0 heads
 *    x, out    [n, ldx] and [n, ldo]: rows of heads * dim elements of dtype dt and odt (QPACK_F32, F16 or BF16), 16-byte
 *              aligned, ldx and ldo >= heads * dim and multiples of 8. out may be x where dt is odt and ldx is ldo; otherwise
 *              the outputs overlap nothing.
 *    weight    [dim] fp32, 16-byte aligned, or NULL
 *  dim         elements of a head, a multiple of 8, 8 to 256
 *  eps         >= 0, finite (used with a weight only; a head of zeros with an eps of 0 is NaN). The mean of squares may lie outside
 *              fp32's range: a head for which it does is scaled by a power of two for it.
 *  rope        NULL (no rotation), or [rope_rows, rope_dim] fp32, 16-byte aligned: row p holds cos (rope_dim / 2) and sin
 *              (rope_dim / 2) of position p (whatever scaling a long context asks for is in the table)
 *  rope_dim    a multiple of 8, at most dim (0 without rope)
 *  interleaved 0: pairs (i, i + rope_dim / 2); 1: pairs (2i, 2i + 1)
 *  t, seqs, pos  token i's position: pos[i] (int32), or where pos is NULL the last one of sequence seqs[i] (NULL: i) of t,
 *              lens - 1. t and pos may both be NULL where rope is. A token whose position is negative is skipped: its
 *              rows of out are left as they were. A sequence or length out of range skips the token, and a position behind
 *              the table leaves its heads without rotation; both set QPACK_FAULT_PAGE. */
typedef struct {
    const void *x;
    void *out;
    const float *weight;
    int64_t ldx, ldo;
    int32_t heads;
    int32_t reserved;       /* 0 */
} qpack_heads_t;
int qpack_qk_norm_rope(const qpack_heads_t *q, const qpack_heads_t *k, int64_t n, int dim, int dt, int odt, float eps,
                       const float *rope, int64_t rope_rows, int rope_dim, int interleaved, const qpack_kv_tables_t *t,
                       const int32_t *seqs, const int32_t *pos, qpack_stream_t stream);

/* The next token of each row from its logits x_0 .. x_{V-1}, by a given random number. With m = max x and
 * w_i = e^{(x_i - m) / T}:
 *   order   tokens by falling logit, the lowest index first among equals
 *   top_k   k of them are kept (k <= 0, or as many as there are: all)
 *   top_p   of these, the shortest run from the top whose weights reach top_p of the sum of these (at least one; >= 1: all)
 *   min_p   of these, the ones with w_i >= min_p (<= 0: all; >= 1: those of the maximum)
 *   token   the lowest index whose sum of kept weights up to and including it passes u times their total
 * Weights and sums are exact to some 2^-43 of the largest weight, and do not depend on the order in which blocks run.
 * A logit of -inf masks its token: it is not counted and never drawn. A row without any other gives token -1 and
 * probability 0. A temperature below 2^-64 (0, negative or NaN too) gives the lowest index of the maximum and probability 1;
 * one above 2^64 counts as 2^64. A NaN among the filters' numbers switches the filter off. u outside [0, 1) counts as the
 * nearest number inside, NaN as 0. A logit of NaN or +inf gives token -1 and probability NaN for its row, and sets
 * QPACK_FAULT_NONFINITE_X.
 *  logits       [B, ld] of dtype dt (QPACK_F32, F16 or BF16), aligned to its elements, ld >= V; V at most 2^20
 *  temperature, top_k, top_p, min_p  [B] fp32 (top_k int32), or NULL: 1, and no filter
 *  u            [B] fp32
 *  tokens       [B] int32;  probs  [B] fp32, or NULL: the token's weight over the total of those kept
 * No output overlaps an input. */
int qpack_sample(const void *logits, int dt, int64_t ld, int64_t V, int64_t B, const float *temperature,
                 const int32_t *top_k, const float *top_p, const float *min_p, const float *u, int32_t *tokens,
                 float *probs, qpack_stream_t stream);

/* Human-readable name of a qpack_status value. Never NULL. */
const char *qpack_status_string(int status);

/* Device-side fault record: bounded waits inside the kernels that give up OR a bit into a per-device word
 * instead of hanging, and the decode products OR in QPACK_FAULT_NONFINITE_X when an activation was inf or nan.
 * Copies the current device's word to *flags (synchronous) and clears it.
 * Returns QPACK_OK or QPACK_ERR_CUDA. A non-zero *flags means some kernel result is invalid. */
#define QPACK_FAULT_NONFINITE_X 16
int qpack_fetch_fault_flags(int32_t *flags);

/* Per-device options (the device current at the call).
 *  QPACK_OPT_WEIGHT_PREFETCH (default 0): when 1, qgemv / qgemm_small launch as programmatic dependents of the
 *  previous kernel in the stream and start streaming their packed weights before that kernel has finished
 *  (activations are still read only after it has finished, and outputs written after). The caller guarantees
 *  that the packed weights and scales of a product are not written by the kernel launched just before it on
 *  that stream (true for a decode loop over resident weights).
 *  QPACK_OPT_PREFILL_TILE_ROWS (default 0): the qgemm_prefill tiling. 256 or 224: pairs of CTAs on two SMs (a
 *  cluster of two), each pair a 512-token x 256- or 224-weight-row block of Y computed by tcgen05 MMAs of M = 256
 *  tokens and N = 256 or 224 weight rows spread over the pair. 112 or 128: one CTA per 512-token x 112- or
 *  128-row block (MMAs of M = 128, N = 112 or 128). 0 (the default) takes the pairs for every format, of 224 rows
 *  where they fill more of the SMs at once (not for Q3S), else of 256. All of them meet the prefill bound.
 * Returns QPACK_OK, QPACK_ERR_ARG (unknown option or value) or QPACK_ERR_CUDA (no current device). Host-only. */
#define QPACK_OPT_WEIGHT_PREFETCH 1
#define QPACK_OPT_PREFILL_TILE_ROWS 2
int qpack_set_option(int option, int value);

/* Library version: major * 10000 + minor * 100 + patch. */
int qpack_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QPACK_H_ */
