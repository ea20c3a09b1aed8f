// qpack_launch.h — host-side interface between the C ABI (qpack_api.cu) and the kernel translation units.
// Argument validation happens in the C ABI layer; these launchers assume valid arguments.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "qpack.h"

namespace qpack {

// Arguments of the per-256-weight-block kernels (quantize / pack / unpack / dequant). Unused pointers are null.
struct BlockArgs {
    const void *W;            // quantize input [N, K] (f32 / f16 / bf16)
    int64_t N, K;
    int64_t nbk;              // 256-weight blocks per row (ceil(K / 256))
    int64_t row_stride;       // packed bytes per row
    int64_t scale_stride;     // Q4G32 packed scale floats per row
    int8_t *codes;            // [N, K] signed codes (written by quantize/unpack, read by pack)
    float *gscale;            // Q4G32 [N, K/32]
    uint8_t *sub_scale;       // [N, nbk * nsub]
    uint8_t *sub_min;         // [N, nbk * nsub] (asymmetric formats)
    uint16_t *d;              // [N, nbk]
    uint16_t *dmin;           // [N, nbk] (asymmetric formats)
    uint8_t *packed;          // packed output
    float *gs_out;            // Q4G32 packed scale output [N, scale_stride]
    const uint8_t *packed_in; // packed input (unpack / dequant)
    const float *gs_in;       // Q4G32 packed scale input
    float *out;               // dequant output [N, K]
    int32_t *status;          // RANGE flag word (quantize modes), may be null
};

// mode: 0 quantize->parts, 1 quantize->packed, 2 parts->packed, 3 packed->parts, 4 packed->fp32
cudaError_t launch_block_op(int fmt, int mode, int wdt, const BlockArgs &a, cudaStream_t s);

// Arguments of the streaming products (qgemv / qgemm_small).
struct GemvArgs {
    const uint8_t *packed;
    const float *gscale;      // Q4G32 packed scales, else null
    int64_t N, K;
    int64_t row_stride;       // bytes
    int64_t scale_stride;     // floats (Q4G32)
    const uint16_t *X;        // [M, ldx] fp16
    int64_t ldx;
    float *Y;                 // [M, ldy] fp32
    int64_t ldy;
    int M;
    int weight_prefetch;      // 1: launched as a programmatic dependent of the previous kernel and allowed to
                              //    stream packed weights before that kernel has finished (caller's opt-in)
    int64_t kc0;              // first K chunk of this launch: it covers columns [kc0 * chunk, kc0 * chunk + K) of
                              //    the packed rows (X already points at column kc0 * chunk)
    int accumulate;           // 1: add the products to Y (a later K split), 0: overwrite Y
};
cudaError_t launch_gemv(int fmt, const GemvArgs &a, cudaStream_t s);

// Arguments of the tensor-core prefill GEMM.
struct PrefillArgs {
    const uint8_t *packed;
    const float *gscale;
    int64_t N, K, M;
    int64_t row_stride;
    int64_t scale_stride;
    const uint16_t *X;        // bf16 [M, ldx]
    int64_t ldx;
    uint16_t *Y;              // bf16 [M, ldy]
    int64_t ldy;
    int vec_y;                // 1 when Y rows allow 16-byte stores (Y 16-byte aligned, ldy % 8 == 0)
};
cudaError_t launch_prefill(int fmt, const PrefillArgs &a, cudaStream_t s);

// Per-translation-unit device fault words (bounded waits that gave up). Read and cleared synchronously.
// 8-bit KV cache (qpack_kv.cu); n a positive multiple of 32, pointers checked by the caller.
cudaError_t launch_kv_quantize(const uint16_t *v, int64_t n, int8_t *q, uint16_t *scales, cudaStream_t s);
cudaError_t launch_kv_dequant(const int8_t *q, const uint16_t *scales, int64_t n, uint16_t *out, cudaStream_t s);
// Addresses of the translation units' fault words on the current device.
cudaError_t fault_word_gemv(int **word);
cudaError_t fault_word_prefill(int **word);

// Paged KV cache (qpack_paged.cu, qpack_attend.cu). The pool and the tables as the C ABI has them, checked.
struct AppendArgs {
    qpack_kv_pool_t pool;
    qpack_kv_tables_t t;
    const int32_t *seqs, *pos;   // null: token i of sequence i / its last token
    int64_t n;
    void *k, *v;                 // read by append, written by read (either may then be null)
    int64_t ldk, ldv;
    const float *rope;           // null: no rotation
    int64_t rope_rows;
    int layer, dt;
};
cudaError_t launch_kv_append(const AppendArgs &a, cudaStream_t s);
cudaError_t launch_kv_read(const AppendArgs &a, cudaStream_t s);

struct AttendArgs {
    qpack_kv_pool_t pool;
    qpack_kv_tables_t t;
    const int32_t *seqs;
    const void *q;
    int64_t ldq;
    const float *rope;
    int64_t rope_rows;
    void *out;
    int64_t ldo;
    float *lse;
    void *ws;
    int64_t window;
    float scale;
    int layer, B, q_heads, qdt, odt;
};
cudaError_t launch_kv_attend(const AttendArgs &a, cudaStream_t s);
int64_t kv_attend_workspace(const qpack_kv_pool_t &pool, int q_heads);

cudaError_t launch_kv_reserve(const qpack_kv_pool_t &p, const qpack_kv_tables_t &t, const int32_t *seqs,
                              const int32_t *add, int n, cudaStream_t s);
cudaError_t launch_kv_fork(const qpack_kv_pool_t &p, const qpack_kv_tables_t &t, const int32_t *src, const int32_t *dst,
                           int n, void *ws, cudaStream_t s);
cudaError_t launch_kv_free(const qpack_kv_tables_t &t, const int32_t *seqs, int n, cudaStream_t s);
cudaError_t launch_kv_compact(const qpack_kv_pool_t &p, const qpack_kv_tables_t &t, int32_t *tables_out,
                              int32_t *refs_out, int32_t *moved, void *ws, cudaStream_t s);
cudaError_t launch_kv_copy_pages(const qpack_kv_pool_t &p, const int32_t *src, const int32_t *dst, int64_t n,
                                 cudaStream_t s);
int64_t kv_page_workspace(const qpack_kv_pool_t &p);
cudaError_t fault_word_paged(int **word);
cudaError_t fault_words_attend(int **words);    // one a cache type
cudaError_t fetch_faults(int32_t *flags);

int num_sms();
int weight_prefetch_enabled();   // per-device option QPACK_OPT_WEIGHT_PREFETCH
int prefill_tile_rows();         // per-device option QPACK_OPT_PREFILL_TILE_ROWS (0: chosen per launch)

}  // namespace qpack
