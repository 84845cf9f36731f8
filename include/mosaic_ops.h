/*
 * mosaic_ops.h -- the operators of libmosaic around a quantized linear layer when a model
 * answers token by token: products of 16-bit activations with the packed NVFP4 weight,
 * head norms with the position rotation, a paged key/value cache in NVFP4, and attention
 * over it. The pages describe the linear layer alone; these have no counterpart there.
 *
 * The conventions of mosaic.h hold (device pointers, caller-owned buffers, asynchronous on
 * `stream`, host-side validation). Two are added:
 *  - 16-bit tensors are bf16 or fp16, one type per call (mq_dtype).
 *  - Index arrays live on the device, so the host cannot check what they hold. The kernels
 *    do: an index out of range is skipped as each call states, never followed, and
 *    MQ_ERR_INVALID_ARG is recorded in the device error word (mq_get_error reports it).
 */
#ifndef MOSAIC_OPS_H_
#define MOSAIC_OPS_H_

#include "mosaic.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MQ_BF16 = 0,
    MQ_F16 = 1
} mq_dtype;

/*
 * A [tokens][heads][D] tensor: element (t, h, d) at data + t * token_stride +
 * h * head_stride + d (strides in elements, >= 0; the D elements are adjacent). data and
 * both strides must be multiples of 16 bytes. Rows of an output must not overlap: one axis
 * lies inside a step of the other.
 */
typedef struct {
    void* data;
    int64_t heads;
    int64_t token_stride;
    int64_t head_stride;
} mq_heads;

/*
 * A paged cache of keys and values in NVFP4. page_size tokens a page (a multiple of 16), D
 * = 64 or 128. Token t of a page lies in record t / 16; a record holds 16 tokens of one
 * head, keys and values, in 18 D bytes:
 *   pages + ((page * heads + head) * (page_size / 16) + t / 16) * 18 D.
 * Inside a record (token i = t % 16, group q = d / 16, L = D / 64):
 *   [0, 8D)    key codes: token i's D/2 bytes at i * D/2 (element 2j in byte j's low nibble)
 *   [8D, 16D)  value codes, 8 bytes a group: + q*128 + (((i/8) ^ (q%2)) * 64) + (i%8)*8
 *   [16D, 17D) key scales (E4M3): + (i%8)*8L + (q/L)*2L + (i/8)*L + q%L
 *   [17D, 18D) value scales: + q*16 + (i%8)/2*4 + (i/8)*2 + i%2
 * so that one bulk copy fetches 16 tokens of one head, and each lane of a warp reads its
 * operands of the tensor-core products from it with few, conflict-free, wide loads.
 * k_scale, v_scale: the fp32 tensor scale g of each head [heads] (positive; NULL = all
 * 1.0), kept for the cache's life. A value stands for val * dec(sf) * g; the rule that
 * picks code and scale is mosaic.h's with this g instead of amax / 2688, so values beyond
 * 2688 g saturate. Slot s is token s % page_size of page s / page_size.
 */
typedef struct {
    uint8_t* pages; /* 128-byte aligned, mq_kv_cache_bytes bytes */
    int num_pages;
    int page_size;
    int heads;
    int D;
    const float* k_scale;
    const float* v_scale;
} mq_kv_cache;

/* num_pages * heads * page_size * 18 D / 16; 0 on a bad shape. */
size_t mq_kv_cache_bytes(int num_pages, int page_size, int heads, int D);

/*
 * Products of 16-bit activations with the packed weight (mq_gemm without quantizing X):
 *   Y[m,n] = rn( g_w * sum_k x[m,k] * ( wh[n,k] + [block (n/64, k/64) selected] rh[n,k] ) ),
 * wh and rh the scaled E2M1 values (val * dec(sf)), the sum in fp32. X: [M][K], row m at
 * m * ldx elements (16-byte aligned, ldx % 8 == 0); Y: [M][N], row m at m * ldy.
 * 1 <= M <= 16 tokens (MQ_ERR_UNSUPPORTED_SHAPE above: mq_gemm serves those), N and K any
 * multiples of 64 (N up to 64 * 65535, MQ_ERR_UNSUPPORTED_SHAPE above). wq: codes, sf_swz (both 16-byte aligned), gscale [1]. r as in
 * mq_gemm, with blk_kt; blocks that tile_ptr puts past the store and columns that blk_kt puts
 * past K are left out and reported. flags: 0 or MQ_GEMM_BASE_ONLY / MQ_GEMM_RESIDUAL_ONLY;
 * MQ_GEMM_WEIGHTS_READY is taken and changes nothing (the weight is read while the activations
 * are prepared in any case). Repeated calls give the same bits. ws: mq_gemv_workspace_bytes,
 * 16-byte aligned, any contents; calls that share one must not overlap on the GPU.
 */
mq_status mq_gemv(const void* X, mq_dtype type, int64_t ldx, const mq_nvfp4_mat* wq, const mq_residual_packed* r,
                  void* Y, int64_t ldy, int M, int N, int K, unsigned flags, void* ws, size_t ws_bytes, mq_stream stream);

/* The activations as a tensor-core operand. 0 on a bad shape. */
size_t mq_gemv_workspace_bytes(int M, int K);

/*
 * RMS norm of every query and key head and the position rotation, in one pass:
 *   u = x * (mean_d x^2 + eps)^(-1/2) * w_d      (q_weight / k_weight NULL: u = x)
 *   (a, b) -> (a cos - b sin, b cos + a sin), angle = pos[t] * freq[i],
 * over the pairs (u_i, u_{i + rot/2}), or (u_2i, u_{2i+1}) if interleaved, i < rot / 2;
 * elements from rot on are not turned. eps >= 0 (with 0, a row of zeros has no norm: NaN). fp32
 * arithmetic, rounded once; the angle is formed
 * and reduced in fp64. q, k: [T][heads][D]; q_out, k_out of the same heads (may be the
 * input itself, not a shifted view of it). pos: [T] (any value within +-2^53), freq: fp64 [rot/2] radians
 * a position. D = 64, 128 or 256, rot a multiple of 16 from 0 to D (0: pos and freq may be
 * NULL). k (with k_out) may be NULL, and so may q (with q_out). T >= 0.
 */
mq_status mq_qk_norm_rope(const mq_heads* q, const mq_heads* k, const mq_heads* q_out, const mq_heads* k_out, int T,
                          int D, mq_dtype type, const void* q_weight, const void* k_weight, float eps,
                          const int64_t* pos, const double* freq, int rot, int interleaved, mq_stream stream);

/*
 * Quantizes K and V rows [T][cache heads][D] into the cache at slots[t]. A negative slot
 * skips its token (padding); one past the cache is skipped and reported. The slots of one
 * call are distinct: a slot named twice ends up with a mixture of its rows. The rows are finite,
 * as mosaic.h's inputs are: sixteen NaN in a row of v would also reach query rows that do not see
 * their token, where others of their sequence do.
 */
mq_status mq_kv_append(const mq_heads* k, const mq_heads* v, int T, mq_dtype type, const int64_t* slots,
                       const mq_kv_cache* cache, mq_stream stream);

/*
 * mq_qk_norm_rope and mq_kv_append in one launch: queries to q_out; the keys, normed,
 * turned and rounded to `type` as there, and the values into the cache. The results are
 * those of the two calls, bit for bit. k_out may be NULL (the keys are kept in the cache
 * alone). D = 64 or 128.
 */
mq_status mq_qkv_append(const mq_heads* q, const mq_heads* k, const mq_heads* v, const mq_heads* q_out,
                        const mq_heads* k_out, int T, mq_dtype type, const void* q_weight, const void* k_weight,
                        float eps, const int64_t* pos, const double* freq, int rot, int interleaved,
                        const int64_t* slots, const mq_kv_cache* cache, mq_stream stream);

/*
 * The cached rows of slots[t] as 16-bit values, rn(val * fp32(dec(sf) * g)): k, v
 * [T][cache heads][D]. The rows of a negative slot are left as they were; so are those of
 * a slot past the cache, which is reported.
 */
mq_status mq_kv_read(const mq_kv_cache* cache, const int64_t* slots, int T, const mq_heads* k, const mq_heads* v,
                     mq_dtype type, mq_stream stream);

/* Workspace of mq_kv_attention for the current device: counters, then partial results of the
 * pieces into which it cuts long sequences. All zero before the first call on a workspace;
 * every call leaves the counters zero (one that ended in MQ_ERR_TIMEOUT may not: zero it
 * again), so calls of any shapes may take turns on one that is large enough for each. Calls
 * that share a workspace must not overlap on the GPU (two captured graphs included). 0 on a
 * bad shape. */
size_t mq_kv_attention_workspace_bytes(int q_heads, int kv_heads, int D, int max_q);

/*
 * Attention of the newest tokens of B sequences over the cache. Sequence b holds
 * kv_len[b] cached tokens (its query tokens' own keys and values among them), token j at
 * page block_table[b * table_stride + j / page_size]. Its query tokens are rows cu_q[b] to
 * cu_q[b+1] of q (cu_q NULL: row b alone, T = B); row i of n sits at position
 * p = kv_len[b] - n + i and sees the cached tokens j <= p, and j > p - window if window > 0.
 *   out = sum_j softmax_j(scale * q . K_j) V_j,   lse = ln sum_j exp(scale * q . K_j).
 * Query head h reads cache head h / (q heads / cache heads). A row that sees nothing gets
 * zeros (lse -inf). Scores, softmax sums and outputs are held in fp32; the softmax weights
 * enter the second product in fp16, and bf16 queries the first one as mq_gemv's activations do. Rows of q that belong to no sequence leave out and lse
 * as they were. A page outside the cache, a length past the table (or 2^30) or a row past T is
 * left out and reported. q, out: [T][q heads][D] (distinct); lse: fp32 [T][q heads] or NULL.
 * max_q: the largest number of query tokens of a sequence that the caller expects (it sizes
 * ws and, with the call's other sizes, picks the kernel; more are served too). Prompts and
 * single tokens may share a call: T other than B * max_q says so, and each sequence goes to the
 * kernel that its own rows and length ask for. q heads a
 * multiple of cache heads.
 * Repeated calls give the same bits. T >= 0, B >= 0.
 */
mq_status mq_kv_attention(const mq_heads* q, const mq_heads* out, float* lse, int T, mq_dtype type,
                          const mq_kv_cache* cache, const int32_t* block_table, int64_t table_stride, int max_pages,
                          int B, const int32_t* cu_q, int max_q, const int32_t* kv_len, float scale, int window,
                          void* ws, size_t ws_bytes, mq_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* MOSAIC_OPS_H_ */
