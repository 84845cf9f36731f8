// Types and launchers of the operators declared in mosaic_ops.h, shared by their kernels
// and the host side (ops.cu).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "mosaic_ops.h"
#include "nvfp4.cuh"

namespace mq {

// Two 16-bit values of a word (the low one first) widened to fp32, and back with one
// rounding to nearest even.
template <bool F16>
__device__ __forceinline__ float2 widen2(uint32_t w) {
    if constexpr (F16)
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    else
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <bool F16>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
    uint32_t w;
    if constexpr (F16)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}

// A [tokens][heads][D] operand of 16-bit elements.
struct HeadsView {
    uint16_t* p;
    int heads;
    int64_t st, sh;
};

struct CacheView {
    uint8_t* pages;
    int num_pages, page_size, heads, D;
    const float *k_scale, *v_scale;  // null: 1.0
};

// Byte offset of (token i, group q) in a record: its 8 value-code bytes, its key scale and
// its value scale (mosaic_ops.h states the layout).
template <int D>
__device__ __forceinline__ int rec_vcodes(int i, int q) {
    return 8 * D + q * 128 + (((i >> 3) ^ (q & 1)) << 6) + ((i & 7) << 3);
}
template <int D>
__device__ __forceinline__ int rec_kscale(int i, int q) {
    constexpr int L = D / 64;
    return 16 * D + (i & 7) * (8 * L) + (q / L) * (2 * L) + (i >> 3) * L + q % L;
}
template <int D>
__device__ __forceinline__ int rec_vscale(int i, int q) {
    return 17 * D + q * 16 + ((i & 7) >> 1) * 4 + ((i >> 3) << 1) + (i & 1);
}

// Records an index that a kernel found out of range in the device error word.
__device__ __forceinline__ void report_index(int* err) { atomicCAS(err, 0, (int)MQ_ERR_INVALID_ARG); }

// Division of n < 2^31 by d >= 1, d known on the host: a multiply and a shift (Granlund and
// Montgomery's round-up method).
struct FastDiv {
    int d;
    uint32_t mul;
    int shift;
    FastDiv() = default;
    explicit FastDiv(int divisor) : d(divisor), shift(0) {
        while ((int64_t(1) << shift) < d) ++shift;
        mul = (uint32_t)(((uint64_t(1) << 32) * ((uint64_t(1) << shift) - (uint64_t)d)) / (uint64_t)d + 1);
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};

struct HeadsParams {
    HeadsView q, k, v, qo, ko;  // p == null: absent
    int T;
    const uint16_t *wq, *wk;    // null: no norm
    float eps;
    const int64_t* pos;
    const double* freq;
    int rot, interleaved;
    const int64_t* slots;       // with a cache
    CacheView cache;            // pages == null: none
    int* err;
    FastDiv by_page;            // tokens of a page
};

struct GemvParams {
    const uint16_t* X;
    int64_t ldx;
    const uint8_t *codes, *sf;
    const float* g_w;
    const uint8_t *blk_codes, *blk_sf;  // null: no residual
    const int32_t *blk_kt, *tile_ptr;
    int nblk;
    uint16_t* Y;
    int64_t ldy;
    int M, N, K;
    int base;     // 0: the residual alone
    uint8_t* xop;  // workspace: the activations as an operand
    int* err;
};

struct AttnParams {
    HeadsView q, o;
    float* lse;  // [T][heads] or null
    int T;
    CacheView cache;
    const int32_t* table;
    int64_t table_stride;
    int max_pages, B;
    const int32_t* cu_q;  // null: one query token a sequence
    const int32_t* kv_len;
    float scale;
    int window;
    float* partial;
    int* counters;
    int* err;
    FastDiv by_group, by_page, by_grid;  // query heads of a cache head, tokens of a page, CTAs
    int split;                           // both kernels run: attn.cuh says which sequences are whose
    int least;                           // with split: the query rows of a sequence that it is about,
    int64_t even;                        // and kRowsWorth rows for each SM
};

// api.cu: a launch's status, counted in mq_launch_count; the current device's error word
mq_status count_launches(cudaError_t e, int kernels);
int* device_error_word();
// a byte matrix in boxes of 128 bytes x 64 rows, 128-byte swizzle; zeros outside
bool tensor_map_w64(CUtensorMap* map, const void* base, uint64_t row_bytes, uint64_t rows);
int device_sms();  // gemm.cu: SMs of the current device (148 without one)

cudaError_t launch_heads(const HeadsParams& p, int D, bool f16, cudaStream_t s);
cudaError_t launch_kv_read(const HeadsParams& p, int D, bool f16, cudaStream_t s);
// tw: the codes (tensor_map_w64)
size_t gemv_workspace(int M, int K);
cudaError_t launch_gemv(const CUtensorMap& tw, const GemvParams& p, bool f16, cudaStream_t s);
// bytes: counters, then partial sums at *partials_at
size_t attn_workspace(int q_heads, int kv_heads, int D, int max_q, size_t* partials_at);
// *kernels: how many were launched
cudaError_t launch_attn(const AttnParams& p, int D, int max_q, bool f16, cudaStream_t s, int* kernels);

}  // namespace mq
