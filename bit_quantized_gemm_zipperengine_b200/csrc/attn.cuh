// What the two attention kernels (attn.cu, attn_rows.cu) share: a sequence's checked extent,
// the tokens that a tile of its rows sees, and the softmax's constants.
#pragma once

#include "ops.cuh"

namespace mq {

constexpr int kStep = 32;         // a tile's tokens begin at a multiple of this
constexpr int kMaxLen = 1 << 30;  // cached tokens of a sequence
constexpr float kShift = 7.0f;    // exponent offset of the fp16 softmax weights
constexpr float kSlack = 8.0f;    // how far a score may pass its row's reference

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Sequence b: its rows of q and its length, checked.
struct Seq {
    int row0, nq, len;
};
__device__ __forceinline__ Seq seq_of(const AttnParams& p, int b, bool report) {
    Seq s;
    s.row0 = p.cu_q ? ld_prior(p.cu_q + b) : b;
    const int hi = p.cu_q ? ld_prior(p.cu_q + b + 1) : b + 1;
    s.nq = hi - s.row0;
    s.len = ld_prior(p.kv_len + b);
    if (s.row0 < 0 || hi < s.row0 || hi > p.T) {
        if (report) report_index(p.err);
        s.row0 = s.nq = 0;
    }
    if (s.len < 0 || s.len > kMaxLen || s.len > (int64_t)p.max_pages * p.cache.page_size) {
        if (report) report_index(p.err);
        s.len = 0;
    }
    return s;
}
// The tokens that rows [r0, r0 + rows) of a sequence's nq * G rows can see: [begin, end), begin
// rounded down to a step.
__device__ __forceinline__ void range_of(const Seq& s, const FastDiv& G, int window, int r0, int rows, int& begin, int& end) {
    const int last = min(r0 + rows, s.nq * G.d) - 1;
    end = max(0, s.len - s.nq + (int)G.div(last) + 1);
    begin = 0;
    if (window > 0) {
        const int64_t lo = (int64_t)s.len - s.nq + (int)G.div(r0) - window + 1;
        begin = lo > 0 ? (int)lo / kStep * kStep : 0;
    }
}
// ln of the sum of 2^z, kept as sum = sum of 2^(z - top + kShift).
__device__ __forceinline__ float lse_of(float top, float sum) {
    return sum == 0.0f ? -INFINITY : (top - kShift + log2f(sum)) * 0.69314718055994531f;
}

// attn_rows.cu: tiles of 256 query rows, D = 128; whether it serves a call (by_group, by_page and the
// scale set as for the other kernel)
bool attn_rows_serves(const AttnParams& p, int D);
cudaError_t launch_attn_rows(const AttnParams& p, bool f16, cudaStream_t s);

}  // namespace mq
