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
// Sum over the warp of values from 0 to 2^58, 22 bits at a time.
__device__ __forceinline__ int64_t warp_sum(int64_t v) {
    constexpr unsigned all = 0xffffffffu, low = (1u << 22) - 1;
    const int64_t a = __reduce_add_sync(all, (unsigned)v & low), b = __reduce_add_sync(all, (unsigned)(v >> 22) & low),
                  c = __reduce_add_sync(all, (unsigned)(v >> 44));
    return a + (b << 22) + (c << 44);
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

// Which sequences of a call are whose. A CTA of attn_rows.cu takes a tile of kRowsTile query rows
// through its tokens alone, kRowsStep a step, at a cost that does not go by how many rows there
// are: about what the other kernel needs for kRowsWorth rows on one SM. The other kernel cuts any
// sequence over all SMs. So attn_rows.cu is given a sequence with `least` rows or more (its tiles
// hold kRowsWorth each then) if its chain of steps is not longer than an SM's even share of what
// all such sequences cost in the other kernel. Both kernels find the same answer, from integers.
constexpr int kRowsTile = 256, kRowsStep = 64, kRowsWorth = 48;
constexpr int kRowsLeast = 56;  // `least` where the numbers of query tokens differ; below it where they do not

__device__ __forceinline__ int64_t rows_steps(const Seq& s, const AttnParams& p) {
    return (p.window > 0 ? min((int64_t)s.len, (int64_t)p.window + s.nq) : (int64_t)s.len) / kRowsStep + 1;
}
// A sequence's query rows times steps, if it has the rows.
__device__ __forceinline__ int64_t rows_work(const Seq& s, const AttnParams& p) {
    const int64_t rows = s.nq * p.by_group.d;
    return rows >= p.least ? rows * p.cache.heads * rows_steps(s, p) : 0;
}
// work: the sum over the call's sequences.
__device__ __forceinline__ bool takes_rows(const Seq& s, const AttnParams& p, int64_t work) {
    return s.nq * p.by_group.d >= p.least && rows_steps(s, p) * p.even <= work;
}

// attn_rows.cu: tiles of 256 query rows, D = 128 (by_group, by_page and the scale set as for the
// other kernel). Which kernels a call runs, and the rows of a sequence that may be that one's:
struct AttnPlan {
    bool other, rows;
    int least;
};
AttnPlan attn_plan(const AttnParams& p, int D, int max_q);
cudaError_t launch_attn_rows(const AttnParams& p, bool f16, cudaStream_t s);

}  // namespace mq
