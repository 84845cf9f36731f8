// Attention of new tokens over the NVFP4 cache:
//   out = sum_j softmax_j(scale q . K_j) V_j over the cached tokens that a query row sees.
//
// What bounds it: the cache's bytes, 9/8 D a token and head, read once for all the query
// rows of a cache head (a "row" is a query token and one of the query heads that share it).
//
// One pass. A warp takes 32 tokens at a time: two records of the cache, one bulk copy each,
// into its own ring in shared memory. Its products run on the tensor cores with the
// *tokens* as the 16-row operand, so eight query rows fill the other one:
//   S^T[token][row] = K[token][d] Q^T[d][row],   O^T[d][row] += V^T[d][token] P^T[token][row].
// E2M1 times E4M3 has at most six significant bits and lies in [2^-10, 2688], so the
// dequantized operand is exact in fp16: one conversion and one packed multiply per two
// elements, no tensor scale (it joins the softmax scale and the last division). The order of d
// inside a product is free, so a lane takes 16 adjacent bytes of a row. V^T wants pairs of
// tokens: two byte permutes per pair of elements. bf16 queries are scaled by a power of two
// per row to fit fp16 (what falls below is under 2^-39 of the row's largest element).
//
// Softmax: p = 2^(z - m + 7), z = scale log2(e) q . K. The reference m of a row is raised only
// when a score passes it by 8 (one vote a step, no shuffles), so p stays under 2^15 and its
// fp16 copy keeps all 11 bits down to 2^-21 of the largest. Sums and outputs are fp32.
//
// Work split: every (sequence, cache head, tile of rows) is a run of 128-token units; the
// units of all runs are numbered through, and CTA w of a grid that just fills the GPU takes the w-th
// equal share, wherever the sequences end. Runs that a share boundary cuts leave partial
// sums in the workspace; whoever finishes a run last adds its parts in their order, so the
// result does not depend on the timing.
#include <cfloat>
#include <climits>

#include "ops.cuh"

namespace mq {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = 32;               // tokens a warp takes at a time
constexpr int kUnit = kStep * kWarps;   // tokens of a unit
constexpr int kStages = 3;              // steps in flight per warp
constexpr float kShift = 7.0f;          // exponent offset of the fp16 softmax weights
constexpr float kSlack = 8.0f;          // how far a score may pass its row's reference

template <int NT>
constexpr int ctas_per_sm() { return NT == 1 ? 3 : 2; }

// Rows, partials and counters: the workspace of a grid.
__host__ __device__ constexpr int slot_floats(int nt, int D) { return 8 * nt * (D + 2); }

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit elements held by the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The eight codes of a word as four fp16 pairs (element 2j, 2j + 1).
__device__ __forceinline__ void e2m1x8_half(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
// Four E4M3 bytes as two fp16 pairs.
__device__ __forceinline__ void e4m3x4_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t low2(uint32_t a) { return __byte_perm(a, a, 0x1010); }
__device__ __forceinline__ uint32_t high2(uint32_t a) { return __byte_perm(a, a, 0x3232); }

// Sequence b: its rows of q and its length, checked.
struct Seq {
    int row0, nq, len;
};
__device__ __forceinline__ Seq seq_of(const AttnParams& p, int b, bool report) {
    Seq s;
    s.row0 = p.cu_q ? __ldg(p.cu_q + b) : b;
    const int hi = p.cu_q ? __ldg(p.cu_q + b + 1) : b + 1;
    s.nq = hi - s.row0;
    s.len = __ldg(p.kv_len + b);
    if (s.row0 < 0 || hi < s.row0 || hi > p.T) {
        if (report) report_index(p.err);
        s.row0 = s.nq = 0;
    }
    if (s.len < 0 || s.len > (int64_t)p.max_pages * p.cache.page_size) {
        if (report) report_index(p.err);
        s.len = 0;
    }
    return s;
}
// The tokens that rows [r0, r0 + rows) of a sequence's nq * G rows can see: [begin, end), begin
// rounded down to a step.
__device__ __forceinline__ void range_of(const Seq& s, int G, int window, int r0, int rows, int& begin, int& end) {
    const int last = min(r0 + rows, s.nq * G) - 1;
    end = max(0, s.len - s.nq + last / G + 1);
    begin = 0;
    if (window > 0) {
        const int64_t lo = (int64_t)s.len - s.nq + r0 / G - window + 1;
        begin = lo > 0 ? (int)lo / kStep * kStep : 0;
    }
}
__device__ __forceinline__ int units_of(const Seq& s, int G, int window, int r0, int rows) {
    int begin, end;
    range_of(s, G, window, r0, rows, begin, end);
    return max(1, (end - begin + kUnit - 1) / kUnit);  // one for rows that see nothing: they are written too
}
// Units of one cache head of a sequence.
__device__ __forceinline__ int64_t seq_units(const Seq& s, int G, int window, int rows) {
    int64_t n = 0;
    for (int r0 = 0; r0 < s.nq * G; r0 += rows) n += units_of(s, G, window, r0, rows);
    return n;
}

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
// ln of the sum of 2^z, kept as sum = sum of 2^(z - top + kShift).
__device__ __forceinline__ float lse_of(float top, float sum) {
    return sum > 0.0f ? (top - kShift + log2f(sum)) * 0.69314718055994531f : -INFINITY;
}

template <int D, int NT, bool F16>
__global__ void __launch_bounds__(kThreads, ctas_per_sm<NT>()) k_attn(const AttnParams p) {
    constexpr bool PAIR = NT == 1;
    constexpr int R = 8 * NT;           // rows of a tile
    constexpr int REC = 18 * D;         // bytes of a record
    constexpr int KS = D / 16;          // products of 16 d per token tile; also d tiles of the output
    constexpr int RS = D + 4;           // floats of a merged row in shared memory
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[kWarps][kStages];
    __shared__ float sm_m[kWarps][R], sm_l[kWarps][R];
    __shared__ int64_t red[kWarps];
    __shared__ int64_t found[4];
    __shared__ int last_part;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int H = p.cache.heads, G = p.q.heads / H;
    if (tid < kWarps * kStages) mbar_init(&full[0][0] + tid, 1);
    mbar_fence_init();
    griddep_wait();
    griddep_launch();

    // total units, then the sequence that holds this CTA's first one
    const int64_t own = tid < p.B ? seq_units(seq_of(p, tid, blockIdx.x == 0), G, p.window, R) * H : 0;
    int64_t mine = own;
    for (int b = tid + kThreads; b < p.B; b += kThreads)
        mine += seq_units(seq_of(p, b, blockIdx.x == 0), G, p.window, R) * H;
    mine = warp_sum(mine);
    if (lane == 0) red[warp] = mine;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += red[w];
    if (total == 0) return;
    const int64_t share = (total + gridDim.x - 1) / gridDim.x;
    const int64_t u0 = share * blockIdx.x, u1 = min(u0 + share, total);
    if (u0 >= u1) return;
    {
        int64_t base = 0;
        for (int b0 = 0; b0 < p.B; b0 += kThreads) {
            const int b = b0 + tid;
            const int64_t n = b0 == 0 ? own : b < p.B ? seq_units(seq_of(p, b, false), G, p.window, R) * H : 0;
            int64_t x = n;  // inclusive scan over the CTA
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            __syncthreads();
            if (lane == 31) red[warp] = x;
            __syncthreads();
            int64_t before = base, all = base;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                before += w < warp ? red[w] : 0;
                all += red[w];
            }
            x += before;
            if (n > 0 && u0 >= x - n && u0 < x) {
                found[0] = b;
                found[1] = x - n;
            }
            base = all;
            if (u0 < base) break;
        }
        __syncthreads();
    }
    int b = (int)found[0], h, r0 = 0, piece;
    Seq s = seq_of(p, b, false);
    int64_t run;  // unit number of the current run's first unit
    {
        const int64_t per = seq_units(s, G, p.window, R);
        int64_t off = u0 - found[1];
        h = (int)(off / per);
        off -= h * per;
        int n;
        while (off >= (n = units_of(s, G, p.window, r0, R))) {
            off -= n;
            r0 += R;
        }
        piece = (int)off;
        run = u0 - piece;
    }

    uint8_t* ring = smem + warp * (kStages * 2 * REC);
    float* merge = reinterpret_cast<float*>(smem);
    uint32_t at = 0, phase = 0;  // ring place and parity of this warp's next step
    bool alive = true;  // false after a wait that gave up
    int64_t u = u0;
    while (true) {
        // ---------------------------------------------------------------- one run, or this CTA's part of it
        int begin, end;
        range_of(s, G, p.window, r0, R, begin, end);
        const int units = max(1, (end - begin + kUnit - 1) / kUnit);
        const int take = (int)min((int64_t)(units - piece), u1 - u);
        const float gk = p.cache.k_scale ? __ldg(p.cache.k_scale + h) : 1.0f;
        const float gv = p.cache.v_scale ? __ldg(p.cache.v_scale + h) : 1.0f;

        // this warp's steps, and their copies: two records each
        const int first = begin + piece * kUnit + warp * kStep;
        const int steps = first < end ? min(take, (end - first + kUnit - 1) / kUnit) : 0;
        uint32_t bad = 0;           // bits 2 i, 2 i + 1: record 0 or 1 of the step in ring place i is not there
        uint32_t to = at;           // ring place of the next issue
        const uint8_t* src = nullptr;  // lane 2 i + r: record r of step 16 k + i (null: not there), 16 steps at a time
        auto issue = [&](int step) {
            if ((step & 15) == 0) {
                const int j = first + (step + (lane >> 1)) * kUnit + 16 * (lane & 1);
                src = nullptr;
                if (j < end) {
                    const int pg = j / p.cache.page_size;
                    const int page = __ldg(p.table + b * p.table_stride + pg);
                    if (page >= 0 && page < p.cache.num_pages)
                        src = p.cache.pages +
                              (((int64_t)page * H + h) * (p.cache.page_size >> 4) + ((j - pg * p.cache.page_size) >> 4)) * REC;
                    else if (step + (lane >> 1) < steps)
                        report_index(p.err);
                }
            }
            const int turn = step & 15;
            const uint32_t have = (__ballot_sync(0xffffffffu, src != nullptr) >> (2 * turn)) & 3u;
            bad = (bad & ~(3u << (2 * to))) | ((~have & 3u) << (2 * to));
            uint64_t* bar = &full[warp][to];
            if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)__popc(have) * REC);
            __syncwarp();
            if ((lane >> 1) == turn && src) bulk_load(ring + to * (2 * REC) + (lane & 1) * REC, src, REC, bar);
            to = to + 1 == kStages ? 0 : to + 1;
        };
#pragma unroll
        for (int i = 0; i < kStages; ++i)
            if (i < steps && alive) issue(i);

        // this lane's query elements (row 8 nt + g, d = t D/4 ...) as the second operand, and
        // the scale and limits of its score columns (rows 8 nt + 2t, + 2t + 1)
        uint32_t qf[NT][KS][2];
        float qs[NT][2];
        int lim[NT][2];
        float m[NT][2], l[NT][2];
        float ref[NT][2];    // m - kShift (0 while m is -inf)
        float limit[NT][2];  // the unscaled score that raises m
        // outputs: with PAIR, o[2 i + e] holds elements e of the d pairs 2 i, 2 i + 1
        float o[KS][NT][4];
        int lim_min = INT_MAX;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = r0 + 8 * nt + g, rows = s.nq * G;
            float inv = 0.0f;
#pragma unroll
            for (int j = 0; j < KS; ++j) qf[nt][j][0] = qf[nt][j][1] = 0u;
            if (row < rows) {
                const int qi = row / G;
                const uint4* src = reinterpret_cast<const uint4*>(p.q.p + (int64_t)(s.row0 + qi) * p.q.st +
                                                                  (int64_t)(h * G + row - qi * G) * p.q.sh + t * (D / 4));
#pragma unroll
                for (int i = 0; i < KS / 2; ++i) {
                    const uint4 v = __ldg(src + i);
                    qf[nt][2 * i][0] = v.x;
                    qf[nt][2 * i][1] = v.y;
                    qf[nt][2 * i + 1][0] = v.z;
                    qf[nt][2 * i + 1][1] = v.w;
                }
                inv = 1.0f;
                if (F16 && p.scale < 0.0f)  // the sign of the scale goes into the query: qs > 0
#pragma unroll
                    for (int j = 0; j < KS; ++j) qf[nt][j][0] ^= 0x80008000u, qf[nt][j][1] ^= 0x80008000u;
            }
            if constexpr (!F16) {
                float top = 0.0f;
#pragma unroll
                for (int j = 0; j < KS; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 f = widen2<false>(qf[nt][j][i]);
                        top = max3(top, fabsf(f.x), fabsf(f.y));
                    }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // the largest element to [2^14, 2^15)
                const uint32_t ex = max(__float_as_uint(top) >> 23, 15u);
                const float up = copysignf(__uint_as_float((268u - ex) << 23), p.scale);
                inv *= __uint_as_float((ex - 14u) << 23);
#pragma unroll
                for (int j = 0; j < KS; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 f = widen2<false>(qf[nt][j][i]);
                        qf[nt][j][i] = narrow2<true>(f.x * up, f.y * up);
                    }
            }
            // never zero: a masked score is -inf before the scale (with this least scale every
            // other score rounds to 0)
            const float z = fmaxf(inv * gk * fabsf(p.scale), FLT_MIN);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                qs[nt][c] = __shfl_sync(0xffffffffu, z, 4 * (2 * t + c));
                const int r = r0 + 8 * nt + 2 * t + c;
                lim[nt][c] = r < rows ? s.len - s.nq + r / G + 1 : INT_MAX;
                lim_min = min(lim_min, lim[nt][c]);
                m[nt][c] = -INFINITY;
                ref[nt][c] = 0.0f;
                limit[nt][c] = -INFINITY;
                l[nt][c] = 0.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < KS; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[j][nt][c] = 0.0f;
        lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, 1));
        lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, 2));
        // the last row's window starts last
        const int lo_max = p.window > 0 ? end - p.window : 0;
        const int lo_min = p.window > 0 ? s.len - s.nq + r0 / G + 1 - p.window : 0;

        for (int step = 0; step < steps && alive; ++step) {
            if (!mbar_wait_err(&full[warp][at], phase, p.err)) alive = false;
            if (!__all_sync(0xffffffffu, alive)) {
                // give the copies behind it their (bounded) time, then leave
                alive = false;
                for (int i = 1; i < min(steps - step, kStages); ++i) {
                    const uint32_t x = at + i;
                    mbar_wait_err(&full[warp][x % kStages], phase ^ (x >= kStages), p.err);
                }
                break;
            }
            const uint8_t* buf = ring + at * (2 * REC);
            const int j0 = first + step * kUnit;
            const uint32_t lost = (bad >> (2 * at)) & 3u;
            // every row sees every token of the step
            const bool whole = j0 + kStep <= lim_min && j0 >= lo_max && lost == 0;

            // ---- scores
            float z[2][NT][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint8_t* rec = buf + r * REC;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) z[r][nt][c] = 0.0f;
                uint32_t ka[KS / 2], kb[KS / 2], s0, s1;  // tokens g and g + 8
                uint32_t sa[2], sb[2];
                if constexpr (D == 128) {
                    const uint4 x = *reinterpret_cast<const uint4*>(rec + g * 64 + t * 16);
                    const uint4 y = *reinterpret_cast<const uint4*>(rec + 512 + g * 64 + t * 16);
                    ka[0] = x.x, ka[1] = x.y, ka[2] = x.z, ka[3] = x.w;
                    kb[0] = y.x, kb[1] = y.y, kb[2] = y.z, kb[3] = y.w;
                    e4m3x4_half(*reinterpret_cast<const uint32_t*>(rec + 16 * D + lane * 4), s0, s1);
                    sa[0] = low2(s0), sa[1] = high2(s0), sb[0] = low2(s1), sb[1] = high2(s1);
                } else {
                    const uint2 x = *reinterpret_cast<const uint2*>(rec + g * 32 + t * 8);
                    const uint2 y = *reinterpret_cast<const uint2*>(rec + 256 + g * 32 + t * 8);
                    ka[0] = x.x, ka[1] = x.y;
                    kb[0] = y.x, kb[1] = y.y;
                    // a lane pair's two scales each lie in one word
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(rec + 16 * D + (lane >> 1) * 4);
                    e4m3x4_half(w, s0, s1);
                    const uint32_t mine2 = (lane & 1) ? s1 : s0;
                    sa[0] = sa[1] = low2(mine2), sb[0] = sb[1] = high2(mine2);
                }
#pragma unroll
                for (int w = 0; w < KS / 2; ++w) {
                    uint32_t x[4], y[4];
                    e2m1x8_half(ka[w], x);
                    e2m1x8_half(kb[w], y);
                    const uint32_t fa = sa[2 * w / (KS / 2)], fb = sb[2 * w / (KS / 2)];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t a[4] = {mul_h2(x[2 * i], fa), mul_h2(y[2 * i], fb), mul_h2(x[2 * i + 1], fa),
                                               mul_h2(y[2 * i + 1], fb)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_f16(z[r][nt], a, qf[nt][2 * w + i][0], qf[nt][2 * w + i][1]);
                    }
                }
            }
            if (!whole) {
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int j = j0 + 16 * r + g + 8 * (c >> 1), top = lim[nt][c & 1];
                            const bool see = j < min(top, end) && (p.window == 0 || j >= top - p.window) && !((lost >> r) & 1u);
                            if (!see) z[r][nt][c] = -INFINITY;
                        }
            }

            // ---- softmax weights
            bool rise = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    rise |= fmaxf(max3(z[0][nt][c], z[0][nt][c + 2], z[1][nt][c]), z[1][nt][c + 2]) > limit[nt][c];
            if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float top = fmaxf(max3(z[0][nt][c], z[0][nt][c + 2], z[1][nt][c]), z[1][nt][c + 2]);
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                        const float mn = fmaxf(m[nt][c], top * qs[nt][c]);
                        const float f = mn == -INFINITY ? 1.0f : ex2(m[nt][c] - mn);
                        m[nt][c] = mn;
                        ref[nt][c] = mn == -INFINITY ? 0.0f : mn - kShift;
                        limit[nt][c] = (mn + kSlack) / qs[nt][c];
                        l[nt][c] *= f;
#pragma unroll
                        for (int j = 0; j < KS; ++j) {
                            o[j][nt][c] *= f;
                            o[j][nt][c + 2] *= f;
                        }
                    }
            }
            uint32_t pb[2][NT][2];  // weights as the second operand: row g, tokens 2t, 2t + 1 and + 8
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float w[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        w[c] = ex2(__fmaf_rn(z[r][nt][c], qs[nt][c & 1], -ref[nt][c & 1]));
                        l[nt][c & 1] += w[c];
                    }
                    pb[r][nt][0] = transpose8x8(narrow2<true>(w[0], w[1]));
                    pb[r][nt][1] = transpose8x8(narrow2<true>(w[2], w[3]));
                }

            // ---- outputs
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint8_t* rec = buf + r * REC;
                uint32_t sc;
                if constexpr (D == 128)
                    sc = *reinterpret_cast<const uint32_t*>(rec + 17 * D + g * 16 + t * 4);
                else
                    sc = *reinterpret_cast<const uint32_t*>(rec + 17 * D + (g >> 1) * 16 + t * 4);
                if (!whole) {
                    // tokens that no row sees may hold anything: their scales become zero
                    uint32_t keep = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = j0 + 16 * r + 2 * t + (i & 1) + 8 * (i >> 1);
                        if (j < end && j >= lo_min && !((lost >> r) & 1u)) keep |= 0xFFu << (8 * i);
                    }
                    sc &= keep;
                }
                uint32_t sab, scd;
                e4m3x4_half(sc, sab, scd);
                const uint32_t f[4] = {low2(sab), high2(sab), low2(scd), high2(scd)};  // tokens 2t, 2t+1, 2t+8, 2t+9
                uint32_t v[4][KS / 4];                                                // their codes of this lane's d
                if constexpr (D == 128) {
                    const uint8_t* base = rec + 8 * D + g * 128 + t * 16;
                    const uint4 x = *reinterpret_cast<const uint4*>(base + ((g & 1) << 6));
                    const uint4 y = *reinterpret_cast<const uint4*>(base + (((g & 1) ^ 1) << 6));
                    v[0][0] = x.x, v[0][1] = x.y, v[1][0] = x.z, v[1][1] = x.w;
                    v[2][0] = y.x, v[2][1] = y.y, v[3][0] = y.z, v[3][1] = y.w;
                } else {
                    const int q = g >> 1;
                    const uint8_t* base = rec + 8 * D + q * 128 + t * 16 + (g & 1) * 4;
                    const uint8_t *x = base + ((q & 1) << 6), *y = base + (((q & 1) ^ 1) << 6);
                    v[0][0] = *reinterpret_cast<const uint32_t*>(x), v[1][0] = *reinterpret_cast<const uint32_t*>(x + 8);
                    v[2][0] = *reinterpret_cast<const uint32_t*>(y), v[3][0] = *reinterpret_cast<const uint32_t*>(y + 8);
                }
#pragma unroll
                for (int w = 0; w < KS / 4; ++w) {
                    uint32_t x[4][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        e2m1x8_half(v[i][w], x[i]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[i][e] = mul_h2(x[i][e], f[i]);
                    }
                    if constexpr (PAIR) {
                        // the product's k pair is the two d of a byte, its row a byte: against (p, 0)
                        // it sums the even d, against (0, p) the odd ones, eight tokens a product
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {  // tokens 0..7, 8..15
                                const uint32_t a[4] = {x[2 * e][2 * i], x[2 * e][2 * i + 1], x[2 * e + 1][2 * i],
                                                       x[2 * e + 1][2 * i + 1]};
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    const uint32_t pr = pb[r][nt][e];
                                    mma_f16(o[2 * (2 * w + i)][nt], a, pr & 0xFFFFu, pr >> 16);
                                    mma_f16(o[2 * (2 * w + i) + 1][nt], a, pr << 16, pr & 0xFFFF0000u);
                                }
                            }
                    } else
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t a[4] = {__byte_perm(x[0][e], x[1][e], 0x5410), __byte_perm(x[0][e], x[1][e], 0x7632),
                                               __byte_perm(x[2][e], x[3][e], 0x5410), __byte_perm(x[2][e], x[3][e], 0x7632)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_f16(o[4 * w + e][nt], a, pb[r][nt][0], pb[r][nt][1]);
                    }
                }
            }
            __syncwarp();
            if (step + kStages < steps) issue(step + kStages);
            if (++at == kStages) at = 0, phase ^= 1u;
        }

        // ---------------------------------------------------------------- join the warps
        // Without PAIR, o[j][.][c] is d = g D/8 + 2 j + (c >> 1). A merged row lies as [j][g][2] (d = g D/8 + 2 j + .), RS floats.
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], x);
        if (g == 0)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    sm_m[warp][8 * nt + 2 * t + c] = m[nt][c];
                    sm_l[warp][8 * nt + 2 * t + c] = l[nt][c];
                }
        __syncthreads();  // every ring is idle: its memory takes the merge
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int row = 8 * nt + 2 * t + c;
                float top = sm_m[0][row];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sm_m[w][row]);
                const float f = m[nt][c] == -INFINITY ? 0.0f : ex2(m[nt][c] - top);
                float2* dst = reinterpret_cast<float2*>(merge + (warp * R + row) * RS) + g;
#pragma unroll
                for (int j = 0; j < KS; ++j)
                    dst[8 * j] = PAIR ? make_float2(o[j & ~1][nt][c + 2 * (j & 1)] * f, o[j | 1][nt][c + 2 * (j & 1)] * f)
                                      : make_float2(o[j][nt][c] * f, o[j][nt][c + 2] * f);
            }
        __syncthreads();
        const int rows = min(R, s.nq * G - r0);
        const int64_t w_first = run / share, w_last = (run + units - 1) / share;
        const int parts = (int)(w_last - w_first + 1);
        constexpr int PAIRS = D / 2, RPP = kThreads / PAIRS;  // float2s of a row, rows per pass
        const int pi = tid % PAIRS;                           // output elements 2 pi, 2 pi + 1
        const int pg = pi / KS, pj = pi % KS;
        if (parts > 1) {
            // slot 0 of a CTA: a run that an earlier CTA began; slot 1: one that it begins itself
            const int64_t slot = 2 * (int64_t)blockIdx.x + (run < u0 ? 0 : 1);
            float* dst = p.partial + slot * slot_floats(NT, D);
            for (int row = tid / PAIRS; row < rows; row += RPP) {
                float2 a = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float2 v = reinterpret_cast<const float2*>(merge + (w * R + row) * RS)[8 * pj + pg];
                    a.x += v.x;
                    a.y += v.y;
                }
                reinterpret_cast<float2*>(dst + row * D)[pi] = a;
                if (pi == 0) {
                    float top = sm_m[0][row], sum = 0.0f;
#pragma unroll
                    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sm_m[w][row]);
#pragma unroll
                    for (int w = 0; w < kWarps; ++w)
                        sum += sm_m[w][row] == -INFINITY ? 0.0f : sm_l[w][row] * ex2(sm_m[w][row] - top);
                    dst[R * D + row] = top;
                    dst[R * D + R + row] = sum;
                }
            }
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const int old = atomicAdd(p.counters + w_first, 1);
                last_part = old == parts - 1;
                if (last_part) p.counters[w_first] = 0;
            }
            __syncthreads();
            if (last_part) __threadfence();
        }
        if (parts == 1) {
            for (int row = tid / PAIRS; row < rows; row += RPP) {
                float2 a = make_float2(0.0f, 0.0f);
                float top = sm_m[0][row], sum = 0.0f;
#pragma unroll
                for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sm_m[w][row]);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float2 v = reinterpret_cast<const float2*>(merge + (w * R + row) * RS)[8 * pj + pg];
                    a.x += v.x;
                    a.y += v.y;
                    sum += sm_m[w][row] == -INFINITY ? 0.0f : sm_l[w][row] * ex2(sm_m[w][row] - top);
                }
                const int qi = (r0 + row) / G, hq = h * G + r0 + row - qi * G;
                const int64_t tok = s.row0 + qi;
                const float inv = sum > 0.0f ? gv / sum : 0.0f;
                *reinterpret_cast<uint32_t*>(p.o.p + tok * p.o.st + hq * p.o.sh + 2 * pi) = narrow2<F16>(a.x * inv, a.y * inv);
                if (p.lse && pi == 0) p.lse[tok * p.q.heads + hq] = lse_of(top, sum);
            }
        } else if (last_part) {
            // part 0 lies in its CTA's slot 1, the others in their CTAs' slots 0. A warp takes a
            // row's maxima and sums and leaves the parts' factors in shared memory; then all
            // threads add the rows, four elements each.
            constexpr int SLOT = slot_floats(NT, D), QUADS = D / 4;
            const float* part0 = p.partial + (2 * w_first + 1) * SLOT;
            const float* parts1 = p.partial + 2 * w_first * SLOT;  // part i > 0 at + 2 i SLOT
            float* fac = merge;                                    // [parts][R]: the merge's rows are not needed any more
            for (int row = warp; row < rows; row += kWarps) {
                float top = -INFINITY, sum = 0.0f;
                for (int i = lane; i < parts; i += 32)
                    top = fmaxf(top, __ldcg((i ? parts1 + (int64_t)2 * i * SLOT : part0) + R * D + row));
                top = warp_max(top);
                for (int i = lane; i < parts; i += 32) {
                    const float* src = (i ? parts1 + (int64_t)2 * i * SLOT : part0) + R * D + row;
                    const float mw = __ldcg(src), f = mw == -INFINITY ? 0.0f : ex2(mw - top);
                    fac[i * R + row] = f;
                    sum = __fmaf_rn(__ldcg(src + R), f, sum);
                }
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                if (lane == 0) {
                    sm_l[0][row] = sum;
                    sm_m[0][row] = top;
                }
            }
            __syncthreads();
            for (int i = tid; i < rows * QUADS; i += kThreads) {
                const int row = i / QUADS, d = 4 * (i - row * QUADS);
                float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                auto add = [&](const float4& v, float f) {
                    a.x = __fmaf_rn(v.x, f, a.x);
                    a.y = __fmaf_rn(v.y, f, a.y);
                    a.z = __fmaf_rn(v.z, f, a.z);
                    a.w = __fmaf_rn(v.w, f, a.w);
                };
                add(__ldcg(reinterpret_cast<const float4*>(part0 + row * D + d)), fac[row]);
                const float* src = parts1 + row * D + d;
                int w = 1;
                for (; w + 8 <= parts; w += 8) {
                    float4 v[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) v[x] = __ldcg(reinterpret_cast<const float4*>(src + (int64_t)2 * (w + x) * SLOT));
#pragma unroll
                    for (int x = 0; x < 8; ++x) add(v[x], fac[(w + x) * R + row]);
                }
                for (; w < parts; ++w) add(__ldcg(reinterpret_cast<const float4*>(src + (int64_t)2 * w * SLOT)), fac[w * R + row]);
                const int qi = (r0 + row) / G, hq = h * G + r0 + row - qi * G;
                const int64_t tok = s.row0 + qi;
                const float sum = sm_l[0][row], inv = sum > 0.0f ? gv / sum : 0.0f;
                *reinterpret_cast<uint2*>(p.o.p + tok * p.o.st + hq * p.o.sh + d) =
                    make_uint2(narrow2<F16>(a.x * inv, a.y * inv), narrow2<F16>(a.z * inv, a.w * inv));
                if (p.lse && d == 0) p.lse[tok * p.q.heads + hq] = lse_of(sm_m[0][row], sum);
            }
        }
        // ---------------------------------------------------------------- the next run
        u += take;
        if (u >= u1) break;
        fence_proxy_async_smem();  // the merge's writes come before the ring's next copies
        __syncthreads();
        run += units;
        piece = 0;
        r0 += R;
        if (r0 >= s.nq * G) {
            r0 = 0;
            if (++h == H) {
                h = 0;
                do s = seq_of(p, ++b, false);
                while (s.nq == 0);
            }
        }
    }
}

template <int D, int NT>
constexpr size_t smem_bytes() {
    const size_t ring = (size_t)kWarps * kStages * 2 * 18 * D, merge = (size_t)kWarps * 8 * NT * (D + 4) * 4;
    return ring > merge ? ring : merge;
}

template <int D, int NT, bool F16>
cudaError_t attn_of(const AttnParams& p, int grid, cudaStream_t s) {
    static std::atomic<bool> done[64];
    const cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(k_attn<D, NT, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<D, NT>());
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(k_attn<D, NT, F16>, dim3(grid), dim3(kThreads), smem_bytes<D, NT>(), s, 1, p);
}

int row_tiles(int q_heads, int kv_heads, int max_q) {
    return (int64_t)(q_heads / kv_heads) * max_q <= 8 ? 1 : 2;
}

int grid_of(int nt) { return device_sms() * (nt == 1 ? ctas_per_sm<1>() : ctas_per_sm<2>()); }

}  // namespace

size_t attn_workspace(int q_heads, int kv_heads, int D, int max_q, size_t* counters_at) {
    const int nt = row_tiles(q_heads, kv_heads, max_q), grid = grid_of(nt);
    *counters_at = (size_t)2 * grid * slot_floats(nt, D) * sizeof(float);
    return *counters_at + (size_t)grid * sizeof(int);
}

cudaError_t launch_attn(const AttnParams& p0, int D, int max_q, bool f16, cudaStream_t s) {
    AttnParams p = p0;
    p.scale *= 1.4426950408889634f;  // scores in powers of two
    const int nt = row_tiles(p.q.heads, p.cache.heads, max_q), grid = grid_of(nt);
    if (D == 64) {
        if (nt == 1) return f16 ? attn_of<64, 1, true>(p, grid, s) : attn_of<64, 1, false>(p, grid, s);
        return f16 ? attn_of<64, 2, true>(p, grid, s) : attn_of<64, 2, false>(p, grid, s);
    }
    if (nt == 1) return f16 ? attn_of<128, 1, true>(p, grid, s) : attn_of<128, 1, false>(p, grid, s);
    return f16 ? attn_of<128, 2, true>(p, grid, s) : attn_of<128, 2, false>(p, grid, s);
}

}  // namespace mq
