// Attention of new tokens over the NVFP4 cache:
//   out = sum_j softmax_j(scale q . K_j) V_j over the cached tokens that a query row sees.
//
// What bounds it: the cache's bytes, 9/8 D a token and head, read once for all the query
// rows of a cache head (a "row" is a query token and one of the query heads that share it).
// Calls, and sequences, with many rows a cache head and D = 128 go to attn_rows.cu (attn.cuh).
//
// Once a long cache streams, the conversions, multiplies and products that share the issue slots
// are the longer half: 4 x 131072 tokens, 64/8 heads take 127 us (4.8 TB/s), the copies alone
// 104, the arithmetic alone 122; half of the issue slots are used, the rest are waits. One sequence
// of 509 tokens takes 9.8 us, all latency.
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
// Work split: every (sequence, cache head, tile of rows) is a run of 128-token units. The grid
// just fills the GPU, and the runs are cut so that every CTA has about the same number of
// units, wherever the sequences end. Runs that are cut leave partial sums in the workspace;
// whoever finishes a run last adds its parts in their order, so the result does not depend on
// the timing.
#include <algorithm>
#include <cfloat>
#include <climits>

#include "attn.cuh"
#include "half_mma.cuh"

namespace mq {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnit = kStep * kWarps;   // tokens of a unit
constexpr int kStages = 2;              // steps in flight per warp (a power of two)
constexpr int kJoin = 4;                // what a second run costs a CTA, in units

template <int NT>
constexpr int ctas_per_sm() { return NT == 1 ? 3 : 2; }

// Rows, partials and counters: the workspace of a grid.
__host__ __device__ constexpr int slot_floats(int nt, int D) { return 8 * nt * (D + 2); }

// Transpose of an 8 x 8 matrix of 16-bit elements held by the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ int units_of(const Seq& s, const FastDiv& G, int window, int r0, int rows) {
    int begin, end;
    range_of(s, G, window, r0, rows, begin, end);
    return max(1, (end - begin + kUnit - 1) / kUnit);  // one for rows that see nothing: they are written too
}
// Units of one cache head of a sequence.
__device__ __forceinline__ int64_t seq_units(const Seq& s, const FastDiv& G, int window, int rows) {
    int64_t n = 0;
    for (int r0 = 0; r0 < s.nq * G.d; r0 += rows) n += units_of(s, G, window, r0, rows);
    return n;
}

// A CTA's part of one run of units: (sequence, cache head, tile of rows), pieces [piece,
// piece + take) of its `units`, its first unit's number, and its tokens.
struct Run {
    Seq s;
    int b, h, r0, piece, units, take, begin, end;
    int64_t unit0;
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
// SPLIT: attn_rows.cu's kernel has some of the sequences (attn.cuh).
template <int D, int NT, bool F16, bool SPLIT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm<NT>()) k_attn(const AttnParams p) {
    constexpr int R = 8 * NT;           // rows of a tile
    constexpr int REC = 18 * D;         // bytes of a record
    constexpr int KS = D / 16;          // products of 16 d per token tile; also d tiles of the output
    constexpr int RS = D + 4;           // floats of a merged row in shared memory
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[kWarps][kStages];
    __shared__ float sm_m[kWarps][R], sm_l[kWarps][R];
    __shared__ int64_t red[kWarps], red2[kWarps];
    __shared__ int64_t found[2];
    __shared__ int counts[kWarps];
    __shared__ int last_part;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int H = p.cache.heads;
    const FastDiv& G = p.by_group;
    if (tid < kWarps * kStages) mbar_init(&full[0][0] + tid, 2);  // the two records' lanes
    mbar_fence_init();
    // With split, attn_rows.cu's kernel is the one before. It waited before it let this one start, so
    // what this one reads is there, and the two may run side by side; the first CTA waits for it at
    // its end, and lets the next kernel start no sooner.
    if constexpr (!SPLIT) {
        griddep_wait();
        griddep_launch();
    }
    auto leave = [&] {
        if (SPLIT && blockIdx.x == 0) {
            griddep_wait();
            griddep_launch();
        }
    };

    // The CTA's work. CTA w takes the w-th equal share of all units, in order; or, with fewer
    // runs than CTAs, every run is cut into equal pieces of at most q units, one CTA each. Then no
    // CTA joins two runs, which costs it about as much as kJoin units (16 sequences of up to
    // 8192 tokens: 33.2 us by shares, 31.8 by pieces; 4 of 131072, where pieces waste 5 of 74
    // units: 126.6 and 132.7).
    Seq own = tid < p.B ? seq_of(p, tid, blockIdx.x == 0) : Seq{0, 0, 0};
    int64_t all_work = 0;
    if constexpr (SPLIT) {
        all_work = rows_work(own, p);
        for (int b = tid + kThreads; b < p.B; b += kThreads) all_work += rows_work(seq_of(p, b, false), p);
        all_work = warp_sum(all_work);
        if (lane == 0) red[warp] = all_work;
        __syncthreads();
        all_work = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) all_work += red[w];
        __syncthreads();
    }
    // a sequence; without query tokens if the other kernel has it
    auto left = [&](Seq s) {
        if (SPLIT && takes_rows(s, p, all_work)) s.nq = 0;
        return s;
    };
    own = left(own);
    const int64_t own_units = seq_units(own, G, p.window, R) * H;
    int64_t mine = own_units, rmine = (int64_t)((own.nq * G.d + R - 1) / R) * H;
    for (int b = tid + kThreads; b < p.B; b += kThreads) {
        const Seq s = left(seq_of(p, b, blockIdx.x == 0));
        mine += seq_units(s, G, p.window, R) * H;
        rmine += (int64_t)((s.nq * G.d + R - 1) / R) * H;
    }
    mine = warp_sum(mine);
    rmine = warp_sum(rmine);
    if (lane == 0) {
        red[warp] = mine;
        red2[warp] = rmine;
    }
    if (tid == 0) found[0] = -1;
    __syncthreads();
    int64_t total = 0, runs = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        total += red[w];
        runs += red2[w];
    }
    if (total == 0) {
        leave();
        return;
    }
    const int grid = (int)gridDim.x;
    const bool fits = total < (1 << 30);  // 32-bit divisions
    const int64_t share = fits ? (int)p.by_grid.div((uint32_t)total + grid - 1) : (total + grid - 1) / grid;
    auto pieces_of = [&](const Seq& s, int q) {  // of one cache head
        int n = 0;
        for (int r0 = 0; r0 < s.nq * G.d; r0 += R) n += (units_of(s, G, p.window, r0, R) + q - 1) / q;
        return n;
    };
    bool cut = false;
    int q = 1;
    if (fits && p.B <= kThreads && runs < grid) {
        // a run's last piece is half empty on average
        const int room = grid - (int)runs / 2;
        q = ((int)total + room - 1) / room;
        if (q <= (int)share + kJoin) {
            const int n = __reduce_add_sync(0xffffffffu, pieces_of(own, q) * H);
            if (lane == 0) counts[warp] = n;
            __syncthreads();
            cut = counts[0] + counts[1] + counts[2] + counts[3] <= grid;
        }
    }
    const int64_t at0 = cut ? blockIdx.x : share * blockIdx.x;  // the CTA's first piece or unit
    int64_t u0, u1;
    const int64_t own_n = cut ? pieces_of(own, q) * H : own_units;
    {
        int64_t base = 0;
        for (int b0 = 0; b0 < p.B; b0 += kThreads) {
            const int b = b0 + tid;
            const int64_t n = b0 == 0 ? own_n : b < p.B ? seq_units(left(seq_of(p, b, false)), G, p.window, R) * H : 0;
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
            if (n > 0 && at0 >= x - n && at0 < x) {
                found[0] = b;
                found[1] = x - n;
            }
            base = all;
            if (at0 < base) break;
        }
        __syncthreads();
    }
    if (found[0] < 0) {  // past the last piece or unit
        leave();
        return;
    }
    Run c;
    c.b = (int)found[0];
    c.s = seq_of(p, c.b, false);
    c.r0 = 0;
    int cut_parts = 0;  // pieces of the run, and the CTA of its first one
    int64_t cut_first = 0;
    {
        const int64_t per = cut ? pieces_of(c.s, q) : seq_units(c.s, G, p.window, R);
        int64_t off = at0 - found[1];
        c.h = fits ? (int)off / (int)per : (int)(off / per);
        off -= c.h * per;
        int n;
        while (true) {
            n = units_of(c.s, G, p.window, c.r0, R);
            const int m = cut ? (n + q - 1) / q : n;
            if (off < m) break;
            off -= m;
            c.r0 += R;
        }
        if (cut) {
            const int i = (int)off;
            cut_parts = (n + q - 1) / q;
            cut_first = blockIdx.x - i;
            const int base = n / cut_parts, rest = n - base * cut_parts;
            c.piece = i * base + min(i, rest);
            u0 = c.piece;
            u1 = u0 + base + (i < rest);
        } else {
            c.piece = (int)off;
            u0 = at0;
            u1 = min(u0 + share, total);
        }
        c.unit0 = u0 - c.piece;
    }
    auto measure = [&](Run& r, int64_t u) {
        range_of(r.s, G, p.window, r.r0, R, r.begin, r.end);
        r.units = max(1, (r.end - r.begin + kUnit - 1) / kUnit);
        r.take = (int)min((int64_t)(r.units - r.piece), u1 - u);
    };
    measure(c, u0);

    // This warp's ring. Step i of a run's part covers tokens first + i * kUnit ... + kStep, one
    // record per lane of a pair; the records' addresses are looked up 16 steps at a time.
    uint8_t* ring = smem + warp * (kStages * 2 * REC);
    uint32_t taken = 0, given = 0;       // steps taken from the ring, and issued into it
    const uint8_t* src = nullptr;        // lane 2 i + r: record r of step 16 k + i (null: not there)
    bool holes = false;                  // a page of the run is not there (every lane knows)
    bool alive = true;                   // false after a wait that gave up
    auto first_of = [&](const Run& r) { return r.begin + r.piece * kUnit + warp * kStep; };
    auto steps_of = [&](const Run& r) {
        const int first = first_of(r);
        return first < r.end ? min(r.take, (r.end - first + kUnit - 1) / kUnit) : 0;
    };
    auto record = [&](const Run& r, int j) -> const uint8_t* {
        const int pg = (int)p.by_page.div(j);
        const int page = ld_prior(p.table + r.b * p.table_stride + pg);
        if (page < 0 || page >= p.cache.num_pages) return nullptr;
        return p.cache.pages + (((int64_t)page * H + r.h) * (p.cache.page_size >> 4) + ((j - pg * p.cache.page_size) >> 4)) * REC;
    };
    auto issue = [&](const Run& r, int step, int steps) {
        const int turn = step & 15;
        if (turn == 0) {
            const int i = step + (lane >> 1), j = first_of(r) + i * kUnit + 16 * (lane & 1);
            const bool want = i < steps && j < r.end;
            src = want ? record(r, j) : nullptr;
            if (want && !src) report_index(p.err);
            holes = __any_sync(0xffffffffu, want && !src) || (step > 0 && holes);
        }
        if ((lane >> 1) == turn) {
            const uint32_t to = given % kStages;
            uint64_t* bar = &full[warp][to];
            if (src) {
                mbar_arrive_expect_tx(bar, REC);
                bulk_load(ring + (2 * to + (lane & 1)) * REC, src, REC, bar);
            } else {
                mbar_arrive(bar);
            }
        }
        ++given;
    };
    int steps = steps_of(c);
#pragma unroll
    for (int i = 0; i < kStages; ++i)
        if (i < steps) issue(c, i, steps);

    float* merge = reinterpret_cast<float*>(smem + kWarps * kStages * 2 * REC);
    int64_t u = u0;
    while (true) {
        // ---------------------------------------------------------------- one run, or this CTA's part of it
        const Seq& s = c.s;
        const int h = c.h, r0 = c.r0, end = c.end;
        const float gk = p.cache.k_scale ? ld_prior(p.cache.k_scale + h) : 1.0f;
        const float gv = p.cache.v_scale ? ld_prior(p.cache.v_scale + h) : 1.0f;
        const int first = first_of(c);

        // this lane's query elements (row 8 nt + g, d = t D/4 ...) as the second operand, and
        // the scale and limits of its score columns (rows 8 nt + 2t, + 2t + 1)
        uint32_t qf[NT][KS][2];
        float qs[NT][2];
        int lim[NT][2];
        float m[NT][2], l[NT][2];
        float ref[NT][2];    // m - kShift (0 while m is -inf)
        float limit[NT][2];  // the unscaled score that raises m
        float o[KS][NT][4];
        int lim_min = INT_MAX;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = r0 + 8 * nt + g, rows = s.nq * G.d;
            float inv = 0.0f;
#pragma unroll
            for (int j = 0; j < KS; ++j) qf[nt][j][0] = qf[nt][j][1] = 0u;
            if (row < rows) {
                const int qi = (int)G.div(row);
                const uint4* src = reinterpret_cast<const uint4*>(p.q.p + (int64_t)(s.row0 + qi) * p.q.st +
                                                                  (int64_t)(h * G.d + row - qi * G.d) * p.q.sh + t * (D / 4));
#pragma unroll
                for (int i = 0; i < KS / 2; ++i) {
                    const uint4 v = ld_prior(src + i);
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
            const float z = fmaxf(inv * (gk * fabsf(p.scale)), FLT_MIN);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                qs[nt][c] = __shfl_sync(0xffffffffu, z, 4 * (2 * t + c));
                const int r = r0 + 8 * nt + 2 * t + c;
                lim[nt][c] = r < rows ? s.len - s.nq + (int)G.div(r) + 1 : INT_MAX;
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
        const int lo_min = p.window > 0 ? s.len - s.nq + (int)G.div(r0) + 1 - p.window : 0;
        // steps [full0, full1): every row sees every token
        const int full0 = lo_max > first ? (lo_max - first + kUnit - 1) / kUnit : 0;
        const int full1 = holes || lim_min < first + kStep ? 0 : (min(lim_min, end) - kStep - first) / kUnit + 1;

        for (int step = 0; step < steps; ++step) {
            const uint32_t at = taken % kStages;
            // the warp decides together; after a wait that gave up (reported) nothing is issued
            // or waited for any more
            const uint32_t parity = (taken / kStages) & 1u;
            if (__any_sync(0xffffffffu, !mbar_try_wait(&full[warp][at], parity)) && alive)
                alive = __all_sync(0xffffffffu, mbar_wait_err(&full[warp][at], parity, p.err));
            ++taken;
            const uint8_t* buf = ring + at * (2 * REC);
            const int j0 = first + step * kUnit;
            const bool whole = step >= full0 && step < full1 && !holes;
            // records that are not there: looked up again, since nothing but a bad page comes here
            uint32_t lost = 0;
            if (holes)
                for (int r = 0; r < 2; ++r)
                    if (j0 + 16 * r < end && !record(c, j0 + 16 * r)) lost |= 1u << r;

            // ---- scores: the two records side by side, as independent chains of products
            float z[2][NT][4];
            uint32_t ka[2][KS / 4], kb[2][KS / 4], ka2[2][KS / 4], kb2[2][KS / 4];  // tokens g and g + 8: low and high half of the lane's codes
            __half2 sa[2][2], sb[2][2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint8_t* rec = buf + r * REC;
                uint32_t s0, s1;
                if constexpr (D == 128) {
                    const uint4 x = *reinterpret_cast<const uint4*>(rec + g * 64 + t * 16);
                    const uint4 y = *reinterpret_cast<const uint4*>(rec + 512 + g * 64 + t * 16);
                    ka[r][0] = x.x, ka[r][1] = x.y, ka2[r][0] = x.z, ka2[r][1] = x.w;
                    kb[r][0] = y.x, kb[r][1] = y.y, kb2[r][0] = y.z, kb2[r][1] = y.w;
                    e4m3x4_half(*reinterpret_cast<const uint32_t*>(rec + 16 * D + lane * 4), s0, s1);
                    sa[r][0] = low2(s0), sa[r][1] = high2(s0), sb[r][0] = low2(s1), sb[r][1] = high2(s1);
                } else {
                    const uint2 x = *reinterpret_cast<const uint2*>(rec + g * 32 + t * 8);
                    const uint2 y = *reinterpret_cast<const uint2*>(rec + 256 + g * 32 + t * 8);
                    ka[r][0] = x.x, ka2[r][0] = x.y;
                    kb[r][0] = y.x, kb2[r][0] = y.y;
                    // a lane pair's two scales each lie in one word
                    e4m3x4_half(*reinterpret_cast<const uint32_t*>(rec + 16 * D + (lane >> 1) * 4), s0, s1);
                    const uint32_t mine2 = (lane & 1) ? s1 : s0;
                    sa[r][0] = sa[r][1] = low2(mine2), sb[r][0] = sb[r][1] = high2(mine2);
                }
            }
#pragma unroll
            for (int w = 0; w < KS / 2; ++w) {
                constexpr int HALF = KS / 4;
                uint32_t x[2][4], y[2][4];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    e2m1x8_half(w < HALF ? ka[r][w] : ka2[r][w - HALF], x[r]);
                    e2m1x8_half(w < HALF ? kb[r][w] : kb2[r][w - HALF], y[r]);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const __half2 fa = sa[r][w / HALF], fb = sb[r][w / HALF];
                        const uint32_t a[4] = {mul_h2(x[r][2 * i], fa), mul_h2(y[r][2 * i], fb), mul_h2(x[r][2 * i + 1], fa),
                                               mul_h2(y[r][2 * i + 1], fb)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (w == 0 && i == 0)
                                mma_f16_first(z[r][nt], a, qf[nt][0][0], qf[nt][0][1]);
                            else
                                mma_f16(z[r][nt], a, qf[nt][2 * w + i][0], qf[nt][2 * w + i][1]);
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
                const __half2 f[4] = {low2(sab), high2(sab), low2(scd), high2(scd)};  // tokens 2t, 2t+1, 2t+8, 2t+9
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
            if (step + kStages < steps && alive) issue(c, step + kStages, steps);
        }

        // the next run's first copies fly while this one is joined
        u += c.take;
        Run nx = c;
        int nsteps = 0;
        if (u < u1) {
            nx.unit0 += nx.units;
            nx.piece = 0;
            nx.r0 += R;
            if (nx.r0 >= nx.s.nq * G.d) {
                nx.r0 = 0;
                if (++nx.h == H) {
                    nx.h = 0;
                    do nx.s = left(seq_of(p, ++nx.b, false));
                    while (nx.s.nq == 0);
                }
            }
            measure(nx, u);
            nsteps = steps_of(nx);
#pragma unroll
            for (int i = 0; i < kStages; ++i)
                if (i < nsteps && alive) issue(nx, i, nsteps);
        }

        // ---------------------------------------------------------------- join the warps
        // o[j][.][c] is d = g D/8 + 2 j + (c >> 1). A merged row lies as [j][g][2], RS floats.
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
        __syncthreads();
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
                    dst[8 * j] = make_float2(o[j][nt][c] * f, o[j][nt][c + 2] * f);
            }
        __syncthreads();
        const int rows = min(R, s.nq * G.d - r0);
        const int64_t w_first = cut ? cut_first : c.unit0 / share;
        const int parts = cut ? cut_parts : (int)((c.unit0 + c.units - 1) / share - w_first + 1);
        constexpr int PAIRS = D / 2, RPP = kThreads / PAIRS;  // float2s of a row, rows per pass
        const int pi = tid % PAIRS;                           // output elements 2 pi, 2 pi + 1
        const int pg = pi / KS, pj = pi % KS;
        if (parts > 1) {
            // slot 0 of a CTA: a run that an earlier CTA began; slot 1: one that it begins itself
            const int64_t slot = 2 * (int64_t)blockIdx.x + (c.unit0 < u0 ? 0 : 1);
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
                        sum += sm_l[w][row] * (sm_m[w][row] == -INFINITY ? 0.0f : ex2(sm_m[w][row] - top));
                    dst[R * D + row] = top;
                    dst[R * D + R + row] = sum;
                }
            }
            __syncthreads();
            if (tid == 0) {
                // release what the CTA wrote, acquire what the other parts' CTAs released
                int old;
                asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(p.counters + w_first) : "memory");
                last_part = old == parts - 1;
                if (last_part) p.counters[w_first] = 0;
            }
            __syncthreads();
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
                    sum += sm_l[w][row] * (sm_m[w][row] == -INFINITY ? 0.0f : ex2(sm_m[w][row] - top));
                }
                const int qi = (int)G.div(r0 + row), hq = h * G.d + r0 + row - qi * G.d;
                const int64_t tok = s.row0 + qi;
                const float inv = sum == 0.0f ? 0.0f : gv / sum;
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
            // the first 32 parts' maxima and sums, read together
            auto stat = [&](int i, int row) { return (i ? parts1 + (int64_t)2 * i * SLOT : part0) + R * D + row; };
            for (int row = warp; row < rows; row += kWarps) {
                const float m0 = lane < parts ? __ldcg(stat(lane, row)) : -INFINITY;
                const float l0 = lane < parts ? __ldcg(stat(lane, row) + R) : 0.0f;
                float top = m0;
                for (int i = lane + 32; i < parts; i += 32) top = fmaxf(top, __ldcg(stat(i, row)));
                top = warp_max(top);
                const float f0 = m0 == -INFINITY ? 0.0f : ex2(m0 - top);
                float sum = l0 * f0;
                if (lane < parts) fac[lane * R + row] = f0;
                for (int i = lane + 32; i < parts; i += 32) {
                    const float mw = __ldcg(stat(i, row)), f = mw == -INFINITY ? 0.0f : ex2(mw - top);
                    fac[i * R + row] = f;
                    sum = __fmaf_rn(__ldcg(stat(i, row) + R), f, sum);
                }
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                if (lane == 0) {
                    sm_l[0][row] = sum;
                    sm_m[0][row] = top;
                }
            }
            __syncthreads();
#pragma unroll 2
            for (int i = tid; i < rows * QUADS; i += kThreads) {
                const int row = i / QUADS, d = 4 * (i - row * QUADS);
                float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (int w = 0; w < parts; w += 8) {
                    float4 v[8];
                    float f[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const bool on = w + x < parts;
                        const float* from = (w + x ? parts1 + (int64_t)2 * (w + x) * SLOT : part0) + row * D + d;
                        v[x] = on ? __ldcg(reinterpret_cast<const float4*>(from)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        f[x] = on ? fac[(w + x) * R + row] : 0.0f;
                    }
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        a.x = __fmaf_rn(v[x].x, f[x], a.x);
                        a.y = __fmaf_rn(v[x].y, f[x], a.y);
                        a.z = __fmaf_rn(v[x].z, f[x], a.z);
                        a.w = __fmaf_rn(v[x].w, f[x], a.w);
                    }
                }
                const int qi = (int)G.div(r0 + row), hq = h * G.d + r0 + row - qi * G.d;
                const int64_t tok = s.row0 + qi;
                const float sum = sm_l[0][row], inv = sum == 0.0f ? 0.0f : gv / sum;
                *reinterpret_cast<uint2*>(p.o.p + tok * p.o.st + hq * p.o.sh + d) =
                    make_uint2(narrow2<F16>(a.x * inv, a.y * inv), narrow2<F16>(a.z * inv, a.w * inv));
                if (p.lse && d == 0) p.lse[tok * p.q.heads + hq] = lse_of(sm_m[0][row], sum);
            }
        }
        // ---------------------------------------------------------------- the next run
        if (u >= u1) break;
        c = nx;
        steps = nsteps;
        __syncthreads();  // the merge's memory is free again
    }
    // a warp that gave up leaves its last copies their (bounded) time
    if (!alive)
        for (uint32_t i = 1; i <= min(given, (uint32_t)kStages); ++i)
            mbar_wait_err(&full[warp][(given - i) % kStages], ((given - i) / kStages) & 1u, p.err);
    leave();
}

// Rings, then the memory of a merge: the warps' rows, or a run's factors (at most one part a CTA).
template <int D, int NT>
size_t smem_bytes(int grid) {
    const size_t rows = (size_t)kWarps * 8 * NT * (D + 4) * 4, factors = (size_t)grid * 8 * NT * 4;
    return (size_t)kWarps * kStages * 2 * 18 * D + (rows > factors ? rows : factors);
}

template <int D, int NT, bool F16, bool SPLIT>
cudaError_t attn_kernel(const AttnParams& p, int grid, cudaStream_t s) {
    static std::atomic<bool> done[64];
    const size_t smem = smem_bytes<D, NT>(grid);
    const cudaError_t e = once_per_device(done, [smem] {
        return cudaFuncSetAttribute(k_attn<D, NT, F16, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(k_attn<D, NT, F16, SPLIT>, dim3(grid), dim3(kThreads), smem, s, 1, p);
}

template <int D, int NT, bool F16>
cudaError_t attn_of(const AttnParams& p, int grid, cudaStream_t s) {
    if constexpr (D == 128)
        if (p.split) return attn_kernel<D, NT, F16, true>(p, grid, s);
    return attn_kernel<D, NT, F16, false>(p, grid, s);
}

int grid_of(int nt) { return device_sms() * (nt == 1 ? ctas_per_sm<1>() : ctas_per_sm<2>()); }

// Eights of query rows that a CTA holds. More rows share a step's copies and conversions, up to what
// the registers hold; with few steps a CTA the shorter step wins. So 17 to 24 rows are one tile where
// the tables' capacity gives a CTA kLong units or more, and two of 16 below (us by 16 and by 24, 20
// rows of 8 cache heads: 8 sequences of up to 4001 tokens, ragged, 26.4 and 29.0; of 4001 tokens 36.3
// and 33.2; of 16384 97 and 81; of 65536 328 and 233); 25 to 32 rows are two of 16 (8 x 65536: 330
// and 435), more rows tiles of 24 (8 sequences of 512 rows: 157 and 143).
constexpr int kLong = 8;
int row_tiles(int64_t rows, bool many_units) { return rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 24 && many_units ? 3 : rows <= 32 ? 2 : 3; }

}  // namespace

// Counters first, in the same place for every shape: the partial sums of one must not fall on
// the counters of another that shares the workspace.
size_t attn_workspace(int q_heads, int kv_heads, int D, int max_q, size_t* partials_at) {
    const int64_t rows = (int64_t)(q_heads / kv_heads) * max_q;
    const int nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 3;  // what fewer rows need, fits too
    *partials_at = ((size_t)device_sms() * ctas_per_sm<1>() * sizeof(int) + 255) / 256 * 256;
    return *partials_at + (size_t)2 * grid_of(nt) * slot_floats(nt, D) * sizeof(float);
}

cudaError_t launch_attn(const AttnParams& p0, int D, int max_q, bool f16, cudaStream_t s, int* kernels) {
    AttnParams p = p0;
    p.by_group = FastDiv(p.q.heads / p.cache.heads);
    p.by_page = FastDiv(p.cache.page_size);
    p.scale *= 1.4426950408889634f;  // scores in powers of two
    const AttnPlan plan = attn_plan(p, D, max_q);
    const int64_t G = p.q.heads / p.cache.heads;
    const int64_t units = (int64_t)p.max_pages * p.cache.page_size / kUnit * p.B * p.cache.heads;
    const bool many_units = units >= (int64_t)kLong * grid_of(2);
    int nt = row_tiles(G * max_q, many_units);
    if (plan.rows) {
        p.split = plan.other;
        p.least = plan.least;
        p.even = (int64_t)kRowsWorth * device_sms();
        const cudaError_t e = launch_attn_rows(p, f16, s);
        if (e != cudaSuccess || !p.split) return e;
        *kernels = 2;
        if (plan.least == kRowsLeast) nt = std::min(nt, row_tiles(G, many_units));  // mostly single tokens are left
    }
    const int grid = grid_of(nt);
    p.by_grid = FastDiv(grid);
    if (D == 64) {
        if (nt == 1) return f16 ? attn_of<64, 1, true>(p, grid, s) : attn_of<64, 1, false>(p, grid, s);
        if (nt == 3) return f16 ? attn_of<64, 3, true>(p, grid, s) : attn_of<64, 3, false>(p, grid, s);
        return f16 ? attn_of<64, 2, true>(p, grid, s) : attn_of<64, 2, false>(p, grid, s);
    }
    if (nt == 1) return f16 ? attn_of<128, 1, true>(p, grid, s) : attn_of<128, 1, false>(p, grid, s);
    if (nt == 3) return f16 ? attn_of<128, 3, true>(p, grid, s) : attn_of<128, 3, false>(p, grid, s);
    return f16 ? attn_of<128, 2, true>(p, grid, s) : attn_of<128, 2, false>(p, grid, s);
}

}  // namespace mq
