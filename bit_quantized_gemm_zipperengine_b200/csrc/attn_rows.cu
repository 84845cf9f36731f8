// Attention over the NVFP4 cache for many query rows a cache head (prompts): the formula, the
// masks and the softmax reference of attn.cu, on tcgen05 with tensor-memory accumulators.
//
// What bounds it: the products, 4 D flops a row and seen token, and one exponential each (16
// a clock and SM, as long as the products of D = 128). 256 query rows (tokens times the
// query heads that share a cache head) share a conversion of the cache, where attn.cu's 24
// spend their time converting: 512 tokens of two sequences behind 8192, 32/8 heads: 162 us, 820
// TFLOP/s, against 599; a prompt of 4096: 178 against 1508 us.
//
// A CTA takes a tile of 256 rows, two operands of 128; the cached tokens pass in steps of 64:
//  - four warps convert: a record (16 tokens) each, codes and scales from global memory, a step
//    ahead in registers, to exact fp16 in shared memory (128-byte swizzle, two buffers);
//  - a warp for each operand issues its products from an elected lane: S = Q K^T (64 columns
//    of tensor memory) and O += P V (128 columns; V's tokens are rows in memory, so it is the
//    operand whose rows run fastest). One warp for both took 217 us: its waits and issues, a
//    hundred cycles each, were the longest chain of a step;
//  - four warps an operand hold a query row a thread: its maximum and sum need no shuffles. S is
//    free for the next step's scores as soon as it is in registers; P goes back in fp16 (two
//    buffers of 32 columns) and is read as an operand from there. O is rescaled in place when a
//    row's reference rises, which the slack of 2^8 makes rare.
// One such CTA fills an SM (512 columns of tensor memory, 128 KB). Two of 128 rows an SM took
// 190 us: every step was converted twice. What is left: a step takes 2400 cycles, its products 1024, the
// exponentials 1024; the rest is the latency of handing S and P over.
#include <algorithm>
#include <cfloat>
#include <climits>

#include "attn.cuh"
#include "half_mma.cuh"

namespace mq {

namespace {

constexpr int kD = 128;
constexpr int kRows = 128;   // query rows of an operand, one softmax thread each
constexpr int kGroups = 2;   // operands of a CTA
constexpr int kBlock = kGroups * kRows;
constexpr int kTile = kRowsStep;  // tokens of a step
static_assert(kBlock == kRowsTile);
// Warps: one a group that issues its products, four that convert, four a group for the query rows.
constexpr int kConvert = kGroups, kSoftmax = kConvert + 4;
constexpr int kThreads = 32 * (kSoftmax + 4 * kGroups);
constexpr int kQ = kRows * kD * 2, kOffK = kGroups * kQ, kKv = kTile * kD * 2, kOffV = kOffK + 2 * kKv;
constexpr int kSmem = kOffV + 2 * kKv;
constexpr uint32_t kCols = 256, kWeightCol = 64, kOutCol = 128;  // tensor memory of a group: S, P, P, O

// fp16 operands, fp32 accumulator: D format 1 (bits 4-5), A and B format 0, bit 16: B's
// rows run fastest, N >> 3 in bits 17-22, M >> 4 in bits 24-28.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_rows_fast) {
    return (1u << 4) | ((b_rows_fast ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// 16 columns of the warp's 32 lanes; complete after tmem_st_wait.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 operations an instruction.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ float2 parts_of(uint64_t v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
    uint64_t v;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}

// Byte of 16-byte piece c of row n in a [rows][64 elements] block with 128-byte swizzle.
__device__ __forceinline__ int swizzled(int n, int c) { return n * 128 + ((c ^ (n & 7)) << 4); }

// The CTA's tile, into work (its sequence, -1 for none; its number there): sequences in order, then
// tiles from the last rows on (they see most), then heads. One warp looks through up to 32
// sequences, all of them (with two barriers a round) through more.
template <bool SPLIT>
__device__ __forceinline__ void find_tile(const AttnParams& p, int* work, int64_t* sums) {
    constexpr int kWarps = kThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool few = p.B <= 32, first = blockIdx.x == 0;  // the first CTA reports what is out of range
    if (few && warp > 0) return;
    const int stride = few ? 32 : kThreads;
    const Seq own = tid < p.B ? seq_of(p, tid, first) : Seq{0, 0, 0};
    int64_t all_work = 0;
    if constexpr (SPLIT) {
        all_work = rows_work(own, p);
        for (int b = tid + stride; b < p.B; b += stride) all_work += rows_work(seq_of(p, b, false), p);
        all_work = warp_sum(all_work);
        if (!few) {
            if (lane == 0) sums[warp] = all_work;
            __syncthreads();
            all_work = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) all_work += sums[w];
            __syncthreads();
        }
    }
    int64_t base = 0;
    for (int b0 = 0; b0 < p.B; b0 += stride) {
        const int b = b0 + tid;
        Seq s = b0 == 0 ? own : b < p.B ? seq_of(p, b, first) : Seq{0, 0, 0};
        if (SPLIT && !takes_rows(s, p, all_work)) s.nq = 0;
        const int64_t n = (int64_t)((s.nq * p.by_group.d + kBlock - 1) / kBlock) * p.cache.heads;
        int64_t x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        int64_t all = __shfl_sync(0xffffffffu, x, 31);
        x += base;
        if (!few) {
            if (lane == 31) sums[warp] = all;
            __syncthreads();
            all = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                x += w < warp ? sums[w] : 0;
                all += sums[w];
            }
            __syncthreads();
        }
        if (n > 0 && (int64_t)blockIdx.x >= x - n && (int64_t)blockIdx.x < x) {
            work[0] = b;
            work[1] = (int)(blockIdx.x - (x - n));
        }
        base += all;
        if (!first && (int64_t)blockIdx.x < base) break;
    }
}

// SPLIT: attn.cu's kernel has some of the sequences.
template <bool F16, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) k_attn_rows(const AttnParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint64_t q_full[kGroups], k_full[2], v_full[2];
    __shared__ uint64_t s_full[kGroups][2], s_free[kGroups], p_full[kGroups][2], done[kGroups][2];
    __shared__ uint32_t tmem_at;
    __shared__ int work[2];
    __shared__ int64_t sums[kThreads / 32];
    __shared__ volatile int lost[4][4];  // of step i at i % 4: written before its keys, read before step i + 4's keys
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int H = p.cache.heads;
    const FastDiv& G = p.by_group;
    if (tid == 0) work[0] = -1;
    if constexpr (SPLIT) {
        // a CTA without a tile leaves at once: the grid has one for every part that sequences may end in
        __syncthreads();
        griddep_wait();
        find_tile<SPLIT>(p, work, sums);
        __syncthreads();
        if (work[0] < 0) {
            griddep_launch();
            return;
        }
    }
    // Tensor memory before the next kernel may start: it could take what is left of it.
    if (warp == 0) {
        tmem_alloc(&tmem_at, kGroups * kCols);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(k_full + b, 128);
            mbar_init(v_full + b, 128);
        }
        for (int g = 0; g < kGroups; ++g) {
            mbar_init(q_full + g, kRows);
            mbar_init(s_free + g, kRows);
            for (int b = 0; b < 2; ++b) {
                mbar_init(&s_full[g][b], 1);
                mbar_init(&p_full[g][b], kRows);
                mbar_init(&done[g][b], 1);
            }
        }
    }
    mbar_fence_init();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_at;
    const bool placed = (smem_u32(smem) & 1023u) == 0;  // the swizzle repeats every 1024 bytes
    if constexpr (!SPLIT) griddep_wait();
    griddep_launch();

    if constexpr (!SPLIT) find_tile<SPLIT>(p, work, sums);
    if (!placed && tid == 0) report_index(p.err);
    __syncthreads();
    if (work[0] >= 0 && placed) {
        const Seq s = seq_of(p, work[0], false);
        const int rows = s.nq * G.d, tiles = (rows + kBlock - 1) / kBlock;
        const int h = work[1] % H, r0 = (tiles - 1 - work[1] / H) * kBlock;
        const int groups = rows - r0 > kRows ? kGroups : 1;  // the last tile may be short
        int begin, end;
        range_of(s, G, p.window, r0, kBlock, begin, end);
        const int steps = end > begin ? (end - begin + kTile - 1) / kTile : 0;

        // the warp decides together; after a wait that gave up (reported) its loop ends
        auto wait = [&](uint64_t* bar, int use) { return __all_sync(0xffffffffu, mbar_wait_err(bar, use & 1, p.err)) != 0; };

        if (warp >= kConvert && warp < kSoftmax) {
            // ------------------------------------------------------------ conversion
            const int r = warp - kConvert, n8 = lane & 7, t = lane >> 3;  // record of a step; token, piece
            const int lo_min = p.window > 0 ? s.len - s.nq + (int)G.div(r0) + 1 - p.window : 0;
            const int32_t* table = p.table + work[0] * p.table_stride;
            // a step's page number (looked at a step later, when it has arrived), and its record
            auto page_of = [&](int step) {
                const int j = begin + step * kTile + 16 * r;
                return step < steps && j < end ? ld_prior(table + p.by_page.div(j)) : 0;
            };
            auto record = [&](int step, int page) -> const uint8_t* {
                const int j = begin + step * kTile + 16 * r;
                if (step >= steps || j >= end) return nullptr;
                if (page < 0 || page >= p.cache.num_pages) {
                    report_index(p.err);
                    return nullptr;
                }
                const int in = j - (int)p.by_page.div(j) * p.cache.page_size;
                return p.cache.pages + (((int64_t)page * H + h) * (p.cache.page_size >> 4) + (in >> 4)) * (18 * kD);
            };
            // a lane's part of a record: keys of tokens n8 and n8 + 8, 32 elements each; values of
            // both tokens in groups t and t + 4
            uint4 kc[2];
            uint2 vc[4];
            uint32_t ks[2], vs[4];
            bool there = false;
            auto fetch = [&](const uint8_t* rec) {
                there = rec != nullptr;
                if (!there) {
                    kc[0] = kc[1] = make_uint4(0, 0, 0, 0);
                    vc[0] = vc[1] = vc[2] = vc[3] = make_uint2(0, 0);
                    ks[0] = ks[1] = vs[0] = vs[1] = vs[2] = vs[3] = 0;
                    return;
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int i = n8 + 8 * u;
                    kc[u] = ld_prior(reinterpret_cast<const uint4*>(rec + i * (kD / 2) + 16 * t));
                    ks[u] = ld_prior(reinterpret_cast<const uint16_t*>(rec + rec_kscale<kD>(i, 2 * t)));
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        vc[2 * u + w] = ld_prior(reinterpret_cast<const uint2*>(rec + rec_vcodes<kD>(i, t + 4 * w)));
                        vs[2 * u + w] = ld_prior(rec + rec_vscale<kD>(i, t + 4 * w));
                    }
                }
            };
            auto put = [&](uint8_t* dst, uint32_t codes, __half2 f) {
                uint32_t x[4];
                e2m1x8_half(codes, x);
                *reinterpret_cast<uint4*>(dst) = make_uint4(mul_h2(x[0], f), mul_h2(x[1], f), mul_h2(x[2], f), mul_h2(x[3], f));
            };
            fetch(record(0, page_of(0)));
            int next = page_of(1);
            for (int i = 0; i < steps; ++i) {
                const int b = i & 1, j0 = begin + i * kTile + 16 * r;
                uint4 k2[2] = {kc[0], kc[1]};
                uint2 v4[4] = {vc[0], vc[1], vc[2], vc[3]};
                const uint32_t ks2 = ks[0] | ks[1] << 16;
                uint32_t vs4 = vs[0] | vs[1] << 8 | vs[2] << 16 | vs[3] << 24;
                const bool here = there;
                fetch(record(i + 1, next));
                next = page_of(i + 2);
                // tokens that no row sees may hold anything: their values' scales become zero
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    if (j0 + n8 + 8 * u >= end || j0 + n8 + 8 * u < lo_min) vs4 &= u ? 0x0000FFFFu : 0xFFFF0000u;
                // the keys' buffer is free when the scores of step i - 2 are there, long before their weights
                if (i >= 2 && !(wait(&s_full[0][b], (i >> 1) - 1) && (groups == 1 || wait(&s_full[1][b], (i >> 1) - 1)))) break;
                uint8_t *K = smem + kOffK + b * kKv, *V = smem + kOffV + b * kKv;
                uint32_t f[2], g[2];
                e4m3x4_half(ks2, f[0], f[1]);
                e4m3x4_half(vs4, g[0], g[1]);
                if (lane == 0) lost[i & 3][r] = !here;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int n = 16 * r + n8 + 8 * u;
                    uint8_t* at = K + (t >> 1) * (kKv / 2);
                    const int c = (t & 1) * 4;
                    put(at + swizzled(n, c), k2[u].x, low2(f[u]));
                    put(at + swizzled(n, c + 1), k2[u].y, low2(f[u]));
                    put(at + swizzled(n, c + 2), k2[u].z, high2(f[u]));
                    put(at + swizzled(n, c + 3), k2[u].w, high2(f[u]));
                }
                fence_proxy_async_smem();
                mbar_arrive(k_full + b);
                if (i >= 2 && !(wait(&done[0][b], (i >> 1) - 1) && (groups == 1 || wait(&done[1][b], (i >> 1) - 1)))) break;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int n = 16 * r + n8 + 8 * u;
#pragma unroll
                    for (int w = 0; w < 2; ++w) {  // group t + 4 w: the w-th 64 elements
                        put(V + w * (kKv / 2) + swizzled(n, 2 * t), v4[2 * u + w].x, w ? high2(g[u]) : low2(g[u]));
                        put(V + w * (kKv / 2) + swizzled(n, 2 * t + 1), v4[2 * u + w].y, w ? high2(g[u]) : low2(g[u]));
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(v_full + b);
            }
        } else if (warp < groups) {
            // ------------------------------------------------------------ a group's products
            constexpr uint32_t iqk = idesc_f16(kRows, kTile, false), ipv = idesc_f16(kRows, kD, true);
            const int g = warp;
            const uint32_t sk = smem_u32(smem) + kOffK, sv = smem_u32(smem) + kOffV, sq = smem_u32(smem) + g * kQ, mine = tmem + g * kCols;
            auto scores = [&](int b) {
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kD / 16; ++k)
                        mma_ss(mine, smem_desc(sq + (k >> 2) * (kQ / 2) + (k & 3) * 32, 16, 1024, 2),
                               smem_desc(sk + b * kKv + (k >> 2) * (kKv / 2) + (k & 3) * 32, 16, 1024, 2), iqk, k > 0);
                    tc_commit(&s_full[g][b]);
                }
                __syncwarp();
            };
            int last = -1;  // the last step whose second product was issued
            if (steps > 0 && wait(k_full, 0) && wait(q_full + g, 0)) {
                tc_fence_after();
                scores(0);
                for (int i = 0; i < steps; ++i) {
                    const int b = i & 1;
                    if (i + 1 < steps) {  // the next scores run beside this step's softmax
                        if (!wait(k_full + (b ^ 1), (i + 1) >> 1) || !wait(s_free + g, i)) break;
                        tc_fence_after();
                        scores(b ^ 1);
                    }
                    if (!wait(v_full + b, i >> 1) || !wait(&p_full[g][b], i >> 1)) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k)
                            mma_ts(mine + kOutCol, mine + kWeightCol + b * (kTile / 2) + 8 * k,
                                   smem_desc(sv + b * kKv + k * 2048, kKv / 2, 1024, 2), ipv, i > 0 || k > 0);
                        tc_commit(&done[g][b]);
                    }
                    __syncwarp();
                    last = i;
                }
                if (last >= 0) wait(&done[g][last & 1], last >> 1);
            }
        } else if (warp >= kSoftmax && warp < kSoftmax + 4 * groups) {
            // ------------------------------------------------------------ a query row a thread
            const int g = (warp - kSoftmax) >> 2, in = 32 * (warp & 3) + lane, row = r0 + g * kRows + in;
            const bool on = row < rows;
            const int qi = on ? (int)G.div(row) : 0, hq = h * G.d + row - qi * G.d;
            const int64_t tok = s.row0 + qi;
            const float gk = p.cache.k_scale ? ld_prior(p.cache.k_scale + h) : 1.0f;
            const float gv = p.cache.v_scale ? ld_prior(p.cache.v_scale + h) : 1.0f;
            float inv = 1.0f;
            {
                const uint4* src = reinterpret_cast<const uint4*>(p.q.p + tok * p.q.st + hq * p.q.sh);
                auto piece = [&](int c) { return on ? ld_prior(src + c) : make_uint4(0, 0, 0, 0); };
                const uint32_t flip = p.scale < 0.0f ? 0x80008000u : 0u;  // the sign of the scale goes into the query: qs > 0
                float up = 1.0f;
                if constexpr (!F16) {
                    uint32_t a = 0;  // the largest element's bits, two at a time
#pragma unroll 4
                    for (int c = 0; c < 16; ++c) {
                        const uint4 v = piece(c);
                        a = __vmaxu2(a, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
                    }
                    const uint32_t ex = max(max(a & 0xFFFFu, a >> 16) >> 7, 15u);  // the largest element to [2^14, 2^15)
                    up = __uint_as_float((268u - ex) << 23);
                    inv = __uint_as_float((ex - 14u) << 23);
                }
#pragma unroll 4
                for (int c = 0; c < 16; ++c) {
                    const uint4 v = piece(c);
                    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        if constexpr (!F16) {
                            const float2 f = widen2<false>(w[x]);
                            w[x] = narrow2<true>(f.x * up, f.y * up);
                        }
                        w[x] ^= flip;
                    }
                    *reinterpret_cast<uint4*>(smem + g * kQ + (c >> 3) * (kQ / 2) + swizzled(in, c & 7)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(q_full + g);
            // never zero: a masked score is -inf before the scale
            const float qs = fmaxf(inv * (gk * fabsf(p.scale)), FLT_MIN);
            const int lim = on ? s.len - s.nq + qi + 1 : INT_MAX;
            const int lim_first = s.len - s.nq + (int)G.div(r0) + 1;
            const uint32_t mine = tmem + g * kCols + ((uint32_t)((warp & 3) * 32) << 16);  // this warp's lanes
            float m = -INFINITY, ref = 0.0f, limit = -INFINITY, l = 0.0f;
            bool alive = true;
            for (int i = 0; i < steps; ++i) {
                const int b = i & 1, j0 = begin + i * kTile;
                alive = wait(&s_full[g][b], i >> 1);
                if (!alive) break;
                tc_fence_after();
                float z[kTile];
                tmem_ld_chunks<kTile / 16>(mine, 0xF, z);
                tc_fence_before();
                mbar_arrive(s_free + g);
                const volatile int* no = lost[i & 3];
                const int gone = no[0] | no[1] << 1 | no[2] << 2 | no[3] << 3;
                const bool whole = gone == 0 && j0 + kTile <= min(lim_first, end) && (p.window == 0 || j0 >= end - p.window);
                if (!whole) {
                    const int hi = min(lim, end) - j0, lo = p.window > 0 ? lim - p.window - j0 : 0;
#pragma unroll
                    for (int c = 0; c < kTile; ++c)
                        if (c >= hi || c < lo || ((gone >> (c >> 4)) & 1)) z[c] = -INFINITY;
                }
                float tops[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    tops[x] = fmaxf(z[16 * x], z[16 * x + 1]);
#pragma unroll
                    for (int c = 2; c < 16; c += 2) tops[x] = max3(tops[x], z[16 * x + c], z[16 * x + c + 1]);
                }
                const float top = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]);
                if (__any_sync(0xffffffffu, top > limit)) {
                    const float mn = fmaxf(m, top * qs);
                    const float f = mn == -INFINITY ? 1.0f : ex2(m - mn);
                    m = mn;
                    ref = mn == -INFINITY ? 0.0f : mn - kShift;
                    limit = (mn + kSlack) / qs;
                    l *= f;
                    if (i > 0) {
                        alive = wait(&done[g][b ^ 1], (i - 1) >> 1);
                        if (!alive) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < kD; c += 16) {
                            uint32_t o[16];
                            tmem_ld16_issue(mine + kOutCol + c, o);
                            tmem_ld_wait16(o);
#pragma unroll
                            for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                            tmem_st16(mine + kOutCol + c, o);
                        }
                    }
                }
                if (i >= 2 && !(alive = wait(&done[g][b], (i >> 1) - 1))) break;
                tc_fence_after();
                const uint64_t q2 = pair_of(qs, qs), r2 = pair_of(-ref, -ref);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int c0 = 0; c0 < kTile; c0 += 32) {
                    uint32_t w[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float2 e = parts_of(fma_pair(pair_of(z[c0 + 2 * c], z[c0 + 2 * c + 1]), q2, r2));
                        const float x = ex2(e.x), y = ex2(e.y);
                        sum[c & 1] = add_pair(sum[c & 1], pair_of(x, y));
                        w[c] = narrow2<true>(x, y);
                    }
                    tmem_st16(mine + kWeightCol + b * (kTile / 2) + c0 / 2, w);
                }
                const float2 both = parts_of(add_pair(sum[0], sum[1]));
                l += both.x + both.y;
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&p_full[g][b]);
            }
            if (steps > 0 && alive) alive = wait(&done[g][(steps - 1) & 1], (steps - 1) >> 1);
            if (alive) {
                tc_fence_after();
                const float back = l == 0.0f ? 0.0f : gv / l;
                uint16_t* dst = p.o.p + tok * p.o.st + hq * p.o.sh;
#pragma unroll 1
                for (int c = 0; c < kD; c += 16) {
                    uint32_t o[16];
                    if (steps > 0) {
                        tmem_ld16_issue(mine + kOutCol + c, o);
                        tmem_ld_wait16(o);
                    } else {
#pragma unroll
                        for (int x = 0; x < 16; ++x) o[x] = 0u;
                    }
                    uint32_t w[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) w[x] = narrow2<F16>(__uint_as_float(o[2 * x]) * back, __uint_as_float(o[2 * x + 1]) * back);
                    if (on) {
                        *reinterpret_cast<uint4*>(dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
                        *reinterpret_cast<uint4*>(dst + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                    }
                }
                if (on && p.lse) p.lse[tok * p.q.heads + hq] = lse_of(m, l);
            }
            tc_fence_before();
        }
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, kGroups * kCols);
}

template <bool F16, bool SPLIT>
cudaError_t rows_of(const AttnParams& p, unsigned grid, cudaStream_t s) {
    static std::atomic<bool> done[64];
    const cudaError_t e = once_per_device(
        done, [] { return cudaFuncSetAttribute(k_attn_rows<F16, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem); });
    if (e != cudaSuccess) return e;
    return launch_pdl(k_attn_rows<F16, SPLIT>, dim3(grid), dim3(kThreads), kSmem, s, 1, p);
}

}  // namespace

// A CTA's step costs the same however many of its rows are there, about as much as attn.cu
// needs for 48 to 58 rows on one SM. So, where all sequences have as many query tokens: that many
// rows for each SM and for each CTA (us here and there: 16 x 8 tokens behind 4096, 64/8
// heads: 65 and 115; 32 x 16 and 32 x 8 behind 2048, 32/8 heads: 73 and 127, 71 and 67; 256
// and 128 tokens behind 8192: 160 and 173, 161 and 102). A sequence that fills the SMs by itself is
// never worse off here, however long it is. If none does, or the numbers of query tokens differ,
// the kernels share the call, sequence by sequence (us by the average of all sequences and by each
// one's own rows: a prompt of 2048 beside 15 single tokens behind 131072, 64/8 heads: 1930 and 545;
// beside one behind 2^20, 32/8 heads: 14500 and 296; 512 tokens beside 15 single ones, all behind
// 8192: 239 and 164; 16 x 8 tokens behind 4096, one of them behind 131072, 64/8 heads: 1820 and
// 250; 1000 sequences of 1 to 20 tokens behind 500: 1393 and 1038). A call that is all one kernel's
// pays up to 2 us, or 2%, for it (prompts of 1000 and 1024 tokens: 42 and 44; eight of 37 to 4000:
// 294 and 300; 32 x 16 behind 2048: 71.8 and 73.4).
AttnPlan attn_plan(const AttnParams& p, int D, int max_q) {
    const int64_t G = p.q.heads / p.cache.heads, H = p.cache.heads, rows = p.T * G;  // rows: of a cache head
    const int64_t fill = (int64_t)kRowsWorth * device_sms();
    const int64_t most = std::min<int64_t>(p.T, std::max<int64_t>(max_q, ((int64_t)p.T + p.B - 1) / p.B));  // query tokens of a sequence
    const AttnPlan other = {true, false, 0};
    if (D != kD || rows * H < fill || (rows / kRowsWorth + p.B) * H >= INT_MAX) return other;
    if (p.T != p.B * most) return most * G >= kRowsLeast ? AttnPlan{true, true, kRowsLeast} : other;
    const int64_t own = rows / p.B;
    if (own < kRowsWorth * ((own + kBlock - 1) / kBlock)) return other;
    return AttnPlan{p.B > 1 && own * H < fill, true, (int)std::min<int64_t>(own, kRowsLeast - 1)};
}

cudaError_t launch_attn_rows(const AttnParams& p, bool f16, cudaStream_t s) {
    const int64_t rows = (int64_t)p.T * (p.q.heads / p.cache.heads);
    // at most: every sequence that is taken ends in a part of a tile
    const int64_t taken = p.split ? std::min<int64_t>(p.B, rows / p.least) : p.B;
    const unsigned grid = (unsigned)((rows / kBlock + taken) * p.cache.heads);
    if (p.split) return f16 ? rows_of<true, true>(p, grid, s) : rows_of<false, true>(p, grid, s);
    return f16 ? rows_of<true, false>(p, grid, s) : rows_of<false, false>(p, grid, s);
}

}  // namespace mq
