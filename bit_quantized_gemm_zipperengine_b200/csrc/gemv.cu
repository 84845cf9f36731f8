// Products of a few tokens of 16-bit activations with the packed NVFP4 weight:
//   Y[m,n] = rn(g_w * sum_k x[m,k] (wh[n,k] + [block selected] rh[n,k])),  wh = val * dec(sf).
//
// What bounds it: the weight's bytes (9/16 a weight, 2304 a residual block), read once.
//
// The work of 64 weight rows is a list of steps: 128 columns of the base each, then two
// residual blocks each (a block row's blocks lie one behind the other). In both a lane of
// a warp takes 32 adjacent columns of its rows, at a column of its own, which a product's
// free order of k allows; so a residual step is as dense as a base step. A step's codes
// (4 KB: one TMA box of 64 bytes x 64 rows, or two packed blocks by one bulk copy) and scales (1 KB, one
// bulk copy) go to the warp's own ring in shared memory. Steps are this short so that 16
// warps fit an SM: with twice the columns and half the warps the waits of a step show
// (28672 x 8192, one token: 45.1 us against TODO).
//
// The weights are the 16-row operand of fp16 tensor-core products (val * dec(sf) is exact
// in fp16), eight tokens the other one. bf16 activations are scaled by a power of two per
// token and step to fit fp16 (what falls below is under 2^-39 of the step's largest), and the
// step's fp32 sums scaled back.
//
// The steps of a row tile are dealt to the warps of a cluster of S CTAs, S so that the CTAs
// about fill the GPU; the warps' sums are added in their order through shared memory, then
// the CTAs' through the cluster's.
#include <algorithm>

#include "half_mma.cuh"
#include "ops.cuh"

namespace mq {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 2;
constexpr int kRows = 64;              // weight rows of a tile (a block row)
constexpr int kCols = 128;             // base columns of a step
constexpr int kCodes = kRows * kCols / 2;
constexpr int kStage = kCodes + 1024;  // codes, then two 512-byte scale chunks
constexpr int kPitch = kRows + 4;      // floats of a token's row in the sums

template <int NT>
constexpr int ctas_per_sm() { return NT == 1 ? 4 : 3; }

template <int NT>
constexpr size_t smem_bytes() { return (size_t)kWarps * (kStages * kStage + NT * 2048 + kStages * 8); }

template <int NT, bool F16>
__global__ void __launch_bounds__(kThreads, ctas_per_sm<NT>()) k_gemv(const __grid_constant__ CUtensorMap tw, const GemvParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t(*full)[kStages] = reinterpret_cast<uint64_t(*)[kStages]>(smem + kWarps * (kStages * kStage + NT * 2048));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int tile = blockIdx.y, S = gridDim.x, rank = blockIdx.x, KC = p.K / 64;
    if (tid < kWarps * kStages) mbar_init(&full[0][0] + tid, 1);
    mbar_fence_init();
    if (tid == 0) tma_prefetch_desc(&tw);
    __syncthreads();
    if (!p.w_ready) {
        griddep_wait();
        griddep_launch();
    }
    const int nbase = p.base ? (KC + 1) / 2 : 0, step0 = rank * kWarps + warp, stride = S * kWarps;
    uint8_t* ring = smem + warp * (kStages * kStage);
    uint8_t* frag = smem + kWarps * kStages * kStage + warp * (NT * 2048);  // this warp's activations as fp16 operands
    int res0 = 0, res1 = 0;

    auto issue = [&](int i) {
        if (lane == 0) {
            const int step = step0 + i * stride;
            uint8_t* dst = ring + (i % kStages) * kStage;
            uint64_t* bar = &full[warp][i % kStages];
            if (step < nbase) {
                const uint32_t sf = (uint32_t)min(2, KC - 2 * step) * 512;
                mbar_arrive_expect_tx(bar, kCodes + sf);
                tma_load_2d(dst, &tw, bar, step * (kCols / 2), tile * kRows);
                bulk_load(dst + kCodes, p.sf + ((int64_t)(tile >> 1) * KC + 2 * step) * 512, sf, bar);
            } else {
                const int e = res0 + 2 * (step - nbase);
                const uint32_t n = (uint32_t)min(2, res1 - e);
                mbar_arrive_expect_tx(bar, n * 2560);
                bulk_load(dst, p.blk_codes + (int64_t)e * 2048, n * 2048, bar);
                bulk_load(dst + kCodes, p.blk_sf + (int64_t)e * 512, n * 512, bar);
            }
        }
    };
    // the first base steps fly before the residual's extent is known
    int ahead = 0;
    while (ahead < kStages && step0 + ahead * stride < nbase) issue(ahead++);
    if (p.blk_codes) {
        res0 = __ldg(p.tile_ptr + tile);
        res1 = __ldg(p.tile_ptr + tile + 1);
    }
    const int total = nbase + (res1 - res0 + 1) / 2;
    const int steps = step0 < total ? (total - step0 + stride - 1) / stride : 0;
    while (ahead < min(kStages, steps)) issue(ahead++);
    // Column chunk c (0 or 1, 64 columns) of a step, -1 past the end.
    auto chunk_of = [&](int i, int c) {
        const int step = step0 + i * stride;
        if (step < nbase) return 2 * step + c < KC ? 2 * step + c : -1;
        const int e = res0 + 2 * (step - nbase) + c;
        return e < res1 ? __ldg(p.blk_kt + e) : -1;
    };
    const int half = lane >> 4, piece = lane & 15;  // of a pair of tokens, and of a token's 128 activations
    int kt = steps > 0 ? chunk_of(0, piece >> 3) : -1;
    // tokens past M are zeros, and stay
    for (int i = lane; i < NT * 128; i += 32) reinterpret_cast<uint4*>(frag)[i] = make_uint4(0, 0, 0, 0);
    if (p.w_ready) {
        griddep_wait();
        griddep_launch();
    }

    uint4 xr[4 * NT];  // eight activations of tokens 2 i + half
    auto load_x = [&](int kt) {
        const uint16_t* src = p.X + 64 * (int64_t)kt + 8 * (piece & 7) + half * p.ldx;
#pragma unroll
        for (int i = 0; i < 4 * NT; ++i)
            if (2 * i < p.M)
                xr[i] = kt >= 0 && 2 * i + half < p.M ? __ldg(reinterpret_cast<const uint4*>(src + 2 * i * p.ldx))
                                                      : make_uint4(0, 0, 0, 0);
    };
    load_x(kt);

    float acc[4][NT][4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[rt][nt][c] = 0.0f;

    bool alive = true;
    for (int i = 0; i < steps; ++i) {
        const int step = step0 + i * stride;
        // columns of this lane's rows
        const bool valid = step < nbase ? 2 * step + (t >> 1) < KC : res0 + 2 * (step - nbase) + (t >> 1) < res1;
        // Activations to fp16, as operands: piece j (two products) of lane l's columns at slot
        // l ^ 2j, so that neither these stores nor the loads below meet in a bank.
        float back[NT][2] = {};  // scale of this lane's result columns, tokens 8 nt + 2t, + 1
#pragma unroll
        for (int m = 0; m < 4 * NT; ++m) {
            if (2 * m >= p.M) continue;
            uint32_t w[4] = {xr[m].x, xr[m].y, xr[m].z, xr[m].w};
            if constexpr (!F16) {
                // the largest element's bits (bf16, two at a time), over a token's 16 lanes
                uint32_t a = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                      __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
                uint32_t top = max(a & 0xFFFFu, a >> 16);
#pragma unroll
                for (int x = 1; x < 16; x <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, x));
                // the largest element to [2^14, 2^15)
                const uint32_t ex = max(top >> 7, 15u);
                const float up = __uint_as_float((268u - ex) << 23);
                const float d = __uint_as_float((ex - 14u) << 23);
                const float d0 = __shfl_sync(0xffffffffu, d, 0), d1 = __shfl_sync(0xffffffffu, d, 16);
                if ((m & 3) == t) {
                    back[m / 4][0] = d0;
                    back[m / 4][1] = d1;
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float2 f = widen2<false>(w[q]);
                    w[q] = narrow2<true>(f.x * up, f.y * up);
                }
            }
            // token 2m + half; its piece 4 t' + j
            const int j = piece & 3, slot = (4 * (2 * (m & 3) + half) + (piece >> 2)) ^ (2 * j);
            *reinterpret_cast<uint4*>(frag + (m / 4) * 2048 + j * 512 + slot * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        kt = i + 1 < steps ? chunk_of(i + 1, piece >> 3) : -1;
        load_x(kt);

        const uint32_t parity = (i / kStages) & 1u;
        // the warp decides together; after a wait that gave up (reported) nothing is issued or waited for
        if (__any_sync(0xffffffffu, !mbar_try_wait(&full[warp][i % kStages], parity)) && alive)
            alive = __all_sync(0xffffffffu, mbar_wait_err(&full[warp][i % kStages], parity, p.err));
        const uint8_t* buf = ring + (i % kStages) * kStage;
        // Scales of rows 16 rt + 8 hf + g in the lane's 32 columns (two groups): a 128-row chunk
        // holds row r's four at (r % 32) * 16 + (r / 32) * 4. Columns past the end may hold
        // anything: zero.
        uint32_t sc[4][2];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const uint2 w = *reinterpret_cast<const uint2*>(buf + kCodes + (t >> 1) * 512 + (16 * q + 8 * hf + g) * 16 + (tile & 1) * 8);
                const uint32_t both = __byte_perm(w.x, w.y, (t & 1) ? 0x7632 : 0x5410);
                e4m3x4_half(valid ? both : 0u, sc[q][hf], sc[q + 2][hf]);
            }
        float cc[4][NT][4];
        // 16 bytes of row g: rows of 64 bytes, or packed blocks (lane pair = half a block)
        const bool isb = step < nbase;
        const uint8_t* codes = isb ? buf + g * 64 + t * 16 : buf + (t >> 1) * 2048 + (t & 1) * 128 + g * 16;
        const int row8 = isb ? 512 : 256;  // eight rows further
        uint4 b[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int w = 0; w < 4; ++w) b[nt][w] = *reinterpret_cast<const uint4*>(frag + nt * 2048 + w * 512 + (lane ^ (2 * w)) * 16);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const uint4 a0 = *reinterpret_cast<const uint4*>(codes + (2 * rt) * row8);
            const uint4 a1 = *reinterpret_cast<const uint4*>(codes + (2 * rt + 1) * row8);
            const uint32_t w0[4] = {a0.x, a0.y, a0.z, a0.w}, w1[4] = {a1.x, a1.y, a1.z, a1.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t x[4], y[4];
                e2m1x8_half(w0[w], x);
                e2m1x8_half(w1[w], y);
                const __half2 f0 = w < 2 ? low2(sc[rt][0]) : high2(sc[rt][0]), f1 = w < 2 ? low2(sc[rt][1]) : high2(sc[rt][1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t a[4] = {mul_h2(x[2 * e], f0), mul_h2(y[2 * e], f1), mul_h2(x[2 * e + 1], f0),
                                           mul_h2(y[2 * e + 1], f1)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint32_t b0 = e ? b[nt][w].z : b[nt][w].x, b1 = e ? b[nt][w].w : b[nt][w].y;
                        if constexpr (F16) {
                            mma_f16(acc[rt][nt], a, b0, b1);
                        } else {
                            if (w == 0 && e == 0)
                                mma_f16_first(cc[rt][nt], a, b0, b1);
                            else
                                mma_f16(cc[rt][nt], a, b0, b1);
                        }
                    }
                }
            }
        }
        if constexpr (!F16)
#pragma unroll
            for (int rt = 0; rt < 4; ++rt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[rt][nt][c] = __fmaf_rn(cc[rt][nt][c], back[nt][c & 1], acc[rt][nt][c]);
        __syncwarp();
        if (i + kStages < steps && alive) issue(i + kStages);
    }
    if (!alive)  // the last copies get their (bounded) time
        for (int i = max(0, steps - kStages); i < steps; ++i)
            mbar_wait_err(&full[warp][i % kStages], (i / kStages) & 1u, p.err);

    // the warps' sums, then the CTAs', each in order
    __syncthreads();
    float* sums = reinterpret_cast<float*>(smem);  // [warp][token][kPitch]
#pragma unroll
    for (int rt = 0; rt < 4; ++rt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                sums[(warp * 8 * NT + 8 * nt + 2 * t + (c & 1)) * kPitch + 16 * rt + g + 8 * (c >> 1)] = acc[rt][nt][c];
    __syncthreads();
    const float gw = __ldg(p.g_w);
    float* mine = sums + kWarps * 8 * NT * kPitch;  // [token][kPitch], this CTA's
    for (int i = tid; i < kRows * p.M; i += kThreads) {
        const int m = i / kRows, n = i % kRows;
        float v = sums[m * kPitch + n];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v += sums[(w * 8 * NT + m) * kPitch + n];
        if (S == 1)
            p.Y[m * p.ldy + tile * kRows + n] = (uint16_t)narrow2<F16>(v * gw, 0.0f);
        else
            mine[m * kPitch + n] = v;
    }
    if (S > 1) {
        cluster_sync();
        for (int i = tid + rank * kThreads; i < kRows * p.M; i += S * kThreads) {
            const int m = i / kRows, n = i % kRows;
            float v = 0.0f;
            for (int r = 0; r < S; ++r) v += ld_dsmem_f32(mine + m * kPitch + n, r);
            p.Y[m * p.ldy + tile * kRows + n] = (uint16_t)narrow2<F16>(v * gw, 0.0f);
        }
        cluster_sync();  // no CTA leaves while another reads its sums
    }
}

template <int NT, bool F16>
cudaError_t gemv_of(const CUtensorMap& tw, const GemvParams& p, int S, cudaStream_t s) {
    static std::atomic<bool> done[64];
    const cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(k_gemv<NT, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<NT>());
    });
    if (e != cudaSuccess) return e;
    return launch_pdl_cluster(k_gemv<NT, F16>, dim3(S, p.N / kRows), dim3(kThreads), smem_bytes<NT>(), s, dim3(S, 1, 1), tw, p);
}

}  // namespace

cudaError_t launch_gemv(const CUtensorMap& tw, const GemvParams& p, bool f16, cudaStream_t s) {
    const int tiles = p.N / kRows, steps = (p.K / 64 + 1) / 2;
    // CTAs that fill the GPU once, none without a step for each of its warps
    const int S = std::max(1, std::min({8, (p.M <= 8 ? ctas_per_sm<1>() : ctas_per_sm<2>()) * device_sms() / tiles, steps / kWarps}));
    if (p.M <= 8) return f16 ? gemv_of<1, true>(tw, p, S, s) : gemv_of<1, false>(tw, p, S, s);
    return f16 ? gemv_of<2, true>(tw, p, S, s) : gemv_of<2, false>(tw, p, S, s);
}

}  // namespace mq
