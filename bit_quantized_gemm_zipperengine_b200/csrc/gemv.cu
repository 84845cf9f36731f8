// Products of a few tokens of 16-bit activations with the packed NVFP4 weight:
//   Y[m,n] = rn(g_w * sum_k x[m,k] (wh[n,k] + [block selected] rh[n,k])),  wh = val * dec(sf).
//
// What bounds it: the weight's bytes (9/16 a weight, 2304 a residual block), read once, and
// waits: 1 token through 28672 x 8192 with a tenth of the blocks takes 37.7 us (3.9 TB/s; half of
// the issue slots and no pipe more than 43% used), 16 through 5120 x 25600 30.0 us (14.3 for the
// copies alone), 1 through 4096 x 4096 8.4 us (4.4).
//
// The work of 64 weight rows is a list of steps: 256 columns of the base each, then four
// residual blocks each (a block row's blocks lie one behind the other). In both a lane of
// a warp takes 64 adjacent columns of its rows, at a column of its own, which a product's
// free order of k allows; so a residual step is as dense as a base step. Two warps share a step,
// each with half of every lane's columns: 16 warps an SM with 160 KB of rings. A step's codes
// (8 KB, one TMA box, 128-byte swizzle; or four packed blocks, one bulk copy) and scales
// (2 KB, one bulk copy) go to the pair's own ring in shared memory.
//
// The weights are the 16-row operand of fp16 tensor-core products (val * dec(sf) is exact
// in fp16), eight tokens the other one. A first kernel writes the activations as that operand: in
// fp16, bf16 ones scaled by a power of two per token (the largest element to [2^14, 2^15); what
// falls below is under 2^-39 of it), in the order in which lanes read them. Formed inside the
// products' kernel instead, by every CTA again, they cost it up to half of its time (16
// tokens through 14336 x 4096: 28.3 us against 17.8). The two kernels overlap: the weight's
// copies do not wait for the first one.
//
// The steps of a row tile are dealt to the pairs of a cluster of S CTAs, S so that the CTAs
// about fill the GPU; the warps' sums are added in their order through shared memory, then
// the CTAs' through the cluster's.
#include <algorithm>

#include "half_mma.cuh"
#include "ops.cuh"

namespace mq {

namespace {

// Pairs of warps of a CTA: what 128 and 168 registers a thread leave room for, two CTAs an SM.
template <int NT>
__host__ __device__ constexpr int pairs() { return NT == 1 ? 4 : 3; }
constexpr int kStages = 2;
constexpr int kRows = 64;              // weight rows of a tile (a block row)
constexpr int kCols = 256;             // base columns of a step
constexpr int kCodes = kRows * kCols / 2;
constexpr int kStage = kCodes + 2048;  // codes, then four 512-byte scale chunks
constexpr int kCtasPerSm = 2;
constexpr int kXThreads = 512, kXKeep = 4;  // of the operand's kernel: 16384 columns are read once
constexpr int kPitch = kRows + 4;      // floats of a token's row in the sums

template <int NT>
constexpr size_t smem_bytes() { return (size_t)pairs<NT>() * kStages * (kStage + 16); }

// Bytes of the operand: per 64-column chunk and eight tokens 1 KB, [piece of 8 columns][token], and
// every token's scale.
size_t operand_bytes(int nt, int K) { return (size_t)(K / 64) * nt * 1024 + 8 * nt * sizeof(float); }

// A CTA a token (those past M: zeros).
template <bool F16>
__global__ void __launch_bounds__(kXThreads) k_gemv_x(const uint16_t* X, int64_t ldx, int M, int NT, int K, uint8_t* out,
                                                      float* back) {
    __shared__ uint32_t tops[kXThreads / 32];
    const int m = blockIdx.x, pieces = K / 8;
    griddep_wait();
    griddep_launch();
    const uint4* src = reinterpret_cast<const uint4*>(X + m * ldx);
    uint4 keep[kXKeep];  // the first pieces, read once
#pragma unroll
    for (int i = 0; i < kXKeep; ++i) {
        const int c = threadIdx.x + i * kXThreads;
        keep[i] = m < M && c < pieces ? ld_prior(src + c) : make_uint4(0, 0, 0, 0);
    }
    uint32_t ex = 15u;
    if constexpr (!F16) {
        // the largest element's bits, two at a time
        auto top_of = [](const uint4& w) {
            return __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu), __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
        };
        uint32_t a = 0;
#pragma unroll
        for (int i = 0; i < kXKeep; ++i) a = __vmaxu2(a, top_of(keep[i]));
        if (m < M)
            for (int c = threadIdx.x + kXKeep * kXThreads; c < pieces; c += kXThreads) a = __vmaxu2(a, top_of(ld_prior(src + c)));
        const uint32_t top = __reduce_max_sync(0xffffffffu, max(a & 0xFFFFu, a >> 16));
        if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
        __syncthreads();
        for (int i = 0; i < kXThreads / 32; ++i) ex = max(ex, tops[i] >> 7);
    }
    const float up = __uint_as_float((268u - ex) << 23);
    auto put = [&](int c, const uint4& v) {
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
        if constexpr (!F16) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 f = widen2<false>(w[q]);
                w[q] = narrow2<true>(f.x * up, f.y * up);
            }
        }
        *reinterpret_cast<uint4*>(out + (((int64_t)(c >> 3) * NT + (m >> 3)) * 8 + (c & 7)) * 128 + (m & 7) * 16) =
            make_uint4(w[0], w[1], w[2], w[3]);
    };
#pragma unroll
    for (int i = 0; i < kXKeep; ++i) {
        const int c = threadIdx.x + i * kXThreads;
        if (c < pieces) put(c, keep[i]);
    }
    for (int c = threadIdx.x + kXKeep * kXThreads; c < pieces; c += kXThreads)
        put(c, m < M ? ld_prior(src + c) : make_uint4(0, 0, 0, 0));
    if (threadIdx.x == 0) back[m] = F16 ? 1.0f : __uint_as_float((ex - 14u) << 23);
}

template <int NT, bool F16>
__global__ void __launch_bounds__(64 * pairs<NT>(), kCtasPerSm) k_gemv(const __grid_constant__ CUtensorMap tw, const GemvParams p) {
    // The swizzle's pattern repeats every 1024 bytes. Without static shared memory the array
    // starts on such a boundary (checked below), and two CTAs fit an SM.
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr int kPairs = pairs<NT>(), kWarps = 2 * kPairs, kThreads = 32 * kWarps;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, pair = warp >> 1, h = warp & 1, g = lane >> 2, t = lane & 3;
    // per pair and stage: its copies have landed, both warps are done with it
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kPairs * kStages * kStage) + pair * (2 * kStages);
    uint64_t* empty = full + kStages;
    const int tile = blockIdx.y, S = gridDim.x, rank = blockIdx.x, KC = p.K / 64;
    if (h == 0 && lane < kStages) {
        mbar_init(full + lane, 1);
        mbar_init(empty + lane, 2);
    }
    mbar_fence_init();
    if (tid == 0) tma_prefetch_desc(&tw);
    __syncthreads();
    if (smem_u32(smem) & 1023u) {
        if (tid == 0) report_index(p.err);
        return;
    }
    const int nbase = p.base ? (KC + 3) / 4 : 0, step0 = rank * kPairs + pair, stride = S * kPairs;
    uint8_t* ring = smem + pair * (kStages * kStage);
    int res0 = 0, res1 = 0;

    auto issue = [&](int i) {
        if (h == 0 && lane == 0) {
            const int step = step0 + i * stride;
            uint8_t* dst = ring + (i % kStages) * kStage;
            uint64_t* bar = full + i % kStages;
            if (step < nbase) {
                const uint32_t sf = (uint32_t)min(4, KC - 4 * step) * 512;
                mbar_arrive_expect_tx(bar, kCodes + sf);
                tma_load_2d(dst, &tw, bar, step * (kCols / 2), tile * kRows);
                bulk_load(dst + kCodes, p.sf + ((int64_t)(tile >> 1) * KC + 4 * step) * 512, sf, bar);
            } else {
                const int e = res0 + 4 * (step - nbase);
                const uint32_t n = (uint32_t)min(4, res1 - e);
                mbar_arrive_expect_tx(bar, n * 2560);
                bulk_load(dst, p.blk_codes + (int64_t)e * 2048, n * 2048, bar);
                bulk_load(dst + kCodes, p.blk_sf + (int64_t)e * 512, n * 512, bar);
            }
        }
    };
    // The operand's kernel lets this one start after its own wait: all that came before it, the
    // weight's writers among them, has ended, so the weight is final (__ldg may read it). The
    // first base steps fly before the residual's extent is known.
    int ahead = 0;
    while (ahead < kStages && step0 + ahead * stride < nbase) issue(ahead++);
    if (p.blk_codes) {
        const int e0 = __ldg(p.tile_ptr + tile), e1 = __ldg(p.tile_ptr + tile + 1);
        res0 = min(max(e0, 0), p.nblk);  // a well-formed range is inside the store
        res1 = min(max(e1, res0), p.nblk);
        if ((res0 != e0 || res1 != e1) && tid == 0) report_index(p.err);
    }
    const int total = nbase + (res1 - res0 + 3) / 4;
    const int steps = step0 < total ? (total - step0 + stride - 1) / stride : 0;
    while (ahead < min(kStages, steps)) issue(ahead++);
    // Column chunk c (0..3, 64 columns) of a step, -1 past the end (a block's: or past K).
    auto chunk_of = [&](int i, int c) {
        const int step = step0 + i * stride;
        if (step < nbase) return 4 * step + c < KC ? 4 * step + c : -1;
        const int e = res0 + 4 * (step - nbase) + c;
        const int kt = e < res1 ? __ldg(p.blk_kt + e) : -1;
        if (e < res1 && (unsigned)kt >= (unsigned)KC) report_index(p.err);
        return (unsigned)kt < (unsigned)KC ? kt : -1;
    };
    const int kt = steps > 0 ? chunk_of(0, t) : -1;
    int ktn = steps > 1 ? chunk_of(1, t) : -1;
    griddep_wait();
    griddep_launch();

    uint4 b[NT][4];  // the lane's operand in the warp's 32 of its 64 columns, a step ahead
    auto load_x = [&](int kt) {
        const uint8_t* src = p.xop + (int64_t)kt * (NT * 1024) + (4 * h) * 128 + g * 16;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int w = 0; w < 4; ++w)
                b[nt][w] = kt >= 0 ? ld_prior(reinterpret_cast<const uint4*>(src + nt * 1024 + w * 128)) : make_uint4(0, 0, 0, 0);
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
        const bool valid = step < nbase ? 4 * step + t < KC : res0 + 4 * (step - nbase) + t < res1;  // columns of this lane's rows
        const uint32_t parity = (i / kStages) & 1u;
        // the warp decides together; after a wait that gave up (reported) nothing is issued or waited for
        if (__any_sync(0xffffffffu, !mbar_try_wait(full + i % kStages, parity)) && alive)
            alive = __all_sync(0xffffffffu, mbar_wait_err(full + i % kStages, parity, p.err));
        const uint8_t* buf = ring + (i % kStages) * kStage;
        // scales of rows 16 rt + 8 hf + g in the lane's 64 columns: a 128-row chunk holds row
        // r's four at (r % 32) * 16 + (r / 32) * 4. Columns past the end may hold anything: zero.
        uint32_t sc[4][2];  // the warp's half: two groups of 16 columns
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const uint2 w = *reinterpret_cast<const uint2*>(buf + kCodes + t * 512 + (16 * q + 8 * hf + g) * 16 + (tile & 1) * 8);
                const uint32_t two = __byte_perm(w.x, w.y, h ? 0x7632 : 0x5410);
                e4m3x4_half(valid ? two : 0u, sc[q][hf], sc[q + 2][hf]);
            }
        // 16-byte piece h of the lane's columns in row r: swizzled rows of 128 bytes, or packed blocks
        const bool isb = step < nbase;
        const uint8_t* codes = isb ? buf + g * 128 : buf + t * 2048 + g * 16;
        const int row8 = isb ? 1024 : 256;  // eight rows further
        {
            const uint8_t* at = codes + (isb ? ((2 * t + h) ^ g) * 16 : h * 128);
            uint4 x0[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int w = 0; w < 4; ++w) x0[nt][w] = b[nt][w];
            load_x(ktn);
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                const uint4 a0 = *reinterpret_cast<const uint4*>(at + (2 * rt) * row8);
                const uint4 a1 = *reinterpret_cast<const uint4*>(at + (2 * rt + 1) * row8);
                const uint32_t s0 = sc[rt][0], s1 = sc[rt][1];
                const uint32_t w0[4] = {a0.x, a0.y, a0.z, a0.w}, w1[4] = {a1.x, a1.y, a1.z, a1.w};
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t x[4], y[4];
                    e2m1x8_half(w0[w], x);
                    e2m1x8_half(w1[w], y);
                    const __half2 f0 = w < 2 ? low2(s0) : high2(s0), f1 = w < 2 ? low2(s1) : high2(s1);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t a[4] = {mul_h2(x[2 * e], f0), mul_h2(y[2 * e], f1), mul_h2(x[2 * e + 1], f0),
                                               mul_h2(y[2 * e + 1], f1)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16(acc[rt][nt], a, e ? x0[nt][w].z : x0[nt][w].x, e ? x0[nt][w].w : x0[nt][w].y);
                    }
                }
            }
        }
        ktn = i + 2 < steps ? chunk_of(i + 2, t) : -1;
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + i % kStages);
        if (h == 0 && i + kStages < steps && alive) {
            // the other warp's half
            if (__any_sync(0xffffffffu, !mbar_try_wait(empty + i % kStages, parity)))
                alive = __all_sync(0xffffffffu, mbar_wait_err(empty + i % kStages, parity, p.err));
            if (alive) issue(i + kStages);
        }
    }
    if (!alive)  // the last copies get their (bounded) time
        for (int i = max(0, steps - kStages); i < steps; ++i) mbar_wait_err(full + i % kStages, (i / kStages) & 1u, p.err);

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
    // the tensor scale before the token's: a sum times a far token's scale alone may pass fp32's range
    const float gw = __ldg(p.g_w);
    const float* back = reinterpret_cast<const float*>(p.xop + (int64_t)KC * (NT * 1024));  // the tokens' scales
    float* mine = sums + kWarps * 8 * NT * kPitch;  // [token][kPitch], this CTA's
    for (int i = tid; i < kRows * p.M; i += kThreads) {
        const int m = i / kRows, n = i % kRows;
        float v = sums[m * kPitch + n];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v += sums[(w * 8 * NT + m) * kPitch + n];
        if (S == 1)
            p.Y[m * p.ldy + tile * kRows + n] = (uint16_t)narrow2<F16>(v * gw * ld_prior(back + m), 0.0f);
        else
            mine[m * kPitch + n] = v;
    }
    if (S > 1) {
        cluster_sync();
        for (int i = tid + rank * kThreads; i < kRows * p.M; i += S * kThreads) {
            const int m = i / kRows, n = i % kRows;
            float v = 0.0f;
            for (int r = 0; r < S; ++r) v += ld_dsmem_f32(mine + m * kPitch + n, r);
            p.Y[m * p.ldy + tile * kRows + n] = (uint16_t)narrow2<F16>(v * gw * ld_prior(back + m), 0.0f);
        }
        cluster_sync();  // no CTA leaves while another reads its sums
    }
}

template <int NT, bool F16>
cudaError_t gemv_of(const CUtensorMap& tw, const GemvParams& p, int S, cudaStream_t s) {
    static std::atomic<bool> done[64];
    cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(k_gemv<NT, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<NT>());
    });
    if (e != cudaSuccess) return e;
    uint8_t* xop = p.xop;
    e = launch_pdl(k_gemv_x<F16>, dim3(8 * NT), dim3(kXThreads), 0, s, 1, p.X, p.ldx, p.M, NT, p.K, xop,
                   reinterpret_cast<float*>(xop + (int64_t)(p.K / 64) * (NT * 1024)));
    if (e != cudaSuccess) return e;
    return launch_pdl_cluster(k_gemv<NT, F16>, dim3(S, p.N / kRows), dim3(64 * pairs<NT>()), smem_bytes<NT>(), s, dim3(S, 1, 1), tw, p);
}

}  // namespace

size_t gemv_workspace(int M, int K) { return operand_bytes(M <= 8 ? 1 : 2, K); }

cudaError_t launch_gemv(const CUtensorMap& tw, const GemvParams& p, bool f16, cudaStream_t s) {
    const int tiles = p.N / kRows, steps = (p.K / 64 + 3) / 4;
    // CTAs that fill the GPU once, none without a step for each of its warps
    const int S = std::max(1, std::min({8, kCtasPerSm * device_sms() / tiles, steps / (p.M <= 8 ? pairs<1>() : pairs<2>())}));
    if (p.M <= 8) return f16 ? gemv_of<1, true>(tw, p, S, s) : gemv_of<1, false>(tw, p, S, s);
    return f16 ? gemv_of<2, true>(tw, p, S, s) : gemv_of<2, false>(tw, p, S, s);
}

}  // namespace mq
