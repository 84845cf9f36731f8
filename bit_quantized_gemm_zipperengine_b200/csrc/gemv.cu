// Products of a few tokens of 16-bit activations with the packed NVFP4 weight:
//   Y[m,n] = rn(g_w * sum_k x[m,k] (wh[n,k] + [block selected] rh[n,k])),  wh = val * dec(sf).
// The floor is the weight's bytes (9/16 a weight, 2304 a residual block), read once.
// One warp a row; a lane takes 32 codes (16 bytes, two scale groups) at a time.
#include "ops.cuh"

namespace mq {

namespace {

constexpr int kWarps = 4;

// acc[m] += sum over 32 elements at column k0: 16 bytes of codes and their two scales.
template <int MT, bool F16>
__device__ __forceinline__ void fma32(const GemvParams& p, const uint4& w, float s0, float s1, int k0, int m0,
                                      float (&acc)[MT]) {
    const uint32_t c[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float v[8];
        e2m1x8_values(c[j], v);
        const float s = j < 2 ? s0 : s1;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= s;  // exact: six significant bits
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if (m0 + m >= p.M) break;
            const uint4 xv = __ldg(reinterpret_cast<const uint4*>(p.X + (m0 + m) * p.ldx + k0 + 8 * j));
            const uint32_t x[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = widen2<F16>(x[i]);
                acc[m] = __fmaf_rn(f.x, v[2 * i], acc[m]);
                acc[m] = __fmaf_rn(f.y, v[2 * i + 1], acc[m]);
            }
        }
    }
}

template <int MT, bool F16>
__global__ void __launch_bounds__(32 * kWarps) k_gemv(const GemvParams p) {
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31, n = blockIdx.x * kWarps + (threadIdx.x >> 5), m0 = blockIdx.y * MT;
    if (n >= p.N) return;
    float acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = 0.0f;
    if (p.base) {
        const uint8_t* row = p.codes + (int64_t)n * (p.K / 2);
        for (int k0 = 32 * lane; k0 < p.K; k0 += 1024) {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(row + k0 / 2));
            const uint8_t* f = p.sf + sf_swz_offset(n, k0 / 16, p.K);
            fma32<MT, F16>(p, w, e4m3_value(f[0]), e4m3_value(f[1]), k0, m0, acc);
        }
    }
    if (p.blk_codes) {
        const int lo = __ldg(p.tile_ptr + n / 64), hi = __ldg(p.tile_ptr + n / 64 + 1), r = n & 63, t = n & 127;
        for (int e = 2 * lo + lane; e < 2 * hi; e += 32) {  // half a block row each
            const int64_t b = e >> 1;
            const int h = e & 1;
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(p.blk_codes + b * 2048 + (r / 8) * 256 + h * 128 + (r % 8) * 16));
            const uint8_t* f = p.blk_sf + b * 512 + (t % 32) * 16 + (t / 32) * 4 + 2 * h;
            fma32<MT, F16>(p, w, e4m3_value(f[0]), e4m3_value(f[1]), 64 * __ldg(p.blk_kt + b) + 32 * h, m0, acc);
        }
    }
    const float g = __ldg(p.g_w);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[m] += __shfl_xor_sync(0xffffffffu, acc[m], o);
        if (lane == 0 && m0 + m < p.M) p.Y[(m0 + m) * p.ldy + n] = (uint16_t)narrow2<F16>(acc[m] * g, 0.0f);
    }
}

}  // namespace

cudaError_t launch_gemv(const GemvParams& p, bool f16, cudaStream_t s) {
    const dim3 grid((p.N + kWarps - 1) / kWarps, (p.M + 3) / 4);
    return f16 ? launch_pdl(k_gemv<4, true>, grid, dim3(32 * kWarps), 0, s, 1, p)
               : launch_pdl(k_gemv<4, false>, grid, dim3(32 * kWarps), 0, s, 1, p);
}

}  // namespace mq
