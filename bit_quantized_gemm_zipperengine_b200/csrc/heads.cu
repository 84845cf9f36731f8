// Per-head work of a new token: RMS norm and position rotation of queries and keys,
// NVFP4 quantization of keys and values into the paged cache, and the way back.
//
//   u = x * (mean_d x^2 + eps)^(-1/2) * w_d,   (a, b) -> (a cos - b sin, b cos + a sin)
//
// Every element is read once and written once, so the floor is the bytes. A row (one head
// of one token) is held by D/8 lanes, 16 bytes each: the sum of squares is a shuffle tree,
// the partner of a rotated half sits rot/16 lanes away, and a group of 16 quantized
// elements is a lane pair. A warp keeps one token and walks heads, so that the token's
// angles (fp64: a far position times a frequency loses its fraction in fp32) are formed once.
#include "ops.cuh"

namespace mq {

namespace {

constexpr int kWarps = 4;

// The angle pos * freq in turns, its fraction in [-1/2, 1/2], then cos and sin in fp32.
__device__ __forceinline__ float2 cos_sin(double pos, double freq) {
    const double turns = pos * freq * 0.15915494309189533577;
    const float r = (float)(turns - rint(turns));
    float c, s;
    sincospif(2.0f * r, &s, &c);
    return make_float2(c, s);
}

// NVFP4 of a group held by two adjacent lanes, eight elements each, with tensor scale g
// (the rule of nvfp4_group): this lane's eight codes; the scale byte in sf.
__device__ __forceinline__ uint32_t quantize_pair(const float (&a)[8], float g, float g6, uint32_t& sf) {
    float m = max3(fabsf(a[0]), fabsf(a[1]), fabsf(a[2]));
    m = max3(m, fabsf(a[3]), fabsf(a[4]));
    m = max3(m, fabsf(a[5]), fabsf(a[6]));
    m = fmaxf(m, fabsf(a[7]));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    sf = e4m3_encode_nonneg(__fdiv_rn(m, g6));
    const float d = __fmul_rn(e4m3_value(sf), g);
    if (!(d > 0.0f)) return sign_nibbles8(a);
    const float r = __frcp_rn(d);
    return e2m1x8(__fmul_rn(a[0], r), __fmul_rn(a[1], r), __fmul_rn(a[2], r), __fmul_rn(a[3], r), __fmul_rn(a[4], r),
                  __fmul_rn(a[5], r), __fmul_rn(a[6], r), __fmul_rn(a[7], r));
}

// One record of the cache for slot (checked by the caller) and head h.
template <int D>
__device__ __forceinline__ uint8_t* record_of(const CacheView& c, int64_t slot, int h) {
    const int64_t page = slot / c.page_size;
    const int rec = (int)(slot - page * c.page_size) >> 4;
    return c.pages + ((page * c.heads + h) * (c.page_size >> 4) + rec) * (18 * D);
}

template <int D, bool F16>
__global__ void __launch_bounds__(32 * kWarps) k_heads(const HeadsParams p, int chunks, int per_warp) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31, li = lane % LPR, sub = lane / LPR;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t t = unit / chunks;
    if (t >= p.T) return;
    const int nq = p.q.p ? p.q.heads : 0, nk = p.k.p ? p.k.heads : 0, nv = p.v.p ? p.v.heads : 0;
    const int h0 = (int)(unit - t * chunks) * per_warp, h1 = min(h0 + per_warp, nq + nk + nv);
    const int e0 = 8 * li, half = p.rot / 2;

    // this lane's angles: of its eight elements (halves), or of its four pairs
    float2 cs[8];
    if (e0 < p.rot) {
        const double pos = (double)__ldg(p.pos + t);
        if (p.interleaved) {
#pragma unroll
            for (int j = 0; j < 4; ++j) cs[j] = cos_sin(pos, __ldg(p.freq + e0 / 2 + j));
        } else {
            const int i0 = e0 < half ? e0 : e0 - half;
#pragma unroll
            for (int j = 0; j < 8; ++j) cs[j] = cos_sin(pos, __ldg(p.freq + i0 + j));
        }
    }
    int64_t slot = -1;
    if (p.cache.pages) {
        slot = __ldg(p.slots + t);
        if (slot >= (int64_t)p.cache.num_pages * p.cache.page_size) {
            if (lane == 0) report_index(p.err);
            slot = -1;
        }
    }
    for (int hb = h0; hb < h1; hb += RPW) {
        const int hg = hb + sub;
        const bool on = hg < h1;
        const int kind = hg < nq ? 0 : hg < nq + nk ? 1 : 2;  // q, k, v
        const HeadsView& in = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
        const int h = kind == 0 ? hg : kind == 1 ? hg - nq : hg - nq - nk;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (on) w = *reinterpret_cast<const uint4*>(in.p + t * in.st + h * in.sh + e0);
        float a[8];
        {
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = widen2<F16>(x[j]);
                a[2 * j] = f.x;
                a[2 * j + 1] = f.y;
            }
        }
        // the warp's rows may be of different kinds: the shuffles run for all of them
        const uint16_t* wt = kind == 0 ? p.wq : kind == 1 ? p.wk : nullptr;
        if (p.wq || p.wk) {
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = __fmaf_rn(a[j], a[j], ss);
#pragma unroll
            for (int o = 1; o < LPR; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (wt) {
                const float r = rsqrtf(ss * (1.0f / D) + p.eps);
                const uint4 g = __ldg(reinterpret_cast<const uint4*>(wt + e0));
                const uint32_t x[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = widen2<F16>(x[j]);
                    a[2 * j] *= r * f.x;
                    a[2 * j + 1] *= r * f.y;
                }
            }
        }
        if (p.rot > 0) {
            if (p.interleaved) {
                if (e0 < p.rot && kind < 2) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float x = a[2 * j], y = a[2 * j + 1];
                        a[2 * j] = __fmaf_rn(x, cs[j].x, -(y * cs[j].y));
                        a[2 * j + 1] = __fmaf_rn(y, cs[j].x, x * cs[j].y);
                    }
                }
            } else {
                const int r2 = p.rot / 16;
                const int src = sub * LPR + (li < r2 ? li + r2 : li < 2 * r2 ? li - r2 : li);
                const float sign = li < r2 ? -1.0f : 1.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float y = __shfl_sync(0xffffffffu, a[j], src);
                    if (e0 < p.rot && kind < 2) a[j] = __fmaf_rn(a[j], cs[j].x, sign * y * cs[j].y);
                }
            }
        }
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = narrow2<F16>(a[2 * j], a[2 * j + 1]);
        if (kind < 2 && on) {
            const HeadsView& out = kind == 0 ? p.qo : p.ko;
            if (out.p)
                *reinterpret_cast<uint4*>(out.p + t * out.st + h * out.sh + e0) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        if constexpr (D <= 128) {
            if (p.cache.pages) {
                // what the cache holds is the rounded row
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = widen2<F16>(o[j]);
                    a[2 * j] = f.x;
                    a[2 * j + 1] = f.y;
                }
                const float* sc = kind == 1 ? p.cache.k_scale : p.cache.v_scale;
                const float g = (sc && on && kind > 0) ? __ldg(sc + h) : 1.0f;
                uint32_t sf;
                const uint32_t codes = quantize_pair(a, g, __fmul_rn(6.0f, g), sf);
                if (on && kind > 0 && slot >= 0) {
                    uint8_t* rec = record_of<D>(p.cache, slot, h);
                    const int i = (int)(slot & 15), q = li >> 1;  // page_size is a multiple of 16
                    const int at = kind == 1 ? i * (D / 2) + 4 * li : rec_vcodes<D>(i, q) + 4 * (li & 1);
                    *reinterpret_cast<uint32_t*>(rec + at) = codes;
                    if (!(li & 1)) rec[kind == 1 ? rec_kscale<D>(i, q) : rec_vscale<D>(i, q)] = (uint8_t)sf;
                }
            }
        }
    }
}

// The cached rows of slots[t]: warp per (token, heads), lanes as above.
template <int D, bool F16>
__global__ void __launch_bounds__(32 * kWarps) k_kv_read(const HeadsParams p) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31, li = lane % LPR, sub = lane / LPR;
    const int H = p.cache.heads, rows = 2 * H;
    const int64_t row = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * RPW + sub;
    const int64_t t = row / rows;
    if (t >= p.T) return;
    const int hg = (int)(row - t * rows), kind = hg >= H, h = kind ? hg - H : hg;
    const int64_t slot = __ldg(p.slots + t);
    if (slot < 0) return;
    if (slot >= (int64_t)p.cache.num_pages * p.cache.page_size) {
        if (li == 0) report_index(p.err);
        return;
    }
    const uint8_t* rec = record_of<D>(p.cache, slot, h);
    const int i = (int)(slot & 15), q = li >> 1;
    const float* sc = kind ? p.cache.v_scale : p.cache.k_scale;
    const float g = sc ? __ldg(sc + h) : 1.0f;
    const uint32_t codes =
        *reinterpret_cast<const uint32_t*>(rec + (kind ? rec_vcodes<D>(i, q) + 4 * (li & 1) : i * (D / 2) + 4 * li));
    const float d = __fmul_rn(e4m3_value(rec[kind ? rec_vscale<D>(i, q) : rec_kscale<D>(i, q)]), g);
    float v[8];
    e2m1x8_values(codes, v);
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = narrow2<F16>(__fmul_rn(v[2 * j], d), __fmul_rn(v[2 * j + 1], d));
    const HeadsView& out = kind ? p.v : p.k;
    *reinterpret_cast<uint4*>(out.p + t * out.st + h * out.sh + 8 * li) = make_uint4(o[0], o[1], o[2], o[3]);
}

template <int D, bool F16>
cudaError_t heads_of(const HeadsParams& p, cudaStream_t s) {
    constexpr int RPW = 32 / (D / 8);
    const int heads = (p.q.p ? p.q.heads : 0) + (p.k.p ? p.k.heads : 0) + (p.v.p ? p.v.heads : 0);
    const int per = RPW * 4;  // heads a warp walks
    const int chunks = (heads + per - 1) / per;
    const int64_t blocks = ((int64_t)p.T * chunks + kWarps - 1) / kWarps;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    return launch_pdl(k_heads<D, F16>, dim3((unsigned)blocks), dim3(32 * kWarps), 0, s, 1, p, chunks, per);
}

template <int D, bool F16>
cudaError_t read_of(const HeadsParams& p, cudaStream_t s) {
    constexpr int rows_per_block = kWarps * (32 / (D / 8));
    const int64_t blocks = ((int64_t)p.T * 2 * p.cache.heads + rows_per_block - 1) / rows_per_block;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    return launch_pdl(k_kv_read<D, F16>, dim3((unsigned)blocks), dim3(32 * kWarps), 0, s, 1, p);
}

}  // namespace

cudaError_t launch_heads(const HeadsParams& p, int D, bool f16, cudaStream_t s) {
    switch (D) {
        case 64: return f16 ? heads_of<64, true>(p, s) : heads_of<64, false>(p, s);
        case 128: return f16 ? heads_of<128, true>(p, s) : heads_of<128, false>(p, s);
        default: return f16 ? heads_of<256, true>(p, s) : heads_of<256, false>(p, s);
    }
}

cudaError_t launch_kv_read(const HeadsParams& p, int D, bool f16, cudaStream_t s) {
    if (D == 64) return f16 ? read_of<64, true>(p, s) : read_of<64, false>(p, s);
    return f16 ? read_of<128, true>(p, s) : read_of<128, false>(p, s);
}

}  // namespace mq
