// Per-head work of a new token: RMS norm and position rotation of queries and keys,
// NVFP4 quantization of keys and values into the paged cache, and the way back.
//
//   u = x * (mean_d x^2 + eps)^(-1/2) * w_d,   (a, b) -> (a cos - b sin, b cos + a sin)
//
// Every element is read once and written once, so the floor is the bytes; few tokens are
// bound by the launch and one chain of loads. A CTA takes a token and some of its heads. Its
// threads form the token's angles once, one each (fp64: a far position times a frequency
// loses its fraction in fp32), and share them. A row (one head) is held by D/8 lanes, 16
// bytes each: the sum of squares is a shuffle tree, the partner of a rotated half sits
// rot/16 lanes away, and a group of 16 quantized elements is a lane pair. A warp's next row is
// in flight while it works on one.
#include <algorithm>

#include "ops.cuh"

namespace mq {

namespace {

constexpr int kWarps = 4;
constexpr int kSpread = 4;  // CTAs an SM that a call should have before a CTA takes a second step

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

// A slot's page and token in the page (slot checked by the caller).
__device__ __forceinline__ void split_slot(const HeadsParams& p, int64_t slot, int64_t& page, int& token) {
    if (slot < 0x7FFFFFFF) {
        const uint32_t q = p.by_page.div((uint32_t)slot);
        page = q;
        token = (int)((uint32_t)slot - q * (uint32_t)p.cache.page_size);
    } else {
        page = slot / p.cache.page_size;
        token = (int)(slot - page * p.cache.page_size);
    }
}

// steps: how many rows a lane group walks (a CTA's rows are dealt to its warps in turn).
template <int D, bool F16>
__global__ void __launch_bounds__(32 * kWarps) k_heads(const HeadsParams p, int steps) {
    constexpr int LPR = D / 8, RPW = 32 / LPR, STEP = kWarps * RPW;
    __shared__ float2 angles[D / 2];
    const int lane = threadIdx.x & 31, li = lane % LPR, e0 = 8 * li, half = p.rot / 2;
    const int64_t t = blockIdx.x;
    const int nq = p.q.heads, nk = p.k.heads, nv = p.v.heads, all = nq + nk + nv;  // 0 heads: absent
    int hg = blockIdx.y * steps * STEP + (threadIdx.x >> 5) * RPW + lane / LPR;     // this lane's row: q, k, then v heads
    const uint16_t *qb = p.q.p + t * p.q.st + e0, *kb = p.k.p + t * p.k.st + e0, *vb = p.v.p + t * p.v.st + e0;
    auto load = [&](int hg) {
        if (hg >= all) return make_uint4(0, 0, 0, 0);
        const uint16_t* src = hg < nq ? qb + hg * p.q.sh : hg < nq + nk ? kb + (hg - nq) * p.k.sh : vb + (hg - nq - nk) * p.v.sh;
        return *reinterpret_cast<const uint4*>(src);
    };
    griddep_wait();
    griddep_launch();
    uint4 next = load(hg);
    uint8_t* rec = nullptr;  // head 0's record of this token's slot
    int tok = 0;             // its token in the record
    if (p.cache.pages) {
        const int64_t slot = __ldg(p.slots + t);
        if (slot >= (int64_t)p.cache.num_pages * p.cache.page_size) {
            if (threadIdx.x == 0) report_index(p.err);
        } else if (slot >= 0) {
            int64_t page;
            split_slot(p, slot, page, tok);
            rec = p.cache.pages + (page * p.cache.heads * (p.cache.page_size >> 4) + (tok >> 4)) * (18 * D);
            tok &= 15;
        }
    }
    if (p.rot > 0) {
        if ((int)threadIdx.x < half) angles[threadIdx.x] = cos_sin((double)__ldg(p.pos + t), __ldg(p.freq + threadIdx.x));
        __syncthreads();
    }
    // this lane's angles: of its eight elements (halves; the sine with its sign), or of its four pairs
    const bool turned = e0 < p.rot;
    const int r2 = p.rot / 16, from = (lane & ~(LPR - 1)) + (li < r2 ? li + r2 : li < 2 * r2 ? li - r2 : li);
    float2 cs[8];
    if (turned) {
        if (p.interleaved) {
#pragma unroll
            for (int j = 0; j < 4; ++j) cs[j] = angles[e0 / 2 + j];
        } else {
            const int i0 = e0 < half ? e0 : e0 - half;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                cs[j] = angles[i0 + j];
                if (e0 < half) cs[j].y = -cs[j].y;
            }
        }
    }
    for (int s = 0; s < steps; ++s, hg += STEP) {
        const uint4 w = next;
        const bool on = hg < all;
        if (s + 1 < steps) next = load(hg + STEP);
        const int kind = hg < nq ? 0 : hg < nq + nk ? 1 : 2;  // q, k, v
        const int h = kind == 0 ? hg : kind == 1 ? hg - nq : hg - nq - nk;
        uint32_t o[4] = {w.x, w.y, w.z, w.w};
        float a[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = widen2<F16>(o[j]);
            a[2 * j] = f.x;
            a[2 * j + 1] = f.y;
        }
        // the warp's rows may be of different kinds: the shuffles run for all of them
        if (p.wq || p.wk) {
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = __fmaf_rn(a[j], a[j], ss);
#pragma unroll
            for (int x = 1; x < LPR; x <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, x);
            const uint16_t* wt = kind == 0 ? p.wq : kind == 1 ? p.wk : nullptr;
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
                if (turned && kind < 2) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float x = a[2 * j], y = a[2 * j + 1];
                        a[2 * j] = __fmaf_rn(x, cs[j].x, -(y * cs[j].y));
                        a[2 * j + 1] = __fmaf_rn(y, cs[j].x, x * cs[j].y);
                    }
                }
            } else {
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = __shfl_sync(0xffffffffu, a[j], from);
                if (turned && kind < 2)
#pragma unroll
                    for (int j = 0; j < 8; ++j) a[j] = __fmaf_rn(a[j], cs[j].x, y[j] * cs[j].y);
            }
        }
        if (kind < 2) {
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = narrow2<F16>(a[2 * j], a[2 * j + 1]);
            const HeadsView& out = kind == 0 ? p.qo : p.ko;
            if (on && out.p)
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
                if (on && kind > 0 && rec) {
                    uint8_t* r = rec + (int64_t)h * ((p.cache.page_size >> 4) * (18 * D));
                    const int q = li >> 1;
                    const int at = kind == 1 ? tok * (D / 2) + 4 * li : rec_vcodes<D>(tok, q) + 4 * (li & 1);
                    *reinterpret_cast<uint32_t*>(r + at) = codes;
                    if (!(li & 1)) r[kind == 1 ? rec_kscale<D>(tok, q) : rec_vscale<D>(tok, q)] = (uint8_t)sf;
                }
            }
        }
    }
}

// The cached rows of slots[t], lanes and warps as above; two of a warp's rows at a time.
template <int D, bool F16>
__global__ void __launch_bounds__(32 * kWarps) k_kv_read(const HeadsParams p) {
    constexpr int LPR = D / 8, RPW = 32 / LPR, STEP = kWarps * RPW;
    const int lane = threadIdx.x & 31, li = lane % LPR, q = li >> 1;
    const int64_t t = blockIdx.x;
    const int H = p.cache.heads;
    griddep_wait();
    griddep_launch();
    const int64_t slot = __ldg(p.slots + t);
    if (slot < 0) return;
    if (slot >= (int64_t)p.cache.num_pages * p.cache.page_size) {
        if (threadIdx.x == 0) report_index(p.err);
        return;
    }
    int64_t page;
    int tok;
    split_slot(p, slot, page, tok);
    const int64_t per_head = (int64_t)(p.cache.page_size >> 4) * (18 * D);
    const uint8_t* rec = p.cache.pages + page * H * per_head + (tok >> 4) * (18 * D);
    tok &= 15;
    const int kat = tok * (D / 2) + 4 * li, vat = rec_vcodes<D>(tok, q) + 4 * (li & 1);
    const int ksat = rec_kscale<D>(tok, q), vsat = rec_vscale<D>(tok, q);
    uint16_t *kb = p.k.p + t * p.k.st + 8 * li, *vb = p.v.p + t * p.v.st + 8 * li;
    for (int h = (threadIdx.x >> 5) * RPW + lane / LPR; h < H; h += STEP) {
        const uint8_t* r = rec + h * per_head;
        const uint32_t kc = *reinterpret_cast<const uint32_t*>(r + kat), vc = *reinterpret_cast<const uint32_t*>(r + vat);
        const uint32_t ks = r[ksat], vs = r[vsat];
        const float gk = p.cache.k_scale ? __ldg(p.cache.k_scale + h) : 1.0f;
        const float gv = p.cache.v_scale ? __ldg(p.cache.v_scale + h) : 1.0f;
        auto put = [&](uint32_t codes, uint32_t sf, float g, uint16_t* dst) {
            const float d = __fmul_rn(e4m3_value(sf), g);
            float v[8];
            e2m1x8_values(codes, v);
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = narrow2<F16>(__fmul_rn(v[2 * j], d), __fmul_rn(v[2 * j + 1], d));
            *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
        };
        put(kc, ks, gk, kb + h * p.k.sh);
        put(vc, vs, gv, vb + h * p.v.sh);
    }
}

template <int D, bool F16>
cudaError_t heads_of(const HeadsParams& p, cudaStream_t s) {
    constexpr int STEP = kWarps * (32 / (D / 8));  // rows of a CTA at a time
    const int steps_all = (p.q.heads + p.k.heads + p.v.heads + STEP - 1) / STEP;
    // few tokens: their heads are spread over more CTAs, down to one step each
    const int spread = (int)std::min<int64_t>(steps_all, std::max<int64_t>(1, (int64_t)kSpread * device_sms() / p.T));
    const int steps = (steps_all + spread - 1) / spread;
    return launch_pdl(k_heads<D, F16>, dim3((unsigned)p.T, (steps_all + steps - 1) / steps), dim3(32 * kWarps), 0, s, 1, p, steps);
}

template <int D, bool F16>
cudaError_t read_of(const HeadsParams& p, cudaStream_t s) {
    return launch_pdl(k_kv_read<D, F16>, dim3((unsigned)p.T), dim3(32 * kWarps), 0, s, 1, p);
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
