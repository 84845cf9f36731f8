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
// in flight while it works on one. 16 tokens of 72 heads take 2.3 us; 8191 of 40 heads, turned,
// 30.8 us (5.5 TB/s; 71% of the issue slots used), and appended, 8 heads, about 15 us (76%, ~40
// instructions for eight quantized values).
#include <algorithm>

#include "ops.cuh"

namespace mq {

namespace {

constexpr int kWarps = 2;
constexpr int kUnroll = 2;  // rows a lane group works on together
constexpr int kReadWarps = 2;
constexpr int kReadUnroll = 2;
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

// How the heads of a call are dealt: kWarps * RPW * kUnroll rows of one kind (q, k, v) a
// step, steps numbered through the kinds; a CTA takes `steps` of them.
struct Deal {
    int q, k, v;  // steps of each kind
    int steps;
};

// TURN: 0 none, 1 halves, 2 interleaved pairs.
template <int D, bool F16, int TURN>
__global__ void __launch_bounds__(32 * kWarps, 32 / kWarps) k_heads(const HeadsParams p, const Deal deal) {
    constexpr int LPR = D / 8, RPW = 32 / LPR, STEP = kWarps * RPW * kUnroll;
    __shared__ float2 angles[TURN ? D / 2 : 1];
    const int lane = threadIdx.x & 31, li = lane % LPR, e0 = 8 * li, half = p.rot / 2;
    const int row = (threadIdx.x >> 5) * RPW + lane / LPR;  // of a step's rows: this one and kUnroll - 1 more, kWarps * RPW apart
    const int64_t t = blockIdx.x;
    int s = blockIdx.y * deal.steps;
    const int s1 = min(s + deal.steps, deal.q + deal.k + deal.v);

    // one step's kind, first head and operands (the same for the whole CTA)
    struct Kind {
        int kind, h0, heads;
        const uint16_t* src;
        int64_t sh;
    };
    auto kind_of = [&](int s) {
        Kind k;
        k.kind = s < deal.q ? 0 : s < deal.q + deal.k ? 1 : 2;
        const HeadsView& in = k.kind == 0 ? p.q : k.kind == 1 ? p.k : p.v;
        k.h0 = (s - (k.kind == 0 ? 0 : k.kind == 1 ? deal.q : deal.q + deal.k)) * STEP;
        k.heads = in.heads;
        k.src = in.p + t * in.st;
        k.sh = in.sh;
        return k;
    };
    uint4 next[kUnroll];
    auto load = [&](const Kind& k) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = k.h0 + row + u * (kWarps * RPW);
            next[u] = h < k.heads ? *reinterpret_cast<const uint4*>(k.src + h * k.sh + e0) : make_uint4(0, 0, 0, 0);
        }
    };
    griddep_wait();
    griddep_launch();
    Kind k = kind_of(s);
    load(k);
    uint8_t* rec = nullptr;  // head 0's record of this token's slot
    int tok = 0;             // its token in the record
    if (p.cache.pages) {
        const int64_t slot = ld_prior(p.slots + t);
        if (slot >= (int64_t)p.cache.num_pages * p.cache.page_size) {
            if (threadIdx.x == 0) report_index(p.err);
        } else if (slot >= 0) {
            int64_t page;
            split_slot(p, slot, page, tok);
            rec = p.cache.pages + (page * p.cache.heads * (p.cache.page_size >> 4) + (tok >> 4)) * (18 * D);
            tok &= 15;
        }
    }
    // this lane's angles: of its eight elements (halves; the sine with its sign), or of its four
    // pairs; a lane past the rotation turns by nothing
    float2 cs[8];
    const int r2 = p.rot / 16, from = (lane & ~(LPR - 1)) + (li < r2 ? li + r2 : li < 2 * r2 ? li - r2 : li);
    if constexpr (TURN != 0) {
        const double pos = (double)ld_prior(p.pos + t);
        for (int i = threadIdx.x; i < half; i += 32 * kWarps) angles[i] = cos_sin(pos, ld_prior(p.freq + i));
        __syncthreads();
#pragma unroll
        for (int j = 0; j < (TURN == 2 ? 4 : 8); ++j) {
            cs[j] = make_float2(1.0f, 0.0f);
            if (e0 < p.rot) {
                cs[j] = angles[TURN == 2 ? e0 / 2 + j : e0 < half ? e0 + j : e0 - half + j];
                if (TURN == 1 && e0 < half) cs[j].y = -cs[j].y;
            }
        }
    }
    for (; s < s1; ++s) {
        const Kind c = k;
        uint4 w[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) w[u] = next[u];
        if (s + 1 < s1) {
            k = kind_of(s + 1);
            load(k);
        }
        const uint16_t* wt = c.kind == 0 ? p.wq : c.kind == 1 ? p.wk : nullptr;
        const HeadsView& out = c.kind == 0 ? p.qo : p.ko;
        const bool store = c.kind < 2 && out.p, quantize = c.kind > 0 && p.cache.pages;
        uint16_t* dst = out.p + t * out.st + e0;
        const float* sc = c.kind == 1 ? p.cache.k_scale : p.cache.v_scale;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = c.h0 + row + u * (kWarps * RPW);
            const bool on = h < c.heads;
            uint32_t o[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
            float a[8];
            if (c.kind < 2) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = widen2<F16>(o[j]);
                    a[2 * j] = f.x;
                    a[2 * j + 1] = f.y;
                }
                if (wt) {
                    float ss = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss = __fmaf_rn(a[j], a[j], ss);
#pragma unroll
                    for (int x = 1; x < LPR; x <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, x);
                    const float r = rsqrtf(ss * (1.0f / D) + p.eps);
                    const uint4 g = ld_prior(reinterpret_cast<const uint4*>(wt + e0));
                    const uint32_t x[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = widen2<F16>(x[j]);
                        a[2 * j] *= r * f.x;
                        a[2 * j + 1] *= r * f.y;
                    }
                }
                if constexpr (TURN == 2) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float x = a[2 * j], y = a[2 * j + 1];
                        a[2 * j] = __fmaf_rn(x, cs[j].x, -(y * cs[j].y));
                        a[2 * j + 1] = __fmaf_rn(y, cs[j].x, x * cs[j].y);
                    }
                } else if constexpr (TURN == 1) {
                    float y[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = __shfl_sync(0xffffffffu, a[j], from);
#pragma unroll
                    for (int j = 0; j < 8; ++j) a[j] = __fmaf_rn(a[j], cs[j].x, y[j] * cs[j].y);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = narrow2<F16>(a[2 * j], a[2 * j + 1]);
                if (store && on) *reinterpret_cast<uint4*>(dst + h * out.sh) = make_uint4(o[0], o[1], o[2], o[3]);
            }
            if constexpr (D <= 128) {
                if (quantize) {
                    // what the cache holds is the rounded row
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = widen2<F16>(o[j]);
                        a[2 * j] = f.x;
                        a[2 * j + 1] = f.y;
                    }
                    const float g = sc && on ? ld_prior(sc + h) : 1.0f;
                    uint32_t sf;
                    const uint32_t codes = quantize_pair(a, g, __fmul_rn(6.0f, g), sf);
                    if (on && rec) {
                        uint8_t* r = rec + (int64_t)h * (p.cache.page_size >> 4) * (18 * D);
                        const int q = li >> 1;
                        const int at = c.kind == 1 ? tok * (D / 2) + 4 * li : rec_vcodes<D>(tok, q) + 4 * (li & 1);
                        *reinterpret_cast<uint32_t*>(r + at) = codes;
                        if (!(li & 1)) r[c.kind == 1 ? rec_kscale<D>(tok, q) : rec_vscale<D>(tok, q)] = (uint8_t)sf;
                    }
                }
            }
        }
    }
}

// The cached rows of slots[t], lanes and warps as above; a lane group fetches kReadUnroll heads' keys
// and values together.
template <int D, bool F16>
__global__ void __launch_bounds__(32 * kReadWarps) k_kv_read(const HeadsParams p) {
    constexpr int LPR = D / 8, RPW = 32 / LPR, STEP = kReadWarps * RPW;
    const int lane = threadIdx.x & 31, li = lane % LPR, q = li >> 1;
    const int64_t t = blockIdx.x;
    const int H = p.cache.heads;
    griddep_wait();
    griddep_launch();
    const int64_t slot = ld_prior(p.slots + t);
    if (slot < 0) return;
    if (slot >= (int64_t)p.cache.num_pages * p.cache.page_size) {
        if (threadIdx.x == 0) report_index(p.err);
        return;
    }
    int64_t page;
    int tok;
    split_slot(p, slot, page, tok);
    const int64_t per_head = (int64_t)(p.cache.page_size >> 4) * (18 * D);
    const uint8_t* rec = p.cache.pages + page * H * per_head + (int64_t)(tok >> 4) * (18 * D);
    tok &= 15;
    const int kat = tok * (D / 2) + 4 * li, vat = rec_vcodes<D>(tok, q) + 4 * (li & 1);
    const int ksat = rec_kscale<D>(tok, q), vsat = rec_vscale<D>(tok, q);
    uint16_t *kb = p.k.p + t * p.k.st + 8 * li, *vb = p.v.p + t * p.v.st + 8 * li;
    auto put = [](uint32_t codes, uint32_t sf, float g, uint16_t* dst) {
        const float d = __fmul_rn(e4m3_value(sf), g);
        float v[8];
        e2m1x8_values(codes, v);
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = narrow2<F16>(__fmul_rn(v[2 * j], d), __fmul_rn(v[2 * j + 1], d));
        *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
    };
    for (int h0 = (threadIdx.x >> 5) * RPW + lane / LPR; h0 < H; h0 += STEP * kReadUnroll) {
        uint32_t kc[kReadUnroll], vc[kReadUnroll], ks[kReadUnroll], vs[kReadUnroll];
        float gk[kReadUnroll], gv[kReadUnroll];
#pragma unroll
        for (int u = 0; u < kReadUnroll; ++u) {
            const int h = min(h0 + u * STEP, H - 1);
            const uint8_t* r = rec + h * per_head;
            kc[u] = *reinterpret_cast<const uint32_t*>(r + kat);
            vc[u] = *reinterpret_cast<const uint32_t*>(r + vat);
            ks[u] = r[ksat];
            vs[u] = r[vsat];
            gk[u] = p.cache.k_scale ? ld_prior(p.cache.k_scale + h) : 1.0f;
            gv[u] = p.cache.v_scale ? ld_prior(p.cache.v_scale + h) : 1.0f;
        }
#pragma unroll
        for (int u = 0; u < kReadUnroll; ++u) {
            const int h = h0 + u * STEP;
            if (h >= H) break;
            put(kc[u], ks[u], gk[u], kb + h * p.k.sh);
            put(vc[u], vs[u], gv[u], vb + h * p.v.sh);
        }
    }
}

template <int D, bool F16>
cudaError_t heads_of(const HeadsParams& p, cudaStream_t s) {
    constexpr int STEP = kWarps * (32 / (D / 8)) * kUnroll;
    Deal d;
    d.q = (p.q.heads + STEP - 1) / STEP;
    d.k = (p.k.heads + STEP - 1) / STEP;
    d.v = (p.v.heads + STEP - 1) / STEP;
    // few tokens: their heads are spread over more CTAs, down to one step each
    const int all = d.q + d.k + d.v;
    const int spread = (int)std::min<int64_t>(all, std::max<int64_t>(1, (int64_t)kSpread * device_sms() / p.T));
    d.steps = (all + spread - 1) / spread;
    const dim3 grid((unsigned)p.T, (all + d.steps - 1) / d.steps), block(32 * kWarps);
    if (p.rot == 0) return launch_pdl(k_heads<D, F16, 0>, grid, block, 0, s, 1, p, d);
    return p.interleaved ? launch_pdl(k_heads<D, F16, 2>, grid, block, 0, s, 1, p, d)
                         : launch_pdl(k_heads<D, F16, 1>, grid, block, 0, s, 1, p, d);
}

template <int D, bool F16>
cudaError_t read_of(const HeadsParams& p, cudaStream_t s) {
    return launch_pdl(k_kv_read<D, F16>, dim3((unsigned)p.T), dim3(32 * kReadWarps), 0, s, 1, p);
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
