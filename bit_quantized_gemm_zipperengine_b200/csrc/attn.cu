// Attention of new tokens over the NVFP4 cache:
//   out = sum_j softmax_j(scale q . K_j) V_j over the cached tokens that a query row sees.
// The floor is the cache's bytes (9/8 D a token and head). One pass: the running maximum m
// and sum l of the softmax are kept, and the sums so far are scaled by 2^(m_old - m_new)
// when the maximum grows. One warp a query row and head; lanes split D.
#include "ops.cuh"

namespace mq {

namespace {

constexpr int kWarps = 4;

template <int D, bool F16>
__global__ void __launch_bounds__(32 * kWarps) k_attn_row(const AttnParams p) {
    constexpr int E = D / 32;  // elements a lane
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t t = unit / p.q.heads;
    const int h = (int)(unit - t * p.q.heads);
    if (t >= p.T) return;
    // the sequence that holds row t
    int b = -1, row0 = 0, n = 1;
    if (p.cu_q) {
        for (int i = 0; i < p.B; ++i) {
            const int lo = __ldg(p.cu_q + i), hi = __ldg(p.cu_q + i + 1);
            if (lo < 0 || hi < lo || hi > p.T) {
                if (lane == 0) report_index(p.err);
                continue;
            }
            if (t >= lo && t < hi) {
                b = i;
                row0 = lo;
                n = hi - lo;
                break;
            }
        }
    } else if (t < p.B) {
        b = (int)t;
        row0 = b;
    }
    if (b < 0) return;
    int64_t len = __ldg(p.kv_len + b);
    if (len < 0 || len > (int64_t)p.max_pages * p.cache.page_size) {
        if (lane == 0) report_index(p.err);
        len = 0;
    }
    const int64_t pos = len - n + (t - row0);
    const int64_t first = p.window > 0 ? max((int64_t)0, pos - p.window + 1) : 0;
    const int kvh = h / (p.q.heads / p.cache.heads), d0 = lane * E;
    const float gk = p.cache.k_scale ? __ldg(p.cache.k_scale + kvh) : 1.0f;
    const float gv = p.cache.v_scale ? __ldg(p.cache.v_scale + kvh) : 1.0f;
    float q[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int j = 0; j < E; j += 2) {
        const float2 f = widen2<F16>(*reinterpret_cast<const uint32_t*>(p.q.p + t * p.q.st + h * p.q.sh + d0 + j));
        q[j] = f.x;
        q[j + 1] = f.y;
        o[j] = o[j + 1] = 0.0f;
    }
    for (int64_t j = first; j <= pos; ++j) {
        const int page = __ldg(p.table + b * p.table_stride + j / p.cache.page_size);
        if (page < 0 || page >= p.cache.num_pages) {
            if (lane == 0) report_index(p.err);
            continue;
        }
        const int in = (int)(j % p.cache.page_size), i = in & 15, g = d0 / 16;
        const uint8_t* rec =
            p.cache.pages + (((int64_t)page * p.cache.heads + kvh) * (p.cache.page_size / 16) + in / 16) * (18 * D);
        // whole words: on this toolchain the E2M1 conversion of a word that was loaded as one
        // or two bytes came out as zeros
        const uint32_t ck = *reinterpret_cast<const uint32_t*>(rec + i * (D / 2) + d0 / 8 * 4) >> (d0 % 8 * 4);
        const uint32_t cv =
            *reinterpret_cast<const uint32_t*>(rec + rec_vcodes<D>(i, g) + (d0 & 15) / 8 * 4) >> (d0 % 8 * 4);
        float k[8], v[8];
        e2m1x8_values(ck, k);
        e2m1x8_values(cv, v);
        const float sk = e4m3_value(rec[rec_kscale<D>(i, g)]), sv = e4m3_value(rec[rec_vscale<D>(i, g)]) * gv;
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = __fmaf_rn(q[e], k[e] * sk, s);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= gk * p.scale;
        const float mn = fmaxf(m, s), c = __expf(m - mn), w = __expf(s - mn);
        l = l * c + w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = __fmaf_rn(w, v[e] * sv, o[e] * c);
        m = mn;
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int j = 0; j < E; j += 2)
        *reinterpret_cast<uint32_t*>(p.o.p + t * p.o.st + h * p.o.sh + d0 + j) = narrow2<F16>(o[j] * inv, o[j + 1] * inv);
    if (p.lse && lane == 0) p.lse[t * p.q.heads + h] = l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t attn_workspace(int, int, int, int, size_t* counters_at) {
    *counters_at = 0;
    return 0;
}

cudaError_t launch_attn(const AttnParams& p, int D, int, bool f16, cudaStream_t s) {
    const int64_t blocks = ((int64_t)p.T * p.q.heads + kWarps - 1) / kWarps;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks), block(32 * kWarps);
    if (D == 64)
        return f16 ? launch_pdl(k_attn_row<64, true>, grid, block, 0, s, 1, p)
                   : launch_pdl(k_attn_row<64, false>, grid, block, 0, s, 1, p);
    return f16 ? launch_pdl(k_attn_row<128, true>, grid, block, 0, s, 1, p)
               : launch_pdl(k_attn_row<128, false>, grid, block, 0, s, 1, p);
}

}  // namespace mq
