// Host side of mosaic_ops.h: argument validation and dispatch.
#include <cmath>
#include <cstring>

#include "ops.cuh"

using namespace mq;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A [tokens][heads][D] operand; rows of an output must not overlap.
bool heads_ok(const mq_heads* h, int T, int D, bool output) {
    if (!h || !h->data || !aligned(h->data, 16) || h->heads <= 0 || h->heads > (1 << 20)) return false;
    if (h->token_stride < 0 || h->head_stride < 0 || h->token_stride % 8 || h->head_stride % 8) return false;
    if (!output || T <= 0) return true;
    // one axis inside the other: its rows side by side, and all of them before the next one's
    const int64_t n[2] = {T, h->heads}, s[2] = {T > 1 ? h->token_stride : INT64_MAX, h->heads > 1 ? h->head_stride : INT64_MAX};
    const int in = s[0] < s[1] ? 0 : 1, out = 1 - in;
    return (n[in] == 1 || s[in] >= D) && (n[out] == 1 || (s[out] - D) / (n[in] - 1) >= s[in]);
}

HeadsView view(const mq_heads* h) {
    if (!h) return HeadsView{nullptr, 0, 0, 0};
    return HeadsView{static_cast<uint16_t*>(h->data), (int)h->heads, h->token_stride, h->head_stride};
}

bool cache_ok(const mq_kv_cache* c) {
    return c && c->pages && aligned(c->pages, 128) && mq_kv_cache_bytes(c->num_pages, c->page_size, c->heads, c->D) > 0;
}

CacheView view(const mq_kv_cache* c) {
    if (!c) return CacheView{nullptr, 0, 0, 0, 0, nullptr, nullptr};
    return CacheView{c->pages, c->num_pages, c->page_size, c->heads, c->D, c->k_scale, c->v_scale};
}

bool type_ok(mq_dtype t) { return t == MQ_BF16 || t == MQ_F16; }

cudaStream_t as_stream(mq_stream s) { return reinterpret_cast<cudaStream_t>(s); }

// The rotation's and the norms' arguments.
bool turn_ok(int D, const void* qw, const void* kw, float eps, const int64_t* pos, const double* freq, int rot) {
    if (rot < 0 || rot > D || rot % 16 || (rot > 0 && (!pos || !freq))) return false;
    if ((qw && !aligned(qw, 16)) || (kw && !aligned(kw, 16))) return false;
    return eps >= 0.0f && std::isfinite(eps);
}

}  // namespace

extern "C" {

size_t mq_kv_cache_bytes(int num_pages, int page_size, int heads, int D) {
    if (num_pages <= 0 || page_size <= 0 || page_size % 16 || heads <= 0 || (D != 64 && D != 128)) return 0;
    return (size_t)num_pages * (size_t)heads * (size_t)(page_size / 16) * (size_t)(18 * D);
}

size_t mq_gemv_workspace_bytes(int M, int K) {
    if (M <= 0 || M > 16 || K <= 0 || K % 64) return 0;
    return gemv_workspace(M, K);
}

mq_status mq_gemv(const void* X, mq_dtype type, int64_t ldx, const mq_nvfp4_mat* wq, const mq_residual_packed* r,
                  void* Y, int64_t ldy, int M, int N, int K, unsigned flags, void* ws, size_t ws_bytes, mq_stream stream) {
    if (!X || !wq || !Y || !type_ok(type) || M <= 0 || N <= 0 || K <= 0 || N % 64 || K % 64) return MQ_ERR_INVALID_ARG;
    if (flags & ~(unsigned)(MQ_GEMM_BASE_ONLY | MQ_GEMM_RESIDUAL_ONLY | MQ_GEMM_WEIGHTS_READY)) return MQ_ERR_INVALID_ARG;
    if ((flags & MQ_GEMM_BASE_ONLY) && (flags & MQ_GEMM_RESIDUAL_ONLY)) return MQ_ERR_INVALID_ARG;
    if (!wq->codes || !wq->sf_swz || !wq->gscale || wq->rows != N || wq->cols != K) return MQ_ERR_INVALID_ARG;
    if (!aligned(X, 16) || !aligned(Y, 2) || !aligned(wq->codes, 16) || !aligned(wq->sf_swz, 16)) return MQ_ERR_INVALID_ARG;
    if (M > 1 && (ldx < K || ldx % 8 || ldy < N)) return MQ_ERR_INVALID_ARG;
    if (r && r->nblk > 0) {
        if (r->N != N || r->K != K || !r->blk_codes || !r->blk_sf || !r->blk_kt || !r->tile_ptr) return MQ_ERR_INVALID_ARG;
        if (!aligned(r->blk_codes, 16) || !aligned(r->blk_sf, 16)) return MQ_ERR_INVALID_ARG;
    }
    if (M > 16 || N / 64 > 65535) return MQ_ERR_UNSUPPORTED_SHAPE;  // a grid's second axis counts the row tiles
    if (!ws || ws_bytes < mq_gemv_workspace_bytes(M, K) || !aligned(ws, 16)) return MQ_ERR_WORKSPACE;
    const bool has_r = r && r->nblk > 0 && !(flags & MQ_GEMM_BASE_ONLY);
    GemvParams p;
    memset(&p, 0, sizeof p);
    p.X = static_cast<const uint16_t*>(X);
    p.ldx = M > 1 ? ldx : 0;
    p.codes = wq->codes;
    p.sf = wq->sf_swz;
    p.g_w = wq->gscale;
    if (has_r) {
        p.blk_codes = r->blk_codes;
        p.blk_sf = r->blk_sf;
        p.blk_kt = r->blk_kt;
        p.tile_ptr = r->tile_ptr;
        p.nblk = r->nblk;
    }
    p.Y = static_cast<uint16_t*>(Y);
    p.ldy = M > 1 ? ldy : 0;
    p.M = M;
    p.N = N;
    p.K = K;
    p.base = (flags & MQ_GEMM_RESIDUAL_ONLY) ? 0 : 1;
    p.xop = static_cast<uint8_t*>(ws);
    p.err = device_error_word();
    CUtensorMap tw;
    if (!p.err || !tensor_map_w64(&tw, wq->codes, (uint64_t)K / 2, (uint64_t)N)) return MQ_ERR_CUDA;
    return count_launches(launch_gemv(tw, p, type == MQ_F16, as_stream(stream)), 2);
}

// q, k, v, q_out, k_out, slots and cache as the entry points say; absent ones are null.
static mq_status heads_impl(const mq_heads* q, const mq_heads* k, const mq_heads* v, const mq_heads* q_out,
                            const mq_heads* k_out, int T, int D, mq_dtype type, const void* qw, const void* kw,
                            float eps, const int64_t* pos, const double* freq, int rot, int interleaved,
                            const int64_t* slots, const mq_kv_cache* cache, mq_stream stream) {
    if (T == 0) return MQ_OK;
    if ((q && (!heads_ok(q, T, D, false) || !heads_ok(q_out, T, D, true) || q_out->heads != q->heads)) ||
        (k && (!heads_ok(k, T, D, false) || (k_out && (!heads_ok(k_out, T, D, true) || k_out->heads != k->heads)))) ||
        (v && !heads_ok(v, T, D, false)))
        return MQ_ERR_INVALID_ARG;
    if (!turn_ok(D, qw, kw, eps, pos, freq, rot)) return MQ_ERR_INVALID_ARG;
    if (cache && (!slots || k->heads != cache->heads || v->heads != cache->heads)) return MQ_ERR_INVALID_ARG;
    HeadsParams p;
    memset(&p, 0, sizeof p);
    p.q = view(q);
    p.k = view(k);
    p.v = view(v);
    p.qo = view(q ? q_out : nullptr);
    p.ko = view(k ? k_out : nullptr);
    p.T = T;
    p.wq = q ? static_cast<const uint16_t*>(qw) : nullptr;
    p.wk = k ? static_cast<const uint16_t*>(kw) : nullptr;
    p.eps = eps;
    p.pos = pos;
    p.freq = freq;
    p.rot = rot;
    p.interleaved = interleaved ? 1 : 0;
    p.slots = slots;
    p.cache = view(cache);
    p.by_page = FastDiv(cache ? cache->page_size : 1);
    p.err = device_error_word();
    if (!p.err) return MQ_ERR_CUDA;
    return count_launches(launch_heads(p, D, type == MQ_F16, as_stream(stream)), 1);
}

mq_status mq_qk_norm_rope(const mq_heads* q, const mq_heads* k, const mq_heads* q_out, const mq_heads* k_out, int T,
                          int D, mq_dtype type, const void* q_weight, const void* k_weight, float eps,
                          const int64_t* pos, const double* freq, int rot, int interleaved, mq_stream stream) {
    if (!type_ok(type) || T < 0 || (D != 64 && D != 128 && D != 256) || (!q && !k) || !q != !q_out || !k != !k_out)
        return MQ_ERR_INVALID_ARG;
    return heads_impl(q, k, nullptr, q_out, k_out, T, D, type, q_weight, k_weight, eps, pos, freq, rot, interleaved,
                      nullptr, nullptr, stream);
}

mq_status mq_kv_append(const mq_heads* k, const mq_heads* v, int T, mq_dtype type, const int64_t* slots,
                       const mq_kv_cache* cache, mq_stream stream) {
    if (!k || !v || !type_ok(type) || T < 0 || !cache_ok(cache)) return MQ_ERR_INVALID_ARG;
    return heads_impl(nullptr, k, v, nullptr, nullptr, T, cache->D, type, nullptr, nullptr, 0.0f, nullptr, nullptr, 0,
                      0, slots, cache, stream);
}

mq_status mq_qkv_append(const mq_heads* q, const mq_heads* k, const mq_heads* v, const mq_heads* q_out,
                        const mq_heads* k_out, int T, mq_dtype type, const void* q_weight, const void* k_weight,
                        float eps, const int64_t* pos, const double* freq, int rot, int interleaved,
                        const int64_t* slots, const mq_kv_cache* cache, mq_stream stream) {
    if (!q || !k || !v || !q_out || !type_ok(type) || T < 0 || !cache_ok(cache)) return MQ_ERR_INVALID_ARG;
    return heads_impl(q, k, v, q_out, k_out, T, cache->D, type, q_weight, k_weight, eps, pos, freq, rot, interleaved,
                      slots, cache, stream);
}

mq_status mq_kv_read(const mq_kv_cache* cache, const int64_t* slots, int T, const mq_heads* k, const mq_heads* v,
                     mq_dtype type, mq_stream stream) {
    if (!k || !v || !type_ok(type) || T < 0 || !cache_ok(cache)) return MQ_ERR_INVALID_ARG;
    if (T == 0) return MQ_OK;
    if (!slots || !heads_ok(k, T, cache->D, true) || !heads_ok(v, T, cache->D, true)) return MQ_ERR_INVALID_ARG;
    if (k->heads != cache->heads || v->heads != cache->heads) return MQ_ERR_INVALID_ARG;
    HeadsParams p;
    memset(&p, 0, sizeof p);
    p.k = view(k);
    p.v = view(v);
    p.T = T;
    p.slots = slots;
    p.cache = view(cache);
    p.by_page = FastDiv(cache ? cache->page_size : 1);
    p.err = device_error_word();
    if (!p.err) return MQ_ERR_CUDA;
    return count_launches(launch_kv_read(p, cache->D, type == MQ_F16, as_stream(stream)), 1);
}

size_t mq_kv_attention_workspace_bytes(int q_heads, int kv_heads, int D, int max_q) {
    if (q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads || (D != 64 && D != 128) || max_q <= 0) return 0;
    size_t at;
    return attn_workspace(q_heads, kv_heads, D, max_q, &at);
}

mq_status mq_kv_attention(const mq_heads* q, const mq_heads* out, float* lse, int T, mq_dtype type,
                          const mq_kv_cache* cache, const int32_t* block_table, int64_t table_stride, int max_pages,
                          int B, const int32_t* cu_q, int max_q, const int32_t* kv_len, float scale, int window,
                          void* ws, size_t ws_bytes, mq_stream stream) {
    if (!type_ok(type) || T < 0 || B < 0 || max_q <= 0 || window < 0 || !std::isfinite(scale) || !cache_ok(cache))
        return MQ_ERR_INVALID_ARG;
    if (T == 0 || B == 0) return MQ_OK;
    const int D = cache->D;
    if (!heads_ok(q, T, D, false) || !heads_ok(out, T, D, true) || out->heads != q->heads || out->data == q->data)
        return MQ_ERR_INVALID_ARG;
    if (q->heads % cache->heads || !block_table || !kv_len || max_pages <= 0 || (B > 1 && table_stride < max_pages))
        return MQ_ERR_INVALID_ARG;
    if (!cu_q && T != B) return MQ_ERR_INVALID_ARG;
    if ((int64_t)T * (q->heads / cache->heads) > (1 << 30)) return MQ_ERR_UNSUPPORTED_SHAPE;  // rows are counted in 32 bits
    size_t partials_at;
    const size_t need = attn_workspace((int)q->heads, cache->heads, D, max_q, &partials_at);
    if (!ws || ws_bytes < need || !aligned(ws, 16)) return MQ_ERR_WORKSPACE;
    AttnParams p;
    memset(&p, 0, sizeof p);
    p.q = view(q);
    p.o = view(out);
    p.lse = lse;
    p.T = T;
    p.cache = view(cache);
    p.table = block_table;
    p.table_stride = table_stride;
    p.max_pages = max_pages;
    p.B = B;
    p.cu_q = cu_q;
    p.kv_len = kv_len;
    p.scale = scale;
    // from the longest length on a window holds everything (and the kernel's sums stay in 32 bits)
    p.window = window < (1 << 30) ? window : 0;
    p.counters = static_cast<int*>(ws);
    p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + partials_at);
    p.err = device_error_word();
    if (!p.err) return MQ_ERR_CUDA;
    int kernels = 1;
    const cudaError_t e = launch_attn(p, D, max_q, type == MQ_F16, as_stream(stream), &kernels);
    return count_launches(e, kernels);
}

}  // extern "C"
