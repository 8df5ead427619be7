// Attention of drafted tokens over a paged latent cache (the absorbed form).
//
// The mathematics: with x_t = log2(e) scale q . c_t, out = sum_t 2^(x_t - m) c'_t / sum_t 2^(x_t - m) in one pass
// over the slots, m the largest x_t so far; O and the sum are scaled where m grows.
#include "fa_attention.cuh"
#include "fa_latent.cuh"

using namespace fa_attention;

namespace {

constexpr int ROWS = 8;

// a warp a row: lane's elements 2 lane + 64 k
template <class T> __global__ void __launch_bounds__(ROWS * 32) k_latent_simple(AttendArgs a, int latent) {
    constexpr int K = 9;
    const int lane = threadIdx.x & 31, D = a.c.head_dim, b = blockIdx.y, row = blockIdx.x * ROWS + (threadIdx.x >> 5);
    if (row >= a.rows) return;
    const int ti = row / a.heads, h = row - ti * a.heads;
    Segment s;
    extent(a, b, s.slots, s.use, s.end);
    s.b = b;
    s.head = 0;
    const T *q = (const T *)a.q + b * a.qb + ti * a.qt + h * a.qh;
    float2 x[K], o[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = 2 * lane + 64 * k;
        o[k] = make_float2(0.0f, 0.0f);
        x[k] = i < D ? make_float2(fa_to_f32(q[i]), fa_to_f32(q[i + 1])) : make_float2(0.0f, 0.0f);
    }
    float m = -INFINITY, l = 0.0f;
    const Rows rows(a, s);
    uint32_t sees = 0;
    for (int t = 0; t < s.end && ti < s.use; ++t) {
        if (t % 32 == 0) sees = seen_bits(a, s, ti, t);
        if (!(sees >> (t & 31) & 1)) continue;
        const int64_t at = rows.row((uint32_t)t);
        if (at < 0) continue;
        const T *c = (const T *)a.c.k + at * D;
        float2 y[K];
        float dot = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = 2 * lane + 64 * k;
            y[k] = i < D ? make_float2(fa_to_f32(c[i]), fa_to_f32(c[i + 1])) : make_float2(0.0f, 0.0f);
            dot = fmaf(x[k].x, y[k].x, fmaf(x[k].y, y[k].y, dot));
        }
        dot = fa_warp_sum(dot) * (a.scale * kLog2e);
        const float top = fmaxf(m, dot), f = m == -INFINITY ? 0.0f : ex2(m - top), p = ex2(dot - top);
        m = top;
        l = l * f + p;
#pragma unroll
        for (int k = 0; k < K; ++k) o[k] = make_float2(fmaf(p, y[k].x, o[k].x * f), fmaf(p, y[k].y, o[k].y * f));
    }
    const int64_t to = ((int64_t)b * a.T + ti) * a.heads + h;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = 2 * lane + 64 * k;
        if (i >= latent) continue;
        ((T *)a.out)[to * latent + i] = fa_from_f32<T>(o[k].x * inv);
        ((T *)a.out)[to * latent + i + 1] = fa_from_f32<T>(o[k].y * inv);
    }
    if (a.lse && lane == 0) a.lse[to] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

size_t workspace_bytes(int latent) { return 256; }

fa_status sizes(const char *fn, int32_t B, int32_t T, int32_t heads) {
    if (B < 0 || B > 65535 || T < 0 || T > FA_MAX_DRAFT || heads < 1 || heads > 1024) return fa_refuse(fn, "B, T or heads out of range");
    if ((int64_t)B * std::max(T, 1) * heads > 2147483647) return fa_refuse(fn, "B * T * heads out of range");
    return FA_OK;
}

}  // namespace

extern "C" fa_status fa_latent_attention_workspace_bytes(int32_t B, int32_t T, int32_t heads, int32_t latent_dim,
                                                         int32_t rope_dim, size_t *bytes) {
    const char *fn = "fa_latent_attention_workspace_bytes";
    if (!bytes) return fa_refuse(fn, "NULL argument");
    fa_status st = sizes(fn, B, T, heads);
    if (st != FA_OK) return st;
    if (latent_dim < 128 || latent_dim > 512 || latent_dim % 128 || rope_dim < 16 || rope_dim > 64 || rope_dim % 16)
        return fa_refuse(fn, "latent_dim or rope_dim out of range");
    *bytes = workspace_bytes(latent_dim);
    return FA_OK;
}

extern "C" fa_status fa_latent_attention(const fa_latent_cache *cache, int32_t dtype, int32_t B, int32_t T, int32_t heads,
                                         const void *q, int64_t q_batch_stride, int64_t q_token_stride,
                                         int64_t q_head_stride, const int32_t *page_table, int32_t max_pages,
                                         const int32_t *length, const int32_t *count, const uint64_t *mask, float scale,
                                         void *out, float *lse, void *workspace, size_t ws_bytes, fa_stream stream) {
    const char *fn = "fa_latent_attention";
    AttendArgs a = {};
    fa_status st = fa_view_latent(fn, cache, page_table, max_pages, &a.c);
    if (st != FA_OK) return st;
    if ((st = sizes(fn, B, T, heads)) != FA_OK) return st;
    if (dtype != FA_DTYPE_F16 && dtype != FA_DTYPE_BF16) return fa_refuse(fn, "q must be fp16 or bf16", FA_ERR_UNSUPPORTED);
    if (cache->format != dtype) return fa_refuse(fn, "the cache must have the type of q", FA_ERR_UNSUPPORTED);
    if (!(scale > 0.0f && scale < INFINITY)) return fa_refuse(fn, "scale must be positive and finite");
    const int64_t slots = (int64_t)max_pages << a.c.page_shift;
    if (slots > 2147483647LL - 4096) return fa_refuse(fn, "max_pages * page_size out of range");
    a.rows = T * heads;
    a.blocks = (a.rows + 63) / 64;
    if ((int64_t)B * a.blocks > 2147483647 || (int64_t)B * a.blocks * ((slots + 63) / 64 + 5) > 2147483647)
        return fa_refuse(fn, "B * row blocks * tiles out of range");
    if (B == 0 || T == 0) return FA_OK;
    if (!q || !out || !length) return fa_refuse(fn, "NULL buffer");
    if ((((uintptr_t)q | (uintptr_t)out) & 15) || ((q_batch_stride | q_token_stride | q_head_stride) & 7))
        return fa_refuse(fn, "q and out must be 16-byte aligned, with strides that are multiples of 8");
    const size_t need = workspace_bytes(cache->latent_dim);
    if (ws_bytes < need || !workspace)
        return fa_refuse(fn, ("workspace needs " + std::to_string(need) + " bytes").c_str(), FA_ERR_WORKSPACE_TOO_SMALL);
    if ((uintptr_t)workspace & 255) return fa_refuse(fn, "workspace not 256-byte aligned");
    a.B = B; a.T = T; a.heads = a.group = heads; a.words = (T + 63) / 64;
    a.q = q; a.qb = q_batch_stride; a.qt = q_token_stride; a.qh = q_head_stride;
    a.length = length; a.count = count; a.mask = mask; a.scale = scale; a.out = out; a.lse = lse;
    const dim3 grid((unsigned)((a.rows + ROWS - 1) / ROWS), (unsigned)B);
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == FA_DTYPE_F16) k_latent_simple<__half><<<grid, ROWS * 32, 0, s>>>(a, cache->latent_dim);
    else k_latent_simple<__nv_bfloat16><<<grid, ROWS * 32, 0, s>>>(a, cache->latent_dim);
    return fa_launch_check("latent attention");
}
