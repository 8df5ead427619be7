// Attention of drafted tokens over a paged cache.
#include "fa_lm.cuh"

namespace {

constexpr int NW = 4;

struct AttendArgs {
    fa_cache_view c;
    int format, T, heads, group, words;
    const void *q;
    int64_t qb, qt, qh;
    const int32_t *length, *count;
    const uint64_t *mask;
    float scale;
    void *out;
    float *lse;
};

__device__ __forceinline__ float cached(const void *p, const float *scale, int format, int64_t row, int D, int d) {
    const int64_t at = row * D + d;
    if (format == FA_CACHE_F16) return __half2float(((const __half *)p)[at]);
    if (format == FA_CACHE_BF16) return __bfloat162float(((const __nv_bfloat16 *)p)[at]);
    const uint32_t h = fa_e4m3x2_to_half2(((const uint8_t *)p)[at]);
    return __half2float(__ushort_as_half((unsigned short)(h & 0xffff))) * scale[row];
}

// One block per (sequence, drafted token, query head): every warp walks every fourth slot with
// its own running maximum and sum (lane l holds elements l, l + 32, ...), then the warps' parts
// are joined.
template <class T>
__global__ void __launch_bounds__(32 * NW) k_attend(AttendArgs a) {
    __shared__ float sm[NW], sl[NW], so[NW][128];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = a.c.head_dim;
    const int64_t r = blockIdx.x;
    const int h = (int)(r % a.heads);
    const int64_t bt = r / a.heads;
    const int b = (int)(bt / a.T), t = (int)(bt % a.T), kv = h / a.group;
    const int64_t n = max(a.length[b], 0);
    const int use = a.count ? min(max(a.count[b], 0), a.T) : a.T;
    const T *q = (const T *)a.q + b * a.qb + t * a.qt + h * a.qh;
    float qf[4], o[4] = {0, 0, 0, 0}, m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) qf[i] = lane + 32 * i < D ? fa_to_f32(q[lane + 32 * i]) * a.scale : 0.0f;
    const int64_t end = t < use ? n + use : 0;
    for (int64_t s = warp; s < end; s += NW) {
        if (s >= n && a.mask) {
            const int j = (int)(s - n);
            if (!(a.mask[bt * a.words + j / 64] >> (j % 64) & 1)) continue;
        }
        const int64_t row = a.c.row(b, s, kv);
        if (row < 0) continue;
        float x = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane + 32 * i < D) x += qf[i] * cached(a.c.k, a.c.k_scale, a.format, row, D, lane + 32 * i);
        x = fa_warp_sum(x);
        const float m2 = fmaxf(m, x), w = expf(m - m2), p = expf(x - m2);
        l = l * w + p;
        m = m2;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane + 32 * i < D) o[i] = o[i] * w + p * cached(a.c.v, a.c.v_scale, a.format, row, D, lane + 32 * i);
    }
    if (lane == 0) { sm[warp] = m; sl[warp] = l; }
#pragma unroll
    for (int i = 0; i < 4; ++i) so[warp][lane + 32 * i] = o[i];
    __syncthreads();
    float mm = -INFINITY, ll = 0.0f;
    for (int w = 0; w < NW; ++w) mm = fmaxf(mm, sm[w]);
    float f[NW];
    for (int w = 0; w < NW; ++w) {
        f[w] = sm[w] == -INFINITY ? 0.0f : expf(sm[w] - mm);
        ll += f[w] * sl[w];
    }
    const int d = threadIdx.x;
    if (d < D) {
        float y = 0.0f;
        for (int w = 0; w < NW; ++w)
            if (f[w] > 0.0f) y += f[w] * so[w][d];
        ((T *)a.out)[r * D + d] = fa_from_f32<T>(ll > 0.0f ? y / ll : mm == -INFINITY ? 0.0f : y / ll);
    }
    if (d == 0 && a.lse) a.lse[r] = mm == -INFINITY ? -INFINITY : mm + logf(ll);
}

// two partial results of up to 256 rows for each of 152 blocks
size_t workspace_bytes(int head_dim) { return (size_t)152 * 2 * 256 * ((head_dim <= 64 ? 64 : 128) + 2) * sizeof(float); }

fa_status sizes(const char *fn, int32_t B, int32_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
    if (B < 0 || B > 65535 || T < 0 || T > FA_MAX_DRAFT) return fa_refuse(fn, "B or T out of range");
    if (kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads) return fa_refuse(fn, "q_heads must be a multiple of kv_heads");
    if ((int64_t)B * T * q_heads > 2147483647) return fa_refuse(fn, "B * T * q_heads out of range");
    if (head_dim < 16 || head_dim % 16) return fa_refuse(fn, "head_dim must be a multiple of 16");
    if (head_dim > 128) return fa_refuse(fn, "head_dim above 128", FA_ERR_UNSUPPORTED);
    return FA_OK;
}

}  // namespace

extern "C" fa_status fa_tree_attention_workspace_bytes(int32_t B, int32_t T, int32_t q_heads, int32_t kv_heads,
                                                       int32_t head_dim, size_t *bytes) {
    const char *fn = "fa_tree_attention_workspace_bytes";
    if (!bytes) return fa_refuse(fn, "NULL argument");
    fa_status st = sizes(fn, B, T, q_heads, kv_heads, head_dim);
    if (st != FA_OK) return st;
    *bytes = workspace_bytes(head_dim);
    return FA_OK;
}

extern "C" fa_status fa_tree_attention(const fa_kv_cache *cache, int32_t dtype, int32_t B, int32_t T, int32_t q_heads,
                                       const void *q, int64_t q_batch_stride, int64_t q_token_stride,
                                       int64_t q_head_stride, const int32_t *page_table, int32_t max_pages,
                                       const int32_t *length, const int32_t *count, const uint64_t *mask, float scale,
                                       void *out, float *lse, void *workspace, size_t ws_bytes, fa_stream stream) {
    const char *fn = "fa_tree_attention";
    AttendArgs a;
    fa_status st = fa_view_cache(fn, cache, page_table, max_pages, &a.c);
    if (st != FA_OK) return st;
    if ((st = sizes(fn, B, T, q_heads, cache->kv_heads, cache->head_dim)) != FA_OK) return st;
    if (dtype != FA_DTYPE_F16 && dtype != FA_DTYPE_BF16) return fa_refuse(fn, "q must be fp16 or bf16", FA_ERR_UNSUPPORTED);
    if (cache->format != FA_CACHE_E4M3 && cache->format != dtype)
        return fa_refuse(fn, "a 16-bit cache must have the type of q", FA_ERR_UNSUPPORTED);
    if (B == 0 || T == 0) return FA_OK;
    if (!q || !out || !length) return fa_refuse(fn, "NULL buffer");
    if (((uintptr_t)q | (uintptr_t)out) & 15 || (q_batch_stride | q_token_stride | q_head_stride) & 7)
        return fa_refuse(fn, "q and out must be 16-byte aligned, with strides that are multiples of 8");
    const size_t need = workspace_bytes(cache->head_dim);
    if (ws_bytes < need || !workspace)
        return fa_refuse(fn, ("workspace needs " + std::to_string(need) + " bytes").c_str(), FA_ERR_WORKSPACE_TOO_SMALL);
    if ((uintptr_t)workspace & 255) return fa_refuse(fn, "workspace not 256-byte aligned");
    a.format = cache->format; a.T = T; a.heads = q_heads; a.group = q_heads / cache->kv_heads; a.words = (T + 63) / 64;
    a.q = q; a.qb = q_batch_stride; a.qt = q_token_stride; a.qh = q_head_stride;
    a.length = length; a.count = count; a.mask = mask; a.scale = scale; a.out = out; a.lse = lse;
    const unsigned grid = (unsigned)((int64_t)B * T * q_heads);
    if (dtype == FA_DTYPE_F16) k_attend<__half><<<grid, 32 * NW, 0, (cudaStream_t)stream>>>(a);
    else k_attend<__nv_bfloat16><<<grid, 32 * NW, 0, (cudaStream_t)stream>>>(a);
    return fa_launch_check("tree attention");
}
