// Rotary positions and the paged, quantised key/value cache: writing, reading back, keeping an
// accepted path, and the mask of a draft tree.
#include "fa_lm.cuh"

namespace {

constexpr int NT = 256;

// mscale * (cos, sin) of position t times phase (a 64-bit fraction of a turn): the product wraps
// around at whole turns, so the angle is exact to 2^-32 turn at any position.
__device__ __forceinline__ float2 turn(int32_t t, uint64_t phase, float mscale, bool inverse) {
    const int32_t frac = (int32_t)(uint32_t)(((uint64_t)(int64_t)t * phase) >> 32);
    float s, c;
    sincospif((float)frac * (1.0f / 2147483648.0f), &s, &c);
    return make_float2(mscale * c, mscale * (inverse ? -s : s));
}

// y = R x per pair.  One thread per element, any strides, any sizes.
template <class T>
__global__ void __launch_bounds__(NT) k_rope(int64_t n_tokens, int heads, int dim, int rot, int interleaved, bool inverse,
                                             const T *x, int64_t xt, int64_t xh, const int32_t *__restrict__ pos,
                                             const uint64_t *__restrict__ phase, float mscale, T *out, int64_t ot,
                                             int64_t oh) {
    const int half = rot / 2, per_head = half + (dim - rot);
    const int64_t total = n_tokens * heads * per_head;
    for (int64_t it = (int64_t)blockIdx.x * NT + threadIdx.x; it < total; it += (int64_t)gridDim.x * NT) {
        const int i = (int)(it % per_head);
        const int64_t nh = it / per_head, n = nh / heads;
        const int h = (int)(nh % heads);
        const T *xr = x + n * xt + h * xh;
        T *yr = out + n * ot + h * oh;
        if (i >= half) {
            yr[rot + i - half] = xr[rot + i - half];
            continue;
        }
        const int a = interleaved ? 2 * i : i, b = interleaved ? 2 * i + 1 : i + half;
        const float2 cs = turn(__ldg(pos + n), __ldg(phase + i), mscale, inverse);
        const float x0 = fa_to_f32(xr[a]), x1 = fa_to_f32(xr[b]);
        yr[a] = fa_from_f32<T>(x0 * cs.x - x1 * cs.y);
        yr[b] = fa_from_f32<T>(x0 * cs.y + x1 * cs.x);
    }
}

struct WriteArgs {
    fa_cache_view c;
    int format, B, T;
    const void *k, *v;
    int64_t kb, kt, kh, vb, vt, vh;
    const int32_t *start, *count, *pos;
    const uint64_t *phase;
    int rot, interleaved;
    float mscale;
};

// One warp per (token, head): the key's row, then the value's.  Lane l holds elements l, l + 32, ...
template <class T>
__global__ void __launch_bounds__(NT) k_cache_write(WriteArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * (NT / 32) + (threadIdx.x >> 5);
    const int H = a.c.kv_heads, D = a.c.head_dim;
    if (w >= (int64_t)a.B * a.T * H) return;
    const int h = (int)(w % H);
    const int64_t bt = w / H;
    const int b = (int)(bt / a.T), t = (int)(bt % a.T);
    if (a.count && t >= a.count[b]) return;
    const int64_t row = a.c.row(b, (int64_t)a.start[b] + t, h);
    if (row < 0) return;
    for (int side = 0; side < 2; ++side) {
        const T *x = side ? (const T *)a.v + b * a.vb + t * a.vt + h * a.vh : (const T *)a.k + b * a.kb + t * a.kt + h * a.kh;
        float f[8], amax = 0.0f;
        bool odd = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int d = lane + 32 * i;
            if (d >= D) { f[i] = 0.0f; continue; }
            f[i] = fa_to_f32(x[d]);
            if (!side && a.pos && d < a.rot) {
                const int half = a.rot / 2;
                const int pair = a.interleaved ? d / 2 : d % half;
                const bool second = a.interleaved ? d & 1 : d >= half;
                const int mate = a.interleaved ? d ^ 1 : (second ? d - half : d + half);
                const float2 cs = turn(a.pos[bt], a.phase[pair], a.mscale, false);
                const float y = fa_to_f32(x[mate]);
                f[i] = second ? y * cs.y + f[i] * cs.x : f[i] * cs.x - y * cs.y;
            }
            odd |= !isfinite(f[i]);
            amax = fmaxf(amax, fabsf(f[i]));
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        odd = __any_sync(0xffffffffu, odd);
        const float scale = odd ? __int_as_float(0x7fffffff) : amax / FA_E4M3_MAX;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int d = lane + 32 * i;
            if (d >= D) continue;
            const int64_t at = row * D + d;
            void *dst = side ? a.c.v : a.c.k;
            if (a.format == FA_CACHE_E4M3)
                ((uint8_t *)dst)[at] = odd || scale == 0.0f ? 0 : (uint8_t)fa_to_e4m3x2(f[i] / scale, 0.0f);
            else if (a.format == FA_CACHE_F16)
                ((__half *)dst)[at] = __float2half_rn(f[i]);
            else
                ((__nv_bfloat16 *)dst)[at] = __float2bfloat16_rn(f[i]);
        }
        if (a.format == FA_CACHE_E4M3 && lane == 0) (side ? a.c.v_scale : a.c.k_scale)[row] = scale;
    }
}

__device__ __forceinline__ float cached(const void *p, const float *scale, int format, int64_t row, int D, int d) {
    const int64_t at = row * D + d;
    if (format == FA_CACHE_F16) return __half2float(((const __half *)p)[at]);
    if (format == FA_CACHE_BF16) return __bfloat162float(((const __nv_bfloat16 *)p)[at]);
    const uint32_t h = fa_e4m3x2_to_half2(((const uint8_t *)p)[at]);
    return __half2float(__ushort_as_half((unsigned short)(h & 0xffff))) * scale[row];
}

template <class T>
__global__ void __launch_bounds__(NT) k_cache_read(fa_cache_view c, int format, int B, int N, const int32_t *length, T *k, T *v) {
    const int H = c.kv_heads, D = c.head_dim;
    const int64_t total = (int64_t)B * N * H * D;
    for (int64_t it = (int64_t)blockIdx.x * NT + threadIdx.x; it < total; it += (int64_t)gridDim.x * NT) {
        const int d = (int)(it % D);
        const int64_t r = it / D;
        const int h = (int)(r % H);
        const int64_t bt = r / H;
        const int b = (int)(bt / N), t = (int)(bt % N);
        const int64_t row = t < length[b] ? c.row(b, t, h) : -1;
        k[it] = row < 0 ? fa_from_f32<T>(0.0f) : fa_from_f32<T>(cached(c.k, c.k_scale, format, row, D, d));
        v[it] = row < 0 ? fa_from_f32<T>(0.0f) : fa_from_f32<T>(cached(c.v, c.v_scale, format, row, D, d));
    }
}

// One block per (sequence, head).  A thread moves the same 16 bytes of every kept row, in order:
// path[i] >= i, so a row still to be read is never one that was written.
__global__ void __launch_bounds__(64) k_cache_keep(fa_cache_view c, int es, int P, const int32_t *length, const int32_t *path) {
    const int b = blockIdx.x / c.kv_heads, h = blockIdx.x % c.kv_heads;
    const int chunks = c.head_dim * es / 16, tid = threadIdx.x;
    const int64_t n = length[b];
    if (n < 0) return;
    int last = -1;
    for (int i = 0; i < P; ++i) {
        const int j = path[(int64_t)b * P + i];
        if (j <= last) return;   // the path's end, or one that does not ascend
        last = j;
        if (j == i) continue;
        const int64_t from = c.row(b, n + j, h), to = c.row(b, n + i, h);
        if (from < 0 || to < 0) return;
        for (int q = tid; q < 2 * chunks; q += 64) {
            uint4 *p = (uint4 *)(q < chunks ? c.k : c.v);
            p[to * chunks + q % chunks] = p[from * chunks + q % chunks];
        }
        if (c.k_scale && tid < 2) {
            float *p = tid ? c.v_scale : c.k_scale;
            p[to] = p[from];
        }
    }
}

// One block per sequence, one thread per drafted token: walk up the ancestors, which come in
// descending order, and store each 64-bit word when the walk leaves it.
__global__ void k_tree_mask(int T, const int32_t *__restrict__ parents, uint64_t *mask, int32_t *depth) {
    __shared__ int32_t par[FA_MAX_DRAFT];
    const int words = (T + 63) / 64;
    const int64_t b = blockIdx.x;
    for (int j = threadIdx.x; j < T; j += blockDim.x) par[j] = parents[b * T + j];
    __syncthreads();
    for (int j = threadIdx.x; j < T; j += blockDim.x) {
        uint64_t *m = mask + (b * T + j) * words;
        int w = words - 1, at = j, n = 0;
        uint64_t bits = 0;
        while (true) {
            while (w > at / 64) { m[w--] = bits; bits = 0; }
            bits |= 1ull << (at % 64);
            const int up = par[at];
            if (up < 0 || up >= at) break;
            at = up;
            ++n;
        }
        for (; w >= 0; --w) { m[w] = bits; bits = 0; }
        if (depth) depth[b * T + j] = n;
    }
}

unsigned blocks_for(int64_t items) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>((items + NT - 1) / NT, 152 * 16)); }

fa_status rope_args(const char *fn, int32_t head_dim, int32_t rot_dim, int32_t interleaved) {
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 2) return fa_refuse(fn, "rot_dim must be even and in [0, head_dim]");
    if (interleaved != 0 && interleaved != 1) return fa_refuse(fn, "interleaved must be 0 or 1");
    return FA_OK;
}

}  // namespace

extern "C" fa_status fa_rope(int32_t dtype, int64_t n_tokens, int32_t n_heads, int32_t head_dim, int32_t rot_dim,
                             int32_t interleaved, int32_t inverse, const void *x, int64_t x_token_stride,
                             int64_t x_head_stride, const int32_t *positions, const uint64_t *phase, float mscale,
                             void *out, int64_t out_token_stride, int64_t out_head_stride, fa_stream stream) {
    const char *fn = "fa_rope";
    if (!fa_dtype_ok(dtype)) return fa_refuse(fn, "unknown dtype");
    if (n_tokens < 0 || n_heads < 0 || head_dim < 1 || head_dim > 1024) return fa_refuse(fn, "sizes out of range");
    fa_status st = rope_args(fn, head_dim, rot_dim, interleaved);
    if (st != FA_OK) return st;
    if (n_tokens == 0 || n_heads == 0) return FA_OK;
    if (!x || !out || (rot_dim > 0 && (!positions || !phase))) return fa_refuse(fn, "NULL buffer");
    cudaStream_t s = (cudaStream_t)stream;
    const int64_t items = n_tokens * n_heads * (head_dim - rot_dim / 2);
    auto go = [&](auto tag) {
        using T = decltype(tag);
        k_rope<T><<<blocks_for(items), NT, 0, s>>>(n_tokens, n_heads, head_dim, rot_dim, interleaved, inverse != 0,
                                                   (const T *)x, x_token_stride, x_head_stride, positions, phase, mscale,
                                                   (T *)out, out_token_stride, out_head_stride);
    };
    if (dtype == FA_DTYPE_F32) go(0.0f);
    else if (dtype == FA_DTYPE_F16) go(__half());
    else go(__nv_bfloat16());
    return fa_launch_check("rope");
}

extern "C" fa_status fa_cache_write(const fa_kv_cache *cache, int32_t dtype, int32_t B, int32_t T, const void *k,
                                    int64_t k_batch_stride, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                                    int64_t v_batch_stride, int64_t v_token_stride, int64_t v_head_stride,
                                    const int32_t *page_table, int32_t max_pages, const int32_t *start,
                                    const int32_t *count, const int32_t *positions, const uint64_t *phase,
                                    int32_t rot_dim, int32_t interleaved, float mscale, fa_stream stream) {
    const char *fn = "fa_cache_write";
    WriteArgs a;
    fa_status st = fa_view_cache(fn, cache, page_table, max_pages, &a.c);
    if (st != FA_OK) return st;
    if (!fa_dtype_ok(dtype)) return fa_refuse(fn, "unknown dtype");
    if (B < 0 || T < 0) return fa_refuse(fn, "B or T negative");
    if ((positions == nullptr) != (phase == nullptr)) return fa_refuse(fn, "positions and phase go together");
    if (positions && (st = rope_args(fn, cache->head_dim, rot_dim, interleaved)) != FA_OK) return st;
    if (B == 0 || T == 0) return FA_OK;
    if (!k || !v || !start) return fa_refuse(fn, "NULL buffer");
    a.format = cache->format; a.B = B; a.T = T;
    a.k = k; a.v = v;
    a.kb = k_batch_stride; a.kt = k_token_stride; a.kh = k_head_stride;
    a.vb = v_batch_stride; a.vt = v_token_stride; a.vh = v_head_stride;
    a.start = start; a.count = count; a.pos = positions; a.phase = phase;
    a.rot = positions ? rot_dim : 0; a.interleaved = interleaved; a.mscale = mscale;
    const int64_t warps = (int64_t)B * T * cache->kv_heads;
    if (warps > (int64_t)2147483647) return fa_refuse(fn, "B * T * kv_heads out of range");
    const unsigned grid = (unsigned)((warps + NT / 32 - 1) / (NT / 32));
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == FA_DTYPE_F32) k_cache_write<float><<<grid, NT, 0, s>>>(a);
    else if (dtype == FA_DTYPE_F16) k_cache_write<__half><<<grid, NT, 0, s>>>(a);
    else k_cache_write<__nv_bfloat16><<<grid, NT, 0, s>>>(a);
    return fa_launch_check("cache write");
}

extern "C" fa_status fa_cache_read(const fa_kv_cache *cache, int32_t dtype, int32_t B, int32_t N,
                                   const int32_t *page_table, int32_t max_pages, const int32_t *length, void *k_out,
                                   void *v_out, fa_stream stream) {
    const char *fn = "fa_cache_read";
    fa_cache_view c;
    fa_status st = fa_view_cache(fn, cache, page_table, max_pages, &c);
    if (st != FA_OK) return st;
    if (!fa_dtype_ok(dtype)) return fa_refuse(fn, "unknown dtype");
    if (B < 0 || N < 0) return fa_refuse(fn, "B or N negative");
    if (B == 0 || N == 0) return FA_OK;
    if (!length || !k_out || !v_out) return fa_refuse(fn, "NULL buffer");
    if (((uintptr_t)k_out | (uintptr_t)v_out) & 15) return fa_refuse(fn, "outputs must be 16-byte aligned");
    const int64_t items = (int64_t)B * N * cache->kv_heads * cache->head_dim;
    cudaStream_t s = (cudaStream_t)stream;
    auto go = [&](auto tag) {
        using T = decltype(tag);
        k_cache_read<T><<<blocks_for(items), NT, 0, s>>>(c, cache->format, B, N, length, (T *)k_out, (T *)v_out);
    };
    if (dtype == FA_DTYPE_F32) go(0.0f);
    else if (dtype == FA_DTYPE_F16) go(__half());
    else go(__nv_bfloat16());
    return fa_launch_check("cache read");
}

extern "C" fa_status fa_cache_keep(const fa_kv_cache *cache, int32_t B, int32_t P, const int32_t *page_table,
                                   int32_t max_pages, const int32_t *length, const int32_t *path, fa_stream stream) {
    const char *fn = "fa_cache_keep";
    fa_cache_view c;
    fa_status st = fa_view_cache(fn, cache, page_table, max_pages, &c);
    if (st != FA_OK) return st;
    if (B < 0 || P < 0 || (int64_t)B * cache->kv_heads > 2147483647) return fa_refuse(fn, "B or P out of range");
    if (B == 0 || P == 0) return FA_OK;
    if (!length || !path) return fa_refuse(fn, "NULL buffer");
    k_cache_keep<<<(unsigned)(B * cache->kv_heads), 64, 0, (cudaStream_t)stream>>>(
        c, cache->format == FA_CACHE_E4M3 ? 1 : 2, P, length, path);
    return fa_launch_check("cache keep");
}

extern "C" fa_status fa_tree_mask(int32_t B, int32_t T, const int32_t *parents, uint64_t *mask, int32_t *depth,
                                  fa_stream stream) {
    const char *fn = "fa_tree_mask";
    if (B < 0 || T < 0 || T > FA_MAX_DRAFT) return fa_refuse(fn, "B or T out of range");
    if (B == 0 || T == 0) return FA_OK;
    if (!parents || !mask) return fa_refuse(fn, "NULL buffer");
    k_tree_mask<<<(unsigned)B, (unsigned)std::min(256, (T + 31) / 32 * 32), 0, (cudaStream_t)stream>>>(T, parents, mask, depth);
    return fa_launch_check("tree mask");
}
