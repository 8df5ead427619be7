// What the model-side operators share: element types, 16-byte vectors of them, argument checks
// and the slots of a paged cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "fa_internal.cuh"

template <class T> struct fa_vec { static constexpr int N = 16 / (int)sizeof(T); };

__device__ __forceinline__ float fa_to_f32(float x) { return x; }
__device__ __forceinline__ float fa_to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float fa_to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T> __device__ __forceinline__ T fa_from_f32(float x);
template <> __device__ __forceinline__ float fa_from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __half fa_from_f32<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 fa_from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// the elements of 16 bytes as floats, and back
__device__ __forceinline__ void fa_unpack(uint4 r, float (&f)[4], float) {
    f[0] = __uint_as_float(r.x); f[1] = __uint_as_float(r.y); f[2] = __uint_as_float(r.z); f[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void fa_unpack(uint4 r, float (&f)[8], __half) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __half2 h;
        memcpy(&h, &w[i], 4);
        const float2 p = __half22float2(h);
        f[2 * i] = p.x; f[2 * i + 1] = p.y;
    }
}
__device__ __forceinline__ void fa_unpack(uint4 r, float (&f)[8], __nv_bfloat16) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 fa_pack(const float (&f)[4], float) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint32_t fa_pack2(float a, float b, __half) {
    const __half2 h = __floats2half2_rn(a, b);
    uint32_t u;
    memcpy(&u, &h, 4);
    return u;
}
__device__ __forceinline__ uint32_t fa_pack2(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    uint32_t u;
    memcpy(&u, &h, 4);
    return u;
}
template <class T> __device__ __forceinline__ uint4 fa_pack(const float (&f)[8], T t) {
    return make_uint4(fa_pack2(f[0], f[1], t), fa_pack2(f[2], f[3], t), fa_pack2(f[4], f[5], t), fa_pack2(f[6], f[7], t));
}

// two e4m3 codes (low byte first) as two halves, exactly
__device__ __forceinline__ uint32_t fa_e4m3x2_to_half2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return h;
}
// two floats as e4m3 codes, nearest even, saturating (low byte = a)
__device__ __forceinline__ uint32_t fa_to_e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// mscale * (cos, sin) of position t times phase (a 64-bit fraction of a turn): the product wraps around at
// whole turns whatever the position, and its upper 32 bits, rounded to fp32, are the angle: off by up to 2^-26
// turn (a tenth of a millionth of a radian), where fp32's own sines and products are off by as much.
__device__ __forceinline__ float2 fa_turn(int32_t t, uint64_t phase, float mscale, bool inverse) {
    const int32_t frac = (int32_t)(uint32_t)(((uint64_t)(int64_t)t * phase) >> 32);
    float s, c;
    sincospif((float)frac * (1.0f / 2147483648.0f), &s, &c);
    return make_float2(mscale * c, mscale * (inverse ? -s : s));
}

#define FA_E4M3_MAX 448.0f

// A paged cache as kernels see it.  Rows are (page, head, place); row r starts at element
// r * head_dim of k and v and has the scales k_scale[r], v_scale[r].
struct fa_cache_view {
    void *k, *v;
    float *k_scale, *v_scale;
    int32_t n_pages, page_shift, kv_heads, head_dim;
    const int32_t *page_table;
    int32_t max_pages;

    // the row of sequence b's slot and head h, or -1 when no page holds it
    __device__ __forceinline__ int64_t row(int b, int64_t slot, int h) const {
        const int64_t p = slot >> page_shift;
        if (slot < 0 || p >= max_pages) return -1;
        const int page = __ldg(page_table + (int64_t)b * max_pages + p);
        if ((unsigned)page >= (unsigned)n_pages) return -1;
        return (((int64_t)page * kv_heads + h) << page_shift) + (slot & ((1 << page_shift) - 1));
    }
};

// A second kernel of an operator is launched while the first one runs: the first allows it when it
// starts, the second waits for all of the first's results.
__device__ __forceinline__ void fa_let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void fa_wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ----------------------------------------------------------------------------- host side

// launch a kernel that calls fa_wait_for_previous() before it touches what the stream's last kernel writes
template <class... P, class... A>
fa_status fa_launch_second(const char *what, void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = dim3(block);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = at;
    c.numAttrs = 1;
    (void)cudaLaunchKernelEx(&c, kernel, args...);   // its error is the one the check reads
    return fa_launch_check(what);
}

inline fa_status fa_refuse(const char *fn, const char *why, fa_status st = FA_ERR_INVALID_ARG) {
    fa_set_error(std::string(fn) + ": " + why);
    return st;
}

inline bool fa_overlap(const void *x, size_t x_bytes, const void *y, size_t y_bytes) {
    return (uintptr_t)x < (uintptr_t)y + y_bytes && (uintptr_t)y < (uintptr_t)x + x_bytes;
}

inline bool fa_dtype_ok(int32_t dtype) { return dtype >= FA_DTYPE_F32 && dtype <= FA_DTYPE_BF16; }
inline int fa_dtype_bytes(int32_t dtype) { return dtype == FA_DTYPE_F32 ? 4 : 2; }

// checks a cache's description and makes the kernels' view of it
inline fa_status fa_view_cache(const char *fn, const fa_kv_cache *c, const int32_t *page_table, int32_t max_pages,
                               fa_cache_view *out) {
    if (!c) return fa_refuse(fn, "NULL cache");
    if (c->format != FA_CACHE_F16 && c->format != FA_CACHE_BF16 && c->format != FA_CACHE_E4M3)
        return fa_refuse(fn, "unknown cache format");
    if (c->n_pages < 0 || c->kv_heads < 1 || c->kv_heads > 65535) return fa_refuse(fn, "cache pages or heads out of range");
    if (c->page_size < 1 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
        return fa_refuse(fn, "page_size must be a power of two in [1, 1024]");
    if (c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16)
        return fa_refuse(fn, "head_dim must be a multiple of 16 in [16, 256]");
    if (max_pages < 0) return fa_refuse(fn, "max_pages < 0");
    if (c->n_pages > 0 && (!c->k || !c->v)) return fa_refuse(fn, "NULL cache buffer");
    if (((uintptr_t)c->k | (uintptr_t)c->v) & 15) return fa_refuse(fn, "cache buffers must be 16-byte aligned");
    if (c->format == FA_CACHE_E4M3 && c->n_pages > 0 && (!c->k_scale || !c->v_scale))
        return fa_refuse(fn, "an 8-bit cache needs k_scale and v_scale");
    if (max_pages > 0 && !page_table) return fa_refuse(fn, "NULL page_table");
    int shift = 0;
    while ((1 << shift) < c->page_size) ++shift;
    *out = fa_cache_view{c->k, c->v, c->k_scale, c->v_scale, c->n_pages, shift, c->kv_heads, c->head_dim, page_table, max_pages};
    return FA_OK;
}
