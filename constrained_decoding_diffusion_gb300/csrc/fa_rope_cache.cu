// Rotary positions and the paged, quantised key/value cache: writing, reading back, keeping an
// accepted path, and the mask of a draft tree.
#include "fa_lm.cuh"

namespace {

constexpr int NT = 256;

// mscale * (cos, sin) of position t times phase (a 64-bit fraction of a turn): the product wraps around at
// whole turns whatever the position, and its upper 32 bits, rounded to fp32, are the angle: off by up to 2^-26
// turn (a tenth of a millionth of a radian), where fp32's own sines and products are off by as much.
__device__ __forceinline__ float2 turn(int32_t t, uint64_t phase, float mscale, bool inverse) {
    const int32_t frac = (int32_t)(uint32_t)(((uint64_t)(int64_t)t * phase) >> 32);
    float s, c;
    sincospif((float)frac * (1.0f / 2147483648.0f), &s, &c);
    return make_float2(mscale * c, mscale * (inverse ? -s : s));
}

unsigned blocks_for(int64_t items) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>((items + NT - 1) / NT, 152 * 16)); }

struct RopeArgs {
    int64_t n_tokens, xt, xh, ot, oh;
    int heads, dim, rot, interleaved, inverse;
    const void *x;
    void *out;
    const int32_t *pos;
    const uint64_t *phase;
    float mscale;
};

// y = R x per pair, element by element: any strides and sizes.
template <class T>
__global__ void __launch_bounds__(NT) k_rope_any(RopeArgs a) {
    const int half = a.rot / 2, per_head = half + (a.dim - a.rot);
    const int64_t total = a.n_tokens * a.heads * per_head;
    for (int64_t it = (int64_t)blockIdx.x * NT + threadIdx.x; it < total; it += (int64_t)gridDim.x * NT) {
        const int i = (int)(it % per_head);
        const int64_t nh = it / per_head, n = nh / a.heads;
        const int h = (int)(nh % a.heads);
        const T *xr = (const T *)a.x + n * a.xt + h * a.xh;
        T *yr = (T *)a.out + n * a.ot + h * a.oh;
        if (i >= half) {
            yr[a.rot + i - half] = xr[a.rot + i - half];
            continue;
        }
        const int p = a.interleaved ? 2 * i : i, q = a.interleaved ? 2 * i + 1 : i + half;
        const float2 cs = turn(__ldg(a.pos + n), __ldg(a.phase + i), a.mscale, a.inverse);
        const float x0 = fa_to_f32(xr[p]), x1 = fa_to_f32(xr[q]);
        yr[p] = fa_from_f32<T>(x0 * cs.x - x1 * cs.y);
        yr[q] = fa_from_f32<T>(x0 * cs.y + x1 * cs.x);
    }
}

// The same in 16-byte vectors of N elements, where every row is aligned and the rotated part is
// whole vectors (half layout: each half).  The bound is memory: x is read and out written
// once.  A block takes a few tokens with all their heads.  Their sines and cosines, one per
// token and pair, are made once in shared memory while the first vectors are on their way; a
// thread keeps its place (head and vector) and walks the tokens, four of them under way at a time,
// so the arithmetic of places is done once.  Measured, 8192 tokens of 32 heads of 128 in bf16, half of a head
// rotated: 25 us (134 MB, 5.4 TB/s, four fifths of a copy).
constexpr int ROPE_TOKENS = 16;
template <class T> constexpr int rope_blocks() { return sizeof(T) == 4 ? 0 : 4; }   // of an SM at least (0: no bound), without spills
template <class T, bool INTERLEAVED>
__global__ void __launch_bounds__(NT, rope_blocks<T>()) k_rope(RopeArgs a, int tokens) {
    // [tokens][pair of a vector][vector]: neighbouring lanes' pairs lie side by side
    extern __shared__ float2 table[];
    constexpr int N = fa_vec<T>::N, U = 4, P = INTERLEAVED ? N / 2 : N;
    const int half = a.rot / 2, tid = threadIdx.x;
    // a head's work items: rotated vectors (pairs of vectors), then the vectors that are copied
    const int turned = INTERLEAVED ? a.rot / N : half / N, items = turned + (a.dim - a.rot) / N, per_token = items * a.heads;
    const int64_t n0 = (int64_t)blockIdx.x * tokens;
    const int here = (int)min((int64_t)tokens, a.n_tokens - n0), step = half / P;
    bool made = false;
    for (int it = tid; it < per_token || !made; it += NT) {
        const int h = it / items, i = it - h * items, col = i < turned ? i * N : a.rot + (i - turned) * N;
        const bool mine = it < per_token, pairs = !INTERLEAVED && i < turned;
        const T *src = (const T *)a.x + n0 * a.xt + h * a.xh + col;
        T *dst = (T *)a.out + n0 * a.ot + h * a.oh + col;
        for (int t0 = 0; t0 < here; t0 += U) {
            uint4 v[U], w[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!mine || t0 + u >= here) continue;
                // (not the read-only path: out may be x)
                v[u] = *reinterpret_cast<const uint4 *>(src + (t0 + u) * a.xt);
                if (pairs) w[u] = *reinterpret_cast<const uint4 *>(src + (t0 + u) * a.xt + half);
            }
            if (!made) {
                for (int j = tid; j < here * half; j += NT) {
                    const int t = j / half, p = j - t * half;
                    table[t * half + p % P * step + p / P] = turn(__ldg(a.pos + n0 + t), __ldg(a.phase + p), a.mscale, a.inverse);
                }
                __syncthreads();
                made = true;
            }
            if (!mine) continue;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t0 + u >= here) break;
                uint4 *to = reinterpret_cast<uint4 *>(dst + (t0 + u) * a.ot);
                if (i >= turned) { *to = v[u]; continue; }
                const float2 *cs = table + (t0 + u) * half + i;
                float x[N];
                fa_unpack(v[u], x, T());
                if (INTERLEAVED) {
#pragma unroll
                    for (int e = 0; e < N; e += 2) {
                        const float2 f = cs[e / 2 * step];
                        const float p = x[e] * f.x - x[e + 1] * f.y;
                        x[e + 1] = x[e] * f.y + x[e + 1] * f.x;
                        x[e] = p;
                    }
                    *to = fa_pack(x, T());
                } else {
                    float y[N];
                    fa_unpack(w[u], y, T());
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        const float2 f = cs[e * step];
                        const float p = x[e] * f.x - y[e] * f.y;
                        y[e] = x[e] * f.y + y[e] * f.x;
                        x[e] = p;
                    }
                    *to = fa_pack(x, T());
                    *reinterpret_cast<uint4 *>(dst + (t0 + u) * a.ot + half) = fa_pack(y, T());
                }
            }
        }
    }
}

template <class T> fa_status launch_rope(const RopeArgs &a, cudaStream_t s) {
    constexpr int N = fa_vec<T>::N;
    const bool aligned = !(((uintptr_t)a.x | (uintptr_t)a.out) & 15) && !((a.xt | a.xh | a.ot | a.oh) % N);
    const bool whole = a.dim % N == 0 && (a.interleaved ? a.rot % N == 0 : a.rot / 2 % N == 0);
    const int64_t per_token = (int64_t)a.heads * ((a.interleaved ? a.rot : a.rot / 2) + a.dim - a.rot) / N;
    if (!aligned || !whole || per_token > (1 << 24)) {
        const int64_t items = a.n_tokens * a.heads * (a.dim - a.rot / 2);
        k_rope_any<T><<<blocks_for(items), NT, 0, s>>>(a);
        return fa_launch_check("rope");
    }
    // Tokens of a block: 16-bit types, as many as make full waves of four blocks an SM (8192 tokens x 32 heads x
    // 128: 23.4 us, 25.7 half rotated, against 23.7 and 28.6 with eight whatever the count); fp32, twice the bytes
    // a token, up to eight and fewer where that leaves SMs without a block (43 us against 46.7 with full waves).
    int64_t tokens;
    if (sizeof(T) == 4) {
        tokens = std::min<int64_t>(8, std::max<int64_t>(1, a.n_tokens / (152 * 4)));
    } else {
        const int64_t resident = 152 * rope_blocks<T>();
        const int64_t most = std::min<int64_t>(ROPE_TOKENS, 40960 / std::max<int64_t>(1, a.rot / 2 * (int64_t)sizeof(float2)));
        const int64_t waves = (a.n_tokens + resident * most - 1) / (resident * most);
        tokens = (a.n_tokens + resident * waves - 1) / (resident * waves);
    }
    const int64_t blocks = (a.n_tokens + tokens - 1) / tokens;
    if (blocks > 2147483647) return fa_refuse("fa_rope", "too many tokens");
    const size_t smem = (size_t)tokens * (a.rot / 2) * sizeof(float2);   // at most 40 KB
    if (a.interleaved) k_rope<T, true><<<(unsigned)blocks, NT, smem, s>>>(a, (int)tokens);
    else k_rope<T, false><<<(unsigned)blocks, NT, smem, s>>>(a, (int)tokens);
    return fa_launch_check("rope");
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

// One warp per (token, head), element by element: any strides and alignment.  Lane l holds elements
// l, l + 32, ...
template <class T>
__global__ void __launch_bounds__(NT) k_cache_write_any(WriteArgs a) {
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

// x / s for |x| <= 448 s, rounded as a division would be: the product with the reciprocal, then one
// step of Markstein's correction (the remainder of an fma times the reciprocal).  The remainder is
// exact unless it falls below the normal range, which the caller excludes.
__device__ __forceinline__ float quotient(float x, float s, float r) {
    const float q = x * r;
    return fmaf(fmaf(-q, s, x), r, q);
}

// the larger magnitude, or NaN if either is one
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// four elements in memory (8 bytes of 16-bit types, 16 bytes of fp32)
__device__ __forceinline__ void load4(const float *p, uint4 &r) { r = __ldg(reinterpret_cast<const uint4 *>(p)); }
template <class T> __device__ __forceinline__ void load4(const T *p, uint2 &r) { r = __ldg(reinterpret_cast<const uint2 *>(p)); }
__device__ __forceinline__ void floats4(uint4 r, float *f, float) {
    f[0] = __uint_as_float(r.x); f[1] = __uint_as_float(r.y); f[2] = __uint_as_float(r.z); f[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void floats4(uint2 r, float *f, __nv_bfloat16) {
    f[0] = __uint_as_float(r.x << 16); f[1] = __uint_as_float(r.x & 0xffff0000u);
    f[2] = __uint_as_float(r.y << 16); f[3] = __uint_as_float(r.y & 0xffff0000u);
}
__device__ __forceinline__ void floats4(uint2 r, float *f, __half) {
    __half2 h[2];
    memcpy(h, &r, 8);
    const float2 a = __half22float2(h[0]), b = __half22float2(h[1]);
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

// The same in vectors: a group of G = 8, 16 or 32 lanes holds a row, a lane eight of its elements as
// two pieces of four, and each row is read once.  In the half layout the pieces of a rotated lane are
// four elements of the first half and their mates of the second, so every pair meets in a lane.
// The bound is memory (keys and values in, codes and scales out) and, before it, the issue of
// instructions: sines and cosines are made once per token in shared memory; a maximum that keeps NaN
// finds the rows to mark; the largest magnitudes of a thread's four vectors are exchanged so that each
// lane divides for one of them; the division by the scale is a multiplication with a correction.  A
// block takes up to 32 tokens with all their heads, a thread two rows' keys and values while the next
// two are under way.  Measured, 16 x 2048 tokens of 8 heads of 128, bf16 to 8 bits: 55 us (3.7 TB/s; 44 M
// warp instructions, two thirds of the issue slots with a third of the warps resident, so latency counts as
// well); to bf16, without maxima and quotients, 3 us less; without rows under way 63, with a pair of floats
// per instruction no faster.
constexpr int WRITE_TOKENS = 32;
template <class T> constexpr int write_blocks() { return sizeof(T) == 4 ? 2 : 3; }   // of an SM, without spills
template <class T, int G, int FORMAT>
__global__ void __launch_bounds__(NT, write_blocks<T>()) k_cache_write(WriteArgs a, int tokens) {
    extern __shared__ float2 table[];           // [tokens][pair of a lane's four][lane]
    __shared__ int64_t row0[WRITE_TOKENS], key0[WRITE_TOKENS], value0[WRITE_TOKENS];   // a token's row of head 0, or -1; its offsets
    typedef typename std::conditional<sizeof(T) == 4, uint4, uint2>::type Raw;
    constexpr int ROWS = NT / G, U = 2;         // rows in step, rows of a thread under way
    const int H = a.c.kv_heads, D = a.c.head_dim, half = a.rot / 2, lanes = half / 4;   // lanes with pairs
    const int g = threadIdx.x % G, r0 = threadIdx.x / G;
    const bool in = g * 8 < D, turned = g < lanes, split = turned && !a.interleaved;
    const int v0 = g * 8, k0 = split ? g * 4 : v0, k1 = split ? half + g * 4 : v0 + 4;   // the pieces
    const unsigned all = (unsigned)a.B * (unsigned)a.T, n0 = blockIdx.x * (unsigned)tokens;   // below 2^31
    const int here = (int)min((unsigned)tokens, all - n0), total = here * H;
    const unsigned mask = G == 32 ? 0xffffffffu : ((1u << G) - 1) << (threadIdx.x % 32 / G * G);
    if ((int)threadIdx.x < here) {
        const unsigned bt = n0 + threadIdx.x, b = bt / (unsigned)a.T;
        const int t = (int)(bt - b * (unsigned)a.T);
        const bool used = !a.count || t < __ldg(a.count + b);
        row0[threadIdx.x] = used ? a.c.row((int)b, (int64_t)__ldg(a.start + b) + t, 0) : -1;
        key0[threadIdx.x] = (int)b * a.kb + t * a.kt;
        value0[threadIdx.x] = (int)b * a.vb + t * a.vt;
    }
    for (int i = threadIdx.x; i < here * half; i += NT) {
        const int t = i / half, p = i - t * half;
        table[t * half + p % 4 * lanes + p / 4] = turn(__ldg(a.pos + n0 + t), __ldg(a.phase + p), a.mscale, false);
    }
    __syncthreads();
    int64_t row[U], next_row[U];
    int tok[U], next_tok[U];
    Raw x[U][4];                                // the key's pieces, the value's
    auto load = [&](int first) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int it = first + u * ROWS;
            next_row[u] = -1;
            if (it >= total) continue;
            next_tok[u] = it / H;
            const int h = it - next_tok[u] * H;
            next_row[u] = row0[next_tok[u]];
            if (next_row[u] < 0) continue;
            next_row[u] += (int64_t)h << a.c.page_shift;
            if (!in) continue;
            const T *k = (const T *)a.k + key0[next_tok[u]] + h * a.kh;
            const T *v = (const T *)a.v + value0[next_tok[u]] + h * a.vh + v0;
            load4(k + k0, x[u][0]);
            load4(k + k1, x[u][1]);
            load4(v, x[u][2]);
            load4(v + 4, x[u][3]);
        }
    };
    load(r0);
    for (int first = r0; first - r0 < total; first += U * ROWS) {
#pragma unroll
        for (int u = 0; u < U; ++u) { row[u] = next_row[u]; tok[u] = next_tok[u]; }
        float f[U][2][8];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                float (&y)[8] = f[u][side];
                if (in && row[u] >= 0) {
                    floats4(x[u][2 * side], y, T());
                    floats4(x[u][2 * side + 1], y + 4, T());
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = 0.0f;
                }
            }
        load(first + U * ROWS);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float (&y)[8] = f[u][0];
            if (turned && row[u] >= 0) {
                const float2 *cs = table + tok[u] * half + g;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 t = cs[e * lanes];
                    auto turn_pair = [&](float &p, float &q) {
                        const float z = p * t.x - q * t.y;
                        q = p * t.y + q * t.x;
                        p = z;
                    };
                    if (a.interleaved) turn_pair(y[2 * e], y[2 * e + 1]);
                    else turn_pair(y[e], y[e + 4]);
                }
            }
        }
        float scale = 0.0f, r = 0.0f;           // lane g: of row g / 2 % 2, side g % 2
        if (FORMAT == FA_CACHE_E4M3) {
            // the largest of every vector, exchanged so that a lane ends with one of the four
            float top[U][2];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int side = 0; side < 2; ++side) {
                    top[u][side] = 0.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) top[u][side] = max_nan(top[u][side], fabsf(f[u][side][e]));
                }
            const bool u1 = g & 2, s1 = g & 1;
            const float t0 = max_nan(u1 ? top[1][0] : top[0][0], __shfl_xor_sync(mask, u1 ? top[0][0] : top[1][0], 2));
            const float t1 = max_nan(u1 ? top[1][1] : top[0][1], __shfl_xor_sync(mask, u1 ? top[0][1] : top[1][1], 2));
            float amax = max_nan(s1 ? t1 : t0, __shfl_xor_sync(mask, s1 ? t0 : t1, 1));
#pragma unroll
            for (int o = G / 2; o >= 4; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(mask, amax, o));
            const bool odd = !(amax < INFINITY);
            scale = odd ? __int_as_float(0x7fffffff) : amax / FA_E4M3_MAX;
            r = odd || amax < 1e-30f ? 0.0f : 1.0f / scale;
            const int64_t mine = u1 ? row[1] : row[0];
            if (g < 4 && mine >= 0) (s1 ? a.c.v_scale : a.c.k_scale)[mine] = scale;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                float (&y)[8] = f[u][side];
                const int64_t at = row[u] * D;
                const int p0 = side ? v0 : k0, p1 = side ? v0 + 4 : k1;
                void *dst = side ? a.c.v : a.c.k;
                if (FORMAT == FA_CACHE_E4M3) {
                    const float sc = __shfl_sync(mask, scale, 2 * u + side, G), rc = __shfl_sync(mask, r, 2 * u + side, G);
                    if (row[u] < 0 || !in) continue;
                    if (rc == 0.0f) {
                        // a row of zeros or one that is marked; tiny values take the plain division
#pragma unroll 1
                        for (int e = 0; e < 8; ++e) {
                            const float q = sc > 0.0f ? y[0] / sc : 0.0f;   // rotate through y[0]
#pragma unroll
                            for (int j = 0; j < 7; ++j) y[j] = y[j + 1];
                            y[7] = q;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] = quotient(y[e], sc, rc);
                    }
                    *reinterpret_cast<uint32_t *>((uint8_t *)dst + at + p0) = fa_to_e4m3x2(y[0], y[1]) | fa_to_e4m3x2(y[2], y[3]) << 16;
                    *reinterpret_cast<uint32_t *>((uint8_t *)dst + at + p1) = fa_to_e4m3x2(y[4], y[5]) | fa_to_e4m3x2(y[6], y[7]) << 16;
                } else if (in && row[u] >= 0) {
                    typedef typename std::conditional<FORMAT == FA_CACHE_F16, __half, __nv_bfloat16>::type O;
                    *reinterpret_cast<uint2 *>((O *)dst + at + p0) = make_uint2(fa_pack2(y[0], y[1], O()), fa_pack2(y[2], y[3], O()));
                    *reinterpret_cast<uint2 *>((O *)dst + at + p1) = make_uint2(fa_pack2(y[4], y[5], O()), fa_pack2(y[6], y[7], O()));
                }
            }
    }
}

template <class T, int G> void launch_write(const WriteArgs &a, unsigned blocks, int tokens, size_t smem, cudaStream_t s) {
    if (a.format == FA_CACHE_E4M3) k_cache_write<T, G, FA_CACHE_E4M3><<<blocks, NT, smem, s>>>(a, tokens);
    else if (a.format == FA_CACHE_F16) k_cache_write<T, G, FA_CACHE_F16><<<blocks, NT, smem, s>>>(a, tokens);
    else k_cache_write<T, G, FA_CACHE_BF16><<<blocks, NT, smem, s>>>(a, tokens);
}

template <class T> fa_status launch_write(const WriteArgs &a, cudaStream_t s) {
    const int H = a.c.kv_heads, D = a.c.head_dim;
    const int64_t all = (int64_t)a.B * a.T;
    const bool aligned = !(((uintptr_t)a.k | (uintptr_t)a.v) & 15) && !((a.kb | a.kt | a.kh | a.vb | a.vt | a.vh) % fa_vec<T>::N);
    if (!aligned || a.rot % 8) {
        k_cache_write_any<T><<<(unsigned)((all * H + NT / 32 - 1) / (NT / 32)), NT, 0, s>>>(a);
        return fa_launch_check("cache write");
    }
    const int G = D <= 64 ? 8 : D <= 128 ? 16 : 32;
    // as many tokens a block as make full waves of blocks (16 tokens whatever the count: 60 us
    // against 55 for 16 x 2048 tokens)
    const int64_t resident = 152 * write_blocks<T>(), waves = (all + resident * WRITE_TOKENS - 1) / (resident * WRITE_TOKENS);
    const int tokens = (int)((all + resident * waves - 1) / (resident * waves));
    const unsigned blocks = (unsigned)((all + tokens - 1) / tokens);
    const size_t smem = (size_t)tokens * (a.rot / 2) * sizeof(float2);   // at most 32 * 128 * 8 bytes
    if (G == 8) launch_write<T, 8>(a, blocks, tokens, smem, s);
    else if (G == 16) launch_write<T, 16>(a, blocks, tokens, smem, s);
    else launch_write<T, 32>(a, blocks, tokens, smem, s);
    return fa_launch_check("cache write");
}

// Slots back as dense rows.  The bound is memory: codes in, twice or four times as many bytes out.
// A thread takes eight elements of a row, the keys' and the values', with two rows under way (four
// cost more in occupancy than they hide); a warp's loads and stores are contiguous.  Measured, 16 x 8192 slots
// of 8 heads of 128, 8 bits to bf16: 131 us (0.81 GB, 6.2 TB/s, 92% of a copy).
template <class T, int FORMAT>
__global__ void __launch_bounds__(NT) k_cache_read(fa_cache_view c, int N, const int32_t *__restrict__ length, T *k_out, T *v_out) {
    constexpr int U = 2;
    typedef typename std::conditional<FORMAT == FA_CACHE_E4M3, uint2, uint4>::type Raw;   // eight elements
    const unsigned H = c.kv_heads, C = c.head_dim / 8, total = (unsigned)N * H * C;
    const int b = blockIdx.y, n = __ldg(length + b);
    const int64_t base = (int64_t)b * total;
    for (unsigned first = blockIdx.x * (NT * U) + threadIdx.x; first < total; first += gridDim.x * NT * U) {
        Raw x[U][2];
        float scale[U][2];
        bool there[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const unsigned it = first + u * NT;
            there[u] = false;
            if (it >= total) continue;
            const unsigned r = it / C, ch = it - r * C, t = r / H, h = r - t * H;
            const int64_t row = (int)t < n ? c.row(b, t, (int)h) : -1;
            if (row < 0) continue;
            there[u] = true;
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                x[u][side] = __ldg((const Raw *)(side ? c.v : c.k) + row * C + ch);
                if (FORMAT == FA_CACHE_E4M3) scale[u][side] = __ldg((side ? c.v_scale : c.k_scale) + row);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const unsigned it = first + u * NT;
            if (it >= total) continue;
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                float f[8];
                if (!there[u]) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = 0.0f;
                } else if constexpr (FORMAT == FA_CACHE_E4M3) {
                    const uint32_t w[2] = {x[u][side].x, x[u][side].y};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t two = fa_e4m3x2_to_half2(w[i / 2] >> (16 * (i & 1)));
                        __half2 hh;
                        memcpy(&hh, &two, 4);
                        const float2 p = __half22float2(hh);
                        f[2 * i] = p.x * scale[u][side];
                        f[2 * i + 1] = p.y * scale[u][side];
                    }
                } else if constexpr (FORMAT == FA_CACHE_F16) {
                    fa_unpack(x[u][side], f, __half());
                } else {
                    fa_unpack(x[u][side], f, __nv_bfloat16());
                }
                uint4 *dst = reinterpret_cast<uint4 *>((side ? v_out : k_out) + (base + it) * 8);
                constexpr int PER = fa_vec<T>::N;
#pragma unroll
                for (int i = 0; i < 8 / PER; ++i) {
                    float p[PER];
#pragma unroll
                    for (int e = 0; e < PER; ++e) p[e] = f[PER * i + e];
                    dst[i] = fa_pack(p, T());
                }
            }
        }
    }
}

// One block per (sequence, head).  A thread moves the same 16 bytes of every kept row, in order:
// path[i] >= i, so a row still to be read is never one that was written.  A slot that no page holds
// reads as zeros and is not written, like everywhere.  What bounds it is the chain of lookups, one row
// after the other (1.3 us a row, of which a path has as many as a draft is deep).  Measured from a cold cache
// with 5 us for the launch, 16 sequences of 8 heads of 128, 8 bits: paths of 5 rows 13 us, of 64 rows 87 us.
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
        if (to < 0) continue;
        for (int q = tid; q < 2 * chunks; q += 64) {
            uint4 *p = (uint4 *)(q < chunks ? c.k : c.v);
            p[to * chunks + q % chunks] = from < 0 ? make_uint4(0, 0, 0, 0) : p[from * chunks + q % chunks];
        }
        if (c.k_scale && tid < 2) {
            float *p = tid ? c.v_scale : c.k_scale;
            p[to] = from < 0 ? 0.0f : p[from];
        }
    }
}

// One block per sequence, one thread per drafted token: walk up the ancestors, which come in
// descending order, and store each 64-bit word when the walk leaves it.  What bounds it is the longest
// walk, a dependent read of shared memory a step.  Measured from a cold cache with 5 us for the launch, 16
// chains of 17 / 64 / 1024 tokens (the deepest trees there are): 9 / 11 / 298 us.
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
    if (n_tokens > ((int64_t)1 << 62) / ((int64_t)n_heads * head_dim)) return fa_refuse(fn, "too many elements");
    cudaStream_t s = (cudaStream_t)stream;
    const RopeArgs a{n_tokens, x_token_stride, x_head_stride, out_token_stride, out_head_stride, n_heads, head_dim, rot_dim,
                     interleaved, inverse != 0, x, out, positions, phase, mscale};
    if (dtype == FA_DTYPE_F32) return launch_rope<float>(a, s);
    if (dtype == FA_DTYPE_F16) return launch_rope<__half>(a, s);
    return launch_rope<__nv_bfloat16>(a, s);
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
    if (rot_dim != 0 && (positions == nullptr) != (phase == nullptr)) return fa_refuse(fn, "positions and phase go together");
    if (positions && phase && (st = rope_args(fn, cache->head_dim, rot_dim, interleaved)) != FA_OK) return st;
    if (B == 0 || T == 0) return FA_OK;
    if (!k || !v || !start) return fa_refuse(fn, "NULL buffer");
    a.format = cache->format; a.B = B; a.T = T;
    a.k = k; a.v = v;
    a.kb = k_batch_stride; a.kt = k_token_stride; a.kh = k_head_stride;
    a.vb = v_batch_stride; a.vt = v_token_stride; a.vh = v_head_stride;
    a.start = start; a.count = count; a.pos = positions; a.phase = phase;
    a.rot = positions && phase ? rot_dim : 0; a.interleaved = interleaved; a.mscale = mscale;
    if ((int64_t)B * T > 2147483647 / cache->kv_heads) return fa_refuse(fn, "B * T * kv_heads out of range");
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == FA_DTYPE_F32) return launch_write<float>(a, s);
    if (dtype == FA_DTYPE_F16) return launch_write<__half>(a, s);
    return launch_write<__nv_bfloat16>(a, s);
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
    const int64_t items = (int64_t)N * cache->kv_heads * (cache->head_dim / 8);
    if (B > 65535 || items > 2147483647 - 152 * 64 * 2 * NT) return fa_refuse(fn, "B or N * kv_heads * head_dim out of range");
    const dim3 grid((unsigned)std::min<int64_t>((items + 2 * NT - 1) / (2 * NT), 152 * 64), (unsigned)B);
    cudaStream_t s = (cudaStream_t)stream;
    auto go = [&](auto tag) {
        using T = decltype(tag);
        T *ko = (T *)k_out, *vo = (T *)v_out;
        if (cache->format == FA_CACHE_E4M3) k_cache_read<T, FA_CACHE_E4M3><<<grid, NT, 0, s>>>(c, N, length, ko, vo);
        else if (cache->format == FA_CACHE_F16) k_cache_read<T, FA_CACHE_F16><<<grid, NT, 0, s>>>(c, N, length, ko, vo);
        else k_cache_read<T, FA_CACHE_BF16><<<grid, NT, 0, s>>>(c, N, length, ko, vo);
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
