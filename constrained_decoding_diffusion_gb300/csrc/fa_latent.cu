// Writing a paged latent cache and keeping an accepted path in it.
#include "fa_latent.cuh"

namespace {

constexpr int NT = 256;

struct WriteArgs {
    void *rows;
    int64_t n_slots, ls, ks;
    int N, latent, rope, interleaved;
    const void *x, *key;
    const int32_t *slot, *pos;
    const uint64_t *phase;
    float mscale;
};

// A warp takes two tokens at a time, so that all that it reads of both is under way before it stores: the latent part in
// vectors of 16 bytes of the source, R a lane (R = 0: one element at a time, where its rows are not aligned), the key
// part a pair a lane.  The bound is memory: a vector is read once and written once.  Measured, 32768 tokens of 512 + 64
// bf16: 14.6 us (75 MB, 5.2 TB/s, 76% of a copy; one token a warp at a time 18.5).
template <class T, class O, int R>
__global__ void __launch_bounds__(NT) k_latent_write(WriteArgs a) {
    constexpr int N = fa_vec<T>::N, U = 2, RR = R > 0 ? R : 1;
    const int lane = threadIdx.x & 31, half = a.rope / 2, vectors = a.latent / N;
    const int64_t n0 = ((int64_t)blockIdx.x * (NT / 32) + (threadIdx.x >> 5)) * U;
    const int p = a.interleaved ? 2 * lane : lane, q = a.interleaved ? 2 * lane + 1 : lane + half;
    int64_t at[U];
    int pos[U];
    uint4 v[U][RR];
    T k0[U], k1[U];
    const uint64_t phase = a.pos && lane < half ? __ldg(a.phase + lane) : 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t n = n0 + u;
        at[u] = n < a.N ? a.slot[n] : -1;
        pos[u] = a.pos && n < a.N ? __ldg(a.pos + n) : 0;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t n = min(n0 + u, (int64_t)a.N - 1);
        const T *x = (const T *)a.x + n * a.ls, *k = (const T *)a.key + n * a.ks;
        if (R > 0)
#pragma unroll
            for (int r = 0; r < RR; ++r)
                if (lane + 32 * r < vectors) v[u][r] = __ldg(reinterpret_cast<const uint4 *>(x) + lane + 32 * r);
        if (lane < half) { k0[u] = k[p]; k1[u] = k[q]; }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (at[u] < 0 || at[u] >= a.n_slots) continue;
        O *row = (O *)a.rows + at[u] * (a.latent + a.rope);
        if (R > 0) {
#pragma unroll
            for (int r = 0; r < RR; ++r) {
                const int c = lane + 32 * r;
                if (c >= vectors) break;
                float f[N];
                fa_unpack(v[u][r], f, T());
                if constexpr (N == 8) reinterpret_cast<uint4 *>(row)[c] = fa_pack(f, O());
                else reinterpret_cast<uint2 *>(row)[c] = make_uint2(fa_pack2(f[0], f[1], O()), fa_pack2(f[2], f[3], O()));
            }
        } else {
            const T *x = (const T *)a.x + (n0 + u) * a.ls;
            for (int c = lane; c < a.latent; c += 32) row[c] = fa_from_f32<O>(fa_to_f32(x[c]));
        }
        if (lane < half) {
            row += a.latent;
            const float x0 = fa_to_f32(k0[u]), x1 = fa_to_f32(k1[u]);
            if (a.pos) {
                const float2 cs = fa_turn(pos[u], phase, a.mscale, false);
                row[p] = fa_from_f32<O>(x0 * cs.x - x1 * cs.y);
                row[q] = fa_from_f32<O>(x0 * cs.y + x1 * cs.x);
            } else {
                row[p] = fa_from_f32<O>(x0);
                row[q] = fa_from_f32<O>(x1);
            }
        }
    }
}

// One block per sequence.  The path's slots are looked up all at once; then its rows move, eight under
// way.  What bounds it is the chain of path, page numbers, rows: paths of 3 rows in 64 sequences 5.9 us from a cold cache.
//  A row is read before it is written over: path[i] >= i, and the rows of a turn are all read before any is written.
__global__ void __launch_bounds__(128) k_latent_keep(fa_cache_view c, int P, const int32_t *__restrict__ length,
                                                     const int32_t *__restrict__ path) {
    __shared__ int from[FA_MAX_DRAFT], to[FA_MAX_DRAFT];   // -1: no page; the host has checked that slots are 32 bits
    __shared__ int end;
    constexpr int U = 8;
    const int64_t b = blockIdx.x;
    const int64_t n = length[b];
    const int tid = threadIdx.x, chunks = c.head_dim / 8;
    if (n < 0) return;
    if (tid == 0) end = P;
    __syncthreads();
    for (int i = tid; i < P; i += 128) {
        const int j = path[b * P + i], last = i > 0 ? path[b * P + i - 1] : -1;
        if (j < 0 || j <= last) atomicMin(&end, i);
        from[i] = (int)c.row((int)b, n + j, 0);
        to[i] = j == i ? -1 : (int)c.row((int)b, n + i, 0);
    }
    __syncthreads();
    uint4 *rows = (uint4 *)c.k;
    if (tid >= chunks) return;
    for (int i0 = 0; i0 < end; i0 += U) {
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u;
            x[u] = make_uint4(0, 0, 0, 0);
            if (i < end && to[i] >= 0 && from[i] >= 0) x[u] = rows[(int64_t)from[i] * chunks + tid];
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u < end && to[i0 + u] >= 0) rows[(int64_t)to[i0 + u] * chunks + tid] = x[u];
    }
}

template <class T, class O> fa_status launch_write(const WriteArgs &a, cudaStream_t s) {
    const bool aligned = !((uintptr_t)a.x & 15) && a.ls % fa_vec<T>::N == 0;
    const unsigned blocks = (unsigned)((((int64_t)a.N + 1) / 2 * 32 + NT - 1) / NT);
    const int each = (a.latent / fa_vec<T>::N + 31) / 32;
    if (!aligned) k_latent_write<T, O, 0><<<blocks, NT, 0, s>>>(a);
    else if (each == 1) k_latent_write<T, O, 1><<<blocks, NT, 0, s>>>(a);
    else if (each == 2) k_latent_write<T, O, 2><<<blocks, NT, 0, s>>>(a);
    else k_latent_write<T, O, 4><<<blocks, NT, 0, s>>>(a);
    return fa_launch_check("latent write");
}

}  // namespace

extern "C" fa_status fa_latent_write(const fa_latent_cache *cache, int32_t dtype, int32_t N, const void *latent,
                                     int64_t latent_stride, const void *key, int64_t key_stride, const int32_t *slot,
                                     const int32_t *positions, const uint64_t *phase, int32_t interleaved, float mscale,
                                     fa_stream stream) {
    const char *fn = "fa_latent_write";
    fa_cache_view c;
    fa_status st = fa_view_latent(fn, cache, nullptr, 0, &c);
    if (st != FA_OK) return st;
    if (!fa_dtype_ok(dtype)) return fa_refuse(fn, "unknown dtype");
    if (N < 0) return fa_refuse(fn, "N negative");
    if ((positions == nullptr) != (phase == nullptr)) return fa_refuse(fn, "positions and phase go together");
    if (interleaved != 0 && interleaved != 1) return fa_refuse(fn, "interleaved must be 0 or 1");
    if (N == 0) return FA_OK;
    if (!latent || !key || !slot) return fa_refuse(fn, "NULL buffer");
    if (((uintptr_t)latent | (uintptr_t)key) % fa_dtype_bytes(dtype)) return fa_refuse(fn, "latent and key must be aligned to their type");
    const WriteArgs a{cache->rows, (int64_t)cache->n_pages * cache->page_size, latent_stride, key_stride, N, cache->latent_dim,
                      cache->rope_dim, interleaved, latent, key, slot, positions, phase, mscale};
    cudaStream_t s = (cudaStream_t)stream;
    auto go = [&](auto tag) {
        using O = decltype(tag);
        if (dtype == FA_DTYPE_F32) return launch_write<float, O>(a, s);
        if (dtype == FA_DTYPE_F16) return launch_write<__half, O>(a, s);
        return launch_write<__nv_bfloat16, O>(a, s);
    };
    return cache->format == FA_CACHE_F16 ? go(__half()) : go(__nv_bfloat16());
}

extern "C" fa_status fa_latent_keep(const fa_latent_cache *cache, int32_t B, int32_t P, const int32_t *page_table,
                                    int32_t max_pages, const int32_t *length, const int32_t *path, fa_stream stream) {
    const char *fn = "fa_latent_keep";
    fa_cache_view c;
    fa_status st = fa_view_latent(fn, cache, page_table, max_pages, &c);
    if (st != FA_OK) return st;
    if (B < 0 || P < 0 || P > FA_MAX_DRAFT) return fa_refuse(fn, "B or P out of range");
    if (B == 0 || P == 0) return FA_OK;
    if (!length || !path) return fa_refuse(fn, "NULL buffer");
    k_latent_keep<<<(unsigned)B, 128, 0, (cudaStream_t)stream>>>(c, P, length, path);
    return fa_launch_check("latent keep");
}
