// Beam selection over beams and vocabulary under an automaton, and the reordering of the beams'
// states.
//
// A cell (beam k, token v) has the value scores[k] + logp[k, v].  Its key is the value's
// order-preserving bit pattern above the complement of its flat index k V + v: keys are distinct,
// larger is better and ties go to the lowest index, so the result does not depend on the order in
// which cells are met.  Selection is one pass over logp.  A block walks batches of 8192 cells of one
// beam, 32 per thread in registers, and keeps the best keys met so far in shared memory; the `top`-th
// best of them is the threshold that nearly every later cell fails.  A thread compares the
// largest of its cells (16-bit types: two at a time), and only where that can pass looks at them one
// by one.  What costs is a list that fills in vain, so every block first takes a threshold from one
// batch of the best beam.  A second launch merges the blocks' lists of a sequence the same way and
// looks up the states.
//
// The floor is memory: logp and the live bits once.  Measured, 16 sequences of 16 beams of 151936
// tokens in bf16, a tenth of them live, top 16: 48 us with merge and reordering, of which the scan
// 41 (2 TB/s); without any cell that passes the scan takes 22, so what bounds it is the threshold's
// rise (most of a block's eight batches still hold a cell that passes) and the barriers around it,
// not the loads.  4 beams of 32000 tokens: 20 us with the reordering, three launches' start and end (2 more
// if a block with a single batch takes a threshold first, too).
#include "fa_lm.cuh"

namespace {

constexpr int NT = 256;
constexpr int PER = 32;            // cells of a batch per thread
constexpr int BATCH = NT * PER;
typedef unsigned long long key_t64;

__device__ __forceinline__ key_t64 cell_key(float v, uint32_t flat) {
    const uint32_t u = __float_as_uint(v + 0.0f);   // -0 becomes 0
    const uint32_t ord = (u >> 31) ? ~u : (u | 0x80000000u);
    return ((key_t64)ord << 32) | (0xffffffffu - flat);
}
__device__ __forceinline__ float key_value(key_t64 k);
// the value below which no cell passes a threshold
__device__ __forceinline__ float passing(key_t64 threshold) { return threshold ? key_value(threshold) : -INFINITY; }
__device__ __forceinline__ float key_value(key_t64 k) {
    const uint32_t ord = (uint32_t)(k >> 32);
    return __uint_as_float((ord >> 31) ? (ord & 0x7fffffffu) : ~ord);
}

// The best keys met so far, at least `top` of them once there are so many: list[0 .. count), all distinct;
// threshold = a key that `top` of them reach, 0 (below every cell's key) before.
struct BestShared {
    key_t64 maxima[NT];
    key_t64 threshold;
    int count, kept, sums[2][NT / 32];
};

// threads that may push in one offer
__host__ __device__ constexpr int pushers(int top) { return 4 * top < NT ? 4 * top : NT; }

// A key that at least `top` of the threads' best keys reach and at most pushers(top) exceed, or 0 where fewer
// than `top` threads have one.  A warp's k-th largest key, k = top / 8 rounded up: the smallest of the
// eight warps' will do, and usually few enough are above it; where not, or where a warp has fewer, the
// top-th largest of all by counting.
__device__ __forceinline__ key_t64 raise(BestShared &sh, int top, key_t64 best) {
    const int tid = threadIdx.x;
    key_t64 x = best, kth = 0;
    for (int i = 0; i < (top + NT / 32 - 1) / (NT / 32); ++i) {
        kth = x;
#pragma unroll
        for (int o = 16; o; o >>= 1) kth = max(kth, __shfl_xor_sync(0xffffffffu, kth, o));
        if (x == kth) x = 0;                       // keys are distinct
    }
    if (tid % 32 == 0) sh.maxima[tid / 32] = kth;
    __syncthreads();
    key_t64 t = sh.maxima[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) t = min(t, sh.maxima[w]);
    t = t ? t - 1 : 0;                             // the least of them still passes
    const int n = __syncthreads_count(best > t);
    if (n <= pushers(top) && (t || n < top)) return t;
    sh.maxima[tid] = best;
    __syncthreads();
    int rank = 0;
    for (int i = 0; i < NT; ++i) rank += sh.maxima[i] > best;
    __syncthreads();
    if (rank == top - 1) sh.maxima[0] = best - 1;
    __syncthreads();
    return sh.maxima[0];
}

// Offer the threads' keys.  pass says whether a thread has one that may be above the threshold,
// best() gives its largest (0 where none can pass) and is asked for only where more threads pass than the
// list has room for; push(t, pass, put) calls put for each key above t of the threads that pass.
// Called by all threads of the block.  The list is cut back to its best `top`, and the threshold raised,
// when it holds twice as many, or `top` before there is a threshold.
constexpr int FULL = 2;
// Keys beyond which a list is searched bit by bit (about 40 counts) and not ranked (a comparison per pair
// of keys).  A list of thousands comes from a first batch with a large `top`: 50257 tokens, top 256, 2030 us
// with ranks alone, 40 to 63 with the search; lists of tens, the common ones, are ranked in less than a
// search's barriers.
constexpr int LONG = 512;
__device__ __forceinline__ void keep_best(BestShared &sh, key_t64 *list, key_t64 *work, int top) {
    const int tid = threadIdx.x, m = sh.count;
    if (m <= top && sh.threshold) return;
    key_t64 least = 0;                             // the smallest of the best `top`
    if (m <= LONG) {
        for (int i = tid; i < m; i += NT) {
            const key_t64 k = list[i];
            int rank = 0;
            for (int j = 0; j < m; ++j) rank += list[j] > k;
            if (rank < top) work[rank] = k;
        }
        __syncthreads();
        if (m >= top) least = work[top - 1];
    } else {
        // bit by bit the largest number that `top` keys reach, until just so many do
        for (int bit = 63; bit >= 0; --bit) {
            const key_t64 t = least | (key_t64)1 << bit;
            int n = 0;
            for (int i = tid; i < m; i += NT) n += list[i] >= t;
            n = __reduce_add_sync(0xffffffffu, n);
            if (tid % 32 == 0) sh.sums[bit & 1][tid / 32] = n;
            __syncthreads();
            n = 0;
#pragma unroll
            for (int w = 0; w < NT / 32; ++w) n += sh.sums[bit & 1][w];
            if (n >= top) least = t;
            if (n == top) break;
        }
        if (tid == 0) sh.kept = 0;
        __syncthreads();
        for (int i = tid; i < m; i += NT)
            if (list[i] >= least) work[atomicAdd(&sh.kept, 1)] = list[i];
        __syncthreads();
    }
    for (int i = tid; i < min(m, top); i += NT) list[i] = work[i];
    if (tid == 0 && m >= top) { sh.count = top; sh.threshold = max(sh.threshold, least); }
    __syncthreads();
}
template <class B, class F>
__device__ __forceinline__ void offer(BestShared &sh, key_t64 *list, key_t64 *work, int top, bool pass, B best, F push) {
    key_t64 thr = sh.threshold;
    const int above = __syncthreads_count(pass);
    if (!above) return;
    if (above > pushers(top) || (!thr && above >= top)) {
        const key_t64 mine = pass ? best() : 0;
        if (__syncthreads_count(mine > thr) > pushers(top) || !thr) thr = max(thr, raise(sh, top, mine));
        pass = mine > thr;
    }
    push(thr, pass, [&](key_t64 k) { list[atomicAdd(&sh.count, 1)] = k; });
    __syncthreads();
    if (sh.count >= (sh.threshold ? FULL * top : top)) keep_best(sh, list, work, top);
}

struct SelectArgs {
    int N, K, V, top, S, words, nb;      // nb blocks per sequence
    const void *logp;
    int64_t ln, lk;
    const float *scores;
    const int32_t *states;
    const int16_t *next;
    const uint32_t *live;
    key_t64 *keys;                       // [N, nb, top]
    float *out_score;
    int32_t *out_parent, *out_token, *out_state;
};

// The larger of two vectors' elements, pairwise in the 16-bit types; a NaN loses.
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b, __half) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b, __nv_bfloat16) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// the largest element of a vector whose bit in m is set (-inf or NaN: none)
__device__ __forceinline__ float top_of(uint4 r, uint32_t m, const uint2 *, float) {
    float t = -INFINITY;
    const float f[4] = {__uint_as_float(r.x), __uint_as_float(r.y), __uint_as_float(r.z), __uint_as_float(r.w)};
#pragma unroll
    for (int e = 0; e < 4; ++e) t = (m >> e & 1) ? fmaxf(t, f[e]) : t;
    return t;
}
// masks: for each nibble of live bits the two words that keep its four elements
template <class T> __device__ __forceinline__ float top_of(uint4 r, uint32_t m, const uint2 *masks, T) {
    constexpr uint32_t low = std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;   // -inf, twice
    const uint2 a = masks[m & 15], b = masks[m >> 4];
    const uint32_t w[4] = {(r.x & a.x) | (low & ~a.x), (r.y & a.y) | (low & ~a.y), (r.z & b.x) | (low & ~b.x), (r.w & b.y) | (low & ~b.y)};
    const uint32_t t = max_pair(max_pair(w[0], w[1], T()), max_pair(w[2], w[3], T()), T());
    float f[8];
    fa_unpack(make_uint4(t, t, t, t), f, T());
    return fmaxf(f[0], f[1]);
}

// the live bits of tokens v0 .. v0 + 31 (v0 may be negative or near the row's end); no row: all of them
__device__ __forceinline__ uint32_t live_word(const uint32_t *row, int words, int v0, int V) {
    if (v0 <= -32 || v0 >= V) return 0;
    uint32_t m = 0xffffffffu;
    if (row) {
        const int w = v0 >> 5, sh = v0 & 31;
        m = w >= 0 ? __ldg(row + w) >> sh : 0u;
        if (sh && w + 1 < words) m |= __ldg(row + w + 1) << (32 - sh);
    }
    if (v0 < 0) m &= 0xffffffffu << -v0;
    if (V - v0 < 32) m &= (1u << (V - v0)) - 1;
    return m;
}

// The sequence's cells from their keys in order, a thread each (0: none).  The beams' scores and states may
// lie where the results go, so every parent's state is read before the first result is written.
__device__ void store_cells(const SelectArgs &a, int n, const key_t64 *keys) {
    static_assert(FA_MAX_BEAM_TOP <= NT, "a thread per result");
    const int i = threadIdx.x;
    const key_t64 k = i < a.top ? keys[i] : 0;
    const uint32_t flat = 0xffffffffu - (uint32_t)k;
    const int parent = k ? (int)(flat / (uint32_t)a.V) : -1, token = k ? (int)(flat % (uint32_t)a.V) : -1;
    int state = -1;
    if (k && a.out_state) state = a.next[(int64_t)a.states[(int64_t)n * a.K + parent] * a.V + token];
    __syncthreads();
    if (i >= a.top) return;
    const int64_t at = (int64_t)n * a.top + i;
    a.out_score[at] = k ? key_value(k) : -INFINITY;
    a.out_parent[at] = parent;
    a.out_token[at] = token;
    if (a.out_state) a.out_state[at] = state;
}

// write the block's best keys: to the outputs when it is the sequence's only block
__device__ void finish(const SelectArgs &a, BestShared &sh, key_t64 *list, key_t64 *work, int n, bool last) {
    __syncthreads();
    if (sh.count > a.top) keep_best(sh, list, work, a.top);
    const int tid = threadIdx.x, m = sh.count;
    if (last) {
        for (int i = tid; i < a.top; i += NT) work[i] = 0;
        __syncthreads();
        for (int i = tid; i < m; i += NT) {
            int rank = 0;
            for (int j = 0; j < m; ++j) rank += list[j] > list[i];
            work[rank] = list[i];
        }
        __syncthreads();
        store_cells(a, n, work);
    } else {
        key_t64 *out = a.keys + ((int64_t)n * a.nb + blockIdx.x) * a.top;
        for (int i = tid; i < a.top; i += NT) out[i] = i < m ? list[i] : 0;
    }
}

template <class T>
__global__ void __launch_bounds__(NT, sizeof(T) == 2 ? 4 : 2) k_beam_scan(SelectArgs a) {
    extern __shared__ key_t64 dyn[];
    __shared__ BestShared sh;
    constexpr int VEC = fa_vec<T>::N, NV = PER / VEC;
    key_t64 *list = dyn, *work = dyn + (size_t)PER * pushers(a.top) + FULL * a.top;
    const int tid = threadIdx.x, n = blockIdx.y;
    __shared__ uint2 masks[16];
    fa_let_next_start();
    if (tid == 0) { sh.threshold = 0; sh.count = 0; }
    if (tid < 16)
        masks[tid] = make_uint2((tid & 1 ? 0x0000ffffu : 0u) | (tid & 2 ? 0xffff0000u : 0u), (tid & 4 ? 0x0000ffffu : 0u) | (tid & 8 ? 0xffff0000u : 0u));
    __syncthreads();
    // the beam with the largest score that is alive, the lowest of equals
    __shared__ key_t64 best_key;
    if (tid == 0) best_key = 0;
    __syncthreads();
    for (int k = tid; k < a.K; k += NT) {
        const float x = __ldg(a.scores + (int64_t)n * a.K + k);
        if (x > -INFINITY && (!a.S || (unsigned)__ldg(a.states + (int64_t)n * a.K + k) < (unsigned)a.S))
            atomicMax(&best_key, cell_key(x, (uint32_t)k));
    }
    __syncthreads();
    const int best_beam = best_key ? (int)(0xffffffffu - (uint32_t)best_key) : 0;
    const int per_beam = (a.V + VEC - 1 + BATCH - 1) / BATCH;   // a misaligned row starts up to VEC - 1 cells early
    const int batches = a.K * per_beam;
    // Which cells of a batch are live: a warp takes 32 x PER consecutive cells, in rows of 32 vectors, and
    // a lane loads the bits of PER of them, one batch ahead of the values.
    static_assert(PER == 32, "a lane's bits are one word");
    constexpr int RPW = 32 / NV;                             // words of bits of a row of vectors
    const int lane = tid & 31, warp_cell = (tid >> 5) * 32 * PER;
    struct Cells {
        uint32_t word;
        const T *row;
        float score;
        int k, first, mis;
    };
    auto find = [&](int bt) {
        Cells x;
        x.word = 0;
        x.k = bt / per_beam;
        x.first = (bt - x.k * per_beam) * BATCH + warp_cell;
        x.score = -INFINITY;
        x.mis = 0;
        x.row = nullptr;
        if (bt >= batches) return x;
        x.score = __ldg(a.scores + (int64_t)n * a.K + x.k);
        const int state = a.S ? __ldg(a.states + (int64_t)n * a.K + x.k) : 0;
        if (!(x.score > -INFINITY) || (a.S && (unsigned)state >= (unsigned)a.S)) return x;   // a dead beam
        x.row = (const T *)a.logp + n * a.ln + x.k * a.lk;
        x.mis = (int)(((uintptr_t)x.row & 15) / sizeof(T));     // the batch's first cell is `first` - mis
        x.word = live_word(a.S ? a.live + (int64_t)state * a.words : nullptr, a.words, x.first - x.mis + 32 * lane, a.V);
        return x;
    };
    // Beams differ by whole units of score, so a block that meets a poor one first would fill its list
    // in vain: every block looks at one batch of the best beam before its own ones, only for a
    // threshold, unless it starts there anyway or has a single batch.
    bool look = batches > (int)gridDim.x && (int)blockIdx.x / per_beam != best_beam;
    Cells next = find(look ? best_beam * per_beam + (int)blockIdx.x % per_beam : blockIdx.x);
    for (int bt = look ? (int)blockIdx.x - (int)gridDim.x : (int)blockIdx.x; bt < batches; bt += gridDim.x, look = false) {
        const Cells c = next;
        const float score = c.score;
        const int cell0 = c.first - c.mis + lane * VEC;      // of vector 0; vector i is 32 i VEC further
        const T *at = c.row + cell0;
        uint32_t bits[NV];
        uint4 raw[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            bits[i] = __shfl_sync(0xffffffffu, c.word, i * RPW + lane / NV) >> lane % NV * VEC & ((1u << VEC) - 1);
            const int v0 = cell0 + 32 * VEC * i;
            raw[i] = make_uint4(0, 0, 0, 0);
            if (!bits[i]) continue;
            if (v0 >= 0 && v0 + VEC <= a.V) {
                raw[i] = __ldg(reinterpret_cast<const uint4 *>(at + 32 * VEC * i));
            } else {
                float f[VEC];
                for (int e = 0; e < VEC; ++e) f[e] = (bits[i] >> e & 1) ? fa_to_f32(at[32 * VEC * i + e]) : 0.0f;
                raw[i] = fa_pack(f, T());
            }
        }
        next = find(bt + gridDim.x);
        // the thread's largest value: the addition is monotone, so it is the score plus the largest cell
        float most = -INFINITY, tops[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            tops[i] = top_of(raw[i], bits[i], masks, T());
            most = fmaxf(most, tops[i]);
        }
        const float top_value = score + most;
        const uint32_t flat0 = (uint32_t)(c.k * a.V + cell0);   // of the thread's first cell
        auto best = [&]() {                                  // the key of the thread's largest cell, the lowest index of equals
            key_t64 key = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float x[VEC];
                fa_unpack(raw[i], x, T());
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if ((bits[i] >> e & 1) && score + x[e] == top_value && !key) key = cell_key(score + x[e], flat0 + 32 * VEC * i + e);
            }
            return key;
        };
        const bool pass = top_value > -INFINITY && !(top_value < passing(sh.threshold));
        if (look) {
            // at least `top` of the batch's cells reach it, so all of the best ones do
            const key_t64 t = raise(sh, a.top, pass ? best() : 0);
            if (tid == 0) sh.threshold = t;
            __syncthreads();
            continue;
        }
        offer(sh, list, work, a.top, pass, best, [&](key_t64 thr, bool mine, auto put) {
            const float least = passing(thr);
            if (mine)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (!(score + tops[i] >= least)) continue;   // nearly all vectors
                    float x[VEC];
                    fa_unpack(raw[i], x, T());
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float v = score + x[e];
                        if ((bits[i] >> e & 1) && v >= least && v > -INFINITY) {
                            const key_t64 key = cell_key(v, flat0 + 32 * VEC * i + e);
                            if (key > thr) put(key);
                        }
                    }
                }
        });
    }
    finish(a, sh, list, work, n, gridDim.x == 1);
}

// merge a sequence's lists
__global__ void __launch_bounds__(NT) k_beam_merge(SelectArgs a) {
    extern __shared__ key_t64 dyn[];
    __shared__ BestShared sh;
    key_t64 *list = dyn, *work = dyn + (size_t)4 * pushers(a.top) + FULL * a.top;
    const int tid = threadIdx.x, n = blockIdx.x;
    if (tid == 0) { sh.threshold = 0; sh.count = 0; }
    __syncthreads();
    fa_wait_for_previous();
    const key_t64 *keys = a.keys + (int64_t)n * a.nb * a.top;
    const int total = a.nb * a.top;
    for (int first = 0; first < total; first += 4 * NT) {
        key_t64 k[4], best = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = first + i * NT + tid;
            k[i] = at < total ? keys[at] : 0;
            best = max(best, k[i]);
        }
        offer(sh, list, work, a.top, best > sh.threshold, [&]() { return best; }, [&](key_t64 thr, bool mine, auto put) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (mine && k[i] > thr) put(k[i]);
        });
    }
    finish(a, sh, list, work, n, true);
}

__global__ void __launch_bounds__(NT) k_beam_reorder(int K, int top, int64_t words, const int32_t *__restrict__ src,
                                                     const int32_t *__restrict__ parent,
                                                     const int32_t *__restrict__ token, int64_t at, int32_t *dst) {
    const int64_t r = blockIdx.x, n = r / top;
    const int p = parent[r];
    const bool found = (unsigned)p < (unsigned)K;
    const int32_t *from = src + (n * K + (found ? p : 0)) * words;
    int32_t *to = dst + r * words;
    for (int64_t w = (int64_t)blockIdx.y * NT + threadIdx.x; w < words; w += (int64_t)gridDim.y * NT)
        to[w] = token && w == at ? token[r] : found ? from[w] : -1;
}

// ----------------------------------------------------------------------------- tables

__global__ void __launch_bounds__(NT) k_table_clear(int64_t n, int16_t *next) {
    for (int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x; i < n; i += (int64_t)gridDim.x * NT) next[i] = -1;
}

// which states reach an accepting one, as bits: backwards over the edges until nothing changes
// (at most S times); one block
__global__ void __launch_bounds__(1024) k_table_reach(int S, int E, const int32_t *accept_mask, const int32_t *src,
                                                      const int32_t *dst, uint32_t *reach) {
    __shared__ uint32_t got[FA_MAX_STATES / 32];
    const int words = (S + 31) / 32, tid = threadIdx.x;
    for (int w = tid; w < words; w += 1024) got[w] = 0;
    __syncthreads();
    for (int s = tid; s < S; s += 1024)
        if (accept_mask[s]) atomicOr(&got[s / 32], 1u << (s % 32));
    __syncthreads();
    for (int round = 0; round < S; ++round) {
        int changed = 0;
        for (int e = tid; e < E; e += 1024) {
            const int s = src[e], d = dst[e];
            if ((got[d / 32] >> (d % 32) & 1) && !(got[s / 32] >> (s % 32) & 1)) {
                atomicOr(&got[s / 32], 1u << (s % 32));
                changed = 1;
            }
        }
        if (!__syncthreads_or(changed)) break;
    }
    for (int w = tid; w < words; w += 1024) reach[w] = got[w];
}

// a block per edge: its tokens lead to its destination, if that can still be accepted
__global__ void __launch_bounds__(NT) k_table_fill(int E, int V, const int64_t *lab_off, const int32_t *lab_tok,
                                                   const int32_t *src, const int32_t *dst, const uint32_t *reach,
                                                   int16_t *next) {
    for (int e = blockIdx.x; e < E; e += gridDim.x) {
        const int s = src[e], d = dst[e];
        if (!(reach[d / 32] >> (d % 32) & 1)) continue;
        for (int64_t i = lab_off[e] + threadIdx.x; i < lab_off[e + 1]; i += NT) next[(int64_t)s * V + lab_tok[i]] = (int16_t)d;
    }
}

// one warp per word
__global__ void __launch_bounds__(NT) k_table_bits(int64_t n_words, int words, int V, const int16_t *next, uint32_t *live) {
    const int lane = threadIdx.x & 31;
    for (int64_t w = (int64_t)blockIdx.x * (NT / 32) + threadIdx.x / 32; w < n_words; w += (int64_t)gridDim.x * (NT / 32)) {
        const int64_t s = w / words;
        const int v = (int)(w % words) * 32 + lane;
        const uint32_t bits = __ballot_sync(0xffffffffu, v < V && next[s * V + v] >= 0);
        if (lane == 0) live[w] = bits;
    }
}

// blocks per sequence: four per SM over all sequences, one batch each at least
int select_blocks(int N, int K, int V) {
    const int64_t batches = (int64_t)K * ((V + 7 + BATCH - 1) / BATCH);
    const int64_t want = std::max<int64_t>(1, (152 * 4 + N - 1) / N);
    return (int)std::min(batches, want);
}

fa_status select_sizes(const char *fn, int32_t N, int32_t K, int32_t V, int32_t top) {
    if (N < 0 || N > 65535 || K < 1 || V < 1 || (int64_t)K * V >= 2147483648LL) return fa_refuse(fn, "N, K or V out of range");
    // the scan counts a row's cells in 32 bits up to two batches past its end, and beams and batches (where V is
    // small as many as beams) up to a launch's blocks past theirs
    if (std::max(K, V) > 2147483647 - 2 * BATCH) return fa_refuse(fn, "K or V out of range");
    if (top < 1 || top > FA_MAX_BEAM_TOP) return fa_refuse(fn, "top must be in [1, FA_MAX_BEAM_TOP]");
    return FA_OK;
}

}  // namespace

extern "C" fa_status fa_beam_select_workspace_bytes(int32_t N, int32_t K, int32_t V, int32_t top, size_t *bytes) {
    const char *fn = "fa_beam_select_workspace_bytes";
    if (!bytes) return fa_refuse(fn, "NULL argument");
    fa_status st = select_sizes(fn, N, K, V, top);
    if (st != FA_OK) return st;
    *bytes = (size_t)N * select_blocks(std::max(N, 1), K, V) * top * sizeof(key_t64);
    return FA_OK;
}

extern "C" fa_status fa_beam_select(int32_t dtype, int32_t N, int32_t K, int32_t V, int32_t top, const void *logp,
                                    int64_t logp_seq_stride, int64_t logp_beam_stride, const float *scores,
                                    const int32_t *states, int32_t S, const int16_t *next, const uint32_t *live,
                                    float *out_score, int32_t *out_parent, int32_t *out_token, int32_t *out_state,
                                    void *workspace, size_t ws_bytes, fa_stream stream) {
    const char *fn = "fa_beam_select";
    if (!fa_dtype_ok(dtype)) return fa_refuse(fn, "unknown dtype");
    fa_status st = select_sizes(fn, N, K, V, top);
    if (st != FA_OK) return st;
    if (S < 0 || S > FA_MAX_STATES) return fa_refuse(fn, "S out of [0, FA_MAX_STATES]");
    const bool aut = S > 0;
    if (aut != (states != nullptr) || aut != (next != nullptr) || aut != (live != nullptr) || aut != (out_state != nullptr))
        return fa_refuse(fn, "states, next, live and out_state go together with S > 0");
    if (N == 0) return FA_OK;
    if (!logp || !scores || !out_score || !out_parent || !out_token) return fa_refuse(fn, "NULL buffer");
    if ((uintptr_t)logp % fa_dtype_bytes(dtype)) return fa_refuse(fn, "logp is not aligned to its type");
    SelectArgs a;
    a.N = N; a.K = K; a.V = V; a.top = top; a.S = S; a.words = (V + 31) / 32;
    a.nb = select_blocks(N, K, V);
    const size_t need = (size_t)N * a.nb * top * sizeof(key_t64);
    if (ws_bytes < need || (need && !workspace))
        return fa_refuse(fn, ("workspace needs " + std::to_string(need) + " bytes").c_str(), FA_ERR_WORKSPACE_TOO_SMALL);
    if ((uintptr_t)workspace & 255) return fa_refuse(fn, "workspace not 256-byte aligned");
    // a sequence's scores and states are read before its results are written, other sequences' may be read later
    const size_t in = (size_t)N * K * 4, out = (size_t)N * top * 4;
    const bool same_rows = K == top || N == 1;
    auto in_place = [&](const void *x, const void *y) { return same_rows && x == y; };
    if ((fa_overlap(scores, in, out_score, out) && !in_place(scores, out_score)) || fa_overlap(scores, in, out_parent, out) ||
        fa_overlap(scores, in, out_token, out) || (aut && fa_overlap(scores, in, out_state, out)))
        return fa_refuse(fn, "scores overlaps an output");
    if (aut && ((fa_overlap(states, in, out_state, out) && !in_place(states, out_state)) || fa_overlap(states, in, out_score, out) ||
                fa_overlap(states, in, out_parent, out) || fa_overlap(states, in, out_token, out)))
        return fa_refuse(fn, "states overlaps an output");
    a.logp = logp; a.ln = logp_seq_stride; a.lk = logp_beam_stride;
    a.scores = scores; a.states = states; a.next = next; a.live = live;
    a.keys = (key_t64 *)workspace;
    a.out_score = out_score; a.out_parent = out_parent; a.out_token = out_token; a.out_state = out_state;
    cudaStream_t s = (cudaStream_t)stream;
    const size_t smem = ((size_t)PER * pushers(top) + (FULL + 1) * top) * 8;
    auto go = [&](auto tag) {
        using T = decltype(tag);
        if (smem > 40 * 1024) {
            cudaError_t e = cudaFuncSetAttribute(k_beam_scan<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return e;
        }
        k_beam_scan<T><<<dim3((unsigned)a.nb, (unsigned)N), NT, smem, s>>>(a);
        return cudaSuccess;
    };
    const cudaError_t e = dtype == FA_DTYPE_F32 ? go(0.0f) : dtype == FA_DTYPE_F16 ? go(__half()) : go(__nv_bfloat16());
    if (e != cudaSuccess) return fa_refuse(fn, cudaGetErrorString(e), FA_ERR_CUDA);
    if ((st = fa_launch_check("beam scan")) != FA_OK || a.nb == 1) return st;
    return fa_launch_second("beam merge", k_beam_merge, dim3((unsigned)N), NT, ((size_t)4 * pushers(top) + (FULL + 1) * top) * 8, s, a);
}

extern "C" fa_status fa_beam_reorder(int32_t N, int32_t K, int32_t top, int64_t words, const int32_t *src,
                                     const int32_t *parent, const int32_t *token, int64_t at, int32_t *dst,
                                     fa_stream stream) {
    const char *fn = "fa_beam_reorder";
    if (N < 0 || K < 0 || top < 0 || words < 0 || (int64_t)N * top > 2147483647) return fa_refuse(fn, "sizes out of range");
    if (token && (at < 0 || at >= words)) return fa_refuse(fn, "at must be in [0, words)");
    if ((int64_t)N * top == 0 || words == 0) return FA_OK;
    if ((K > 0 && !src) || !parent || !dst) return fa_refuse(fn, "NULL buffer");
    const unsigned gy = (unsigned)std::min<int64_t>((words + NT * 4 - 1) / (NT * 4), 1024);
    k_beam_reorder<<<dim3((unsigned)(N * top), gy), NT, 0, (cudaStream_t)stream>>>(K, top, words, src, parent, token, at, dst);
    return fa_launch_check("beam reorder");
}

extern "C" fa_status fa_beam_tables(const fa_automaton *aut, int16_t *next, uint32_t *live, fa_stream stream) {
    const char *fn = "fa_beam_tables";
    if (!aut) return fa_refuse(fn, "NULL automaton");
    if (!aut->is_dfa) return fa_refuse(fn, "the automaton is not deterministic", FA_ERR_UNSUPPORTED);
    if (!next || !live) return fa_refuse(fn, "NULL buffer");
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fa_refuse(fn, cudaGetErrorString(e), FA_ERR_CUDA);
    if (dev != aut->device) return fa_refuse(fn, "current device differs from the automaton's device");
    cudaStream_t s = (cudaStream_t)stream;
    const int S = aut->S, V = aut->V, E = aut->E, words = (V + 31) / 32;
    k_table_clear<<<152 * 8, NT, 0, s>>>((int64_t)S * V, next);
    fa_status st = fa_launch_check("beam tables");
    if (st != FA_OK) return st;
    // live is free until the last kernel: its first words hold the reachable states meanwhile
    k_table_reach<<<1, 1024, 0, s>>>(S, E, aut->accept_mask, aut->edge_src, aut->edge_dst, live);
    if ((st = fa_launch_check("beam tables")) != FA_OK) return st;
    if (E > 0) {
        k_table_fill<<<(unsigned)std::min(E, 152 * 64), NT, 0, s>>>(E, V, aut->lab_off, aut->lab_tok, aut->edge_src, aut->edge_dst, live, next);
        if ((st = fa_launch_check("beam tables")) != FA_OK) return st;
    }
    k_table_bits<<<152 * 16, NT, 0, s>>>((int64_t)S * words, words, V, next, live);
    return fa_launch_check("beam tables");
}
