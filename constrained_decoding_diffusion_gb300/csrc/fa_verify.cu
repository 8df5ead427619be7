// Verification of drafted tokens against a target's probabilities.
//
// The mathematics.  At a node with the target's row p (sum S0) and the draft's row q (sum Q), the distribution left
// after k rejections is r_k = max(p - l_k q, 0) / S_k with l_0 = 0, since
//     max(r_k - q / Q, 0) = max(p - l_k q - (S_k / Q) q, 0) / S_k,
// so l_{k+1} = l_k + S_k / Q and S_{k+1} = sum_v max(p(v) - l_{k+1} q(v), 0): a rejection costs one pass over the
// two rows and stores none.  Child x is accepted if u S_k q(x) < max(p(x) - l_k q(x), 0) Q.  Without a draft row q is
// one at x: accepted if u S_k < p(x), else S_{k+1} = S_k - p(x), with no pass at all.  The next token is found in
// the sums of the vocabulary's segments (one a warp) and then in its segment.
//
// Under an automaton both rows are those of its tokens alone, and a child with another token is passed over.  Of children
// drawn from the whole row those that are left are draws from the restricted one, so the result has the target's distribution
// whether or not the drafter knew the automaton; a rejection of the others would take from the target what they cannot stand for.
//
// A draw compares u with a sum over the vocabulary, so everything is kept as unevaluated sums of two floats (Knuth's and
// Dekker's exact additions and products, 46 bits or more): fp64 runs at two lanes a clock and SM here.  A row whose sum is far
// from one is taken times a power of two, so that S_k / Q and the low parts stay within fp32's range.
//
// A cluster of blocks takes a sequence: each block a slice of the vocabulary, from node to node, so that only the rows of
// nodes that are visited are read.  Every block gets every segment's sums and decides for itself, so that the cluster meets
// once a row; what else a decision rests on is read by the first block and sent to all, so that they never part ways
// whatever the inputs hold.
//
// What bounds it is the chain from node to node.  In eight blocks a row of 151936 takes 5.5 us with a draft (2900 cycles of
// additions, 14 a token, and their loads 6700 clocks; the sums of warps, the cluster's meeting and the decision 3500)
// and 4 without, the draw 3.  Measured in a graph: 64 sequences of 9 x 151936 fp32 with a draft 88 to 100 us (206 MB read, 2.3
// TB/s; the longest path takes 10 rows or more, and 36 clusters run at a time), 16 trees of 17 x 151936 bf16 under an automaton 25
// to 28, a chain of 5 x 32000 14 to 16.
// Tried and dropped: a ring of asynchronous copies in shared memory (5% slower, more instructions), two sums at a time in
// packed registers against one (equal: the packed addition takes twice as long), the next vectors loaded while
// these are added up (10% slower, registers), three blocks an SM with fewer vectors under way (8 to 15% slower), arrivals on
// barriers in the other blocks' memory for the cluster's (equal: either waits for the stores before), one block that decides
// and tells the others in a second meeting (5 to 9% slower).
#include <atomic>

#include <cooperative_groups.h>

#include "fa_lm.cuh"
#include "fa_verify_blocks.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int NT_LOG = 8, NT = 1 << NT_LOG, WARPS = NT / 32, MAX_CLUSTER = 16, SEGS = MAX_CLUSTER * WARPS, ROWS = 32;   // rows of a segment that the draw takes at a time

struct Sum { float h, l; };   // h + l

__device__ __forceinline__ Sum two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Sum fast_two_sum(float a, float b) {   // |a| >= |b|
    const float s = __fadd_rn(a, b);
    return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Sum operator+(Sum a, Sum b) {
    const Sum s = two_sum(a.h, b.h);
    return fast_two_sum(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
// Two floats in a register pair: one instruction adds, subtracts or multiplies both.
typedef unsigned long long Two;
__device__ __forceinline__ Two two(float a, float b) {
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 apart(Two a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}
__device__ __forceinline__ Two add2(Two a, Two b) { Two r; asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b)); return r; }
__device__ __forceinline__ Two sub2(Two a, Two b) { Two r; asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b)); return r; }
__device__ __forceinline__ Two mul2(Two a, Two b) { Two r; asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b)); return r; }
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) { Two r; asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c)); return r; }

// Two running sums: what each addition loses is added up apart.  Every few dozen terms the low parts are folded into the high
// ones: they would else grow with the terms and lose bits of their own.  Emulated in fp32, log-normal weights (sigma 4),
// 2048 lanes: a row's sum is off by 2^-41 at V = 10^7 and 2^-38 at 2.4 10^7 without it, by 2^-47 and 2^-48 with it
// (64 x 9 x 151936 90.5 -> 90.7 us; behind the additions rather than before the next loads 91.3).
struct Sums {
    Two h, l;
    __device__ __forceinline__ void add(Two b) {
        const Two s = add2(h, b), t = sub2(s, h);
        l = add2(l, add2(sub2(h, sub2(s, t)), sub2(b, t)));
        h = s;
    }
    __device__ __forceinline__ void add(Two b, Two low) {
        add(b);
        l = add2(l, low);
    }
    __device__ __forceinline__ void fold() {
        const Two s = add2(h, l);
        l = sub2(l, sub2(s, h));
        h = s;
    }
    __device__ __forceinline__ Sum first() const { return fast_two_sum(apart(h).x, apart(l).x); }
    __device__ __forceinline__ Sum second() const { return fast_two_sum(apart(h).y, apart(l).y); }
};
__device__ __forceinline__ Sum operator*(Sum a, float b) {
    const float h = __fmul_rn(a.h, b);
    return fast_two_sum(h, __fmaf_rn(a.l, b, __fmaf_rn(a.h, b, -h)));
}
__device__ __forceinline__ Sum operator-(Sum a) { return {-a.h, -a.l}; }
__device__ __forceinline__ bool operator<(Sum a, Sum b) { return (a + -b).h < 0.0f; }
// a / b: two quotients and what they leave over
__device__ __forceinline__ Sum operator/(Sum a, Sum b) {
    const float q0 = __fdiv_rn(a.h, b.h);
    const Sum r = a + -(b * q0);
    const float q1 = __fdiv_rn(r.h, b.h);
    const Sum t = r + -(b * q1);
    return fast_two_sum(q0, __fadd_rn(q1, __fdiv_rn(t.h, b.h)));
}
__device__ __forceinline__ Sum shfl_xor(Sum a, int o) {
    return {__shfl_xor_sync(0xffffffffu, a.h, o), __shfl_xor_sync(0xffffffffu, a.l, o)};
}
// without bringing the low part below the high one's last place, which a chain of sums needs only once
__device__ __forceinline__ Sum loosely(Sum a, Sum b) {
    const Sum s = two_sum(a.h, b.h);
    return {s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l))};
}
__device__ __forceinline__ Sum warp_sum(Sum a) {
#pragma unroll
    for (int o = 16; o; o >>= 1) a = loosely(a, shfl_xor(a, o));
    return fast_two_sum(a.h, a.l);
}
// two sums over the warp, side by side
__device__ __forceinline__ void warp_sums(Sum &a, Sum &b) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const Sum x = shfl_xor(a, o), y = shfl_xor(b, o);
        a = loosely(a, x);
        b = loosely(b, y);
    }
    a = fast_two_sum(a.h, a.l);
    b = fast_two_sum(b.h, b.l);
}
// inclusive sums over the lanes
__device__ __forceinline__ Sum warp_scan(Sum a) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sum up = {__shfl_up_sync(0xffffffffu, a.h, o), __shfl_up_sync(0xffffffffu, a.l, o)};
        if ((threadIdx.x & 31) >= o) a = loosely(up, a);
    }
    return fast_two_sum(a.h, a.l);
}

// max(p - l q, 0) as two floats
__device__ __forceinline__ Sum left(float p, float q, Sum l) {
    const float h = __fmul_rn(l.h, q), e = __fmaf_rn(l.l, q, __fmaf_rn(l.h, q, -h));
    const Sum d = two_sum(p, -h);
    const Sum r = fast_two_sum(d.h, __fsub_rn(d.l, e));
    return r.h > 0.0f ? r : Sum{0.0f, 0.0f};
}

// the same for two elements
__device__ __forceinline__ void left2(Two p, Two q, Two lh, Two ll, Two &high, Two &low) {
    const Two n = mul2(lh, q ^ 0x8000000080000000ull);   // -l q
    const Two e = fma2(ll, q, fma2(lh, q, n));            // and what that lacks
    const Two s = add2(p, n), t = sub2(s, p), d = sub2(add2(sub2(p, sub2(s, t)), sub2(n, t)), e);
    const Two r = add2(s, d);
    const float2 h = apart(r), l = apart(sub2(d, sub2(r, s)));
    high = two(h.x > 0.0f ? h.x : 0.0f, h.y > 0.0f ? h.y : 0.0f);
    low = two(h.x > 0.0f ? l.x : 0.0f, h.y > 0.0f ? l.y : 0.0f);
}

// x 2^e for |e| < 250, by two powers that are floats themselves; exact but for bits below 2^-149
__device__ __forceinline__ float scaled(float x, int e) {
    auto power = [](int i) { return __int_as_float((127 + i) << 23); };
    return x * power(e / 2) * power(e - e / 2);
}
// A sum beyond 2^48, not finite, or below 2^-48.  (Sums between leave quotients and products that fp32 holds with their low parts.
// fp16's sums are all between: its weights lie within 2^-24 and 2^16, and a row has fewer than 2^31.)
__device__ __forceinline__ bool far(float h) { return !(h >= 0x1p-48f && h < 0x1p48f); }
// the power of two that brings such a sum near one (a draft's beyond fp32 is 2^159 at most, of finite weights); 0: none does, or need be
__device__ __forceinline__ int power_for(float h) {
    if (!far(h) || h == 0.0f) return 0;
    return h < INFINITY ? 127 - (__float_as_int(h) >> 23) : -140;
}

// x where it is a positive finite number, else 0
__device__ __forceinline__ float weight(float x) { return __float_as_uint(x) - 1u < 0x7f7fffffu ? x : 0.0f; }

struct VerifyArgs {
    int B, T, V, S, words;
    const void *target, *draft;
    int64_t tb, tr, db, dr;
    const int32_t *tokens, *parents, *count;
    const float *u;
    const int32_t *states;
    const int16_t *next;
    const uint32_t *live;
    int32_t *path, *kept, *token, *state;
};

struct Plan {          // what a block's first warp tells the others
    int action;        // draw from segment `segment`, go to `node` with `state`, or sweep again, with l or for other powers
    int node, state, segment, tried;
    int ep, eq;        // powers of two by which both rows are multiplied
    Sum l, before, goal;   // the sum before the segment, and what the draw looks for
};
enum { DRAW = 0, NODE = 1, SWEEP = 2, RESUM = 3 };

struct Shared {
    Plan plan;
    Sum seg[2][SEGS], seg_q[2][SEGS];   // the sums of all segments, of this sweep and the next (zero where there are fewer)
    Sum row[ROWS];                      // (the draw) of the rows of one segment
    int use, last;
};

// A drafted token.
struct __align__(16) Child { int parent, token; float u, unused; };
constexpr size_t kBytesOfToken = sizeof(Child) + sizeof(float2) + 3 * sizeof(int);   // with its weights, place on the path ...

// A row of the vocabulary in vectors of 16 bytes, counted from the aligned address at or before its start.
template <class T> struct Row {
    static constexpr int N = fa_vec<T>::N;
    const T *p;
    int V;
    // elements i .. i + N - 1, zero outside the row
    __device__ __forceinline__ uint4 load(int i) const {
        if (i >= 0 && i <= V - N && !((uintptr_t)(p + i) & 15)) return __ldg(reinterpret_cast<const uint4 *>(p + i));
        float f[N];
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] = i + e >= 0 && i + e < V ? fa_to_f32(p[i + e]) : 0.0f;
        return fa_pack(f, T());
    }
};

// bits i .. i + 7 of a row of live bits (any past its end), -8 < i; without a branch, so that loads go on behind it
__device__ __forceinline__ uint32_t bits_at(const uint32_t *live, int words, int i) {
    const int w = max(i, 0) >> 5;
    const uint32_t lo = __ldg(live + w), hi = __ldg(live + min(w + 1, words - 1));
    return i < 0 ? lo << (-i & 31) : __funnelshift_r(lo, hi, i & 31);
}

// What a block knows of the current node.
template <class T, bool DRAFT> struct Node {
    static constexpr int N = fa_vec<T>::N;
    Row<T> p, q;
    const uint32_t *live;
    int words, lead, chunks, per;                        // of the row: first element's place, vectors, vectors of a segment
    Sum lam;
    __device__ __forceinline__ uint32_t bits(int c) const { return live ? bits_at(live, words, c * N - lead) : 0xffffffffu; }
    __device__ __forceinline__ int segment(int x) const { return (x + lead) / N / per; }
    // two elements' worth of sums for every vector: fresh, the target's and the draft's sum; else those of even and of odd
    // elements
    template <bool FRESH, bool LIVE> __device__ __forceinline__ void take(Sums &run, uint4 x, uint4 y, uint32_t b) const {
        float f[N], g[N];
        fa_unpack(x, f, T());
        if (DRAFT) fa_unpack(y, g, T());
        // all of them nonnegative and finite: the common case
        uint32_t most = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) most = max(most, max(__float_as_uint(f[e]), DRAFT ? __float_as_uint(g[e]) : 0u));
        if (most >= 0x7f800000u) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                f[e] = weight(f[e]);
                if (DRAFT) g[e] = weight(g[e]);
            }
        }
        if (LIVE) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int in = (int)(b << (31 - e)) >> 31;
                f[e] = __int_as_float(__float_as_int(f[e]) & in);
                if (DRAFT) g[e] = __int_as_float(__float_as_int(g[e]) & in);
            }
        }
        if (DRAFT && FRESH) {
#pragma unroll
            for (int e = 0; e < N; ++e) run.add(two(f[e], g[e]));
        } else {
            const Two lh = two(lam.h, lam.h), ll = two(lam.l, lam.l);
#pragma unroll
            for (int e = 0; e < N; e += 2) {
                if (!DRAFT) { run.add(two(f[e], f[e + 1])); continue; }
                Two high, low;
                left2(two(f[e], f[e + 1]), two(g[e], g[e + 1]), lh, ll, high, low);
                run.add(high, low);
            }
        }
    }
    // vectors c, c + step, ... below c1 of both rows (zeros past it): plain loads for those that the row fills, all
    // issued before the row's ends or a draft row of another alignment are looked after
    template <int U> __device__ __forceinline__ void fetch(int c, int step, int c1, uint4 (&x)[U], uint4 (&y)[U]) const {
        const int from = lead ? 1 : 0, to = (p.V + lead) % N ? chunks - 1 : chunks;
        const uint4 *pv = reinterpret_cast<const uint4 *>(p.p - lead) + c, *qv = reinterpret_cast<const uint4 *>(q.p - lead) + c;
        const bool together = !((uintptr_t)qv & 15);
        bool left_over = false;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int at = c + step * k;
            const bool whole = at >= from && at < min(to, c1);
            x[k] = y[k] = make_uint4(0, 0, 0, 0);
            if (whole) x[k] = __ldg(pv + step * k);
            if (DRAFT && whole && together) y[k] = __ldg(qv + step * k);
            left_over |= at < c1 && !(whole && (!DRAFT || together));
        }
        if (left_over) {
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int at = c + step * k;
                if (at >= c1) continue;
                x[k] = p.load(at * N - lead);
                if (DRAFT) y[k] = q.load(at * N - lead);
            }
        }
    }
    // the sums of vectors c0 + lane, c0 + lane + 32, ... below c1, U of them under way; FRESH: l = 0, and the draft's sum too
    template <bool FRESH, bool LIVE> __device__ __forceinline__ void sweep(int c0, int c1, Sum &w, Sum &wq) const {
        constexpr int U = DRAFT ? 5 : 8;
        Sums run = {0ull, 0ull};
        for (int c = c0 + (threadIdx.x & 31); c < c1; c += 32 * U) {
            run.fold();
            uint4 x[U], y[U];
            uint32_t b[U];
#pragma unroll
            for (int k = 0; k < U; ++k) b[k] = LIVE && c + 32 * k < c1 ? bits_at(live, words, (c + 32 * k) * N - lead) : 0u;
            fetch(c, 32, c1, x, y);
#pragma unroll
            for (int k = 0; k < U; ++k) take<FRESH, LIVE>(run, x[k], y[k], b[k]);
        }
        w = run.first();
        wq = run.second();
        if (!(DRAFT && FRESH)) w = w + wq;
    }
    // the weights of vector c for the draw, without the n tokens of `tried`, and their sum
    __device__ __forceinline__ Sum weigh(int c, uint4 x, uint4 y, uint32_t b, Sum (&v)[N], const int *tried, int n) const {
        const int i = c * N - lead;
        float f[N], g[N];
        fa_unpack(x, f, T());
        if (DRAFT) fa_unpack(y, g, T());
        for (int k = 0; k < n; ++k) {
            const uint32_t e = (uint32_t)(tried[k] - i);
            if (e < N) b &= ~(1u << e);
        }
        Sum sum = {0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float pe = b >> e & 1 ? weight(f[e]) : 0.0f;
            v[e] = DRAFT ? left(pe, weight(g[e]), lam) : Sum{pe, 0.0f};
            sum = sum + v[e];
        }
        return sum;
    }
};

// What few rows need lies apart from the kernel, which slows down with the code between its loops (64 x 9 x 151936 fp32: a choice in
// the loops 96 us, beside them 93, apart 91, and no scales at all 90).

// elements times 2^e
template <class T> __device__ __noinline__ uint4 scaled_vector(uint4 x, int e) {
    float f[fa_vec<T>::N];
    fa_unpack(x, f, T());
#pragma unroll
    for (float &y : f) y = scaled(y, e);
    return fa_pack(f, T());
}
// The sums of a segment of rows that are scaled, a vector at a time.
struct Pair { Sum w, wq; };
template <class T, bool DRAFT>
__device__ __noinline__ Pair sweep_scaled(const T *p, const T *q, int V, const uint32_t *live, int words, Sum lam, int ep, int eq, bool fresh,
                                          int c0, int c1, int lead, int chunks) {
    const Node<T, DRAFT> at = {{p, V}, {q, V}, live, words, lead, chunks, 0, lam};
    Sums run = {0ull, 0ull};
    for (int c = c0 + (threadIdx.x & 31); c < c1; c += 32) {
        uint4 x[1], y[1];
        at.fetch(c, 32, c1, x, y);
        x[0] = scaled_vector<T>(x[0], ep);
        if (DRAFT) y[0] = scaled_vector<T>(y[0], eq);
        if (fresh || !DRAFT) at.template take<true, true>(run, x[0], y[0], at.bits(c));
        else at.template take<false, true>(run, x[0], y[0], at.bits(c));
        run.fold();
    }
    Pair r = {run.first(), run.second()};
    if (!(DRAFT && fresh)) r.w = r.w + r.wq;
    return r;
}

template <class T, bool DRAFT>
__global__ void __launch_bounds__(NT, 2) k_verify(VerifyArgs a) {
    constexpr int N = fa_vec<T>::N;
    constexpr bool SCALES = !std::is_same<T, __half>::value;
    __shared__ Shared sh;
    extern __shared__ Child child[];
    float2 *pq = reinterpret_cast<float2 *>(child + a.T);   // the target's and the draft's weight
    int *after = reinterpret_cast<int *>(pq + a.T), *path = after + a.T, *tried = path + a.T;
    const cg::cluster_group cluster = cg::this_cluster();
    const int C = cluster.num_blocks(), log_c = 31 - __clz(C), rank = cluster.block_rank(), b = blockIdx.x >> log_c;
    // (what all threads of a warp have alike goes through a shuffle where later shuffles depend on it)
    auto alike = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    const int tid = threadIdx.x, warp = alike(tid >> 5), lane = tid & 31;
    const int use = a.count ? min(max(a.count[b], 0), a.T) : a.T;
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    path[0] = 0;
    for (int i = C * WARPS + tid; i < SEGS; i += NT)
        for (int k = 0; k < 2; ++k) sh.seg[k][i] = sh.seg_q[k][i] = {0.0f, 0.0f};
    // the drafted token j, and its weights in its parent's rows
    auto read = [&](int j) {
        const int64_t i = (int64_t)b * a.T + j;
        return Child{a.parents[i], a.tokens[i], a.u[i], 0.0f};
    };
    auto weights = [&](int j, Child c) {
        float2 w = {0.0f, 0.0f};
        if ((unsigned)c.parent < (unsigned)j && (unsigned)c.token < (unsigned)a.V) {
            w.x = fa_to_f32(((const T *)a.target + b * a.tb + c.parent * a.tr)[c.token]);
            if (DRAFT) w.y = fa_to_f32(((const T *)a.draft + b * a.db + c.parent * a.dr)[c.token]);
        }
        return w;
    };
    Child own = {-1, -1, 0.0f, 0.0f};
    if (rank == 0 && tid < a.T) own = read(tid);
    // all blocks have started before the first store to another
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    // stores x at y in every block
    auto tell = [&](auto *y, auto x) {
#pragma unroll
        for (int c = 0; c < MAX_CLUSTER; ++c)
            if (c < C) *cluster.map_shared_rank(y, c) = x;
    };
    float2 own_pq = {0.0f, 0.0f};
    if (rank == 0) {
        for (int j = tid; j < a.T; j += NT) tell(child + j, j == tid ? own : read(j));
        if (tid == 0) tell(&sh.use, use);
        if (tid < a.T) own_pq = weights(tid, own);        // under way during the first sweep
    }
    // kept by a block's first lane, and the same in all blocks
    int j = 1, kept = use > 0 ? 1 : 0, n_tried = 0;
    Sum l = {0.0f, 0.0f}, old_l = l;
    bool again = false;                                  // this sweep only restores the sums of old_l
    bool probing = false;                                // this sweep is a rejection's
    Sum total_q = {0.0f, 0.0f};
    int node = 0, state = a.S ? a.states[b] : 0;
    bool entered = true, fresh = true, first = true;     // a new node, sums with l = 0, the first turn
    int ep = 0, eq = 0;
    Node<T, DRAFT> at;
    at.words = a.words;
    __syncthreads();
    for (int turn = 0;; turn ^= 1) {
        Sum *const seg = sh.seg[turn], *const seg_q = sh.seg_q[turn];
        // (nothing that a block reads for itself decides how often the cluster meets)
        const bool any = use > 0 && (!a.S || (unsigned)state < (unsigned)a.S);
        if (entered) {
            at.p = {(const T *)a.target + b * a.tb + node * a.tr, a.V};
            at.q = {DRAFT ? (const T *)a.draft + b * a.db + node * a.dr : nullptr, a.V};
            at.live = a.S && any ? a.live + (int64_t)state * a.words : nullptr;
            at.lead = (int)(((uintptr_t)at.p.p / sizeof(T)) % N);
            at.chunks = (int)(((int64_t)a.V + at.lead + N - 1) / N);
            at.per = ((at.chunks + (NT << log_c) - 1) >> (NT_LOG + log_c)) * 32;
            at.lam = {0.0f, 0.0f};
        }
        // where the automaton goes by a child, one a thread (and the rest of a long draft below): under way during the sweep
        const int mine_too = node + 1 + tid;
        auto is_child = [&](int j) { return child[j].parent == node && (unsigned)child[j].token < (unsigned)a.V; };
        auto goes = [&](int j) { return any ? a.next[(int64_t)state * a.V + child[j].token] : -1; };
        const bool moves = a.S && rank == 0 && entered && mine_too < use && is_child(mine_too);
        const int to = moves ? goes(mine_too) : -1;
        // ---- this warp's segment
        const int mine = rank * WARPS + warp, s0 = mine * at.per, s1 = min(s0 + at.per, at.chunks);
        Sum w = {0.0f, 0.0f}, wq = {0.0f, 0.0f};
        if (any) {
            if (SCALES && (ep | eq)) {
                const Pair r = sweep_scaled<T, DRAFT>(at.p.p, at.q.p, a.V, at.live, at.words, at.lam, ep, eq, fresh, s0, s1, at.lead, at.chunks);
                w = r.w;
                wq = r.wq;
            } else if (fresh || !DRAFT) {
                if (at.live) at.template sweep<true, true>(s0, s1, w, wq);
                else at.template sweep<true, false>(s0, s1, w, wq);
            } else {
                if (at.live) at.template sweep<false, true>(s0, s1, w, wq);
                else at.template sweep<false, false>(s0, s1, w, wq);
            }
        }
        if (DRAFT && fresh) warp_sums(w, wq);
        else w = warp_sum(w);
        // (the first lane's, to the last bit, for all blocks)
        w = {__shfl_sync(0xffffffffu, w.h, 0), __shfl_sync(0xffffffffu, w.l, 0)};
        if (DRAFT && fresh) wq = {__shfl_sync(0xffffffffu, wq.h, 0), __shfl_sync(0xffffffffu, wq.l, 0)};
        if (lane < C) {
            *cluster.map_shared_rank(seg + mine, lane) = w;
            if (DRAFT && fresh) *cluster.map_shared_rank(seg_q + mine, lane) = wq;
        }
        if (moves) tell(after + mine_too, to);
        if (rank == 0 && first) {
            for (int j = tid; j < a.T; j += NT) {
                const float2 x = j == tid ? own_pq : weights(j, child[j]);
                tell(pq + j, make_float2(weight(x.x), weight(x.y)));
            }
        }
        if (a.S && rank == 0 && entered)
            for (int j = mine_too + NT; j < use; j += NT)
                if (is_child(j)) tell(after + j, goes(j));
        first = false;
        cluster.sync();
        if (warp == 0) {
            const int use = sh.use;
            static_assert(SEGS == 128, "four segments of a lane at most");
            const int each = C * WARPS > 64 ? 4 : 2;      // segments of a lane
            auto of_lane = [&](const Sum *x) {
                Sum y = x[lane * each] + x[lane * each + 1];
                if (each == 4) y = y + (x[lane * 4 + 2] + x[lane * 4 + 3]);
                return y;
            };
            Sum total = of_lane(seg), t = {0.0f, 0.0f};
            if (DRAFT && fresh) t = of_lane(seg_q);
            if (fresh) {
                n_tried = 0;
                l = {0.0f, 0.0f};
                if (DRAFT) warp_sums(total, t);
                total_q = t;
            }
            if (!DRAFT || !fresh) total = warp_sum(total);
            Plan plan = {};
            const bool some = total.h > 0.0f && total.h < INFINITY;
            if (lane == 0) {
                // Rows whose sums are far from one are summed again, times powers of two that bring them near it, so that quotients,
                // products and their low parts stay within fp32.
                const bool again_scaled = SCALES && fresh && some && !(ep | eq) && (far(total.h) || (DRAFT && far(total_q.h)));
                if (again_scaled) {
                    ep = power_for(total.h);
                    eq = DRAFT ? power_for(total_q.h) : 0;
                }
                if (again_scaled && (ep | eq)) {
                    plan.action = RESUM;
                } else if (probing && !again && !(total.h > 0.0f)) {
                    // nothing would be left: the distribution stays as it was
                    l = old_l;
                    plan.action = SWEEP;
                    plan.l = l;
                    again = true;
                } else {
                    again = probing = false;
                    if (!some) j = use;                              // nothing can be accepted
                    const bool drafts = DRAFT && total_q.h > 0.0f;   // a row without weight: q(x) = 0
                    for (; j < use; ++j) {
                        const Child x = child[j];
                        if (x.parent != node || (unsigned)x.token >= (unsigned)a.V) continue;
                        if (a.S && after[j] < 0) continue;           // not of the distributions that are compared
                        float p = pq[j].x, q = pq[j].y;
                        if (SCALES && (ep | eq)) {
                            p = scaled(p, ep);
                            q = scaled(q, eq);
                        }
                        bool take, known = false;
                        Sum ratio = {0.0f, 0.0f};
                        if (DRAFT) {
                            // 24 bits mostly tell, without the quotient; where they do not, or leave fp32's range, 48 do
                            const Sum rest = left(p, q, l);
                            const float less = total.h * q * x.u, more = rest.h * total_q.h;
                            take = less > 1e-30f && more < 1e30f && less * 1.0001f < more;
                            if (!take) {
                                if (drafts) ratio = total / total_q;
                                take = ratio * q * x.u < rest;
                            }
                        } else {
                            for (int i = 0; i < n_tried; ++i) known |= tried[i] == x.token;
                            take = !known && total * x.u < Sum{p, 0.0f};
                        }
                        if (take) {
                            plan.action = NODE;
                            plan.node = j;
                            plan.state = after[j];
                            path[kept++] = j;
                            ++j;
                            break;
                        }
                        if (DRAFT) {
                            if (!drafts) continue;
                            old_l = l;
                            l = l + ratio;
                            plan.action = SWEEP;
                            plan.l = l;
                            probing = true;
                            ++j;
                            break;
                        }
                        if (known || p == 0.0f) continue;
                        const Sum rest = total + Sum{-p, 0.0f};
                        if (!(rest.h > 0.0f)) continue;
                        total = rest;
                        Sum &from = seg[at.segment(x.token)];
                        from = from + Sum{-p, 0.0f};
                        tried[n_tried++] = x.token;
                    }
                    plan.goal = total * child[0].u;
                }
            }
            plan.action = __shfl_sync(0xffffffffu, plan.action, 0);
            if (plan.action == DRAW) {
                __syncwarp();                             // what the first lane took from segments is seen
                // the segment that holds the draw
                const Sum goal = {__shfl_sync(0xffffffffu, plan.goal.h, 0), __shfl_sync(0xffffffffu, plan.goal.l, 0)};
                const int i0 = lane * each, i1 = i0 + each;
                Sum here = {0.0f, 0.0f};
                bool weighs = false;
                for (int i = i0; i < i1; ++i) {
                    here = here + seg[i];
                    weighs |= seg[i].h > 0.0f;
                }
                const Sum upto = warp_scan(here);
                const Sum start = {__shfl_up_sync(0xffffffffu, upto.h, 1), __shfl_up_sync(0xffffffffu, upto.l, 1)};
                const uint32_t past = __ballot_sync(0xffffffffu, weighs && goal < upto), all = __ballot_sync(0xffffffffu, weighs);
                const int who = past ? __ffs(past) - 1 : all ? 31 - __clz(all) : 0;
                plan.segment = -1;
                if (lane == who && all && some) {
                    Sum before = lane ? start : Sum{0.0f, 0.0f};
                    for (int i = i0; i < i1; ++i) {
                        if (!(seg[i].h > 0.0f)) continue;
                        const Sum next = before + seg[i];
                        plan.segment = i;                 // the last one if rounding hides all others
                        plan.before = before;
                        if (goal < next) break;
                        before = next;
                    }
                }
                plan.segment = __shfl_sync(0xffffffffu, plan.segment, who);
                plan.before = {__shfl_sync(0xffffffffu, plan.before.h, who), __shfl_sync(0xffffffffu, plan.before.l, who)};
                plan.goal = goal;
            }
            plan.node = __shfl_sync(0xffffffffu, plan.node, 0);
            plan.state = __shfl_sync(0xffffffffu, plan.state, 0);
            plan.l.h = __shfl_sync(0xffffffffu, plan.l.h, 0);
            plan.l.l = __shfl_sync(0xffffffffu, plan.l.l, 0);
            plan.tried = __shfl_sync(0xffffffffu, n_tried, 0);
            plan.ep = ep;
            plan.eq = eq;
            if (lane == 0) sh.plan = plan;
        }
        __syncthreads();
        const int action = alike(sh.plan.action);
        entered = action == NODE;
        fresh = entered || action == RESUM;
        if (entered) {
            node = alike(sh.plan.node);
            state = alike(sh.plan.state);
            ep = eq = 0;
            continue;
        }
        if (SCALES && action == RESUM) {
            ep = alike(sh.plan.ep);
            eq = alike(sh.plan.eq);
            continue;
        }
        if (action == SWEEP) {
            at.lam = sh.plan.l;
            continue;
        }
        break;
    }
    // ---- the draw: the block that has the segment sums its rows of 32 vectors, and a warp takes the row that holds it
    // (nothing is read from or written to another block from here on: each may end)
    const int segment = alike(sh.plan.segment), n = DRAFT ? 0 : alike(sh.plan.tried);
    if (segment < 0 && n == 0) {
        if (rank == 0 && tid == 0) {
            a.token[b] = -1;
            if (a.state) a.state[b] = -1;
        }
    } else if (rank == max(segment, 0) / WARPS) {
        Sum goal = sh.plan.goal;
        Sum before = sh.plan.before;
        Sum v[N];
        auto scale = [&](auto &x, auto &y) {
            if (SCALES && (ep | eq))
                for (auto &v : x) v = scaled_vector<T>(v, ep);
            if (SCALES && DRAFT && (ep | eq))
                for (auto &v : y) v = scaled_vector<T>(v, eq);
        };
        // Where tried tokens have left a rounding of a segment and no other weight, the first weight behind it is the next token,
        // or the last before it.
        int c0 = max(segment, 0) * at.per, c1 = segment < 0 ? 0 : min(c0 + at.per, at.chunks);
        int held = -1;                                    // the last row with a weight so far
        for (int look = 0; look < (n ? 3 : 1) && held < 0; ++look) {
            if (look == 1) {
                c0 = c1;
                c1 = at.chunks;
                before = {0.0f, 0.0f};
                goal = {-1.0f, 0.0f};
            } else if (look == 2) {
                c1 = segment * at.per;
                c0 = 0;
            }
            bool found_row = false;
            for (int r0 = c0; r0 < c1; r0 += 32 * ROWS) {
                constexpr int U = ROWS / WARPS;
                Sum sums[U];
                uint4 x[U], y[U];
                uint32_t bits[U];
                const int c = r0 + tid;
                at.fetch(c, NT, c1, x, y);
                scale(x, y);
#pragma unroll
                for (int k = 0; k < U; ++k) bits[k] = c + NT * k < c1 ? at.bits(c + NT * k) : 0u;
#pragma unroll
                for (int k = 0; k < U; ++k) sums[k] = at.weigh(c + NT * k, x[k], y[k], bits[k], v, tried, n);
#pragma unroll
                for (int k = 0; k < ROWS / WARPS; k += 2) warp_sums(sums[k], sums[k + 1]);
                __syncthreads();                          // the last rows' sums have been read
                if (lane == 0)
#pragma unroll
                    for (int k = 0; k < ROWS / WARPS; ++k) sh.row[warp + WARPS * k] = sums[k];
                __syncthreads();
                // the rows' sums in the lanes
                const Sum mine = sh.row[lane], upto = warp_scan(lane ? mine : before + mine);
                const uint32_t holds = __ballot_sync(0xffffffffu, mine.h > 0.0f && goal < upto), some = __ballot_sync(0xffffffffu, mine.h > 0.0f);
                if (some) held = r0 + 32 * (31 - __clz(some));
                const int who = holds ? __ffs(holds) - 1 : 31;
                if (holds) held = r0 + 32 * who;
                const int prior = holds ? who - 1 : 31;
                const Sum next = {__shfl_sync(0xffffffffu, upto.h, max(prior, 0)), __shfl_sync(0xffffffffu, upto.l, max(prior, 0))};
                if (prior >= 0) before = next;
                if (holds) { found_row = true; break; }
            }
            if (!found_row) goal = {INFINITY, 0.0f};   // rounding hid the draw: the last element with a weight
        }
        if (warp == 0 && held >= 0) {
            const int c = held + lane;
            uint4 x[1], y[1];
            at.fetch(c, 32, c1, x, y);
            scale(x, y);
            const Sum sum = at.weigh(c, x[0], y[0], c < c1 ? at.bits(c) : 0u, v, tried, n), upto = warp_scan(lane ? sum : before + sum);
            const uint32_t past = __ballot_sync(0xffffffffu, sum.h > 0.0f && goal < upto), some = __ballot_sync(0xffffffffu, sum.h > 0.0f);
            const int pick = past ? __ffs(past) - 1 : 31 - __clz(some);
            Sum run = {__shfl_up_sync(0xffffffffu, upto.h, 1), __shfl_up_sync(0xffffffffu, upto.l, 1)};   // of the lanes before, then through the elements
            if (lane == 0) run = before;
            if (lane == pick) {
                int found = -1;
                bool done = false;
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    if (done || !(v[e].h > 0.0f)) continue;
                    run = run + v[e];
                    found = c * N - at.lead + e;
                    done = goal < run;
                }
                a.token[b] = found;
                if (a.state) a.state[b] = a.next[(int64_t)state * a.V + found];
            }
        } else if (tid == 0 && held < 0) {                // all that weighed has been tried
            a.token[b] = -1;
            if (a.state) a.state[b] = -1;
        }
    }
    if (rank == 0) {
        if (tid == 0) { sh.last = kept; a.kept[b] = kept; }
        __syncthreads();
        const int n = sh.last;
        for (int i = tid; i < a.T; i += NT) a.path[(int64_t)b * a.T + i] = i < n ? path[i] : -1;
    }
}

template <class T, bool DRAFT> cudaLaunchConfig_t config(cudaLaunchAttribute *at, int B, int cluster, int tokens, cudaStream_t s) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)B * cluster);
    c.blockDim = dim3(NT);
    c.dynamicSmemBytes = tokens * kBytesOfToken;
    c.stream = s;
    c.attrs = at;
    c.numAttrs = 1;
    return c;
}

// The clusters of sixteen blocks that the current device runs at a time: 0 where it has none that large, which is beyond the portable
// size.  Asked once a device, for the longest draft.
template <class T, bool DRAFT> int wide_clusters() {
    constexpr int DEVICES = 64;
    static std::atomic<int> known[DEVICES];               // one more than the answer
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = DEVICES;
    if (dev < DEVICES && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n - 1;
    cudaLaunchAttribute at[1];
    const cudaLaunchConfig_t c = config<T, DRAFT>(at, 1, MAX_CLUSTER, FA_MAX_DRAFT, nullptr);
    cudaError_t e = cudaFuncSetAttribute(k_verify<T, DRAFT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, k_verify<T, DRAFT>, &c);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();                         // the launch's own is the one that counts
        n = 0;
    }
    if (dev < DEVICES) known[dev].store(n + 1, std::memory_order_relaxed);
    return n;
}

template <class T, bool DRAFT> void launch(const VerifyArgs &a, cudaStream_t s) {
    auto blocks = [&](int wide) { return fa_verify_blocks(a.B, a.V, sizeof(T), DRAFT, a.S > 0, wide); };
    int cluster = blocks(a.V >= 98304 ? wide_clusters<T, DRAFT>() : 0);
    if (cluster > 8 && cudaFuncSetAttribute(k_verify<T, DRAFT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
        (void)cudaGetLastError();
        cluster = blocks(0);
    }
    cudaLaunchAttribute at[1];
    const cudaLaunchConfig_t c = config<T, DRAFT>(at, a.B, cluster, a.T, s);
    (void)cudaLaunchKernelEx(&c, k_verify<T, DRAFT>, a);   // its error is the one the check reads
}

}  // namespace

extern "C" fa_status fa_verify(int32_t dtype, int32_t B, int32_t T, int32_t V, const void *target, int64_t target_batch_stride,
                               int64_t target_row_stride, const void *draft, int64_t draft_batch_stride,
                               int64_t draft_row_stride, const int32_t *tokens, const int32_t *parents, const int32_t *count,
                               const float *u, const int32_t *states, int32_t S, const int16_t *next, const uint32_t *live,
                               int32_t *path, int32_t *kept, int32_t *token, int32_t *state, fa_stream stream) {
    const char *fn = "fa_verify";
    if (!fa_dtype_ok(dtype)) return fa_refuse(fn, "unknown dtype");
    if (B < 0 || B > 65535 || T < 1 || T > FA_MAX_DRAFT || V < 1 || V >= 2147483647 - 65536)
        return fa_refuse(fn, "B, T or V out of range");
    if (S < 0 || S > FA_MAX_STATES) return fa_refuse(fn, "S out of range");
    if ((S > 0) != (states != nullptr) || (S > 0) != (next != nullptr) || (S > 0) != (live != nullptr))
        return fa_refuse(fn, "states, next and live go together with S");
    if (B == 0) return FA_OK;
    if (!target || !tokens || !parents || !u || !path || !kept || !token || (S > 0 && !state)) return fa_refuse(fn, "NULL buffer");
    const int es = fa_dtype_bytes(dtype);
    if (((uintptr_t)target | (uintptr_t)draft) % es) return fa_refuse(fn, "target and draft must be aligned to their type");
    const VerifyArgs a{B, T, V, S, (V + 31) / 32, target, draft, target_batch_stride, target_row_stride, draft_batch_stride,
                       draft_row_stride, tokens, parents, count, u, states, next, live, path, kept, token, S > 0 ? state : nullptr};
    auto go = [&](auto tag) {
        using T_ = decltype(tag);
        if (draft) launch<T_, true>(a, (cudaStream_t)stream);
        else launch<T_, false>(a, (cudaStream_t)stream);
    };
    if (dtype == FA_DTYPE_F32) go(0.0f);
    else if (dtype == FA_DTYPE_F16) go(__half());
    else go(__nv_bfloat16());
    return fa_launch_check("verify");
}
