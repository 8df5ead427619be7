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
// A draw compares u with a sum over the vocabulary, so everything is kept as unevaluated sums of two floats (Knuth's and
// Dekker's exact additions and products, 46 bits or more): fp64 runs at two lanes a clock and SM here.
//
// A cluster of blocks takes a sequence: each block a slice of the vocabulary, from node to node.  The first
// block decides and tells the others, so that they never part ways whatever the inputs hold.
#include <cooperative_groups.h>

#include "fa_lm.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int NT = 512, WARPS = NT / 32, MAX_CLUSTER = 8;

// vectors of a thread under way, and the distance from one to the next (the target's and the draft's) in the ring
template <bool DRAFT> constexpr int RING = DRAFT ? 5 : 8;
template <bool DRAFT> constexpr int PER = DRAFT ? 2 * NT : NT;

__device__ __forceinline__ void cp_async16(uint4 *to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}

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
// a running sum: what each addition loses is added up apart (a few dozen terms lose less than 2^-46 of the sum)
__device__ __forceinline__ void add(Sum &a, float b) {
    const Sum s = two_sum(a.h, b);
    a.h = s.h;
    a.l = __fadd_rn(a.l, s.l);
}
__device__ __forceinline__ void add(Sum &a, Sum b) {
    const Sum s = two_sum(a.h, b.h);
    a.h = s.h;
    a.l = __fadd_rn(a.l, __fadd_rn(s.l, b.l));
}
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
__device__ __forceinline__ Sum warp_sum(Sum a) {
#pragma unroll
    for (int o = 16; o; o >>= 1) a = a + shfl_xor(a, o);
    return a;
}
// inclusive sums over the lanes
__device__ __forceinline__ Sum warp_scan(Sum a) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sum up = {__shfl_up_sync(0xffffffffu, a.h, o), __shfl_up_sync(0xffffffffu, a.l, o)};
        if ((threadIdx.x & 31) >= o) a = up + a;
    }
    return a;
}

// max(p - l q, 0) as two floats
__device__ __forceinline__ Sum left(float p, float q, Sum l) {
    const float h = __fmul_rn(l.h, q), e = __fmaf_rn(l.l, q, __fmaf_rn(l.h, q, -h));
    const Sum d = two_sum(p, -h);
    const Sum r = fast_two_sum(d.h, __fsub_rn(d.l, e));
    return r.h > 0.0f ? r : Sum{0.0f, 0.0f};
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

struct Plan {          // what the first block tells the others
    int action;        // draw from segment `segment`, go to `node` with `state`, or sweep again with l
    int node, state, segment, tried;
    Sum l, before, goal;   // the sum before the segment, and what the draw looks for
};
enum { DRAW = 0, NODE = 1, SWEEP = 2 };

struct Shared {
    Plan plan;
    Sum seg[MAX_CLUSTER * WARPS], seg_q[MAX_CLUSTER * WARPS];   // (first block) the sums of all segments
    Sum row[WARPS];                                             // (the draw) of the rows of one segment
};

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

// bits i .. i + 7 of a row of live bits
__device__ __forceinline__ uint32_t bits_at(const uint32_t *live, int words, int i) {
    if (i < 0) return __ldg(live) << -i;                // -8 < i
    const int w = i >> 5;
    const uint32_t lo = __ldg(live + w);
    if (!(i & 7)) return lo >> (i & 31);
    return __funnelshift_r(lo, w + 1 < words ? __ldg(live + w + 1) : 0u, i & 31);
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
    // vector c of the rows to the thread's place of the ring: an asynchronous copy where it is aligned
    __device__ __forceinline__ void fetch(uint4 *to, int c) const {
        const int i = c * N - lead;
        const bool inside = i >= 0 && i <= V() - N;
        if (inside) cp_async16(to, p.p + i);             // (p's vectors are aligned by their count)
        else *to = p.load(i);
        if (DRAFT) {
            if (inside && !((uintptr_t)(q.p + i) & 15)) cp_async16(to + NT, q.p + i);
            else to[NT] = q.load(i);
        }
    }
    __device__ __forceinline__ int V() const { return p.V; }
    // The sums of vectors c0 + lane, c0 + lane + 32, ... below c1; FRESH: l = 0, and the draft's sum too.  The vectors
    // come through a ring in shared memory, which keeps more of them under way than registers would; a thread
    // reads what it has copied itself.
    template <bool FRESH> __device__ __forceinline__ void sweep(uint4 *ring, int c0, int c1, Sum &w, Sum &wq) const {
        ring += threadIdx.x;
        int put = c0 + (threadIdx.x & 31);
#pragma unroll
        for (int k = 0; k < RING<DRAFT>; ++k, put += 32) {
            if (put < c1) fetch(ring + k * PER<DRAFT>, put);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        int k = 0;
        for (int c = c0 + (threadIdx.x & 31); c < c1; c += 32, put += 32) {
            asm volatile("cp.async.wait_group %0;" ::"n"(RING<DRAFT> - 1) : "memory");
            uint4 *at = ring + k * PER<DRAFT>;
            const uint4 x = *at, y = DRAFT ? at[NT] : x;
            const uint32_t b = live ? bits(c) : 0xffffffffu;
            float f[N], g[N];
            fa_unpack(x, f, T());
            if (DRAFT) fa_unpack(y, g, T());
            // all of them nonnegative and finite, and allowed: the common case
            uint32_t most = 0;
#pragma unroll
            for (int e = 0; e < N; ++e) most = max(most, max(__float_as_uint(f[e]), DRAFT ? __float_as_uint(g[e]) : 0u));
            if (most >= 0x7f800000u || (b & ((1u << N) - 1)) != (1u << N) - 1) {
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const bool in = b >> e & 1;
                    f[e] = in ? weight(f[e]) : 0.0f;
                    if (DRAFT) g[e] = in ? weight(g[e]) : 0.0f;
                }
            }
#pragma unroll
            for (int e = 0; e < N; ++e) {
                if (DRAFT && !FRESH) {
                    add(w, left(f[e], g[e], lam));
                } else {
                    add(w, f[e]);
                    if (DRAFT) add(wq, g[e]);
                }
            }
            if (put < c1) fetch(at, put);
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (++k == RING<DRAFT>) k = 0;
        }
    }
};

template <class T, bool DRAFT>
__global__ void __launch_bounds__(NT, 2) k_verify(VerifyArgs a) {
    constexpr int N = fa_vec<T>::N;
    __shared__ Shared sh;
    extern __shared__ uint4 ring[];
    int *dyn = reinterpret_cast<int *>(ring + RING<DRAFT> * PER<DRAFT>);
    int *parent = dyn, *tok = dyn + a.T, *path = dyn + 2 * a.T, *after = dyn + 3 * a.T, *tried = dyn + 4 * a.T;
    float *us = (float *)(dyn + 5 * a.T), *px = us + a.T, *qx = px + a.T;
    const cg::cluster_group cluster = cg::this_cluster();
    const int C = cluster.num_blocks(), rank = cluster.block_rank(), b = blockIdx.x / C;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Shared *first = cluster.map_shared_rank(&sh, 0);
    const int use = a.count ? min(max(a.count[b], 0), a.T) : a.T;
    if (rank == 0)
        for (int j = tid; j < a.T; j += NT) {
            parent[j] = a.parents[(int64_t)b * a.T + j];
            tok[j] = a.tokens[(int64_t)b * a.T + j];
            us[j] = a.u[(int64_t)b * a.T + j];
            path[j] = 0;
        }
    // kept by the first block's first lane
    int j = 1, kept = use > 0 ? 1 : 0, n_tried = 0;
    Sum l = {0.0f, 0.0f}, old_l = l;
    bool again = false;                                  // this sweep only restores the sums of old_l
    bool probing = false;                                // this sweep is a rejection's
    Sum total_q = {0.0f, 0.0f};
    int node = 0, state = a.S ? a.states[b] : 0;
    bool fresh = true;
    Node<T, DRAFT> at;
    at.words = a.words;
    __syncthreads();
    while (true) {
        // (nothing that a block reads for itself decides how often the cluster meets)
        const bool any = use > 0 && (!a.S || (unsigned)state < (unsigned)a.S);
        if (fresh) {
            at.p = {(const T *)a.target + b * a.tb + node * a.tr, a.V};
            at.q = {DRAFT ? (const T *)a.draft + b * a.db + node * a.dr : nullptr, a.V};
            at.live = a.S && any ? a.live + (int64_t)state * a.words : nullptr;
            at.lead = (int)(((uintptr_t)at.p.p / sizeof(T)) % N);
            at.chunks = (int)(((int64_t)a.V + at.lead + N - 1) / N);
            at.per = (at.chunks + C * NT - 1) / (C * NT) * 32;
            at.lam = {0.0f, 0.0f};
            if (rank == 0) {
                // what the tests of this node's children need
                for (int i = node + 1 + tid; i < use; i += NT) {
                    if (parent[i] != node) continue;
                    const int x = tok[i];
                    px[i] = qx[i] = 0.0f;
                    after[i] = -1;
                    if ((unsigned)x >= (unsigned)a.V || !any) continue;
                    const int to = a.S ? a.next[(int64_t)state * a.V + x] : 0;
                    after[i] = to;
                    if (to < 0) continue;
                    px[i] = weight(fa_to_f32(at.p.p[x]));
                    if (DRAFT) qx[i] = weight(fa_to_f32(at.q.p[x]));
                }
            }
        }
        // ---- this warp's segment
        const int mine = rank * WARPS + warp, s0 = mine * at.per, s1 = min(s0 + at.per, at.chunks);
        Sum w = {0.0f, 0.0f}, wq = {0.0f, 0.0f};
        if (any) {
            if (fresh || !DRAFT) at.template sweep<true>(ring, s0, s1, w, wq);
            else at.template sweep<false>(ring, s0, s1, w, wq);
        }
        w = warp_sum(fast_two_sum(w.h, w.l));
        if (DRAFT && fresh) wq = warp_sum(fast_two_sum(wq.h, wq.l));
        if (lane == 0) {
            first->seg[mine] = w;
            if (DRAFT && fresh) first->seg_q[mine] = wq;
        }
        cluster.sync();
        if (rank == 0 && warp == 0) {
            const int each = (C * WARPS + 31) / 32;       // segments of a lane
            Sum total = {0.0f, 0.0f}, t = {0.0f, 0.0f};
            for (int i = lane * each; i < min((lane + 1) * each, C * WARPS); ++i) {
                total = total + sh.seg[i];
                if (DRAFT && fresh) t = t + sh.seg_q[i];
            }
            total = warp_sum(total);
            if (fresh) {
                n_tried = 0;
                l = {0.0f, 0.0f};
                if (DRAFT) total_q = warp_sum(t);
            }
            Plan plan = {};
            const bool some = total.h > 0.0f && total.h < INFINITY;
            if (lane == 0) {
                if (probing && !again && !(total.h > 0.0f)) {
                    // nothing would be left: the distribution stays as it was
                    l = old_l;
                    plan.action = SWEEP;
                    plan.l = l;
                    again = true;
                } else {
                    again = probing = false;
                    if (!some) j = use;                              // nothing can be accepted
                    const bool drafts = DRAFT && total_q.h > 0.0f;   // a row without weight: q(x) = 0
                    Sum ratio = {0.0f, 0.0f};
                    if (drafts && j < use) ratio = total / total_q;
                    for (; j < use; ++j) {
                        if (parent[j] != node || (unsigned)tok[j] >= (unsigned)a.V) continue;
                        const float u = us[j], x = px[j];
                        bool take, known = false;
                        if (DRAFT) {
                            take = ratio * qx[j] * u < left(x, qx[j], l);
                        } else {
                            for (int i = 0; i < n_tried; ++i) known |= tried[i] == tok[j];
                            take = !known && total * u < Sum{x, 0.0f};
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
                        if (known || x == 0.0f) continue;
                        const Sum rest = total + Sum{-x, 0.0f};
                        if (!(rest.h > 0.0f)) continue;
                        total = rest;
                        Sum &from = sh.seg[at.segment(tok[j])];
                        from = from + Sum{-x, 0.0f};
                        tried[n_tried++] = tok[j];
                    }
                    plan.goal = total * us[0];
                }
            }
            plan.action = __shfl_sync(0xffffffffu, plan.action, 0);
            if (plan.action == DRAW) {
                // the segment that holds the draw
                const Sum goal = {__shfl_sync(0xffffffffu, plan.goal.h, 0), __shfl_sync(0xffffffffu, plan.goal.l, 0)};
                const int i0 = lane * each, i1 = min(i0 + each, C * WARPS);
                Sum here = {0.0f, 0.0f};
                bool weighs = false;
                for (int i = i0; i < i1; ++i) {
                    here = here + sh.seg[i];
                    weighs |= sh.seg[i].h > 0.0f;
                }
                const Sum upto = warp_scan(here);
                const Sum start = {__shfl_up_sync(0xffffffffu, upto.h, 1), __shfl_up_sync(0xffffffffu, upto.l, 1)};
                const uint32_t past = __ballot_sync(0xffffffffu, weighs && goal < upto), all = __ballot_sync(0xffffffffu, weighs);
                const int who = past ? __ffs(past) - 1 : all ? 31 - __clz(all) : 0;
                plan.segment = -1;
                if (lane == who && all && some) {
                    Sum before = lane ? start : Sum{0.0f, 0.0f};
                    for (int i = i0; i < i1; ++i) {
                        if (!(sh.seg[i].h > 0.0f)) continue;
                        const Sum next = before + sh.seg[i];
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
            if (lane < C) cluster.map_shared_rank(&sh, lane)->plan = plan;
        }
        cluster.sync();
        const int action = sh.plan.action;
        fresh = action == NODE;
        if (action == NODE) {
            node = sh.plan.node;
            state = sh.plan.state;
            continue;
        }
        if (action == SWEEP) {
            at.lam = sh.plan.l;
            continue;
        }
        break;
    }
    // ---- the draw: the block that has the segment takes it row by row of 32 vectors, a warp a row
    const int segment = sh.plan.segment;
    if (segment < 0) {
        if (rank == 0 && tid == 0) {
            a.token[b] = -1;
            if (a.state) a.state[b] = -1;
        }
    } else if (rank == segment / WARPS) {
        const int n = DRAFT ? 0 : sh.plan.tried, c0 = segment * at.per, c1 = min(c0 + at.per, at.chunks);
        const Sum goal = sh.plan.goal;
        if (!DRAFT && rank != 0) {
            const int *theirs = cluster.map_shared_rank(tried, 0);
            for (int i = tid; i < n; i += NT) tried[i] = theirs[i];
            __syncthreads();
        }
        Sum before = sh.plan.before;
        int last = -1;                                    // the last element with a weight so far
        for (int r0 = c0; r0 < c1; r0 += NT) {
            const int c = r0 + tid, i = c * N - at.lead;
            float f[N], g[N];
            uint32_t bits = 0;
            uint4 x = make_uint4(0, 0, 0, 0), y = x;
            if (c < c1) {
                x = at.p.load(i);
                if (DRAFT) y = at.q.load(i);
                bits = at.bits(c);
            }
            fa_unpack(x, f, T());
            if (DRAFT) fa_unpack(y, g, T());
            Sum sum = {0.0f, 0.0f};
            int best = -1;
            uint32_t in = 0;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                bool out = !(bits >> e & 1);
                for (int k = 0; k < n; ++k) out |= tried[k] == i + e;
                const float pe = out ? 0.0f : weight(f[e]), qe = DRAFT ? weight(g[e]) : 0.0f;
                const Sum v = DRAFT ? left(pe, qe, at.lam) : Sum{pe, 0.0f};
                if (v.h > 0.0f) { best = i + e; in |= 1u << e; }
                add(sum, v);
            }
            const Sum upto = warp_scan(fast_two_sum(sum.h, sum.l));
            if (lane == 31) sh.row[warp] = upto;
            __syncthreads();
            // the rows' sums in the lanes; the warp whose row holds the draw
            const Sum mine = lane < WARPS ? sh.row[lane] : Sum{0.0f, 0.0f}, rows = warp_scan(lane ? mine : before + mine);
            const uint32_t holds = __ballot_sync(0xffffffffu, mine.h > 0.0f && goal < rows);
            const int who = holds ? __ffs(holds) - 1 : -1, prior = max(who - 1, 0);
            Sum start = {__shfl_sync(0xffffffffu, rows.h, prior), __shfl_sync(0xffffffffu, rows.l, prior)};
            if (who <= 0) start = before;
            const Sum end = {__shfl_sync(0xffffffffu, rows.h, 31), __shfl_sync(0xffffffffu, rows.l, 31)};
            if (warp == who) {
                const Sum lanes = {__shfl_up_sync(0xffffffffu, upto.h, 1), __shfl_up_sync(0xffffffffu, upto.l, 1)};
                const uint32_t past = __ballot_sync(0xffffffffu, in && goal < start + upto), some = __ballot_sync(0xffffffffu, in != 0);
                const int pick = past ? __ffs(past) - 1 : 31 - __clz(some);
                if (lane == pick) {
                    Sum run = lane ? start + lanes : start;   // of the lanes before, then through the elements
                    int found = best;
                    bool done = false;
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        if (!(in >> e & 1) || done) continue;
                        const float pe = weight(f[e]), qe = DRAFT ? weight(g[e]) : 0.0f;
                        const Sum v = DRAFT ? left(pe, qe, at.lam) : Sum{pe, 0.0f};
                        run = run + fast_two_sum(v.h, v.l);
                        if (goal < run) { found = i + e; done = true; }
                    }
                    a.token[b] = found;
                    if (a.state) a.state[b] = a.next[(int64_t)state * a.V + found];
                }
            }
            if (who >= 0) { last = -1; break; }
            best = __reduce_max_sync(0xffffffffu, best);
            __syncthreads();                              // the rows' sums have been read
            if (lane == 0) sh.row[warp].h = __int_as_float(best);
            __syncthreads();
            for (int k = 0; k < WARPS; ++k) last = max(last, __float_as_int(sh.row[k].h));
            __syncthreads();
            before = end;
        }
        if (last >= 0 && tid == 0) {                      // rounding hid the draw: the last element with a weight
            a.token[b] = last;
            if (a.state) a.state[b] = a.next[(int64_t)state * a.V + last];
        }
    }
    if (rank == 0) {
        __syncthreads();                                  // the rows' sums have been read
        if (tid == 0) { sh.row[0].h = __int_as_float(kept); a.kept[b] = kept; }
        __syncthreads();
        const int n = __float_as_int(sh.row[0].h);
        for (int i = tid; i < a.T; i += NT) a.path[(int64_t)b * a.T + i] = i < n ? path[i] : -1;
    }
    cluster.sync();                                       // no block leaves while another reads its list
}

template <class T, bool DRAFT> void launch(const VerifyArgs &a, int cluster, cudaStream_t s) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)a.B * cluster);
    c.blockDim = dim3(NT);
    c.dynamicSmemBytes = sizeof(uint4) * RING<DRAFT> * PER<DRAFT> + (size_t)a.T * 8 * sizeof(int);
    c.stream = s;
    c.attrs = at;
    c.numAttrs = 1;
    if (cudaFuncSetAttribute(k_verify<T, DRAFT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)c.dynamicSmemBytes) == cudaSuccess)
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
    const int cluster = V > 4096 ? MAX_CLUSTER : 1;
    auto go = [&](auto tag) {
        using T_ = decltype(tag);
        if (draft) launch<T_, true>(a, cluster, (cudaStream_t)stream);
        else launch<T_, false>(a, cluster, (cudaStream_t)stream);
    };
    if (dtype == FA_DTYPE_F32) go(0.0f);
    else if (dtype == FA_DTYPE_F16) go(__half());
    else go(__nv_bfloat16());
    return fa_launch_check("verify");
}
