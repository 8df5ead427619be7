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
// A draw compares u with a sum over the vocabulary, so sums are kept as unevaluated sums of two floats (Knuth's and
// Dekker's exact additions, 46 bits or more): fp64 runs at two lanes a clock and SM here.
//
// A cluster of blocks takes a sequence: each block a slice of the vocabulary, from node to node.  The first
// block decides and tells the others, so that they never part ways whatever the inputs hold.
#include <cooperative_groups.h>

#include "fa_lm.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int NT = 512, WARPS = NT / 32, MAX_CLUSTER = 8;

struct Sum { float h, l; };   // h + l, |l| at most half a unit of h's last place

__device__ __forceinline__ Sum two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Sum fast_two_sum(float a, float b) {   // |a| >= |b|
    const float s = __fadd_rn(a, b);
    return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Sum operator+(Sum a, Sum b) {
    Sum s = two_sum(a.h, b.h);
    return fast_two_sum(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Sum operator+(Sum a, float b) {
    Sum s = two_sum(a.h, b);
    return fast_two_sum(s.h, __fadd_rn(s.l, a.l));
}
__device__ __forceinline__ double value(Sum a) { return (double)a.h + (double)a.l; }
__device__ __forceinline__ Sum split(double x) {
    const float h = (float)x;
    return {h, (float)(x - (double)h)};
}
__device__ __forceinline__ Sum warp_sum(Sum a) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
        a = a + Sum{__shfl_xor_sync(0xffffffffu, a.h, o), __shfl_xor_sync(0xffffffffu, a.l, o)};
    return a;
}

// max(p - l q, 0)
__device__ __forceinline__ Sum left(float p, float q, Sum l) {
    const float h = __fmul_rn(l.h, q), e = __fmaf_rn(l.l, q, __fmaf_rn(l.h, q, -h));
    const Sum d = two_sum(p, -h), r = fast_two_sum(d.h, __fsub_rn(d.l, e));
    return r.h > 0.0f ? r : Sum{0.0f, 0.0f};
}

__device__ __forceinline__ float weight(float x) { return x > 0.0f && x < INFINITY ? x : 0.0f; }

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
    int action;        // draw from the segment sums, go to `node` with `state`, or sweep again with l
    int node, state, owner;
    Sum l;
    double before;     // the sum before the owner's slice, and what the draw looks for
    double goal;
};
enum { DRAW = 0, NODE = 1, SWEEP = 2 };

struct Shared {
    Plan plan;
    Sum seg[WARPS], seg_q[WARPS];                       // this block's segments
    Sum part[MAX_CLUSTER], part_q[MAX_CLUSTER];         // (first block) every block's slice
    int picked;
};

// A row of the vocabulary in vectors of 16 bytes, counted from the aligned address at or before its start.
template <class T> struct Row {
    static constexpr int N = fa_vec<T>::N;
    const T *p;
    int V;
    // elements i .. i + N - 1, zero outside the row
    __device__ __forceinline__ void load(int i, float (&f)[N]) const {
        if (i >= 0 && i <= V - N && !((uintptr_t)(p + i) & 15)) {
            fa_unpack(__ldg(reinterpret_cast<const uint4 *>(p + i)), f, T());
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) f[e] = i + e >= 0 && i + e < V ? fa_to_f32(p[i + e]) : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] = weight(f[e]);
    }
};

// bits i .. i + 7 of a row of live bits
__device__ __forceinline__ uint32_t bits_at(const uint32_t *live, int words, int i) {
    if (i < 0) return __ldg(live) << -i;                // -8 < i
    const int w = i >> 5;
    const uint32_t lo = __ldg(live + w), hi = w + 1 < words ? __ldg(live + w + 1) : 0u;
    return __funnelshift_r(lo, hi, i & 31);
}

template <class T, bool DRAFT>
__global__ void __launch_bounds__(NT) k_verify(VerifyArgs a) {
    constexpr int N = fa_vec<T>::N;
    __shared__ Shared sh;
    extern __shared__ int dyn[];
    int *parent = dyn, *tok = dyn + a.T, *path = dyn + 2 * a.T, *after = dyn + 3 * a.T, *tried = dyn + 4 * a.T;
    float *us = (float *)(dyn + 5 * a.T), *px = us + a.T, *qx = px + a.T;
    const cg::cluster_group cluster = cg::this_cluster();
    const int C = cluster.num_blocks(), rank = cluster.block_rank(), b = blockIdx.x / C;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Shared *first = cluster.map_shared_rank(&sh, 0);
    const int use = a.count ? min(max(a.count[b], 0), a.T) : a.T;
    for (int j = tid; j < a.T; j += NT) {
        parent[j] = a.parents[(int64_t)b * a.T + j];
        tok[j] = a.tokens[(int64_t)b * a.T + j];
        us[j] = a.u[(int64_t)b * a.T + j];
    }
    // kept by the first block's first thread
    int j = 1, kept = 0, n_tried = 0;
    double l = 0.0, old_l = 0.0;
    bool again = false;                                  // this sweep only restores the sums of old_l
    bool probing = false;                                // this sweep is a rejection's
    Sum total = {0.0f, 0.0f}, total_q = {0.0f, 0.0f};
    int node = 0, state = a.S ? a.states[b] : 0;
    Sum lam = {0.0f, 0.0f};
    bool fresh = true;
    const int known = a.S;                               // states
    if (tid == 0 && use > 0) path[0] = 0;
    kept = use > 0 ? 1 : 0;
    __syncthreads();
    while (true) {
        // (nothing that a block reads for itself decides how often the cluster meets)
        const bool any = use > 0 && (!known || (unsigned)state < (unsigned)known);
        const T *p = (const T *)a.target + b * a.tb + node * a.tr, *q = DRAFT ? (const T *)a.draft + b * a.db + node * a.dr : nullptr;
        const int lead = (int)(((uintptr_t)p / sizeof(T)) % N);
        const int chunks = (int)(((int64_t)a.V + lead + N - 1) / N);
        const int per = (chunks + C * NT - 1) / (C * NT) * 32;               // chunks of a segment
        const uint32_t *live = known && any ? a.live + (int64_t)state * a.words : nullptr;
        if (rank == 0 && fresh) {
            // what the tests of this node's children need
            for (int i = tid; i < use; i += NT) {
                if (parent[i] != node || i <= node) continue;
                const int x = tok[i];
                px[i] = qx[i] = 0.0f;
                after[i] = -1;
                if ((unsigned)x >= (unsigned)a.V || !any) continue;
                const int to = known ? a.next[(int64_t)state * a.V + x] : 0;
                after[i] = to;
                if (to < 0) continue;
                px[i] = weight(fa_to_f32(p[x]));
                if (DRAFT) qx[i] = weight(fa_to_f32(q[x]));
            }
        }
        // ---- this warp's segment
        const int s0 = (rank * WARPS + warp) * per, s1 = min(s0 + per, chunks);
        const Row<T> rp{p, a.V}, rq{q, a.V};
        Sum w = {0.0f, 0.0f}, wq = {0.0f, 0.0f};
        constexpr int U = 4;
        if (any)
            for (int c = s0 + lane; c < s1; c += 32 * U) {
                float f[U][N], g[U][N];
                uint32_t bits[U];
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int i = (c + 32 * k) * N - lead;
                    bits[k] = 0;
                    if (c + 32 * k >= s1) continue;
                    bits[k] = live ? bits_at(live, a.words, i) : 0xffffffffu;
                    rp.load(i, f[k]);
                    if (DRAFT) rq.load(i, g[k]);
                }
#pragma unroll
                for (int k = 0; k < U; ++k)
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        if (!(bits[k] >> e & 1)) continue;
                        if (DRAFT) {
                            wq = wq + g[k][e];
                            w = w + left(f[k][e], g[k][e], lam);
                        } else {
                            w = w + f[k][e];
                        }
                    }
            }
        w = warp_sum(w);
        if (DRAFT) wq = warp_sum(wq);
        if (lane == 0) { sh.seg[warp] = w; if (DRAFT) sh.seg_q[warp] = wq; }
        __syncthreads();
        if (tid == 0) {
            Sum s = {0.0f, 0.0f}, t = {0.0f, 0.0f};
            for (int i = 0; i < WARPS; ++i) { s = s + sh.seg[i]; if (DRAFT) t = t + sh.seg_q[i]; }
            first->part[rank] = s;
            first->part_q[rank] = t;
        }
        cluster.sync();
        if (rank == 0 && tid == 0) {
            Sum s = {0.0f, 0.0f}, t = {0.0f, 0.0f};
            for (int i = 0; i < C; ++i) { s = s + sh.part[i]; t = t + sh.part_q[i]; }
            if (fresh) { n_tried = 0; l = 0.0; total_q = t; }
            Plan plan;
            plan.action = DRAW;
            bool restore = false;
            if (probing && !again && !(value(s) > 0.0)) { restore = true; l = old_l; }
            total = s;
            if (restore) {
                plan.action = SWEEP;
                plan.l = split(l);
                again = true;
            } else {
                again = probing = false;
                double S = value(total);
                const double Q = DRAFT ? value(total_q) : 1.0;
                if (!(S > 0.0 && S < INFINITY)) j = use;         // nothing can be accepted
                for (; j < use; ++j) {
                    if (parent[j] != node || (unsigned)tok[j] >= (unsigned)a.V) continue;
                    const double u = us[j], x = px[j];
                    bool take, known_token = false;
                    if (DRAFT) {
                        const double y = qx[j], r = x - l * y;
                        take = u * S * y < (r > 0.0 ? r : 0.0) * (Q > 0.0 ? Q : 1.0);   // a row without weight: q(x) = 0
                    } else {
                        for (int i = 0; i < n_tried; ++i) known_token |= tried[i] == tok[j];
                        take = !known_token && u * S < x;
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
                        if (!(Q > 0.0)) continue;
                        old_l = l;
                        l += S / Q;
                        plan.action = SWEEP;
                        plan.l = split(l);
                        probing = true;
                        ++j;
                        break;
                    }
                    if (known_token || x == 0.0) continue;
                    const Sum rest = total + (float)-x;
                    if (!(value(rest) > 0.0)) continue;
                    total = rest;
                    S = value(total);
                    tried[n_tried++] = tok[j];
                }
                if (plan.action == DRAW) {
                    // the slice that holds the draw: without what was tried
                    plan.goal = (double)us[0] * S;
                    plan.owner = -1;
                    plan.before = 0.0;
                    int last = -1;
                    double last_before = 0.0;
                    if (S > 0.0 && S < INFINITY)
                        for (int c = 0; c < C; ++c) {
                            Sum here = sh.part[c];
                            if (!DRAFT)
                                for (int i = 0; i < n_tried; ++i)
                                    if ((tried[i] + lead) / N / per / WARPS == c) here = here + -weight(fa_to_f32(p[tried[i]]));
                            const double v = value(here);
                            if (!(v > 0.0)) continue;
                            last = c;
                            last_before = plan.before;
                            if (plan.goal < plan.before + v) { plan.owner = c; break; }
                            plan.before += v;
                        }
                    if (plan.owner < 0) { plan.owner = last; plan.before = last_before; }
                    plan.node = n_tried;
                }
            }
            for (int c = 0; c < C; ++c) cluster.map_shared_rank(&sh, c)->plan = plan;
        }
        cluster.sync();
        const Plan plan = sh.plan;
        fresh = plan.action == NODE;
        if (plan.action == NODE) {
            node = plan.node;
            state = plan.state;
            lam = {0.0f, 0.0f};
            continue;
        }
        if (plan.action == SWEEP) {
            lam = plan.l;
            continue;
        }
        // ---- the draw
        if (plan.owner < 0) {
            if (rank == 0 && tid == 0) {
                a.token[b] = -1;
                if (a.state) a.state[b] = -1;
            }
        } else {
            const int *list = tried;
            if (!DRAFT && plan.owner != 0 && rank == plan.owner) {
                const int *theirs = cluster.map_shared_rank(tried, 0);
                for (int i = tid; i < plan.node; i += NT) tried[i] = theirs[i];
                __syncthreads();
            }
            if (rank == plan.owner && warp == 0) {
                const int n = DRAFT ? 0 : plan.node;
                int pick = -1, last = -1;
                double before = plan.before, last_before = 0.0;
                if (lane == 0) {
                    for (int k = 0; k < WARPS; ++k) {
                        Sum here = sh.seg[k];
                        for (int i = 0; i < n; ++i)
                            if ((list[i] + lead) / N / per == rank * WARPS + k) here = here + -weight(fa_to_f32(p[list[i]]));
                        const double v = value(here);
                        if (!(v > 0.0)) continue;
                        last = k;
                        last_before = before;
                        if (plan.goal < before + v) { pick = k; break; }
                        before += v;
                    }
                    if (pick < 0) { pick = last; before = last_before; }
                }
                pick = __shfl_sync(0xffffffffu, pick, 0);
                before = __shfl_sync(0xffffffffu, before, 0);
                int found = -1, best = -1;                // best: the last element with a weight
                if (pick >= 0) {
                    const int c0 = (rank * WARPS + pick) * per, c1 = min(c0 + per, chunks);
                    for (int c = c0; c < c1 && found < 0; c += 32) {
                        const int i = (c + lane) * N - lead;
                        float f[N], g[N];
                        Sum x[N], sum = {0.0f, 0.0f};
                        const uint32_t bits = c + lane < c1 ? live ? bits_at(live, a.words, i) : 0xffffffffu : 0u;
                        if (c + lane < c1) {
                            rp.load(i, f);
                            if (DRAFT) rq.load(i, g);
                        }
#pragma unroll
                        for (int e = 0; e < N; ++e) {
                            x[e] = {0.0f, 0.0f};
                            if (!(bits >> e & 1)) continue;
                            bool out = false;
                            for (int k = 0; k < n; ++k) out |= list[k] == i + e;
                            if (out) continue;
                            if (DRAFT) x[e] = left(f[e], g[e], lam);
                            else x[e] = {f[e], 0.0f};
                            if (x[e].h > 0.0f) best = i + e;
                            sum = sum + x[e];
                        }
                        Sum upto = sum;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const Sum up = {__shfl_up_sync(0xffffffffu, upto.h, o), __shfl_up_sync(0xffffffffu, upto.l, o)};
                            if (lane >= o) upto = up + upto;
                        }
                        const double end = before + value(upto);
                        const uint32_t past = __ballot_sync(0xffffffffu, end > plan.goal && sum.h > 0.0f);
                        if (past) {
                            const int who = __ffs(past) - 1;
                            // the lanes before
                            const Sum start = {__shfl_up_sync(0xffffffffu, upto.h, 1), __shfl_up_sync(0xffffffffu, upto.l, 1)};
                            if (lane == who) {
                                Sum at = lane ? start : Sum{0.0f, 0.0f};
                                int mine = -1, some = -1;
#pragma unroll
                                for (int e = 0; e < N; ++e) {
                                    at = at + x[e];
                                    if (!(x[e].h > 0.0f)) continue;
                                    some = i + e;
                                    if (mine < 0 && before + value(at) > plan.goal) mine = i + e;
                                }
                                found = mine >= 0 ? mine : some;
                            }
                            found = __shfl_sync(0xffffffffu, found, who);
                        }
                        before = __shfl_sync(0xffffffffu, end, 31);
                    }
                    if (found < 0) found = __reduce_max_sync(0xffffffffu, best);
                }
                if (lane == 0) {
                    a.token[b] = found;
                    if (a.state) a.state[b] = found >= 0 ? a.next[(int64_t)state * a.V + found] : -1;
                }
            }
        }
        break;
    }
    __syncthreads();
    if (rank == 0) {
        if (tid == 0) { sh.picked = kept; a.kept[b] = kept; }
        __syncthreads();
        for (int i = tid; i < a.T; i += NT) a.path[(int64_t)b * a.T + i] = i < sh.picked ? path[i] : -1;
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
    c.dynamicSmemBytes = (size_t)a.T * 8 * sizeof(int);
    c.stream = s;
    c.attrs = at;
    c.numAttrs = 1;
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
