// Attention of few rows (up to 16 for a key/value head: single tokens with their group of query
// heads, short drafts) over a paged cache.
//
// The mathematics is that of fa_tree_attention.cu.  The bound is memory: every cached key and value
// is read once and used for at most 16 rows.  Nothing is shared between warps: a warp owns an
// equal run of the list of all tiles of all units, copies its tiles (4 KB of keys, 4 KB of
// values) asynchronously into three buffers of its own, two of them under way, and keeps its rows'
// queries, statistics and results in registers, so no barrier joins warps and eight warps an SM have
// 128 KB of loads in flight.  The products are 16 x 8 x 16 tensor instructions on fragments made in
// registers; a contraction's order is free, so every lane takes 16 consecutive bytes of a key or
// value and the other operand follows that order: codes become fp16 there (exactly) without a pass
// through shared memory.  Tiles are swizzled so that the reads of both kinds are free of bank
// conflicts.  A unit that is cut leaves partial results, joined by the same kernel as the larger one's.
//
// Measured (head_dim 128, 8 key/value heads): 32 sequences of 8192 slots, 8-bit cache, 4 rows 101 us
// (545 MB, 5.4 TB/s), 16 rows 121 us (the instructions of two halves of the left operand begin to count);
// 16-bit cache 176 us (1.07 GB, 6.1 TB/s).  32 ragged sequences of up to 8192 slots, 8-bit:
// 61 us (285 MB; 56 the kernel, 5 the join).  4 sequences of 509 slots: 12 us replayed in a graph, 14 called one by
// one: two launches' start and end.  Up to eight rows leave the operand's second half out (R16 = false: 104 us at 8
// rows).
#include "fa_attention.cuh"

using namespace fa_attention;

namespace {

constexpr int NW = FA_FEW_WARPS, NB = 3, BUF = 4096;   // warps, buffers of a warp, bytes of a tile's keys

template <int DP, bool E4M3> struct Few {
    static constexpr int ROWB = DP * (E4M3 ? 1 : 2), CH = BUF / ROWB, C16 = ROWB / 16;   // bytes of a row, slots of a tile, 16-byte chunks of a row
    static constexpr int STAGE = 2 * BUF + (E4M3 ? 2 * CH * 4 : 0);
    static constexpr int SMEM = NW * NB * STAGE;
    // where a row's chunk c lies: keys are read by 8 rows x 4 chunks, values by rows 2t and 2t + 1 (t < 4) x 8 chunks
    static __device__ __forceinline__ int key_chunk(int r, int c) { return C16 >= 8 ? c ^ ((r & 1) << 2) : c; }
    static __device__ __forceinline__ int value_chunk(int r, int c) { return C16 >= 8 ? c ^ (((r >> 1) & 3) << 1) : c ^ ((r >> 1) & 3); }
    // the first of the four query columns that lane quarter t contracts in step s
    static __device__ __forceinline__ int query_col(int s, int t) {
        return E4M3 ? 16 * (t + 4 * (s >> 2)) + 4 * (s & 3) : 8 * (4 * (s >> 1) + t) + 4 * (s & 1);
    }
    // the column of the result's block jj of eight values with n = 0, and the stride of n
    static constexpr int NSTEP = E4M3 && DP == 128 ? 16 : 8;
    static __device__ __forceinline__ int out_col(int n, int jj) { return n * NSTEP + jj * (NSTEP == 16 ? 8 : 64); }
};

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1, __half) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1, __nv_bfloat16) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

// M: the tensor instructions' type; T: q's and out's; R16: more than eight rows
template <int DP, bool E4M3, class T, class M, bool R16>
__global__ void __launch_bounds__(32 * NW, 1) k_attend_few(AttendArgs a) {
    typedef Few<DP, E4M3> F;
    constexpr int CH = F::CH, C16 = F::C16, RPI = 32 / C16, NJ = DP / 8, KS = DP / 16, NBK = CH / 8, RR = R16 ? 2 : 1;
    constexpr int SLOTS = (CH + 31) / 32;                    // slots a lane looks up per tile
    constexpr float OFF = std::is_same<M, __half>::value ? 4.0f : 0.0f;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Work work;
    fa_let_next_start();
    plan(a, work);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3, D = a.c.head_dim;
    const int run = blockIdx.x * NW + warp;
    unsigned char *mine = smem + warp * (NB * F::STAGE);
    const Walk start(a, work, run, gridDim.x * NW);

    // ---- tiles on their way
    Walk ahead = start;
    Segment sa;
    sa.n = 0;
    int ia = 0, issued = 0;
    bool more = ahead.next(a, sa);
    Rows rows_a(a, sa);
    uint32_t page[SLOTS];
    auto look = [&]() {
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            const uint32_t slot = (uint32_t)(sa.t0 + ia) * CH + 32 * i + lane;
            page[i] = (CH >= 32 || lane < CH) && slot < (uint32_t)sa.end ? rows_a.page(slot) : 0xffffffffu;
        }
    };
    if (more) look();
    const int copy_c = lane % C16, copy_r = lane / C16;
    const bool column = copy_c * 16 < D * (E4M3 ? 1 : 2);
    auto issue = [&]() {
        if (more) {
            unsigned char *stage = mine + issued % NB * F::STAGE;
            const uint32_t dst = smem_u32(stage), first = (uint32_t)(sa.t0 + ia) * CH;
            const uint32_t row_bytes = D * (E4M3 ? 1 : 2);
#pragma unroll
            for (int it = 0; it < CH / RPI; ++it) {
                const int r = it * RPI + copy_r;
                const uint32_t p = __shfl_sync(0xffffffffu, page[it * RPI / 32], r & 31);
                const int64_t row = rows_a.row(p, first + r);
                const bool there = row >= 0 && column;
                const int64_t off = there ? row * row_bytes + copy_c * 16 : 0;
                cp_async16(dst + r * F::ROWB + F::key_chunk(r, copy_c) * 16, (const unsigned char *)a.c.k + off, there);
                cp_async16(dst + BUF + r * F::ROWB + F::value_chunk(r, copy_c) * 16, (const unsigned char *)a.c.v + off, there);
            }
            if (E4M3)
#pragma unroll
                for (int i = 0; i < SLOTS; ++i) {
                    const int64_t row = rows_a.row(page[i], first + 32 * i + lane);
                    cp_async4(dst + 2 * BUF + (32 * i + lane) * 4, a.c.k_scale + max(row, (int64_t)0), row >= 0);
                    cp_async4(dst + 2 * BUF + (CH + 32 * i + lane) * 4, a.c.v_scale + max(row, (int64_t)0), row >= 0);
                }
            ++issued;
            if (++ia == sa.n) {
                ia = 0;
                more = ahead.next(a, sa);
                if (more) rows_a = Rows(a, sa);
            }
            if (more) look();
        }
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < NB - 1; ++i) issue();

    Walk walk = start;
    Segment s;
    int done = 0;
    while (walk.next(a, s)) {
        const Rows rows(a, s);
        // ---- the rows' queries, as left operands in the order of the contraction
        int ti[RR];
        bool live[RR], used[RR];
        float c[RR], m[RR], l[RR], bias[RR];
        float ev[RR];                           // whole numbers
        int64_t orow[RR];
        uint32_t qf[KS][2 * RR];
#pragma unroll
        for (int h = 0; h < RR; ++h) {
            const int row = g + 8 * h;
            live[h] = row < s.rows;
            ti[h] = live[h] ? row / a.group : 0;
            const int hq = s.head * a.group + (live[h] ? row - ti[h] * a.group : 0);
            used[h] = live[h] && ti[h] < s.use;
            orow[h] = ((int64_t)s.b * a.T + ti[h]) * a.heads + hq;
            m[h] = -INFINITY;
            l[h] = bias[h] = 0.0f;
            ev[h] = E4M3 ? kLeastScale : 0.0f;
            const T *q = (const T *)a.q + s.b * a.qb + ti[h] * a.qt + hq * a.qh;
            float top = 0.0f;
            uint2 raw[KS];
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const int col = F::query_col(k, t);
                raw[k] = live[h] && col < D ? __ldg(reinterpret_cast<const uint2 *>(q + col)) : make_uint2(0, 0);
            }
            c[h] = a.scale * kLog2e;
            if constexpr (!E4M3) {
#pragma unroll
                for (int k = 0; k < KS; ++k) { qf[k][2 * h] = raw[k].x; qf[k][2 * h + 1] = raw[k].y; }
            } else {
                // scaled by a power of two, the largest element to [2^8, 2^9)
                auto four = [&](uint2 r, float (&f)[4]) {
                    float f8[8];
                    fa_unpack(make_uint4(r.x, r.y, 0, 0), f8, T());
#pragma unroll
                    for (int j = 0; j < 4; ++j) f[j] = f8[j];
                };
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    float f[4];
                    four(raw[k], f);
#pragma unroll
                    for (int j = 0; j < 4; ++j) top = fmaxf(top, fabsf(f[j]));
                }
                top = quad_max(top);
                const int e = top > 0.0f && top < INFINITY ? max(min(fa_exponent(top) - 8, 120), -120) : 0;
                const float pow = pow2(-e);
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    float f[4];
                    four(raw[k], f);
                    qf[k][2 * h] = fa_pack2(f[0] * pow, f[1] * pow, M());
                    qf[k][2 * h + 1] = fa_pack2(f[2] * pow, f[3] * pow, M());
                }
                c[h] *= pow2(e);
            }
        }
        float o[NJ][4];
#pragma unroll
        for (int j = 0; j < NJ; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
        bool odd = false;                       // a drafted value is not finite (the same for the warp)

        for (int tile = 0; tile < s.n; ++tile, ++done) {
            issue();
            cp_wait<NB - 1>();
            __syncwarp();
            unsigned char *kb = mine + done % NB * F::STAGE, *vb = kb + BUF;
            const float *ks = reinterpret_cast<const float *>(kb + 2 * BUF), *vs = ks + CH;
            const int first = (s.t0 + tile) * CH;
            // ---- scores
            float x[NBK][4];
#pragma unroll
            for (int nb = 0; nb < NBK; ++nb) {
                x[nb][0] = x[nb][1] = x[nb][2] = x[nb][3] = 0.0f;
                const int r = nb * 8 + g;
                const unsigned char *kr = kb + r * F::ROWB;
#pragma unroll
                for (int j = 0; j < C16 / 4; ++j) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(kr + F::key_chunk(r, 4 * j + t) * 16);
                    const uint32_t word[4] = {w.x, w.y, w.z, w.w};
                    if constexpr (E4M3) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t (&q)[2 * RR] = qf[4 * j + i];
                            mma(x[nb], q[0], R16 ? q[2 * RR - 2] : 0u, q[1], R16 ? q[2 * RR - 1] : 0u,
                                fa_e4m3x2_to_half2(word[i]), fa_e4m3x2_to_half2(word[i] >> 16), M());
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t (&q)[2 * RR] = qf[2 * j + i];
                            mma(x[nb], q[0], R16 ? q[2 * RR - 2] : 0u, q[1], R16 ? q[2 * RR - 1] : 0u, word[2 * i], word[2 * i + 1], M());
                        }
                    }
                }
            }
            // ---- which slots the rows see
            const bool whole = first + CH <= s.slots;
            uint32_t see[RR][SLOTS];
            bool all = whole;
            {
                uint32_t held[SLOTS];
#pragma unroll
                for (int i = 0; i < SLOTS; ++i) {
                    const uint32_t slot = first + 32 * i + lane;
                    held[i] = __ballot_sync(0xffffffffu, (CH >= 32 || lane < CH) && slot < (uint32_t)s.end && rows.page(slot) < rows.n_pages);
                    all &= held[i] == (CH >= 32 ? 0xffffffffu : (1u << (CH & 31)) - 1);
                }
#pragma unroll
                for (int h = 0; h < RR; ++h)
#pragma unroll
                    for (int i = 0; i < SLOTS; ++i)
                        see[h][i] = all ? 0xffffffffu : used[h] ? held[i] & seen_bits(a, s, ti[h], first + 32 * i) : 0u;
            }
            if (first + CH > s.slots) {
                // drafted values that are not finite are left out of the product (they join the rows that
                // see them at the end), and so are scales
                bool here = false;
                for (int i = lane; i < BUF / 16; i += 32) {
                    const int r = i / C16;
                    if (first + r < s.slots) continue;
                    uint4 *p = reinterpret_cast<uint4 *>(vb) + i;
                    uint4 v = *p;
                    if constexpr (E4M3) {
                        uint32_t w[4] = {v.x, v.y, v.z, v.w};
                        bool bad = false;
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if ((w[j / 4] >> (8 * (j & 3)) & 0x7f) == 0x7f) { w[j / 4] &= ~(0xffu << (8 * (j & 3))); bad = true; }
                        if (bad) *p = make_uint4(w[0], w[1], w[2], w[3]);
                        here |= bad;
                    } else {
                        if (zero_odd<M>(v)) { *p = v; here = true; }
                    }
                }
                if (E4M3)
                    for (int r = lane; r < CH; r += 32)
                        if (first + r >= s.slots && !(fabsf(vs[r]) < INFINITY)) { const_cast<float *>(vs)[r] = 0.0f; here = true; }
                odd |= __any_sync(0xffffffffu, here);
                __syncwarp();
            }
            // ---- weights
            float2 kk[NBK], vv[NBK];
            if (E4M3)
#pragma unroll
                for (int nb = 0; nb < NBK; ++nb) {
                    kk[nb] = *reinterpret_cast<const float2 *>(ks + nb * 8 + 2 * t);
                    vv[nb] = *reinterpret_cast<const float2 *>(vs + nb * 8 + 2 * t);
                }
            uint32_t p[NBK][RR];
            float f[RR];
            bool moved = false;
#pragma unroll
            for (int h = 0; h < RR; ++h) {
                float mx = -INFINITY, vmx = 0.0f;
#pragma unroll
                for (int nb = 0; nb < NBK; ++nb) {
                    float &x0 = x[nb][2 * h], &x1 = x[nb][2 * h + 1];
                    if (E4M3) { x0 = __fmul_rn(x0, kk[nb].x); x1 = __fmul_rn(x1, kk[nb].y); }
                    if (!all) {
                        const uint32_t z = see[h][nb / 4] >> (8 * (nb & 3) + 2 * t);
                        x0 = z & 1 ? x0 : -INFINITY;
                        x1 = z & 2 ? x1 : -INFINITY;
                        if (E4M3) {
                            if (z & 1) vmx = fmaxf(vmx, vv[nb].x);
                            if (z & 2) vmx = fmaxf(vmx, vv[nb].y);
                        }
                    } else if (E4M3) {
                        vmx = fmaxf(vmx, fmaxf(vv[nb].x, vv[nb].y));
                    }
                    mx = fmaxf(mx, fmaxf(x0, x1));
                }
                mx = quad_max(mx);
                if (E4M3) vmx = quad_max(vmx);
                // (as in the larger kernel: products are looked at only where their bound says so)
                const float by_score = (mx - m[h]) * c[h];
                bool move = by_score > (E4M3 ? fminf(kGrow, ev[h] + kProductGrow - lg2(vmx)) : kGrow);
                float e2 = ev[h];
                if (E4M3 && __any_sync(0xffffffffu, move)) {
                    const float m2 = fmaxf(m[h], mx);
                    float most = -INFINITY;
#pragma unroll
                    for (int nb = 0; nb < NBK; ++nb) {
                        most = fmaxf(most, fmaf(x[nb][2 * h] - m2, c[h], lg2(vv[nb].x)));
                        most = fmaxf(most, fmaf(x[nb][2 * h + 1] - m2, c[h], lg2(vv[nb].y)));
                    }
                    most = quad_max(most);
                    const float now = m[h] > -INFINITY ? (m[h] - m2) * c[h] + ev[h] : -INFINITY;
                    move = move && (by_score > kGrow || most > now + kProductGrow);
                    e2 = scale_power(fmaxf(now, most));
                }
                f[h] = 1.0f;
                if (move) {
                    const bool had = m[h] > -INFINITY;
                    const float m0 = m[h], up = e2 - ev[h];
                    m[h] = fmaxf(m[h], mx);
                    ev[h] = e2;
                    const float b2 = m[h] * c[h] + ev[h] - OFF;
                    const float by = fmaxf(fabsf(bias[h]), fabsf(b2)) > kFar ? (m0 - m[h]) * c[h] - up : bias[h] - b2;
                    f[h] = had ? ex2(by) : 0.0f;
                    bias[h] = b2;
                    l[h] *= E4M3 ? (had ? ex2(up + by) : 0.0f) : f[h];
                    moved = true;
                }
                const bool far = fabsf(bias[h]) > kFar;
                const float ref = far ? ev[h] - OFF : bias[h];
                if (__any_sync(0xffffffffu, far))
#pragma unroll
                    for (int nb = 0; nb < NBK; ++nb) {
                        x[nb][2 * h] -= far ? m[h] : 0.0f;
                        x[nb][2 * h + 1] -= far ? m[h] : 0.0f;
                    }
                float sum = 0.0f;
#pragma unroll
                for (int nb = 0; nb < NBK; ++nb) {
                    float y0 = ex2(fmaf(x[nb][2 * h], c[h], -ref)), y1 = ex2(fmaf(x[nb][2 * h + 1], c[h], -ref));
                    sum += y0 + y1;
                    if (E4M3) { y0 *= vv[nb].x; y1 *= vv[nb].y; }
                    p[nb][h] = fa_pack2(y0, y1, M());
                }
                l[h] += sum * pow2(ev[h]);
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    o[j][0] *= f[0];
                    o[j][1] *= f[0];
                    if (R16) { o[j][2] *= f[RR - 1]; o[j][3] *= f[RR - 1]; }
                }
            }
            // ---- values
#pragma unroll
            for (int kg = 0; kg < CH / 16; ++kg) {
                const uint32_t a0 = p[2 * kg][0], a1 = R16 ? p[2 * kg][RR - 1] : 0u, a2 = p[2 * kg + 1][0], a3 = R16 ? p[2 * kg + 1][RR - 1] : 0u;
                const int r0 = 16 * kg + 2 * t;                // rows r0, r0 + 1, r0 + 8, r0 + 9
                if constexpr (E4M3) {
                    constexpr int W = DP / 32;                 // 4-byte words of a lane's codes
                    uint32_t w[4][W];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = r0 + (i & 1) + 8 * (i >> 1);
                        const unsigned char *vr = vb + r * F::ROWB;
                        if constexpr (DP == 128) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(vr + F::value_chunk(r, g) * 16);
                            w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
                        } else {
                            const uint2 v = *reinterpret_cast<const uint2 *>(vr + F::value_chunk(r, g >> 1) * 16 + (g & 1) * 8);
                            w[i][0] = v.x; w[i][1] = v.y;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        const uint32_t b0l = __byte_perm(w[0][i], w[1][i], 0x5140), b0h = __byte_perm(w[0][i], w[1][i], 0x7362);
                        const uint32_t b1l = __byte_perm(w[2][i], w[3][i], 0x5140), b1h = __byte_perm(w[2][i], w[3][i], 0x7362);
                        mma(o[4 * i], a0, a1, a2, a3, fa_e4m3x2_to_half2(b0l), fa_e4m3x2_to_half2(b1l), M());
                        mma(o[4 * i + 1], a0, a1, a2, a3, fa_e4m3x2_to_half2(b0l >> 16), fa_e4m3x2_to_half2(b1l >> 16), M());
                        mma(o[4 * i + 2], a0, a1, a2, a3, fa_e4m3x2_to_half2(b0h), fa_e4m3x2_to_half2(b1h), M());
                        mma(o[4 * i + 3], a0, a1, a2, a3, fa_e4m3x2_to_half2(b0h >> 16), fa_e4m3x2_to_half2(b1h >> 16), M());
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < DP / 64; ++q) {        // chunks g and g + 8
                        uint4 w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = r0 + (i & 1) + 8 * (i >> 1);
                            w[i] = *reinterpret_cast<const uint4 *>(vb + r * F::ROWB + F::value_chunk(r, g + 8 * q) * 16);
                        }
                        const uint32_t w0[4] = {w[0].x, w[0].y, w[0].z, w[0].w}, w1[4] = {w[1].x, w[1].y, w[1].z, w[1].w};
                        const uint32_t w2[4] = {w[2].x, w[2].y, w[2].z, w[2].w}, w3[4] = {w[3].x, w[3].y, w[3].z, w[3].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            mma(o[8 * q + 2 * i], a0, a1, a2, a3, __byte_perm(w0[i], w1[i], 0x5410), __byte_perm(w2[i], w3[i], 0x5410), M());
                            mma(o[8 * q + 2 * i + 1], a0, a1, a2, a3, __byte_perm(w0[i], w1[i], 0x7632), __byte_perm(w2[i], w3[i], 0x7632), M());
                        }
                    }
                }
            }
            __syncwarp();                                      // the buffer may be filled again
        }
        // ---- the segment's result: the sum of the weights is l 2^(bias - ev), that of values o 2^bias
        const bool partial = s.n < s.nt;
        const int64_t prow0 = ((int64_t)run * 2 + (s.t0 == 0 ? 1 : 0)) * FA_FEW_ROWS;
#pragma unroll
        for (int h = 0; h < RR; ++h) {
            float total = l[h];
            total += __shfl_xor_sync(0xffffffffu, total, 1);
            total += __shfl_xor_sync(0xffffffffu, total, 2);
            const float inv = total == 0.0f ? 0.0f : pow2(ev[h]) / total;
            const bool some = used[h] && total != 0.0f;
            if (live[h]) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int jj = 0; jj < NJ / 8; ++jj) {
                        const int col = F::out_col(2 * t + n, jj);
                        float y[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] = some ? o[8 * jj + e][2 * h + n] * inv : 0.0f;
                        if (odd && used[h]) add_odd<E4M3, T, 8>(a, s, rows, ti[h], col, y);
                        if (partial) {
                            float4 *dst = reinterpret_cast<float4 *>(a.part_o + (prow0 + g + 8 * h) * DP + col);
                            dst[0] = make_float4(y[0], y[1], y[2], y[3]);
                            dst[1] = make_float4(y[4], y[5], y[6], y[7]);
                        } else if (col < D) {
                            *reinterpret_cast<uint4 *>((T *)a.out + orow[h] * D + col) = fa_pack(y, T());
                        }
                    }
                if (t == 0) {
                    const float lse = some ? bias[h] - ev[h] + log2f(total) : -INFINITY;
                    if (partial) a.part_lse[prow0 + g + 8 * h] = lse;
                    else if (a.lse) a.lse[orow[h]] = lse * kLn2;
                }
            }
        }
    }
    cp_wait<0>();
}

template <int DP, bool E4M3, class T, class M, bool R16>
fa_status launch_few(const AttendArgs &a, int ctas, cudaStream_t s) {
    const cudaError_t e = cudaFuncSetAttribute(k_attend_few<DP, E4M3, T, M, R16>, cudaFuncAttributeMaxDynamicSharedMemorySize, Few<DP, E4M3>::SMEM);
    if (e != cudaSuccess) return fa_refuse("fa_tree_attention", cudaGetErrorString(e), FA_ERR_CUDA);
    k_attend_few<DP, E4M3, T, M, R16><<<ctas, 32 * NW, Few<DP, E4M3>::SMEM, s>>>(a);
    return fa_launch_check("tree attention (few rows)");
}
template <int DP, bool E4M3, class T, class M> fa_status launch_few(const AttendArgs &a, int ctas, cudaStream_t s) {
    return a.rows > 8 ? launch_few<DP, E4M3, T, M, true>(a, ctas, s) : launch_few<DP, E4M3, T, M, false>(a, ctas, s);
}
template <bool E4M3, class T, class M> fa_status launch_few(const AttendArgs &a, int ctas, cudaStream_t s) {
    return a.c.head_dim <= 64 ? launch_few<64, E4M3, T, M>(a, ctas, s) : launch_few<128, E4M3, T, M>(a, ctas, s);
}

}  // namespace

int fa_attend_few_tile_shift(int head_dim, bool e4m3) {
    const int slots = head_dim <= 64 ? (e4m3 ? Few<64, true>::CH : Few<64, false>::CH) : (e4m3 ? Few<128, true>::CH : Few<128, false>::CH);
    int shift = 0;
    while (1 << shift < slots) ++shift;
    return shift;
}

fa_status fa_attend_few(const AttendArgs &a, int format, int dtype, int ctas, cudaStream_t s) {
    if (format == FA_CACHE_E4M3)
        return dtype == FA_DTYPE_F16 ? launch_few<true, __half, __half>(a, ctas, s) : launch_few<true, __nv_bfloat16, __half>(a, ctas, s);
    return dtype == FA_DTYPE_F16 ? launch_few<false, __half, __half>(a, ctas, s) : launch_few<false, __nv_bfloat16, __nv_bfloat16>(a, ctas, s);
}
