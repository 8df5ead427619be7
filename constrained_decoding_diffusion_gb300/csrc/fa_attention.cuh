// What the two kernels of the attention of drafted tokens share: the work list, slots and pages, masks.
#pragma once

#include "fa_lm.cuh"

namespace fa_attention {

constexpr int MAX_CTAS = 152;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kGrow = 6.0f;                // how far a score may exceed the reference (log2)
// With an 8-bit cache a weight is rounded together with its value's scale.  The reference follows the
// largest such product a row has met: it lies a whole power of two from the largest score's, and the
// weights' own sum is kept without that power.  The power ends at 2^-108, where a tile's weights, up to
// 2^(kGrow + 4 + 108) each, still add up in fp32 (smaller values lose bits of their weights), and at 2^120.
constexpr float kLeastScale = -108.0f;
constexpr float kProductGrow = 10.0f;        // how far a product may exceed the reference: 2^(4 + 10) is below fp16's largest
constexpr uint32_t kAlike = 4u << 23;        // scales whose bits differ by no more are alike: the largest is at most 16 times the least

// Beyond this a reference, times the scale, is rounded so coarsely that a row's largest weight could leave the
// range of fp32 (at 2^30), so scores are taken less the largest one first, which is one more instruction each.
constexpr float kFar = 4194304.0f;

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// the power of the reference for a largest product 2^x times the largest score's weight (NaN: the least)
__device__ __forceinline__ float scale_power(float x) { return fminf(fmaxf(rintf(x), kLeastScale), 120.0f); }

__device__ __forceinline__ float pow2(int e) { return __int_as_float((127 + e) << 23); }   // -126 <= e <= 127
// of a whole number: the sum's last bits are e
__device__ __forceinline__ float pow2(float e) { return __int_as_float((__float_as_int(e + 12582912.0f) << 23) + 0x3f800000); }

struct AttendArgs {
    fa_cache_view c;
    int B, T, heads, group, words, rows, blocks;   // rows of a unit's problem, row blocks of 256
    const void *q;
    int64_t qb, qt, qh;
    const int32_t *length, *count;
    const uint64_t *mask;
    float scale;
    void *out;
    float *lse;
    float *part_o, *part_lse;                      // [MAX_CTAS, 2, 256, DP], [MAX_CTAS, 2, 256]
    int *status;                                   // [MAX_CTAS]
    int box_rows;                                  // rows of a tensor-map box, 0 = no tensor maps
    int tile_shift, unit_cost;                     // log2 of the slots of a tile; what starting a unit costs, in tiles
    int part_rows;                                 // rows of a partial result
    int inject;                                    // (failure tests) a wait of the first block's runs out
};

// ----------------------------------------------------------------------------- the work list

// sequence b's slots: before the draft (up to the table's end), drafted, and the end of what can be
// read.  The host has checked that slots and the number of tiles of all units stay below 2^31.
__device__ __forceinline__ void extent(const AttendArgs &a, int b, int &n, int &use, int &end) {
    const int cap = a.c.max_pages << a.c.page_shift;
    n = min(max(__ldg(a.length + b), 0), cap);
    use = a.count ? min(max(__ldg(a.count + b), 0), a.T) : a.T;
    end = min(n + use, cap);
}
__device__ __forceinline__ int tiles_of(const AttendArgs &a, int b) {
    int n, use, end;
    extent(a, b, n, use, end);
    return max(1, (end + (1 << a.tile_shift) - 1) >> a.tile_shift);   // an empty sequence's rows are written by one masked tile
}
// A unit's share of the work list: its tiles, then unit_cost places that stand for its start (its
// queries, its masked tile, its result) and hold no tile.
__device__ __forceinline__ int places_of(const AttendArgs &a, int b) { return tiles_of(a, b) + a.unit_cost; }

constexpr int RUNS = 64;
struct Work {
    int cum[RUNS + 2];   // places of one (head, row block) before each of 64 runs of sequences
};
__device__ __forceinline__ int run_length(const AttendArgs &a) { return (a.B + RUNS - 1) / RUNS; }

// all threads of the block, 64 at least
__device__ __forceinline__ void plan(const AttendArgs &a, Work &w) {
    const int tid = threadIdx.x, per = run_length(a);
    if (tid < RUNS) {
        int s = 0;
        for (int b = tid * per; b < min(a.B, (tid + 1) * per); ++b) s += places_of(a, b);
        w.cum[tid] = s;
    }
    __syncthreads();
    if (tid < 32) {
        const int s0 = w.cum[2 * tid], s = s0 + w.cum[2 * tid + 1];
        int before = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, before, o);
            if (tid >= o) before += up;
        }
        w.cum[2 * tid] = before - s;
        w.cum[2 * tid + 1] = before - s + s0;
        if (tid == 31) w.cum[RUNS] = before;
    }
    __syncthreads();
}

// the first place of run c, of `total` places over `ctas` runs
__device__ __forceinline__ int run_start(int total, int c, int ctas) { return (int)((int64_t)total * c / ctas); }

struct Segment {
    int b, head, block;       // the unit
    int nt, t0, n;            // its tiles, the first of this segment, how many
    int rows;                 // rows of the row block (up to 256)
    int slots, use, end;      // before the draft, drafted, the end of what can be read
    // (tensor cores) two row tiles of 128 over the same key/value tiles, or one over alternate ones
    __device__ __forceinline__ bool two() const { return rows > 128; }
};

struct Walk {
    int left, t0;             // places of the run still to come; the next place of the unit
    int b, head, block;       // the unit
    __device__ __forceinline__ Walk(const AttendArgs &a, const Work &w, int cta, int ctas) {
        const int units = a.c.kv_heads * a.blocks, total = w.cum[RUNS] * units;
        ctas = min(total, ctas);                    // no run is empty
        left = t0 = b = head = block = 0;
        if (cta >= ctas) return;
        const int g = run_start(total, cta, ctas);
        left = run_start(total, cta + 1, ctas) - g;
        int lo = 0, hi = RUNS;                      // the last run that starts at or before g
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (w.cum[mid] * units <= g) lo = mid; else hi = mid;
        }
        b = lo * run_length(a);
        int base = w.cum[lo] * units, places;
        while (true) {
            places = places_of(a, b);
            if (g < base + places * units) break;
            base += places * units;
            ++b;
        }
        const int u = (g - base) / places;
        t0 = g - base - u * places;
        head = u / a.blocks;
        block = u - head * a.blocks;
    }
    __device__ __forceinline__ bool next(const AttendArgs &a, Segment &s) {
        while (left > 0) {
            extent(a, b, s.slots, s.use, s.end);
            s.b = b;
            s.head = head;
            s.block = block;
            s.nt = max(1, (s.end + (1 << a.tile_shift) - 1) >> a.tile_shift);
            s.t0 = t0;
            s.n = min(s.nt - t0, left);
            s.rows = min(a.rows - 256 * block, 256);
            left -= s.nt + a.unit_cost - t0;
            t0 = 0;
            if (++block == a.blocks) {
                block = 0;
                if (++head == a.c.kv_heads) { head = 0; ++b; }
            }
            if (s.n > 0) return true;               // the run may begin behind a unit's last tile
        }
        return false;
    }
};

// zero the elements of eight 16-bit floats that are not finite; true if there was one
template <class M> __device__ __forceinline__ bool zero_odd(uint4 &x) {
    constexpr uint32_t em = sizeof(M) == 2 && std::is_same<M, __half>::value ? 0x7c00u : 0x7f80u;
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((w[i] & em) == em) { w[i] &= 0xffff0000u; odd = true; }
        if ((w[i] >> 16 & em) == em) { w[i] &= 0x0000ffffu; odd = true; }
    }
    x = make_uint4(w[0], w[1], w[2], w[3]);
    return odd;
}

// Where a sequence's slots lie for one head.  The slot is below Segment::end, so its page number is
// in the table.
struct Rows {
    const int32_t *pages;
    uint32_t n_pages, heads, head, shift;
    __device__ __forceinline__ Rows() {}
    __device__ __forceinline__ Rows(const AttendArgs &a, const Segment &s)
        : pages(a.c.page_table + (int64_t)s.b * a.c.max_pages), n_pages(a.c.n_pages), heads(a.c.kv_heads), head(s.head),
          shift(a.c.page_shift) {}
    __device__ __forceinline__ uint32_t page(uint32_t slot) const { return (uint32_t)__ldg(pages + (slot >> shift)); }
    // the row of a slot in a page, or -1 when there is no such page
    __device__ __forceinline__ int64_t row(uint32_t page, uint32_t slot) const {
        if (page >= n_pages) return -1;
        return ((int64_t)(page * heads + head) << shift) + (slot & ((1u << shift) - 1));
    }
    __device__ __forceinline__ int64_t row(uint32_t slot) const { return row(page(slot), slot); }
};

// which of the 32 slots from `first` on drafted token i of sequence b sees
__device__ __forceinline__ uint32_t seen_bits(const AttendArgs &a, const Segment &s, int i, int first) {
    const int d0 = first - s.slots;
    if (d0 <= -32) return 0xffffffffu;
    const int from = min(max(d0, 0), s.use);
    uint32_t v = 0xffffffffu;
    if (a.mask && from < s.use) {
        const uint64_t *m = a.mask + ((int64_t)s.b * a.T + i) * a.words;
        const int w = from >> 6, sh = from & 63;
        uint64_t x = __ldg(m + w) >> sh;
        if (sh > 32 && w + 1 < a.words) x |= __ldg(m + w + 1) << (64 - sh);
        v = (uint32_t)x;
    }
    const int left = s.use - from;
    if (left < 32) v &= left > 0 ? (1u << left) - 1 : 0u;
    if (d0 < 0) v = v << -d0 | ((1u << -d0) - 1);
    return v;
}

template <class T> __device__ __forceinline__ T bits_as(uint16_t u) {
    T x;
    memcpy(&x, &u, 2);
    return x;
}

// Drafted values that are not finite are left out of the products (a row that does not see them must
// not meet them); here they join the rows that do: N columns from col on of drafted token t's result.
template <bool E4M3, class T, int N>
__device__ __forceinline__ void add_odd(const AttendArgs &a, const Segment &s, const Rows &rows, int t, int col, float (&o)[N]) {
#pragma unroll 1
    for (int j = 0; j < s.use; ++j) {
        const int slot = s.slots + j;
        if (slot < s.t0 << a.tile_shift || slot >= (s.t0 + s.n) << a.tile_shift || slot >= s.end || !(seen_bits(a, s, t, slot) & 1)) continue;
        const int64_t at = rows.row((uint32_t)slot);
        if (at < 0) continue;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            if (col + e >= a.c.head_dim) break;
            const int64_t x = at * a.c.head_dim + col + e;
            float y;
            if (E4M3) y = (((const uint8_t *)a.c.v)[x] & 0x7f) == 0x7f || !(fabsf(a.c.v_scale[at]) < INFINITY) ? NAN : 0.0f;
            else y = fa_to_f32(((const T *)a.c.v)[x]);
            if (!isfinite(y)) o[e] += y;
        }
    }
}

}  // namespace fa_attention

// up to 16 rows a unit (fa_tree_attention_few.cu)
int fa_attend_few_tile_shift(int head_dim, bool e4m3);
fa_status fa_attend_few(const fa_attention::AttendArgs &a, int format, int dtype, int ctas, cudaStream_t s);
constexpr int FA_FEW_ROWS = 16, FA_FEW_WARPS = 8;
