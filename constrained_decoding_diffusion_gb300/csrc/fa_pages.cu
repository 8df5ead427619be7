// Pages of a cache handed out on the device, and the slots of a ragged batch of tokens.
//
// Both are prefix sums over the sequences followed by independent moves, so that a decoding loop that gains and
// loses sequences needs no host synchronisation.
#include <cooperative_groups.h>

#include "fa_lm.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int NT = 1024;

// inclusive sums of x over the block, and the block's total; all threads
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t *warps, int64_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += up;
    }
    __syncthreads();                     // the last call's sums have been read
    if (lane == 31) warps[warp] = x;
    __syncthreads();
    int64_t before = 0;
    total = 0;
    for (int i = 0; i < n; ++i) {
        before += i < warp ? warps[i] : 0;
        total += warps[i];
    }
    return before + x;
}

struct PagesArgs {
    int B, max_pages, shift, n_pages;
    const int32_t *want;
    int32_t *table, *held, *free_pages, *n_free, *status;
};

// what sequence b holds and wants
__device__ __forceinline__ void sequence(const PagesArgs &a, int b, int &held, int64_t &need) {
    held = min(max(a.held[b], 0), a.max_pages);
    need = ((int64_t)max(a.want[b], 0) + (1 << a.shift) - 1) >> a.shift;
}

// the sequence of the tile whose pages' range holds move k: sums[i] is the number of moves before sequence i
__device__ __forceinline__ int owner(const int64_t *sums, int n, int64_t k) {
    int lo = 0, hi = n;                  // sums[lo] <= k < sums[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= k) lo = mid; else hi = mid;
    }
    return lo;
}

// One cluster.  Every block makes the sums itself, over the sequences in tiles of NT, and moves its part of the
// pages; what is read stays unchanged until all blocks have read it.
__global__ void __launch_bounds__(NT) k_pages_resize(PagesArgs a) {
    __shared__ int64_t warps[NT / 32], sums[NT + 1];
    const cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, part = cluster.block_rank() * NT + tid, parts = cluster.num_blocks() * NT;
    const int64_t n_free = min(max(*a.n_free, 0), a.n_pages);
    // what is given back in all
    int64_t mine = 0, returned, total;
    for (int b = tid; b < a.B; b += NT) {
        int held;
        int64_t need;
        sequence(a, b, held, need);
        mine += max((int64_t)held - need, (int64_t)0);
    }
    block_scan(mine, warps, returned);
    const int64_t there = n_free + returned;
    // pages given back
    int64_t before = 0;
    for (int b0 = 0; b0 < a.B && returned > 0; b0 += NT) {
        int held = 0;
        int64_t need = 0;
        if (b0 + tid < a.B) sequence(a, b0 + tid, held, need);
        const int64_t sum = block_scan(max((int64_t)held - need, (int64_t)0), warps, total);
        sums[tid + 1] = sum;
        if (tid == 0) sums[0] = 0;
        __syncthreads();
        for (int64_t k = part; k < total; k += parts) {
            const int i = owner(sums, NT, k), b = b0 + i;
            int h;
            int64_t n;
            sequence(a, b, h, n);
            int32_t *entry = a.table + (int64_t)b * a.max_pages + n + (k - sums[i]);
            const int64_t to = there - 1 - (before + k);
            if (to < a.n_pages) a.free_pages[to] = *entry;
            *entry = -1;
        }
        before += total;
    }
    __threadfence();
    cluster.sync();
    // pages taken; granted while the sum of all that is wanted up to here is there
    before = 0;
    int64_t taken = 0;
    for (int b0 = 0; b0 < a.B; b0 += NT) {
        int held = 0;
        int64_t need = 0;
        if (b0 + tid < a.B) sequence(a, b0 + tid, held, need);
        const int64_t grow = need <= a.max_pages ? max(need - held, (int64_t)0) : 0;
        const int64_t sum = block_scan(grow, warps, total);
        // a sequence that is refused takes nothing: the sums end before it
        sums[tid + 1] = before + sum <= there ? sum : -1;
        if (tid == 0) sums[0] = 0;
        __syncthreads();
        int n = NT;
        if (sums[NT] < 0) {
            int lo = 0, hi = NT;         // sums[lo] >= 0, sums[hi] < 0
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (sums[mid] >= 0) lo = mid; else hi = mid;
            }
            n = lo;
        }
        const int64_t here = sums[n];
        for (int64_t k = part; k < here; k += parts) {
            const int i = owner(sums, n, k), b = b0 + i;
            const int64_t from = there - 1 - (before + k);
            const int h = min(max(a.held[b], 0), a.max_pages);
            a.table[(int64_t)b * a.max_pages + h + (k - sums[i])] = from < a.n_pages ? a.free_pages[from] : -1;
            if (from < a.n_pages) a.free_pages[from] = -1;
        }
        taken += here;
        before += total;
    }
    cluster.sync();                      // all blocks have read what changes now
    if (cluster.block_rank() != 0) return;
    before = 0;
    for (int b0 = 0; b0 < a.B; b0 += NT) {
        const int b = b0 + tid;
        int held = 0;
        int64_t need = 0;
        if (b < a.B) sequence(a, b, held, need);
        const int64_t grow = need <= a.max_pages ? max(need - held, (int64_t)0) : 0;
        const int64_t sum = before + block_scan(grow, warps, total);
        if (b < a.B) {
            const bool fits = need <= a.max_pages, granted = grow == 0 || sum <= there;
            a.held[b] = fits && granted ? (int)need : held;
            a.status[b] = !fits ? FA_PAGES_TOO_LONG : granted ? FA_PAGES_OK : FA_PAGES_SHORT;
        }
        before += total;
    }
    if (tid == 0) *a.n_free = (int)min(there - taken, (int64_t)a.n_pages);
}

struct MapArgs {
    int B, N, shift, n_pages, max_pages;
    const int32_t *table, *start, *count;
    int32_t *slot, *seq, *position, *offset;
};

// Block (tile of MT sequences, part of their tokens).
constexpr int MT = 256;
__global__ void __launch_bounds__(MT) k_slot_map(MapArgs a) {
    __shared__ int64_t warps[MT / 32], sums[MT + 1];
    const int tid = threadIdx.x, b0 = blockIdx.x * MT, b = b0 + tid;
    int64_t mine = 0, before, total;
    for (int i = tid; i < b0; i += MT) mine += max(a.count[i], 0);
    block_scan(mine, warps, before);
    const int64_t n = b < a.B ? max(a.count[b], 0) : 0;
    const int64_t sum = block_scan(n, warps, total);
    sums[tid + 1] = sum;
    if (tid == 0) sums[0] = 0;
    __syncthreads();
    if (a.offset && blockIdx.y == 0) {
        if (b < a.B) a.offset[b] = (int)min(before + sum - n, (int64_t)a.N);
        if (b == a.B - 1 || (a.B == 0 && tid == 0)) a.offset[a.B] = (int)min(before + sum, (int64_t)a.N);
    }
    const int64_t end = min(total, a.N - before), step = (int64_t)gridDim.y * MT;
    for (int64_t k = (int64_t)blockIdx.y * MT + tid; k < end; k += step) {
        const int i = owner(sums, MT, k), s = b0 + i;
        const int64_t pos = a.start[s] + (k - sums[i]), page_at = pos >> a.shift, at = before + k;
        int page = -1;
        if (pos >= 0 && page_at < a.max_pages) page = a.table[(int64_t)s * a.max_pages + page_at];
        if ((unsigned)page >= (unsigned)a.n_pages) page = -1;
        a.slot[at] = page < 0 ? -1 : (int)((page << a.shift) + (pos & ((1 << a.shift) - 1)));
        if (a.seq) a.seq[at] = s;
        if (a.position) a.position[at] = (int)pos;
    }
    if (blockIdx.x != gridDim.x - 1) return;
    for (int64_t at = before + total + (int64_t)blockIdx.y * MT + tid; at < a.N; at += step) {
        a.slot[at] = -1;
        if (a.seq) a.seq[at] = -1;
        if (a.position) a.position[at] = -1;
    }
}

// the shift of a page's size, or -1
int page_shift(int32_t page_size) {
    int shift = 0;
    while (shift < 10 && (1 << shift) < page_size) ++shift;
    return page_size == 1 << shift ? shift : -1;
}

}  // namespace

extern "C" fa_status fa_pages_resize(int32_t B, int32_t max_pages, int32_t page_size, int32_t n_pages, const int32_t *want,
                                     int32_t *page_table, int32_t *held, int32_t *free_pages, int32_t *n_free,
                                     int32_t *status, fa_stream stream) {
    const char *fn = "fa_pages_resize";
    const int shift = page_shift(page_size);
    if (shift < 0) return fa_refuse(fn, "page_size must be a power of two in [1, 1024]");
    if (B < 0 || B > 65535 || max_pages < 0 || n_pages < 0 || (int64_t)B * max_pages > 2147483647)
        return fa_refuse(fn, "B, max_pages or n_pages out of range");
    if (B == 0) return FA_OK;
    if (!want || !held || !n_free || !status || (max_pages > 0 && !page_table) || (n_pages > 0 && !free_pages))
        return fa_refuse(fn, "NULL buffer");
    const PagesArgs a{B, max_pages, shift, n_pages, want, page_table, held, free_pages, n_free, status};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 8;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(8);
    c.blockDim = dim3(NT);
    c.stream = (cudaStream_t)stream;
    c.attrs = at;
    c.numAttrs = 1;
    (void)cudaLaunchKernelEx(&c, k_pages_resize, a);   // its error is the one the check reads
    return fa_launch_check("pages resize");
}

extern "C" fa_status fa_slot_map(int32_t B, int32_t N, int32_t page_size, int32_t n_pages, const int32_t *page_table,
                                 int32_t max_pages, const int32_t *start, const int32_t *count, int32_t *slot, int32_t *seq,
                                 int32_t *position, int32_t *offset, fa_stream stream) {
    const char *fn = "fa_slot_map";
    const int shift = page_shift(page_size);
    if (shift < 0) return fa_refuse(fn, "page_size must be a power of two in [1, 1024]");
    if (B < 0 || B > 65535 || N < 0 || max_pages < 0 || n_pages < 0 || ((int64_t)n_pages << shift) > 2147483647)
        return fa_refuse(fn, "B, N, max_pages or n_pages out of range");
    if (B == 0 && N == 0 && !offset) return FA_OK;
    if ((B > 0 && (!start || !count)) || (N > 0 && !slot) || (B > 0 && max_pages > 0 && !page_table))
        return fa_refuse(fn, "NULL buffer");
    const MapArgs a{B, N, shift, n_pages, max_pages, page_table, start, count, slot, seq, position, offset};
    const unsigned tiles = (unsigned)std::max(1, (B + MT - 1) / MT);
    const unsigned split = (unsigned)std::max<int64_t>(1, std::min<int64_t>((N + 4 * MT - 1) / (4 * MT), 8 * 152 / tiles));
    k_slot_map<<<dim3(tiles, split), MT, 0, (cudaStream_t)stream>>>(a);
    return fa_launch_check("slot map");
}
