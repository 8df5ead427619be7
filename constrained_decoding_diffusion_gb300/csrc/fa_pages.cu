// Pages of a cache handed out on the device, and the slots of a ragged batch of tokens.
//
// Both are prefix sums over the sequences followed by independent moves, so that a decoding loop that gains and
// loses sequences needs no host synchronisation.
#include <cooperative_groups.h>

#include "fa_lm.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int NT = 1024;

// inclusive sums of x over the block's n warps, and the block's total; all threads
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t *warps, int n, int64_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += up;
    }
    __syncthreads();                     // the last call's sums have been read
    if (lane == 31) warps[warp] = x;
    __syncthreads();
    // every warp adds up the warps' sums itself
    int64_t all = lane < n ? warps[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, all, o);
        if (lane >= o) all += up;
    }
    total = __shfl_sync(0xffffffffu, all, 31);
    const int64_t before = __shfl_sync(0xffffffffu, all, max(warp - 1, 0));
    return warp ? before + x : x;
}

struct PagesArgs {
    int B, max_pages, shift, n_pages;
    const int32_t *want;
    int32_t *table, *held, *free_pages, *n_free, *status;
};

// The sequences of a tile: what each holds and wants, and the pages given back and wanted before each.
struct Tile {
    int64_t warps[NT / 32];
    int32_t held[NT], need[NT], back[NT + 1], grow[NT + 1];
};

// the sequence of a tile of N (a power of two) whose range holds move k: sums[i] is the number of moves before sequence i
template <int N, class S> __device__ __forceinline__ int owner(const S *sums, int64_t k) {
    int lo = 0;                          // sums[lo] <= k < sums[N]
#pragma unroll
    for (int step = N / 2; step; step /= 2)
        if (sums[lo + step] <= k) lo += step;
    return lo;
}

// One block, or a cluster of them whose blocks all make the sums and move a part of the pages each.  Sequences come in
// tiles of a block's threads; up to one tile (the common case) is read and summed up once.
// What bounds it is the chain of steps: lengths, their sums, the copies down and up the stack with a barrier between.
// Measured in a graph: 64 sequences that take a page each 3.3 us, 1024 5.7, 102400 pages moved 12 (8 bytes a page: 0.07
// TB/s), a million 81.
template <bool CLUSTER> __global__ void __launch_bounds__(NT) k_pages_resize(PagesArgs a) {
    constexpr int U = 4;                 // moves of a thread under way
    __shared__ Tile t;
    const cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, rank = CLUSTER ? cluster.block_rank() : 0, parts = CLUSTER ? cluster.num_blocks() * NT : NT;
    const int part = rank * NT + tid;
    const bool single = a.B <= NT;
    auto meet = [&]() {                  // the others' writes are seen after
        if (CLUSTER) { __threadfence(); cluster.sync(); }
        else __syncthreads();
    };
    int held = 0;                        // of the thread's sequence of the tile
    int64_t need = 0, grow = 0, upto = 0;
    auto load = [&](int b) {
        held = 0;
        need = 0;
        if (b < a.B) {
            held = min(max(a.held[b], 0), a.max_pages);
            need = ((int64_t)max(a.want[b], 0) + (1 << a.shift) - 1) >> a.shift;
        }
        grow = need <= a.max_pages ? max(need - held, (int64_t)0) : 0;
    };
    // the tile's sums, pages given back in the low half and wanted in the high one (the host has checked that both fit)
    int64_t tile_back, tile_grow;
    auto sum = [&](int b0) {
        load(b0 + tid);
        int64_t total;
        const int64_t both = block_scan(max((int64_t)held - need, (int64_t)0) + (grow << 32), t.warps, NT / 32, total);
        tile_back = total & 0xffffffff;
        tile_grow = total >> 32;
        upto = both >> 32;
        t.held[tid] = held;
        t.need[tid] = (int)min(need, (int64_t)a.max_pages);
        t.back[tid + 1] = (int)(both & 0xffffffff);
        t.grow[tid + 1] = (int)upto;
        if (tid == 0) t.back[0] = t.grow[0] = 0;
        __syncthreads();
    };
    const int64_t n_free = min(max(*a.n_free, 0), a.n_pages);
    int64_t returned = 0;
    if (single) {
        sum(0);
        returned = tile_back;
    } else {
        int64_t mine = 0;
        for (int b = tid; b < a.B; b += NT) { load(b); mine += max((int64_t)held - need, (int64_t)0); }
        block_scan(mine, t.warps, NT / 32, returned);
    }
    const int64_t there = n_free + returned;
    // ---- pages given back: move k goes k places below the new top
    int64_t before = 0;
    for (int b0 = 0; b0 < a.B && returned > 0; b0 += NT) {
        if (!single) sum(b0);
        for (int64_t k0 = part; k0 < tile_back; k0 += U * parts) {
            int32_t *entry[U], page[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t k = k0 + u * parts;
                if (k >= tile_back) break;
                const int i = owner<NT>(t.back, k);
                entry[u] = a.table + (int64_t)(b0 + i) * a.max_pages + t.need[i] + (k - t.back[i]);
                page[u] = *entry[u];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t k = k0 + u * parts, to = there - 1 - (before + k);
                if (k >= tile_back) break;
                if (to < a.n_pages) a.free_pages[to] = page[u];
                *entry[u] = -1;
            }
        }
        before += tile_back;
    }
    if (returned > 0 || CLUSTER) meet();
    // ---- pages taken, from the top: granted while the sum of all that is wanted up to here is there
    before = 0;
    int64_t taken = 0;
    for (int b0 = 0; b0 < a.B; b0 += NT) {
        if (!single) sum(b0);
        int n = NT;                      // the sequences that take theirs
        if (before + tile_grow > there) {
            int lo = 0, hi = NT;         // grow[lo] is there, grow[hi] is not
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (before + t.grow[mid] <= there) lo = mid; else hi = mid;
            }
            n = before <= there ? lo : 0;
        }
        const int64_t here = t.grow[n];
        for (int64_t k0 = part; k0 < here; k0 += U * parts) {
            int32_t page[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t k = k0 + u * parts, from = there - 1 - (before + k);
                page[u] = k < here && from < a.n_pages ? a.free_pages[from] : -1;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t k = k0 + u * parts, from = there - 1 - (before + k);
                if (k >= here) break;
                const int i = owner<NT>(t.grow, k);
                if (from < a.n_pages) a.free_pages[from] = -1;
                a.table[(int64_t)(b0 + i) * a.max_pages + t.held[i] + (k - t.grow[i])] = page[u];
            }
        }
        taken += here;
        before += tile_grow;
    }
    // ---- what changed, once all blocks have read what was (a single tile: before the last meeting)
    if (!single) meet();
    if (rank != 0) return;
    before = 0;
    for (int b0 = 0; b0 < a.B; b0 += NT) {
        if (!single) sum(b0);
        const int b = b0 + tid;
        if (b < a.B) {
            const bool fits = need <= a.max_pages, granted = grow == 0 || before + upto <= there;
            a.held[b] = fits && granted ? (int)need : held;
            a.status[b] = !fits ? FA_PAGES_TOO_LONG : granted ? FA_PAGES_OK : FA_PAGES_SHORT;
        }
        before += tile_grow;
    }
    if (tid == 0) *a.n_free = (int)min(there - taken, (int64_t)a.n_pages);
}

struct MapArgs {
    int B, N, shift, n_pages, max_pages;
    const int32_t *table, *start, *count;
    int32_t *slot, *seq, *position, *offset;
};

// Block (tile of MT sequences, part of their tokens).  What bounds it is the chain of counts, sums, search and page
// number: 64 sequences of a token each 4.0 us in a graph, 65536 tokens of 256 sequences 4.4.
constexpr int MT = 256;
__global__ void __launch_bounds__(MT) k_slot_map(MapArgs a) {
    __shared__ int64_t warps[MT / 32], sums[MT + 1];
    const int tid = threadIdx.x, b0 = blockIdx.x * MT, b = b0 + tid;
    int64_t mine = 0, before, total;
    for (int i = tid; i < b0; i += MT) mine += max(a.count[i], 0);
    block_scan(mine, warps, MT / 32, before);
    const int64_t n = b < a.B ? max(a.count[b], 0) : 0;
    const int64_t sum = block_scan(n, warps, MT / 32, total);
    sums[tid + 1] = sum;
    if (tid == 0) sums[0] = 0;
    __syncthreads();
    if (a.offset && blockIdx.y == 0) {
        if (b < a.B) a.offset[b] = (int)min(before + sum - n, (int64_t)a.N);
        if (b == a.B - 1 || (a.B == 0 && tid == 0)) a.offset[a.B] = (int)min(before + sum, (int64_t)a.N);
    }
    const int64_t end = min(total, a.N - before), step = (int64_t)gridDim.y * MT;
    for (int64_t k = (int64_t)blockIdx.y * MT + tid; k < end; k += step) {
        const int i = owner<MT>(sums, k), s = b0 + i;
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
    cudaStream_t s = (cudaStream_t)stream;
    // One block where the tables are small.  One block / a cluster of eight: 64 sequences of up to 257 pages that take or
    // give back a page each 3.3 / 4.1 us, 200 pages each 10.4 / 5.3; 256 of 528 with a page each 3.3 / 4.2, with 400 pages
    // each 58 / 12 (the number of pages that move is known on the device only).
    if ((int64_t)B * max_pages <= 65536) {
        k_pages_resize<false><<<1, NT, 0, s>>>(a);
    } else {
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 8;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t c = {};
        c.gridDim = dim3(8);
        c.blockDim = dim3(NT);
        c.stream = s;
        c.attrs = at;
        c.numAttrs = 1;
        (void)cudaLaunchKernelEx(&c, k_pages_resize<true>, a);   // its error is the one the check reads
    }
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
    const unsigned split = (unsigned)std::max<int64_t>(1, std::min<int64_t>(((int64_t)N + 4 * MT - 1) / (4 * MT), 8 * 152 / tiles));
    k_slot_map<<<dim3(tiles, split), MT, 0, (cudaStream_t)stream>>>(a);
    return fa_launch_check("slot map");
}
