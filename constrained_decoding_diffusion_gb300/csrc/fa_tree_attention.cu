// Attention of drafted tokens over a paged cache, on the 5th-generation tensor cores.
//
// The mathematics.  A row is one query (drafted token i, query head) of a sequence and a
// key/value head; it sees the slots before the draft and the drafted slots its mask allows.  With
// x_t = log2(e) scale q . k_t, out = sum_t 2^(x_t) v_t / sum_t 2^(x_t), computed in one pass
// over the slots: every weight is taken relative to a reference B of the row, p_t = 2^(x_t - B),
// with l = sum p_t and O = sum p_t v_t; when a tile's largest x_t exceeds the reference's by more
// than 6 (a factor of 64), B moves and O and l are scaled by 2^(B_old - B_new).  out = O / l
// and lse = (B + log2 l) ln 2 for any B, and parts over disjoint slots join by their lse.
//
// An 8-bit cache (codes times one scale per slot and head): the key's scale multiplies the
// score, the value's the weight, so the codes themselves go to the tensor cores, as fp16 (exact).
// q is scaled per row by a power of two into the middle of the fp16 range (exact but for elements below 2^-22 of
// the row's largest, whose last bits fp16 drops) and the factor
// goes to the exponent; B follows the largest product of a weight and its value's scale that a row
// meets, so that the products stay in fp16's range with 24 bits or more below the largest.  Where all
// slots of a tile are seen and their scales are within 16 times one another, the largest score with
// the largest scale stands for the tile's largest product; else the products are looked at one by one
// (2 x 98304 slots x 64 rows: 185 us, 247 if every tile took that path).
//
// The layout.  All query heads of one key/value head and all drafted tokens are rows of one
// problem, so a cached tile is read once for up to 256 rows: two tiles of 128 rows are two
// streams (a warpgroup each, its own scores and accumulator in tensor memory) over the same key
// and value tiles.  With up to 128 rows the two streams take alternate key/value tiles of the
// same rows instead, and their results are joined at the end: either way the tensor cores work on
// one stream while the other one's softmax runs.  The work is the list of all tiles of 128
// slots of all (sequence, head, row block) units; one block per SM takes an equal run of it,
// whatever the lengths, which are read on the device.  A unit that is cut by the runs leaves
// partial results, joined by a second small kernel in a fixed order.  Problems of up to 16 rows go
// to a kernel without shared tiles (fa_tree_attention_few.cu).
//
// Roles (20 warps): warps 0-7 the two softmax warpgroups (a thread per row), warps 8-15 load and
// convert (16-byte asynchronous copies into 128-byte-swizzled tiles), warp 16 issues the MMAs
// (17-19 only complete its warpgroup, whose registers go to the softmax):
// S = Q K^T (both from shared memory), P overwrites S in tensor memory as the 16-bit left operand
// of O += P V, with V read from the same layout as K but as the MN-major operand.
//
// What bounds it, and what it measured (head_dim 128, 8 key/value heads, replayed in a graph).  16-bit
// cache: 16 sequences of 8192 slots x 256 rows 152 us, 549 MB read (3.6 TB/s) and 140 GFLOP (0.9
// PFLOP/s): per tile of 128 slots 2.1 us an SM, of which the softmax of 256 rows takes most (copies
// 1.45, MMA 1.7); about 40 us are fixed (launch, first tiles, results).  8-bit cache: 2 x 98304 slots
// x 64 rows 185 us (2.2 TB/s): the conversion of a tile takes 1.6 us, its copy 0.7.
//
// Roundings.  Both operands of the second product have one 16-bit type, so the weights take the cache's: bf16
// (8 bits) on a bf16 cache, else fp16.  The sum of the weights is taken before that, in fp32, which costs no
// instruction and keeps lse free of the rounding; the result then carries the roundings of single
// weights.  Against 64 bits, 16 x 8192 slots in bf16: 0.0023 of the result, where its own rounding alone is
// 0.0017.
//
// Every wait is bounded (about a second).  A wait that runs out marks the block's status; the
// joining kernel then sets the rows the block had a part in to NaN.
#include "fa_attention.cuh"
#include "fa_tensor.cuh"

using namespace fa_attention;

namespace {

constexpr int TS = 128;                      // slots of a tile, rows of a stream
constexpr int NLOAD = 8 * 32, NTHR = 20 * 32;
// registers a thread of each role, of the 96 the block is launched with: 256 softmax + 256 load +
// 128 MMA threads use 640 * 96 either way.  16-bit, 16 x 8192 slots x 256 rows: 112, 80 and 96 157 us, 120, 72 and
// 96 153 (head_dim up to 64: the loads would spill), 128, 64 and 96 157.  8-bit, where the code of masked tiles
// spills a few either way: 128, 72 and 80 and 136, 64 and 80 measured 3% and 2% slower than 128, 64 and 96.
template <int DP, bool E4M3> struct Regs {
    static constexpr int SOFTMAX = E4M3 ? 128 : DP == 128 ? 120 : 112, LOAD = E4M3 ? 64 : DP == 128 ? 72 : 80, MMA = 96;
};
constexpr int kUnitCost = 3;                 // what starting a unit costs, in tiles

// The order in which a segment's key and value tiles are consumed: with two row tiles K0 V0 K1 V1
// ...; with alternating streams K0 K1 V0 K2 V1 ... (the next tile's scores are started before the
// previous tile's weights are ready).
__device__ __forceinline__ void item_of(const Segment &s, int i, int &tile, bool &value) {
    if (s.two() || s.n == 1) { tile = i >> 1; value = i & 1; return; }
    if (i < 2) { tile = i; value = false; return; }
    const int j = (i - 2) >> 1;
    value = !(i & 1) || j + 2 >= s.n;
    tile = !(i & 1) ? j : j + 2 < s.n ? j + 2 : s.n - 1;
}

// ----------------------------------------------------------------------------- the kernel

template <int DP, bool E4M3>
struct Shape {
    static constexpr int TILE = TS * DP * 2;                       // a 16-bit tile in shared memory
    static constexpr int NS = E4M3 ? (DP == 64 ? 4 : 3) : (DP == 64 ? 10 : 5);   // tiles in the ring
    static constexpr int RAW = TS * DP, NR = E4M3 ? (DP == 64 ? 8 : 4) : 0;      // raw 8-bit tiles in flight
    static constexpr int Q = 0, RING = 2 * TILE, RAWS = RING + NS * TILE, MISC = RAWS + NR * RAW;
};

struct Misc {
    uint64_t full[10], empty[10], s_full[2], p_full[2], pv_done[2], q_full[2], done;
    uint64_t raw_full[8], raw_empty[8];
    uint64_t by_hand[16];             // tile by hand & 15: its place in the ring is free
    uint32_t raw_rows[8][4];          // which rows of a raw tile were copied
    uint32_t tmem;
    int fail;
    // A drafted value, or a scale, that is not finite is marked by its segment's number, so that nothing
    // has to be cleared: the loading warps, at most six segments ahead of stream 0, by odd[segment & 7];
    // each stream by an entry of its own, since stream 1 passes over segments of a single tile and may be
    // any number of them ahead of stream 0.
    int odd[8], odd_scale[2];         // 1 + the last segment that was marked
    int hole[16];                     // key tile & 15: a slot of the tile has no page or lies past the end
    float vtop[2][4];                 // per stream: log2 of the largest value scale of 32 slots, inf where they differ widely
};
struct Scales { float k[2][TS], v[2][TS]; };   // per stream, of its tile

template <int DP, bool E4M3> constexpr size_t smem_bytes() {
    return Shape<DP, E4M3>::MISC + sizeof(Misc) + sizeof(Work) + (E4M3 ? sizeof(Scales) : 0);
}

// where chunk c (16 bytes = 8 elements) of row r lies in a 128-byte-swizzled tile: halves of 64
// columns, rows of 128 bytes, the eight chunks of a row permuted by the row's low bits
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    return (uint32_t)((c >> 3) * (TS * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// The key and value tiles of a block's work in the order of their consumption.
struct Feed {
    Walk walk;
    Segment s;
    int i, seg, tile;
    bool value;
    __device__ __forceinline__ Feed(const Walk &w) : walk(w), i(0), seg(-1) { s.n = 0; }
    __device__ __forceinline__ bool next(const AttendArgs &a) {
        if (i == 2 * s.n) {
            i = 0;
            if (!walk.next(a, s)) { s.n = 0; return false; }
            ++seg;
        }
        item_of(s, i++, tile, value);
        return true;
    }
    __device__ __forceinline__ uint32_t first() const { return (uint32_t)(s.t0 + tile) * TS; }
    // drafted values may be hidden from some rows
    __device__ __forceinline__ bool draft() const { return value && (s.t0 + tile + 1) * TS > s.slots; }
    // a 16-bit tile that the loading warps bring themselves: a page may end in it, or its values need
    // a look; all others come by tensor copies
    __device__ __forceinline__ bool by_hand(const AttendArgs &a) const {
        return !a.box_rows || (s.t0 + tile + 1) * TS > s.end || draft();
    }
};

// A loading thread's share of a tile: one 16-byte chunk of every STEP-th row.  The page numbers of
// the next tile are fetched while the current one is issued.  A page's rows of one head are
// contiguous, and the place of a tile's row in its page depends on the tile only when a page is
// longer than a tile.
template <int STEP>
struct Share {
    static constexpr int ITER = TS / STEP;
    uint32_t page[ITER];
    uint32_t n_pages, in_page, page_bytes, row_bytes, r0;
    __device__ __forceinline__ Share(const AttendArgs &a, int r0_, int row_bytes_)
        : n_pages(a.c.n_pages), in_page((1u << a.c.page_shift) - 1), row_bytes(row_bytes_), r0(r0_) {
        page_bytes = (uint32_t)row_bytes << a.c.page_shift;
    }
    __device__ __forceinline__ void look(const AttendArgs &a, const Feed &f) {
        const int32_t *pages = a.c.page_table + (int64_t)f.s.b * a.c.max_pages;
        const uint32_t first = f.first() + r0, end = (uint32_t)f.s.end;
#pragma unroll
        for (int q = 0; q < ITER; ++q)
            page[q] = first + q * STEP < end ? (uint32_t)__ldg(pages + ((first + q * STEP) >> a.c.page_shift)) : 0xffffffffu;
    }
    // the bytes of the q-th row, from the head's bytes in page 0
    __device__ __forceinline__ const unsigned char *at(const unsigned char *base, uint64_t stride, uint32_t first, int q) const {
        return base + (page[q] < n_pages ? page[q] : 0) * stride + ((first + q * STEP) & in_page) * row_bytes;
    }
    __device__ __forceinline__ bool held(int q) const { return page[q] < n_pages; }
};

// M: the tensor cores' 16-bit type; T: q's and out's
template <int DP, bool E4M3, class T, class M>
__global__ void __launch_bounds__(NTHR, 1) k_attend(AttendArgs a, const __grid_constant__ CUtensorMap map_k,
                                                    const __grid_constant__ CUtensorMap map_v) {
    using S = Shape<DP, E4M3>;
    extern __shared__ __align__(1024) unsigned char smem[];
    constexpr size_t MISC = S::MISC + (E4M3 ? sizeof(Scales) : 0);
    static_assert(S::MISC % 16 == 0 && MISC % 8 == 0 && sizeof(Misc) % 8 == 0, "alignment of the parts");
    Scales &sc = *reinterpret_cast<Scales *>(smem + S::MISC);       // first: read in 16-byte pieces
    Misc &sh = *reinterpret_cast<Misc *>(smem + MISC);
    Work &work = *reinterpret_cast<Work *>(smem + MISC + sizeof(Misc));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr bool F16 = std::is_same<M, __half>::value;
    constexpr float OFF = F16 ? 4.0f : 0.0f;          // fp16 weights reach 2^10 above and 2^-28 below a row's largest
    const int D = a.c.head_dim;
    volatile int *fail = &sh.fail;
    if (smem_u32(smem) & 1023) {           // the swizzled tiles need it
        if (tid == 0) a.status[blockIdx.x] = 1;
        return;
    }

    if (tid == 0) {
        for (int i = 0; i < S::NS; ++i) { mbar_init(&sh.full[i], NLOAD / 32); mbar_init(&sh.empty[i], 1); }
        for (int i = 0; i < S::NR; ++i) { mbar_init(&sh.raw_full[i], 1); mbar_init(&sh.raw_empty[i], NLOAD / 32); }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i], 4);
            mbar_init(&sh.pv_done[i], 1);
            mbar_init(&sh.q_full[i], 4);
        }
        for (int i = 0; i < 16; ++i) mbar_init(&sh.by_hand[i], 1);
        mbar_init(&sh.done, 1);
        sh.fail = 0;
        for (int i = 0; i < 8; ++i) sh.odd[i] = 0;
        sh.odd_scale[0] = sh.odd_scale[1] = 0;
        for (int i = 0; i < 16; ++i) sh.hole[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 16) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    fa_let_next_start();
    plan(a, work);
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    Walk walk(a, work, blockIdx.x, gridDim.x);
    Segment s;

    if (warp >= 16) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<DP, E4M3>::MMA));
        if (warp == 16 && lane == 0) {
            // ---- the MMAs
            constexpr uint32_t fmt = F16 ? 0u : 1u;
            constexpr uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(TS >> 4) << 24);
            constexpr uint32_t idesc_s = idesc | ((uint32_t)(TS >> 3) << 17);                 // S: N = 128 slots
            constexpr uint32_t idesc_o = idesc | ((uint32_t)(DP >> 3) << 17) | (1u << 16);    // O: N = DP, V is MN-major
            Ring<S::NS> get;
            int nq[2] = {0, 0}, np[2] = {0, 0};
            const uint32_t q0 = smem_u32(smem + S::Q), ring = smem_u32(smem + S::RING);
            auto next_tile = [&]() -> int {
                const int slot = get.slot;
                if (!mbar_wait(&sh.full[slot], get.phase, fail)) return -1;
                ++get;
                return slot;
            };
            auto scores = [&](int st, int slot) {
                const uint64_t qd = umma_desc(q0 + st * S::TILE, 16), kd = umma_desc(ring + slot * S::TILE, 16);
                const uint32_t d = tmem + st * TS;
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    const uint32_t off = ((k >> 2) * (TS * 128) + (k & 3) * 32) / 16;
                    umma_ss(d, qd + off, kd + off, idesc_s, k > 0);
                }
                umma_commit(&sh.s_full[st]);
            };
            auto values = [&](int st, int slot, bool first, bool last) {
                const uint64_t vd = umma_desc(ring + slot * S::TILE, TS * 128);
                const uint32_t d = tmem + 256 + st * DP, p = tmem + st * TS;
#pragma unroll
                for (int k = 0; k < TS / 16; ++k) umma_ts(d, p + k * 8, vd + k * (2048 / 16), idesc_o, !first || k > 0);
                if (last) umma_commit(&sh.pv_done[st]);   // else the next scores' barrier says it too
            };
            auto wait_p = [&](int st) {
                const bool ok = mbar_wait(&sh.p_full[st], (uint32_t)np[st] & 1, fail);
                ++np[st];
                tc_fence_after();
                return ok;
            };
            if (a.inject && blockIdx.x == 0) {   // a failure test: only this thread completes `done`, later
                const long long t0 = clock64();
                while (!mbar_try_wait(&sh.done, 0) && clock64() - t0 < kInjectCycles) {}
                *fail = 1;
            }
            while (!*fail && walk.next(a, s)) {
                const int streams = s.two() || s.n > 1 ? 2 : 1;
                bool ok = true;
                for (int st = 0; st < streams; ++st) ok &= mbar_wait(&sh.q_full[st], (uint32_t)nq[st]++ & 1, fail);
                if (!ok) break;
                tc_fence_after();
                int slot;
                if (s.two()) {
                    if ((slot = next_tile()) < 0) break;
                    scores(0, slot);
                    scores(1, slot);
                    umma_commit(&sh.empty[slot]);
                    for (int j = 0; j < s.n && ok; ++j) {
                        const int vs = next_tile();
                        if (vs < 0 || !wait_p(0)) { ok = false; break; }
                        values(0, vs, j == 0, j + 1 == s.n);
                        int ks = -1;
                        if (j + 1 < s.n) {
                            if ((ks = next_tile()) < 0) { ok = false; break; }
                            scores(0, ks);
                        }
                        if (!wait_p(1)) { ok = false; break; }
                        values(1, vs, j == 0, j + 1 == s.n);
                        umma_commit(&sh.empty[vs]);
                        if (ks >= 0) {
                            scores(1, ks);
                            umma_commit(&sh.empty[ks]);
                        }
                    }
                } else {
                    for (int j = 0; j < streams && ok; ++j) {
                        if ((slot = next_tile()) < 0) { ok = false; break; }
                        scores(j, slot);
                        umma_commit(&sh.empty[slot]);
                    }
                    for (int j = 0; j < s.n && ok; ++j) {
                        const int st = j & 1;
                        if ((slot = next_tile()) < 0 || !wait_p(st)) { ok = false; break; }
                        values(st, slot, j < 2, j + 2 >= s.n);
                        umma_commit(&sh.empty[slot]);
                        if (j + 2 < s.n) {
                            if ((slot = next_tile()) < 0) { ok = false; break; }
                            scores(st, slot);
                            umma_commit(&sh.empty[slot]);
                        }
                    }
                }
                if (!ok) break;
            }
            // every MMA issued has completed before tensor memory is released
            umma_commit(&sh.done);
            const long long t0 = clock64();
            while (!mbar_try_wait(&sh.done, 0))
                if (clock64() - t0 > kSpinCycles) { *fail = 1; break; }
        }
        if constexpr (E4M3) {
        if (warp == 17) {
            // ---- raw codes: one bulk copy for the slots of a tile that share a page
            Feed f(walk);
            Rows rows;
            uint32_t page[4];
            auto look = [&]() {
                rows = Rows(a, f.s);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t slot = f.first() + 32 * w + lane;
                    page[w] = slot < (uint32_t)f.s.end ? rows.page(slot) : 0xffffffffu;
                }
            };
            const uint32_t in_page = (1u << a.c.page_shift) - 1;
            bool more = f.next(a);
            if (more) look();
            int it = 0, keys = 0;
            Ring<S::NR> put;
            for (; more; ++it) {
                const int slot = put.slot;
                if (it >= S::NR && !mbar_wait(&sh.raw_empty[slot], put.phase ^ 1, fail)) break;
                __syncwarp();
                uint32_t there[4], n = 0;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    there[w] = __ballot_sync(0xffffffffu, page[w] < rows.n_pages);
                    n += __popc(there[w]);
                }
                if (lane == 0) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) sh.raw_rows[slot][w] = there[w];
                    if (!f.value) sh.hole[keys & 15] = n < TS;
                    mbar_expect(&sh.raw_full[slot], n * D);
                }
                __syncwarp();
                keys += !f.value;
                const uint8_t *src = (const uint8_t *)(f.value ? a.c.v : a.c.k);
                const uint32_t dst = smem_u32(smem + S::RAWS) + slot * S::RAW;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t r = 32 * w + lane, at = f.first() + r;
                    if (page[w] < rows.n_pages && ((at & in_page) == 0 || r == 0)) {
                        const uint32_t len = min(min(in_page + 1 - (at & in_page), TS - r), (uint32_t)f.s.end - at);
                        bulk_copy(dst + r * D, src + rows.row(page[w], at) * D, len * D, &sh.raw_full[slot]);
                    }
                }
                ++put;
                more = f.next(a);
                if (more) look();
            }
            // no copy may land after the block has gone
            for (int i = max(it - S::NR, 0); i < it; ++i) {
                const long long t0 = clock64();
                while (!mbar_try_wait(&sh.raw_full[i % S::NR], (uint32_t)(i / S::NR) & 1) && clock64() - t0 < kSpinCycles) {}
            }
        }
        } else if (warp == 17 && a.box_rows) {
            // ---- 16-bit tiles by tensor copies: a lane per box of (a page's rows) x 64 columns
            Feed f(walk);
            const int boxes = TS / a.box_rows, mine = lane % boxes, half = lane / boxes;
            const bool copies_box = half < DP / 64;
            const uint32_t in_page = (1u << a.c.page_shift) - 1;
            uint32_t page = 0;
            auto look = [&]() {
                if (!f.by_hand(a) && copies_box)
                    page = (uint32_t)__ldg(a.c.page_table + (int64_t)f.s.b * a.c.max_pages +
                                           ((f.first() + mine * a.box_rows) >> a.c.page_shift));
            };
            bool more = f.next(a), again = false;
            if (more) look();
            int keys = 0, hand = 0;
            Ring<S::NS> put;
            uint32_t copied = 0, copied_phase = 0;   // bit i: slot i's last tile came by copies, and its phase
            for (; more;) {
                if (again && !mbar_wait(&sh.empty[put.slot], put.phase ^ 1, fail)) break;
                __syncwarp();
                if (!f.by_hand(a)) {
                    const bool held = !copies_box || page < (uint32_t)a.c.n_pages;
                    const bool hole = __any_sync(0xffffffffu, !held);
                    if (lane == 0) {
                        if (!f.value) sh.hole[keys & 15] = hole;
                        mbar_expect(&sh.full[put.slot], S::TILE);
                    }
                    __syncwarp();
                    if (lane > 0 && lane < NLOAD / 32) mbar_arrive(&sh.full[put.slot]);
                    if (copies_box) {
                        const uint32_t first = f.first() + mine * a.box_rows;
                        const int y = held ? (int)(((page * a.c.kv_heads + f.s.head) << a.c.page_shift) + (first & in_page))
                                           : a.c.n_pages * a.c.kv_heads << a.c.page_shift;   // past the end: zeros
                        tensor_copy(smem_u32(smem + S::RING) + put.slot * S::TILE + half * (TS * 128) + mine * a.box_rows * 128,
                                    f.value ? &map_v : &map_k, half * 64, y, &sh.full[put.slot]);
                    }
                    copied |= 1u << put.slot;
                    copied_phase = (copied_phase & ~(1u << put.slot)) | put.phase << put.slot;
                } else {
                    // at most NS tiles are under way, so the loading warps are never 16 behind
                    if (lane == 0) mbar_arrive(&sh.by_hand[hand & 15]);
                    ++hand;
                    copied &= ~(1u << put.slot);   // the place is free: its last copy has landed
                }
                keys += !f.value;
                ++put;
                again |= put.slot == 0;
                more = f.next(a);
                if (more) look();
            }
            // no copy may land after the block has gone
            for (int i = 0; i < S::NS; ++i)
                if (copied >> i & 1) {
                    const long long t0 = clock64();
                    while (!mbar_try_wait(&sh.full[i], copied_phase >> i & 1) && clock64() - t0 < kSpinCycles) {}
                }
        }
    } else if (warp >= 8) {
        // ---- loading
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<DP, E4M3>::LOAD));
        const int lt = tid - 256;
        const uint32_t ring = smem_u32(smem + S::RING);
        Ring<S::NS> put;                         // the tile to fill: free at first, then when it has been used
        bool again = false;
        auto wait_empty = [&]() { return !again || mbar_wait(&sh.empty[put.slot], put.phase ^ 1, fail); };
        auto advance = [&]() {
            ++put;
            again |= put.slot == 0;
        };
        Feed f(walk);
        if constexpr (!E4M3) {
            int keys = 0, hand = 0;
            constexpr int CPR = DP / 8, STEP = NLOAD / CPR;
            const int c = lt % CPR, r0 = lt / CPR;
            const uint32_t to = chunk_at(r0, c);
            const bool column = c * 8 < D;
            Share<STEP> x(a, r0, D * 2);
            const uint64_t stride = (uint64_t)x.page_bytes * a.c.kv_heads;
            while (f.next(a)) {
                if (!f.by_hand(a)) {
                    keys += !f.value;
                    advance();
                    continue;
                }
                x.look(a, f);
                const uint32_t first = f.first() + r0;
                const unsigned char *src = (const unsigned char *)(f.value ? a.c.v : a.c.k) + (uint64_t)f.s.head * x.page_bytes + c * 16;
                // with tensor copies their warp says when a place is free: only it follows every round of
                // the ring
                if (!(a.box_rows ? mbar_wait(&sh.by_hand[hand & 15], (uint32_t)hand >> 4 & 1, fail) : wait_empty())) break;
                ++hand;
                if (!f.value) {
                    bool hole = false;
#pragma unroll
                    for (int q = 0; q < x.ITER; ++q) hole |= !x.held(q);
                    if (hole) sh.hole[keys & 15] = 1;
                }
                if (!a.box_rows && lt == 0 && !f.value) sh.hole[(keys + 8) & 15] = 0;   // at most NS tiles are under way
                keys += !f.value;
                if (!f.draft()) {
                    const uint32_t dst = ring + put.slot * S::TILE + to;
#pragma unroll
                    for (int q = 0; q < x.ITER; ++q)
                        cp_async16(dst + q * STEP * 128, x.at(src, stride, first, q), x.held(q) && column);
                    cp_commit();
                    cp_wait<0>();
                } else {
                    unsigned char *dst = smem + S::RING + put.slot * S::TILE + to;
                    uint4 v[x.ITER];
#pragma unroll
                    for (int q = 0; q < x.ITER; ++q) {
                        v[q] = make_uint4(0, 0, 0, 0);
                        if (x.held(q) && column) v[q] = __ldg(reinterpret_cast<const uint4 *>(x.at(src, stride, first, q)));
                    }
#pragma unroll
                    for (int q = 0; q < x.ITER; ++q) {
                        if (first + q * STEP >= (uint32_t)f.s.slots && zero_odd<M>(v[q])) sh.odd[f.seg & 7] = f.seg + 1;
                        *reinterpret_cast<uint4 *>(dst + q * STEP * 128) = v[q];
                    }
                }
                proxy_fence();
                warp_arrive(&sh.full[put.slot]);
                advance();
            }
        } else {
            // a thread converts one 16-byte chunk of every STEP-th row
            constexpr int RPR = DP / 16, STEP = NLOAD / RPR, ITER = TS / STEP;
            const int c = lt % RPR, r0 = lt / RPR;
            const uint32_t to0 = chunk_at(r0, 2 * c), to1 = chunk_at(r0, 2 * c + 1);
            const bool column = c * 16 < D;
            Ring<S::NR> from;
            while (f.next(a)) {
                if (!mbar_wait(&sh.raw_full[from.slot], from.phase, fail)) break;
                const unsigned char *raw = smem + S::RAWS + from.slot * S::RAW + (r0 * D + c * 16);
                uint4 w[ITER];
#pragma unroll
                for (int q = 0; q < ITER; ++q) {
                    const int r = r0 + q * STEP;
                    const bool there = column && (sh.raw_rows[from.slot][r >> 5] >> (r & 31) & 1);
                    w[q] = there ? *reinterpret_cast<const uint4 *>(raw + q * STEP * D) : make_uint4(0, 0, 0, 0);
                }
                if (!wait_empty()) break;
                unsigned char *dst = smem + S::RING + put.slot * S::TILE;
                // drafted values that are not finite are left out
                const uint32_t odd_from = f.draft() ? (uint32_t)f.s.slots - f.first() : 0xffffffffu;
#pragma unroll
                for (int q = 0; q < ITER; ++q) {
                    uint4 lo = make_uint4(fa_e4m3x2_to_half2(w[q].x), fa_e4m3x2_to_half2(w[q].x >> 16),
                                          fa_e4m3x2_to_half2(w[q].y), fa_e4m3x2_to_half2(w[q].y >> 16));
                    uint4 hi = make_uint4(fa_e4m3x2_to_half2(w[q].z), fa_e4m3x2_to_half2(w[q].z >> 16),
                                          fa_e4m3x2_to_half2(w[q].w), fa_e4m3x2_to_half2(w[q].w >> 16));
                    if (odd_from != 0xffffffffu && r0 + q * STEP >= (int)odd_from) {
                        const bool o1 = zero_odd<M>(lo), o2 = zero_odd<M>(hi);
                        if (o1 || o2) sh.odd[f.seg & 7] = f.seg + 1;
                    }
                    *reinterpret_cast<uint4 *>(dst + to0 + q * STEP * 128) = lo;
                    *reinterpret_cast<uint4 *>(dst + to1 + q * STEP * 128) = hi;
                }
                warp_arrive(&sh.raw_empty[from.slot]);
                proxy_fence();
                warp_arrive(&sh.full[put.slot]);
                ++from;
                advance();
            }
        }
    } else {
        // ---- softmax: stream st, row r of its tile
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Regs<DP, E4M3>::SOFTMAX));
        const int st = warp >> 2, r = tid & 127;
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + lane_base + st * TS, to = tmem + lane_base + 256 + st * DP;
        int ns = 0, npv = 0, seg = 0, keys = 0;   // keys: key tiles of both streams before the segment's
        float *given = reinterpret_cast<float *>(smem + S::Q + S::TILE);   // stream 1's statistics, where its Q was
        while (walk.next(a, s)) {
            const int step = s.two() ? 1 : 2, begin = s.two() ? 0 : st, mine = s.two() ? s.n : (s.n + 1 - st) / 2;
            const int sg = seg++;
            const int keys_before = keys;
            keys += s.n;
            if (mine <= 0) continue;                       // a single tile: stream 1 has none
            // Up to 64 (32) rows lie two (four) times in the 128 lanes: copy `copy` weighs its part of
            // a tile's columns and gives the others no weight, and the copies are joined at the end.
            const int copies = s.rows <= 32 ? 4 : s.rows <= 64 ? 2 : 1, pad = TS / copies;
            const int copy = r / pad, w_begin = copy * (4 / copies), w_end = w_begin + 4 / copies;
            const int row = (s.two() ? st * TS : 0) + r - copy * pad;   // of the row block
            const bool live = row < s.rows;
            const bool warp_live = row - lane < s.rows;    // the same for the whole warp
            const int rr = 256 * s.block + row, ti = live ? rr / a.group : 0;
            const int hq = s.head * a.group + (live ? rr - ti * a.group : 0);
            const bool used = live && ti < s.use;
            float c = a.scale * kLog2e;
            if (warp_live) {
                // The warp's rows of Q into the stream's tile, DP / 8 lanes to a row of 16-byte chunks.
                // (This and the result run once a unit, from a cold instruction cache: short loops.)
                constexpr int LPR = DP / 8, RPI = 32 / LPR;       // lanes per row, rows per step
                unsigned char *dst = smem + S::Q + st * S::TILE;
                const int ch = lane % LPR, sub = lane / LPR, w0 = 32 * (warp & 3);
                const long long mine_at = s.b * a.qb + ti * a.qt + hq * a.qh;
                const int rows_here = min(s.rows - (row - lane), 32);
#pragma unroll 1
                for (int of = sub; of - sub < rows_here; of += RPI) {
                    const long long at = __shfl_sync(0xffffffffu, mine_at, of & 31);
                    const bool there = of < rows_here && ch < D / 8;
                    cp_async16(smem_u32(dst) + chunk_at(w0 + of, ch), (const T *)a.q + (there ? at + ch * 8 : 0), there);
                }
                cp_commit();
                cp_wait<0>();
                if (E4M3) {
                    __syncwarp();
                    uint32_t top = 0;                             // the row's largest magnitude, as bits of T
#pragma unroll 1
                    for (int ch2 = 0; ch2 < LPR; ++ch2) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(dst + chunk_at(r, ch2));
                        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) top = max(top, max(x[j] & 0x7fffu, x[j] >> 16 & 0x7fffu));
                    }
                    const float big = fa_to_f32(bits_as<T>((uint16_t)top));
                    // the largest element of the row to [2^8, 2^9)
                    const int e = big > 0.0f && big < INFINITY ? max(min(fa_exponent(big) - 8, 120), -120) : 0;
                    const float pow = pow2(-e);
#pragma unroll 1
                    for (int ch2 = 0; ch2 < LPR; ++ch2) {
                        uint4 *v = reinterpret_cast<uint4 *>(dst + chunk_at(r, ch2));
                        float f[8];
                        fa_unpack(*v, f, T());
#pragma unroll
                        for (int j = 0; j < 8; ++j) f[j] *= pow;
                        *v = fa_pack(f, M());
                    }
                    c *= pow2(e);
                }
                proxy_fence();
            }
            warp_arrive(&sh.q_full[st]);
            float m = -INFINITY, l = 0.0f, bias = 0.0f;
            bool any_far = false;                          // a reference of the warp's is
            float ev = E4M3 ? kLeastScale : 0.0f;          // a whole number
            // the scales of slot r of each tile are fetched one tile ahead, its page's number two
            float ks = 0.0f, vs = 0.0f;
            const Rows rows(a, s);
            auto page_of = [&](int tile) {
                const uint32_t slot = (uint32_t)(s.t0 + tile) * TS + r;
                return tile < s.n && slot < (uint32_t)s.end ? rows.page(slot) : 0xffffffffu;
            };
            auto fetch = [&](int tile, uint32_t page) {
                const int64_t at = rows.row(page, (uint32_t)(s.t0 + tile) * TS + r);
                ks = at >= 0 ? __ldg(a.c.k_scale + at) : 0.0f;
                vs = at >= 0 ? __ldg(a.c.v_scale + at) : 0.0f;
            };
            uint32_t next_page = 0;
            if (E4M3) {
                next_page = page_of(begin + step);
                fetch(begin, page_of(begin));
            }
            // with four copies a warp weighs the very slots whose scales it fetches
            auto scales_sync = [&]() {
                if (copies == 4) __syncwarp();
                else bar_sync(1 + st, TS);
            };
            for (int q = 0; q < mine; ++q) {
                const int tile = begin + q * step;
                const int first = (s.t0 + tile) * TS;
                if (E4M3) {
                    // (as bits: scales are not negative, and infinities and NaN are the largest)
                    const uint32_t vt = __reduce_max_sync(0xffffffffu, __float_as_uint(vs)), vl = __reduce_min_sync(0xffffffffu, __float_as_uint(vs));
                    if (q > 0) scales_sync();             // the previous tile's have been read
                    if (lane == 0) sh.vtop[st][warp & 3] = vt < 0x7f800000u && vt - vl <= kAlike ? lg2(__uint_as_float(vt)) : INFINITY;
                    if (first + r >= s.slots && !(fabsf(vs) < INFINITY)) { vs = 0.0f; sh.odd_scale[st] = sg + 1; }
                    sc.k[st][r] = ks;
                    sc.v[st][r] = vs;
                    if (q + 1 < mine) {
                        fetch(tile + step, next_page);
                        next_page = page_of(tile + 2 * step);
                    }
                    scales_sync();
                }
                mbar_wait(&sh.s_full[st], (uint32_t)ns++ & 1, fail);
                __syncwarp();
                tc_fence_after();
                float vmx = 0.0f;                          // log2 of the tile's largest value scale
                if (E4M3) {
                    vmx = -INFINITY;
                    for (int w = w_begin; w < w_end; ++w) vmx = fmaxf(vmx, sh.vtop[st][w]);
                }
                const bool whole = first + TS <= s.slots && !sh.hole[(keys_before + tile) & 15] && vmx < INFINITY;
                // The tile's scores to weights.  WHOLE: every row sees every slot, and the value scales are
                // alike; the code of the other tiles is kept apart so that the common one stays short.
                auto weigh = [&](auto whole_tag) {
                    constexpr bool WHOLE = decltype(whole_tag)::value;
                    float x[32];
                    // which of chunk w's slots the row sees
                    auto seen = [&](int w) {
                        if (WHOLE) return 0xffffffffu;
                        const uint32_t slot = first + 32 * w + lane;
                        const uint32_t held = __ballot_sync(0xffffffffu, slot < (uint32_t)s.end && rows.page(slot) < rows.n_pages);
                        return used ? held & seen_bits(a, s, ti, first + 32 * w) : 0u;
                    };
                    // chunk w of 32 scores, times the keys' scales (rounded, so that the largest less itself is
                    // zero), hidden ones to -inf
                    auto load_chunk = [&](int w, uint32_t z) {
                        if (!WHOLE) __syncwarp();
                        tmem_ld32(ts + 32 * w, x);
                        if (E4M3)
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const float4 f = *reinterpret_cast<const float4 *>(&sc.k[st][32 * w + e]);
                                x[e] = __fmul_rn(x[e], f.x);
                                x[e + 1] = __fmul_rn(x[e + 1], f.y);
                                x[e + 2] = __fmul_rn(x[e + 2], f.z);
                                x[e + 3] = __fmul_rn(x[e + 3], f.w);
                            }
                        if (!WHOLE)
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[e] = (z >> e & 1) ? x[e] : -INFINITY;
                    };
                    // the largest score (before the scale) that the row sees
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int w = w_begin; w < w_end; ++w) {
                        load_chunk(w, seen(w));
                        float top[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
#pragma unroll
                            for (int j = 0; j < 4; ++j) top[j] = fmaxf(fmaxf(top[j], x[e + 2 * j]), x[e + 2 * j + 1]);
                        mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                    }
                    // The reference moves where the largest score exceeds it by too much, or the largest product does:
                    // where scales are alike the largest score with the largest scale stands for it, else the
                    // products themselves.  (No score yet: m is -inf, and where there is still none the differences
                    // are not numbers.)
                    const float by_score = (mx - m) * c, m2 = fmaxf(m, mx);
                    const float now = (m - m2) * c + ev;  // the reference's product, less the largest score
                    float most = vmx + (mx - m2) * c;     // the tile's
                    if (E4M3 && !WHOLE) {
                        most = -INFINITY;
#pragma unroll 1
                        for (int w = w_begin; w < w_end; ++w) {
                            load_chunk(w, seen(w));
#pragma unroll
                            for (int e = 0; e < 32; ++e) most = fmaxf(most, fmaf(x[e] - m2, c, lg2(sc.v[st][32 * w + e])));
                        }
                    }
                    const bool move = live && (by_score > kGrow || (E4M3 && most > now + kProductGrow));
                    if (__any_sync(0xffffffffu, move)) {
                        float f = 1.0f;
                        if (move) {
                            const bool had = m > -INFINITY;
                            const float m0 = m, ev0 = ev;
                            m = m2;
                            if (E4M3) ev = scale_power(had ? fmaxf(now, most) : most);
                            const float up = ev - ev0;
                            const float b2 = m * c + ev - OFF;
                            // (m0 - m) c - up, exactly that of the weights' references
                            const float by = fmaxf(fabsf(bias), fabsf(b2)) > kFar ? (m0 - m) * c - up : bias - b2;
                            f = had ? ex2(by) : 0.0f;
                            bias = b2;
                            l *= E4M3 ? (had ? ex2(up + by) : 0.0f) : f;
                        }
                        any_far = __any_sync(0xffffffffu, fabsf(bias) > kFar);
                        if (q > 0) {
                            // (the previous tile's values were added before these scores were made)
#pragma unroll 1
                            for (int w = 0; w < DP / 32; ++w) {
                                float o[32];
                                tmem_ld32(to + 32 * w, o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] *= f;
                                tmem_st32(to + 32 * w, o);
                            }
                        }
                    }
                    const bool far = fabsf(bias) > kFar;
                    const float ref = far ? ev - OFF : bias;
                    float sum[4] = {0, 0, 0, 0};
#pragma unroll 1
                    for (int w = w_begin; w < w_end; ++w) {
                        uint32_t p[16];
                        if (copies < 4) load_chunk(w, seen(w));   // else the one chunk is still there
                        if (any_far)
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[e] = far ? x[e] - m : x[e];
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            float y[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                y[j] = ex2(fmaf(x[e + j], c, -ref));
                                sum[j] += y[j];
                            }
                            if (E4M3) {
                                const float4 g = *reinterpret_cast<const float4 *>(&sc.v[st][32 * w + e]);
                                y[0] *= g.x; y[1] *= g.y; y[2] *= g.z; y[3] *= g.w;
                            }
                            p[e / 2] = fa_pack2(y[0], y[1], M());
                            p[e / 2 + 1] = fa_pack2(y[2], y[3], M());
                        }
                        tmem_st16(ts + 16 * w, p);
                    }
                    if (copies > 1) {
                        const uint32_t none[16] = {};
#pragma unroll 1
                        for (int w = 0; w < 4; ++w)
                            if (w < w_begin || w >= w_end) tmem_st16(ts + 16 * w, none);
                    }
                    l += ((sum[0] + sum[1]) + (sum[2] + sum[3])) * pow2(ev);
                    tmem_st_wait();
                };
                if (warp_live) {
                    if (whole) weigh(std::true_type());
                    else weigh(std::false_type());
                }
                tc_fence_before();
                warp_arrive(&sh.p_full[st]);
            }
            // ---- the segment's result: the sum of the weights is l 2^bias, that of values o pow2(ev) 2^bias
            bias -= ev;
            mbar_wait(&sh.pv_done[st], (uint32_t)npv++ & 1, fail);
            __syncwarp();
            tc_fence_after();
            // (after the streams' barrier where both had tiles of the segment)
            auto any_odd = [&]() {
                return sh.odd[sg & 7] == sg + 1 || sh.odd_scale[0] == sg + 1 || sh.odd_scale[1] == sg + 1;
            };
            const bool pair_up = !s.two() && s.n > 1, join = pair_up && copies == 1, partial = s.n < s.nt;
            // of the block's partial results, slot 1 is a unit's first part, slot 0 a later one
            const int64_t prow0 = ((int64_t)blockIdx.x * 2 + (s.t0 == 0 ? 1 : 0)) * 256;
            if (copies > 1) {
                // join the copies (of both streams) through shared memory, where the queries were
                const int streams = pair_up ? 2 : 1, threads = streams * TS, me = st * TS + r, parts = copies * streams;
                float *stats = reinterpret_cast<float *>(smem + S::Q);             // 2 threads floats, then the sums
                float *acc = stats + 512;
                // columns at a time: all of them when the rows are few
                const int room = S::TILE * streams / 4 - 512;
                const int cols = parts * s.rows * DP <= room ? DP : parts * s.rows * (DP / 2) <= room ? DP / 2 : DP / 4;
                auto sync = [&]() { bar_sync(pair_up ? 3 : 1, threads); };
                sync();                                            // all products with the queries are done
                stats[me] = bias;
                stats[threads + me] = l;
                sync();
                float top = -INFINITY, sum = 0.0f;
                for (int i = 0; i < parts; ++i) {
                    const int at = row + i * pad;
                    if (!(stats[threads + at] == 0.0f)) top = fmaxf(top, stats[at]);
                }
                for (int i = 0; i < parts; ++i) {
                    const int at = row + i * pad;
                    const float li = stats[threads + at];
                    if (!(li == 0.0f)) sum += li * ex2(stats[at] - top);
                }
                const float f = l == 0.0f || !used ? 0.0f : ex2(bias - top) * (pow2(ev) / sum);
                const bool odd = any_odd();
                const int groups = cols / 4, part = st * copies + copy;
#pragma unroll 1
                for (int col0 = 0; col0 < DP; col0 += cols) {
                    if (warp_live) {
#pragma unroll 1
                        for (int w = 0; w < cols; w += 16) {
                            float o[16];
                            __syncwarp();
                            tmem_ld16(to + col0 + w, o);
                            if (live)
#pragma unroll
                                for (int g = 0; g < 4; ++g)
                                    *reinterpret_cast<float4 *>(acc + (part * s.rows + row) * cols + (((w / 4 + g) ^ (row & 3)) << 2)) =
                                        f == 0.0f ? make_float4(0, 0, 0, 0)
                                                  : make_float4(o[4 * g] * f, o[4 * g + 1] * f, o[4 * g + 2] * f, o[4 * g + 3] * f);
                        }
                    }
                    sync();
                    for (int x = me; x < s.rows * groups; x += threads) {
                        const int q = x / groups, g = x - q * groups, col = col0 + 4 * g;
                        float4 y = make_float4(0, 0, 0, 0);
                        for (int i = 0; i < parts; ++i) {
                            const float4 z = *reinterpret_cast<const float4 *>(acc + (i * s.rows + q) * cols + ((g ^ (q & 3)) << 2));
                            y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
                        }
                        const int qr = 256 * s.block + q, t = qr / a.group;
                        if (odd && t < s.use) {
                            float o[4] = {y.x, y.y, y.z, y.w};
                            add_odd<E4M3, T, 4>(a, s, rows, t, col, o);
                            y = make_float4(o[0], o[1], o[2], o[3]);
                        }
                        if (partial) {
                            *reinterpret_cast<float4 *>(a.part_o + (prow0 + q) * DP + col) = y;
                        } else if (col < D) {
                            T *dst = (T *)a.out + (((int64_t)s.b * a.T + t) * a.heads + s.head * a.group + qr - t * a.group) * D + col;
                            *reinterpret_cast<uint2 *>(dst) = make_uint2(fa_pack2(y.x, y.y, T()), fa_pack2(y.z, y.w, T()));
                        }
                    }
                    if (col0 + cols < DP) sync();
                }
                if (st == 0 && copy == 0 && live) {
                    const float lse = used && sum != 0.0f ? top + log2f(sum) : -INFINITY;
                    if (partial) a.part_lse[prow0 + row] = lse;
                    else if (a.lse) a.lse[((int64_t)s.b * a.T + ti) * a.heads + hq] = lse * kLn2;
                }
                tc_fence_before();
                sync();
                continue;
            }
            float f0 = 0.0f, f1 = 0.0f;
            if (join) {
                if (st == 1) { given[r] = bias; given[TS + r] = l; given[2 * TS + r] = pow2(ev); tc_fence_before(); }
                bar_sync(3, 2 * TS);
                tc_fence_after();
                if (st == 0) {
                    const float b1 = given[r], l1 = given[TS + r];
                    const bool h0 = !(l == 0.0f), h1 = !(l1 == 0.0f);   // a stream that saw something (or NaN)
                    const float top = h0 && h1 ? fmaxf(bias, b1) : h1 ? b1 : bias;
                    f0 = h0 ? ex2(bias - top) : 0.0f;
                    f1 = h1 ? ex2(b1 - top) : 0.0f;
                    l = l * f0 + l1 * f1;
                    bias = top;
                    f0 *= pow2(ev) / l;
                    f1 *= given[2 * TS + r] / l;
                }
            } else {
                f0 = pow2(ev) / l;
            }
            if (st == 0 || s.two()) {
                const bool odd = any_odd();
                const int64_t orow = ((int64_t)s.b * a.T + ti) * a.heads + hq, prow = prow0 + row;
                if (warp_live) {
                    // Rows leave through shared memory (the stream's queries are done with), so that a
                    // row's stores are contiguous: the 16-bit result whole, fp32 parts in two halves.
                    constexpr int LPR = DP / 8, RPI = 32 / LPR;
                    unsigned char *stage = smem + S::Q + st * S::TILE;
                    const int w0 = 32 * (warp & 3), ch = lane % LPR, sub = lane / LPR;
                    const int rows_here = min(s.rows - (row - lane), 32);
                    const int per_turn = partial ? DP / 2 : DP;         // columns staged at a time
#pragma unroll 1
                    for (int turn = 0; turn < DP; turn += per_turn) {
#pragma unroll 1
                        for (int w = turn; w < turn + per_turn; w += 32) {
                            float o[32];
                            __syncwarp();
                            tmem_ld32(to + w, o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= f0;
                            if (join) {
                                float o1[32];
                                tmem_ld32(to + DP + w, o1);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] += o1[e] * f1;
                            }
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = used && l != 0.0f ? o[e] : 0.0f;
                            if (odd && used) add_odd<E4M3, T, 32>(a, s, rows, ti, w, o);
                            if (partial) {
#pragma unroll
                                for (int e = 0; e < 32; e += 4)
                                    *reinterpret_cast<float4 *>(stage + chunk_at(r, (w - turn + e) / 4)) =
                                        make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; e += 8) {
                                    const float f[8] = {o[e], o[e + 1], o[e + 2], o[e + 3], o[e + 4], o[e + 5], o[e + 6], o[e + 7]};
                                    *reinterpret_cast<uint4 *>(stage + chunk_at(r, (w + e) / 8)) = fa_pack(f, T());
                                }
                            }
                        }
                        __syncwarp();
#pragma unroll 4
                        for (int i = 0; i < LPR; ++i) {
                            const int of = i * RPI + sub;
                            const long long at = __shfl_sync(0xffffffffu, partial ? (long long)prow : (long long)orow, of);
                            const uint4 v = *reinterpret_cast<const uint4 *>(stage + chunk_at(w0 + of, ch));
                            if (of >= rows_here) continue;
                            if (partial) *reinterpret_cast<uint4 *>(a.part_o + at * DP + turn + ch * 4) = v;
                            else if (ch * 8 < D) *reinterpret_cast<uint4 *>((T *)a.out + at * D + ch * 8) = v;
                        }
                        __syncwarp();
                    }
                }
                if (live) {
                    const float lse = used && l != 0.0f ? bias + log2f(l) : -INFINITY;
                    if (partial) a.part_lse[prow] = lse;
                    else if (a.lse) a.lse[orow] = lse * kLn2;
                }
            }
            tc_fence_before();
            // stream 1 may go on: its accumulator and its mark have been read
            if (join || s.two()) bar_sync(3, 2 * TS);
            else bar_sync(1 + st, TS);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0) a.status[blockIdx.x] = sh.fail;
    if (warp == 16) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Joins the parts of units that were cut, in an order that depends on nothing but the lengths.  Block
// (unit, RB rows).  With RB = 8, 16 or 32 a warp adds up every eighth row, its lanes across the columns;
// the lanes make the weights of a row each.  With fewer rows 8 / RB warps share a row's parts, their
// lanes make the weights of a part each, and their sums are added up.
template <int DP, class T, int RB>
__global__ void __launch_bounds__(256) k_attend_join(AttendArgs a, int runs, int statuses) {
    constexpr int NE = DP / 32, SUBS = RB < 8 ? 8 / RB : 1, R = RB < 8 ? 1 : RB / 8;
    struct alignas(4 * NE) Vec { float x[NE]; };
    __shared__ Work work;
    __shared__ int before;
    plan(a, work);
    const int units = a.c.kv_heads * a.blocks;
    const int b = (int)(blockIdx.x / units), u = (int)(blockIdx.x % units);
    if (threadIdx.x == 0) {
        const int per = run_length(a);
        int g = work.cum[b / per];
        for (int i = b / per * per; i < b; ++i) g += places_of(a, i);
        before = g;
    }
    __syncthreads();
    const int nt = tiles_of(a, b), total = work.cum[RUNS] * units, g0 = before * units + u * (nt + a.unit_cost), g1 = g0 + nt - 1;
    runs = min(total, runs);
    // the runs that hold the unit's first and last tile
    const int c0 = (int)((((int64_t)g0 + 1) * runs - 1) / total), c1 = (int)((((int64_t)g1 + 1) * runs - 1) / total);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, head = u / a.blocks, block = u % a.blocks;
    const int rows = min(a.rows - 256 * block, 256), row0 = RB * blockIdx.y, D = a.c.head_dim, parts = c1 - c0 + 1;
    fa_wait_for_previous();                     // by every block: the next kernel waits for this one only
    if (row0 >= rows) return;
    bool failed = false;
    if (statuses)
        for (int c = c0; c <= c1; ++c) failed |= a.status[c] != 0;
    if (parts == 1 && !failed) return;
    // of a run's two partial results the second holds a unit's first part
    auto part = [&](int i, int row) { return ((int64_t)(c0 + i) * 2 + (i == 0 ? 1 : 0)) * a.part_rows + row; };
    auto add = [&](float w, int i, int row, float (&o)[NE]) {
        const Vec p = *reinterpret_cast<const Vec *>(a.part_o + part(i, row) * DP + lane * NE);
#pragma unroll
        for (int e = 0; e < NE; ++e) o[e] = fmaf(w, p.x[e], o[e]);
    };
    auto store = [&](int row, const float (&o)[NE], float inv) {
        const int rr = 256 * block + row, ti = rr / a.group;
        const int64_t at = (((int64_t)b * a.T + ti) * a.heads + head * a.group + rr - ti * a.group) * D + lane * NE;
        T y[NE];
#pragma unroll
        for (int e = 0; e < NE; ++e) y[e] = fa_from_f32<T>(failed ? NAN : o[e] * inv);
        if (lane * NE < D) memcpy((T *)a.out + at, y, sizeof y);
    };
    auto store_lse = [&](int row, float top, float l) {
        const int rr = 256 * block + row, ti = rr / a.group;
        if (a.lse)
            a.lse[((int64_t)b * a.T + ti) * a.heads + head * a.group + rr - ti * a.group] =
                failed ? NAN : l == 0.0f ? -INFINITY : (top + log2f(l)) * kLn2;
    };
    float top = -INFINITY, l = 0.0f, o[R][NE] = {};
    if (SUBS == 1) {
        const int mine = min(row0 + min(lane, RB - 1), rows - 1);
        for (int i = 0; i < parts; ++i) top = fmaxf(top, a.part_lse[part(i, mine)]);   // a NaN is met below
        if (parts > 1)
#pragma unroll 2
            for (int i = 0; i < parts; ++i) {
                const float x = a.part_lse[part(i, mine)], f = x == -INFINITY ? 0.0f : ex2(x - top);
                l += f;
#pragma unroll
                for (int r = 0; r < R; ++r)
                    add(__shfl_sync(0xffffffffu, f, warp + 8 * r), i, min(row0 + warp + 8 * r, rows - 1), o[r]);
            }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float w = __shfl_sync(0xffffffffu, inv, warp + 8 * r);
            if (row0 + warp + 8 * r < rows) store(row0 + warp + 8 * r, o[r], w);
        }
        if (warp == 0 && lane < RB && row0 + lane < rows) store_lse(mine, top, l);
    } else {
        __shared__ float sums[8][DP], totals[8];
        const int row = row0 + warp / SUBS, sub = warp % SUBS;
        if (row < rows) {
            for (int i = lane; i < parts; i += 32) top = fmaxf(top, a.part_lse[part(i, row)]);
#pragma unroll
            for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            if (parts > 1)
                for (int first = sub; first < parts; first += 32 * SUBS) {
                    const int mine = first + lane * SUBS, n = min(32, (parts - first + SUBS - 1) / SUBS);
                    const float x = mine < parts ? a.part_lse[part(mine, row)] : -INFINITY;
                    const float f = x == -INFINITY ? 0.0f : ex2(x - top);
#pragma unroll 8
                    for (int i = 0; i < n; ++i) {
                        const float w = __shfl_sync(0xffffffffu, f, i);
                        l += w;
                        add(w, first + i * SUBS, row, o[0]);
                    }
                }
        }
#pragma unroll
        for (int e = 0; e < NE; ++e) sums[warp][lane * NE + e] = o[0][e];
        if (lane == 0) totals[warp] = l;
        __syncthreads();
        if (sub || row >= rows) return;
#pragma unroll
        for (int i = 1; i < SUBS; ++i) {
            l += totals[warp + i];
#pragma unroll
            for (int e = 0; e < NE; ++e) o[0][e] += sums[warp + i][lane * NE + e];
        }
        store(row, o[0], l == 0.0f ? 0.0f : 1.0f / l);
        if (lane == 0) store_lse(row, top, l);
    }
}

// two partial results of up to 256 rows and a status for each block
size_t workspace_bytes(int head_dim) {
    const size_t dp = head_dim <= 64 ? 64 : 128;
    return (size_t)MAX_CTAS * 2 * 256 * (dp + 1) * sizeof(float) + MAX_CTAS * sizeof(int);
}

// Tensor maps of a 16-bit cache: rows of head_dim elements, boxes of up to 128 rows of one page by
// 64 columns, 128-byte swizzled.  False where the cache cannot have them (pages of fewer than the
// eight rows of a swizzle atom, more rows than a coordinate holds).
bool make_maps(const fa_kv_cache *c, int box_rows, CUtensorMap (&maps)[2]) {
    const fa_encode_t encode = fa_tensor_map_encoder();
    const int64_t rows = (int64_t)c->n_pages * c->kv_heads * c->page_size;
    if (!encode || box_rows < 8 || rows < 1 || rows > 2147483647) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)c->head_dim, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)c->head_dim * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, step[2] = {1, 1};
    for (int i = 0; i < 2; ++i)
        if (encode(&maps[i], CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, i ? c->v : c->k, dims, strides, box, step,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    return true;
}

template <int DP, class T> fa_status join(const AttendArgs &a, int runs, int statuses, cudaStream_t s) {
    const int64_t units = (int64_t)a.B * a.c.kv_heads * a.blocks;
    const int rows = std::min(a.rows, 256);
    // Few units are cut into many parts: as few rows a block as keep all blocks on the GPU at once.
    // Against 32 rows always: 2 x 98304 slots, 16 units of 64 rows 192 -> 181 us in all, 4 x 509 slots, 32
    // units of 4 rows 14 -> 12 us.
    int rb = 1;
    while (rb < 32 && units * ((rows + rb - 1) / rb) > 8 * MAX_CTAS) rb *= 2;
    const dim3 grid((unsigned)units, (unsigned)((rows + rb - 1) / rb));
    void (*const kernel)(AttendArgs, int, int) = rb == 1   ? k_attend_join<DP, T, 1>
                                                 : rb == 2 ? k_attend_join<DP, T, 2>
                                                 : rb == 4 ? k_attend_join<DP, T, 4>
                                                 : rb == 8 ? k_attend_join<DP, T, 8>
                                                 : rb == 16 ? k_attend_join<DP, T, 16>
                                                            : k_attend_join<DP, T, 32>;
    return fa_launch_second("tree attention join", kernel, grid, 256, 0, s, a, runs, statuses);
}

template <int DP, bool E4M3, class T, class M>
fa_status launch(AttendArgs a, const CUtensorMap (&maps)[2], cudaStream_t s) {
    constexpr size_t smem = smem_bytes<DP, E4M3>();
    static_assert(smem <= 232448, "shared memory of a block");
    int ctas = 0;
    cudaError_t e = block_count(&ctas);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_attend<DP, E4M3, T, M>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return fa_refuse("fa_tree_attention", cudaGetErrorString(e), FA_ERR_CUDA);
    a.inject = fa_take_injected_timeout();
    k_attend<DP, E4M3, T, M><<<ctas, NTHR, smem, s>>>(a, maps[0], maps[1]);
    fa_status st = fa_launch_check("tree attention");
    if (st != FA_OK) return st;
    return join<DP, T>(a, ctas, 1, s);
}

fa_status sizes(const char *fn, int32_t B, int32_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
    if (B < 0 || B > 65535 || T < 0 || T > FA_MAX_DRAFT) return fa_refuse(fn, "B or T out of range");
    if (kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads) return fa_refuse(fn, "q_heads must be a multiple of kv_heads");
    if ((int64_t)B * std::max(T, 1) * q_heads > 2147483647) return fa_refuse(fn, "B * T * q_heads out of range");
    if (head_dim < 16 || head_dim % 16) return fa_refuse(fn, "head_dim must be a multiple of 16");
    if (head_dim > 128) return fa_refuse(fn, "head_dim above 128", FA_ERR_UNSUPPORTED);
    return FA_OK;
}

}  // namespace

extern "C" fa_status fa_tree_attention_workspace_bytes(int32_t B, int32_t T, int32_t q_heads, int32_t kv_heads,
                                                       int32_t head_dim, size_t *bytes) {
    const char *fn = "fa_tree_attention_workspace_bytes";
    if (!bytes) return fa_refuse(fn, "NULL argument");
    fa_status st = sizes(fn, B, T, q_heads, kv_heads, head_dim);
    if (st != FA_OK) return st;
    *bytes = workspace_bytes(head_dim);
    return FA_OK;
}

extern "C" fa_status fa_tree_attention(const fa_kv_cache *cache, int32_t dtype, int32_t B, int32_t T, int32_t q_heads,
                                       const void *q, int64_t q_batch_stride, int64_t q_token_stride,
                                       int64_t q_head_stride, const int32_t *page_table, int32_t max_pages,
                                       const int32_t *length, const int32_t *count, const uint64_t *mask, float scale,
                                       void *out, float *lse, void *workspace, size_t ws_bytes, fa_stream stream) {
    const char *fn = "fa_tree_attention";
    AttendArgs a;
    fa_status st = fa_view_cache(fn, cache, page_table, max_pages, &a.c);
    if (st != FA_OK) return st;
    if ((st = sizes(fn, B, T, q_heads, cache->kv_heads, cache->head_dim)) != FA_OK) return st;
    if (dtype != FA_DTYPE_F16 && dtype != FA_DTYPE_BF16) return fa_refuse(fn, "q must be fp16 or bf16", FA_ERR_UNSUPPORTED);
    if (cache->format != FA_CACHE_E4M3 && cache->format != dtype)
        return fa_refuse(fn, "a 16-bit cache must have the type of q", FA_ERR_UNSUPPORTED);
    if (!(scale > 0.0f && scale < INFINITY)) return fa_refuse(fn, "scale must be positive and finite");
    const int64_t slots = (int64_t)max_pages << a.c.page_shift;
    if (slots > 2147483647LL - 4096) return fa_refuse(fn, "max_pages * page_size out of range");
    if ((int64_t)cache->n_pages * cache->kv_heads > 2147483647LL) return fa_refuse(fn, "n_pages * kv_heads out of range");
    if (B == 0 || T == 0) return FA_OK;
    if (!q || !out || !length) return fa_refuse(fn, "NULL buffer");
    if ((((uintptr_t)q | (uintptr_t)out) & 15) || ((q_batch_stride | q_token_stride | q_head_stride) & 7))
        return fa_refuse(fn, "q and out must be 16-byte aligned, with strides that are multiples of 8");
    const size_t need = workspace_bytes(cache->head_dim);
    if (ws_bytes < need || !workspace)
        return fa_refuse(fn, ("workspace needs " + std::to_string(need) + " bytes").c_str(), FA_ERR_WORKSPACE_TOO_SMALL);
    if ((uintptr_t)workspace & 255) return fa_refuse(fn, "workspace not 256-byte aligned");
    a.B = B; a.T = T; a.heads = q_heads; a.group = q_heads / cache->kv_heads; a.words = (T + 63) / 64;
    if ((int64_t)T * a.group > 1 << 24) return fa_refuse(fn, "T * group out of range");
    a.rows = T * a.group;
    a.blocks = (a.rows + 255) / 256;
    const int least = a.rows <= FA_FEW_ROWS ? 16 : TS;   // slots of the smallest tile
    if ((int64_t)B * cache->kv_heads * a.blocks * ((slots + least - 1) / least + 5) > 2147483647)
        return fa_refuse(fn, "B * kv_heads * row blocks * tiles out of range");
    a.q = q; a.qb = q_batch_stride; a.qt = q_token_stride; a.qh = q_head_stride;
    a.length = length; a.count = count; a.mask = mask; a.scale = scale; a.out = out; a.lse = lse;
    const size_t dp = cache->head_dim <= 64 ? 64 : 128;
    a.part_o = (float *)workspace;
    a.part_lse = a.part_o + (size_t)MAX_CTAS * 2 * 256 * dp;
    a.status = (int *)(a.part_lse + (size_t)MAX_CTAS * 2 * 256);
    cudaStream_t s = (cudaStream_t)stream;
    const bool f16 = dtype == FA_DTYPE_F16, e4m3 = cache->format == FA_CACHE_E4M3;
    if (a.rows <= FA_FEW_ROWS) {
        // Few rows leave most of a 128-row tile empty; the kernel without shared tiles reads at the same
        // rate with less to start.  Measured, this kernel against that one: 8-bit cache, 32 x 8192 slots,
        // 4 / 16 rows 220 / 226 against 101 / 121 us; 1 x 65536 70 / 76 against 41 / 46; 4 x 509 19 / 22
        // against 12 / 15.  16-bit: 32 x 8192 165 / 170 against 176 / 181; 1 x 65536 58 / 65 against
        // 57 / 60; 4 x 509 16 / 20 against 12 / 15 (replayed in a graph).  Lengths are known on the device only, so
        // one rule serves them all: a 16-bit cache gains a quarter where calls are short and loses 6% where many
        // sequences are long.
        a.tile_shift = fa_attend_few_tile_shift(cache->head_dim, e4m3);
        a.unit_cost = 4;                         // 32 ragged sequences of up to 8192 slots: 1 / 2 / 4 / 7 give 74 / 64 / 63 / 64 us
        a.part_rows = FA_FEW_ROWS;
        int ctas = 0;
        const cudaError_t e = block_count(&ctas);
        if (e != cudaSuccess) return fa_refuse(fn, cudaGetErrorString(e), FA_ERR_CUDA);
        if ((st = fa_attend_few(a, cache->format, dtype, ctas, s)) != FA_OK) return st;
        const int runs = ctas * FA_FEW_WARPS;
        if (dp == 64) return f16 ? join<64, __half>(a, runs, 0, s) : join<64, __nv_bfloat16>(a, runs, 0, s);
        return f16 ? join<128, __half>(a, runs, 0, s) : join<128, __nv_bfloat16>(a, runs, 0, s);
    }
    a.tile_shift = 7;
    a.inject = 0;
    a.unit_cost = kUnitCost;
    a.part_rows = 256;
    CUtensorMap maps[2] = {};
    const int box_rows = std::min(cache->page_size, TS);
    a.box_rows = cache->format != FA_CACHE_E4M3 && make_maps(cache, box_rows, maps) ? box_rows : 0;
    if (cache->format == FA_CACHE_E4M3) {
        if (dp == 64) return f16 ? launch<64, true, __half, __half>(a, maps, s) : launch<64, true, __nv_bfloat16, __half>(a, maps, s);
        return f16 ? launch<128, true, __half, __half>(a, maps, s) : launch<128, true, __nv_bfloat16, __half>(a, maps, s);
    }
    if (dp == 64) return f16 ? launch<64, false, __half, __half>(a, maps, s) : launch<64, false, __nv_bfloat16, __nv_bfloat16>(a, maps, s);
    return f16 ? launch<128, false, __half, __half>(a, maps, s) : launch<128, false, __nv_bfloat16, __nv_bfloat16>(a, maps, s);
}
