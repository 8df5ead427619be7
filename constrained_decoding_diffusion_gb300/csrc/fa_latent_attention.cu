// Attention of drafted tokens over a paged latent cache (the absorbed form), on the 5th-generation tensor cores.
//
// The mathematics: with x_t = scale q . c_t, out = sum_t e^(x_t) c'_t / sum_t e^(x_t) in one pass over the slots, c' the
// latent part of c.  Every weight is taken relative to a reference m of the row, p_t = e^(x_t - m), with l = sum p_t and
// O = sum p_t c'_t; where a tile's largest score exceeds the reference's by more than 6 / log2(e) (a factor of 64), m moves
// and O and l are scaled.  Parts over disjoint slots join by their log-sum.
//
// The layout.  All heads of all drafted tokens are rows of one problem, 64 to a block, so a slot is read once for 64
// rows and serves as key and as value.  The accumulator of 64 rows by 512 columns takes half of tensor
// memory only if it is transposed, with a full 128 lanes of columns: O^T = C'^T P^T, C' read from the very
// tile that was the key of S = Q C^T, as the MN-major left operand.  (Untransposed, 128 rows would take all of tensor memory
// and leave no room for S, and 64 rows would leave half the lanes idle.)  S is not transposed, so that a row's maximum and
// sum lie in four lanes of a warp.  A tile is 64 slots: two of them, the queries and the weights fill shared memory.
//
// The work is the list of all tiles of all (sequence, row block) units; one block per SM takes an equal run of it.
// A unit that is cut leaves partial results, joined by a second small kernel in a fixed order.  (The list does not look
// at the mask: a tile of drafted slots is computed for row blocks that see none of it.)
//
// What bounds it, and what it measured (latent 512 + 64 bf16, replayed in a graph).  Up to 64 rows the slots' bytes: 32
// ragged sequences of up to 8192 slots x 32 rows 49 us, 157 MB read; in the loop a tile takes 2.1 us an SM (5.3 TB/s, 78% of
// a copy), about 15 us are start, results and join.  Two tiles are all that shared memory holds, so a place is
// refilled only when the tile before has been weighed and used: 1.2 us of products and softmax, 1.0 and up for the copy.
// Beyond that the tensor cores' shared memory: 16 sequences of 4096 slots x 1024 rows 212 us (147 GFLOP, 0.69 PFLOP/s), 2900
// clocks a tile of 64 slots x 64 rows, where the products themselves take 1200 (S: 64 rows are half of the instruction's
// rate) and 750 (O) and move 245 KB of operands at 128 bytes a clock, besides the 74 KB that come.  Latents of 256 + 32:
// 2 x 98304 slots x 256 rows 70 us (55 GFLOP, 0.78 PFLOP/s).
// Tried and dropped: eight softmax warps of half a tile each (a barrier more; 4 to 13% slower), a tile's columns refilled as
// the values' product leaves them (the copies' issue takes 1.7 times as long), one three-dimensional copy a tile, scores
// issued in pieces between which the other product has its turn, the blocks of rows of a sequence side by side on neighbouring
// SMs, so that a slot is read from memory once, where the slots are more than 128 MiB (16 x 8192 slots x 128 rows equal, 256
// 131 -> 121, 512 232 -> 207, 1024 414 -> 398, but 2 to 4 us more in every other call with more than one block of rows).
//
// Roundings.  Both operands of the second product have one 16-bit type, so the weights take the cache's: bf16 (8 bits), or
// fp16 with 2^8 for the reference's weight, so that all down to 2^-22 of it keep 11 bits.  The sum of the weights is taken before
// that, in fp32.  Against 64 bits, 16 x 4096 slots in bf16: 0.0020 of the result, where its own rounding alone is 0.0017.
//
// Roles (14 warps): warps 0-3 softmax and results, warp 4 issues the MMAs, warp 5 the tensor copies of
// whole tiles before the draft, warps 6-13 load the queries and the tiles in which the draft lies or a sequence ends.
// Every wait is bounded (about a second).  A wait that runs out marks the block's status; the joining kernel then sets
// the rows the block had a part in to NaN.
#include "fa_latent.cuh"
#include "fa_tensor.cuh"

using namespace fa_attention;

namespace {

constexpr int TS = 64, RB = 64;              // slots of a tile, rows of a block
constexpr int NLOAD = 8 * 32, NTHR = 14 * 32;
constexpr int GROUP = 64 * 128;              // 64 rows of 64 columns, 128-byte swizzled
// What a unit costs besides its tiles, in tiles: its queries, its tiles by hand (whose masks are looked up where several
// tokens are drafted) and its result.  Without it / 2 / 4 / 6 / 8: 32 ragged sequences of up to 8192 slots x 32 rows
// 52.8 / 48.8 / 48.8 / 50.4 / 50.3 us, 16 ragged ones of up to 4096 x 1024 rows of 32 tokens 273 / 201 / 142 / 133 / 130.
constexpr int kUnitCost = 4, kDraftCost = 3;

// QR: rows that the queries' and the weights' places hold, 64 or, for problems of no more, 16 (S reads on past them, into what
// lies behind, for rows that nobody looks at).  With 16 there is room for a third tile of 512 columns: 32 ragged sequences of
// up to 8192 slots x 16 rows 47.2 -> 40.5 us.  (Tiles of 32 slots, five of them: 45.6, and 47.1 against 48.3 for 32 rows: an
// instruction of 32 columns takes 26 clocks, one of 64 takes 33.)
template <int L, int QR> struct Shape {
    // A tile's latent columns lie in one of NS places, its key part (padded to 64 columns), which only the scores need,
    // in one of NK.  A single place is filled while the next tile's scores over the latent columns are computed, and has
    // barriers of its own.
    static constexpr int G = L / 64 + 1, TILE = (G - 1) * GROUP;
    static constexpr int NS = L == 128 ? 6 : L == 256 ? 4 : L == 384 || QR == 16 ? 3 : 2, NK = L < 384 ? NS : 1;
    static constexpr int QG = QR * 128, Q = 0, RING = G * QG, KEYS = RING + NS * TILE, P = KEYS + NK * GROUP, MISC = P + 2 * QG;
};

struct Misc {
    uint64_t full[6], empty[6], s_full[2], by_hand[8], p_full[2], pv_done[2], keys_full, keys_used, q_full, q_free, o_free, done;
    uint32_t there[6][2];              // per place of the ring: slots that a page holds
    uint8_t odd[6][8];                 // (by hand) bit k of byte w: slot w + 8 k, which loading warp w brought, holds an element that is not finite
    alignas(16) float factor[2][RB];   // read four at a time
    alignas(16) float inverse[2][RB];
    uint32_t tmem;
    int fail;
};

template <int L, int QR> constexpr size_t smem_bytes() { return Shape<L, QR>::MISC + sizeof(Misc) + sizeof(Work); }

// where chunk c (16 bytes = 8 elements) of row r lies in 128-byte-swizzled groups of 64 columns, each `group` bytes long
__device__ __forceinline__ uint32_t chunk_at(int r, int c, int group = GROUP) {
    return (uint32_t)((c >> 3) * group + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
// a tile that the loading warps bring: the draft or a sequence's end lies in it
__device__ __forceinline__ bool by_hand(const AttendArgs &a, const Segment &s, int tile) {
    return !a.box_rows || (s.t0 + tile + 1) * TS > s.slots;
}
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// 16 lanes by 64 columns: r[4 j + e] is row lane / 4 + 8 (e / 2), column 8 j + 2 (lane % 4) + e % 2
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, float (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
          "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
          "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr)
        : "memory");
}
// whether any of the four softmax warps says so; what they wrote to shared memory before is seen after
__device__ __forceinline__ bool any_warp(bool x) {
    uint32_t y;
    __syncwarp();
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
        : "=r"(y)
        : "r"((uint32_t)x)
        : "memory");
    return y != 0;
}

template <int L, class T, int QR>
__global__ void __launch_bounds__(NTHR, 1) k_latent(AttendArgs a, const __grid_constant__ CUtensorMap map) {
    using S = Shape<L, QR>;
    constexpr int G = S::G;
    extern __shared__ __align__(1024) unsigned char smem[];
    static_assert(S::MISC % 16 == 0 && alignof(Misc) == 16 && sizeof(Misc) % alignof(Work) == 0, "alignment of the parts");
    Misc &sh = *reinterpret_cast<Misc *>(smem + S::MISC);
    Work &work = *reinterpret_cast<Work *>(smem + S::MISC + sizeof(Misc));
    // (the warp's number by way of a shuffle: 2 x 98304 slots x 256 rows 83 -> 69 us)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    constexpr bool F16 = std::is_same<T, __half>::value;
    constexpr float OFF = F16 ? 8.0f : 0.0f;      // fp16 weights reach from 2^14 down to 2^-24, with 2^8 for the reference
    const int D = a.c.head_dim;
    volatile int *fail = &sh.fail;
    if (smem_u32(smem) & 1023) {                  // the swizzled tiles need it
        if (tid == 0) a.status[blockIdx.x] = 1;
        return;
    }
    if (tid == 0) {
        if (a.box_rows) asm volatile("prefetch.tensormap [%0];" ::"l"(&map) : "memory");
        for (int i = 0; i < S::NS; ++i) { mbar_init(&sh.full[i], NLOAD / 32); mbar_init(&sh.empty[i], 1); }
        for (int i = 0; i < 2; ++i) mbar_init(&sh.s_full[i], 1);
        for (int i = 0; i < 8; ++i) mbar_init(&sh.by_hand[i], 1);
        for (int i = 0; i < 2; ++i) { mbar_init(&sh.p_full[i], 4); mbar_init(&sh.pv_done[i], 1); }
        mbar_init(&sh.keys_full, NLOAD / 32);
        mbar_init(&sh.keys_used, 1);
        mbar_init(&sh.q_full, NLOAD / 32);
        mbar_init(&sh.q_free, 1);
        mbar_init(&sh.o_free, 4);
        mbar_init(&sh.done, 1);
        sh.fail = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 4) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    fa_let_next_start();
    plan(a, work);
    tc_fence_after();
    const uint32_t tmem = sh.tmem, ring = smem_u32(smem + S::RING), keys = smem_u32(smem + S::KEYS);
    Walk walk(a, work, blockIdx.x, gridDim.x);
    Segment s;

    if (warp == 4) {
        // ---- the MMAs: the warp runs as one
        constexpr uint32_t fmt = F16 ? 0u : 1u, idesc = (1u << 4) | (fmt << 7) | (fmt << 10);
        constexpr uint32_t idesc_s = idesc | (uint32_t)(RB >> 4) << 24 | (uint32_t)(TS >> 3) << 17;
        const uint64_t qd = umma_desc(smem_u32(smem + S::Q), 16), pd = umma_desc(smem_u32(smem + S::P), 16);
        Ring<S::NS> get, use;                     // the next tile's place for scores, and for values
        uint32_t ns = 0, np = 0, nseg = 0, tiles = 0;
        const int last_steps = (D - L) / 16;
        if (a.inject && blockIdx.x == 0) {        // a failure test: only this warp completes `done`, later
            const long long t0 = clock64();
            while (!mbar_try_wait(&sh.done, 0) && clock64() - t0 < kInjectCycles) {}
            *fail = 1;
            __syncwarp();
        }
        // (all steps in one piece of straight code: with a choice of pieces between which the other product has its turn, the
        // issue takes twice as long as the product)
        auto scores = [&]() {
            tc_fence_after();
            const uint64_t cd = umma_desc(ring + get.slot * S::TILE, 16), kd = umma_desc(keys + (S::NK == 1 ? 0 : get.slot) * GROUP, 16);
            const uint32_t d = tmem + 256 + (ns & 1) * TS;
#pragma unroll
            for (int k = 0; k < L / 16; ++k) {
                umma_ss_warp(d, qd + ((k >> 2) * S::QG + (k & 3) * 32) / 16, cd + ((k >> 2) * GROUP + (k & 3) * 32) / 16, idesc_s, k > 0);
            }
            if (S::NK < S::NS) {                           // (should the wait run out, what is there is as good as anything)
                mbar_wait(&sh.keys_full, tiles & 1, fail);
                __syncwarp();
                ++tiles;
                tc_fence_after();
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < last_steps) umma_ss_warp(d, qd + ((G - 1) * S::QG + k * 32) / 16, kd + k * 32 / 16, idesc_s, 1);
            umma_commit_warp(&sh.s_full[ns & 1]);
            if (S::NK < S::NS) umma_commit_warp(&sh.keys_used);
            ++ns;
            ++get;
        };
        bool ok = !__any_sync(0xffffffffu, *fail);
        while (ok && walk.next(a, s)) {
            if (!__all_sync(0xffffffffu, mbar_wait(&sh.q_full, nseg & 1, fail))) break;
            const int rows = min(a.rows - RB * s.block, RB);
            const uint32_t idesc_o = idesc | (uint32_t)(128 >> 4) << 24 | (uint32_t)((rows + 15) / 16 * 2) << 17 | 1u << 15;
            int issued = 0;
            for (int j = 0; j < s.n; ++j) {
                const long long t0 = clock64();
                while (true) {
                    // the next tile's scores as soon as it has come, these weights' product as soon as they are there
                    if (issued < s.n && issued <= j + 1 && __all_sync(0xffffffffu, mbar_test(&sh.full[get.slot], get.phase))) {
                        scores();
                        if (++issued == s.n) umma_commit_warp(&sh.q_free);
                    }
                    if (issued > j && __all_sync(0xffffffffu, mbar_test(&sh.p_full[np & 1], np >> 1 & 1))) break;
                    if (__any_sync(0xffffffffu, *fail || clock64() - t0 > kSpinCycles)) { *fail = 1; ok = false; break; }
                }
                if (!ok) break;
                const uint64_t pj = pd + (np & 1) * (S::QG / 16);
                if (j == 0 && nseg > 0 && !__all_sync(0xffffffffu, mbar_wait(&sh.o_free, (nseg - 1) & 1, fail))) { ok = false; break; }
                tc_fence_after();
                const uint64_t vd = umma_desc(ring + use.slot * S::TILE, GROUP);
#pragma unroll
                for (int c = 0; c < L / 128; ++c)
#pragma unroll
                    for (int k = 0; k < TS / 16; ++k)
                        umma_ss_warp(tmem + c * RB, vd + (2 * c * GROUP + k * 2048) / 16, pj + k * 32 / 16, idesc_o, j > 0 || k > 0);
                umma_commit_warp(&sh.empty[use.slot]);
                umma_commit_warp(&sh.pv_done[np & 1]);
                ++np;
                ++use;
            }
            ++nseg;
        }
        // every MMA issued has completed before tensor memory is released
        umma_commit_warp(&sh.done);
        const long long t0 = clock64();
        while (!mbar_try_wait(&sh.done, 0))
            if (clock64() - t0 > kSpinCycles) { *fail = 1; break; }
        __syncwarp();
    } else if (warp == 5) {
        // ---- tensor copies: a lane per box of (a page's rows) x 64 columns
        const int box = a.box_rows ? a.box_rows : TS, boxes = TS / box, mine = lane % boxes;
        const uint32_t in_page = (1u << a.c.page_shift) - 1;
        Ring<S::NS> put;
        bool again = false, ok = true;
        bool keys_copied = false;
        uint32_t keys_phase = 0;
        uint32_t hand = 0, tile = 0, copied = 0, copied_phase = 0;   // bit i: place i's last tile came by copies, and its phase
        while (ok && walk.next(a, s)) {
            const int32_t *pages = a.c.page_table + (int64_t)s.b * a.c.max_pages;
            for (int j = 0; j < s.n; ++j) {
                const bool hand_tile = by_hand(a, s, j);
                const uint32_t first = (uint32_t)(s.t0 + j) * TS + mine * box;
                uint32_t page = 0;
                if (!hand_tile) page = (uint32_t)__ldg(pages + (first >> a.c.page_shift));
                if (again && !__all_sync(0xffffffffu, mbar_wait(&sh.empty[put.slot], put.phase ^ 1, fail))) { ok = false; break; }
                if (!hand_tile) {
                    const bool held = page < (uint32_t)a.c.n_pages;
                    const uint32_t all = __ballot_sync(0xffffffffu, held);
                    if (lane == 0) {
                        uint64_t there = ~0ull;
                        if (all != 0xffffffffu)
                            for (int i = 0; i < boxes; ++i)
                                if (!(all >> i & 1)) there &= ~((box == 64 ? ~0ull : (1ull << box) - 1) << (i * box));
                        sh.there[put.slot][0] = (uint32_t)there;
                        sh.there[put.slot][1] = (uint32_t)(there >> 32);
                        mbar_expect(&sh.full[put.slot], S::NK < S::NS ? S::TILE : S::TILE + GROUP);
                    }
                    __syncwarp();
                    if (lane > 0 && lane < NLOAD / 32) mbar_arrive(&sh.full[put.slot]);
                    const int y = held ? (int)((page << a.c.page_shift) + (first & in_page)) : a.c.n_pages << a.c.page_shift;   // past the end: zeros
                    const uint32_t dst = ring + put.slot * S::TILE, key = keys + (S::NK == 1 ? 0 : put.slot) * GROUP;
                    for (int i = 0; i < boxes; ++i) {
                        const int yi = __shfl_sync(0xffffffffu, y, i);
#pragma unroll
                        for (int g = 0; g < G - 1; ++g)
                            tensor_copy_warp(dst + g * GROUP + i * box * 128, &map, g * 64, yi, &sh.full[put.slot]);
                    }
                    // (should the wait run out the tile still comes whole, so that its copies can be waited for)
                    uint64_t *const bar = S::NK < S::NS ? &sh.keys_full : &sh.full[put.slot];
                    if (S::NK < S::NS) {
                        if (tile > 0) ok = __all_sync(0xffffffffu, mbar_wait(&sh.keys_used, (tile - 1) & 1, fail));
                        if (lane == 0) mbar_expect(bar, GROUP);
                        else if (lane < NLOAD / 32) mbar_arrive(bar);
                    }
                    __syncwarp();
                    for (int i = 0; i < boxes; ++i)
                        tensor_copy_warp(key + i * box * 128, &map, L, __shfl_sync(0xffffffffu, y, i), bar);
                    keys_copied = true;
                    keys_phase = tile & 1;
                    copied |= 1u << put.slot;
                    copied_phase = (copied_phase & ~(1u << put.slot)) | put.phase << put.slot;
                } else {
                    if (S::NK < S::NS && tile > 0 && !__all_sync(0xffffffffu, mbar_wait(&sh.keys_used, (tile - 1) & 1, fail))) { ok = false; break; }
                    // at most NS tiles are under way, so the loading warps are never 8 behind
                    if (lane == 0) mbar_arrive(&sh.by_hand[hand & 7]);
                    ++hand;
                    copied &= ~(1u << put.slot);           // the place is free: its last copy has landed
                    keys_copied = false;
                }
                ++put;
                ++tile;
                again |= put.slot == 0;
                if (!ok) break;
            }
        }
        // no copy may land after the block has gone
        for (int i = 0; i < S::NS; ++i)
            if (copied >> i & 1) {
                const long long t0 = clock64();
                while (!mbar_try_wait(&sh.full[i], copied_phase >> i & 1) && clock64() - t0 < kSpinCycles) {}
            }
        if (S::NK < S::NS && keys_copied) {
            const long long t0 = clock64();
            while (!mbar_try_wait(&sh.keys_full, keys_phase) && clock64() - t0 < kSpinCycles) {}
        }
    } else if (warp > 5) {
        // ---- queries, and tiles by hand
        // A warp has every eighth row, its lanes the row's chunks.
        const int lw = warp - 6;
        constexpr int CPR = G * 8, LANES = (CPR + 31) / 32, MINE = RB / 8;   // chunks of a row; a lane's; a warp's rows
        Ring<S::NS> put;
        uint32_t nseg = 0, hand = 0;
        bool ok = true;
        while (ok && walk.next(a, s)) {
            if (nseg > 0 && !__all_sync(0xffffffffu, mbar_wait(&sh.q_free, (nseg - 1) & 1, fail))) break;
            const int rows = min(a.rows - RB * s.block, RB);   // (what the others' places hold is of no account)
            const uint32_t q_at = smem_u32(smem + S::Q);
#pragma unroll 2
            for (int r = lw; r < rows; r += 8) {
                const int rr = RB * s.block + r, ti = rr / a.heads;
                const T *src = (const T *)a.q + s.b * a.qb + ti * a.qt + (rr - ti * a.heads) * a.qh;
#pragma unroll
                for (int i = 0; i < LANES; ++i) {
                    const int ch = lane + 32 * i;
                    if (ch < CPR) cp_async16(q_at + chunk_at(r, ch, S::QG), src + (ch * 8 < D ? ch * 8 : 0), ch * 8 < D);
                }
            }
            cp_commit();
            cp_wait<0>();
            proxy_fence();
            warp_arrive(&sh.q_full);
            ++nseg;
            const Rows at(a, s);
            for (int j = 0; j < s.n; ++j, ++put) {
                if (!by_hand(a, s, j)) continue;
                const uint32_t first = (uint32_t)(s.t0 + j) * TS;
                const bool draft = first + TS > (uint32_t)s.slots;
                int64_t row[MINE];
#pragma unroll
                for (int k = 0; k < MINE; ++k) {
                    const uint32_t t = first + lw + 8 * k;
                    row[k] = t < (uint32_t)s.end ? at.row(t) : -1;
                }
                if (!__all_sync(0xffffffffu, mbar_wait(&sh.by_hand[hand & 7], hand >> 3 & 1, fail))) { ok = false; break; }
                ++hand;
                // where a row's chunk goes: the latent columns' place, or the key part's
                const uint32_t dst = S::RING + put.slot * S::TILE, key = S::KEYS + (S::NK == 1 ? 0 : put.slot) * GROUP;
                auto place = [&](int r, int ch) { return ch < (G - 1) * 8 ? dst + chunk_at(r, ch) : key + chunk_at(r, ch - (G - 1) * 8); };
#pragma unroll
                for (int k = 0; k < MINE; ++k) {
                    const T *src = (const T *)a.c.k + (row[k] >= 0 ? row[k] * D : 0);
#pragma unroll
                    for (int i = 0; i < LANES; ++i) {
                        const int ch = lane + 32 * i;
                        const bool there = row[k] >= 0 && ch * 8 < D;
                        if (ch < CPR) cp_async16(smem_u32(smem) + place(lw + 8 * k, ch), src + (there ? ch * 8 : 0), there);
                    }
                }
                cp_commit();
                if (lw == 0) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t t = first + 32 * h + lane;
                        const bool there = t < (uint32_t)s.end && at.page(t) < at.n_pages;
                        const uint32_t bits = __ballot_sync(0xffffffffu, there);
                        if (lane == 0) sh.there[put.slot][h] = bits;
                    }
                }
                cp_wait<0>();
                // drafted elements that are not finite are left out, and their slots marked
                uint32_t marks = 0;
                if (draft)
#pragma unroll 4
                    for (int k = 0; k < MINE; ++k) {
                        const int r = lw + 8 * k;
                        bool odd = false;
                        if (first + r >= (uint32_t)s.slots && first + r < (uint32_t)s.end)
#pragma unroll
                            for (int i = 0; i < LANES; ++i) {
                                const int ch = lane + 32 * i;
                                if (ch >= CPR) continue;
                                uint4 *v = reinterpret_cast<uint4 *>(smem + place(r, ch));
                                uint4 x = *v;
                                if (zero_odd<T>(x)) { *v = x; odd = true; }
                            }
                        marks |= (uint32_t)__any_sync(0xffffffffu, odd) << k;
                    }
                if (lane == 0) sh.odd[put.slot][lw] = (uint8_t)marks;
                proxy_fence();
                warp_arrive(&sh.full[put.slot]);
                if (S::NK < S::NS) warp_arrive(&sh.keys_full);
            }
        }
    } else {
        // ---- softmax: a thread has the rows r0 and r0 + 8, columns 8 i + 2 (lane % 4) and the next
        const int r0 = 16 * warp + (lane >> 2), col = 2 * (lane & 3);
        const uint32_t lanes = (uint32_t)(32 * warp) << 16, to = tmem + lanes;
        const float c = a.scale * kLog2e;
        unsigned char *const p_at = smem + S::P + r0 * 128 + (lane & 3) * 4;
        Ring<S::NS> get;
        uint32_t tiles = 0, nseg = 0;
        // tile t's product with the values is done (asked for no later than two tiles after)
        auto done = [&](uint32_t t) { mbar_wait(&sh.pv_done[t & 1], t >> 1 & 1, fail); };
        while (walk.next(a, s)) {
            const int rows = min(a.rows - RB * s.block, RB);
            int ti[2];
            bool used[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int row = r0 + 8 * q;
                ti[q] = (RB * s.block + row) / a.heads;
                used[q] = row < rows && ti[q] < s.use;
            }
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
            for (int j = 0; j < s.n; ++j) {
                const int first = (s.t0 + j) * TS;
                mbar_wait(&sh.full[get.slot], get.phase, fail);            // (its marks)
                mbar_wait(&sh.s_full[tiles & 1], tiles >> 1 & 1, fail);
                __syncwarp();
                tc_fence_after();
                float x[32];
                tmem_ld_rows(to + 256 + (tiles & 1) * TS, x);
                const bool hand = by_hand(a, s, j);
                const uint32_t there0 = sh.there[get.slot][0], there1 = sh.there[get.slot][1];
                if (hand || (there0 & there1) != 0xffffffffu) {
                    uint32_t marks[2] = {0, 0};
                    if (hand)
                        for (int w = 0; w < 8; ++w)
                            if (const uint32_t bits = sh.odd[get.slot][w])
                                for (int k = 0; k < 8; ++k) marks[k >> 2] |= (bits >> k & 1) << (w + 8 * (k & 3));
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t see[2] = {0, 0};
                        if (used[q]) {
                            see[0] = there0 & seen_bits(a, s, ti[q], first);
                            see[1] = there1 & seen_bits(a, s, ti[q], first + 32);
                        }
                        const uint32_t odd[2] = {see[0] & marks[0], see[1] & marks[1]};
#pragma unroll
                        for (int i = 0; i < 8; ++i)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float &y = x[4 * i + 2 * q + e];
                                const int at = 8 * (i & 3) + col + e;
                                if (!(see[i >> 2] >> at & 1)) y = -INFINITY;
                                if (odd[i >> 2] >> at & 1) y = NAN;
                            }
                    }
                }
                float f[2];
                bool grow = false;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float top = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = fmaxf(top, fmaxf(x[4 * i + 2 * q], x[4 * i + 2 * q + 1]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    f[q] = 1.0f;
                    if (r0 + 8 * q < rows && (top - m[q]) * c > kGrow) {   // (not where both are -inf)
                        f[q] = ex2((m[q] - top) * c);
                        m[q] = top;
                        grow = true;
                    }
                    const float ref = m[q] == -INFINITY ? 0.0f : m[q];
                    l[q] *= f[q];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float &y = x[4 * i + 2 * q + e];
                            y = ex2(fmaf(y - ref, c, OFF));
                            l[q] += y;
                        }
                }
                bool scale_now = false;
                if (j > 0) {
                    if ((lane & 3) == 0) {
                        sh.factor[tiles & 1][r0] = f[0];
                        sh.factor[tiles & 1][r0 + 8] = f[1];
                    }
                    scale_now = any_warp(grow);
                    // the weights' place is free, and the accumulator, if it is to be scaled
                    if (scale_now) done(tiles - 1);
                    else if (j > 1) done(tiles - 2);
                    __syncwarp();
                    tc_fence_after();
                }
                if (scale_now) {
                    const float *by = sh.factor[tiles & 1];
#pragma unroll 1
                    for (int w = 0; w < L / 128 * RB; w += 32) {
                        if ((w & (RB - 1)) >= rows) continue;
                        float o[32];
                        tmem_ld32(to + w, o);
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float4 y = *reinterpret_cast<const float4 *>(by + (w & (RB - 1)) + i);
                            o[i] *= y.x; o[i + 1] *= y.y; o[i + 2] *= y.z; o[i + 3] *= y.w;
                        }
                        tmem_st32(to + w, o);
                    }
                    tmem_st_wait();
                }
                if (16 * warp < QR) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        unsigned char *at = p_at + (tiles & 1) * S::QG + ((i ^ (lane >> 2)) << 4);
                        *reinterpret_cast<uint32_t *>(at) = fa_pack2(x[4 * i], x[4 * i + 1], T());
                        *reinterpret_cast<uint32_t *>(at + 8 * 128) = fa_pack2(x[4 * i + 2], x[4 * i + 3], T());
                    }
                }
                proxy_fence();
                tc_fence_before();
                warp_arrive(&sh.p_full[tiles & 1]);
                ++tiles;
                ++get;
            }
            // ---- the result
            const bool partial = s.n < s.nt;
            const int64_t prow = ((int64_t)blockIdx.x * 2 + (s.t0 == 0 ? 1 : 0)) * RB, orow = (int64_t)s.b * a.T * a.heads + RB * s.block;
            float *inverse = sh.inverse[nseg & 1];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int row = r0 + 8 * q;
                l[q] += __shfl_xor_sync(0xffffffffu, l[q], 1);
                l[q] += __shfl_xor_sync(0xffffffffu, l[q], 2);
                if ((lane & 3) == 0) {
                    const bool some = used[q] && l[q] != 0.0f;
                    inverse[row] = some ? 1.0f / l[q] : 0.0f;
                    const float lse = some ? fmaf(m[q], c, log2f(l[q]) - OFF) : -INFINITY;
                    if (row < rows) {
                        if (partial) a.part_lse[prow + row] = lse;
                        else if (a.lse) a.lse[orow + row] = lse * kLn2;
                    }
                }
            }
            done(tiles - 1);
            bar_sync(1, 128);
            tc_fence_after();
            auto store = [&](auto *out) {
                typedef typename std::remove_pointer<decltype(out)>::type O;
#pragma unroll 1
                for (int w = 0; w < L / 128 * RB; w += 32) {
                    const int row = w & (RB - 1);
                    if (row >= rows) continue;
                    float o[32];
                    tmem_ld32(to + w, o);
                    O *dst = out + row * L + (w / RB) * 128;
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        if (row + i >= rows) break;
                        const float4 by = *reinterpret_cast<const float4 *>(inverse + row + i);
                        const float f[4] = {by.x, by.y, by.z, by.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (row + i + e < rows) dst[(i + e) * L] = fa_from_f32<O>(f[e] == 0.0f ? 0.0f : o[i + e] * f[e]);
                    }
                }
            };
            if (partial) store(a.part_o + prow * L + 32 * warp + lane);
            else store((T *)a.out + orow * L + 32 * warp + lane);
            tc_fence_before();
            warp_arrive(&sh.o_free);
            ++nseg;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0) a.status[blockIdx.x] = sh.fail;
    if (warp == 4) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// The rows of a unit whose tiles lie in the runs c0 to c1: 8 / N warps share a row's parts, their lanes across the columns, and their
// sums are added up.
template <int L, class T, int N> struct JoinMemory {
    float4 sums[8 / N > 1 ? 8 : 1][L / 128][32];
    float totals[8];
};
template <int L, class T, int N>
__device__ __forceinline__ void join_unit(const AttendArgs &a, int b, int block, int c0, int c1, int row, int rows, JoinMemory<L, T, N> &sh) {
    constexpr int SUBS = 8 / N, V = L / 128;               // vectors of four columns a lane
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), sub = warp % SUBS, parts = c1 - c0 + 1;
    bool failed = false;
    for (int c = c0; c <= c1; ++c) failed |= a.status[c] != 0;
    if (parts == 1 && !failed) return;
    // of a run's two partial results the second holds a unit's first part
    auto part = [&](int i) { return ((int64_t)(c0 + i) * 2 + (i == 0 ? 1 : 0)) * RB + row; };
    float top = -INFINITY, l = 0.0f;
    float4 o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (row < rows && parts > 1) {
        for (int i = lane; i < parts; i += 32) top = fmaxf(top, a.part_lse[part(i)]);   // a NaN is met below
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        for (int first = sub; first < parts; first += 32 * SUBS) {
            const int mine = first + lane * SUBS, n = min(32, (parts - first + SUBS - 1) / SUBS);
            const float x = mine < parts ? a.part_lse[part(mine)] : -INFINITY, f = x == -INFINITY ? 0.0f : ex2(x - top);
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
                const float w = __shfl_sync(0xffffffffu, f, i);
                const float4 *src = reinterpret_cast<const float4 *>(a.part_o + part(first + i * SUBS) * L) + lane;
                l += w;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float4 y = src[32 * v];
                    o[v].x = fmaf(w, y.x, o[v].x); o[v].y = fmaf(w, y.y, o[v].y);
                    o[v].z = fmaf(w, y.z, o[v].z); o[v].w = fmaf(w, y.w, o[v].w);
                }
            }
        }
    }
    if (SUBS > 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) sh.sums[warp][v][lane] = o[v];
        if (lane == 0) sh.totals[warp] = l;
        __syncthreads();
        if (sub) return;
#pragma unroll
        for (int i = 1; i < SUBS; ++i) {
            l += sh.totals[warp + i];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float4 y = sh.sums[warp + i][v][lane];
                o[v].x += y.x; o[v].y += y.y; o[v].z += y.z; o[v].w += y.w;
            }
        }
    }
    if (row >= rows) return;
    const float inv = failed ? NAN : l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t at = (int64_t)b * a.T * a.heads + RB * block + row;
#pragma unroll
    for (int v = 0; v < V; ++v)
        *reinterpret_cast<uint2 *>((T *)a.out + at * L + 128 * v + 4 * lane) =
            make_uint2(fa_pack2(o[v].x * inv, o[v].y * inv, T()), fa_pack2(o[v].z * inv, o[v].w * inv, T()));
    if (a.lse && lane == 0) a.lse[at] = failed ? NAN : l == 0.0f ? -INFINITY : (top + log2f(l)) * kLn2;
}

// Joins the parts of units that were cut, in an order that depends on nothing but the lengths.  Block (unit, N rows).
template <int L, class T, int N>
__global__ void __launch_bounds__(256) k_latent_join(AttendArgs a, int runs) {
    constexpr int SUBS = 8 / N;
    __shared__ Work work;
    __shared__ int before;
    __shared__ JoinMemory<L, T, N> sh;
    plan(a, work);
    const int b = (int)(blockIdx.x / a.blocks), block = (int)(blockIdx.x % a.blocks);
    if (threadIdx.x == 0) {
        const int per = run_length(a);
        int g = work.cum[b / per];
        for (int i = b / per * per; i < b; ++i) g += places_of(a, i);
        before = g;
    }
    __syncthreads();
    const int nt = tiles_of(a, b), total = work.cum[RUNS] * a.blocks, g0 = before * a.blocks + block * (nt + a.unit_cost), g1 = g0 + nt - 1;
    runs = min(total, runs);
    // the runs that hold the unit's first and last tile
    const int c0 = (int)((((int64_t)g0 + 1) * runs - 1) / total), c1 = (int)((((int64_t)g1 + 1) * runs - 1) / total);
    // (the warp's number by way of a shuffle, as above: 16 x 4096 slots x 1024 rows 215 -> 212 us)
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int rows = min(a.rows - RB * block, RB), row = N * blockIdx.y + warp / SUBS;
    fa_wait_for_previous();                                // by every block: the next kernel waits for this one only
    if (N * (int)blockIdx.y >= rows) return;
    join_unit<L, T, N>(a, b, block, c0, c1, row, rows, sh);
}

// The same of many sequences.  Every block makes the plan, so with a block a unit the work grows with the square of the sequences;
// the units that are cut are fewer than the runs, and here block x looks at run x: it joins the unit that the run begins in, if it is
// the first to, and looks after the whole units of a run that failed.  A block a unit / a run, B sequences of 64 slots x 16 rows:
// 256 23.0 / 21.3 us, 1024 43.6 / 38.6, 4096 245 / 130, 16384 2302 / 482, 65535 32746 / 1908, but 16 x 4096 slots x 1024
// rows (256 units) 213.8 / 216.2.
constexpr int kManySequences = 512;                        // (more than the runs)
template <int L, class T>
__global__ void __launch_bounds__(256) k_latent_join_many(AttendArgs a, int runs) {
    __shared__ Work work;
    __shared__ JoinMemory<L, T, 8> sh;
    plan(a, work);
    const int lane = threadIdx.x & 31, run = blockIdx.x, row = 8 * blockIdx.y + (threadIdx.x >> 5), total = work.cum[RUNS] * a.blocks;
    Walk walk(a, work, run, runs);
    runs = min(total, runs);
    fa_wait_for_previous();
    if (run >= runs) return;
    const int b = walk.b, block = walk.block, nt = tiles_of(a, b), g0 = run_start(total, run, runs) - walk.t0, g1 = g0 + nt - 1;
    const bool cut = walk.t0 > 0 && walk.t0 < nt;
    if (a.status[run] != 0) {
        Segment s;
        while (walk.next(a, s)) {
            if (s.n < s.nt || row >= min(a.rows - RB * s.block, RB)) continue;
            const int64_t at = (int64_t)s.b * a.T * a.heads + RB * s.block + row;
            for (int c = lane; c < L; c += 32) ((T *)a.out)[at * L + c] = fa_from_f32<T>(NAN);
            if (a.lse && lane == 0) a.lse[at] = NAN;
        }
    }
    const int c0 = (int)((((int64_t)g0 + 1) * runs - 1) / total), c1 = (int)((((int64_t)g1 + 1) * runs - 1) / total);
    const int rows = min(a.rows - RB * block, RB);
    if (cut && c0 == run - 1 && 8 * (int)blockIdx.y < rows) join_unit<L, T, 8>(a, b, block, c0, c1, row, rows, sh);
}

// two partial results of 64 rows and a status for each block
size_t workspace_bytes(int latent) { return (size_t)MAX_CTAS * 2 * RB * (latent + 1) * sizeof(float) + MAX_CTAS * sizeof(int); }

// The cache's tensor map: rows of its elements, boxes of one page's rows by 64 columns, 128-byte swizzled.  False where
// it cannot have one (pages of fewer than the eight rows of a swizzle atom).  (One box of three dimensions for a whole
// tile takes 3100 clocks to arrive, nine of two dimensions side by side 600 to 1500.)
bool make_map(const fa_latent_cache *c, int box_rows, CUtensorMap *map) {
    const fa_encode_t encode = fa_tensor_map_encoder();
    const int64_t rows = (int64_t)c->n_pages * c->page_size;
    if (!encode || box_rows < 8 || rows < 1) return false;
    const cuuint64_t dim = (cuuint64_t)(c->latent_dim + c->rope_dim), dims[2] = {dim, (cuuint64_t)rows}, strides[1] = {dim * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, step[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, c->rows, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int L, class T, int QR> fa_status launch(AttendArgs a, const CUtensorMap &map, cudaStream_t s) {
    constexpr size_t smem = smem_bytes<L, QR>();
    static_assert(smem <= 232448, "shared memory of a block");
    int ctas = 0;
    cudaError_t e = block_count(&ctas);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k_latent<L, T, QR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return fa_refuse("fa_latent_attention", cudaGetErrorString(e), FA_ERR_CUDA);
    a.inject = fa_take_injected_timeout();
    k_latent<L, T, QR><<<ctas, NTHR, smem, s>>>(a, map);
    fa_status st = fa_launch_check("latent attention");
    if (st != FA_OK) return st;
    const int64_t units = (int64_t)a.B * a.blocks;
    const int rows = std::min(a.rows, RB);
    // A block has 8 / n warps for each of its n rows: as few rows as keep all blocks on the GPU at once, but not more
    // warps than a row of an evenly cut list has parts.
    int n = 1;
    while (n < 8 && (units * ((rows + n - 1) / n) > 8 * MAX_CTAS || 8 / n > ctas / units)) n *= 2;
    if (a.B >= kManySequences)
        return fa_launch_second("latent attention join", k_latent_join_many<L, T>, dim3((unsigned)ctas, (unsigned)((rows + 7) / 8)), 256, 0, s, a, ctas);
    void (*const join)(AttendArgs, int) = n == 1 ? k_latent_join<L, T, 1> : n == 2 ? k_latent_join<L, T, 2> : n == 4 ? k_latent_join<L, T, 4> : k_latent_join<L, T, 8>;
    return fa_launch_second("latent attention join", join, dim3((unsigned)units, (unsigned)((rows + n - 1) / n)), 256, 0, s, a, ctas);
}

template <class T> fa_status launch(const AttendArgs &a, int latent, const CUtensorMap &map, cudaStream_t s) {
    if (latent == 128) return launch<128, T, RB>(a, map, s);
    if (latent == 256) return launch<256, T, RB>(a, map, s);
    if (latent == 384) return launch<384, T, RB>(a, map, s);
    return a.rows <= 16 ? launch<512, T, 16>(a, map, s) : launch<512, T, RB>(a, map, s);
}

fa_status sizes(const char *fn, int32_t B, int32_t T, int32_t heads) {
    if (B < 0 || B > 65535 || T < 0 || T > FA_MAX_DRAFT || heads < 1 || heads > 1024) return fa_refuse(fn, "B, T or heads out of range");
    if ((int64_t)B * std::max(T, 1) * heads > 2147483647) return fa_refuse(fn, "B * T * heads out of range");
    return FA_OK;
}

}  // namespace

extern "C" fa_status fa_latent_attention_workspace_bytes(int32_t B, int32_t T, int32_t heads, int32_t latent_dim,
                                                         int32_t rope_dim, size_t *bytes) {
    const char *fn = "fa_latent_attention_workspace_bytes";
    if (!bytes) return fa_refuse(fn, "NULL argument");
    fa_status st = sizes(fn, B, T, heads);
    if (st != FA_OK) return st;
    if (latent_dim < 128 || latent_dim > 512 || latent_dim % 128 || rope_dim < 16 || rope_dim > 64 || rope_dim % 16)
        return fa_refuse(fn, "latent_dim or rope_dim out of range");
    *bytes = workspace_bytes(latent_dim);
    return FA_OK;
}

extern "C" fa_status fa_latent_attention(const fa_latent_cache *cache, int32_t dtype, int32_t B, int32_t T, int32_t heads,
                                         const void *q, int64_t q_batch_stride, int64_t q_token_stride,
                                         int64_t q_head_stride, const int32_t *page_table, int32_t max_pages,
                                         const int32_t *length, const int32_t *count, const uint64_t *mask, float scale,
                                         void *out, float *lse, void *workspace, size_t ws_bytes, fa_stream stream) {
    const char *fn = "fa_latent_attention";
    AttendArgs a = {};
    fa_status st = fa_view_latent(fn, cache, page_table, max_pages, &a.c);
    if (st != FA_OK) return st;
    if ((st = sizes(fn, B, T, heads)) != FA_OK) return st;
    if (dtype != FA_DTYPE_F16 && dtype != FA_DTYPE_BF16) return fa_refuse(fn, "q must be fp16 or bf16", FA_ERR_UNSUPPORTED);
    if (cache->format != dtype) return fa_refuse(fn, "the cache must have the type of q", FA_ERR_UNSUPPORTED);
    if (!(scale > 0.0f && scale < INFINITY)) return fa_refuse(fn, "scale must be positive and finite");
    const int64_t slots = (int64_t)max_pages << a.c.page_shift;
    if (slots > 2147483647LL - 4096) return fa_refuse(fn, "max_pages * page_size out of range");
    a.rows = T * heads;
    a.blocks = (a.rows + RB - 1) / RB;
    if ((int64_t)B * a.blocks > 2147483647 || (int64_t)B * a.blocks * ((slots + TS - 1) / TS + 8) > 2147483647)
        return fa_refuse(fn, "B * row blocks * tiles out of range");
    if (B == 0 || T == 0) return FA_OK;
    if (!q || !out || !length) return fa_refuse(fn, "NULL buffer");
    if ((((uintptr_t)q | (uintptr_t)out) & 15) || ((q_batch_stride | q_token_stride | q_head_stride) & 7))
        return fa_refuse(fn, "q and out must be 16-byte aligned, with strides that are multiples of 8");
    const size_t need = workspace_bytes(cache->latent_dim);
    if (ws_bytes < need || !workspace)
        return fa_refuse(fn, ("workspace needs " + std::to_string(need) + " bytes").c_str(), FA_ERR_WORKSPACE_TOO_SMALL);
    if ((uintptr_t)workspace & 255) return fa_refuse(fn, "workspace not 256-byte aligned");
    a.B = B; a.T = T; a.heads = a.group = heads; a.words = (T + 63) / 64;
    a.q = q; a.qb = q_batch_stride; a.qt = q_token_stride; a.qh = q_head_stride;
    a.length = length; a.count = count; a.mask = mask; a.scale = scale; a.out = out; a.lse = lse;
    a.part_o = (float *)workspace;
    a.part_lse = a.part_o + (size_t)MAX_CTAS * 2 * RB * cache->latent_dim;
    a.status = (int *)(a.part_lse + (size_t)MAX_CTAS * 2 * RB);
    a.tile_shift = 6;
    a.unit_cost = kUnitCost + (T > 1 ? kDraftCost : 0);
    CUtensorMap map = {};
    const int box_rows = std::min(cache->page_size, TS);
    a.box_rows = make_map(cache, box_rows, &map) ? box_rows : 0;
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == FA_DTYPE_F16) return launch<__half>(a, cache->latent_dim, map, s);
    return launch<__nv_bfloat16>(a, cache->latent_dim, map, s);
}
