// latent_absorbed.cu -- attention over a block-paged cache of latent rows, with the key
// and value projections absorbed into the query and the output (sm_103a).
//
// A cached row holds a token's latent vector c (R columns) and its rotary key part r (64
// columns); every head shares it.  With the key projection folded into the query, head h
// of query token i computes
//     s_ij = scale * (q_i,h . [c_j ; r_j]),   out_i,h = sum_j softmax_j(s_ij) c_j
// so one row serves as key (R + 64 columns) and as value (its first R columns) of all heads.
//
// Bound.  A cached token costs 2 (R + 64) bytes once per 64 query rows, and 2 * 64 * (2R + 64)
// multiply-adds: at R = 512, 1152 bytes against 69,632 MACs, i.e. 49 cycles of one SM's
// share of the HBM bandwidth against 17 cycles of its tensor pipe at the full rate.  Up to
// 64 rows a token is HBM-bound if the MMAs stay near half rate and loads never pause.  (That counts
// operations.  Both operands come from shared memory: a 16-deep step of QK, M = N = 64, has 4 KB of them
// for 16 cycles of products, one of PV, M = 128, N = 64, 6 KB for 32.  Were they read at 128 bytes a
// cycle, which is not measured here, a tile's 36 and 16 steps would take 1,900 cycles, not 1,100.)
//
// Layout
//  * A work item is 64 query rows (row = token * heads + head) of one sequence; its units
//    are tiles of 64 cached tokens.  A persistent grid takes equal contiguous shares of the
//    flat unit list (pkv_split.cuh); items cut by a share boundary leave
//    parts that a second kernel joins (latent_merge.cuh).
//  * A tile arrives in two halves, one TMA box a block (32 tokens of a larger one) with all its
//    64-column chunks.  In shared memory every 8 tokens are [chunk][8 tokens][128 bytes], 128-byte
//    swizzled, whatever the block size: the 8-row groups of a tile are a constant distance apart,
//    which is what both operand descriptors need.
//  * S = Q K^T runs with the rows on M = 64 and the tile's tokens on N = 64, so a row's scores stay
//    in the four threads of a quad.  O^T += C^T P^T runs with the latent columns on M = 128 (R / 128 blocks),
//    the rows on N and the tokens on K: the tile is read transposed in place (A MN-major) and P
//    is the K-major B operand.  O^T of 64 rows then takes R / 2 TMEM columns; with the rows
//    on M it would take all 512 and leave none for S.
//  * QK of tile t+1 runs during the softmax of tile t; a tile's stage is free after its PV, half
//    by half.
//
// Measured, with the join: one token of 128 sequences of 500 to 2500 tokens, 64 heads, R = 512:
// 62 us, 3.9 TB/s of what has to be read; 1 to 4 tokens of 32 sequences at 128 heads 130 us.  Two
// tiles of 72 KiB are all that fits beside Q, and a stage is loading for about 5,000 of 8,400 cycles
// at one item a sequence (the rest are its two products and the weights between them): that, the
// 9,000 cycles before the first tile and the join are what is left to the floor of 36 us.
//  * Waits are bounded in time; no CTA waits on another CTA.
#include "attn_block.cuh"
#include "fp32x2.cuh"
#include "latent_absorbed.cuh"
#include "latent_merge.cuh"
#include "latent_walk.cuh"
#include "pkv_split.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace {

// A small batch is spread until a CTA has one tile: its time is that of the longest chain, and a
// second item's loads, products and output one behind the other cost more than a join (four
// requests of up to 100 tokens, 16 heads: 9.2 us; with two tiles at least 15.9).
constexpr int kMinTilesPerCta = 1;

// A row's reference maximum moves, and O^T is rescaled, only when a tile's maximum exceeds it by
// this much (log2 units).  bf16 weights and fp32 sums keep their relative precision up to 2^24
// and far from overflow, and a move is rare enough to be handled off the critical path.
constexpr float kAbsorbedSlack = 24.0f;

constexpr int kMaxStages = 4;

template <int R>
struct AbsorbedSmem {
    static constexpr int NCH = R / 64 + 1;                    // 64-column chunks of a row, rotary last
    static constexpr uint32_t GROUP = NCH * 1024;             // 8 tokens, all chunks
    static constexpr uint32_t HALF = kLatentTile / 16 * GROUP;
    static constexpr uint32_t STAGE = 2 * HALF;               // one tile
    static constexpr uint32_t Q_CH = kLatentRows * 128;       // 64 rows x 64 columns
    static constexpr uint32_t OFF_Q = 0;
    static constexpr uint32_t OFF_P = NCH * Q_CH;             // P: 64 rows x 64 tokens, bf16
    static constexpr uint32_t OFF_STAGES = OFF_P + kLatentRows * 128;
    static constexpr uint32_t MISC = 2048;
    static constexpr uint32_t LIMIT = 232448 - 1024 - MISC;
    static constexpr int NST = (LIMIT - OFF_STAGES) / STAGE > kMaxStages ? kMaxStages : (LIMIT - OFF_STAGES) / STAGE;
    static constexpr uint32_t OFF_MISC = OFF_STAGES + NST * STAGE;
    static constexpr uint32_t BYTES = OFF_MISC + MISC + 1024;
    static constexpr uint32_t COL_O = 128;                    // S: columns 0..63 and 64..127
    static_assert(NST >= 2, "two tiles in flight at least");
};

// Where a share begins: 64-row group grp of the sequence, unit `at` of the item.
struct AbsorbedStart {
    WalkStart seq;
    int grp, at;
};

struct AbsorbedMisc {
    uint64_t q_full, q_empty, o_free, qk_over, pv_over, group, rescaled;
    uint64_t pv_done, p_full[2];  // p_full: by half of the tile
    uint64_t s_full[2], s_free[2];
    uint64_t kv_full[kMaxStages], kv_empty[kMaxStages][2];
    uint32_t tmem_slot;
    int abort_flag;
    int64_t scan[8];
    AbsorbedStart start;
    int moved[2][4];  // by tile parity and softmax warp: a row's reference maximum moved
    float alpha[2][kLatentRows];
    float inv[kLatentRows];
};
static_assert(sizeof(AbsorbedMisc) <= 2048, "fits its place");

// What an item costs besides its tiles, in tiles: its units are kItemCost ones without work, then
// one a tile, so that a share of many short items has fewer tiles.  (Its output takes 4,000 to 6,000
// cycles, a tile 3,300 to 4,200.  With shares of equally many tiles the slowest CTA took 1.4 times
// another's time.)  Measured, us:
//                                                        R = 512              R = 256
//   cost                                             0    2    4    6     0    2    4    6
//   1 to 4 tokens of 32 sequences, 128 heads       172  143  130  134    98   80   74   68
//   one token of 128 sequences, 64 heads          65.3 61.3 62.1 63.6  38.1 35.6 35.2 35.4
//   one of 64, four of them long, 16 heads        56.9 51.1 50.9 52.4  36.4 31.3 30.4 30.9
constexpr int kItemCost = 4;

// Units of a sequence: 64-row groups x (64-token tiles and the item's cost).
struct AbsorbedUnits {
    int num_heads;
    __device__ __forceinline__ int64_t operator()(const SeqInfo &q) const {
        const int64_t groups = ((int64_t)q.q_len * num_heads + kLatentRows - 1) / kLatentRows;
        return groups * ((q.ctx + kLatentTile - 1) / kLatentTile + kItemCost);
    }
};

// The part of one item that lies in the CTA's share.
struct AbsorbedSegment {
    int64_t row0;        // the item's first query row (token * heads + head)
    int row_in_seq;      // the same, counted inside the sequence
    int rows;            // live rows, <= 64
    int kb, tiles;       // first tile of the segment, tiles in it
    bool whole;          // the segment is the whole item
};

// A warp's walk over the items of its CTA's share: steps from the start, which one thread found,
// without a division.  (The first pass through any code waits for its instructions: what every role
// runs before its first tile is kept short.)
struct ItemWalk {
    SeqWalk<AbsorbedUnits> w;
    int64_t left;  // units of the share from here on; 0 if there is no tile among them
    int grp, at;   // 64-row group of the sequence, unit of the item
    __device__ __forceinline__ ItemWalk(const AbsorbedStart &st, int64_t units) : left(units), grp(st.grp), at(st.at) {
        w.start(st.seq);
        if (at + left <= kItemCost) left = 0;
    }
    __device__ __forceinline__ AbsorbedSegment segment(int num_heads) const {
        AbsorbedSegment g;
        const int nk = (w.q.ctx + kLatentTile - 1) / kLatentTile;
        g.kb = max(0, at - kItemCost);
        g.tiles = (int)min64(nk, at + left - kItemCost) - g.kb;
        g.row_in_seq = grp * kLatentRows;
        g.row0 = (int64_t)w.q.q0 * num_heads + g.row_in_seq;
        g.rows = min(kLatentRows, w.q.q_len * num_heads - g.row_in_seq);
        g.whole = g.tiles == nk;
        return g;
    }
    // past the segment
    __device__ __forceinline__ void advance(const SeqBatch &sb, const AbsorbedUnits &u, const AbsorbedSegment &g) {
        left -= g.kb + g.tiles + kItemCost - at;
        at = 0;
        if (left <= kItemCost) left = 0;
        if (++grp * kLatentRows < w.q.q_len * u.num_heads || left == 0) return;
        grp = 0;
        w.seek(sb, u, w.pre + w.units);
    }
};

}  // namespace

template <int R>
__global__ void __launch_bounds__(kAbsorbedThreads, 1)
latent_absorbed_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap kv_map,
                       const AbsorbedArgs a) {
    using L = AbsorbedSmem<R>;
    constexpr int NCH = L::NCH, NST = L::NST;
    constexpr int MB = R / 128;  // M blocks of O^T
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = smem + L::OFF_Q, *sP = smem + L::OFF_P, *sKV = smem + L::OFF_STAGES;
    AbsorbedMisc &ms = *reinterpret_cast<AbsorbedMisc *>(smem + L::OFF_MISC);
    volatile int *abort_flag = &ms.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x;

    if (threadIdx.x == 0) {
        mbar_init(&ms.q_full, 1);
        mbar_init(&ms.q_empty, 1);
        mbar_init(&ms.pv_done, 1);
        mbar_init(&ms.o_free, 4);
        mbar_init(&ms.qk_over, 1);
        mbar_init(&ms.pv_over, 1);
        mbar_init(&ms.group, 4);
        mbar_init(&ms.rescaled, 4);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ms.s_full[i], 1);
            mbar_init(&ms.s_free[i], 4);  // one arrival per softmax warp
            mbar_init(&ms.p_full[i], 4);
        }
        for (int i = 0; i < NST; ++i) {
            mbar_init(&ms.kv_full[i], 2);  // the tile's halves
            for (int h = 0; h < 2; ++h) mbar_init(&ms.kv_empty[i][h], 1);
        }
        ms.abort_flag = 0;
        fence_barrier_init();
    }
    if (threadIdx.x == 32) {
        tma_prefetch_desc(&q_map);
        tma_prefetch_desc(&kv_map);
    }
    // Before the previous kernel's end is waited for: a CTA of this kernel has the SM's shared
    // memory, so no other holder of TMEM is there.
    if (warp == 1) tmem_alloc(&ms.tmem_slot, 512);
    pdl_wait();
    pdl_trigger();

    const SeqBatch sb{a.query_start_loc, a.context_lens, a.num_seqs, a.total_q,
                      (int64_t)a.max_blocks_per_seq << a.block_shift, a.err};
    const AbsorbedUnits units{a.num_heads};
    const auto sc = scan_batch<kAbsorbedThreads>(sb, ms.scan, c == 0, units);
    const int64_t T = sc.total[0];
    const int ge = split_ctas(T, a.grid, kMinTilesPerCta);
    const bool works = T > 0 && c < ge;
    const int64_t lo = works ? quotient(c * T, ge) : 0, hi = works ? quotient((c + 1) * T, ge) : 0;
    if (works && find_unit(sb, units, sc, 0, lo, &ms.start.seq)) {
        const int64_t n = (ms.start.seq.q.ctx + kLatentTile - 1) / kLatentTile + kItemCost;
        const int64_t o = lo - ms.start.seq.pre, grp = quotient(o, n);
        ms.start.grp = (int)grp;
        ms.start.at = (int)(o - grp * n);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ms.tmem_slot;
    if (warp >= 2 && warp < 6) {
        // The merge job of the boundary before this CTA's share: the item split there, when that
        // is its first split.
        if (threadIdx.x == 64) {
            LatentJob j{0, -1, -1, 0};
            if (works && c > 0) {
                const SeqInfo q = ms.start.seq.q;
                const int grp = ms.start.grp, nk = (q.ctx + kLatentTile - 1) / kLatentTile;
                const int kb = ms.start.at - kItemCost;
                const int64_t begin = lo - kb;  // the item's first tile
                if (kb > 0 && begin >= quotient((c - 1) * T, ge)) {
                    j.out_off = ((int64_t)q.q0 * a.num_heads + grp * kLatentRows) * R;
                    j.c0 = c - 1;
                    j.c1 = share_owner(begin + nk - 1, T, ge);
                    j.rows = min(kLatentRows, q.q_len * a.num_heads - grp * kLatentRows);
                }
            }
            if (c > 0) a.ws_jobs[c - 1] = j;
            if (c == a.grid - 1) {
                j.c0 = -1;
                a.ws_jobs[c] = j;
            }
        }
        __syncwarp();
        zero_dead_rows(sb, c, a.grid, a.out, (int64_t)a.num_heads * R, warp - 2, 4);
    }
    if (!works) {
        __syncwarp();
        if (warp == 1) tmem_dealloc(tmem, 512);
        return;
    }
    ItemWalk iw(ms.start, hi - lo);
    SeqWalk<AbsorbedUnits> &w = iw.w;
    if (warp != 0) w.ahead(sb);  // the producer is on the critical path

    if (warp == 0) {
        // ------------------------------ TMA producer ------------------------------
        const uint64_t once = l2_policy_evict_first(), again = l2_policy_evict_normal();
        uint32_t st = 0, ph = 0, fill = 0;  // ring slot and phase of the next tile; halves issued
        uint32_t qloads = 0;
        const int bshift = min(a.block_shift, 5);                      // log2 of a box's tokens
        const int per_half = kLatentTile / 2 >> bshift;                 // boxes of half a tile
        const int box_bytes = L::GROUP << (bshift - 3);
        const uint32_t kv0 = smem_u32(sKV);
        auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.wait_ns));
        };
        bool ok = true;
        while (iw.left > 0 && ok) {
            const AbsorbedSegment g = iw.segment(a.num_heads);
            // A sequence of one item is read once, and its tiles make room in L2 for the parts; those of
            // several are read by each.  (128 sequences of one: 69.3 -> 65.9 us; all of them once, where
            // up to eight items read a sequence: 175 -> 182.)
            const uint64_t policy = w.q.q_len * a.num_heads <= kLatentRows ? once : again;
            // A window of 32 boxes (blocks, or 32 tokens of a larger one), one a lane; the block ids of
            // the next window are loaded while the current one is issued.
            const int32_t *table = a.block_tables + (int64_t)w.s * a.max_blocks_per_seq;
            const int64_t tok0 = (int64_t)g.kb * kLatentTile;
            const int64_t tok1 = min64(w.q.ctx, tok0 + (int64_t)g.tiles * kLatentTile);
            const int nboxes = (int)((tok1 - tok0 + (1 << bshift) - 1) >> bshift);
            auto entry = [&](int i) -> int {
                return i + lane < nboxes ? table[(tok0 + ((int64_t)(i + lane) << bshift)) >> a.block_shift] : 0;
            };
            // looked at only when its window begins, so that nothing waits for the load before
            auto checked = [&](int id) -> int {
                if (id >= 0 && id < a.num_blocks) return id;
                flag_error(a.err, PKV_DEVERR_BLOCK_ID);
                return -1;  // an out-of-range box is filled with zeros
            };
            int bid = 0, next = entry(0);  // under way while Q is asked for
            if (lane == 0) {
                if (qloads > 0) ok = mbar_wait(&ms.q_empty, (qloads - 1) & 1, abort_flag, a.wait_ns);
                if (ok) {
                    mbar_arrive_expect_tx(&ms.q_full, NCH * L::Q_CH);
                    tma_load_3d(sQ, &q_map, &ms.q_full, 0, (int)g.row0, 0, once);
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            ++qloads;
            int i0 = 0;                                                  // next box
            int grp = (int)(tok0 & ((1 << a.block_shift) - 1)) >> 3;     // its 8-token group in its block
            for (int t = 0; t < g.tiles && ok; ++t) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if ((i0 & 31) == 0) {
                        const int raw = next;
                        next = entry(i0 + 32);
                        bid = checked(raw);
                    }
                    ok = wait_all(&ms.kv_empty[st][h], ph ^ 1);
                    if (!ok) break;
                    const int boxes = max(0, min(per_half, nboxes - i0));
                    mbar_arrive_expect_tx_warp(&ms.kv_full[st], boxes * box_bytes);
                    uint32_t dst = kv0 + st * L::STAGE + h * L::HALF;
#pragma unroll 1
                    for (int i = 0; i < boxes; ++i) {
                        const int id = __shfl_sync(0xffffffffu, bid, (i0 + i) & 31);
                        tma_load_5d_warp(dst, &kv_map, &ms.kv_full[st], 0, 0, 0, grp, id, policy);
                        dst += box_bytes;
                        if (a.block_shift > 5) grp ^= 4;  // the other 32 tokens of a 64-token block
                    }
                    i0 += per_half;
                    ++fill;
                }
                if (++st == NST) { st = 0; ph ^= 1; }
                w.ahead(sb);
            }
            iw.advance(sb, units, g);
        }
        if (lane == 0) {
            if (!ok) {
                flag_error(a.err, PKV_DEVERR_TIMEOUT);
                *abort_flag = 1;
                // a stage of which only one half was asked for: its phase ends with that half
                if (fill & 1) mbar_arrive(&ms.kv_full[fill / 2 % NST]);
            }
            // The copies land before this CTA ends, whoever else has given up waiting for them.
            const uint32_t issued = (fill + 1) / 2, pending = minu32(issued, NST);  // fill counts halves
            for (uint32_t k = issued - pending; k < issued; ++k)
                mbar_wait(&ms.kv_full[k % NST], (k / NST) & 1, nullptr);
            if (qloads > 0) mbar_wait(&ms.q_full, (qloads - 1) & 1, nullptr);
        }
    } else if (warp == 1) {
        // ------------------------------ QK issuer ------------------------------
        // The issuers are whole warps on uniform values of which one elected lane issues
        // (tcgen05.cuh).  QK and PV have a warp each: a tile that is late holds up no finished
        // one, and the tensor pipe takes from both.
        auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.wait_ns));
        };
        constexpr uint32_t IDESC_QK = umma_idesc_bf16(kLatentRows, kLatentTile, 0, 0);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t dq = umma_desc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t dk0 = umma_desc_sw128(smem_u32(sKV), 16, L::GROUP);
        uint32_t st = 0, ph = 0;  // ring slot of the next tile
        uint32_t gq = 0;          // tiles issued
        uint32_t seg_i = 0;
        bool ok = true;
        while (iw.left > 0 && ok) {
            const AbsorbedSegment g = iw.segment(a.num_heads);
            const int tiles = __shfl_sync(0xffffffffu, g.tiles, 0);
            ok = wait_all(&ms.q_full, seg_i & 1);
            for (int t = 0; t < tiles && ok; ++t) {
                // S has two places: the scores of two tiles before have been read
                if (gq >= 2 && !wait_all(&ms.s_free[gq & 1], ((gq >> 1) - 1) & 1)) { ok = false; break; }
                const uint32_t tS = tm + (gq & 1) * kLatentTile;
                if (!wait_all(&ms.kv_full[st], ph)) { ok = false; break; }
                tc_fence_after();
                const uint64_t dk = dk0 + st * (L::STAGE >> 4);
#pragma unroll
                for (int k = 0; k < NCH * 4; ++k)
                    umma_bf16_warp(tS, dq + (((k / 4) * L::Q_CH + (k % 4) * 32) >> 4),
                                   dk + (((k / 4) * 1024 + (k % 4) * 32) >> 4), IDESC_QK, k > 0);
                umma_commit_warp(&ms.s_full[gq & 1]);
                ++gq;
                if (++st == NST) { st = 0; ph ^= 1; }
            }
            umma_commit_warp(&ms.q_empty);
            iw.advance(sb, units, g);
            ++seg_i;
        }
        if (!ok) {
            if (lane == 0) flag_error(a.err, PKV_DEVERR_TIMEOUT);
            *abort_flag = 1;
        }
        umma_commit_warp(&ms.qk_over);  // every MMA is done before TMEM is released
        mbar_wait(&ms.qk_over, 0, nullptr);
        __syncwarp();
    } else if (warp == 6) {
        // ------------------------------ PV issuer ------------------------------
        auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.wait_ns));
        };
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t dv0 = umma_desc_sw128(smem_u32(sKV), 1024, L::GROUP);
        const uint64_t dp = umma_desc_sw128(smem_u32(sP), 16, 1024);
        uint32_t st = 0, gv = 0, seg_i = 0, moves = 0;
        bool ok = true;
        while (iw.left > 0 && ok) {
            const AbsorbedSegment g = iw.segment(a.num_heads);
            const int tiles = __shfl_sync(0xffffffffu, g.tiles, 0);
            const int n = __shfl_sync(0xffffffffu, (g.rows + 15) & ~15, 0);
            const uint32_t idesc_pv = umma_idesc_bf16(128, n, 1, 0);
            if (seg_i > 0) ok = wait_all(&ms.o_free, (seg_i - 1) & 1);
            for (int t = 0; t < tiles && ok; ++t) {
                // in the halves in which the weights come and the stage is given back
                const uint64_t dv = dv0 + st * (L::STAGE >> 4);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!wait_all(&ms.p_full[h], gv & 1)) { ok = false; break; }
                    if (h == 0) {
                        const volatile int *mv = ms.moved[gv & 1];
                        if (__any_sync(0xffffffffu, mv[0] | mv[1] | mv[2] | mv[3])) {
                            if (!wait_all(&ms.rescaled, moves & 1)) { ok = false; break; }
                            ++moves;
                        }
                    }
                    tc_fence_after();
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                        for (int ks = 2 * h; ks < 2 * h + 2; ++ks)
                            umma_bf16_warp(tm + L::COL_O + mb * kLatentRows, dv + ((mb * 2048 + ks * 2 * L::GROUP) >> 4),
                                           dp + ((ks * 32) >> 4), idesc_pv, t > 0 || ks > 0);
                    umma_commit_warp(&ms.kv_empty[st][h]);
                }
                if (!ok) break;
                umma_commit_warp(&ms.pv_done);
                ++gv;
                if (++st == NST) st = 0;
            }
            iw.advance(sb, units, g);
            ++seg_i;
        }
        if (!ok) {
            if (lane == 0) flag_error(a.err, PKV_DEVERR_TIMEOUT);
            *abort_flag = 1;
        }
        umma_commit_warp(&ms.pv_over);
        mbar_wait(&ms.pv_over, 0, nullptr);
        __syncwarp();
    } else {
        // ------------- softmax: M = 64 puts row 16 q + i on TMEM lane 32 q + i, i < 16 -------------
        const int quarter = warp & 3;  // the TMEM lanes this warp may access
        const int tid = threadIdx.x - 64;
        const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t tO = tl + L::COL_O;
        // S is read 16 lanes at a time over all 32 threads (tmem_ld_16x32): this thread has rows
        // ra and ra + 8, a quarter of the columns of each.
        const int ra = quarter * 16 + (lane >> 2);
        const int c0 = 2 * (lane & 3);
        const float sl2 = a.scale_log2;
        // where this lane's stmatrix rows go: rows 0..7 and 8..15 of the quarter, two 16-byte
        // chunks of P at a time
        const int pr = quarter * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
        const uint32_t p_row = smem_u32(sP) + pr * 128;
        uint32_t gt = 0;    // tiles seen
        uint32_t meets = 0; // meetings of the four warps
        bool ok = true;
        // Waits that the warp leaves together, so that its warp-wide TMEM accesses stay converged.
        auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.wait_ns));
        };
        // Meeting of the four warps (a barrier with a limit, unlike bar.sync).
        auto meet = [&]() -> bool {
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.group);
            return wait_all(&ms.group, meets++ & 1);
        };
        // O^T, after tile `tile`'s predecessors and before its own PV: every column (= row of the
        // item) times the factor by which its reference maximum moved in that tile.
        auto rescale_if_moved = [&](uint32_t tile, int ncols) -> bool {
            if (!wait_all(&ms.p_full[0], tile & 1)) return false;  // every warp's say about the tile
            const volatile int *mv = ms.moved[tile & 1];
            if (!__any_sync(0xffffffffu, mv[0] | mv[1] | mv[2] | mv[3])) return true;
            if (tile > 0 && !wait_all(&ms.pv_done, (tile - 1) & 1)) return false;
            tc_fence_after();
#pragma unroll 1
            for (int mb = 0; mb < MB; ++mb)
#pragma unroll 1
                for (int cb = 0; cb < ncols; cb += 32) {
                    uint32_t r[32];
                    tmem_ld32(tO + mb * kLatentRows + cb, r);
                    tmem_wait_ld();
                    reg_order32(r);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        r[j] = __float_as_uint(__uint_as_float(r[j]) * ms.alpha[tile & 1][cb + j]);
                    tmem_st32(tO + mb * kLatentRows + cb, r);
                }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.rescaled);
            return true;
        };
        while (iw.left > 0 && ok) {
            const AbsorbedSegment g = iw.segment(a.num_heads);
            const int ctx = w.q.ctx;
            const bool live[2] = {ra < g.rows, ra + 8 < g.rows};
            int lim[2];  // keys the rows may see; rows past the item mask nothing
#pragma unroll
            for (int k = 0; k < 2; ++k)
                lim[k] = !live[k] || !a.causal
                             ? ctx
                             : ctx - w.q.q_len + (g.row_in_seq + ra + 8 * k) / a.num_heads + 1;
            const int ncols = (g.rows + 31) & ~31;  // TMEM columns of O^T to visit
            float m_ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
            for (int t = 0; t < g.tiles; ++t, ++gt) {
                const int64_t key0 = (int64_t)(g.kb + t) * kLatentTile;
                if (t > 0 && !rescale_if_moved(gt - 1, ncols)) { ok = false; break; }  // its PV may wait for it
                if (!wait_all(&ms.s_full[gt & 1], (gt >> 1) & 1)) { ok = false; break; }
                tc_fence_after();
                uint32_t v[2][16];  // by half of the tile
                tmem_ld_16x32(tl + (gt & 1) * kLatentTile, v[0]);
                tmem_ld_16x32(tl + (gt & 1) * kLatentTile + 32, v[1]);
                tmem_wait_ld();
                reg_order16(v[0]);
                reg_order16(v[1]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.s_free[gt & 1]);
                const int vis0 = (int)min64(lim[0] - key0, kLatentTile), vis1 = (int)min64(lim[1] - key0, kLatentTile);
                if (!__all_sync(0xffffffffu, vis0 >= kLatentTile && vis1 >= kLatentTile)) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (8 * (j >> 2) + c0 + (j & 1) >= ((j & 2) ? vis1 : vis0))
                            v[j >> 4][j & 15] = __float_as_uint(-INFINITY);
                }
                bool up[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        mx = fmax3(mx, __uint_as_float(v[i >> 2][4 * (i & 3) + 2 * k]),
                                   __uint_as_float(v[i >> 2][4 * (i & 3) + 2 * k + 1]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * sl2;  // scale > 0 keeps the order
                    up[k] = live[k] && mx > m_ref[k] + kAbsorbedSlack;
                    const float alpha = up[k] ? fast_exp2(m_ref[k] - mx) : 1.f;
                    if (up[k]) {
                        l[k] *= alpha;
                        m_ref[k] = mx;
                    }
                    if ((lane & 3) == 0) ms.alpha[gt & 1][ra + 8 * k] = alpha;
                }
                const bool moved = __any_sync(0xffffffffu, (up[0] || up[1]) && t > 0);
                if (lane == 0) ms.moved[gt & 1][quarter] = moved;
                // The weights, half a tile at a time, so that PV of the first half runs under the
                // exponentials of the second.  The sum adds them as rounded, so a row that one key
                // dominates loses nothing to their rounding.
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t pk[8];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float base = m_ref[k] == -INFINITY ? 0.f : m_ref[k];
                        float s0 = 0.f, s1 = 0.f;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float e0 = fast_exp2(fmaf(__uint_as_float(v[h][4 * i + 2 * k]), sl2, -base));
                            const float e1 = fast_exp2(fmaf(__uint_as_float(v[h][4 * i + 2 * k + 1]), sl2, -base));
                            pk[2 * i + k] = pack_bf16x2(e0, e1);
                            s0 += bf16_lo(pk[2 * i + k]);
                            s1 += bf16_hi(pk[2 * i + k]);
                        }
                        l[k] += s0 + s1;
                    }
                    // P has one place: the last tile's PV comes first
                    if (h == 0 && gt > 0 && !wait_all(&ms.pv_done, (gt - 1) & 1)) { ok = false; break; }
#pragma unroll
                    for (int i = 0; i < 4; i += 2)  // 16-byte chunks i and i + 1 of the half's P rows
                        stmatrix_x4(p_row + (((4 * h + i + (lane >> 4)) ^ (pr & 7)) << 4), pk[2 * i], pk[2 * i + 1],
                                    pk[2 * i + 2], pk[2 * i + 3]);
                    if (h == 0 && key0 + kLatentTile > ctx) {
                        // Slots past the context may hold NaN, and 0 * NaN would reach O^T: their value
                        // columns are zeroed once the copy has landed.
                        const uint32_t st = gt % NST;
                        if (!wait_all(&ms.kv_full[st], (gt / NST) & 1)) { ok = false; break; }
                        const int r0 = (int)(ctx - key0), pieces = (kLatentTile - r0) * (R / 8);
                        for (int i = tid; i < pieces; i += 128) {
                            const int rr = r0 + i / (R / 8), x = i % (R / 8);
                            *reinterpret_cast<uint4 *>(sKV + st * L::STAGE + (rr >> 3) * L::GROUP + (x >> 3) * 1024 +
                                                       (rr & 7) * 128 + ((x & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    fence_async_smem();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ms.p_full[h]);
                }
                if (!ok) break;
            }
            if (!ok) break;
            if (!rescale_if_moved(gt - 1, ncols)) { ok = false; break; }
            // ---- epilogue: O / l of a whole item, or the part for the merge ----
            if (!wait_all(&ms.pv_done, (gt - 1) & 1)) { ok = false; break; }
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 2; ++k) {  // the four threads of a row hold its sum in parts
                l[k] += __shfl_xor_sync(0xffffffffu, l[k], 1);
                l[k] += __shfl_xor_sync(0xffffffffu, l[k], 2);
                if ((lane & 3) == 0) ms.inv[ra + 8 * k] = 1.f / l[k];
            }
            if (!meet()) { ok = false; break; }
            const int slot = g.whole ? 0 : latent_slot(c, g.kb == 0);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (!g.whole && live[k] && (lane & 3) == 0)
                    a.ws_ml[(int64_t)slot * kLatentRows + ra + 8 * k] = make_float2(m_ref[k], l[k]);
            const int odd = lane & 1;
#pragma unroll 1
            for (int mb = 0; mb < MB; ++mb)
#pragma unroll 1
                for (int cb = 0; cb < ncols; cb += 32) {
                    uint32_t r[32];
                    tmem_ld32(tO + mb * kLatentRows + cb, r);
                    tmem_wait_ld();
                    reg_order32(r);
                    const int col = mb * 128 + quarter * 32 + lane;  // this lane's latent column
                    if (g.whole) {
                        // lanes of a pair swap, so that the even one stores its two columns of row j
                        // and the odd one those of row j + 1, 4 bytes each
                        __nv_bfloat16 *o = a.out + (g.row0 + cb) * R + (col & ~1);
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            const float x0 = __uint_as_float(r[j]) * ms.inv[cb + j];
                            const float x1 = __uint_as_float(r[j + 1]) * ms.inv[cb + j + 1];
                            const float y = __shfl_xor_sync(0xffffffffu, odd ? x0 : x1, 1);
                            const uint32_t pair = odd ? pack_bf16x2(y, x1) : pack_bf16x2(x0, y);
                            if (cb + j + odd < g.rows)
                                *reinterpret_cast<uint32_t *>(o + (int64_t)(j + odd) * R) = pair;
                        }
                    } else {
                        float *o = a.ws_o + ((int64_t)slot * kLatentRows + cb) * R + col;
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (cb + j < g.rows) o[(int64_t)j * R] = __uint_as_float(r[j]);
                    }
                }
            tc_fence_before();
            if (lane == 0) mbar_arrive(&ms.o_free);
            // inv is written again only behind the next item's tiles, whose weights every warp's
            // arrival is part of
            iw.advance(sb, units, g);
        }
        if (!ok) {
            if (lane == 0) flag_error(a.err, PKV_DEVERR_TIMEOUT);
            *abort_flag = 1;
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

void plan_absorbed(int latent_dim, int sms, AbsorbedPlan *p) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    p->grid = sms;
    p->off_jobs = 0;
    p->off_ml = up(sizeof(LatentJob) * (size_t)p->grid);
    p->off_o = p->off_ml + up(2 * (size_t)p->grid * kLatentRows * sizeof(float2));
    p->ws_bytes = p->off_o + up(2 * (size_t)p->grid * kLatentRows * latent_dim * sizeof(float));
}

template <int R>
static cudaError_t launch_absorbed(const CUtensorMap &q_map, const CUtensorMap &kv_map, const AbsorbedArgs &a,
                                   cudaStream_t stream) {
    static SmemAllowance allowed;
    cudaError_t e = allow_dynamic_smem(latent_absorbed_kernel<R>, AbsorbedSmem<R>::BYTES, allowed);
    if (e != cudaSuccess) return e;
    e = launch_pdl(latent_absorbed_kernel<R>, dim3(a.grid), dim3(kAbsorbedThreads), AbsorbedSmem<R>::BYTES, stream,
                   q_map, kv_map, a);
    if (e != cudaSuccess) return e;
    return launch_latent_merge<R, kLatentRows, false>(a.ws_jobs, a.ws_ml, a.ws_o, a.out, R, a.grid, stream);
}

cudaError_t launch_latent_absorbed(int latent_dim, const CUtensorMap &q_map, const CUtensorMap &kv_map,
                                   const AbsorbedArgs &a, cudaStream_t stream) {
    return latent_dim == 512 ? launch_absorbed<512>(q_map, kv_map, a, stream)
                             : launch_absorbed<256>(q_map, kv_map, a, stream);
}

}  // namespace pkv
