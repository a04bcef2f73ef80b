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
// 64 rows a token is HBM-bound if the MMAs stay near half rate and loads never pause.
//
// Layout
//  * A work item is 64 query rows (row = token * heads + head) of one sequence; its units
//    are tiles of 64 cached tokens.  A persistent grid takes equal contiguous shares of the
//    flat unit list (pkv_split.cuh); items cut by a share boundary are merged by
//    log-sum-exp weights (merge.cuh).
//  * A tile arrives as eight TMA boxes of 8 tokens x all 64-column chunks, so any block
//    size that is a multiple of 8 works and eight requests move 72 KiB.  In shared memory
//    box b holds [chunk][8 tokens][128 bytes], 128-byte swizzled: the 8-row groups of a tile
//    are a constant distance apart, which is what both operand descriptors need.
//  * S = Q K^T runs with the rows on M = 64 and the tile's tokens on N = 64, so the softmax has
//    one row per thread.  O^T += C^T P^T runs with the latent columns on M = 128 (R / 128 blocks),
//    the rows on N and the tokens on K: the tile is read transposed in place (A MN-major) and P
//    is the K-major B operand.  O^T of 64 rows then takes R / 2 TMEM columns; with the rows
//    on M it would take all 512 and leave none for S.
//  * The MMA warp issues QK of tile t+1 before PV of tile t, so the tensor pipe works during
//    the softmax; a tile's stage is free after its PV.
//  * Waits are bounded in time; no CTA waits on another CTA.
#include "attn_block.cuh"
#include "latent_absorbed.cuh"
#include "latent_walk.cuh"
#include "pkv_split.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace {

constexpr int kMinTilesPerCta = 2;

template <int R>
struct AbsorbedSmem {
    static constexpr int NCH = R / 64 + 1;                    // 64-column chunks of a row, rotary last
    static constexpr uint32_t BOX = NCH * 1024;               // 8 tokens, all chunks
    static constexpr uint32_t STAGE = 8 * BOX;                // one tile
    static constexpr uint32_t Q_CH = kLatentRows * 128;       // 64 rows x 64 columns
    static constexpr uint32_t OFF_Q = 0;
    static constexpr uint32_t OFF_P = NCH * Q_CH;             // P: 64 rows x 64 tokens, bf16
    static constexpr uint32_t OFF_STAGES = OFF_P + kLatentRows * 128;
    static constexpr uint32_t MISC = 2048;
    static constexpr uint32_t LIMIT = 232448 - 1024 - MISC;
    static constexpr int NST = (LIMIT - OFF_STAGES) / STAGE > 4 ? 4 : (LIMIT - OFF_STAGES) / STAGE;
    static constexpr uint32_t OFF_MISC = OFF_STAGES + NST * STAGE;
    static constexpr uint32_t BYTES = OFF_MISC + MISC + 1024;
    static constexpr uint32_t COL_O = 128;                    // S: columns 0..63 and 64..127
    static_assert(NST >= 2, "two tiles in flight at least");
};

struct AbsorbedMisc {
    uint64_t q_full, q_empty, pv_done, p_full, o_free, mma_done, group;
    uint64_t s_full[2];
    uint64_t kv_full[4], kv_empty[4];
    uint32_t tmem_slot;
    int abort_flag;
    int64_t scan[8];
    int64_t start_pre;
    int start_seq;
    int flag[2][4];
    float alpha[2][kLatentRows];
    float inv[kLatentRows];
};
static_assert(sizeof(AbsorbedMisc) <= 2048, "fits its place");

// Units of a sequence: 64-row groups x 64-token tiles.
struct AbsorbedUnits {
    int num_heads;
    __device__ __forceinline__ int64_t operator()(const SeqInfo &q) const {
        const int64_t groups = ((int64_t)q.q_len * num_heads + kLatentRows - 1) / kLatentRows;
        return groups * ((q.ctx + kLatentTile - 1) / kLatentTile);
    }
};

// The part of one item that lies in the CTA's share.
struct AbsorbedSegment {
    int64_t item_begin;  // the item's first unit
    int64_t row0;        // its first query row (token * heads + head)
    int row_in_seq;      // the same, counted inside the sequence
    int rows;            // live rows, <= 64
    int kb, tiles;       // first tile of the segment, tiles in it
    bool whole;          // the segment is the whole item
};

__device__ __forceinline__ AbsorbedSegment segment_at(const AbsorbedArgs &a, const SeqInfo &q, int64_t pre,
                                                      int64_t f, int64_t hi) {
    AbsorbedSegment g;
    const int nk = (q.ctx + kLatentTile - 1) / kLatentTile;
    const int64_t o = f - pre;
    const int64_t grp = o / nk;
    g.kb = (int)(o - grp * nk);
    g.item_begin = f - g.kb;
    g.tiles = (int)min64(nk - g.kb, hi - f);
    g.row_in_seq = (int)(grp * kLatentRows);
    g.row0 = (int64_t)q.q0 * a.num_heads + g.row_in_seq;
    g.rows = (int)min64(kLatentRows, (int64_t)q.q_len * a.num_heads - g.row_in_seq);
    g.whole = g.kb == 0 && g.tiles == nk;
    return g;
}

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
        mbar_init(&ms.p_full, 4);  // one arrival per softmax warp
        mbar_init(&ms.o_free, 4);
        mbar_init(&ms.mma_done, 1);
        mbar_init(&ms.group, 4);
        for (int i = 0; i < 2; ++i) mbar_init(&ms.s_full[i], 1);
        for (int i = 0; i < NST; ++i) {
            mbar_init(&ms.kv_full[i], 1);
            mbar_init(&ms.kv_empty[i], 1);
        }
        ms.abort_flag = 0;
        fence_barrier_init();
    }
    if (threadIdx.x == 32) {
        tma_prefetch_desc(&q_map);
        tma_prefetch_desc(&kv_map);
    }
    pdl_wait();
    pdl_trigger();

    const SeqBatch sb{a.query_start_loc, a.context_lens, a.num_seqs, a.total_q,
                      (int64_t)a.max_blocks_per_seq << a.block_shift, a.err};
    const AbsorbedUnits units{a.num_heads};
    const BatchScan sc = scan_batch(sb, units, ms.scan, c == 0);
    const int64_t T = sc.total;
    const int ge = split_ctas(T, a.grid, kMinTilesPerCta);
    const bool works = T > 0 && c < ge;
    const int64_t lo = works ? share_begin(c, T, ge) : 0, hi = works ? share_begin(c + 1, T, ge) : 0;
    if (works) find_unit(sb, units, sc, lo, &ms.start_seq, &ms.start_pre);
    __syncthreads();

    // The merge job of the boundary before this CTA's share: the item split there, when that
    // is its first split.
    if (threadIdx.x == 0) {
        MergeJob j;
        no_job(j);
        if (works && c > 0) {
            const SeqInfo q = read_seq(sb, ms.start_seq, false);
            const int64_t nk = (q.ctx + kLatentTile - 1) / kLatentTile;
            const int64_t grp = (lo - ms.start_pre) / nk, begin = ms.start_pre + grp * nk;
            if (begin != lo && begin >= share_begin(c - 1, T, ge)) {
                j.item_begin = begin;
                j.total_units = T;
                j.out_row0 = (int64_t)q.q0 * a.num_heads + grp * kLatentRows;
                j.c0 = c - 1;
                j.c1 = share_owner(begin + nk - 1, T, ge);
                j.ge = ge;
                j.rows = (int)min64(kLatentRows, (int64_t)q.q_len * a.num_heads - grp * kLatentRows);
                j.rows_per_token = 1;
                j.head0 = 0;
            }
        }
        if (c > 0) a.ws_jobs[c - 1] = j;
        if (c == a.grid - 1) {
            no_job(j);
            a.ws_jobs[c] = j;
        }
    }
    zero_dead_rows(sb, c, a.grid, a.out, (int64_t)a.num_heads * R);
    if (!works) return;

    if (warp == 1) tmem_alloc(&ms.tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ms.tmem_slot;
    SeqWalk<AbsorbedUnits> w;
    w.start(sb, units, ms.start_seq, ms.start_pre);

    if (warp == 0) {
        // ------------------------------ TMA producer ------------------------------
        const uint64_t policy = l2_policy_evict_normal();
        uint32_t st = 0, ph = 0, fill = 0;  // ring slot and phase of the next tile; tiles issued
        uint32_t qloads = 0;
        bool ok = true;
        for (int64_t f = lo; f < hi && ok;) {
            w.seek(sb, units, f);
            const AbsorbedSegment g = segment_at(a, w.q, w.pre, f, hi);
            if (lane == 0) {
                if (qloads > 0) ok = mbar_wait(&ms.q_empty, (qloads - 1) & 1, abort_flag, a.wait_ns);
                if (ok) {
                    mbar_arrive_expect_tx(&ms.q_full, NCH * L::Q_CH);
#pragma unroll 1
                    for (int ch = 0; ch < NCH; ++ch)
                        tma_load_2d(sQ + ch * L::Q_CH, &q_map, &ms.q_full, ch * 64, (int)g.row0, policy);
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            ++qloads;
            // A window is 4 tiles = 32 groups of 8 tokens, one group a lane; the block ids of the
            // next window are loaded while the current one is issued.
            const int32_t *table = a.block_tables + (int64_t)w.s * a.max_blocks_per_seq;
            const int ctx = w.q.ctx;
            const int64_t first = (int64_t)g.kb * kLatentTile + 8 * lane;
            const int64_t last = min64(ctx, (int64_t)(g.kb + g.tiles) * kLatentTile);
            auto block_of = [&](int tile) -> int {
                const int64_t pos = first + (int64_t)tile * kLatentTile;
                if (pos >= last) return -1;
                const int id = table[pos >> a.block_shift];
                if (id >= 0 && id < a.num_blocks) return id;
                flag_error(a.err, PKV_DEVERR_BLOCK_ID);
                return -1;  // an out-of-range box is filled with zeros
            };
            const int in_block = (int)(first & ((1 << a.block_shift) - 1));  // a tile is a multiple of any block
            int bid = -1, bid_next = block_of(0);
            for (int t = 0; t < g.tiles; ++t) {
                if ((t & 3) == 0) {
                    bid = bid_next;
                    bid_next = block_of(t + 4);
                }
                const int64_t key0 = (int64_t)(g.kb + t) * kLatentTile;
                const int boxes = (int)min64(8, (ctx - key0 + 7) >> 3);
                if (lane == 0) {
                    ok = mbar_wait(&ms.kv_empty[st], ph ^ 1, abort_flag, a.wait_ns);
                    if (ok) mbar_arrive_expect_tx(&ms.kv_full[st], boxes * L::BOX);
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                if ((lane >> 3) == (t & 3) && (lane & 7) < boxes)
                    tma_load_4d(sKV + st * L::STAGE + (lane & 7) * L::BOX, &kv_map, &ms.kv_full[st], 0, in_block, 0,
                                bid, policy);
                ++fill;
                if (++st == NST) { st = 0; ph ^= 1; }
            }
            f += g.tiles;
        }
        if (!ok && lane == 0) {
            flag_error(a.err, PKV_DEVERR_TIMEOUT);
            *abort_flag = 1;
            // copies in flight land before the shared memory is given back
            const uint32_t pending = minu32(fill, NST);
            for (uint32_t k = fill - pending; k < fill; ++k) mbar_wait(&ms.kv_full[k % NST], (k / NST) & 1, nullptr);
            if (qloads > 0) mbar_wait(&ms.q_full, (qloads - 1) & 1, nullptr);
        }
    } else if (warp == 1) {
        // ------------------------------ MMA issuer ------------------------------
        // The whole warp runs on uniform values; one elected lane issues (tcgen05.cuh).
        auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.wait_ns));
        };
        constexpr uint32_t IDESC_QK = umma_idesc_bf16(kLatentRows, kLatentTile, 0, 0);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t dq = umma_desc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t dk0 = umma_desc_sw128(smem_u32(sKV), 16, L::BOX);
        const uint64_t dv0 = umma_desc_sw128(smem_u32(sKV), 1024, L::BOX);
        const uint64_t dp = umma_desc_sw128(smem_u32(sP), 16, 1024);
        uint32_t st = 0, ph = 0;   // ring slot of the next tile's QK
        uint32_t vst = 0;          // ring slot of the next tile's PV
        uint32_t gq = 0, gv = 0;   // tiles whose QK / PV has been issued
        uint32_t seg_i = 0;
        bool ok = true, issued = false;
        auto issue_qk = [&]() -> bool {
            if (!wait_all(&ms.kv_full[st], ph)) return false;
            tc_fence_after();
            const uint64_t dk = dk0 + st * (L::STAGE >> 4);
            const uint32_t tS = tm + (gq & 1) * kLatentTile;
#pragma unroll
            for (int ks = 0; ks < NCH * 4; ++ks)
                umma_bf16_warp(tS, dq + (((ks / 4) * L::Q_CH + (ks % 4) * 32) >> 4),
                               dk + (((ks / 4) * 1024 + (ks % 4) * 32) >> 4), IDESC_QK, ks > 0);
            umma_commit_warp(&ms.s_full[gq & 1]);
            issued = true;
            ++gq;
            if (++st == NST) { st = 0; ph ^= 1; }
            return true;
        };
        for (int64_t f = lo; f < hi && ok;) {
            w.seek(sb, units, f);
            const AbsorbedSegment g = segment_at(a, w.q, w.pre, f, hi);
            const int tiles = __shfl_sync(0xffffffffu, g.tiles, 0);
            const int n = __shfl_sync(0xffffffffu, (g.rows + 15) & ~15, 0);
            const uint32_t idesc_pv = umma_idesc_bf16(128, n, 1, 0);
            if (!wait_all(&ms.q_full, seg_i & 1) || !issue_qk()) { ok = false; break; }
            if (tiles == 1) umma_commit_warp(&ms.q_empty);
            for (int t = 0; t < tiles; ++t) {
                if (t + 1 < tiles) {
                    if (!issue_qk()) { ok = false; break; }
                    if (t + 2 == tiles) umma_commit_warp(&ms.q_empty);
                }
                if (t == 0 && seg_i > 0 && !wait_all(&ms.o_free, (seg_i - 1) & 1)) { ok = false; break; }
                if (!wait_all(&ms.p_full, gv & 1)) { ok = false; break; }
                tc_fence_after();
                const uint64_t dv = dv0 + vst * (L::STAGE >> 4);
#pragma unroll
                for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                    for (int ks = 0; ks < kLatentTile / 16; ++ks)
                        umma_bf16_warp(tm + L::COL_O + mb * kLatentRows, dv + ((mb * 2048 + ks * 2 * L::BOX) >> 4),
                                       dp + ((ks * 32) >> 4), idesc_pv, t > 0 || ks > 0);
                umma_commit_warp(&ms.kv_empty[vst]);
                umma_commit_warp(&ms.pv_done);
                ++gv;
                if (++vst == NST) vst = 0;
            }
            f += g.tiles;
            ++seg_i;
        }
        if (!ok) {
            if (lane == 0) flag_error(a.err, PKV_DEVERR_TIMEOUT);
            *abort_flag = 1;
        }
        if (issued) {  // every MMA is done before TMEM is released
            umma_commit_warp(&ms.mma_done);
            mbar_wait(&ms.mma_done, 0, nullptr);
        }
        __syncwarp();
    } else {
        // ------------- softmax: M = 64 puts row 16 q + i on TMEM lane 32 q + i -------------
        const int quarter = warp & 3;  // the TMEM lanes this warp may access
        const int tid = threadIdx.x - 64;
        const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t tO = tl + L::COL_O;
        const bool has_row = lane < 16;
        const int row = quarter * 16 + (lane & 15);
        const float sl2 = a.scale_log2;
        uint32_t gt = 0;    // tiles seen
        uint32_t meets = 0; // meetings of the four warps
        bool ok = true;
        // Waits that the warp leaves together, so that its warp-wide TMEM accesses stay converged.
        auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.wait_ns));
        };
        // Meeting of the four warps that also tells whether any thread brought `x` (a barrier
        // with a limit, unlike bar.sync).  Flags alternate: a warp writes meeting m + 2's only
        // after every warp reached m + 1, past its reads of m.
        auto meet = [&](bool x, bool &any) -> bool {
            const bool mine = __any_sync(0xffffffffu, x);
            int *fl = ms.flag[meets & 1];
            if (lane == 0) {
                fl[quarter] = mine;
                mbar_arrive(&ms.group);
            }
            if (!wait_all(&ms.group, meets & 1)) return false;
            any = (fl[0] | fl[1] | fl[2] | fl[3]) != 0;
            ++meets;
            return true;
        };
        for (int64_t f = lo; f < hi && ok;) {
            w.seek(sb, units, f);
            const AbsorbedSegment g = segment_at(a, w.q, w.pre, f, hi);
            const int ctx = w.q.ctx;
            const bool live = has_row && row < g.rows;
            // keys this row may see; lanes without a row mask nothing
            const int lim = !live || !a.causal ? ctx : ctx - w.q.q_len + (g.row_in_seq + row) / a.num_heads + 1;
            const int ncols = (g.rows + 31) & ~31;  // TMEM columns of O^T to visit
            float m_ref = -INFINITY, l = 0.f;
            for (int t = 0; t < g.tiles; ++t, ++gt) {
                const int64_t key0 = (int64_t)(g.kb + t) * kLatentTile;
                if (!wait_all(&ms.s_full[gt & 1], (gt >> 1) & 1)) { ok = false; break; }
                tc_fence_after();
                uint32_t v[64];
                float red0, red1;
                const uint32_t tS = tl + (gt & 1) * kLatentTile;
                tmem_ld32_max(tS, reinterpret_cast<uint32_t(&)[32]>(v[0]), red0);
                tmem_ld32_max(tS + 32, reinterpret_cast<uint32_t(&)[32]>(v[32]), red1);
                tmem_wait_ld();
                reg_order32(reinterpret_cast<uint32_t(&)[32]>(v[0]));
                reg_order32(reinterpret_cast<uint32_t(&)[32]>(v[32]));
                float rm = fmaxf(red0, red1);
                const int vis = (int)max64(0, min64(lim - key0, kLatentTile));
                if (!__all_sync(0xffffffffu, vis >= kLatentTile)) {
                    rm = -INFINITY;
#pragma unroll
                    for (int j = 0; j < 64; ++j) {
                        if (j >= vis) v[j] = __float_as_uint(-INFINITY);
                        rm = fmaxf(rm, __uint_as_float(v[j]));
                    }
                }
                const float mx = rm * sl2;
                const bool up = live && mx > m_ref + kRescaleSlack;
                const float alpha = up ? fast_exp2(m_ref - mx) : 1.f;
                if (up) {
                    l *= alpha;
                    m_ref = mx;
                }
                if (has_row) ms.alpha[gt & 1][row] = alpha;
                __syncwarp();
                bool rescale = false;
                if (!meet(up && t > 0, rescale)) { ok = false; break; }
                // The weights, while the tensor pipe finishes the last tile's PV.  The sum adds them as
                // rounded, so a row that one key dominates loses nothing to their rounding.
                const float base = m_ref == -INFINITY ? 0.f : m_ref;
                uint32_t pk[32];
                float s0 = 0.f, s1 = 0.f;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const float e0 = fast_exp2(fmaf(__uint_as_float(v[2 * j]), sl2, -base));
                    const float e1 = fast_exp2(fmaf(__uint_as_float(v[2 * j + 1]), sl2, -base));
                    pk[j] = pack_bf16x2(e0, e1);
                    s0 += bf16_lo(pk[j]);
                    s1 += bf16_hi(pk[j]);
                }
                l += s0 + s1;
                if (gt > 0) {
                    if (!wait_all(&ms.pv_done, (gt - 1) & 1)) { ok = false; break; }
                    tc_fence_after();
                }
                if (rescale) {
                    // O^T's columns are the rows: scale each by its row's factor (rare: the first
                    // tiles of an item and jumps of a maximum by more than 2^8)
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
                                r[j] = __float_as_uint(__uint_as_float(r[j]) * ms.alpha[gt & 1][cb + j]);
                            tmem_st32(tO + mb * kLatentRows + cb, r);
                        }
                    tmem_wait_st();
                }
                if (has_row) {
#pragma unroll
                    for (int cc = 0; cc < 8; ++cc)
                        *reinterpret_cast<uint4 *>(sP + row * 128 + ((cc ^ (row & 7)) << 4)) =
                            make_uint4(pk[4 * cc], pk[4 * cc + 1], pk[4 * cc + 2], pk[4 * cc + 3]);
                }
                if (key0 + kLatentTile > ctx) {
                    // Slots past the context may hold NaN, and 0 * NaN would reach O^T: their value
                    // columns are zeroed once the copy has landed.
                    const uint32_t st = gt % NST;
                    if (!wait_all(&ms.kv_full[st], (gt / NST) & 1)) { ok = false; break; }
                    const int r0 = (int)(ctx - key0), pieces = (kLatentTile - r0) * (R / 8);
                    for (int i = tid; i < pieces; i += 128) {
                        const int rr = r0 + i / (R / 8), x = i % (R / 8);
                        *reinterpret_cast<uint4 *>(sKV + st * L::STAGE + (rr >> 3) * L::BOX + (x >> 3) * 1024 +
                                                   (rr & 7) * 128 + ((x & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.p_full);
            }
            if (!ok) break;
            // ---- epilogue: O / l of a whole item, or the part for the merge ----
            if (!wait_all(&ms.pv_done, (gt - 1) & 1)) { ok = false; break; }
            tc_fence_after();
            if (has_row) ms.inv[row] = l > 0.f ? 1.f / l : 0.f;
            __syncwarp();
            bool any;
            if (!meet(false, any)) { ok = false; break; }
            const int slot = g.whole ? 0 : part_slot(c, g.item_begin, T, ge);
            if (!g.whole && live) a.ws_ml[(int64_t)slot * kLatentRows + row] = make_float2(m_ref, l);
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
            // inv is written again only after the next item's first meeting, which every warp
            // reaches past its reads
            f += g.tiles;
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
    p->grid = sms < kMergeMaxParts ? sms : kMergeMaxParts;
    p->off_jobs = 0;
    p->off_ml = up(sizeof(MergeJob) * (size_t)p->grid);
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
    const MergeArgs m{a.ws_jobs, a.ws_ml, a.ws_o, a.out, kLatentRows, 1};
    return launch_merge<R>(m, a.grid, stream);
}

cudaError_t launch_latent_absorbed(int latent_dim, const CUtensorMap &q_map, const CUtensorMap &kv_map,
                                   const AbsorbedArgs &a, cudaStream_t stream) {
    return latent_dim == 512 ? launch_absorbed<512>(q_map, kv_map, a, stream)
                             : launch_absorbed<256>(q_map, kv_map, a, stream);
}

}  // namespace pkv
