// latent_expand.cu -- per-head keys and values from the block-paged latent cache (sm_103a).
//
//   k[h][j] = W_k[h] c_j (128 columns),  v[h][j] = W_v[h] c_j (128 columns)
// for every cached token j of the sequences with query rows: a matrix product of the gathered
// latent rows [tokens, R] with the stacked weights [256 rows a head, R], written as rows of
// 256 16-bit columns a (head, token), and the rotary parts copied beside them.  Keys are
// rounded to bf16, values to fp16 (see latent_expanded.cu).  fp16 reaches from 2^16 down to 2^-14 with
// all its bits, and values may be of any size: those of 32 tokens of a head are stored 2^-x times as
// large, their largest between 2^14 and 2^15, and x beside them (x >= -64, reached by a largest of
// 2^-50).  A value is so off by 2^-11 of itself, by 2^-39 of that largest or by 2^-89.  x stays at 0
// from 2^14 on; a finite value past fp16's range is clamped to it and flagged PKV_DEVERR_VALUE.
//
// Bound: tensor.  2 * 256 * R operations against 512 bytes written a (token, head): 512
// operations a byte at R = 512.  What feeds the tensor pipe is the question: a CTA keeps 128
// tokens (all of R) in shared memory and streams the weights of one head after the other past
// them, 64 bytes a cycle at the full rate, about as much as an SM takes in, with three 32 KiB
// stages of room.  So two CTAs with a token tile each form a pair (cta_group::2): one MMA
// multiplies 256 tokens, each CTA holds one half of every weight chunk (its keys' rows or its
// values' rows) for both, and the same room makes six stages.  The accumulator (128 tokens x 256
// columns a CTA, half of TMEM) is double-buffered, so the stores of one head run under the
// products of the next.  Units are (pair of token tiles, head), cut into equal contiguous
// shares, so a pair reloads its tokens only when its share crosses tiles.
// Measured at 16,896 tokens x 64 heads, R = 512 (283 GFLOP, 554 MB written): 292 us for single
// CTAs, 228 with every chunk's halves multicast to both CTAs of a cluster, 212 as pairs, some 175 with
// the epilogue on eight warps that store whole lines.  The value warps' first pass over a unit, for its
// largest values, is not in these: with it eight prompts' 311 MB take 138 us, without it 130, both under
// the counters.  What is left is the writes: a plain fill of the 554 MB takes
// 140 us (3.9 TB/s; the products alone are 148 us at the peak rate), and without its stores the call is
// 45 us shorter.
// Waits are bounded in time.  The CTAs of a pair (always resident together) wait for each other;
// no pair waits for another.
#include "attn_block.cuh"
#include "fp32x2.cuh"
#include "latent_expanded.cuh"
#include "latent_walk.cuh"
#include "pkv_split.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace {

constexpr int kExpandThreads = 320;  // loads, MMAs, eight epilogue warps

template <int R>
struct ExpandSmem {
    static constexpr int KCH = R / 64;
    static constexpr uint32_t GROUP = KCH * 1024;         // 8 tokens, all latent chunks
    static constexpr uint32_t A_BYTES = (kExpTile / 8) * GROUP;
    static constexpr uint32_t W_STAGE = 128 * 128;        // this CTA's 128 weight rows x 64 columns
    static constexpr int NST = 6;
    static constexpr uint32_t OFF_W = A_BYTES;
    static constexpr uint32_t OFF_MISC = OFF_W + NST * W_STAGE;
    static constexpr uint32_t BYTES = OFF_MISC + 1024 + 1024;
    static_assert(BYTES <= 232448, "fits one CTA");
};

struct ExpandMisc {
    uint64_t a_full, a_empty, mma_done;
    uint64_t w_full[6], w_empty[6];
    uint64_t acc_full[2], acc_free[2];
    int64_t scan[kExpandThreads / 32];
    WalkStart start;
    uint32_t tmem_slot;
    int abort_flag;
};
static_assert(sizeof(ExpandMisc) <= 1024, "fits its place");

// Clamps a finite value to fp16's range; true if that changed it.
__device__ __forceinline__ bool clamp_f16(uint32_t &x) {
    const float v = __uint_as_float(x);
    if (!(fabsf(v) > 65504.f) || fabsf(v) == INFINITY) return false;
    x = __float_as_uint(copysignf(65504.f, v));
    return true;
}

__device__ __forceinline__ uint32_t pack_16(bool f16, uint32_t lo, uint32_t hi) {
    return f16 ? pack_f16x2(__uint_as_float(lo), __uint_as_float(hi))
               : pack_bf16x2(__uint_as_float(lo), __uint_as_float(hi));
}

// The rotary parts of a warp's 32 rows of a tile, 8 lanes a row: cache rows tok0 + r of sequence s
// (zeros past the context and for bad block ids) to padded rows row0 + r.
template <int R>
__device__ __forceinline__ void copy_rope(const ExpandArgs &a, int s, int64_t tok0, int64_t row0, int quarter,
                                          int valid) {
    const int lane = threadIdx.x & 31, er = lane >> 3, ec = lane & 7;
    const int32_t *table = a.block_tables + (int64_t)s * a.max_blocks_per_seq;
    uint4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int r = quarter * 32 + 4 * k + er;
        const int64_t t = tok0 + r;
        const int id = r < valid ? table[t >> a.block_shift] : -1;
        x[k] = make_uint4(0u, 0u, 0u, 0u);
        if (id >= 0 && id < a.num_blocks) {
            const int64_t slot = ((int64_t)id << a.block_shift) + (t & ((1 << a.block_shift) - 1));
            x[k] = __ldg(reinterpret_cast<const uint4 *>(a.cache + slot * (R + kExpRope) + R) + ec);
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        reinterpret_cast<uint4 *>(a.buf.rope + (row0 + quarter * 32 + 4 * k + er) * kExpRope)[ec] = x[k];
}

}  // namespace

// Units of a sequence: 128-token tiles.
struct ExpandUnits {
    __device__ __forceinline__ int64_t operator()(const SeqInfo &q) const { return (q.ctx + kExpTile - 1) / kExpTile; }
};

template <int R>
__global__ void __launch_bounds__(kExpandThreads, 1)
latent_expand_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap wk_map,
                     const __grid_constant__ CUtensorMap wv_map, const ExpandArgs a) {
    using L = ExpandSmem<R>;
    constexpr int NST = L::NST, KCH = L::KCH;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sA = smem, *sW = smem + L::OFF_W;
    ExpandMisc &ms = *reinterpret_cast<ExpandMisc *>(smem + L::OFF_MISC);
    volatile int *abort_flag = &ms.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int H = a.num_heads;
    const int rank = (int)cluster_rank(), c = blockIdx.x >> 1, nc = a.grid >> 1;  // cluster, clusters

    if (threadIdx.x == 0) {
        // Those the issuer waits for (a_full, w_full, acc_free) are used in the even CTA only and
        // signalled by both; the others are signalled by the issuer in both.
        mbar_init(&ms.a_full, 2);
        mbar_init(&ms.a_empty, 1);
        mbar_init(&ms.mma_done, 1);
        for (int i = 0; i < NST; ++i) {
            mbar_init(&ms.w_full[i], 1);
            mbar_init(&ms.w_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ms.acc_full[i], 1);
            mbar_init(&ms.acc_free[i], 16);  // one arrival per epilogue warp
        }
        ms.abort_flag = 0;
        fence_barrier_init();
    }
    if (threadIdx.x == 32) {
        tma_prefetch_desc(&kv_map);
        tma_prefetch_desc(&wk_map);
        tma_prefetch_desc(&wv_map);
    }
    if (warp == 1) tmem_alloc_pair(&ms.tmem_slot, 512);
    pdl_wait();
    pdl_trigger();
    const SeqBatch sb{a.query_start_loc, a.context_lens, a.num_seqs, a.total_q,
                      (int64_t)a.max_blocks_per_seq << a.block_shift, a.err};
    const ExpandUnits units{};
    const auto sc = scan_batch<kExpandThreads>(sb, ms.scan, blockIdx.x == 0, units);
    // A batch with more tokens than the caller counted is refused whole; the attention kernel
    // sees the same sum and writes zero rows.
    const int64_t NT = sc.total[0] <= a.buf.padded / kExpTile ? sc.total[0] : 0;
    if (blockIdx.x == 0 && NT != sc.total[0] && threadIdx.x == 0) flag_error(a.err, PKV_DEVERR_CONTEXT_LEN);
    const int64_t T = (NT + 1) / 2 * H;  // (pair, head) units
    const int ge = split_ctas(T, nc, 1);
    const bool works = T > 0 && c < ge;
    const int64_t lo = works ? quotient(c * T, ge) : 0, hi = works ? quotient((c + 1) * T, ge) : 0;
    const int64_t g0 = 2 * quotient(lo, H) + rank;  // this CTA's first token tile
    if (works) find_unit(sb, units, sc, 0, g0, &ms.start);
    tc_fence_before();
    cluster_barrier();  // the barriers of both CTAs are there before either is signalled
    tc_fence_after();
    const uint32_t tmem = ms.tmem_slot;
    auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.wait_ns));
    };
    bool ok = true;
    SeqWalk<ExpandUnits> w;
    if (works && g0 < NT) w.start(ms.start);  // (ms.start is written for these only)

    if (!works) {
        // nothing to do but to meet the other CTA at the end
    } else if (warp == 0) {
        // ------------------------------ TMA producer ------------------------------
        const uint64_t policy = l2_policy_evict_normal();
        const CUtensorMap *w_map = rank == 0 ? &wk_map : &wv_map;
        const uint32_t a_full = smem_of_cta(&ms.a_full, 0), w_full0 = smem_of_cta(&ms.w_full[0], 0);
        uint32_t st = 0, ph = 0, fill = 0, aloads = 0;
        int64_t p = quotient(lo, H);
        int h = (int)(lo - p * H);
        for (int64_t f = lo; f < hi && ok; ++f) {
            const int64_t g = 2 * p + rank;
            if (f == lo || h == 0) {
                ok = aloads == 0 || wait_all(&ms.a_empty, (aloads - 1) & 1);
                if (!ok) break;
                int boxes = 0;
                if (g < NT) {
                    w.seek(sb, units, g);
                    // the tile's boxes (blocks, or 32 tokens of a larger one), one a lane, at most 16
                    const int bshift = min(a.block_shift, 5);
                    const int64_t t0 = (g - w.pre) * kExpTile;
                    boxes = (int)((min64(kExpTile, w.q.ctx - t0) + (1 << bshift) - 1) >> bshift);
                    const int box_bytes = L::GROUP << (bshift - 3);
                    int bid = -1;
                    if (lane < boxes) {
                        bid = a.block_tables[(int64_t)w.s * a.max_blocks_per_seq +
                                             ((t0 + ((int64_t)lane << bshift)) >> a.block_shift)];
                        if (bid < 0 || bid >= a.num_blocks) {
                            flag_error(a.err, PKV_DEVERR_BLOCK_ID);
                            bid = -1;  // an out-of-range box is filled with zeros
                        }
                    }
                    if (lane == 0) mbar_arrive_expect_tx_cluster(a_full, boxes * box_bytes);
#pragma unroll 1
                    for (int i = 0; i < boxes; ++i) {
                        const int id = __shfl_sync(0xffffffffu, bid, i);
                        const int grp = ((i << bshift) & ((1 << a.block_shift) - 1)) >> 3;  // (a tile starts a block)
                        if (lane == 0)
                            tma_load_5d_pair(smem_u32(sA) + i * box_bytes, &kv_map, a_full, 0, 0, 0, grp, id, policy);
                    }
                } else if (lane == 0) {
                    mbar_arrive_cluster(a_full);  // no tile of its own: nothing to load
                }
                ++aloads;
            }
            if (lane == 0) {
#pragma unroll 1
                for (int kc = 0; kc < KCH; ++kc) {
                    ok = mbar_wait(&ms.w_empty[st], ph ^ 1, abort_flag, a.wait_ns);
                    if (!ok) break;
                    if (rank == 0) mbar_arrive_expect_tx(&ms.w_full[st], 2 * L::W_STAGE);  // both CTAs' halves
                    tma_load_5d_pair(smem_u32(sW) + st * L::W_STAGE, w_map, w_full0 + st * 8, kc * 64, 0, 0, 0,
                                     h * (kExpHeadDim / 64), policy);
                    ++fill;
                    if (++st == NST) { st = 0; ph ^= 1; }
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (g < NT) w.ahead(sb);
            if (++h == H) { h = 0; ++p; }
        }
        if (lane == 0) {
            const uint32_t pending = minu32(fill, NST);
            // The issuer's last arrivals at this CTA's barriers come before it ends; with them the copies
            // have landed, for the products read them.
            for (uint32_t k = fill - pending; k < fill && ok; ++k)
                ok = mbar_wait(&ms.w_empty[k % NST], (k / NST) & 1, abort_flag, a.wait_ns);
            if (ok && aloads > 0) ok = mbar_wait(&ms.a_empty, (aloads - 1) & 1, abort_flag, a.wait_ns);
            if (!ok) {
                flag_error(a.err, PKV_DEVERR_TIMEOUT);
                *abort_flag = 1;
                // copies in flight land first; their barriers are in the even CTA
                if (rank == 0) {
                    for (uint32_t k = fill - pending; k < fill; ++k)
                        mbar_wait(&ms.w_full[k % NST], (k / NST) & 1, nullptr, kCopyLandsNs);
                    if (aloads > 0) mbar_wait(&ms.a_full, (aloads - 1) & 1, nullptr, kCopyLandsNs);
                } else {
                    const uint64_t t0 = globaltimer_ns();
                    while (globaltimer_ns() - t0 < kCopyLandsNs) {
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------ MMA issuer ------------------------------
        // The even CTA issues for both.  Where the odd one has no tile of its own (the last pair of
        // an odd count) the products run over whatever its shared memory holds; nothing of them is
        // stored.
        constexpr uint32_t IDESC = umma_idesc_bf16(2 * kExpTile, 256, 0, 0);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t da = umma_desc_sw128(smem_u32(sA), 16, L::GROUP);
        const uint64_t dw0 = umma_desc_sw128(smem_u32(sW), 16, 1024);
        uint32_t st = 0, ph = 0, n = 0, atiles = 0;
        int64_t p = quotient(lo, H);
        int h = (int)(lo - p * H);
        for (int64_t f = lo; f < hi && ok && rank == 0; ++f, ++n) {
            if (f == lo || h == 0) {
                if (!wait_all(&ms.a_full, atiles & 1)) { ok = false; break; }
                ++atiles;
            }
            if (n >= 2 && !wait_all(&ms.acc_free[n & 1], ((n >> 1) - 1) & 1)) { ok = false; break; }
#pragma unroll 1
            for (int kc = 0; kc < KCH; ++kc) {
                if (!wait_all(&ms.w_full[st], ph)) { ok = false; break; }
                tc_fence_after();
                const uint64_t dw = dw0 + st * (L::W_STAGE >> 4);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    umma2_bf16_warp(tm + (n & 1) * 256, da + ((kc * 1024 + ks * 32) >> 4), dw + ((ks * 32) >> 4), IDESC,
                                   kc > 0 || ks > 0);
                umma2_commit_warp(&ms.w_empty[st], 3);
                if (++st == NST) { st = 0; ph ^= 1; }
            }
            if (!ok) break;
            umma2_commit_warp(&ms.acc_full[n & 1], 3);
            if (++h == H || f + 1 == hi) umma2_commit_warp(&ms.a_empty, 3);
            if (h == H) {
                h = 0;
                ++p;
            }
        }
        if (!ok) {
            if (lane == 0) flag_error(a.err, PKV_DEVERR_TIMEOUT);
            *abort_flag = 1;
        }
        if (rank == 0) {  // every MMA is done before TMEM is released
            umma2_commit_warp(&ms.mma_done, 1);
            mbar_wait(&ms.mma_done, 0, nullptr);
        }
        __syncwarp();
    } else {
        // ------------- epilogue -------------
        // Four warps write the keys, four the values.  The accumulator is read so that a row's 64
        // columns lie in four threads, 16 each (tmem_ld_16x64), which are 32 bytes of the stored row:
        // four threads store a whole line.  What order the stored columns have follows from the order
        // in which the weight maps load the weights' rows.  (With a row a thread, 32 lines a store, a
        // unit's stores took 5,500 cycles, its products 4,100.)
        const int quarter = warp & 3;
        const bool is_v = warp >= 6;
        const int row = quarter * 32 + (lane >> 2), part = lane & 3;
        const uint32_t acc_free0 = smem_of_cta(&ms.acc_free[0], 0);
        uint32_t n = 0;
        int64_t p = quotient(lo, H);
        int h = (int)(lo - p * H);
        for (int64_t f = lo; f < hi && ok; ++f, ++n) {
            const int64_t g = 2 * p + rank, row0 = g * kExpTile;  // the tile's first padded token
            int valid = 0;
            if (g < NT) {
                w.seek(sb, units, g);
                valid = (int)min64(kExpTile, w.q.ctx - (g - w.pre) * kExpTile);
                if (h == 0 && !is_v) copy_rope<R>(a, w.s, (g - w.pre) * kExpTile, row0, quarter, valid);
            }
            if (!wait_all(&ms.acc_full[n & 1], (n >> 1) & 1)) { ok = false; break; }
            tc_fence_after();
            if (g < NT) {
                uint16_t *dst = a.buf.kv + ((int64_t)(h * 4 + 2 * is_v) * a.buf.padded + row0) * 64 + part * 16;
                // a 64-column piece, 16 of the warp's rows; past the context the product saw whatever the
                // slots held
                auto load = [&](int i, uint32_t(&r)[32]) {
                    tmem_ld_16x64(tmem + ((uint32_t)(quarter * 32 + (i & 1) * 16) << 16) + (n & 1) * 256 + is_v * 128 +
                                      (i >> 1) * 64, r);
                    tmem_wait_ld();
                    reg_order32(r);
                    if (valid < kExpTile) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (row + (i & 1) * 16 + (j & 2) * 4 >= valid) r[j] = 0u;
                    }
                };
                float grow = 1.f;   // 2^-x
                bool past = false;  // a value is past fp16's range
                if (is_v) {
                    float top = 0.f;  // of the warp's 32 tokens (NaN does not take part)
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        uint32_t r[32];
                        load(i, r);
#pragma unroll
                        for (int j = 0; j < 32; j += 2)
                            top = fmax3(top, fabsf(__uint_as_float(r[j])), fabsf(__uint_as_float(r[j + 1])));
                    }
                    const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
                    const int x = max(kValueExpMin, min(0, (int)(bits >> 23) - 127 - 14));
                    grow = __uint_as_float((uint32_t)(127 - x) << 23);
                    past = __uint_as_float(bits) > 65504.f;
                    if (lane == 0) a.buf.value_exp[(int64_t)h * (a.buf.padded / 32) + row0 / 32 + quarter] = (int8_t)x;
                }
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    const int q = i >> 1, r0 = row + (i & 1) * 16;
                    uint32_t r[32];
                    load(i, r);
                    if (is_v) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * grow);
                        if (past) {
                            bool over = false;
#pragma unroll
                            for (int j = 0; j < 32; ++j) over |= clamp_f16(r[j]);
                            if (over) flag_error(a.err, PKV_DEVERR_VALUE);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {  // rows r0 and r0 + 8
                        uint32_t x[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = pack_16(is_v, r[4 * j + 2 * k], r[4 * j + 2 * k + 1]);
                        st_global_32(dst + (int64_t)q * a.buf.padded * 64 + (r0 + 8 * k) * 64, x);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(acc_free0 + (n & 1) * 8);
            if (++h == H) { h = 0; ++p; }
        }
        if (!ok) {
            if (lane == 0) flag_error(a.err, PKV_DEVERR_TIMEOUT);
            *abort_flag = 1;
        }
    }
    __syncwarp();
    tc_fence_before();
    cluster_barrier();  // the other CTA signals and fills this one's shared memory up to here
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

template <int R>
static cudaError_t launch_expand(const CUtensorMap &kv_map, const CUtensorMap &wk_map, const CUtensorMap &wv_map,
                                 const ExpandArgs &a, cudaStream_t stream) {
    static SmemAllowance allowed;
    const cudaError_t e = allow_dynamic_smem(latent_expand_kernel<R>, ExpandSmem<R>::BYTES, allowed);
    if (e != cudaSuccess) return e;
    return launch_pdl_cluster(latent_expand_kernel<R>, dim3(a.grid), dim3(kExpandThreads), 2, ExpandSmem<R>::BYTES,
                              stream, kv_map, wk_map, wv_map, a);
}

cudaError_t launch_latent_expand(int latent_dim, const CUtensorMap &kv_map, const CUtensorMap &wk_map,
                                 const CUtensorMap &wv_map, const ExpandArgs &a, cudaStream_t stream) {
    return latent_dim == 512 ? launch_expand<512>(kv_map, wk_map, wv_map, a, stream)
                             : launch_expand<256>(kv_map, wk_map, wv_map, a, stream);
}

}  // namespace pkv
