// paged_shared.cu -- decode attention of a batch in which groups of sequences share a cached prefix:
// the shared rows read and multiplied once for all of a group, the own rows of each sequence by the
// decode kernel's CTAs, in one launch, and the join of the parts.
//
// softmax over [shared ; own] keys splits into parts (m_p, l_p, o_p), each relative to its own
// maximum, that add up exactly:
//     out = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p,  M = max_p m_p.
//
// A group of n sequences with P shared and R own tokens each reads P + n R rows in place of n (P + R).
// Bound: HBM for the own rows (decode_cta.cuh), the tensor cores for the shared ones when a group has
// many rows (prefix_cta.cuh).  The two run side by side: every CTA works out who shares what and the
// two amounts of work, and takes a role as in paged_varlen.cu.
//
// Measured (64 query heads over 8, d 128; the kernels of a call, L2 as they leave it): 128 sequences with
// up to 512 own tokens behind 8192 shared ones 56 us (193 MB of DRAM, which a copy would move in 28; 3.5 us
// until the roles begin, 4.5 until the first scores, the sides done at 47 to 50, the join 8), 64 sequences
// on two prefixes of 32,768 102 us (578 MB, 5.7 TB/s), 96 sequences on 12 documents over an FP8 cache 72 us
// (263 MB).  Each sequence alone (pkv_paged_attention_decode) the same batches take 277, 790 and 182 us.
#include "decode_cta.cuh"
#include "paged_shared.cuh"
#include "prefix_cta.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace {

// The last group that begins at or before sequence s (gs[0] <= s).
__device__ __forceinline__ int group_of(const int32_t *gs, int groups, int s) {
    int lo = 0, hi = groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (gs[mid] <= s) lo = mid; else hi = mid;
    }
    return lo;
}

// CTAs of the own side out of G, when both sides have work: the one at which the slower side is
// fastest, a unit (and, on the own side, an item) costing its side's CTAs its SM time and the own side
// never less than HBM allows.
__device__ __forceinline__ int own_ctas(int units, int items, int wide, int narrow, int G, const SharedCosts &c) {
    const float d = (float)units * c.own_unit_us + (float)items * c.own_item_us;
    const float p = (float)wide * c.wide_us + (float)narrow * c.narrow_us;
    const float t = fmaxf((d + p) / (float)G, (float)units * c.own_unit_hbm_us);
    // Near what HBM gives both sides get slower than their costs say: the CTAs that neither needs to be done in
    // that time are halved between them.
    return max(1, min(G - 1, (int)(0.5f * (d / t + (float)G - p / t) + 0.5f)));
}

// Two values as e4m3 codes, to nearest (ties to even, NaN stays), the first in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace

// A sequence shares the whole 16-token units of its group's prefix when its context holds the prefix,
// another sequence of the group does too, and the group is worth a tile; the others attend to all their
// tokens alone, as all do when group_start is not ascending within the batch.  So the result does not depend on
// the grouping, as long as the tables of a group agree.
// 384 threads leave 168 registers.  <128, FP8, two n-tiles> spills 44 bytes and loads 60 (the decode kernel of
// that form 72 and 104); the others spill nothing.
template <int D, bool FP8, int NTH>
__global__ void __launch_bounds__(kSharedThreads, 1)
paged_shared_kernel(const __grid_constant__ CUtensorMap dk_map, const __grid_constant__ CUtensorMap dv_map,
                    const __grid_constant__ CUtensorMap pq_map, const __grid_constant__ CUtensorMap pk_map,
                    const __grid_constant__ CUtensorMap pv_map,
                    const DecodeArgs ad, const PrefixArgs ap, const SharedArgs as, const SharedCosts costs) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int S = ap.num_seqs, G = ap.num_groups, nt = blockDim.x, tid = threadIdx.x;
    int32_t *skip = reinterpret_cast<int32_t *>(smem_raw + as.table_offset);  // [S], and
    int32_t *pre = skip + S;                                                  // [G + 1] for the roles
    // scratch until the roles begin: sums, the groups' starts, lengths and sharers, the contexts
    int32_t *tmp = reinterpret_cast<int32_t *>(base), *gs = tmp + 128, *len = gs + G + 1, *count = len + G;
    int32_t *ctx = count + G;
    const bool report = blockIdx.x == 0;
    if (tid == 0) {
        tma_prefetch_desc(&dk_map);
        tma_prefetch_desc(&dv_map);
        if (ap.q_boxes) tma_prefetch_desc(&pq_map);
        tma_prefetch_desc(&pk_map);
        tma_prefetch_desc(&pv_map);
    }
    const int64_t room = (int64_t)ap.max_blocks_per_seq * ap.block_size;
    pdl_wait();
    pdl_trigger();
    for (int i = tid; i < G || i < S; i += nt) {
        if (i < G) {
            gs[i] = ap.group_start[i];
            len[i] = as.prefix_lens[i];
            count[i] = 0;
        }
        if (i < S) ctx[i] = ad.context_lens[i];
    }
    if (tid == 0) gs[G] = G > 0 ? ap.group_start[G] : 0;
    __syncthreads();
    bool good = true;
    for (int g = tid; g < G; g += nt) {
        good = good && gs[g] >= 0 && gs[g] <= gs[g + 1] && gs[g + 1] <= S;
        if (len[g] < 0 || len[g] > room) {
            if (report) flag_error(ap.err, PKV_DEVERR_CONTEXT_LEN);
            len[g] = 0;
        }
    }
    good = __syncthreads_and(good);
    if (!good && report && tid == 0) flag_error(ap.err, PKV_DEVERR_SEQ);
    const int first = good && G > 0 ? gs[0] : S, last = good && G > 0 ? gs[G] : S;
    for (int s = tid; s < S; s += nt) {
        int32_t group = -1;
        if (s >= first && s < last) {
            group = group_of(gs, G, s);
            if (len[group] < kBS || ctx[s] < len[group] || ctx[s] > room) group = -1;
            else atomicAdd(count + group, 1);
        }
        skip[s] = group;
    }
    __syncthreads();
    // A group whose sequences would read the prefix in less SM time than its tiles take does not share it.
    // HBM is left out, so groups of two that it bounds do not share (32 behind 8192 tokens, 64 heads over 8: 315
    // us alone, 190 shared; groups of three share: 191, alone 462).
    for (int g = tid; g < G; g += nt) {
        if (count[g] < 2 || costs.mode == 2) continue;
        const int seqs = gs[g + 1] - gs[g], tiles = prefix_tiles(seqs, ap.group);
        const bool narrow = (seqs - (tiles - 1) * (kPrefixRows / ap.group)) * ap.group <= kPrefixRows / 2;
        const float tile_us = (float)(tiles - 1) * costs.wide_us + (narrow ? costs.narrow_us : costs.wide_us);
        const float shared_us = tile_us * (float)(ap.num_kv_heads * prefix_units(len[g] / kBS));
        const float alone_us = (float)count[g] * (float)(len[g] / kBS * ad.head_tiles) * costs.own_unit_us;
        if (costs.mode == 0 || alone_us < shared_us) count[g] = 0;
    }
    __syncthreads();
    // own units of all sequences; units of the groups
    int32_t own = 0, items = 0, mine = 0, narrow = 0;
    for (int s = tid; s < S; s += nt) {
        const int32_t group = skip[s], units = group >= 0 && count[group] > 1 ? len[group] / kBS : 0;
        skip[s] = units;
        const int32_t rest = ctx[s] > 0 && ctx[s] <= room ? (ctx[s] + kBS - 1) / kBS - units : 0;
        own += rest * ad.head_tiles;
        items += rest > 0 ? ad.head_tiles : 0;
    }
    const int per = (G + nt - 1) / nt, g0 = min(G, tid * per), g1 = min(G, g0 + per);
    auto units_of = [&](int g) -> int32_t {
        return good && count[g] > 1
                   ? prefix_tiles(gs[g + 1] - gs[g], ap.group) * ap.num_kv_heads * prefix_units(len[g] / kBS)
                   : 0;
    };
    for (int g = g0; g < g1; ++g) {
        const int units = units_of(g), seqs = gs[g + 1] - gs[g], tiles = prefix_tiles(seqs, ap.group);
        mine += units;
        // the last tile may be narrow
        if (units > 0 && (seqs - (tiles - 1) * (kPrefixRows / ap.group)) * ap.group <= kPrefixRows / 2) narrow += units / tiles;
    }
    int32_t td = 0, ti = 0, tn = 0;
    {
        const int lane = tid & 31, warp = tid >> 5;
        int32_t x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        own = __reduce_add_sync(0xffffffffu, own);
        items = __reduce_add_sync(0xffffffffu, items);
        narrow = __reduce_add_sync(0xffffffffu, narrow);
        if (lane == 31) {
            tmp[warp] = x;
            tmp[32 + warp] = own;
            tmp[64 + warp] = items;
            tmp[96 + warp] = narrow;
        }
        __syncthreads();
        int32_t run = x - mine;
        for (int w = 0; w < nt / 32; ++w) {
            if (w < warp) run += tmp[w];
            td += tmp[32 + w];
            ti += tmp[64 + w];
            tn += tmp[96 + w];
        }
        for (int g = g0; g < g1; ++g) {
            pre[g] = run;
            run += units_of(g);
        }
        if (tid == nt - 1) pre[G] = run;
        __syncthreads();
    }
    const int tp = pre[G];
    const int grid = (int)gridDim.x;
    const int k = tp == 0 ? grid : td == 0 ? 1 : own_ctas(td, ti, tp - tn, tn, grid, costs);
    // for the join: the parts of each (sequence, KV head) over shared units
    for (int i = (int)blockIdx.x * nt + tid; i < S * ap.num_kv_heads; i += grid * nt) {
        const int s = i / ap.num_kv_heads, kvh = i - s * ap.num_kv_heads;
        int4 parts = make_int4(-1, 0, 0, 0);
        if (skip[s] > 0) {
            const Shares shares(tp, split_ctas(tp, grid - k, kPrefixMinUnits));
            const int g = group_of(gs, G, s), place = s - gs[g], per_tile = kPrefixRows / ap.group, tile = place / per_tile;
            const int units = prefix_units(skip[s]);
            const int begin = pre[g] + (kvh * prefix_tiles(gs[g + 1] - gs[g], ap.group) + tile) * units;
            // the first part is left by the CTA that has the tile's first chunk
            const int c0 = shares.owner(begin + kPrefixSwitch), c1 = shares.owner(begin + units - 1);
            parts = make_int4(shares.owner(begin) == c1 ? -1 : shares.slot(c0, begin), c1 - c0 + 1,
                              (place - tile * per_tile) * ap.group, 0);
        }
        as.prefix_parts[i] = parts;
    }
    hand_over_smem();  // the scratch is free for the roles
    if ((int)blockIdx.x < k) decode_cta<D, FP8, NTH, true>(dk_map, dv_map, ad, (int)blockIdx.x, k, false, skip);
    else prefix_cta<D, FP8>(pq_map, pk_map, pv_map, ap, pre, skip, (int)blockIdx.x - k, grid - k);
}

// A query row for the prefix CTAs of an FP8 cache: q 2^s, with the row's largest element in [2^7, 2^8), as
// two rows of e4m3, the first four significant bits of each element and the other four, and the unit
// 2^-s.  They add up to bf16's value exactly for elements down to 2^-9 of the row's largest, and to within
// 2^-16 of that largest below.  A row that holds an infinity gets NaN in its place: it has no softmax
// either way.  A warp a row.  (In the prefix CTAs, for each tile anew, this took 3 us a tile.)
__global__ void __launch_bounds__(256) split_queries_kernel(const uint2 *q, uint32_t *q8, float *q_unit, int64_t rows) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const uint2 w = q[row * 32 + lane];  // four elements
    const uint32_t m = __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu);
    const int expo = (int)(__reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16)) >> 7);  // biased; 255: not finite
    const int s = min(134 - expo, 126);
    const __nv_bfloat162 up = __float2bfloat162_rn(__int_as_float((s + 127) << 23));
    uint32_t hi = 0, lo = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t x = i == 0 ? w.x : w.y;
        __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&x), up);
        if (expo == 255) v = __hadd2(v, __hsub2(v, v));
        const uint32_t h = *reinterpret_cast<const uint32_t *>(&v) & 0xfff0fff0u;
        const __nv_bfloat162 rest = __hsub2(v, *reinterpret_cast<const __nv_bfloat162 *>(&h));
        const uint32_t l = *reinterpret_cast<const uint32_t *>(&rest);
        hi |= to_e4m3x2(bf16_lo(h), bf16_hi(h)) << (16 * i);
        lo |= to_e4m3x2(bf16_lo(l), bf16_hi(l)) << (16 * i);
    }
    q8[row * 32 + lane] = hi;
    q8[(rows + row) * 32 + lane] = lo;
    if (lane == 0) q_unit[row] = __int_as_float((127 - s) << 23);
}

cudaError_t launch_split_queries(const __nv_bfloat16 *q, uint8_t *q8, float *q_unit, int64_t rows, cudaStream_t stream) {
    return launch_pdl(split_queries_kernel, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, stream,
                      reinterpret_cast<const uint2 *>(q), reinterpret_cast<uint32_t *>(q8), q_unit, rows);
}

// Output rows from their parts: D / 8 threads a row, each with eight columns.  The parts of an item
// that one CTA worked on whole stand at its rows; those of a split one in the slots of the CTAs whose
// shares touch it.  Each thread works out where one part is and loads its (m, l), so that the index
// arithmetic of a row is done once, whatever the number of its parts.  Bound: the latency of two rounds of
// loads from L2 where rows are few (8192 rows of four to six parts, 20 MB: 8 us), its instructions where
// they are many (44,000 rows of two: 17 us).
struct JoinArgs {
    __nv_bfloat16 *out;
    const int32_t *context_lens;
    const int4 *prefix_parts;  // [num_seqs][num_kv_heads]
    const int2 *own_parts;     // [num_seqs][head_tiles]
    const float2 *own_ml, *own_whole_ml, *pre_ml, *pre_whole_ml;
    const float *own_o, *own_whole_o, *pre_o, *pre_whole_o;
    int num_seqs, num_heads, num_kv_heads, group, heads_per_cta, head_tiles;
    float inv_group, inv_heads_per_cta;
    int64_t room;  // tokens of a table row
};

template <int D>
__global__ void __launch_bounds__(256, 3) join_kernel(const JoinArgs a) {
    constexpr int CG = D / 8;
    const int cg = threadIdx.x % CG, s = blockIdx.y, h = blockIdx.x * (256 / CG) + threadIdx.x / CG;
    // Exact: kvh * group <= 2^20 (8192 items of up to 8 heads, 128 rows), so a quotient is off by at most
    // 2^-23 * 2^20 / group = 1 / (8 group), and the half added leaves 1 / (2 group)
    const int kvh = (int)(((float)h + 0.5f) * a.inv_group), hg = h - kvh * a.group;
    const int ht = (int)(((float)kvh + 0.5f) * a.inv_heads_per_cta);
    const int64_t row = (int64_t)s * a.num_heads + h;
    pdl_wait();
    pdl_trigger();
    if (h >= a.num_heads) return;
    const int ctx = a.context_lens[s];
    const int4 shared = a.prefix_parts[(int64_t)s * a.num_kv_heads + kvh];
    const int2 own = a.own_parts[(int64_t)s * a.head_tiles + ht];
    uint4 *out = reinterpret_cast<uint4 *>(a.out + row * D) + cg;
    if (ctx < 1 || ctx > a.room) {
        *out = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    // parts over the shared tokens first, then those over the own ones
    const int n = shared.y + own.y;
    const uint32_t lanes = ((1u << CG) - 1) << (threadIdx.x % 32 / CG * CG);  // of this row
    float M = -INFINITY, sum = 0.f;
    float acc[8] = {};
    for (int i0 = 0; i0 < n; i0 += CG) {
        const int i = i0 + cg;
        const float2 *ml = nullptr;
        const float *o = nullptr;
        if (i < n) {
            const bool of_shared = i < shared.y;
            const int p = of_shared ? i : i - shared.y, first = of_shared ? shared.x : own.x;
            int64_t r = row;  // of a whole item
            if (first >= 0) {
                const int slot = p == 0 ? first : 2 * ((first >> 1) + p);
                r = of_shared ? (int64_t)slot * kPrefixRows + shared.z + hg
                              : ((int64_t)slot * a.heads_per_cta + kvh - ht * a.heads_per_cta) * a.group + hg;
            }
            ml = (of_shared ? (first < 0 ? a.pre_whole_ml : a.pre_ml) : (first < 0 ? a.own_whole_ml : a.own_ml)) + r;
            o = (of_shared ? (first < 0 ? a.pre_whole_o : a.pre_o) : (first < 0 ? a.own_whole_o : a.own_o)) + r * D;
        }
        const float2 x = ml ? __ldcg(ml) : make_float2(-INFINITY, 0.f);
        // The first kPC parts' columns are asked for before the weights are worked out.
        constexpr int kPC = 4;  // parts in flight
        const uint64_t at = reinterpret_cast<uint64_t>(o);
        const int here = min(CG, n - i0);
        float4 v[kPC][2];
        auto load = [&](int q0) {
#pragma unroll
            for (int q = 0; q < kPC; ++q) {
                if (q0 + q >= here) break;
                const float4 *src = reinterpret_cast<const float4 *>(__shfl_sync(lanes, at, q0 + q, CG)) + 2 * cg;
                v[q][0] = __ldcg(src);
                v[q][1] = __ldcg(src + 1);
            }
        };
        load(0);
        float top = x.x;
#pragma unroll
        for (int k = CG / 2; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(lanes, top, k));
        top = fmaxf(top, M);
        // a part whose scores are all -infinity or NaN keeps the weight 1: it holds zeros or NaN
        const float base = top == -INFINITY ? 0.f : top;
        const float w0 = M == -INFINITY ? 1.f : fast_exp2(M - base);
        const float w = !ml ? 0.f : x.x == -INFINITY ? 1.f : fast_exp2(x.x - base);
        float l = w * x.y;
#pragma unroll
        for (int k = CG / 2; k > 0; k >>= 1) l += __shfl_xor_sync(lanes, l, k);
        sum = sum * w0 + l;
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] *= w0;
        M = top;
        for (int q0 = 0;;) {
#pragma unroll
            for (int q = 0; q < kPC; ++q) {
                if (q0 + q >= here) break;
                const float wq = __shfl_sync(lanes, w, q0 + q, CG);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    acc[4 * c] += wq * v[q][c].x;
                    acc[4 * c + 1] += wq * v[q][c].y;
                    acc[4 * c + 2] += wq * v[q][c].z;
                    acc[4 * c + 3] += wq * v[q][c].w;
                }
            }
            if ((q0 += kPC) >= here) break;
            load(q0);
        }
    }
    const float inv = 1.f / sum;
    *out = make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                      pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
}

// ---- host side -------------------------------------------------------------------

int plan_shared(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int head_tiles, int grid, int smem_room,
                bool fp8, SharedPlan *p) {
    // Q; barriers, a narrow tile's second half, the TMEM slot and the abort flag
    const size_t stage = (size_t)kPrefixKeys * head_dim * 2, stage8 = (size_t)kPrefixKeys * head_dim;
    size_t fixed = 1024 + (size_t)(head_dim / 64) * 2 * 128 * 128 + 8 * 12 + 8 * 128 + 8;
    if (fp8) fixed += kPrefixV16 * (stage + 16) + kPrefixV8 * (stage8 + 16);
    const size_t per = (fp8 ? stage8 : stage) + 16;
    int nst = (int)(((int64_t)smem_room - (int64_t)fixed) / (int64_t)per);
    if (nst > 4) nst = 4;
    if (nst < (fp8 ? 2 : 3)) return PKV_ERR_UNSUPPORTED;
    p->num_stages = nst;
    p->smem = fixed + nst * per;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t rows = (size_t)num_seqs * num_heads, slots = 2 * (size_t)grid * kPrefixRows;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += up(bytes);
        return o;
    };
    p->off_prefix_parts = take(sizeof(int4) * (size_t)num_seqs * num_kv_heads);
    p->off_own_parts = take(sizeof(int2) * (size_t)num_seqs * head_tiles);
    p->off_whole_own = take(4 * rows * head_dim);
    p->off_whole_own_ml = take(8 * rows);
    p->off_whole_pre = take(4 * rows * head_dim);
    p->off_whole_pre_ml = take(8 * rows);
    p->off_ml = take(8 * slots);
    p->off_o = take(4 * slots * head_dim);
    p->off_q8 = take(2 * rows * head_dim);  // FP8 cache
    p->off_unit = take(4 * rows);
    p->bytes = at;
    return PKV_OK;
}

template <int D, bool FP8, int NTH>
static cudaError_t launch_shared_d(const CUtensorMap &dk, const CUtensorMap &dv, const DecodeArgs &ad,
                                   const CUtensorMap &pq, const CUtensorMap &pk, const CUtensorMap &pv,
                                   const PrefixArgs &ap, const SharedArgs &as, const SharedCosts &costs,
                                   size_t smem, cudaStream_t stream) {
    auto kernel = paged_shared_kernel<D, FP8, NTH>;
    static SmemAllowance allowed;
    cudaError_t e = allow_dynamic_smem(kernel, smem, allowed);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3(ad.grid), dim3(kSharedThreads), smem, stream, dk, dv, pq, pk, pv, ad, ap, as, costs);
    if (e != cudaSuccess) return e;
    JoinArgs j;
    j.out = ad.out;
    j.context_lens = ad.context_lens;
    j.prefix_parts = as.prefix_parts;
    j.own_parts = ad.own_parts;
    j.own_ml = ad.ws_ml;
    j.own_o = ad.ws_o;
    j.own_whole_ml = ad.whole_ml;
    j.own_whole_o = ad.whole_o;
    j.pre_ml = ap.ws_ml;
    j.pre_o = ap.ws_o;
    j.pre_whole_ml = ap.whole_ml;
    j.pre_whole_o = ap.whole_o;
    j.num_seqs = ad.num_seqs;
    j.num_heads = ad.num_heads;
    j.num_kv_heads = ap.num_kv_heads;
    j.group = ad.group;
    j.inv_group = 1.f / (float)ad.group;
    j.inv_heads_per_cta = 1.f / (float)ad.heads_per_cta;
    j.heads_per_cta = ad.heads_per_cta;
    j.head_tiles = ad.head_tiles;
    j.room = (int64_t)ad.max_blocks_per_seq * ad.block_size;
    constexpr int per = 256 / (D / 8);  // rows of a CTA
    // y has 16 bits: the sequences (8192 at most), not the heads (2^20)
    return launch_pdl(join_kernel<D>, dim3((ad.num_heads + per - 1) / per, ad.num_seqs), dim3(256), 0, stream, j);
}

cudaError_t launch_paged_shared(int head_dim, bool fp8, const CUtensorMap &dk, const CUtensorMap &dv,
                                const DecodeArgs &ad, const CUtensorMap &pq, const CUtensorMap &pk,
                                const CUtensorMap &pv, const PrefixArgs &ap, const SharedArgs &as, const SharedCosts &costs,
                                   size_t smem,
                                cudaStream_t stream) {
    const bool two = ad.group > 8;  // n-tiles of 8 query heads a consumer warp of the own side
    if (fp8) {
        if (head_dim != 128) return cudaErrorInvalidValue;
        return two ? launch_shared_d<128, true, 2>(dk, dv, ad, pq, pk, pv, ap, as, costs, smem, stream)
                   : launch_shared_d<128, true, 1>(dk, dv, ad, pq, pk, pv, ap, as, costs, smem, stream);
    }
    if (head_dim == 128)
        return two ? launch_shared_d<128, false, 2>(dk, dv, ad, pq, pk, pv, ap, as, costs, smem, stream)
                   : launch_shared_d<128, false, 1>(dk, dv, ad, pq, pk, pv, ap, as, costs, smem, stream);
    return two ? launch_shared_d<64, false, 2>(dk, dv, ad, pq, pk, pv, ap, as, costs, smem, stream)
               : launch_shared_d<64, false, 1>(dk, dv, ad, pq, pk, pv, ap, as, costs, smem, stream);
}

}  // namespace pkv
