// latent_merge.cuh -- the join of work items that share boundaries cut (both latent-attention
// kernels).
//
// Each CTA that touched an item leaves, per row, its reference maximum m_p, sum l_p and
// unnormalised output o_p; with M = max_p m_p
//     out = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p,
// exact, as every part's weights are relative to its own m_p.
//
// Bound: L2, which holds the parts just written.  A thread has 4 columns of kJoinRows rows, and
// the loads of four parts of each are in flight together: with one row a thread and a (job, row)
// grid the join of 128 items of 64 x 512 took 15 us behind its kernel, so 11 (12 alone with an
// empty L2).  Registers for three CTAs an SM without a spill: 16 bytes of it cost 5 to 10 us.
#pragma once

#include "attn_block.cuh"

namespace pkv {

// An item whose units lie in the shares of CTAs c0 .. c1 (c0 < 0: none); written by CTA c0 + 1,
// whose share begins inside it.
struct LatentJob {
    int64_t out_off;  // element of out at which the item's first row begins
    int32_t c0, c1, rows;
};

constexpr int kJoinRows = 2;

// A CTA has at most one part that begins inside its item, and one that begins with it.
__device__ __forceinline__ int latent_slot(int c, bool begins) { return 2 * c + begins; }

// Parts lie as [2 * grid][SLOT_ROWS] (m, l) and [2 * grid][SLOT_ROWS][D] o.  BARE: a part that
// saw nothing of a row (m = -inf) need not have left an output there.
template <int D, int SLOT_ROWS, bool BARE>
__global__ void __launch_bounds__(256, 3)
latent_merge_kernel(const LatentJob *jobs, const float2 *ws_ml, const float *ws_o, __nv_bfloat16 *out,
                    int64_t out_stride) {
    constexpr int CG = D / 4, SETS = 256 / CG;  // threads of a row, rows side by side
    constexpr int U = 4;                        // parts in flight
    pdl_wait();
    const LatentJob j = jobs[blockIdx.x];
    if (j.c0 < 0) return;
    const int nparts = j.c1 - j.c0 + 1;
    const int cg = threadIdx.x % CG, row0 = blockIdx.y * (SETS * kJoinRows) + threadIdx.x / CG;
    float M[kJoinRows], Ls[kJoinRows];
    float4 acc[kJoinRows];
#pragma unroll
    for (int k = 0; k < kJoinRows; ++k) {
        M[k] = -INFINITY;
        Ls[k] = 0.f;
        acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int p0 = 0; p0 < nparts; p0 += U) {
        float2 ml[U][kJoinRows];
        float4 o[U][kJoinRows];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = min(p0 + u, nparts - 1);
            const int64_t slot = latent_slot(j.c0 + p, p == 0);
#pragma unroll
            for (int k = 0; k < kJoinRows; ++k) {
                const int row = row0 + k * SETS;
                ml[u][k] = make_float2(-INFINITY, 0.f);
                o[u][k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (p0 + u < nparts && row < j.rows) {
                    ml[u][k] = __ldcg(ws_ml + slot * SLOT_ROWS + row);
                    o[u][k] = __ldcg(reinterpret_cast<const float4 *>(ws_o + (slot * SLOT_ROWS + row) * D) + cg);
                    if (BARE && ml[u][k].x == -INFINITY) o[u][k] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kJoinRows; ++k) {
            float mc = M[k];
#pragma unroll
            for (int u = 0; u < U; ++u) mc = fmaxf(mc, ml[u][k].x);
            const float base = mc == -INFINITY ? 0.f : mc;  // nothing seen yet
            const float s = fast_exp2(M[k] - base);
            M[k] = mc;
            Ls[k] *= s;
            acc[k].x *= s;
            acc[k].y *= s;
            acc[k].z *= s;
            acc[k].w *= s;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float w = fast_exp2(ml[u][k].x - base);
                Ls[k] = fmaf(w, ml[u][k].y, Ls[k]);
                acc[k].x = fmaf(w, o[u][k].x, acc[k].x);
                acc[k].y = fmaf(w, o[u][k].y, acc[k].y);
                acc[k].z = fmaf(w, o[u][k].z, acc[k].z);
                acc[k].w = fmaf(w, o[u][k].w, acc[k].w);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kJoinRows; ++k) {
        const int row = row0 + k * SETS;
        if (row >= j.rows) continue;
        const float inv = Ls[k] > 0.f ? 1.f / Ls[k] : 0.f;
        const uint2 v = make_uint2(pack_bf16x2(acc[k].x * inv, acc[k].y * inv),
                                   pack_bf16x2(acc[k].z * inv, acc[k].w * inv));
        reinterpret_cast<uint2 *>(out + j.out_off + row * out_stride)[cg] = v;
    }
}

template <int D, int SLOT_ROWS, bool BARE>
cudaError_t launch_latent_merge(const LatentJob *jobs, const float2 *ws_ml, const float *ws_o, __nv_bfloat16 *out,
                                int64_t out_stride, int grid, cudaStream_t stream) {
    constexpr int per = 256 / (D / 4) * kJoinRows;
    return launch_pdl(latent_merge_kernel<D, SLOT_ROWS, BARE>, dim3(grid, SLOT_ROWS / per), dim3(256), 0, stream, jobs,
                      ws_ml, ws_o, out, out_stride);
}

}  // namespace pkv
