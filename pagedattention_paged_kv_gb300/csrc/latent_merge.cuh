// latent_merge.cuh -- the join of work items that share boundaries cut (both latent-attention
// kernels).
//
// Each CTA that touched an item leaves, per row, its reference maximum m_p, sum l_p and
// unnormalised output o_p; with M = max_p m_p
//     out = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p,
// exact, as every part's weights are relative to its own m_p.
//
// Bound: latency of the L2, which holds the parts just written.  A thread has 4 columns of one row and
// the loads of three parts of it in flight, five CTAs an SM: most items have two or three parts, and
// four parts of two rows a thread (three CTAs an SM) took 1 us more of 11 for 128 items of 64 x 512.
// One 32k context of 23 parts likes four or six in flight better, by less than that.
#pragma once

#include "attn_block.cuh"

namespace pkv {

// An item whose units lie in the shares of CTAs c0 .. c1 (c0 < 0: none); written by CTA c0 + 1,
// whose share begins inside it.
struct LatentJob {
    int64_t out_off;  // element of out at which the item's first row begins
    int32_t c0, c1, rows;
};

// A CTA has at most one part that begins inside its item, and one that begins with it.
__device__ __forceinline__ int latent_slot(int c, bool begins) { return 2 * c + begins; }

// Parts lie as [2 * grid][SLOT_ROWS] (m, l) and [2 * grid][SLOT_ROWS][D] o.  BARE: a part that
// saw nothing of a row (l = 0) need not have left an output there.  (m = -inf does not tell: it is
// that of a part with scores of NaN alone too, whose l and o are NaN.)
template <int D, int SLOT_ROWS, bool BARE>
__global__ void __launch_bounds__(256, 5)
latent_merge_kernel(const LatentJob *jobs, const float2 *ws_ml, const float *ws_o, __nv_bfloat16 *out,
                    int64_t out_stride) {
    constexpr int CG = D / 4, SETS = 256 / CG;  // threads of a row, rows side by side
    constexpr int U = 3;                        // parts in flight
    pdl_wait();
    const LatentJob j = jobs[blockIdx.x];
    const int cg = threadIdx.x % CG, row = blockIdx.y * SETS + threadIdx.x / CG;
    if (j.c0 < 0 || row >= j.rows) return;
    const int nparts = j.c1 - j.c0 + 1;
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < nparts; p0 += U) {
        float2 ml[U];
        float4 o[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            ml[u] = make_float2(-INFINITY, 0.f);
            o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            const int p = p0 + u;
            if (p < nparts) {
                const int64_t at = (int64_t)latent_slot(j.c0 + p, p == 0) * SLOT_ROWS + row;
                ml[u] = __ldcg(ws_ml + at);
                o[u] = __ldcg(reinterpret_cast<const float4 *>(ws_o + at * D) + cg);
                if (BARE && ml[u].y == 0.f) o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        float mc = M;
#pragma unroll
        for (int u = 0; u < U; ++u) mc = fmaxf(mc, ml[u].x);
        const float base = mc == -INFINITY ? 0.f : mc;  // nothing seen yet
        const float s = fast_exp2(M - base);
        M = mc;
        L *= s;
        acc.x *= s;
        acc.y *= s;
        acc.z *= s;
        acc.w *= s;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float w = fast_exp2(ml[u].x - base);
            L = fmaf(w, ml[u].y, L);
            acc.x = fmaf(w, o[u].x, acc.x);
            acc.y = fmaf(w, o[u].y, acc.y);
            acc.z = fmaf(w, o[u].z, acc.z);
            acc.w = fmaf(w, o[u].w, acc.w);
        }
    }
    const float inv = 1.f / L;  // L = 0: every score is -inf, the row NaN by definition
    reinterpret_cast<uint2 *>(out + j.out_off + row * out_stride)[cg] =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

template <int D, int SLOT_ROWS, bool BARE>
cudaError_t launch_latent_merge(const LatentJob *jobs, const float2 *ws_ml, const float *ws_o, __nv_bfloat16 *out,
                                int64_t out_stride, int grid, cudaStream_t stream) {
    return launch_pdl(latent_merge_kernel<D, SLOT_ROWS, BARE>, dim3(grid, SLOT_ROWS * (D / 4) / 256), dim3(256), 0,
                      stream, jobs, ws_ml, ws_o, out, out_stride);
}

}  // namespace pkv
