// latent_cache_write.cu -- the write of new tokens' latent rows into the block-paged latent
// cache (sm_103a).
//
// Token t's latent vector (latent_dim values) and its rotary key part (rope_dim values) become
// the one row [latent ; rope] of slot slot_mapping[t], unchanged.  Bound: HBM, every byte read
// once and written once; a few tokens are bound by the launch.  A CTA takes a run of tokens and
// its threads the 16-byte pieces of their rows, four loads in flight a thread before the first
// store, so rows whose piece count is no multiple of a warp (72 at 512 + 64) leave no lane idle.
#include "attn_block.cuh"
#include "pkv_common.cuh"

namespace pkv {

__global__ void __launch_bounds__(256)
latent_cache_write_kernel(uint4 *__restrict__ cache, const uint4 *__restrict__ latent,
                          const uint4 *__restrict__ rope, const int64_t *__restrict__ slot_mapping,
                          int64_t num_tokens, int64_t num_slots, int latent_vecs, int rope_vecs,
                          int tokens_per_cta, int *err) {
    pdl_wait();  // the rows and slots may come from the previous kernel in the stream
    pdl_trigger();
    const int64_t t0 = (int64_t)blockIdx.x * tokens_per_cta;
    const int row = latent_vecs + rope_vecs;
    const int n = (int)min64(tokens_per_cta, num_tokens - t0) * row;
    for (int i0 = threadIdx.x; i0 < n; i0 += 4 * 256) {
        uint4 x[4];
        int64_t dst[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + k * 256;
            dst[k] = -1;
            if (i >= n) continue;
            const int tl = i / row, v = i - tl * row;
            const int64_t t = t0 + tl, slot = slot_mapping[t];
            if (slot < 0) continue;  // padding token
            if (slot >= num_slots) {
                if (v == 0) flag_error(err, PKV_DEVERR_SLOT);
                continue;
            }
            dst[k] = slot * row + v;
            x[k] = v < latent_vecs ? __ldcs(latent + t * latent_vecs + v)
                                   : __ldcs(rope + t * rope_vecs + (v - latent_vecs));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (dst[k] >= 0) cache[dst[k]] = x[k];
    }
}

cudaError_t launch_latent_cache_write(void *cache, const void *latent, const void *rope,
                                      const int64_t *slot_mapping, int64_t num_tokens, int64_t num_slots,
                                      int latent_bytes, int rope_bytes, int num_sms, int *err,
                                      cudaStream_t stream) {
    // Runs long enough to fill a CTA's four loads a thread once every SM has work, one token a
    // CTA below that.
    int64_t per = num_tokens / (4 * (int64_t)num_sms);
    per = per < 1 ? 1 : per > 16 ? 16 : per;
    while ((num_tokens + per - 1) / per > 0x7fffffff) per *= 2;
    return launch_pdl(latent_cache_write_kernel, dim3((unsigned)((num_tokens + per - 1) / per)), dim3(256), 0, stream,
                      static_cast<uint4 *>(cache), static_cast<const uint4 *>(latent),
                      static_cast<const uint4 *>(rope), slot_mapping, num_tokens, num_slots, latent_bytes / 16,
                      rope_bytes / 16, (int)per, err);
}

}  // namespace pkv
