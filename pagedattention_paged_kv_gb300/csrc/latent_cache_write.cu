// latent_cache_write.cu -- the write of new tokens' latent rows into the block-paged latent
// cache (sm_103a).
//
// Token t's latent vector (latent_dim values) and its rotary key part (rope_dim values) become
// the one row [latent ; rope] of slot slot_mapping[t], unchanged.  Bound: HBM, every byte read
// once and written once; a few tokens are bound by the launch.  A thread has one 16-byte place of
// a row and walks a run of tokens, four rows in flight: the threads of a block are a whole number
// of rows (72 places at 512 + 64 columns), so none idles and no index is divided on the way.
#include "attn_block.cuh"
#include "pkv_common.cuh"

namespace pkv {

constexpr int kWriteInFlight = 4;

// blockDim.x = rows_side_by_side * min(row, kMaxRowThreads); wider rows take several rounds.
constexpr int kMaxRowThreads = 256;

__global__ void __launch_bounds__(512)
latent_cache_write_kernel(uint4 *__restrict__ cache, const uint4 *__restrict__ latent,
                          const uint4 *__restrict__ rope, const int64_t *__restrict__ slot_mapping,
                          int64_t num_tokens, int64_t num_slots, int latent_vecs, int rope_vecs,
                          int side, int tokens_per_cta, int *err) {
    pdl_wait();  // the rows and slots may come from the previous kernel in the stream
    pdl_trigger();
    const int row = latent_vecs + rope_vecs, width = blockDim.x / side;
    const int sub = threadIdx.x / width;
    const int64_t t0 = (int64_t)blockIdx.x * tokens_per_cta, t1 = min64(num_tokens, t0 + tokens_per_cta);
    for (int v = threadIdx.x - sub * width; v < row; v += width) {
        const bool in_latent = v < latent_vecs;
        const uint4 *src = in_latent ? latent + v : rope + (v - latent_vecs);
        const int64_t pitch = in_latent ? latent_vecs : rope_vecs;
        for (int64_t t = t0 + sub; t < t1; t += side * kWriteInFlight) {
            uint4 x[kWriteInFlight];
            int64_t slot[kWriteInFlight];
#pragma unroll
            for (int k = 0; k < kWriteInFlight; ++k) {
                const int64_t tk = t + k * side;
                slot[k] = -1;
                if (tk < t1) {
                    slot[k] = slot_mapping[tk];
                    x[k] = __ldcs(src + tk * pitch);
                }
            }
#pragma unroll
            for (int k = 0; k < kWriteInFlight; ++k) {
                if (slot[k] < 0) continue;  // padding token
                if (slot[k] >= num_slots) {
                    if (v == 0) flag_error(err, PKV_DEVERR_SLOT);
                    continue;
                }
                __stcs(cache + slot[k] * row + v, x[k]);
            }
        }
    }
}

cudaError_t launch_latent_cache_write(void *cache, const void *latent, const void *rope,
                                      const int64_t *slot_mapping, int64_t num_tokens, int64_t num_slots,
                                      int latent_bytes, int rope_bytes, int num_sms, int *err,
                                      cudaStream_t stream) {
    const int row = (latent_bytes + rope_bytes) / 16;
    const int width = row < kMaxRowThreads ? row : kMaxRowThreads;
    // Few tokens: one each CTA, spread over the SMs.  Many: CTAs of about 300 threads that keep
    // four rows a thread in flight.
    const bool few = num_tokens <= 4 * (int64_t)num_sms;
    int side = few ? 1 : 320 / width;
    if (side < 1) side = 1;
    int64_t per = few ? 1 : side * kWriteInFlight;
    while ((num_tokens + per - 1) / per > 0x7fffffff) per *= 2;
    return launch_pdl(latent_cache_write_kernel, dim3((unsigned)((num_tokens + per - 1) / per)), dim3(side * width), 0,
                      stream, static_cast<uint4 *>(cache), static_cast<const uint4 *>(latent),
                      static_cast<const uint4 *>(rope), slot_mapping, num_tokens, num_slots, latent_bytes / 16,
                      rope_bytes / 16, side, (int)per, err);
}

}  // namespace pkv
