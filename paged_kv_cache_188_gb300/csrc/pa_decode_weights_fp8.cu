// pa_decode_weights_fp8.cu -- kernel instances of decode attention with
// attention weights over the block-scaled e4m3 cache.
#include "pa_decode_block_host.h"

namespace pa {
pa_status decode_block_weights(const BlkArgs &a, int head_dim, cudaStream_t st)
{
    return dispatch_block<true, true>(a, head_dim, st);
}
}  // namespace pa
