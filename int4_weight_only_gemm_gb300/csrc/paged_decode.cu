// The small-row kernel of the paged attention (paged_decode.cuh) for causal tokens and draft blocks.
#include "paged_decode.cuh"

namespace w4a16 {

template cudaError_t launch_paged_decode<false>(const PagedAttnParams&, bool, int, int, cudaStream_t, bool);

size_t paged_decode_part_bytes(int d, int sms) {
    return (size_t)2 * sms * (d == 128 ? kDecPart<128> : kDecPart<64>) * sizeof(float);
}

}  // namespace w4a16
