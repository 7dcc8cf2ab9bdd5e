// The chunk kernel of the paged attention (paged_chunk.cuh) for causal tokens and draft blocks.
#include "paged_chunk.cuh"

namespace w4a16 {

template cudaError_t launch_paged_chunk<false>(const PagedAttnParams&, bool, int, bool, int, cudaStream_t, bool);
template int paged_chunk_status<false>();

size_t paged_chunk_part_bytes(int d, int sms) {
    return (size_t)4 * sms * (d == 128 ? Ch<128, false>::kPartHalf : Ch<64, false>::kPartHalf) * sizeof(float);
}

int chunk_read_status() {
    const int a = paged_chunk_status<false>(), b = paged_chunk_status<true>();
    return a == W4A16_ECUDA || b == W4A16_ECUDA ? W4A16_ECUDA : a ? a : b;
}

}  // namespace w4a16
