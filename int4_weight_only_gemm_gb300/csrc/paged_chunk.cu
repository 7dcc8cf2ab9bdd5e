// The chunk kernel of the paged attention (paged_chunk.cuh) for causal tokens and draft blocks.
#include "paged_chunk.cuh"

namespace w4a16 {

template cudaError_t launch_paged_chunk<false, false>(const PagedAttnParams&, bool, int, bool, int, cudaStream_t, bool);
template int paged_chunk_status<false, false>();

size_t paged_chunk_part_bytes(int d, int sms) {
    return (size_t)4 * sms * (d == 128 ? Ch<128, false>::kPartHalf : Ch<64, false>::kPartHalf) * sizeof(float);
}

int chunk_read_status() {
    int status = 0;
    for (int s : {paged_chunk_status<false, false>(), paged_chunk_status<true, false>(), paged_chunk_status<false, true>(),
                  paged_chunk_status<true, true>()}) {
        if (s == W4A16_ECUDA) return s;
        if (status == 0) status = s;
    }
    return status;
}

}  // namespace w4a16
