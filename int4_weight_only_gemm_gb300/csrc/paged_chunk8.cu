// The chunk kernel of the paged attention (paged_chunk.cuh) for an 8-bit cache, causal tokens and draft blocks.
#include "paged_chunk.cuh"

namespace w4a16 {

template cudaError_t launch_paged_chunk<false, true>(const PagedAttnParams&, bool, int, bool, int, cudaStream_t, bool);
template int paged_chunk_status<false, true>();

}  // namespace w4a16
