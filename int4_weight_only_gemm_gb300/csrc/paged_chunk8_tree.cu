// The chunk kernel of the paged attention (paged_chunk.cuh) for an 8-bit cache and trees of drafted tokens.
#include "paged_chunk.cuh"

namespace w4a16 {

template cudaError_t launch_paged_chunk<true, true>(const PagedAttnParams&, bool, int, bool, int, cudaStream_t, bool);
template int paged_chunk_status<true, true>();

}  // namespace w4a16
