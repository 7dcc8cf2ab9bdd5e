// The small-row kernel of the paged attention (paged_decode.cuh) for trees of drafted tokens.
#include "paged_decode.cuh"

namespace w4a16 {

template cudaError_t launch_paged_decode<true>(const PagedAttnParams&, bool, int, int, cudaStream_t, bool);

}  // namespace w4a16
