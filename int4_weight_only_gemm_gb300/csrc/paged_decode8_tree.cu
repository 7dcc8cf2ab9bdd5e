// The small-row kernel over 8-bit caches (paged_decode8.cuh) for trees of drafted tokens.
#include "paged_decode8.cuh"

namespace w4a16 {

template cudaError_t launch_paged_decode8<true>(const PagedAttnParams&, bool, int, bool, int, cudaStream_t, bool);

}  // namespace w4a16
