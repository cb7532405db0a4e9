// Single tokens over 16-bit pages; the kernel is in paged_decode.cuh.
#include "paged_decode.cuh"

namespace bsa {

cudaError_t launch_paged_decode(const DecodeArgs &a, cudaStream_t st) { return launch_decode<false>(a, st); }

}  // namespace bsa
