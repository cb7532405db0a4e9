// Single tokens over 8-bit pages; the kernel is in paged_decode.cuh.
#include "paged_decode.cuh"

namespace bsa {

cudaError_t launch_paged_decode8(const DecodeArgs &a, cudaStream_t st) { return launch_decode<true>(a, st); }

}  // namespace bsa
