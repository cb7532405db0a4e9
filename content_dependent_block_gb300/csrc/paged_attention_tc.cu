// New tokens over 16-bit pages, many rows at a time; the kernel is in
// paged_attention_tc.cuh.
#include "paged_attention_tc.cuh"

namespace bsa {

cudaError_t launch_attention_tiles(const AttentionArgs &a, cudaStream_t st) {
    return launch_tiles_form<false>(a, st);
}

}  // namespace bsa
