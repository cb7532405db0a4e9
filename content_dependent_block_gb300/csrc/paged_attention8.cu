// New tokens over 8-bit pages, few rows at a time; the kernel is in
// paged_attention.cuh.
#include "paged_attention.cuh"

namespace bsa {

cudaError_t launch_attention_rows8(const AttentionArgs &a, cudaStream_t st) {
    return launch_rows_form<true>(a, st);
}

}  // namespace bsa
