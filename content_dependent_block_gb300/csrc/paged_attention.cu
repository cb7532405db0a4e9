// New tokens over 16-bit pages, few rows at a time; the kernel is in
// paged_attention.cuh.
#include "paged_attention.cuh"

namespace bsa {

cudaError_t launch_attention_rows(const AttentionArgs &a, cudaStream_t st) {
    return launch_rows_form<false>(a, st);
}

cudaError_t launch_paged_attention(const AttentionArgs &a, cudaStream_t st) {
    return a.ks != nullptr ? launch_attention_rows8(a, st) : launch_attention_rows(a, st);
}

}  // namespace bsa
