// New tokens over 16-bit pages, few rows at a time; the kernel is in
// paged_attention.cuh.
#include "paged_attention.cuh"

namespace bsa {

cudaError_t launch_attention_rows(const AttentionArgs &a, cudaStream_t st) {
    return launch_rows_form<false>(a, st);
}

// Sixteen rows of a sequence and cache head are what the few-row form takes at
// once; with more it would read K and V again for each sixteen.
cudaError_t launch_paged_attention(const AttentionArgs &a, cudaStream_t st) {
    const int64_t mean = (a.tokens + a.seqs - 1) / a.seqs;
    if (mean * (a.q_heads / a.c.heads) > kMaxRows)
        return a.ks != nullptr ? launch_attention_tiles8(a, st) : launch_attention_tiles(a, st);
    return a.ks != nullptr ? launch_attention_rows8(a, st) : launch_attention_rows(a, st);
}

}  // namespace bsa
