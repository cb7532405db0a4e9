// New tokens over 16-bit pages, few rows at a time; the kernel is in
// paged_attention.cuh.
#include "paged_attention.cuh"

namespace bsa {

cudaError_t launch_attention_rows(const AttentionArgs &a, cudaStream_t st) {
    return launch_rows_form<false>(a, st);
}

// Few rows: what the register tiles take at once, eight or sixteen of a sequence
// and cache head; with more they would read K and V again for each sixteen.
// Sixteen are two tiles side by side, of which 16-bit pages leave two CTAs to an
// SM: the tensor cores' form is faster there unless there are few keys (64
// sequences, 4 tokens, 32 heads over 8, d 128: 4096 keys 241 us against 213,
// 512 keys 50 against 58; 16 sequences of 4096 to 32768 keys 301 against 223;
// over 8-bit pages 220 against 356 and 277 against 314; with eight rows 200
// against 211 and, 24 sequences, 216 against 222).
cudaError_t launch_paged_attention(const AttentionArgs &a, cudaStream_t st) {
    const int64_t rows = (a.tokens + a.seqs - 1) / a.seqs * (a.q_heads / a.c.heads);
    const int64_t held = int64_t(a.width) * a.c.page, window = int64_t(a.window) + a.sinks;
    const bool short_keys = (a.window > 0 && window < held ? window : held) <= 1024;
    if (rows > (a.ks != nullptr || short_keys ? kMaxRows : kMaxRows / 2))
        return a.ks != nullptr ? launch_attention_tiles8(a, st) : launch_attention_tiles(a, st);
    return a.ks != nullptr ? launch_attention_rows8(a, st) : launch_attention_rows(a, st);
}

}  // namespace bsa
