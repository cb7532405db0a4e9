// What the kernels over the paged cache share: whose tokens a work item has.
#pragma once

#include "bsa_device.cuh"
#include "bsa_internal.h"

namespace bsa {

// The n tokens of a sequence touch at most floor(n / size) + 2 of the runs of
// `size` that its positions are cut into, so sequence s owns the work items
// [c / size + 2 s, c' / size + 2 (s + 1)), c and c' the tokens before and after
// its own: no item list has to be made, and spare items return at once.  The
// same numbers serve runs that start with the sequence's first token.
struct Item {
    int64_t seq, item;        // the sequence and which of its items
    int64_t lo, hi;           // its tokens
};

__device__ __forceinline__ int64_t first_item(const int32_t *cu, int64_t s, int64_t size) {
    return (int64_t(cu[s]) - cu[0]) / size + 2 * s;
}

// The item of number `number`, found by whole warps; false if its sequence's
// bounds make no sense.  Without bounds every sequence has as many tokens, and
// items_each items.
__device__ __forceinline__ bool find_item(const int32_t *cu, int64_t seqs, int64_t tokens,
                                          int64_t size, int64_t items_each, int64_t number, Item *it) {
    if (cu == nullptr) {
        const int64_t n = tokens / seqs;
        it->seq = number / items_each;
        it->item = number - it->seq * items_each;
        it->lo = it->seq * n;
        it->hi = it->lo + n;
        return true;
    }
    // the last sequence whose items start at or before this one: 32-way search,
    // every lane probing one sequence
    int64_t s0 = 0, s1 = seqs;          // in [s0, s1)
    const int lane = threadIdx.x & 31;
    while (s1 - s0 > 1) {
        const int64_t step = (s1 - s0 + 31) / 32;
        const int64_t s = s0 + lane * step;
        const bool at = s < s1 && first_item(cu, s, size) <= number;
        const uint32_t m = __ballot_sync(0xffffffffu, at);
        const int last = m == 0 ? 0 : 31 - __clz(m);
        s0 += last * step;
        s1 = i64min(s1, s0 + step);
    }
    it->seq = s0;
    it->item = number - first_item(cu, s0, size);
    it->lo = cu[s0];
    it->hi = cu[s0 + 1];
    return it->lo >= 0 && it->hi >= it->lo && it->hi <= tokens && it->item >= 0;
}

// Where cu falls, the search may pass over sequences (and over the items of
// others), so each of them is looked at by a thread: `mine` is the thread's
// number in the grid, which has more of them than there are sequences.
__device__ __forceinline__ void check_bounds(const int32_t *cu, int64_t seqs, int64_t tokens,
                                             int64_t mine, int32_t *status) {
    if (cu == nullptr || mine >= seqs) return;
    const int32_t c0 = cu[mine], c1 = cu[mine + 1];
    if (c0 < 0 || c1 < c0 || c1 > tokens) report_status(status, kStatusInvalidArg);
}

// ---- what a new token sees ----------------------------------------------
// Token i of its sequence's n new ones: the keys [lo, hi), the first `sinks`
// of them too where lo > 0, and of the keys from `start` on those whose bit is
// set in `tree`.
struct Sight {
    int32_t lo, hi;
    uint64_t tree;
};

// Without a tree a token is at position start + i and sees the keys up to its
// own.  With one it is at position start + (how many others it sees), and the
// window and the sinks go by positions.
__device__ __forceinline__ Sight sight_of(const AttentionArgs &a, int64_t start, int64_t lo, int n, int i) {
    Sight s;
    if (a.tree == nullptr) {
        s.hi = int32_t(start + i + 1);
        s.lo = a.window > 0 ? int32_t(i64max(0, int64_t(s.hi) - a.window)) : 0;
        s.tree = 0;
        return s;
    }
    const uint64_t all = n < 64 ? (uint64_t(1) << n) - 1 : ~uint64_t(0);
    s.hi = int32_t(start);
    s.lo = 0;
    s.tree = a.tree[lo + i] & all;
    if (a.window > 0) {
        const int depth = __popcll(s.tree & ~(uint64_t(1) << i));
        s.lo = int32_t(i64min(s.hi, i64max(0, start + depth + 1 - a.window)));
        for (uint64_t left = s.tree; left != 0; left &= left - 1) {
            const int j = __ffsll(int64_t(left)) - 1;
            const int other = __popcll(a.tree[lo + j] & all & ~(uint64_t(1) << j));
            if (depth - other >= a.window && start + other >= a.sinks) s.tree &= ~(uint64_t(1) << j);
        }
    }
    return s;
}

// A tile's tokens and the keys they may see: [0, sinks_end) and [first, end).
struct Reach {
    int64_t seq, lo, start;   // the sequence, its first new token, its keys before
    int n, t0, nt;            // its new tokens; the tile's: first and how many
    int32_t sinks_end, first, end;
};

// Tile `number` of `size` tokens; false if there is nothing to do (or, reported,
// nothing that can be done).
__device__ __forceinline__ bool find_reach(const AttentionArgs &a, int size, int64_t items_each,
                                           int64_t number, bool reports, Reach *r) {
    Item it;
    if (!find_item(a.cu, a.seqs, a.tokens, size, items_each, number, &it)) return false;
    const int64_t n = it.hi - it.lo, t0 = it.item * size;
    if (t0 >= n) return false;
    r->seq = it.seq;
    r->lo = it.lo;
    r->start = a.start[it.seq];
    const int64_t end = r->start + n;
    if (r->start < 0 || end > int64_t(a.width) * a.c.page || end > kMostKeys ||
        (a.tree != nullptr && n > kTreeTokens)) {
        if (reports) report_status(a.status, kStatusInvalidArg);
        return false;
    }
    r->n = int(n);
    r->t0 = int(t0);
    r->nt = int(i64min(size, n - t0));
    r->end = int32_t(a.tree != nullptr ? end : r->start + t0 + r->nt);
    r->first = 0;
    r->sinks_end = 0;
    if (a.window > 0) {
        // of the first token, or in a tree of one that sees no other
        r->first = int32_t(i64max(0, r->start + (a.tree != nullptr ? 0 : t0) + 1 - a.window));
        r->sinks_end = min(a.sinks, r->first);
    }
    return true;
}

}  // namespace bsa
