// kv4_counts.cuh -- where a decode step over a cache in 4 bits counts the partial
// states that CTAs leave of a pair they share.  The kernel and the CPU tests
// compile this same header.
//
// A pair's CTAs [c0, c1] are joined in groups of kSub, beginning with c0, and what
// the groups leave in a second step.  The counts lie in the workspace header's words
// behind the status word, which every call leaves at 0, so that a workspace may
// serve any calls.
//   First step: a byte for two CTAs.  A CTA begins one group of two states or more
//   at most, and none inside another group: an even one's that ends in the next CTA
//   has 2 bits, the odd one's, or an even one's that is longer, the upper 5.
//   Second: 5 bits (of 31 groups at most) for each kSub CTAs, of which one begins a
//   pair of more than kSub: the next such pair begins where it ends.
#pragma once

#if defined(__CUDACC__)
#define SPARK_KC __host__ __device__ __forceinline__
#else
#define SPARK_KC inline
#endif

namespace spark {

constexpr int kSub = 16;
constexpr int kMostCtas = 456;
constexpr int kFirstWords = kMostCtas / 8;
constexpr int kCountWords = kFirstWords + (kMostCtas / kSub + 6) / 6;
static_assert(kMostCtas / kSub + 1 <= 31 && kSub < 32, "the counts fit their bits");

// A count of `bits` bits, from bit `shift` of a word on.
struct StateCount {
    int word, shift, bits;
};

// Of group [from, to] of a pair, to > from.
SPARK_KC StateCount kv4_first_count(int from, int to) {
    const int byte = 8 * (from >> 1 & 3);
    const bool upper = (from & 1) || to - from > 1;
    return StateCount{from >> 3, upper ? byte + 3 : byte, upper ? 5 : 2};
}

// Of the groups of a pair that begins in CTA c0.
SPARK_KC StateCount kv4_second_count(int c0) {
    const int at = c0 / kSub;
    return StateCount{kFirstWords + at / 6, 5 * (at % 6), 5};
}

// The group that a CTA of a pair belongs to, and how many the pair has.
struct StateGroup {
    int from, to, groups;
};

SPARK_KC StateGroup kv4_group(int c0, int c1, int cta) {
    StateGroup g;
    g.from = cta - (cta - c0) % kSub;
    g.to = g.from + kSub - 1 < c1 ? g.from + kSub - 1 : c1;
    g.groups = (c1 - c0) / kSub + 1;
    return g;
}

}  // namespace spark
