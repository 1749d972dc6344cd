// Host side of the divided prefill (kda_gdr_tc.cu): which sequences are cut into segments.
// Plain C++ without CUDA, so that the tests can build it alone.
#pragma once

#include <stdint.h>

namespace kda {

constexpr int kSplitChunk = 64;     // tokens of a chunk
constexpr int kSplitSms = 148;      // CTAs at once: a split fills them at most once per launch
constexpr int kMinSplit = 16 * kSplitChunk, kMaxParts = 64;   // tokens of a call; segments of a sequence
constexpr int kSplitCost = 3;                                 // of the two more launches, in chunks

struct SplitBatch {
    int32_t num_seqs, total_tokens, H;
    const int32_t *cu_host;         // host offsets, or nullptr: the lengths are taken as equal
};

// Chunks of sequence n.
inline int chunks_of(const SplitBatch &b, int n)
{
    const int64_t L = b.cu_host ? (int64_t)b.cu_host[n + 1] - b.cu_host[n]
                                : ((int64_t)b.total_tokens + b.num_seqs - 1) / b.num_seqs;
    return (int)((L + kSplitChunk - 1) / kSplitChunk);
}

// Segments of at most `chunks` chunks, for a sequence of n of them.
inline int parts_of(int n, int chunks) { return n > chunks ? (n + chunks - 1) / chunks : 1; }

inline bool may_split(const SplitBatch &b)
{
    return b.num_seqs > 0 && (int64_t)b.H * ((int64_t)b.num_seqs + 1) <= kSplitSms && b.total_tokens >= kMinSplit;
}

// The segment size (in chunks) of the split that ends first, or 0 where whole sequences do.  Both
// launches fit the device once.
inline int plan_split(const SplitBatch &b)
{
    if (!may_split(b)) return 0;
    int lens[kSplitSms], longest = 0;
    for (int n = 0; n < b.num_seqs; ++n) {
        lens[n] = chunks_of(b, n);
        longest = lens[n] > longest ? lens[n] : longest;
    }
    auto fits = [&](int chunks) {
        int64_t first = 0, all = 0;
        for (int n = 0; n < b.num_seqs; ++n) {
            const int P = parts_of(lens[n], chunks);
            if (P > kMaxParts) return false;
            first += P > 1 ? 2 * P - 3 : 0;
            all += P;
        }
        return first * b.H <= kSplitSms && all * b.H <= kSplitSms;
    };
    int lo = 1, hi = longest;      // fits(hi): whole sequences
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (fits(mid)) hi = mid; else lo = mid + 1;
    }
    // In chunks (3.15 us): both passes, a join per segment, and the two more launches.  Slow decays:
    // 32 heads over one sequence of 4096 tokens: 175 us in 3 segments, 216 us whole; 2 heads over
    // 40000: 251 us in 38, 1946 us whole; 1 head over 4096: 223 us in 64 segments, 87 us in 11, 214 us
    // whole; 16 heads over 1100: 58 us in 3, 71 us whole.
    int best = 0, cost = longest;
    for (int P = parts_of(longest, hi); P > 1; --P) {
        // (Not below hi: the longest sequence's even division may cut others into more than fits.)
        const int even = (longest + P - 1) / P, chunks = even > hi ? even : hi, c = 2 * chunks + P + kSplitCost;
        if (c < cost) { best = chunks; cost = c; }
    }
    return best;
}

}  // namespace kda
