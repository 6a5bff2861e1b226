// Completion counters in workspaces that nobody clears.
#pragma once

#include <cstdint>

namespace mxfp4 {

// Count this CTA into `word` and report whether that made `want`.
// The word holds (epoch << 32) | done; a word tagged with another call's
// epoch (never written, or left by a call that stopped on a timeout) counts
// as zero, so the workspace needs no clearing.  The CTA that completes the
// count resets the word to 0, so a replay of a captured call, which repeats
// the tag, starts from zero too.  Lock-free: each failed exchange means
// another CTA of the tile got its increment in.
__device__ __forceinline__ bool count_done(unsigned long long *word, uint32_t epoch, int want)
{
    unsigned long long cur = atomicAdd(word, 0ull);
    for (;;) {
        const unsigned long long next = (static_cast<uint32_t>(cur >> 32) == epoch)
                                            ? cur + 1ull
                                            : ((static_cast<unsigned long long>(epoch) << 32) | 1ull);
        const unsigned long long prev = atomicCAS(word, cur, next);
        if (prev == cur)
            return static_cast<int>(next & 0xFFFFFFFFull) == want;
        cur = prev;
    }
}

}  // namespace mxfp4
