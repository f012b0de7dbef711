// attn_split.h -- arithmetic on sizes that the host does before it launches decode
// attention.  Plain C++, no CUDA: a test compiles it by itself.
#pragma once

namespace qre {

// Whether the join of shared prefixes (attn_shared.cu), which counts the places of the sequences' own positions in 31
// bits (64-bit divisions take long there), may join them: n queries with at most `places` each, for each of `units` head
// blocks.  If not, the decode kernel's own join does, a launch of its own that counts in 64 bits.
inline bool shared_join_counts(long long n, long long places, long long units) {
  return n * places <= 0x7fffffffll / units;
}

}  // namespace qre
