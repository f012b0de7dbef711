// attn_split.h -- arithmetic on sizes that the host does before it launches decode
// attention.  Plain C++, no CUDA: a test compiles it by itself.
#pragma once

namespace qre {

// CTAs of the decode kernel on an SM: as many as its registers leave (`most`), fewer where two stages of the ring and what
// a CTA keeps of each query do not fit (1 KB of each is the system's, and the kernel's static arrays).  In 4 bits at
// head_dim 128, of three: beyond 233 queries two (with holes beyond 116), beyond 3476 one.
inline long long decode_room(int ctas, long long max_smem, long long of_queries) {
  return (max_smem + 1024) / ctas - 1024 - 256 - of_queries;
}
inline int decode_ctas(int most, long long max_smem, long long of_queries, long long two_stages) {
  int ctas = most;
  while (ctas > 1 && decode_room(ctas, max_smem, of_queries) < two_stages) --ctas;
  return ctas;
}

// Whether the join of shared prefixes (attn_shared.cu), which counts the places of the sequences' own positions in 31
// bits (64-bit divisions take long there), may join them: n queries with at most `places` each, for each of `units` head
// blocks.  If not, the decode kernel's own join does, a launch of its own that counts in 64 bits.
inline bool shared_join_counts(long long n, long long places, long long units) {
  return n * places <= 0x7fffffffll / units;
}

// Warps of the join for a query head.  Few heads with many parts of the prefix each get more, while SMs have room (two
// CTAs on each); the parts of a unit of unit_rows rows are as many as its share of the `grid` ranges, two of a range where
// its chains take tiles in turn, and a warp has `ahead` on their way.  (16 sequences behind 32,768, us with one warp /
// this: 2 KV heads of 64 50 / 32, 8 of 128 61 / 58; 64 behind 8192 with 2 of 64 29 / 27.)  Without groups nothing is
// shared, and a warp is enough.
inline int shared_join_ways(long long n, int n_heads, int n_kv_heads, int n_groups, int grid, int unit_rows, int ahead) {
  if (n_groups <= 0) return 1;
  const long long heads = n * n_heads, rows = n * (n_heads / n_kv_heads) / n_groups;
  const long long units = (long long)n_groups * n_kv_heads * ((rows + unit_rows - 1) / unit_rows);
  const long long parts = (2 * rows <= unit_rows ? 2 : 1) * grid / (units > 0 ? units : 1);
  int ways = 1;
  while (ways < 8 && parts > (long long)ahead * ways && heads * ways <= 8ll * grid) ways *= 2;
  return ways;
}

}  // namespace qre
