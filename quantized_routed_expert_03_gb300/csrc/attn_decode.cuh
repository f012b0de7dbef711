// attn_decode.cuh -- attention of one new token per sequence over the paged cache.
//
// o = sum_j softmax_j(scale q . k_j) v_j over the positions j that the token
// sees, for every head, in one pass over K and V: with the running maximum m and
// sum l (fp32, base 2),
//   m' = max(m, max s), l' = l 2^(m - m') + sum 2^(s - m'), o' alike,
// and the same formula joins parts of a sequence.
//
// Bound: every K and V row is read once, 4 g flops per element (g query heads
// share a KV head), so the memory bounds it, and what counts is how many bytes
// are in flight.
//
// Work split.  A chunk is CK positions of one KV head (K and V, 8 KB together);
// the chunks of all (sequence, KV head) units in a row are cut into equal
// contiguous ranges, one per warp of the grid, whatever the lengths are; a unit
// counts kUnitCost chunks more than it has, its queries, first maximum and result
// (without that, ranges of many short units end last: SMs were idle for 28 % of a
// call with 256 sequences of 1 to 2000 positions).  The
// lengths stay on the device: every CTA sums them up for itself.  A unit that lies
// inside one range is finished there; one that is cut leaves a part (o, m, l in
// fp32) per range in the workspace, and a second, dependent launch joins the
// parts in the order of the ranges, so results do not depend on timing.
// Where max_len or the window says that all units are short, none is cut and there
// is no join launch.  Units of up to two chunks (four when there are more units than
// CTAs) are left whole, each to one warp.  When a unit can have a CTA or a cluster of
// 2, 4 or 8 to itself, its warps share its chunks, up to eight each, and meet in
// shared memory.  The ways that lengths of one size took, 32 heads on 8, D = 128, us:
//   sequences x positions   cut    whole   shared by (warps)
//         1 x   64          9.0     7.4      7.3 (4)
//         1 x  777         10.9    42.4     16.6 (4)  10.4 (16)   9.1 (32)
//         1 x 4096         14.8   202       31.8 (8)  19.8 (16)  14.2 (32)
//         9 x  777         16.3    42.7     12.7 (8)  11.2 (16)  23.5 (32: two waves)
//        16 x 2048         20.1   104       21.3 (8)
//        38 x  256         12.4    17.5     11.0 (4)
//        76 x   64         11.6     8.8     15.3 (4: two waves)
//
// A warp runs on its own, with no barrier (with ranges of CTAs, whose warps met at
// the end of every unit, 256 sequences of up to 1500 positions took 57 us instead
// of 53): it fills a ring of chunks in shared memory with cp.async (16-byte pieces, rows that are not seen zero-filled,
// so what they hold never reaches a product) and multiplies with mma.sync
// (m16n8k16), keys and dimensions on the 16 side, heads on the 8 side:
//   S^T = K Q^T (16 keys x 8 heads), O^T += V^T P^T (16 dimensions x 8 heads);
// P turns from the first product's layout into the second's by one 8 x 8
// transpose (movmatrix).  Nothing is padding with 8 heads per KV head; tcgen05
// would want 128 rows.  More than 16 heads per KV head run as several units over
// the same keys, which then come from L2.
// A unit's first chunk sets the reference of its weights; later ones look for no
// maximum (and shuffle nothing) unless a sum of weights grows too large.
// An E4M3 cache is multiplied as fp16, which holds every E4M3 value; a bf16 query
// is brought into fp16's range by a power of two per head.  So is an E2M1 cache: a
// code times its block's scale has at most 6 bits and lies between 2^-10 and 2688, so
// fp16 holds that product exactly too.
//
// What it measured in 4 bits: 4 sequences of 131,072 positions, 64 heads on 8, D = 128: 130 us, 4.6 TB/s (128 heads:
// 163); 256 of up to 2000, window 1500, 28 on 4, D = 64: 30.8 (56 heads: 37.8).  There the conversions' latency bounds it, not
// the memory: 64 of K and V for 16 keys, as many multiplications by scales, of some 310 instructions; 2.2 instructions a
// cycle come from 3 warps a scheduler, the ALUs are busy for 50 % of the time.  Steps of the first: 176 as the other
// types, 2 CTAs per SM and the halves of V's conversions exchanged; 3 CTAs and whole chunks fetched without a look at
// each row 159; the loader's places kept 154; chunks of 64 keys, the weights spread 134.  4 CTAs (128 registers) need
// chunks of 32 keys: 149.
// Registers that do not fit: 4 to 12 bytes of spills at D = 64 with more than 8 heads per KV head, with holes 20 to 28
// there and 12 at D = 128.  The third CTA of D = 128 needs room beside its ring for what it keeps of each query: beyond
// 233 there are two (256 sequences of 2048: 155 us, 230: 133).
//
// SH: some positions of a query are somebody else's (attn_shared.cu): its hole.
// The result of such a query is a part in fp32, not o.
#pragma once

#include <type_traits>

#include "attn_split.h"
#include "internal.h"
#include "kv_rows.cuh"

namespace qre {
namespace {

constexpr int kWarps = 4;
// (a 4-bit cache is bound by its conversions' latency more than by the memory: three CTAs where registers last for it)
constexpr int ctas_per_sm(int cache_type, int head_dim, bool wide) { return cache_type == QRE_E2M1 && !(head_dim == 128 && wide) ? 3 : 2; }
// Positions of a chunk of a 4-bit cache (D = 64, 256 sequences of up to 2000: 31.2 us with 32, 38.5 with 64).
constexpr int chunk4(int head_dim) { return head_dim == 64 ? 32 : 64; }
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 4096;           // bytes of K (and of V) in a chunk (see Decode)
constexpr int kRows = 16;             // query heads of a unit at most
constexpr int kMaxCtas = 1024;        // of the main kernel
constexpr int kUnitCost = 2;          // chunks that the begin and the end of a unit are worth (see below)
constexpr int kMostWays = 32;         // warps of a cluster of 8 CTAs
constexpr int kMostShare = 8;         // chunks of a warp that shares a unit
constexpr int kMinChunks = 2;         // of a range: fewer would save nothing and leave more parts to join

// What the main kernel leaves for the join, in the workspace.
struct Header {
  long long total;    // places of the call: chunks, and kUnitCost in front of each unit's
  int ranges, pad;
};                    // followed at kFirstsAt by the places before each query's first unit, n + 1 int32
constexpr int kFirstsAt = 256;

__device__ __forceinline__ long long range_begin(int b, int ranges, long long total) { return total * b / ranges; }
// The range that chunk i lies in: the last b with total b / ranges < i + 1.
__device__ __forceinline__ int range_of(long long i, int ranges, long long total) {
  return (int)(((i + 1) * ranges - 1) / total);
}

__device__ __forceinline__ void cp_async_16_zfill(uint32_t dst, const void* src, bool valid) {
  const int bytes = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 8 x 8 transpose of 16-bit elements held as ldmatrix leaves them.
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         const uint32_t (&b)[2]) {
  if (BF)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ void cp_async_16_to(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_8_zfill(uint32_t dst, const void* src, bool valid) {
  const int bytes = valid ? 8 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_4_zfill(uint32_t dst, const void* src, bool valid) {
  const int bytes = valid ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t low_half2(uint32_t a) { return h2_as_u32(__low2half2(u32_as_h2(a))); }
__device__ __forceinline__ uint32_t high_half2(uint32_t a) { return h2_as_u32(__high2half2(u32_as_h2(a))); }
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) { return h2_as_u32(__hmul2(u32_as_h2(a), u32_as_h2(b))); }
// Two E4M3 bytes, the low or the high half of b, as an fp16 pair (the conversion takes either half of a register).
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t b) {
  uint32_t r;
  asm("{.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_high_to_half2(uint32_t b) {
  uint32_t r;
  asm("{.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(b));
  return r;
}

// DT: type of q and o; CT: type of the cache; NH: query heads of a unit in eights.
template <int DT, int CT, int D, int NH>
struct Decode {
  static constexpr bool F8 = CT == QRE_E4M3, F4 = CT == QRE_E2M1;
  static constexpr bool LOW = F8 || F4;           // multiplied as fp16, with a scale per head
  static constexpr bool BF = CT == QRE_BF16;      // type of the products
  static constexpr int RB = F4 ? D / 2 : F8 ? D : 2 * D;   // bytes of a row (of codes)
  static constexpr int SB = F4 ? D / kBlock4 : 0; // bytes of a row's scales, behind the codes of the tile
  static constexpr int CK = F4 ? chunk4(D) : kTile / RB; // positions of a chunk
  static constexpr int CODES = CK * RB;           // bytes of a tile's rows
  static constexpr int TILE = CODES + CK * SB;
  static constexpr int PR = RB / 16;              // 16-byte pieces of a row
  static constexpr int RI = 32 / PR;              // rows that the warp's 32 lanes fetch at once
  static constexpr int NP = CK / 16;              // runs of 16 positions (each inside one page)
  static constexpr int SUBS = F4 ? CK / 32 : 1;        // parts of a chunk that are multiplied one after the other (registers)
  static constexpr int NS = NP / SUBS;
  // How V of an E2M1 cache is multiplied.  A conversion gives two dimensions of one key; the product wants two keys of
  // one dimension.  With one block of heads the weights are spread instead, a zero between two: then the two halves are
  // two steps of the product, and even and odd dimensions are products of their own, twice as many (a quarter of the
  // conversions' instructions less).  With two blocks the products would bound it; the halves are exchanged.
  static constexpr bool SPREAD = F4 && NH == 1;
  static constexpr int KS = D / 16;
  static constexpr int PT = BF ? QRE_BF16 : QRE_FP16;
  // Largest sum of a chunk's weights against a standing reference: fp16 weights end at 65504, and values enter
  // the accumulators times weights of up to this, so that finite ones must not overflow there.
  static constexpr float kMost = 32768.0f;
  // The reference lies this far (base 2) below the maximum that sets it.  fp16 ends at 2^-24 below: with the
  // maximum itself, keys whose weights are under 2^-25 of it would count in the sum and not in O, and in a long
  // sequence they weigh something.  A lane's eight weights of 2^kUp stay under kMost with room for a maximum that grows.
  static constexpr float kUp = BF ? 0.0f : 10.0f;

  // Byte offset of piece `col` of row `row` in a tile: pieces of a 128-byte line
  // are permuted by the row, so the eight rows that ldmatrix reads at one column
  // lie in different banks.
  static __device__ __forceinline__ uint32_t at(int row, int col) {
    return (uint32_t)(row * RB + 16 * (PR >= 8 ? col ^ (row & 7) : PR == 4 ? col ^ ((row >> 1) & 3) : col ^ ((row >> 2) & 1)));
  }
};

// Floats of a part: eight heads at a time by D, and (m, l) of each head.
template <int D, int NH>
constexpr int part_floats() {
  return 8 * NH * (D + 2);
}

// The positions of a query that are computed elsewhere, [from, to) (none: from = to), and where the part over
// its other positions goes: o in fp32 before the division by the sum, the reference (base 2) and the sum.
struct Own {
  const int2* hole;   // [n]
  float* o;           // [n][n_heads][D]
  float2* ml;         // [n][n_heads]
  // The launch before this one in the stream (the prefixes) computes the holes' positions; this one needs nothing of it,
  // only of the ones before.  So it begins where SMs are free already, and its first CTA waits for that launch at its end:
  // then what comes behind this launch comes behind both.  What the ones before wrote it has from the plan: that one waits
  // for all that is older, and its last act is to release *start, the call's token above the number of this kernel's CTAs
  // that have work (the SMs that the prefixes leave).  A thread that acquires the token has seen it all; one that does not
  // waits for the prefixes to end, as any other kernel would.  The plan sets *start to 0 first, and every call has another
  // token (a graph's its own again each time it is replayed, behind that 0), so that an older one is none.  (Released by the prefixes, and the number of CTAs read behind it, calls took 2 us
  // more.)
  int late;
  uint32_t token;
  const unsigned long long* start;   // (read if late)
};

__device__ __forceinline__ void release_start(unsigned long long* p, uint32_t token, int ctas) {
  asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(p), "l"((unsigned long long)token << 32 | (uint32_t)ctas) : "memory");
}
__device__ __forceinline__ unsigned long long acquire_start(const unsigned long long* p) {
  unsigned long long v;
  asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
  return v;
}

template <bool SH>
struct Seq {
  int row, len, first;   // table row, length, places of the queries before (for one unit each)
};
template <>
struct Seq<true> {
  int row, len, first;
  int2 hole;
};

// Keys [lo, hi) that belong to chunk x of a query, and the chunk's first position.
struct Span {
  int pos0, lo, hi;
};
// A query sees [lo, len) but its hole: chunks of what lies before the hole, then of what lies behind it.
template <int CK, bool SH>
struct Seen {
  int lo, len, before, behind;   // before: chunks before the hole; behind: first position behind it
  int from;
  __device__ __forceinline__ Seen(const Seq<SH>& s, int window) {
    len = s.len;
    lo = window > 0 && len > window ? len - window : 0;
    before = 0;
    behind = lo;
    from = lo;
    if constexpr (SH) {
      if (s.hole.y > s.hole.x) {
        from = s.hole.x;
        before = from > lo ? (from + CK - 1) / CK - lo / CK : 0;
        behind = s.hole.y > lo ? s.hole.y : lo;
      }
    }
  }
  __device__ __forceinline__ int chunks() const {
    return before + (len > behind ? (len + CK - 1) / CK - behind / CK : 0);
  }
  __device__ __forceinline__ Span span(int x) const {
    if (SH && x < before) return Span{(lo / CK + x) * CK, lo, from};
    return Span{(behind / CK + x - before) * CK, behind, len};
  }
};

// Parts of four outputs of a unit, with a running maximum and sum: the heads r0 + 2 j of one dimension,
// as they lie in a part (slot: 16 bytes of it).
struct Joined {
  float m[4], l[4], x[4];
  __device__ __forceinline__ Joined() {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      m[j] = -INFINITY;
      l[j] = x[j] = 0.0f;
    }
  }
  __device__ __forceinline__ void add(const float4& y4, const float2 (&e)[4]) {
    const float y[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float to = fmaxf(m[j], e[j].x);
      // what saw nothing (m = -inf) counts nothing; a NaN in l stays one
      const float f = m[j] == to ? 1.0f : ex2(m[j] - to), fe = e[j].x == to ? 1.0f : ex2(e[j].x - to);
      m[j] = to;
      l[j] = l[j] * f + e[j].y * fe;
      x[j] = x[j] * f + y[j] * fe;
    }
  }
  // o = x / l of the j-th head of a slot (and lse, with the head's first dimension)
  template <int DT, int CT, int D, int NH>
  static __device__ __forceinline__ void write(const qre_attn& a, int slot, int j, int t, int h0, int rows, float vs, float M,
                                               float L, float X, uint16_t* o, float* lse, const Own* own) {
    const int reg = slot >> 3, i = (reg >> 2) / NH, high = (reg >> 1) & 1;
    const int r = 8 * ((reg >> 2) % NH) + (reg & 1) + 2 * j;
    const int d = CT == QRE_E2M1 ? 32 * (i >> 1) + 4 * (slot & 7) + (NH == 1 ? (i & 1) + 2 * high : 2 * (i & 1) + high)
                                 : 16 * i + (CT == QRE_E4M3 ? 2 * (slot & 7) + high : (slot & 7) + 8 * high);
    if (r >= rows) return;
    if (own) {
      own->o[((size_t)t * a.n_heads + h0 + r) * D + d] = X * vs;
      if (d == 0) own->ml[(size_t)t * a.n_heads + h0 + r] = make_float2(M, L);
      return;
    }
    o[(size_t)t * a.o_token + (size_t)(h0 + r) * a.o_head + d] =
        (uint16_t)pack2<DT>(L == 0.0f ? 0.0f : X * (vs / L), 0.0f);
    if (lse && d == 0) lse[(size_t)t * a.n_heads + h0 + r] = L == 0.0f ? -INFINITY : M * kLn2 + logf(L);
  }
};

__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();   // the aligned form wants the whole warp
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// What lies at a shared address in CTA `rank` of the cluster.
__device__ __forceinline__ float4 peer_float4(uint32_t addr, int rank) {
  float4 r;
  asm volatile("{.reg .b32 p;\n\tmapa.shared::cluster.u32 p, %4, %5;\n\tld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [p];\n\t}"
               : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w)
               : "r"(addr), "r"(rank)
               : "memory");
  return r;
}
__device__ __forceinline__ float2 peer_float2(uint32_t addr, int rank) {
  float2 r;
  asm volatile("{.reg .b32 p;\n\tmapa.shared::cluster.u32 p, %2, %3;\n\tld.shared::cluster.v2.f32 {%0, %1}, [p];\n\t}"
               : "=f"(r.x), "=f"(r.y)
               : "r"(addr), "r"(rank)
               : "memory");
  return r;
}

template <int DT, int CT, int D, int NH, bool SH>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(CT, D, NH > 1))
    attn_decode_kernel(const __grid_constant__ qre_attn a, const __grid_constant__ qre_kv_cache c, int layer, int n,
                       const int32_t* __restrict__ seqs, int row0, const uint16_t* __restrict__ q, uint16_t* __restrict__ o,
                       float* __restrict__ lse, Header* __restrict__ header, float* __restrict__ parts, int stages,
                       int ways, const __grid_constant__ Own own, int* status) {
  using K = Decode<DT, CT, D, NH>;
  using Seq = Seq<SH>;
  constexpr int CK = K::CK, KS = K::KS;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem + (size_t)(threadIdx.x >> 5) * stages * 2 * K::TILE;   // this warp's
  Seq* sq = reinterpret_cast<Seq*>(smem + (size_t)kWarps * stages * 2 * K::TILE);   // [n + 1]
  __shared__ int scan_part[kWarps];
  __shared__ int scan_total;
  __shared__ int has_part[kWarps];
  __shared__ float2 joined[8 * NH];   // (m, l) of the heads
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = a.n_heads / a.n_kv_heads;
  const int blocks = (g + kRows - 1) / kRows;       // head blocks of a KV head
  const int units = a.n_kv_heads * blocks;          // units of a sequence
  const int ps_shift = 31 - __clz(c.page_size);

  // (late: see Own)
  const bool late = SH && own.late;
  int work_ctas = (int)gridDim.x;
  if (late) {
    unsigned long long start = acquire_start(own.start);
    if ((uint32_t)(start >> 32) != own.token) {
      grid_dependency_wait();
      start = acquire_start(own.start);
    }
    work_ctas = (int)(uint32_t)start;
  } else {
    grid_dependency_wait();
  }
  grid_dependents_launch();
  auto leave = [&]() {
    if (SH && late && blockIdx.x == 0) grid_dependency_wait();
  };
  int grid = (int)gridDim.x;
  if constexpr (SH) {
    if (late && ways <= 1) grid = max(1, min(work_ctas, grid));
    if ((int)blockIdx.x >= grid) return;   // never the first, which waits for the launch before
  }

  // ---- the plan: chunks of every query, summed up
  constexpr int kEach = 4;   // queries of a thread at a time: their loads are in flight together
  int before = 0;
  for (int t0 = 0; t0 < n; t0 += kEach * kThreads) {
    int row[kEach], len[kEach], ch[kEach], mine = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int t = t0 + kEach * tid + i;
      row[i] = t < n ? (seqs ? seqs[t] : row0 + t) : -1;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) len[i] = row[i] >= 0 && row[i] < c.max_seqs ? c.seq_len[row[i]] : -1;
    int2 hole[SH ? kEach : 1];
    if constexpr (SH)
#pragma unroll
      for (int i = 0; i < kEach; ++i) hole[i] = t0 + kEach * tid + i < n ? own.hole[t0 + kEach * tid + i] : make_int2(0, 0);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (len[i] < 0 || len[i] > (long long)c.max_pages * c.page_size) {
        if (blockIdx.x == 0 && t0 + kEach * tid + i < n) set_status(status, QRE_DEV_BAD_INDEX);
        len[i] = row[i] = 0;
      }
      Seq s{};
      s.len = len[i];
      if constexpr (SH) s.hole = hole[i];
      const int chunks = Seen<CK, SH>(s, a.window).chunks();
      ch[i] = chunks > 0 ? chunks + kUnitCost : 0;
      mine += ch[i];
    }
    int inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += u;
    }
    if (lane == 31) scan_part[warp] = inc;
    __syncthreads();
    int first = before + inc - mine;
    for (int w = 0; w < warp; ++w) first += scan_part[w];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int t = t0 + kEach * tid + i;
      if (t < n) {
        sq[t].row = row[i];
        sq[t].len = len[i];
        sq[t].first = first;
        if constexpr (SH) sq[t].hole = hole[i];
      }
      first += ch[i];
    }
    if (tid == kThreads - 1) scan_total = first;
    __syncthreads();
    before = scan_total;
  }
  if (tid == 0) sq[n].first = before;
  __syncthreads();
  const long long total = (long long)before * units;
  const bool together = ways > 1;   // a cluster has one unit, `ways` warps share its chunks
  const long long want = ways ? (long long)n * units : (total + kMinChunks - 1) / kMinChunks;
  const long long all = (long long)grid * kWarps;
  const int ranges = (int)(together ? all : want < all ? want : all);
  // this warp's range: few ranges spread over the SMs
  const int me = together ? (int)blockIdx.x * kWarps + warp : warp * grid + (int)blockIdx.x;
  // the place at which range b begins: any, or a unit's first, or one of `ways` shares of a unit
  auto begin = [&](int b) {
    if (!ways) return range_begin(b, ranges, total);
    const long long u = together ? b / ways : (long long)n * units * b / ranges;
    const int t = (int)(u / units);
    if (t >= n) return total;
    const int nch = sq[t + 1].first - sq[t].first, i = together ? b % ways : 0;
    return (long long)sq[t].first * units + (u - (long long)t * units) * nch +
           (i && nch ? kUnitCost + (long long)(nch - kUnitCost) * i / ways : 0);
  };

  // queries that see nothing
  for (int t = blockIdx.x; t < n; t += grid) {
    if (sq[t + 1].first != sq[t].first) continue;
    if constexpr (SH) {
      if (sq[t].hole.y > sq[t].hole.x) {   // what it sees is all in its hole
        for (int i = tid; i < a.n_heads * (D / 4); i += kThreads)
          reinterpret_cast<float4*>(own.o + (size_t)t * a.n_heads * D)[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int h = tid; h < a.n_heads; h += kThreads) own.ml[(size_t)t * a.n_heads + h] = make_float2(-INFINITY, 0.0f);
        continue;
      }
    }
    for (int i = tid; i < a.n_heads * (D / 8); i += kThreads) {
      const int h = i / (D / 8), d = (i - h * (D / 8)) * 8;
      *reinterpret_cast<uint4*>(o + (size_t)t * a.o_token + (size_t)h * a.o_head + d) = make_uint4(0, 0, 0, 0);
    }
    if (lse)
      for (int h = tid; h < a.n_heads; h += kThreads) lse[(size_t)t * a.n_heads + h] = -INFINITY;
  }
  if (blockIdx.x == 0 && !ways) {
    if (tid == 0) *header = Header{total, ranges, 0};
    int32_t* firsts = reinterpret_cast<int32_t*>(reinterpret_cast<char*>(header) + kFirstsAt);
    for (int t = tid; t <= n; t += kThreads) firsts[t] = sq[t].first;
  }
  if (me >= ranges) {
    leave();
    return;
  }
  const long long c0 = begin(me), c1 = begin(me + 1);
  if (c0 >= c1 && !together) {
    leave();
    return;
  }

  if (together && lane == 0) has_part[warp] = 0;
  __syncwarp();
  if (c0 < c1) {   // (always, unless together)
  // the query that chunk c0 belongs to
  int t_first;
  {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if ((long long)sq[mid].first * units <= c0) lo = mid;
      else hi = mid - 1;
    }
    t_first = lo;   // the last one that begins at or before c0: it has chunks
  }

  // A place in the list: place ck of nch of the unit; its chunks begin at place kUnitCost.
  struct Place {
    int t, unit, ck, nch;
  };
  auto place_of = [&](long long i, int t) {
    while ((long long)sq[t + 1].first * units <= i) ++t;
    Place p;
    p.t = t;
    p.nch = sq[t + 1].first - sq[t].first;
    const long long rest = i - (long long)sq[t].first * units;
    p.unit = (int)(rest / p.nch);
    p.ck = (int)(rest - (long long)p.unit * p.nch);
    return p;
  };
  auto advance = [&](Place& p, int by) {   // not past the end of the list
    p.ck += by;
    while (p.ck >= p.nch) {
      p.ck -= p.nch;
      if (++p.unit == units) {
        p.unit = 0;
        do {
          ++p.t;
          if (p.t >= n) return;
          p.nch = sq[p.t + 1].first - sq[p.t].first;
        } while (p.nch == 0);
      }
    }
  };

  // ---- loader
  long long li = c0;                 // place of the next chunk to fetch
  Place lp = place_of(li, t_first);
  auto to_chunk = [&]() {
    if (lp.ck < kUnitCost) {
      li += kUnitCost - lp.ck;
      lp.ck = kUnitCost;
    }
  };
  to_chunk();
  // E2M1, where the loader's arithmetic counts: what holds for the unit that is fetched
  long long code_at = 0;             // lane j: byte of run j's codes in the pool
  Span load_span = {};               // of chunk li
  int load_jump = -1;                // the chunk behind the hole
  const int32_t* load_row = nullptr;
  long long load_head = 0;           // byte of the KV head in page 0
  const size_t head_bytes = (size_t)c.page_size * (K::RB + K::SB);
  const long long page_bytes = (long long)c.n_kv_heads * (long long)head_bytes;
  auto enter = [&]() {
    const Seen<CK, SH> se(sq[lp.t], a.window);
    load_span = se.span(lp.ck - kUnitCost);
    if (SH) load_jump = se.before > 0 ? se.before + kUnitCost : -1;
    load_row = c.page_table + (size_t)sq[lp.t].row * c.max_pages;
    load_head = (long long)layer * c.n_pages * page_bytes + (long long)(lp.unit / blocks) * (long long)head_bytes;
  };
  if constexpr (K::F4)
    if (li < c1) enter();
  int pages = 0;                     // lane j: page of positions 16 j .. 16 j + 15 of that chunk, -1 missing, -2 not seen
  auto look_up = [&]() {
    pages = -2;
    if (li < c1 && lane < K::NP) {
      const Span sp = K::F4 ? load_span : Seen<CK, SH>(sq[lp.t], a.window).span(lp.ck - kUnitCost);
      const int pos = sp.pos0 + 16 * lane;
      if (pos < sp.hi && pos + 16 > sp.lo) {
        pages = K::F4 ? load_row[pos >> ps_shift] : c.page_table[(size_t)sq[lp.t].row * c.max_pages + (pos >> ps_shift)];
        if (pages < 0 || pages >= c.n_pages) {
          pages = -1;
          set_status(status, QRE_DEV_BAD_INDEX);
        }
      }
      if constexpr (K::F4) code_at = load_head + pages * page_bytes + (pos & (c.page_size - 1)) * K::RB;
    }
  };
  const uint8_t* pool_k = static_cast<const uint8_t*>(c.k);
  const uint8_t* pool_v = static_cast<const uint8_t*>(c.v);
  uint32_t missing = 0;              // bit NP * slot + j: run j of that ring slot has no page
  auto fetch = [&](int slot) {       // fetches chunk li into the slot and moves on
    if (li < c1) {
      const Span sp = K::F4 ? load_span : Seen<CK, SH>(sq[lp.t], a.window).span(lp.ck - kUnitCost);
      const int pos0 = sp.pos0, lo = sp.lo, len = sp.hi;
      const uint32_t gone = __ballot_sync(0xffffffffu, pages == -1);
      missing = (missing & ~(((1u << K::NP) - 1u) << (K::NP * slot))) | (gone << (K::NP * slot));
      const uint32_t dst = smem_addr(ring + (size_t)slot * 2 * K::TILE);
      const int r0 = lane / K::PR, col = lane % K::PR;
      if (K::F4 && !gone && pos0 >= lo && pos0 + CK <= len) {   // all of it is seen: the loader's arithmetic counts here
#pragma unroll
        for (int j = 0; j < K::NP; ++j) {
          const long long at = __shfl_sync(0xffffffffu, code_at, j);
          const int row0 = (pos0 + 16 * j) & (c.page_size - 1);
          const uint8_t *ck = pool_k + at + (r0 * K::RB + 16 * col), *cv = pool_v + at + (r0 * K::RB + 16 * col);
#pragma unroll
          for (int r = 0; r < 16; r += K::RI) {
            cp_async_16_to(dst + K::at(16 * j + r + r0, col), ck + r * K::RB);
            cp_async_16_to(dst + K::TILE + K::at(16 * j + r + r0, col), cv + r * K::RB);
          }
          const uint8_t* sc = (lane < 16 ? pool_k : pool_v) + at + (c.page_size * K::RB - row0 * (K::RB - K::SB) + (lane & 15) * K::SB);
          const uint32_t to = dst + (lane < 16 ? 0 : K::TILE) + K::CODES + (16 * j + (lane & 15)) * K::SB;
          if (K::SB == 8) cp_async_8_zfill(to, sc, true);
          else cp_async_4_zfill(to, sc, true);
        }
      } else {
        const int hk = lp.unit / blocks;
#pragma unroll
        for (int j = 0; j < K::NP; ++j) {
          const int page = __shfl_sync(0xffffffffu, pages, j);
          const int row0 = (pos0 + 16 * j) & (c.page_size - 1);
          const size_t head = page < 0 ? 0 : (((size_t)layer * c.n_pages + page) * c.n_kv_heads + hk) * head_bytes;
          const size_t base = page < 0 ? 0 : head + (size_t)row0 * K::RB;
#pragma unroll
          for (int r = 0; r < 16; r += K::RI) {
            const int row = 16 * j + r + r0, pos = pos0 + row;
            const bool ok = page >= 0 && pos >= lo && pos < len;
            const size_t off = ok ? base + (size_t)((r + r0) * K::RB + 16 * col) : 0;
            cp_async_16_zfill(dst + K::at(row, col), pool_k + off, ok);
            cp_async_16_zfill(dst + K::TILE + K::at(row, col), pool_v + off, ok);
          }
          if constexpr (K::F4) {   // the scales: a row a lane, 16 of K and 16 of V
            const int r = lane & 15, pos = pos0 + 16 * j + r;
            const bool ok = page >= 0 && pos >= lo && pos < len;
            const size_t off = ok ? head + (size_t)c.page_size * K::RB + (size_t)(row0 + r) * K::SB : 0;
            const uint32_t to = dst + (lane < 16 ? 0 : K::TILE) + K::CODES + (16 * j + r) * K::SB;
            const uint8_t* pool = lane < 16 ? pool_k : pool_v;
            if (K::SB == 8) cp_async_8_zfill(to, pool + off, ok);
            else cp_async_4_zfill(to, pool + off, ok);
          }
        }
      }
      ++li;
      if (li < c1) {
        if (K::F4 && lp.ck + 1 < lp.nch) {
          if (++lp.ck == load_jump) enter();
          else load_span.pos0 += CK;
        } else {
          advance(lp, 1);
          to_chunk();
          if constexpr (K::F4) enter();
        }
      }
      look_up();
    }
    cp_async_commit();
  };
  look_up();
  for (int s = 0; s < stages - 1; ++s) fetch(s);
  int slot_in = stages - 1, slot = 0;

  // ---- the units of this range, one after the other
  const size_t si = (size_t)layer * c.n_kv_heads;
  const int r4 = lane >> 2, j4 = lane & 3;
  // A unit's queries as the B operand: head 8 nh + lane / 4, zero beyond the unit's heads.  The words
  // are asked for one unit ahead.
  uint32_t qw[KS][NH][2];
  auto heads_of = [&](const Place& p, int& hk, int& h0) {
    hk = p.unit / blocks;
    h0 = hk * g + (p.unit - hk * blocks) * kRows;
    return (hk + 1) * g - h0 < kRows ? (hk + 1) * g - h0 : kRows;
  };
  auto ask_queries = [&](const Place& p) {
    int hk, h0;
    const int rows = heads_of(p, hk, h0);
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
      const int r = 8 * nh + r4;
      const uint16_t* qr = q + (size_t)p.t * a.q_token + (size_t)(h0 + (r < rows ? r : 0)) * a.q_head;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        if (K::F4) {   // of the E2M1 products: k = 2 j + e is dimension 8 j + e of 32, 8 + 2 j + e is 8 j + 2 + e; then 4 further
          const uint2 x = *reinterpret_cast<const uint2*>(qr + 32 * (k / 2) + 8 * j4 + 4 * (k & 1));
          qw[k][nh][0] = r < rows ? x.x : 0;
          qw[k][nh][1] = r < rows ? x.y : 0;
        } else if (K::F8) {   // element order of the E4M3 products: k = 2 j + e is dimension 4 j + e, 8 + 2 j + e is 4 j + 2 + e
          const uint2 x = *reinterpret_cast<const uint2*>(qr + 16 * k + 4 * j4);
          qw[k][nh][0] = r < rows ? x.x : 0;
          qw[k][nh][1] = r < rows ? x.y : 0;
        } else {
          const uint32_t x = *reinterpret_cast<const uint32_t*>(qr + 16 * k + 2 * j4);
          const uint32_t y = *reinterpret_cast<const uint32_t*>(qr + 16 * k + 8 + 2 * j4);
          qw[k][nh][0] = r < rows ? x : 0;
          qw[k][nh][1] = r < rows ? y : 0;
        }
      }
    }
  };
  long long s0 = c0;
  Place cp = place_of(c0, t_first);
  ask_queries(cp);
  while (s0 < c1) {
    const long long u0 = s0 - cp.ck, u1 = u0 + cp.nch, k0 = u0 + kUnitCost;   // k0: its first chunk
    const long long s1 = u1 < c1 ? u1 : c1;
    const int t = cp.t;
    int hk, h0;
    const int rows = heads_of(cp, hk, h0);
    const Seen<CK, SH> seen(sq[t], a.window);
    const float ks = K::LOW && c.k_scale ? c.k_scale[si + hk] : 1.0f;
    const float vs = K::LOW && c.v_scale ? c.v_scale[si + hk] : 1.0f;

    uint32_t qb[KS][NH][2];
    float s2[NH][2];                 // score factor of heads 2 j and 2 j + 1, base 2
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
      float own = a.scale * kLog2e * ks;   // of head lane / 4
      float f = 1.0f;
      if (K::LOW && DT == QRE_BF16) {
        float big = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            big = fmaxf(big, fmaxf(fabsf(bits_to_float<DT>(qw[k][nh][e] & 0xffffu)), fabsf(bits_to_float<DT>(qw[k][nh][e] >> 16))));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // largest element to [2^14, 2^15): exact but for elements 2^-29 times smaller, which round to 2^-39 of it
        const int e = (int)((__float_as_uint(big) >> 23) & 255) - 127;
        const int up = e >= 128 || big == 0.0f ? 0 : (14 - e < 126 ? 14 - e : 126);
        f = __uint_as_float((uint32_t)(up + 127) << 23);
        own *= __uint_as_float((uint32_t)(127 - up) << 23);
      }
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          qb[k][nh][e] = K::LOW && DT == QRE_BF16
                             ? pack2<QRE_FP16>(bits_to_float<DT>(qw[k][nh][e] & 0xffffu) * f, bits_to_float<DT>(qw[k][nh][e] >> 16) * f)
                             : qw[k][nh][e];
      s2[nh][0] = __shfl_sync(0xffffffffu, own, 8 * j4);
      s2[nh][1] = __shfl_sync(0xffffffffu, own, 8 * j4 + 4);
    }

    Place np = cp;                   // the next unit: its queries come meanwhile
    if (s1 < c1) {
      advance(np, (int)(s1 - s0));
      ask_queries(np);
    }

    float acc[D / 16][NH][4];        // O^T: dimensions by heads 2 j, 2 j + 1
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) acc[i][nh][0] = acc[i][nh][1] = acc[i][nh][2] = acc[i][nh][3] = 0.0f;
    float m[NH][2], l[NH][2];        // reference (base 2) and this lane's share of the sum
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
      m[nh][0] = m[nh][1] = -INFINITY;
      l[nh][0] = l[nh][1] = 0.0f;
    }

    for (long long next = s0 < k0 ? k0 : s0; next < s1; ++next) {
      fetch(slot_in);
      slot_in = slot_in + 1 == stages ? 0 : slot_in + 1;
      if (stages == 2) cp_async_wait_group<1>();
      else cp_async_wait_group<2>();
      __syncwarp();
      const uint32_t tile = smem_addr(ring + (size_t)slot * 2 * K::TILE);
      const int m8 = lane >> 3, l8 = lane & 7;
      const Span sp = seen.span((int)(next - k0));
      const uint32_t gone = (missing >> (K::NP * slot)) & ((1u << K::NP) - 1u);
      const bool cut = sp.pos0 < sp.lo || sp.pos0 + CK > sp.hi || gone;

#pragma unroll 1
      for (int sub = 0; sub < K::SUBS; ++sub) {
        const uint32_t kt = tile + sub * 16 * K::NS * K::RB, vt = kt + K::TILE;
        const uint32_t kst = tile + K::CODES + sub * 16 * K::NS * K::SB, vst = kst + K::TILE;
        // E2M1: the scales of a key's row.  Bytes 2 p and 2 p + 1 are of piece p; a lane's dimensions have one of them
        uint2 ksc[K::F4 ? K::NS : 1][2];
        const uint32_t ksel = (uint32_t)(j4 >> 1) * 0x11u + 0x20u;
        auto scales_of = [&](const uint2& row, int p) {   // of pieces p and p + 1
          return e4m3x2_to_half2(__byte_perm(p < 2 ? row.x : row.y, 0, ksel));
        };
        if constexpr (K::F4) {
#pragma unroll
          for (int i = 0; i < K::NS; ++i)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const uint32_t at = kst + (16 * i + 8 * b + r4) * K::SB;
              ksc[i][b] = K::SB == 8 ? lds64(at) : make_uint2(lds32(at), 0);
            }
        }

        float s[K::NS][NH][4];
#pragma unroll
        for (int i = 0; i < K::NS; ++i) {
#pragma unroll
          for (int nh = 0; nh < NH; ++nh) s[i][nh][0] = s[i][nh][1] = s[i][nh][2] = s[i][nh][3] = 0.0f;
          // pieces p and p + 1 of 16 keys: keys 0-7 and 8-15 of each
#pragma unroll
          for (int p = 0; p < K::PR; p += 2) {
            uint32_t x[4];
            ldmatrix_x4(x, kt + K::at(16 * i + 8 * (m8 & 1) + l8, p + (m8 >> 1)));
            if constexpr (K::F4) {
              // a register has 8 codes of key lane / 4 (or 8 more), dimensions 32 p + 8 j and on: two steps of the product
              const uint32_t s0 = scales_of(ksc[i][0], p), s1 = scales_of(ksc[i][1], p);
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                // (one half for both: the multiplication takes it so)
                const uint32_t sa = b ? high_half2(s0) : low_half2(s0), sb = b ? high_half2(s1) : low_half2(s1);
                uint32_t ya[4], yb[4];
                e2m1x8_to_half2(x[2 * b], ya);
                e2m1x8_to_half2(x[2 * b + 1], yb);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t a0 = mul_half2(ya[2 * e], sa), a1 = mul_half2(yb[2 * e], sb);
                  const uint32_t a2 = mul_half2(ya[2 * e + 1], sa), a3 = mul_half2(yb[2 * e + 1], sb);
#pragma unroll
                  for (int nh = 0; nh < NH; ++nh) mma16816<false>(s[i][nh], a0, a1, a2, a3, qb[2 * (p + b) + e][nh]);
                }
              }
            } else {
#pragma unroll
              for (int nh = 0; nh < NH; ++nh) {
                if (!K::F8) {
                  mma16816<K::BF>(s[i][nh], x[0], x[1], x[2], x[3], qb[p / 2][nh]);
                } else {
                  mma16816<false>(s[i][nh], e4m3x2_to_half2(x[0]), e4m3x2_to_half2(x[1]),
                                  e4m3x2_high_to_half2(x[0]), e4m3x2_high_to_half2(x[1]), qb[p][nh]);
                  mma16816<false>(s[i][nh], e4m3x2_to_half2(x[2]), e4m3x2_to_half2(x[3]),
                                  e4m3x2_high_to_half2(x[2]), e4m3x2_high_to_half2(x[3]), qb[p + 1][nh]);
                }
              }
            }
          }
        }

        if (cut) {                     // what is not seen: -inf
#pragma unroll
          for (int i = 0; i < K::NS; ++i)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const int run = sub * K::NS + i, pos = sp.pos0 + 16 * run + 4 * e + r4;
              if (pos < sp.lo || pos >= sp.hi || ((gone >> run) & 1u)) {
#pragma unroll
                for (int nh = 0; nh < NH; ++nh) s[i][nh][e] = s[i][nh][e + 1] = -INFINITY;
              }
            }
        }
        float p[K::NS][NH][4], sum[NH][2];
        auto weights = [&]() {
#pragma unroll
          for (int nh = 0; nh < NH; ++nh) {
            sum[nh][0] = sum[nh][1] = 0.0f;
#pragma unroll
            for (int i = 0; i < K::NS; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float mm = m[nh][e & 1];
                p[i][nh][e] = ex2(fmaf(s[i][nh][e], s2[nh][e & 1], mm == -INFINITY ? 0.0f : -mm));
                sum[nh][e & 1] += p[i][nh][e];
              }
          }
        };
        weights();
        bool redo = false;
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int e = 0; e < 2; ++e) redo |= m[nh][e] == -INFINITY || sum[nh][e] > K::kMost;
        if (__any_sync(0xffffffffu, redo)) {   // the reference moves with the maximum so far
#pragma unroll
          for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mx = -INFINITY;
#pragma unroll
              for (int i = 0; i < K::NS; ++i) mx = fmaxf(mx, fmaxf(s[i][nh][e], s[i][nh][e + 2]));
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
              const float to = fmaxf(m[nh][e], mx * s2[nh][e] - K::kUp);
              const float f = m[nh][e] == to ? 1.0f : ex2(m[nh][e] - to);   // 2^-inf = 0 for the first keys
              m[nh][e] = to;
              l[nh][e] *= f;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                acc[i][nh][e] *= f;
                acc[i][nh][e + 2] *= f;
              }
            }
          weights();
        }
        // O^T += V^T P^T: the weights are rounded to the products' type (the sum l keeps them in fp32)
#pragma unroll
        for (int i = 0; i < K::NS; ++i) {
          uint32_t pb[NH][2];
#pragma unroll
          for (int nh = 0; nh < NH; ++nh) {
            pb[nh][0] = movmatrix(pack2<K::PT>(p[i][nh][0], p[i][nh][1]));
            pb[nh][1] = movmatrix(pack2<K::PT>(p[i][nh][2], p[i][nh][3]));
          }
          uint32_t spread[K::SPREAD ? 2 : 1][2][2];   // [keys 0-7, 8-15][even, odd dimensions]: step 2 j is key 2 j, 2 j + 8 key 2 j + 1
          if constexpr (K::SPREAD) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              spread[b][0][0] = pb[0][b] & 0xffffu;
              spread[b][0][1] = pb[0][b] >> 16;
              spread[b][1][0] = pb[0][b] << 16;
              spread[b][1][1] = pb[0][b] & 0xffff0000u;
            }
          }
          // E2M1: the scales of keys 2 j and 2 j + 1 (and of 8 further), a row each
          uint4 vsc[K::F4 ? 2 : 1];
          auto pair_scale = [&](const uint4& w, int p) {   // of the piece's dimensions 4 r .. 4 r + 3
            const uint32_t sel = (uint32_t)(r4 >> 2) * 0x11u + 0x40u + (p & 1 ? 0x22u : 0u);
            return e4m3x2_to_half2(__byte_perm(p < 2 ? w.x : w.y, p < 2 ? w.z : w.w, sel));
          };
          if constexpr (K::F4) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const uint32_t at = vst + (16 * i + 8 * b + 2 * j4) * K::SB;
              if (K::SB == 8) {
                vsc[b] = lds128(at);
              } else {
                const uint2 w = lds64(at);
                vsc[b] = make_uint4(w.x, 0, w.y, 0);
              }
            }
          }
#pragma unroll
          for (int d = 0; d < K::PR; d += 2) {
            uint32_t x[4];
            if constexpr (K::F4) {
              // as for E4M3, with four codes for two values: a register has keys 2 j, 2 j + 1 of dimensions 4 r .. 4 r + 3
              // of the piece's 32.  Row r of the first product is dimension 4 r, row r + 8 the next, of the second 4 r + 2,
              // 4 r + 3; with the weights spread 4 r and 4 r + 2 of the first, 4 r + 1 and 4 r + 3 of the second
              ldmatrix_x4_trans(x, vt + K::at(16 * i + 8 * (m8 & 1) + l8, d + (m8 >> 1)));
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                if constexpr (K::SPREAD) {
#pragma unroll
                  for (int b = 0; b < 2; ++b) {   // keys 0-7 or 8-15
                    const uint32_t sc = pair_scale(vsc[b], d + e), s0 = low_half2(sc), s1 = high_half2(sc);
                    uint32_t u[4];     // dimensions 4 r, 4 r + 1 and 4 r + 2, 4 r + 3 of key 2 j, then of key 2 j + 1
                    e2m1x8_to_half2(x[2 * e + b], u);
                    const uint32_t a0 = mul_half2(u[0], s0), a1 = mul_half2(u[1], s0), a2 = mul_half2(u[2], s1), a3 = mul_half2(u[3], s1);
                    mma16816<false>(acc[2 * (d + e)][0], a0, a1, a2, a3, spread[b][0]);
                    mma16816<false>(acc[2 * (d + e) + 1][0], a0, a1, a2, a3, spread[b][1]);
                  }
                } else {
                  uint32_t y[2][2][2];   // keys 0-7 or 8-15, product, row r or r + 8
#pragma unroll
                  for (int b = 0; b < 2; ++b) {
                    const uint32_t sc = pair_scale(vsc[b], d + e);
                    uint32_t u[4];       // dimensions 4 r, 4 r + 1 and 4 r + 2, 4 r + 3 of key 2 j, then of key 2 j + 1
                    e2m1x8_to_half2(x[2 * e + b], u);
#pragma unroll
                    for (int m2 = 0; m2 < 2; ++m2) {
                      y[b][m2][0] = mul_half2(__byte_perm(u[m2], u[m2 + 2], 0x5410), sc);
                      y[b][m2][1] = mul_half2(__byte_perm(u[m2], u[m2 + 2], 0x7632), sc);
                    }
                  }
#pragma unroll
                  for (int m2 = 0; m2 < 2; ++m2)
#pragma unroll
                    for (int nh = 0; nh < NH; ++nh)
                      mma16816<false>(acc[2 * (d + e) + m2][nh], y[0][m2][0], y[0][m2][1], y[1][m2][0], y[1][m2][1], pb[nh]);
                }
              }
            } else if (!K::F8) {
              // 16 dimensions: pieces d and d + 1 of keys 0-7, then of keys 8-15
              ldmatrix_x4_trans(x, vt + K::at(16 * i + 8 * (m8 >> 1) + l8, d + (m8 & 1)));
#pragma unroll
              for (int nh = 0; nh < NH; ++nh) mma16816<K::BF>(acc[d / 2][nh], x[0], x[1], x[2], x[3], pb[nh]);
            } else {
              // piece d of keys 0-7 and 8-15, then piece d + 1; a register holds keys 2 j, 2 j + 1 of dimensions
              // 2 r, 2 r + 1: row r of the product is dimension 2 r, row r + 8 dimension 2 r + 1
              ldmatrix_x4_trans(x, vt + K::at(16 * i + 8 * (m8 & 1) + l8, d + (m8 >> 1)));
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t y0 = __byte_perm(x[2 * e], 0, 0x3120), y1 = __byte_perm(x[2 * e + 1], 0, 0x3120);
                const uint32_t a0 = e4m3x2_to_half2(y0), a1 = e4m3x2_high_to_half2(y0);
                const uint32_t a2 = e4m3x2_to_half2(y1), a3 = e4m3x2_high_to_half2(y1);
#pragma unroll
                for (int nh = 0; nh < NH; ++nh) mma16816<false>(acc[d + e][nh], a0, a1, a2, a3, pb[nh]);
              }
            }
          }
        }
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
          l[nh][0] += sum[nh][0];
          l[nh][1] += sum[nh][1];
        }
      }
      slot = slot + 1 == stages ? 0 : slot + 1;
      __syncwarp();
    }

    // ---- end of the unit in this range
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nh][e] += __shfl_xor_sync(0xffffffffu, l[nh][e], d);
    bool holed = false;
    if constexpr (SH) holed = sq[t].hole.y > sq[t].hole.x;
    if (s1 <= k0) {               // none of its chunks
    } else if (SH && holed && !together && s0 <= k0 && s1 == u1) {   // whole, and a part of a query
#pragma unroll
      for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * nh + 2 * j4 + e;
          if (r >= rows) continue;
          float* out = own.o + ((size_t)t * a.n_heads + h0 + r) * D;
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int high = 0; high < 2; ++high) {
              const int d = K::F4 ? 32 * (i >> 1) + 4 * r4 + (K::SPREAD ? (i & 1) + 2 * high : 2 * (i & 1) + high) : 16 * i + (K::F8 ? 2 * r4 + high : r4 + 8 * high);
              out[d] = acc[i][nh][e + 2 * high] * vs;
            }
          if (r4 == 0) own.ml[(size_t)t * a.n_heads + h0 + r] = make_float2(m[nh][e], l[nh][e]);
        }
    } else if (!together && s0 <= k0 && s1 == u1) {   // whole: o = O / l, transposed so that a lane has neighbouring dimensions of head lane / 4
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) {
        float inv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          inv[e] = l[nh][e] == 0.0f ? 0.0f : vs / l[nh][e];
          const int r = 8 * nh + 2 * j4 + e;
          if (lse && r4 == 0 && r < rows)
            lse[(size_t)t * a.n_heads + h0 + r] = l[nh][e] == 0.0f ? -INFINITY : m[nh][e] * kLn2 + logf(l[nh][e]);
        }
        const int r = 8 * nh + r4;
        uint16_t* out = o + (size_t)t * a.o_token + (size_t)(h0 + r) * a.o_head;
        if constexpr (K::F4) {   // x of 2 d: dimensions 8 j, 8 j + 4 of 32 d and on, y: 8 j + 1, 8 j + 5; of 2 d + 1: two further
#pragma unroll
          for (int d = 0; d < D / 32; ++d) {
            uint32_t z[2][2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const float(&y)[4] = acc[2 * d + b][nh];
              z[b][0] = movmatrix(pack2<DT>(y[0] * inv[0], y[1] * inv[1]));
              z[b][1] = movmatrix(pack2<DT>(y[2] * inv[0], y[3] * inv[1]));
            }
            if (K::SPREAD) {         // b: odd dimensions, the second of each two further: as the others lie
              const uint32_t w = z[0][1];
              z[0][1] = z[1][0];
              z[1][0] = w;
            }
            if (r < rows)
              *reinterpret_cast<uint4*>(out + 32 * d + 8 * j4) =
                  make_uint4(__byte_perm(z[0][0], z[0][1], 0x5410), __byte_perm(z[1][0], z[1][1], 0x5410),
                             __byte_perm(z[0][0], z[0][1], 0x7632), __byte_perm(z[1][0], z[1][1], 0x7632));
          }
        } else {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint32_t x = movmatrix(pack2<DT>(acc[i][nh][0] * inv[0], acc[i][nh][1] * inv[1]));
            const uint32_t y = movmatrix(pack2<DT>(acc[i][nh][2] * inv[0], acc[i][nh][3] * inv[1]));
            if (r < rows) {
              if (K::F8) {   // x: dimensions 4 j, 4 j + 2; y: 4 j + 1, 4 j + 3
                *reinterpret_cast<uint2*>(out + 16 * i + 4 * j4) = make_uint2(__byte_perm(x, y, 0x5410), __byte_perm(x, y, 0x7632));
              } else {
                *reinterpret_cast<uint32_t*>(out + 16 * i + 2 * j4) = x;
                *reinterpret_cast<uint32_t*>(out + 16 * i + 8 + 2 * j4) = y;
              }
            }
          }
        }
      }
    } else {                      // a part, as it lies in the registers
      float* part = together ? reinterpret_cast<float*>(ring) : parts + ((size_t)2 * me + (s0 == c0 ? 0 : 1)) * part_floats<D, NH>();
      if (together) {            // over the ring, from which nothing more is read
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        if (lane == 0) has_part[warp] = 1;
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int e = 0; e < 4; ++e) part[((i * NH + nh) * 4 + e) * 32 + lane] = acc[i][nh][e];
      float2* ml = reinterpret_cast<float2*>(part + 8 * NH * D);
      if (r4 == 0)
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int e = 0; e < 2; ++e) ml[8 * nh + 2 * j4 + e] = make_float2(m[nh][e], l[nh][e]);
    }
    s0 = s1;
    cp = np;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  }
  if (!together) {
    leave();
    return;
  }
  // ---- the shares of the unit meet: those of a CTA in its first warp's ring, then those of the CTAs,
  // each of which finishes some of the outputs
  constexpr int kSlots = 2 * NH * D;   // four outputs each, see Joined
  const int ctas = ways / kWarps, rank = (int)blockIdx.x % ctas, u = (int)blockIdx.x / ctas;
  uint8_t* rings = ring - (size_t)warp * stages * 2 * K::TILE;
  __syncthreads();
  for (int slot = tid; slot < kSlots; slot += kThreads) {
    const int reg = slot >> 3, r0 = 8 * ((reg >> 2) % NH) + (reg & 1);
    Joined x;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (!has_part[w]) continue;
      const float* part = reinterpret_cast<const float*>(rings + (size_t)w * stages * 2 * K::TILE);
      const float2* ml = reinterpret_cast<const float2*>(part + 8 * NH * D) + r0;
      const float2 e[4] = {ml[0], ml[2], ml[4], ml[6]};
      x.add(*reinterpret_cast<const float4*>(part + 4 * slot), e);
    }
    *reinterpret_cast<float4*>(rings + 16 * slot) = make_float4(x.x[0], x.x[1], x.x[2], x.x[3]);
    if ((reg >> 2) < NH && !(reg & 2) && !(slot & 7))
#pragma unroll
      for (int j = 0; j < 4; ++j) joined[r0 + 2 * j] = make_float2(x.m[j], x.l[j]);
  }
  cluster_arrive();
  cluster_wait();
  const int t = u / units, unit = u - t * units, hk = unit / blocks, h0 = hk * g + (unit - hk * blocks) * kRows;
  const int rows = (hk + 1) * g - h0 < kRows ? (hk + 1) * g - h0 : kRows;
  const float vs = K::LOW && c.v_scale ? c.v_scale[(size_t)layer * c.n_kv_heads + hk] : 1.0f;
  bool holed = false;
  if constexpr (SH) holed = t < n && sq[t].hole.y > sq[t].hole.x;
  for (int i = tid; i < kSlots / ctas; i += kThreads) {
    const int slot = rank * (kSlots / ctas) + i, reg = slot >> 3, r0 = 8 * ((reg >> 2) % NH) + (reg & 1);
    Joined x;
    const uint32_t at = smem_addr(rings + 16 * slot), ml = smem_addr(joined + r0);
#pragma unroll 4
    for (int b = 0; b < ctas; ++b) {
      float2 e[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) e[j] = peer_float2(ml + 16 * j, b);
      x.add(peer_float4(at, b), e);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      Joined::write<DT, CT, D, NH>(a, slot, j, t, h0, rows, vs, x.m[j], x.l[j], x.x[j], o, lse, holed ? &own : nullptr);
  }
  cluster_arrive();   // nobody leaves while its memory is read
  cluster_wait();
  leave();
}

// Joins the parts of a unit that was cut, with a running maximum and sum.  A thread
// has four outputs of the unit, the heads 8 nh + odd + 2 j of one dimension, as the
// parts lie in memory.  SPLIT: a CTA has 32 such groups and its warps take the
// parts in turn and meet in shared memory (few units, many parts each); else a
// thread goes through all parts.  blockIdx.x is the unit (by_cut == 0), or the begin
// of a range: then the unit that it cuts, if no earlier begin cuts it too.
template <int DT, int CT, int D, int NH, bool SPLIT, bool SH>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ qre_attn a, int n, int by_cut,
                                                        const float* __restrict__ v_scale, uint16_t* __restrict__ o,
                                                        float* __restrict__ lse, const Header* __restrict__ header,
                                                        const float* __restrict__ parts, const __grid_constant__ Own own) {
  constexpr int PF = part_floats<D, NH>();
  grid_dependency_wait();
  grid_dependents_launch();
  const Header h = *header;
  if (h.total == 0) return;
  const int32_t* firsts = reinterpret_cast<const int32_t*>(reinterpret_cast<const char*>(header) + kFirstsAt);
  const int g = a.n_heads / a.n_kv_heads, blocks = (g + kRows - 1) / kRows, units = a.n_kv_heads * blocks;
  int t, unit;
  long long u0;
  int nch;
  if (!by_cut) {
    t = blockIdx.x / units;
    unit = blockIdx.x - t * units;
    nch = firsts[t + 1] - firsts[t];
    u0 = (long long)firsts[t] * units + (long long)unit * nch;
    if (nch == 0) return;
  } else {
    const int b = blockIdx.x + 1;
    if (b >= h.ranges) return;
    const long long x = range_begin(b, h.ranges, h.total);
    int lo = 0, hi = n - 1;   // the last query that begins at or before x
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if ((long long)firsts[mid] * units <= x) lo = mid;
      else hi = mid - 1;
    }
    t = lo;
    nch = firsts[t + 1] - firsts[t];
    const long long rest = x - (long long)firsts[t] * units;
    unit = (int)(rest / nch);
    u0 = x - (rest - (long long)unit * nch);
    // only the begin of the second range that has chunks of the unit
    if (x <= u0 + kUnitCost || range_begin(b - 1, h.ranges, h.total) > u0 + kUnitCost) return;
  }
  const int b0 = range_of(u0 + kUnitCost, h.ranges, h.total), np = range_of(u0 + nch - 1, h.ranges, h.total) - b0 + 1;
  if (np < 2) return;
  // the first part lies in its range's first place when the unit begins there too; the others begin theirs
  const float* first = parts + ((size_t)2 * b0 + (range_begin(b0, h.ranges, h.total) >= u0 ? 0 : 1)) * PF;
  const int hk = unit / blocks, h0 = hk * g + (unit - hk * blocks) * kRows;
  const int rows = (hk + 1) * g - h0 < kRows ? (hk + 1) * g - h0 : kRows;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slot = SPLIT ? 32 * blockIdx.y + lane : (int)blockDim.x * blockIdx.y + tid, reg = slot >> 3, r0 = 8 * ((reg >> 2) % NH) + (reg & 1);
  Joined x;
#pragma unroll 4
  for (int i = SPLIT ? warp : 0; i < np; i += SPLIT ? 8 : 1) {
    const float* part = i == 0 ? first : parts + (size_t)2 * (b0 + i) * PF;
    const float2* ml = reinterpret_cast<const float2*>(part + 8 * NH * D) + r0;
    const float2 e[4] = {ml[0], ml[2], ml[4], ml[6]};
    x.add(*reinterpret_cast<const float4*>(part + 4 * slot), e);
  }
  const float vs = v_scale ? v_scale[hk] : 1.0f;
  bool holed = false;
  if constexpr (SH) {
    const int2 hole = own.hole[t];
    holed = hole.y > hole.x;
  }
  auto write = [&](int sl, int j, float M, float L, float X) {
    Joined::write<DT, CT, D, NH>(a, sl, j, t, h0, rows, vs, M, L, X, o, lse, holed ? &own : nullptr);
  };
  if constexpr (SPLIT) {
    __shared__ float ms[8][32][4], ls[8][32][4], xs[8][32][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ms[warp][lane][j] = x.m[j];
      ls[warp][lane][j] = x.l[j];
      xs[warp][lane][j] = x.x[j];
    }
    __syncthreads();
    if (tid >= 128) return;
    const int k = tid >> 2, j = tid & 3;   // slot of the CTA, head
    float M = -INFINITY, L = 0.0f, X = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) M = fmaxf(M, ms[w][k][j]);
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const float f = ms[w][k][j] == M ? 1.0f : ex2(ms[w][k][j] - M);
      L += ls[w][k][j] * f;
      X += xs[w][k][j] * f;
    }
    write(32 * blockIdx.y + k, j, M, L, X);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) write(slot, j, x.m[j], x.l[j], x.x[j]);
  }
}

int decode_grid(int ctas_sm) {
  const int sms = device_sm_count();
  const int n = (sms <= 0 ? 152 : sms) * ctas_sm;
  return n < kMaxCtas ? n : kMaxCtas;
}

size_t header_bytes(int n) { return (kFirstsAt + (size_t)(n + 1) * sizeof(int32_t) + 255) & ~(size_t)255; }

// Positions of a chunk of a cache, and bytes of its tile of K (or of V).
int chunk_of(const qre_kv_cache& c) { return c.dtype == QRE_E2M1 ? chunk4(c.head_dim) : kTile / (c.head_dim * (c.dtype == QRE_E4M3 ? 1 : 2)); }
int tile_of(const qre_kv_cache& c) { return c.dtype == QRE_E2M1 ? chunk4(c.head_dim) * (c.head_dim / 2 + c.head_dim / kBlock4) : kTile; }

size_t decode_ws_bytes(const qre_attn& a, const qre_kv_cache& c, int n) {
  const int grid = decode_grid(ctas_per_sm(c.dtype, a.head_dim, a.n_heads / a.n_kv_heads > 8));
  return header_bytes(n) + (size_t)2 * grid * kWarps * kRows * (a.head_dim + 2) * sizeof(float);
}

// What the join of a launch reads: the cut of its work, and the parts.
struct Cuts {
  const Header* header;   // NULL: no unit was cut
  const float* parts;
};

// What a CTA keeps in shared memory of n queries, and how many CTAs of a launch of n queries an SM holds.
template <bool SH>
size_t of_queries(int n) {
  return (size_t)(n + 1) * sizeof(Seq<SH>);
}
template <bool SH>
int fitting_ctas(const qre_attn& a, const qre_kv_cache& c, int n) {
  return decode_ctas(ctas_per_sm(c.dtype, a.head_dim, a.n_heads / a.n_kv_heads > 8), device_max_smem_optin(),
                     (long long)of_queries<SH>(n), 2ll * kWarps * 2 * tile_of(c));
}

// One launch (and its join; with `left` the join is left to the caller, if there is one): n queries whose places sum up below 2^31; without ids, of the rows from row0 on.
template <bool SH>
cudaError_t launch_part(const qre_attn& a, const qre_kv_cache& c, int layer, int n, const int32_t* seqs, int row0,
                        int max_len, const void* q, void* o, float* lse, const Own& own, void* ws, int* status,
                        cudaStream_t stream, Cuts* left = nullptr) {
  const int g = a.n_heads / a.n_kv_heads;
  const size_t fixed = of_queries<SH>(n);
  const int tile = tile_of(c);
  const int ctas_sm = fitting_ctas<SH>(a, c, n);
  const int grid = decode_grid(ctas_sm);
  const int stages = decode_room(ctas_sm, device_max_smem_optin(), (long long)fixed) >= 3ll * kWarps * 2 * tile ? 3 : 2;
  const size_t smem = (size_t)stages * kWarps * 2 * tile + fixed;
  Header* header = static_cast<Header*>(ws);
  float* parts = reinterpret_cast<float*>(static_cast<char*>(ws) + header_bytes(n));
  const long long all_units = (long long)n * a.n_kv_heads * ((g + kRows - 1) / kRows);
  const int cuts = grid * kWarps - 1;   // at most as many units are cut
  const int by_cut = all_units > cuts;
  const float* v_scale = (c.dtype == QRE_E4M3 || c.dtype == QRE_E2M1) && c.v_scale ? c.v_scale + (size_t)layer * c.n_kv_heads : nullptr;
  // parts by warps where units are few (8 units of 49 chunks each: 7.4 us by threads, 6.3 us by warps;
  // 512 units of two or three parts: 16.7 us by warps, 9 us by threads)
  const bool split = all_units <= 64;
  // Units are not cut at the warps' convenience where the caller's bound or the window says that all
  // are short: left whole, or shared by the warps of a cluster (see above)
  const int most = a.window > 0 && (max_len == 0 || a.window < max_len) ? a.window : max_len;
  const int chunk = chunk_of(c), chunks = (int)(((long long)most + chunk - 1) / chunk);
  int ways = 0;
  if (chunks > 0 && chunks <= (all_units > grid ? 4 : 2)) {
    ways = 1;
  } else if (chunks > 0 && all_units <= grid) {
    ways = kWarps;
    while (2 * chunks > 3 * ways && ways < kMostWays && all_units * (2 * ways / kWarps) <= grid) ways *= 2;
    if (chunks > kMostShare * ways) ways = 0;
  }
  auto go = [&](auto kernel, auto join, int slots) -> cudaError_t {
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), (int)smem);
    if (e != cudaSuccess) return e;
    const int ctas = ways / kWarps;
    e = launch_dependent_cluster(kernel, dim3(ctas ? (unsigned)all_units * ctas : grid), dim3(kThreads), ctas ? ctas : 1,
                                 smem, stream, a, c, layer, n, seqs, row0, static_cast<const uint16_t*>(q),
                                 static_cast<uint16_t*>(o), lse, header, parts, stages, ways, own, status);
    if (left) *left = ways ? Cuts{nullptr, nullptr} : Cuts{header, parts};
    if (e != cudaSuccess || ways || left) return e;
    const int threads = split || slots > 256 ? 256 : slots;
    return launch_dependent(join, dim3((unsigned)(by_cut ? cuts : all_units), slots / (split ? 32 : threads)),
                            dim3(threads), 0, stream, a, n, by_cut, v_scale, static_cast<uint16_t*>(o), lse,
                            const_cast<const Header*>(header), const_cast<const float*>(parts), own);
  };
  auto pick = [&](auto dt, auto ct, auto d) {
    constexpr int DT = decltype(dt)::value, CT = decltype(ct)::value, D = decltype(d)::value;
    if (g > 8)
      return split ? go(attn_decode_kernel<DT, CT, D, 2, SH>, attn_join_kernel<DT, CT, D, 2, true, SH>, 4 * D)
                   : go(attn_decode_kernel<DT, CT, D, 2, SH>, attn_join_kernel<DT, CT, D, 2, false, SH>, 4 * D);
    return split ? go(attn_decode_kernel<DT, CT, D, 1, SH>, attn_join_kernel<DT, CT, D, 1, true, SH>, 2 * D)
                 : go(attn_decode_kernel<DT, CT, D, 1, SH>, attn_join_kernel<DT, CT, D, 1, false, SH>, 2 * D);
  };
  using B = std::integral_constant<int, QRE_BF16>;
  using H = std::integral_constant<int, QRE_FP16>;
  using E = std::integral_constant<int, QRE_E4M3>;
  using F = std::integral_constant<int, QRE_E2M1>;
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  const bool bf = a.dtype == QRE_BF16, d64 = a.head_dim == 64;
  if (c.dtype == QRE_E2M1) {
    if (bf) return d64 ? pick(B{}, F{}, D64{}) : pick(B{}, F{}, D128{});
    return d64 ? pick(H{}, F{}, D64{}) : pick(H{}, F{}, D128{});
  }
  if (c.dtype == QRE_E4M3) {
    if (bf) return d64 ? pick(B{}, E{}, D64{}) : pick(B{}, E{}, D128{});
    return d64 ? pick(H{}, E{}, D64{}) : pick(H{}, E{}, D128{});
  }
  if (bf) return d64 ? pick(B{}, B{}, D64{}) : pick(B{}, B{}, D128{});
  return d64 ? pick(H{}, H{}, D64{}) : pick(H{}, H{}, D128{});
}

}  // namespace
}  // namespace qre
