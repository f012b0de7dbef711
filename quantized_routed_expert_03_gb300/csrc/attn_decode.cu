// attn_decode.cu -- attention of one new token per sequence over the paged cache.
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
// is brought into fp16's range by a power of two per head.
#include <cuda_fp8.h>

#include <type_traits>

#include "attn.cuh"
#include "internal.h"

namespace qre {
namespace {

constexpr int kWarps = 4;
constexpr int kCtasPerSm = 2;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 4096;           // bytes of K (and of V) in a chunk
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
// Two E4M3 bytes (low half of b) as an fp16 pair.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t b) {
  uint32_t r;
  asm("{.reg .b16 lo;\n\tcvt.u16.u32 lo, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(b));
  return r;
}

// DT: type of q and o; CT: type of the cache; NH: query heads of a unit in eights.
template <int DT, int CT, int D, int NH>
struct Decode {
  static constexpr bool F8 = CT == QRE_E4M3;
  static constexpr bool BF = CT == QRE_BF16;      // type of the products
  static constexpr int RB = D * (F8 ? 1 : 2);     // bytes of a row
  static constexpr int CK = kTile / RB;           // positions of a chunk
  static constexpr int PR = RB / 16;              // 16-byte pieces of a row
  static constexpr int RI = 32 / PR;              // rows that the warp's 32 lanes fetch at once
  static constexpr int NP = CK / 16;              // runs of 16 positions (each inside one page)
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
    return (uint32_t)(row * RB + 16 * (PR >= 8 ? col ^ (row & 7) : col ^ ((row >> 1) & 3)));
  }
};

// Floats of a part: eight heads at a time by D, and (m, l) of each head.
template <int D, int NH>
constexpr int part_floats() {
  return 8 * NH * (D + 2);
}

struct Seq {
  int row, len, first;   // table row, length, places of the queries before (for one unit each)
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
  template <int DT, bool F8, int NH>
  static __device__ __forceinline__ void write(const qre_attn& a, int slot, int j, int t, int h0, int rows, float vs, float M,
                                               float L, float X, uint16_t* o, float* lse) {
    const int reg = slot >> 3, i = (reg >> 2) / NH, high = (reg >> 1) & 1;
    const int r = 8 * ((reg >> 2) % NH) + (reg & 1) + 2 * j;
    const int d = 16 * i + (F8 ? 2 * (slot & 7) + high : (slot & 7) + 8 * high);
    if (r >= rows) return;
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

template <int DT, int CT, int D, int NH>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    attn_decode_kernel(const __grid_constant__ qre_attn a, const __grid_constant__ qre_kv_cache c, int layer, int n,
                       const int32_t* __restrict__ seqs, int row0, const uint16_t* __restrict__ q, uint16_t* __restrict__ o,
                       float* __restrict__ lse, Header* __restrict__ header, float* __restrict__ parts, int stages,
                       int ways, int* status) {
  using K = Decode<DT, CT, D, NH>;
  constexpr int CK = K::CK, KS = K::KS;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem + (size_t)(threadIdx.x >> 5) * stages * 2 * kTile;   // this warp's
  Seq* sq = reinterpret_cast<Seq*>(smem + (size_t)kWarps * stages * 2 * kTile);   // [n + 1]
  __shared__ int scan_part[kWarps];
  __shared__ int scan_total;
  __shared__ int has_part[kWarps];
  __shared__ float2 joined[8 * NH];   // (m, l) of the heads
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = a.n_heads / a.n_kv_heads;
  const int blocks = (g + kRows - 1) / kRows;       // head blocks of a KV head
  const int units = a.n_kv_heads * blocks;          // units of a sequence
  const int ps_shift = 31 - __clz(c.page_size);

  grid_dependency_wait();
  grid_dependents_launch();

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
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (len[i] < 0 || len[i] > (long long)c.max_pages * c.page_size) {
        if (blockIdx.x == 0 && t0 + kEach * tid + i < n) set_status(status, QRE_DEV_BAD_INDEX);
        len[i] = row[i] = 0;
      }
      const int lo = a.window > 0 && len[i] > a.window ? len[i] - a.window : 0;
      ch[i] = len[i] > 0 ? (len[i] + CK - 1) / CK - lo / CK + kUnitCost : 0;
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
      if (t < n) sq[t] = Seq{row[i], len[i], first};
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
  const long long all = (long long)gridDim.x * kWarps;
  const int ranges = (int)(together ? all : want < all ? want : all);
  // this warp's range: few ranges spread over the SMs
  const int me = together ? (int)blockIdx.x * kWarps + warp : warp * (int)gridDim.x + (int)blockIdx.x;
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
  for (int t = blockIdx.x; t < n; t += gridDim.x) {
    if (sq[t + 1].first != sq[t].first) continue;
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
  if (me >= ranges) return;
  const long long c0 = begin(me), c1 = begin(me + 1);
  if (c0 >= c1 && !together) return;

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
  int pages = 0;                     // lane j: page of positions 16 j .. 16 j + 15 of that chunk, -1 missing, -2 not seen
  auto look_up = [&]() {
    pages = -2;
    if (li < c1 && lane < K::NP) {
      const int len = sq[lp.t].len;
      const int lo = a.window > 0 && len > a.window ? len - a.window : 0;
      const int pos = (lo / CK + lp.ck - kUnitCost) * CK + 16 * lane;
      if (pos < len && pos + 16 > lo) {
        pages = c.page_table[(size_t)sq[lp.t].row * c.max_pages + (pos >> ps_shift)];
        if (pages < 0 || pages >= c.n_pages) {
          pages = -1;
          set_status(status, QRE_DEV_BAD_INDEX);
        }
      }
    }
  };
  const uint8_t* pool_k = static_cast<const uint8_t*>(c.k);
  const uint8_t* pool_v = static_cast<const uint8_t*>(c.v);
  const size_t head_bytes = (size_t)c.page_size * K::RB;
  uint32_t missing = 0;              // bit NP * slot + j: run j of that ring slot has no page
  auto fetch = [&](int slot) {       // fetches chunk li into the slot and moves on
    if (li < c1) {
      const int len = sq[lp.t].len;
      const int lo = a.window > 0 && len > a.window ? len - a.window : 0;
      const int pos0 = (lo / CK + lp.ck - kUnitCost) * CK;
      const int hk = lp.unit / blocks;
      const uint32_t gone = __ballot_sync(0xffffffffu, pages == -1);
      missing = (missing & ~(((1u << K::NP) - 1u) << (K::NP * slot))) | (gone << (K::NP * slot));
      const uint32_t dst = smem_addr(ring + (size_t)slot * 2 * kTile);
      const int r0 = lane / K::PR, col = lane % K::PR;
#pragma unroll
      for (int j = 0; j < K::NP; ++j) {
        const int page = __shfl_sync(0xffffffffu, pages, j);
        const size_t base = page < 0 ? 0
                                     : (((size_t)layer * c.n_pages + page) * c.n_kv_heads + hk) * head_bytes +
                                           (size_t)((pos0 + 16 * j) & (c.page_size - 1)) * K::RB;
#pragma unroll
        for (int r = 0; r < 16; r += K::RI) {
          const int row = 16 * j + r + r0, pos = pos0 + row;
          const bool ok = page >= 0 && pos >= lo && pos < len;
          const size_t off = ok ? base + (size_t)((r + r0) * K::RB + 16 * col) : 0;
          cp_async_16_zfill(dst + K::at(row, col), pool_k + off, ok);
          cp_async_16_zfill(dst + kTile + K::at(row, col), pool_v + off, ok);
        }
      }
      ++li;
      if (li < c1) {
        advance(lp, 1);
        to_chunk();
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
        if (K::F8) {   // element order of the E4M3 products: k = 2 j + e is dimension 4 j + e, 8 + 2 j + e is 4 j + 2 + e
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
    const int len = sq[t].len, lo = a.window > 0 && len > a.window ? len - a.window : 0;
    const float ks = K::F8 && c.k_scale ? c.k_scale[si + hk] : 1.0f;
    const float vs = K::F8 && c.v_scale ? c.v_scale[si + hk] : 1.0f;

    uint32_t qb[KS][NH][2];
    float s2[NH][2];                 // score factor of heads 2 j and 2 j + 1, base 2
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
      float own = a.scale * kLog2e * ks;   // of head lane / 4
      float f = 1.0f;
      if (K::F8 && DT == QRE_BF16) {
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
          qb[k][nh][e] = K::F8 && DT == QRE_BF16
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
      const uint32_t kt = smem_addr(ring + (size_t)slot * 2 * kTile), vt = kt + kTile;
      const int m8 = lane >> 3, l8 = lane & 7;

      float s[K::NP][NH][4];
#pragma unroll
      for (int i = 0; i < K::NP; ++i) {
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) s[i][nh][0] = s[i][nh][1] = s[i][nh][2] = s[i][nh][3] = 0.0f;
        // pieces p and p + 1 of 16 keys: keys 0-7 and 8-15 of each
#pragma unroll
        for (int p = 0; p < K::PR; p += 2) {
          uint32_t x[4];
          ldmatrix_x4(x, kt + K::at(16 * i + 8 * (m8 & 1) + l8, p + (m8 >> 1)));
#pragma unroll
          for (int nh = 0; nh < NH; ++nh) {
            if (!K::F8) {
              mma16816<K::BF>(s[i][nh], x[0], x[1], x[2], x[3], qb[p / 2][nh]);
            } else {
              mma16816<false>(s[i][nh], e4m3x2_to_half2(x[0] & 0xffffu), e4m3x2_to_half2(x[1] & 0xffffu),
                              e4m3x2_to_half2(x[0] >> 16), e4m3x2_to_half2(x[1] >> 16), qb[p][nh]);
              mma16816<false>(s[i][nh], e4m3x2_to_half2(x[2] & 0xffffu), e4m3x2_to_half2(x[3] & 0xffffu),
                              e4m3x2_to_half2(x[2] >> 16), e4m3x2_to_half2(x[3] >> 16), qb[p + 1][nh]);
            }
          }
        }
      }

      const int pos0 = (lo / CK + (int)(next - k0)) * CK;
      const uint32_t gone = (missing >> (K::NP * slot)) & ((1u << K::NP) - 1u);
      if (pos0 < lo || pos0 + CK > len || gone) {   // what is not seen: -inf
#pragma unroll
        for (int i = 0; i < K::NP; ++i)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const int pos = pos0 + 16 * i + 4 * e + r4;
            if (pos < lo || pos >= len || ((gone >> i) & 1u)) {
#pragma unroll
              for (int nh = 0; nh < NH; ++nh) s[i][nh][e] = s[i][nh][e + 1] = -INFINITY;
            }
          }
      }
      float p[K::NP][NH][4], sum[NH][2];
      auto weights = [&]() {
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
          sum[nh][0] = sum[nh][1] = 0.0f;
#pragma unroll
          for (int i = 0; i < K::NP; ++i)
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
            for (int i = 0; i < K::NP; ++i) mx = fmaxf(mx, fmaxf(s[i][nh][e], s[i][nh][e + 2]));
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
      for (int i = 0; i < K::NP; ++i) {
        uint32_t pb[NH][2];
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
          pb[nh][0] = movmatrix(pack2<K::PT>(p[i][nh][0], p[i][nh][1]));
          pb[nh][1] = movmatrix(pack2<K::PT>(p[i][nh][2], p[i][nh][3]));
        }
#pragma unroll
        for (int d = 0; d < K::PR; d += 2) {
          uint32_t x[4];
          if (!K::F8) {
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
              const uint32_t a0 = e4m3x2_to_half2(y0 & 0xffffu), a1 = e4m3x2_to_half2(y0 >> 16);
              const uint32_t a2 = e4m3x2_to_half2(y1 & 0xffffu), a3 = e4m3x2_to_half2(y1 >> 16);
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
    if (s1 <= k0) {               // none of its chunks
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
  if (!together) return;
  // ---- the shares of the unit meet: those of a CTA in its first warp's ring, then those of the CTAs,
  // each of which finishes some of the outputs
  constexpr int kSlots = 2 * NH * D;   // four outputs each, see Joined
  const int ctas = ways / kWarps, rank = (int)blockIdx.x % ctas, u = (int)blockIdx.x / ctas;
  uint8_t* rings = ring - (size_t)warp * stages * 2 * kTile;
  __syncthreads();
  for (int slot = tid; slot < kSlots; slot += kThreads) {
    const int reg = slot >> 3, r0 = 8 * ((reg >> 2) % NH) + (reg & 1);
    Joined x;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (!has_part[w]) continue;
      const float* part = reinterpret_cast<const float*>(rings + (size_t)w * stages * 2 * kTile);
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
  const float vs = K::F8 && c.v_scale ? c.v_scale[(size_t)layer * c.n_kv_heads + hk] : 1.0f;
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
      Joined::write<DT, K::F8, NH>(a, slot, j, t, h0, rows, vs, x.m[j], x.l[j], x.x[j], o, lse);
  }
  cluster_arrive();   // nobody leaves while its memory is read
  cluster_wait();
}

// Joins the parts of a unit that was cut, with a running maximum and sum.  A thread
// has four outputs of the unit, the heads 8 nh + odd + 2 j of one dimension, as the
// parts lie in memory.  SPLIT: a CTA has 32 such groups and its warps take the
// parts in turn and meet in shared memory (few units, many parts each); else a
// thread goes through all parts.  blockIdx.x is the unit (by_cut == 0), or the begin
// of a range: then the unit that it cuts, if no earlier begin cuts it too.
template <int DT, bool F8, int D, int NH, bool SPLIT>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ qre_attn a, int n, int by_cut,
                                                        const float* __restrict__ v_scale, uint16_t* __restrict__ o,
                                                        float* __restrict__ lse, const Header* __restrict__ header,
                                                        const float* __restrict__ parts) {
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
  auto write = [&](int sl, int j, float M, float L, float X) {
    Joined::write<DT, F8, NH>(a, sl, j, t, h0, rows, vs, M, L, X, o, lse);
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

int decode_grid() {
  const int sms = device_sm_count();
  const int n = (sms <= 0 ? 152 : sms) * kCtasPerSm;
  return n < kMaxCtas ? n : kMaxCtas;
}

size_t header_bytes(int n) { return (kFirstsAt + (size_t)(n + 1) * sizeof(int32_t) + 255) & ~(size_t)255; }

}  // namespace

size_t attn_decode_ws_bytes(const qre_attn& a, const qre_kv_cache&, int n) {
  const int grid = decode_grid();
  return header_bytes(n) + (size_t)2 * grid * kWarps * kRows * (a.head_dim + 2) * sizeof(float);
}

namespace {

// One launch (and its join): n queries whose places sum up below 2^31; without ids, of the rows from row0 on.
cudaError_t launch_part(const qre_attn& a, const qre_kv_cache& c, int layer, int n, const int32_t* seqs, int row0,
                        int max_len, const void* q, void* o, float* lse, void* ws, int* status, cudaStream_t stream) {
  const int grid = decode_grid();
  const int g = a.n_heads / a.n_kv_heads;
  const size_t fixed = (size_t)(n + 1) * sizeof(Seq);
  // what the CTAs of an SM share (1 KB of each is the system's, and the kernel's static arrays)
  const long long room = ((long long)device_max_smem_optin() + 1024) / kCtasPerSm - 1024 - 256 - (long long)fixed;
  const int stages = room >= 3ll * kWarps * 2 * kTile ? 3 : 2;
  const size_t smem = (size_t)stages * kWarps * 2 * kTile + fixed;
  Header* header = static_cast<Header*>(ws);
  float* parts = reinterpret_cast<float*>(static_cast<char*>(ws) + header_bytes(n));
  const long long all_units = (long long)n * a.n_kv_heads * ((g + kRows - 1) / kRows);
  const int cuts = grid * kWarps - 1;   // at most as many units are cut
  const int by_cut = all_units > cuts;
  const float* v_scale = c.dtype == QRE_E4M3 && c.v_scale ? c.v_scale + (size_t)layer * c.n_kv_heads : nullptr;
  // parts by warps where units are few (8 units of 49 chunks each: 7.4 us by threads, 6.3 us by warps;
  // 512 units of two or three parts: 16.7 us by warps, 9 us by threads)
  const bool split = all_units <= 64;
  // Units are not cut at the warps' convenience where the caller's bound or the window says that all
  // are short: left whole, or shared by the warps of a cluster (see above)
  const int most = a.window > 0 && (max_len == 0 || a.window < max_len) ? a.window : max_len;
  const int chunk = kTile / (a.head_dim * (c.dtype == QRE_E4M3 ? 1 : 2)), chunks = (int)(((long long)most + chunk - 1) / chunk);
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
                                 static_cast<uint16_t*>(o), lse, header, parts, stages, ways, status);
    if (e != cudaSuccess || ways) return e;
    const int threads = split || slots > 256 ? 256 : slots;
    return launch_dependent(join, dim3((unsigned)(by_cut ? cuts : all_units), slots / (split ? 32 : threads)),
                            dim3(threads), 0, stream, a, n, by_cut, v_scale, static_cast<uint16_t*>(o), lse,
                            const_cast<const Header*>(header), const_cast<const float*>(parts));
  };
  auto pick = [&](auto dt, auto ct, auto d) {
    constexpr int DT = decltype(dt)::value, CT = decltype(ct)::value, D = decltype(d)::value;
    constexpr bool F8 = CT == QRE_E4M3;
    if (g > 8)
      return split ? go(attn_decode_kernel<DT, CT, D, 2>, attn_join_kernel<DT, F8, D, 2, true>, 4 * D)
                   : go(attn_decode_kernel<DT, CT, D, 2>, attn_join_kernel<DT, F8, D, 2, false>, 4 * D);
    return split ? go(attn_decode_kernel<DT, CT, D, 1>, attn_join_kernel<DT, F8, D, 1, true>, 2 * D)
                 : go(attn_decode_kernel<DT, CT, D, 1>, attn_join_kernel<DT, F8, D, 1, false>, 2 * D);
  };
  using B = std::integral_constant<int, QRE_BF16>;
  using H = std::integral_constant<int, QRE_FP16>;
  using E = std::integral_constant<int, QRE_E4M3>;
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  const bool bf = a.dtype == QRE_BF16, d64 = a.head_dim == 64;
  if (c.dtype == QRE_E4M3) {
    if (bf) return d64 ? pick(B{}, E{}, D64{}) : pick(B{}, E{}, D128{});
    return d64 ? pick(H{}, E{}, D64{}) : pick(H{}, E{}, D128{});
  }
  if (bf) return d64 ? pick(B{}, B{}, D64{}) : pick(B{}, B{}, D128{});
  return d64 ? pick(H{}, H{}, D64{}) : pick(H{}, H{}, D128{});
}

}  // namespace

cudaError_t launch_attn_decode(const qre_attn& a, const qre_kv_cache& c, int layer, int n, const int32_t* seqs,
                               int max_len, const void* q, void* o, float* lse, void* ws, int* status,
                               cudaStream_t stream) {
  // The kernel counts the places of a launch in 32 bits.  A sequence has at most as many as its table row (or the
  // window) allows, 2^27 and a few, so a launch takes at least 15; a call is split only where rows hold millions
  // of positions.
  const long long chunk = kTile / (a.head_dim * (c.dtype == QRE_E4M3 ? 1 : 2)), held = (long long)c.max_pages * c.page_size;
  const long long places = (a.window > 0 && a.window < held ? a.window : held) / chunk + 2 + kUnitCost;
  const int most = 0x7fffffffll / places < n ? (int)(0x7fffffffll / places) : n;
  for (int i = 0; i < n; i += most) {
    const int m = n - i < most ? n - i : most;
    const cudaError_t e =
        launch_part(a, c, layer, m, seqs ? seqs + i : nullptr, i, max_len, static_cast<const uint16_t*>(q) + i * a.q_token,
                    static_cast<uint16_t*>(o) + i * a.o_token, lse ? lse + (size_t)i * a.n_heads : nullptr, ws, status, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace qre
