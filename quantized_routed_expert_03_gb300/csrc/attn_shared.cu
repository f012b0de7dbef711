// attn_shared.cu -- attention of one new token for sequences that share the pages of a prefix.
//
// The softmax of a query over [0, len) is joined from two parts, the group's common positions (its hole) and its own:
//   m = max m_i, l = sum l_i 2^(m_i - m), o = sum o_i 2^(m_i - m) / l   (base 2, in fp32).
//
// Bound: the prefix is read once for a group, and each sequence's own positions once; 4 flops an element for each query
// head.  The rows of a group that share a KV head, members x heads, are multiplied with a tile of keys together: at 128
// rows a tile of 128 keys (64 KB in 16 bits at D = 128) takes the tensor cores 1024 cycles and the memory 2800.
//
// Steps: a plan (one CTA: what each group shares, in tiles of 128 keys, and how many SMs it is worth); the prefixes
// (below); beside them, on the other SMs, the decode kernel over what lies outside the holes; the join.
//
// Prefixes: units are (group, KV head, 256 rows); their tiles in a row are cut into equal ranges, one per CTA (one on an
// SM), as the decode kernel cuts its chunks.  A CTA multiplies with tcgen05, S and P in tensor memory, O beside it, in
// two chains, each with a softmax of 128 threads, one row each: with more than 128 rows a chain has 128 of them, with
// less both have the same rows and take the tiles in turn, so that one's products run beside the other's softmax.  K and
// V come through a ring by TMA out of the pages; rows of 8 and 4 bits come as bytes and are widened to fp16 in shared
// memory by eight warps of their own.  No row needs a mask: a hole begins where all of the group's windows have, at a
// whole tile, and ends with a common page, behind which the last tile's rows are zeroed.
//
// What it measured (calls with the common lengths found in front of them, us): 64 sequences of up to 1500 positions
// behind 16,384, 32 heads on 8, D = 128, bf16: 73 (E4M3: 64; each by itself 446; the bytes take 39); 8 groups of 8 behind up to 8192:
// 51 (98; 24); 32 behind 32,768 in 4 bits, 64 heads on 8: 62 (E4M3: 63; 265; the products take 18).  10 us of a launch of the
// prefixes are its begin (the plan, the queries, the first tile's references) and 3 its end (parts).  Steps, on the
// first: 119 at first; queries by asynchronous copies, one copy of the softmax's code, 32-bit places and a join that asks
// for its parts at once 97; the own positions begun beside the prefixes 91; the last join for all parts 84; SMs for the
// prefixes and others for the own positions, not all for both in turn, 72.  The last one: 67, then 62 with the turn
// handed over behind the scores and four widened tiles in the ring, not three (4600 -> 3950 cycles a tile).  No gain: a round of the softmax's code before
// the plan is there, for the instruction cache.  In 4 bits 4 warps that widen took 2 us more than 8.
#include <atomic>
#include <type_traits>

#include "attn_decode.cuh"
#include "attn_split.h"
#include "tc.cuh"

namespace qre {
namespace {

constexpr int kM = 128;              // rows of a chain
constexpr int kUnitRows = 2 * kM;
constexpr int kN = 128;              // keys of a tile
constexpr int kTileCost = 2;         // tiles that the begin and the end of a unit are worth
constexpr int kMinTiles = 3;         // places of a range, at least
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kS = 0, kO = 256, kChain = 128;   // tensor-memory columns, from one chain to the other; P overwrites its S
// A row's weights are taken against a reference that stays while the sum of a tile's weights is at most this (fp16
// weights end at 65504, and values enter the accumulators times weights of up to this).
constexpr float kMostSum = 65504.0f;
// The weight, in base 2, of the maximum that sets the reference: fp16 ends at 2^-24, so weights below 2^-33 of the
// largest are lost; 128 weights of it stay below kMostSum with room for a maximum that doubles.
template <bool BF>
constexpr float kLift = BF ? 0.0f : 8.0f;

struct Group {
  int c0, m;             // queries
  int ha, hb;            // positions [ha, hb): ha a whole tile
  int before;            // queries of the groups before that share something
  int tiles;
  int pad[2];
};
// Places are counted in 31 bits (a call with more shares nothing): 64-bit divisions take long, most of all in
// code that is not in the instruction cache yet.
struct PlanHead {
  int total;             // places
  int ranges;
  int each, rest;        // total / ranges, total % ranges
  __device__ __forceinline__ int begin(int b) const { return each * b + (int)((unsigned)rest * (unsigned)b / (unsigned)ranges); }
  // the range that place i lies in
  __device__ __forceinline__ int range_of(int i) const {
    int b = (int)((float)i * ((float)ranges / (float)total));
    b = b < ranges ? b : ranges - 1;
    while (begin(b) > i) --b;
    while (begin(b + 1) <= i) ++b;
    return b;
  }
};
// What the join wants to know of a query, in one place: its loads are a chain as it is.
struct alignas(16) Query {
  int c0, m, before, tiles;   // of its group; no tiles: it is complete already
  int first;                  // places before the group's
  int pad[3];
};
// The workspace.
struct Space {
  PlanHead* head;
  unsigned long long* start;   // see Own
  int32_t* first;        // [n_groups + 1] places of the groups before
  Group* groups;         // [n_groups]
  int2* hole;            // [n]
  Query* query;          // [n]
  float* own_o;          // [n][n_heads][D]
  float2* own_ml;        // [n][n_heads]
  float* part_o;         // [rows][D]
  float2* part_ml;       // [rows]
  void* decode;
  size_t bytes;
};

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

int shared_grid() {
  const int sms = device_sm_count();
  return sms <= 0 ? 152 : sms;
}

constexpr long long kWorthBytes = 200000000;   // see launch_attn_decode_shared
constexpr int kPartQueries = 1024;   // of a launch of the decode kernel: it keeps 24 bytes of each in shared memory

Space space_of(const qre_attn& a, const qre_kv_cache& c, int n, int n_groups, void* ws) {
  Space s;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = static_cast<char*>(ws) + at;
    at += up256(bytes);
    return p;
  };
  const size_t heads = (size_t)n * a.n_heads;
  // pieces of units: rows once or twice, and 256 for each range's end
  const size_t rows = 2 * heads + (size_t)kUnitRows * shared_grid();
  s.head = reinterpret_cast<PlanHead*>(take(sizeof(PlanHead)));
  s.start = reinterpret_cast<unsigned long long*>(take(sizeof(unsigned long long)));
  s.first = reinterpret_cast<int32_t*>(take(((size_t)n_groups + 1) * sizeof(int32_t)));
  s.groups = reinterpret_cast<Group*>(take((size_t)n_groups * sizeof(Group)));
  s.hole = reinterpret_cast<int2*>(take((size_t)n * sizeof(int2)));
  s.query = reinterpret_cast<Query*>(take((size_t)n * sizeof(Query)));
  s.own_o = reinterpret_cast<float*>(take(heads * a.head_dim * sizeof(float)));
  s.own_ml = reinterpret_cast<float2*>(take(heads * sizeof(float2)));
  s.part_o = reinterpret_cast<float*>(take(rows * a.head_dim * sizeof(float)));
  s.part_ml = reinterpret_cast<float2*>(take(rows * sizeof(float2)));
  s.decode = take(decode_ws_bytes(a, c, n));
  s.bytes = at;
  return s;
}

// ---------------------------------------------------------------- the plan

// What the work takes, ns of an SM: a tile of a unit, and a position and a unit of the sequences' own.  Fitted to calls
// that gave the prefixes 16 to 151 of the 152 SMs; with these, seven calls of all types and head sizes came within 4 % of
// their best split.
struct Costs {
  float tile, position, unit;
  int ctas_sm;           // CTAs of the decode kernel on an SM
};

Costs costs_of(const qre_kv_cache& c, int ctas_sm) {
  const bool d64 = c.head_dim == 64;
  if (c.dtype == QRE_E2M1) return d64 ? Costs{1650.0f, 2.7f, 500.0f, ctas_sm} : Costs{1800.0f, 3.8f, 600.0f, ctas_sm};
  if (c.dtype == QRE_E4M3) return d64 ? Costs{1550.0f, 2.9f, 400.0f, ctas_sm} : Costs{1750.0f, 5.1f, 500.0f, ctas_sm};
  return d64 ? Costs{1100.0f, 3.7f, 400.0f, ctas_sm} : Costs{1270.0f, 7.4f, 400.0f, ctas_sm};
}

// One CTA, a warp per group: the positions that it shares, [ha, hb): hb the common length in whole runs of 16 whose
// pages are there, ha a whole tile at or behind the first position that every member sees.
__global__ void __launch_bounds__(1024) shared_plan_kernel(const __grid_constant__ qre_kv_cache c, int n,
                                                           const int32_t* __restrict__ seqs, int n_groups,
                                                           const int32_t* __restrict__ cu_group,
                                                           const int32_t* __restrict__ common_len, int window, int g,
                                                           int n_kv_heads, int min_positions, int grid, Costs costs,
                                                           Space s, uint32_t token, int* status) {
  __shared__ long long scan[33];
  __shared__ int scan_m[33];
  __shared__ long long places_of[32];
  __shared__ int shared_of[32];
  __shared__ float own_of[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dependency_wait();
  grid_dependents_launch();
  if (tid == 0) *s.start = 0;
  int bad = 0;
  for (int i = tid; i < n_groups; i += 1024) {
    const int a = cu_group[i], b = cu_group[i + 1];
    bad |= a < 0 || b < a || b > n || (i == 0 && a != 0) || (i == n_groups - 1 && b != n);
  }
  for (int i = tid; i < n; i += 1024) {
    s.hole[i] = make_int2(0, 0);
    s.query[i].tiles = 0;
  }
  bad = __syncthreads_or(bad || (n_groups == 0 && n > 0));
  if (bad) {   // nothing is shared
    if (tid == 0) {
      set_status(status, QRE_DEV_BAD_INDEX);
      *s.head = PlanHead{0, 0, 0, 0};
      release_start(s.start, token, grid * costs.ctas_sm);
    }
    return;
  }
  const int ps_shift = 31 - __clz(c.page_size);
  long long total = 0;
  int before = 0;
  float own = 0.0f;                  // positions of this warp's sequences that are not shared
  for (int g0 = 0; g0 < n_groups; g0 += 32) {
    const int gi = g0 + warp;
    Group x = {};
    if (gi < n_groups) {
      x.c0 = cu_group[gi];
      x.m = cu_group[gi + 1] - x.c0;
      const int common = common_len[gi];
      int least = 0x7fffffff, most = 0, row = -1;
      float seen = 0.0f;
      for (int i = lane; i < x.m; i += 32) {
        const int id = seqs ? seqs[x.c0 + i] : x.c0 + i;
        const int len = id >= 0 && id < c.max_seqs ? c.seq_len[id] : -1;
        if (i == 0) row = id;
        least = min(least, len);
        most = max(most, len);
        seen += (float)(len < 0 ? 0 : window > 0 && window < len ? window : len);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) seen += __shfl_xor_sync(0xffffffffu, seen, d);
      least = __reduce_min_sync(0xffffffffu, least);
      most = __reduce_max_sync(0xffffffffu, most);
      row = __shfl_sync(0xffffffffu, row, 0);
      const bool ok = least >= 0 && common >= 0 && common <= least && (long long)most <= (long long)c.max_pages * c.page_size;
      if (x.m > 0 && least >= 0 && !ok && lane == 0) set_status(status, QRE_DEV_BAD_INDEX);
      int hb = ok && x.m > 1 ? common & ~15 : 0;
      const int lo = window > 0 && most > window ? most - window : 0;
      x.ha = (int)min(((long long)lo + kN - 1) / kN * kN, (long long)hb);
      // up to the first page that is missing: what lies behind counts as not seen, each sequence for itself
      const int col0 = x.ha >> ps_shift, cols = (hb + c.page_size - 1) >> ps_shift;
      int gone = cols;
      for (int k0 = col0; k0 < cols && gone == cols; k0 += 32 * 8) {
        int p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = k0 + 32 * e + lane < cols ? c.page_table[(size_t)row * c.max_pages + k0 + 32 * e + lane] : 0;
        int first = cols;
#pragma unroll
        for (int e = 7; e >= 0; --e)
          if (p[e] < 0 || p[e] >= c.n_pages) first = k0 + 32 * e + lane;
        gone = __reduce_min_sync(0xffffffffu, first);
      }
      if (gone < cols) hb = gone << ps_shift;
      if (hb - x.ha < min_positions) hb = x.ha = 0;
      x.hb = hb;
      x.tiles = (hb - x.ha + kN - 1) / kN;
      own += seen - (float)x.m * (float)(hb - x.ha);
    }
    const int blocks = (x.m * g + kUnitRows - 1) / kUnitRows;
    if (lane == 0) {
      places_of[warp] = x.tiles ? (long long)n_kv_heads * blocks * (x.tiles + kTileCost) : 0;
      shared_of[warp] = x.tiles ? x.m : 0;
    }
    __syncthreads();
    if (warp == 0) {
      long long p = places_of[lane];
      int q = shared_of[lane];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, p, d);
        const int v = __shfl_up_sync(0xffffffffu, q, d);
        if (lane >= d) {
          p += u;
          q += v;
        }
      }
      scan[lane + 1] = p;
      scan_m[lane + 1] = q;
      if (lane == 0) scan[0] = scan_m[0] = 0;
    }
    __syncthreads();
    x.before = before + scan_m[warp];
    const int first = (int)(total + scan[warp]);
    if (gi < n_groups && lane == 0) {
      s.groups[gi] = x;
      s.first[gi] = first;
    }
    if (x.tiles)
      for (int i = lane; i < x.m; i += 32) {
        s.hole[x.c0 + i] = make_int2(x.ha, x.hb);
        s.query[x.c0 + i] = Query{x.c0, x.m, x.before, x.tiles, first, {}};
      }
    total += scan[32];
    before += scan_m[32];
    __syncthreads();
  }
  if (total > 0x7fffffff - 1024) {   // (the same in all threads)
    for (int i = tid; i < n; i += 1024) {
      s.hole[i] = make_int2(0, 0);
      s.query[i].tiles = 0;
    }
    __syncthreads();
    if (tid == 0) {
      *s.head = PlanHead{0, 0, 0, 0};
      release_start(s.start, token, grid * costs.ctas_sm);
    }
    return;
  }
  if (lane == 0) own_of[warp] = own;
  __syncthreads();
  if (tid == 0) {
    s.first[n_groups] = (int)total;
    float positions = 0.0f;
    for (int i = 0; i < 32; ++i) positions += own_of[i];
    // The prefixes and the sequences' own positions run side by side: SMs in the proportion of what they take
    const float a = costs.tile * (float)total, b = n_kv_heads * (costs.position * positions + costs.unit * (float)n);
    int mine = (int)((float)grid * a / (a + b) + 0.5f);
    mine = mine < 1 ? 1 : mine < grid - 1 ? mine : grid - 1;
    const int most = (int)((total + kMinTiles - 1) / kMinTiles), ranges = most < mine ? most : mine;
    *s.head = PlanHead{(int)total, ranges, ranges ? (int)total / ranges : 0, ranges ? (int)total % ranges : 0};
    release_start(s.start, token, (grid - ranges) * costs.ctas_sm);   // two (or three) on each SM that the ranges leave
  }
}

// ---------------------------------------------------------------- the prefixes

template <int DT, int CT, int D>
struct Shape {
  static constexpr bool F8 = CT == QRE_E4M3, F4 = CT == QRE_E2M1, LOW = F8 || F4;
  static constexpr bool BF = CT == QRE_BF16;         // type of the products
  static constexpr int PT = BF ? QRE_BF16 : QRE_FP16;
  static constexpr int HALF = kN * 128;              // 64 columns of a 128-row tile, 128-byte rows
  static constexpr int TILE = HALF * (D / 64);
  static constexpr int RB = F4 ? D / 2 : F8 ? D : 2 * D;   // bytes of a stored row, without scales
  static constexpr int SB = F4 ? D / kBlock4 : 0;
  static constexpr int RAW = kN * (RB + SB);         // bytes of a stored tile
  static constexpr int SLOTS = D == 128 ? (LOW ? 4 : 5) : (LOW ? 8 : 10);
  static constexpr int STAGES = !LOW ? 0 : F8 ? (D == 128 ? 2 : 4) : (D == 128 ? 3 : 6);
  static constexpr int THREADS = LOW ? 640 : 384;
  // Registers: 384 x 168 at launch = 256 x 208 + 128 x 88; 640 x 96 = 61,440 > 256 x 152 + 384 x 56 (the kernels that widen
  // spill 68 to 72 bytes with these).
  static constexpr int SOFT_REGS = LOW ? 152 : 208, OTHER_REGS = LOW ? 56 : 88;
  static constexpr int BYTES = 2 * TILE + SLOTS * TILE + STAGES * RAW + 2048;
  // warps 0-7: the two chains' softmax; then
  static constexpr int kTma = 8, kMma = 9 /* and 10 */, kWiden = 12, kWidenWarps = 8;
};

__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, volatile int* abort, int* status, uint64_t limit_ns) {
  return __all_sync(0xffffffffu, mbar_wait_inline(bar, parity, abort, status, limit_ns) ? 1 : 0) != 0;
}

// A piece of work: some tiles of a unit.
struct Piece {
  int c0, rows0, rows;     // first query of the group; rows [rows0, rows0 + rows) of the KV head's
  int hk;
  int pos0, hb;            // first position, end of the group's common positions
  int tiles;
  long long out;           // first row of its parts
  __device__ __forceinline__ bool both() const { return rows > kM; }   // each chain has rows of its own
  // the tiles of chain t: begin, step, number
  __device__ __forceinline__ int first(int t) const { return both() ? 0 : t; }
  __device__ __forceinline__ int step() const { return both() ? 1 : 2; }
  __device__ __forceinline__ int count(int t) const { return both() ? tiles : (tiles + 1 - t) / 2; }
  __device__ __forceinline__ int valid(int t) const { return both() ? (t ? rows - kM : kM) : rows; }
};

// The pieces of one range, in order.  Every warp goes through them for itself.
class Pieces {
 public:
  __device__ __forceinline__ Pieces(const Space& s, int g, int n_heads) : s_(s), g_(g), heads_(n_heads), gi_(-1) {}
  // Reads the plan.
  __device__ __forceinline__ void begin(int n_groups) {
    const Space& s = s_;
    const PlanHead h = *s.head;
    b_ = blockIdx.x;
    at_ = end_ = 0;
    if (b_ >= h.ranges) return;
    at_ = h.begin(b_);
    end_ = h.begin(b_ + 1);
    int lo = 0, hi = n_groups - 1;   // the last group that begins at or before at_
    while (lo < hi) {                // 32 at a time
      const int lane = threadIdx.x & 31, step = (hi - lo + 31) / 32;
      const int i = lo + (lane + 1) * step;
      const unsigned le = __ballot_sync(0xffffffffu, i <= hi && s.first[i <= hi ? i : hi] <= at_);
      const int k = __popc(le);      // first[] ascends: the lanes with a bit come first
      lo += k * step;
      if (lo + step - 1 < hi) hi = lo + step - 1;
    }
    gi_ = lo;
    load();
  }
  __device__ __forceinline__ bool next(Piece& p) {
    while (at_ < end_) {
      while (at_ >= next_) {         // (groups that share nothing have no place)
        ++gi_;
        load();
      }
      const int per = x_.tiles + kTileCost;
      const int unit = (at_ - first_) / per, in = at_ - first_ - unit * per, left = end_ - at_;
      const int to = left < per - in ? in + left : per;
      const int t0 = in > kTileCost ? in - kTileCost : 0, t1 = to - kTileCost;
      at_ += to - in;
      if (t1 <= t0) continue;
      const int rows = x_.m * g_, blocks = (rows + kUnitRows - 1) / kUnitRows, block = unit % blocks;
      p.hk = unit / blocks;
      p.c0 = x_.c0;
      p.rows0 = block * kUnitRows;
      p.rows = rows - p.rows0 < kUnitRows ? rows - p.rows0 : kUnitRows;
      p.pos0 = x_.ha + t0 * kN;
      p.hb = x_.hb;
      p.tiles = t1 - t0;
      p.out = 2 * ((long long)x_.before * heads_ + (long long)p.hk * rows + p.rows0) + (long long)kUnitRows * b_;
      return true;
    }
    return false;
  }

 private:
  __device__ __forceinline__ void load() {
    x_ = s_.groups[gi_];
    first_ = s_.first[gi_];
    next_ = s_.first[gi_ + 1];
  }
  const Space& s_;
  int g_, heads_, gi_, b_;
  int at_ = 0, end_ = 0, first_ = 0, next_ = 0;
  Group x_;
};

template <int DT, int CT, int D>
__global__ void __launch_bounds__(Shape<DT, CT, D>::THREADS, 1)
    shared_prefix_kernel(const __grid_constant__ qre_attn a, const __grid_constant__ qre_kv_cache c, int layer,
                         const int32_t* __restrict__ seqs, int n_groups, const uint16_t* __restrict__ q,
                         const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                         const __grid_constant__ CUtensorMap tk16, const __grid_constant__ CUtensorMap tv16, int box_rows,
                         const __grid_constant__ Space space, uint64_t limit_ns, uint64_t stall_ns, int* status) {
  using P = Shape<DT, CT, D>;
  extern __shared__ __align__(1024) uint8_t tiles_smem[];   // the swizzle goes by addresses; no static shared memory beside it
  uint8_t* sq = tiles_smem;                   // two query tiles
  uint8_t* skv = tiles_smem + 2 * P::TILE;         // ring of key and value tiles
  uint8_t* sraw = skv + P::SLOTS * P::TILE;  // ring of stored tiles
  uint64_t* full = reinterpret_cast<uint64_t*>(sraw + P::STAGES * P::RAW);   // [SLOTS]
  uint64_t* empty = full + P::SLOTS;         // [SLOTS]
  uint64_t* raw_full = empty + P::SLOTS;     // [STAGES]
  uint64_t* raw_empty = raw_full + P::STAGES;
  uint64_t* q_full = raw_empty + P::STAGES;
  uint64_t* q_free = q_full + 1;
  uint64_t* s_full = q_free + 1;             // [2]
  uint64_t* p_full = s_full + 2;             // [2]
  uint64_t* o_done = p_full + 2;             // [2]
  uint64_t* turn = o_done + 2;               // [2]
  uint64_t* drain = turn + 2;                // [2]
  float* row_scale = reinterpret_cast<float*>(drain + 2);   // [2][kM]: factor of a row's scores
  uint32_t* tmem_p = reinterpret_cast<uint32_t*>(row_scale + 2 * kM);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_p + 1);   // a wait gave up
  int* issued = const_cast<int*>(reinterpret_cast<volatile int*>(tmem_p + 2));   // tiles whose loads were issued
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = a.n_heads / a.n_kv_heads;

  if (tid == 0) {
    for (int s = 0; s < P::SLOTS; ++s) {
      mbar_init(&full[s], P::LOW ? P::kWidenWarps : 1);
      mbar_init(&empty[s], 2);
    }
    for (int s = 0; s < P::STAGES; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], P::kWidenWarps);
    }
    mbar_init(q_full, 8);
    mbar_init(q_free, 8);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 4);
      mbar_init(&o_done[t], 1);
      mbar_init(&turn[t], 1);
      mbar_init(&drain[t], 1);
    }
    *abort_flag = 0;
    *issued = 0;
    fence_barrier_init();
  }
  if (warp == P::kMma) {
    tmem_alloc(tmem_p, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_p;
  auto wait_for = [&](uint64_t* b, int n) { return wait_bounded(b, n & 1, abort_flag, status, limit_ns); };   // phase n
  Piece w;
  Pieces pieces(space, g, a.n_heads);
  auto begin = [&]() {
    grid_dependency_wait();
    grid_dependents_launch();
    pieces.begin(n_groups);
  };
  const int ps_shift = 31 - __clz(c.page_size);
  if (warp >= 8 && warp < P::kWiden) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(P::OTHER_REGS));
    if (warp == P::kTma) {
      // ---- fetches the tiles: a lane has one run of rows of one page
      begin();
      if (stall_ns && blockIdx.x == 0) debug_stall_inline(stall_ns);   // test hook
      int i = 0;                       // tiles so far, K and V in turn
      bool ok = true;
      const size_t head_bytes = (size_t)c.page_size * (P::RB + P::SB);
      while (ok && pieces.next(w)) {
        const int id = seqs ? seqs[w.c0] : w.c0;
        const int32_t* table = c.page_table + (size_t)id * c.max_pages;
        for (int j = 0; ok && j < w.tiles; ++j) {
          const int pos0 = w.pos0 + j * kN, rows = w.hb - pos0 < kN ? w.hb - pos0 : kN;
          const bool whole = rows == kN;
          const int run = whole || P::LOW ? box_rows : 16, runs = (rows + run - 1) / run;
          int page = 0;
          if (lane < runs) page = table[(pos0 + lane * run) >> ps_shift];
          const int off = (pos0 + lane * run) & (c.page_size - 1);
          for (int x = 0; ok && x < 2; ++x, ++i) {
            const bool is_v = x == 1;
            if constexpr (!P::LOW) {
              const int s = i % P::SLOTS;
              ok = i < P::SLOTS || wait_for(&empty[s], i / P::SLOTS - 1);
              if (!ok) break;
              uint8_t* tile = skv + s * P::TILE;
              if (is_v && !whole) {    // what lies behind the end is multiplied by weights of 0
                for (int e = lane; e < (kN - rows) * 8 * (D / 64); e += 32) {
                  const int half = e / ((kN - rows) * 8), r = e - half * (kN - rows) * 8;
                  reinterpret_cast<uint4*>(tile + half * P::HALF + rows * 128)[r] = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
              }
              if (lane == 0) {
                mbar_arrive_expect_tx(&full[s], (uint32_t)(rows * 2 * D));
                *issued = i + 1;
              }
              __syncwarp();
              if (lane < runs) {
                const CUtensorMap* map = whole ? (is_v ? &tv : &tk) : (is_v ? &tv16 : &tk16);
                const int row = (page * c.n_kv_heads + w.hk) * c.page_size + off;
                for (int h = 0; h < D / 64; ++h)
                  tma_load_2d(tile + h * P::HALF + lane * run * 128, map, 64 * h, row, &full[s]);
              }
            } else {
              const int s = i % P::STAGES;
              ok = i < P::STAGES || wait_for(&raw_empty[s], i / P::STAGES - 1);
              if (!ok) break;
              uint8_t* raw = sraw + s * P::RAW;
              if (lane == 0) {
                mbar_arrive_expect_tx(&raw_full[s], (uint32_t)(rows * (P::RB + P::SB)));
                *issued = i + 1;
              }
              __syncwarp();
              if (lane < runs) {
                const int mine = rows - lane * run < run ? rows - lane * run : run;
                const uint8_t* base = static_cast<const uint8_t*>(is_v ? c.v : c.k) +
                                      (((size_t)layer * c.n_pages + page) * c.n_kv_heads + w.hk) * head_bytes;
                bulk_copy_g2s(raw + lane * run * P::RB, base + (size_t)off * P::RB, (uint32_t)(mine * P::RB), &raw_full[s]);
                if constexpr (P::F4)
                  bulk_copy_g2s(raw + kN * P::RB + lane * run * P::SB, base + (size_t)c.page_size * P::RB + (size_t)off * P::SB,
                                (uint32_t)(mine * P::SB), &raw_full[s]);
              }
            }
            __syncwarp();
          }
        }
      }
    } else if (warp == P::kMma || warp == P::kMma + 1) {
      // ---- products: the whole warp, so that the operands stay in uniform registers; a chain each
      // (what an MMA takes comes out of a shuffle from lane 0, so that the compiler knows it is the warp's: as each lane's
      // own it moves to the uniform registers anew for every MMA, and one takes some 110 cycles to issue, not 64)
      auto of_warp = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
      const int t = of_warp(warp - P::kMma);
      const uint32_t lead = elect_lane();
      const uint32_t id_s = P::BF ? umma_idesc_bf16(kM, kN) : umma_idesc_f16(kM, kN);
      const uint32_t id_o = (P::BF ? umma_idesc_bf16(kM, D) : umma_idesc_f16(kM, D)) | kUmmaBMnMajor;
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), ts = tm + kS + t * kChain, td = tm + kO + t * kChain;
      const uint64_t kd = umma_desc_sw128(smem_addr(skv)), vd = umma_desc_sw128_mn(smem_addr(skv), P::HALF);
      int i0 = 0, np = 0, n = 0, turns = 0;   // ring tiles, pieces, key tiles and turns of this chain so far
      bool ok = true;
      auto wait_tile = [&](int i) { return wait_for(&full[i % P::SLOTS], i / P::SLOTS); };
      begin();
      while (ok && pieces.next(w)) {
        const bool both = w.both();
        const uint64_t qd = umma_desc_sw128(smem_addr(sq) + (uint32_t)of_warp(both ? t : 0) * P::TILE);
        auto scores = [&](int i) {     // S = Q K_j^T
          const int slot = of_warp(i % P::SLOTS);
          const uint64_t k0 = kd + (uint32_t)slot * (P::TILE >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k / 4) * P::HALF + (k % 4) * 32) >> 4;
            umma_f16_lead(ts, qd + off, k0 + off, id_s, k ? 1u : 0u, lead);
          }
          umma_commit_lead(&s_full[t], lead);
          umma_commit_lead(&empty[slot], lead);
        };
        ok = wait_for(q_full, np);
        ++np;
        // Steps of a chain: P V of a tile and the scores of its next one.  The chains take them in turn, 0 first, and hand
        // the turn over behind the scores: if the other's P V may come between the two, the chains fall into step, both
        // softmaxes (1200 cycles) run at once and then all products (2150): 3400 cycles a tile, 2950 so.  The turn is
        // handed over where the other chain has a step next; it has as many as this one, or chain 1 one less.  The next
        // scores wait for no slot that the other chain's step frees: there are four at least.
        const int first = w.first(t), step = w.step(), count = w.count(t), other = w.count(t ^ 1);
        auto pass_by = [&](int j) {      // the other chain's tile: not read here
          ok = wait_tile(i0 + 2 * j) && wait_tile(i0 + 2 * j + 1);
          if (ok && lead) {
            mbar_arrive(&empty[(i0 + 2 * j) % P::SLOTS]);
            mbar_arrive(&empty[(i0 + 2 * j + 1) % P::SLOTS]);
          }
          __syncwarp();
        };
        if (!both)
          for (int j = 0; ok && j < first && j < w.tiles; ++j) pass_by(j);
        if (ok && count > 0) {
          ok = wait_tile(i0 + 2 * first);
          if (ok) {
            tc_fence_after();
            scores(i0 + 2 * first);
          }
        }
        for (int k = 0; ok && k < count; ++k) {
          const int j = first + k * step, iv = i0 + 2 * j + 1;
          ok = wait_tile(iv) && wait_for(&p_full[t], n);
          if (ok && (t || k > 0)) {   // (chain 1 has had a step before each of chain 0's but the first)
            ok = wait_for(&turn[t], turns);
            ++turns;
          }
          if (!ok) break;
          tc_fence_after();
          const int slot = of_warp(iv % P::SLOTS);
          const uint64_t v0 = vd + (uint32_t)slot * (P::TILE >> 4);
#pragma unroll
          for (int e = 0; e < kN / 16; ++e)   // O += P V_j
            umma_f16_tmem_a_lead(td, ts + 8 * e, v0 + e * (2048 >> 4), id_o, k || e ? 1u : 0u, lead);
          umma_commit_lead(&o_done[t], lead);
          umma_commit_lead(&empty[slot], lead);
          ++n;
          if (!both && j + 1 < w.tiles) pass_by(j + 1);
          if (ok && k + 1 < count) {     // over P: issued behind the product that reads it
            ok = wait_tile(i0 + 2 * (j + step));
            if (!ok) break;
            tc_fence_after();
            scores(i0 + 2 * (j + step));
          }
          if (ok && lead && (t ? k + 1 < other : k < other)) mbar_arrive(&turn[t ^ 1]);
          __syncwarp();
        }
        i0 += 2 * w.tiles;
      }
    }
  } else if (warp >= P::kWiden) {
    // ---- stored tiles to fp16: a thread has 16 elements of a row at a time
    if constexpr (P::LOW) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(P::OTHER_REGS));
      begin();
      constexpr int PR = D / 16;
      const int me = tid - 32 * P::kWiden, p = me % PR, swap = (p / 4) & 1, c0 = 2 * (p % 4) + swap;
      int i = 0;
      bool ok = true;
      while (ok && pieces.next(w)) {
        for (int j = 0; ok && j < w.tiles; ++j) {
          const int rows = w.hb - (w.pos0 + j * kN) < kN ? w.hb - (w.pos0 + j * kN) : kN;
          for (int x = 0; ok && x < 2; ++x, ++i) {
            const int st = i % P::STAGES, sl = i % P::SLOTS;
            ok = wait_for(&raw_full[st], i / P::STAGES) && (i < P::SLOTS || wait_for(&empty[sl], i / P::SLOTS - 1));
            if (!ok) break;
            const uint8_t* raw = sraw + st * P::RAW;
            uint8_t* to = skv + sl * P::TILE + (p / 4) * P::HALF;
            constexpr int kRowsAt = 32 * P::kWidenWarps / PR, kAhead = kN / kRowsAt;   // rows at a time; blocks of a thread: all of a tile
#pragma unroll 1
            for (int r0 = me / PR; r0 < kN; r0 += kAhead * kRowsAt) {
              uint4 u[kAhead];       // E2M1: codes and the scale
#pragma unroll
              for (int k = 0; k < kAhead; ++k) {
                const int row = r0 + k * kRowsAt;
                if constexpr (P::F8) {
                  u[k] = *reinterpret_cast<const uint4*>(raw + row * P::RB + 16 * p);
                } else {
                  const uint2 x2 = *reinterpret_cast<const uint2*>(raw + row * P::RB + 8 * p);
                  u[k] = make_uint4(x2.x, x2.y, raw[kN * P::RB + row * P::SB + p], 0);
                }
              }
#pragma unroll
              for (int k = 0; k < kAhead; ++k) {
                const int row = r0 + k * kRowsAt;
                uint32_t y[8];
                if constexpr (P::F8) {
                  const uint32_t b4[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
                  for (int e = 0; e < 8; ++e) y[e] = e & 1 ? e4m3x2_high_to_half2(b4[e / 2]) : e4m3x2_to_half2(b4[e / 2]);
                } else {
                  const uint32_t s2 = e4m3x2_to_half2(__byte_perm(u[k].z, 0, 0x4400));
                  e2m1x8_to_half2(u[k].x, *reinterpret_cast<uint32_t(*)[4]>(y));
                  e2m1x8_to_half2(u[k].y, *reinterpret_cast<uint32_t(*)[4]>(y + 4));
#pragma unroll
                  for (int e = 0; e < 8; ++e) y[e] = mul_half2(y[e], s2);
                }
                const uint4 zero = make_uint4(0, 0, 0, 0);
                const uint4 z0 = row < rows ? make_uint4(y[0], y[1], y[2], y[3]) : zero;
                const uint4 z1 = row < rows ? make_uint4(y[4], y[5], y[6], y[7]) : zero;
                // (lanes of the second 64 columns store their second piece first: other banks than the first 64's)
                uint8_t* line = to + row * 128;
                *reinterpret_cast<uint4*>(line + 16 * (c0 ^ (row & 7))) = swap ? z1 : z0;
                *reinterpret_cast<uint4*>(line + 16 * (c0 ^ 1 ^ (row & 7))) = swap ? z0 : z1;
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&full[sl]);
              mbar_arrive(&raw_empty[st]);
            }
            __syncwarp();
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(P::SOFT_REGS));
    // ---- softmax: thread r of four warps owns row r of its chain
    const int t = warp >> 2, row = 32 * (warp & 3) + lane;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t sc = lanes + kS + t * kChain, oc = lanes + kO + t * kChain;
    const float base = a.scale * kLog2e;
    int np = 0, cnt = 0;             // pieces, key tiles of this chain so far
    bool ok = true;
    begin();
    while (ok && pieces.next(w)) {
      {
        // the queries: 16 or 8 lanes a row, all eight warps both tiles
        if (np > 0) ok = wait_for(q_free, np - 1);   // all rows of the piece before have seen their last scores
        if (!ok) break;
        constexpr int LR = D / 8;
        const float ks = base * (P::LOW && c.k_scale ? c.k_scale[(size_t)layer * c.n_kv_heads + w.hk] : 1.0f);
        const int rows = w.both() ? 2 * kM : kM, p = lane % LR;
        const uint32_t at = smem_addr(sq) + (p / 8) * P::HALF;
        // (loops that are hardly unrolled: this code is cold, and fetching it took 26,000 cycles)
        constexpr int kStep = 8 * (32 / LR);   // rows of all warps at a time
        const int r_first = warp * (32 / LR) + lane / LR, di = kStep / g, dh = kStep - di * g;
        const int i_first = (w.rows0 + r_first) / g;
        int h = w.rows0 + r_first - i_first * g;
        const long long by = di * a.q_token + dh * a.q_head, carry = a.q_token - g * a.q_head;
        const uint16_t* from = q + (w.c0 + i_first) * a.q_token + (w.hk * g + h) * a.q_head + 8 * p;
        uint32_t to = at + r_first * 128 + 16 * ((p % 8) ^ (r_first & 7));   // (kStep is a multiple of 8)
#pragma unroll 2
        for (int r = r_first; r < rows; r += kStep) {
          if (r - kM >= 0 && r - kM < kStep) to += P::TILE - P::HALF;   // into the second tile (its rows follow on the first's)
          cp_async_16_zfill(to, r < w.rows ? from : q, r < w.rows);
          if (p == 0 && !(P::LOW && DT == QRE_BF16)) row_scale[r] = ks;
          to += kStep * 128;
          from += by;
          h += dh;
          if (h >= g) {
            h -= g;
            from += carry;
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if constexpr (P::LOW && DT == QRE_BF16) {
          // to fp16: the largest element of a row to [2^14, 2^15): exact but for elements 2^-29 times smaller, which
          // round to 2^-39 of it
          __syncwarp();
          constexpr int kAhead = 4;  // rows of a lane at a time (rows is a multiple of kAhead * kStep)
          uint8_t* line = sq + (p / 8) * P::HALF + 16 * ((p % 8) ^ (r_first & 7));
#pragma unroll 1
          for (int r0 = r_first; r0 < rows; r0 += kAhead * kStep) {
            uint4* word[kAhead];
            uint4 x[kAhead];
            float big[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
              const int r = r0 + u * kStep;
              word[u] = reinterpret_cast<uint4*>(line + r / kM * P::TILE + r % kM * 128);
              x[u] = *word[u];
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
              float y[8];
              unpack8<DT>(x[u], y);
              big[u] = 0.0f;
#pragma unroll
              for (int e = 0; e < 8; ++e) big[u] = fmaxf(big[u], fabsf(y[e]));
            }
#pragma unroll
            for (int d = LR / 2; d > 0; d >>= 1)
#pragma unroll
              for (int u = 0; u < kAhead; ++u) big[u] = fmaxf(big[u], __shfl_xor_sync(0xffffffffu, big[u], d));
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
              const int e = (int)((__float_as_uint(big[u]) >> 23) & 255) - 127;
              const int up = e >= 128 || big[u] == 0.0f ? 0 : (14 - e < 126 ? 14 - e : 126);
              const float f = __uint_as_float((uint32_t)(up + 127) << 23);
              float y[8];
              unpack8<DT>(x[u], y);
#pragma unroll
              for (int e2 = 0; e2 < 8; ++e2) y[e2] *= f;
              *word[u] = pack8<QRE_FP16>(y);
              if (p == 0) row_scale[r0 + u * kStep] = ks * __uint_as_float((uint32_t)(127 - up) << 23);
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
        ok = wait_for(q_full, np);   // all rows' factors are there
        ++np;
        if (!ok) break;
      }
      const int valid = w.valid(t);
      const float s2 = row_scale[(w.both() ? t * kM : 0) + row];
      const bool idle = 32 * (warp & 3) >= valid;   // rows that do not exist: whatever P holds stays in their own O
      float m = -INFINITY, l = 0.0f;                // reference (base 2) and sum
      const int tiles = w.count(t);
      for (int jj = 0; jj < tiles; ++jj, ++cnt) {
        const int j = w.first(t) + jj * w.step();
        const int seen = w.hb - (w.pos0 + j * kN);   // keys of the tile
        ok = wait_for(&s_full[t], cnt);
        if (!ok) break;
        if (!idle) {
          tc_fence_after();
          if (seen < kN) {           // the last tile: what is behind the end scores -infinity
#pragma unroll 1
            for (int b = seen / 32; b < 4; ++b) {
              uint32_t x[32];
              tmem_ld_32x32b_x32(sc + 32 * b, x);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (32 * b + e >= seen) x[e] = 0xff800000u;
              tmem_st_32x32b_x32(sc + 32 * b, x);
            }
            tmem_st_wait();
          }
          uint32_t p[64];
          float sum;
          // Once, or again with the reference moved
#pragma unroll 1
          for (bool moved = false;; moved = true) {
            const float off = m == -INFINITY ? 0.0f : -m;
            const uint64_t s22 = pair(s2, s2), off2 = pair(off, off);
            uint64_t part[2] = {0, 0};
            uint32_t xs[2][32];      // the next 32 scores come meanwhile
            tmem_ld_32x32b_x32(sc, xs[0]);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              tmem_ld_wait();
              if (b < 3) tmem_ld_32x32b_x32(sc + 32 * (b + 1), xs[(b + 1) & 1]);
              uint32_t(&x)[32] = xs[b & 1];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float2 z = unpair(fma2(pair(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), s22, off2));
                const float p0 = ex2(z.x), p1 = ex2(z.y);
                part[e & 1] = add2(part[e & 1], pair(p0, p1));
                p[16 * b + e] = pack2<P::PT>(p0, p1);   // the weights of the product are rounded; the sum is not
              }
            }
            const float2 u = unpair(add2(part[0], part[1]));
            sum = u.x + u.y;
            if (moved || !__any_sync(0xffffffffu, m == -INFINITY || sum > kMostSum)) break;
            // the reference moves with the maximum so far
            float mx = -INFINITY;
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
              uint32_t x[32];
              tmem_ld_32x32b_x32(sc + 32 * b, x);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; e += 2) mx = max3(mx, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
            }
            const float to = fmaxf(m, mx * s2 - kLift<P::BF>);
            const float f = m == to ? 1.0f : ex2(m - to);   // 2^-inf = 0 for the first keys
            m = to;
            l *= f;
            if (jj > 0) {            // behind the product of the tile before
              ok = wait_for(&o_done[t], cnt - 1);
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int b = 0; b < D / 32; ++b) {
                uint32_t x[32];
                tmem_ld_32x32b_x32(oc + 32 * b, x);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
                tmem_st_32x32b_x32(oc + 32 * b, x);
              }
            }
          }
          if (!ok) break;
          l += sum;
          tmem_st_32x32b_x32(sc, *reinterpret_cast<uint32_t(*)[32]>(p));
          tmem_st_32x32b_x32(sc + 32, *reinterpret_cast<uint32_t(*)[32]>(p + 32));
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t]);
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(q_free);
      // the part: O, reference and sum
      if (tiles > 0) ok = wait_for(&o_done[t], cnt - 1);
      if (!ok) break;
      if (!idle) {
        const long long at = w.out + (w.both() ? t * kM : t * w.rows) + row;
        if (tiles > 0) {
          tc_fence_after();
#pragma unroll 1
          for (int b = 0; b < D / 32; ++b) {
            uint32_t x[32];
            tmem_ld_32x32b_x32(oc + 32 * b, x);
            tmem_ld_wait();
            if (row < valid) {
              float* out = space.part_o + (size_t)at * D + 32 * b;
#pragma unroll
              for (int e = 0; e < 32; e += 8) st_global_32(out + e, x + e);
            }
          }
          tc_fence_before();
        }
        if (row < valid) space.part_ml[at] = make_float2(m, l);   // without tiles: -inf, and O is not read
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // a wait gave up: the loads and tensor-core work already issued complete before the CTA exits
    if (tid == 0) {
      const int n = *issued, ring = P::LOW ? P::STAGES : P::SLOTS;
      uint64_t* bars = P::LOW ? raw_full : full;
      for (int i = n - ring > 0 ? n - ring : 0; i < n; ++i) mbar_wait_drain(&bars[i % ring], (i / ring) & 1, status);
    }
    if (warp == P::kMma || warp == P::kMma + 1) {
      uint64_t* d = drain + (warp - P::kMma);
      if (elect_lane()) {
        umma_commit(d);
        mbar_wait_drain(d, 0, status);
      }
      __syncwarp();
    }
  }
  __syncthreads();
  if (warp == P::kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------- the join

// Where dimension d of head r of a unit lies in a part that the decode kernel left (floats; see Joined::write).
__device__ __forceinline__ int part_index(int cache_type, bool wide, int r, int d) {
  int i, row, high;
  if (cache_type == QRE_E2M1) {
    const int m = d & 3;
    row = (d & 31) >> 2;
    i = 2 * (d >> 5) + (wide ? m >> 1 : m & 1);
    high = wide ? m & 1 : m >> 1;
  } else if (cache_type == QRE_E4M3) {
    i = d >> 4;
    row = (d & 15) >> 1;
    high = d & 1;
  } else {
    i = d >> 4;
    row = d & 7;
    high = (d >> 3) & 1;
  }
  return (((wide ? 2 * i + (r >> 3) : i) * 4 + (r & 1) + 2 * high) << 5) + 4 * row + ((r & 7) >> 1);
}

// `ways` warps per query head: its own part (or parts, where the decode kernel's ranges cut its positions and the join is
// left to this kernel: a launch of its own took 5 us; their places are below 2^31 then, see attn_split.h) and those of the prefix in the order of the ranges, 20 at a time by
// a warp, the warps' results in their order.
constexpr int kAhead = 20;             // parts of a warp whose O is on its way together
template <int DT, int D>
__global__ void __launch_bounds__(256) shared_join_kernel(const __grid_constant__ qre_attn a, int n, int cache_type,
                                                          const float* __restrict__ v_scale, uint16_t* __restrict__ o,
                                                          float* __restrict__ lse, const __grid_constant__ Space s, Cuts cuts, int ways) {
  constexpr int E = D / 32;
  __shared__ float2 way_ml[8];
  __shared__ float way_x[8][D];
  grid_dependency_wait();
  grid_dependents_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, way = warp & (ways - 1);
  const long long id = ((long long)blockIdx.x * 8 + warp) / ways;
  if (id >= (long long)n * a.n_heads) return;   // (all of a CTA's warps where they have others to wait for)
  const int t = (int)(id / a.n_heads), h = (int)(id - (long long)t * a.n_heads);
  // what does not depend on the plan's answer is on its way beside it
  const Query x = s.query[t];
  const PlanHead head = *s.head;
  const float2 own_ml = s.own_ml[id];
  float own[E];
#pragma unroll
  for (int e = 0; e < E; ++e) own[e] = s.own_o[(size_t)id * D + E * lane + e];
  Header cut = {};
  int f0 = 0, f1 = 0;
  if (cuts.header) {
    const int32_t* firsts = reinterpret_cast<const int32_t*>(reinterpret_cast<const char*>(cuts.header) + kFirstsAt);
    cut = *cuts.header;
    f0 = firsts[t];
    f1 = firsts[t + 1];
  }
  const int g = a.n_heads / a.n_kv_heads, hk = h / g;
  const float vs = v_scale ? v_scale[hk] : 1.0f;
  float M = way ? -INFINITY : own_ml.x, L = way ? 0.0f : own_ml.y, X[E];
#pragma unroll
  for (int e = 0; e < E; ++e) X[e] = M == -INFINITY ? 0.0f : own[e];
  bool joined = false;               // of parts, all of its result if it has no hole
  if (f1 > f0) {
    const int blocks = (g + kRows - 1) / kRows, in_kv = h - hk * g, unit = hk * blocks + in_kv / kRows, r = in_kv % kRows;
    const int nch = f1 - f0, u0 = f0 * a.n_kv_heads * blocks + unit * nch;
    const PlanHead by{(int)cut.total, cut.ranges, (int)cut.total / cut.ranges, (int)cut.total % cut.ranges};
    const int b0 = by.range_of(u0 + kUnitCost), b1 = by.range_of(u0 + nch - 1);
    if (b1 > b0) {                   // cut: what lies in own was not written
      const bool wide = g > 8;
      const size_t floats = (size_t)(wide ? 16 : 8) * (D + 2);
      joined = true;
      M = -INFINITY;
      L = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) X[e] = 0.0f;
      int at[E];
#pragma unroll
      for (int e = 0; e < E; ++e) at[e] = part_index(cache_type, wide, r, E * lane + e);
#pragma unroll 4
      for (int b = way ? b1 + 1 : b0; b <= b1; ++b) {
        // the first part lies in its range's first place when the unit begins there too; the others begin theirs
        const float* part = cuts.parts + ((size_t)2 * b + (b == b0 && by.begin(b0) < u0 ? 1 : 0)) * floats;
        const float2 ml = reinterpret_cast<const float2*>(part + (wide ? 16 : 8) * D)[r];
        float y[E];
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = part[at[e]];
        const float to = fmaxf(M, ml.x);
        const float f = M == to ? 1.0f : ex2(M - to), fe = ml.x == to ? 1.0f : ex2(ml.x - to);
        M = to;
        L = L * f + ml.y * fe;
#pragma unroll
        for (int e = 0; e < E; ++e) X[e] = X[e] * f + y[e] * (fe * vs);
      }
    }
  }
  if (x.tiles == 0 && !joined) return;   // complete already
  if (x.tiles > 0) {
    const int rows = x.m * g, r = (t - x.c0) * g + h - hk * g, blocks = (rows + kUnitRows - 1) / kUnitRows, block = r / kUnitRows;
    const int per = x.tiles + kTileCost, in_block = rows - block * kUnitRows < kUnitRows ? rows - block * kUnitRows : kUnitRows;
    const int u0 = x.first + (hk * blocks + block) * per;
    const int b0 = head.range_of(u0 + kTileCost), b1 = head.range_of(u0 + per - 1);
    const long long base = 2 * ((long long)x.before * a.n_heads + (long long)hk * rows + block * kUnitRows) + r - block * kUnitRows;
    const int copies = in_block > kM ? 1 : 2, parts = (b1 - b0 + 1) * copies;
    auto row_of = [&](int i) {         // part i of the prefix
      const int b = b0 + i / copies, k = i - i / copies * copies;
      return base + (long long)kUnitRows * b + (long long)k * in_block;
    };
    for (int i0 = kAhead * way; i0 < parts; i0 += kAhead * ways) {   // a lane has a part's reference and sum
      const int mine = parts - i0 < kAhead ? parts - i0 : kAhead;
      float2 ml = make_float2(-INFINITY, 0.0f);
      if (lane < mine) ml = s.part_ml[row_of(i0 + lane)];
      float y[kAhead][E];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
#pragma unroll
        for (int e = 0; e < E; ++e) y[u][e] = 0.0f;
        if (u < mine) {
          const float* from = s.part_o + (size_t)row_of(i0 + u) * D + E * lane;
          if (E == 4) {
            const float4 z = *reinterpret_cast<const float4*>(from);
            y[u][0] = z.x, y[u][1] = z.y, y[u][E - 2] = z.z, y[u][E - 1] = z.w;
          } else {
            const float2 z = *reinterpret_cast<const float2*>(from);
            y[u][0] = z.x, y[u][1] = z.y;
          }
        }
      }
      const bool empty = ml.x == -INFINITY && ml.y == 0.0f;   // saw nothing: its O was not written
      float to = ml.x;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, d));
      to = fmaxf(M, to);
      const float f = M == to ? 1.0f : ex2(M - to), fe = empty ? 0.0f : ml.x == to ? 1.0f : ex2(ml.x - to);
      float sum = empty ? 0.0f : ml.y * fe;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      M = to;
      L = L * f + sum;
      const uint32_t there = __ballot_sync(0xffffffffu, !empty);
#pragma unroll
      for (int e = 0; e < E; ++e) X[e] *= f;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const float w = __shfl_sync(0xffffffffu, fe, u) * vs;
        if ((there >> u) & 1u)
#pragma unroll
          for (int e = 0; e < E; ++e) X[e] = fmaf(y[u][e], w, X[e]);
      }
    }
  }
  if (ways > 1) {                      // (what is asked above is the same for all warps of a head)
    if (way) {
      if (lane == 0) way_ml[warp] = make_float2(M, L);
#pragma unroll
      for (int e = 0; e < E; ++e) way_x[warp][E * lane + e] = X[e];
    }
    asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / ways), "r"(32 * ways) : "memory");
    if (way) return;
    for (int w = warp + 1; w < warp + ways; ++w) {
      const float2 ml = way_ml[w];
      if (ml.x == -INFINITY && ml.y == 0.0f) continue;
      const float to = fmaxf(M, ml.x);
      const float f = M == to ? 1.0f : ex2(M - to), fe = ml.x == to ? 1.0f : ex2(ml.x - to);
      M = to;
      L = L * f + ml.y * fe;
#pragma unroll
      for (int e = 0; e < E; ++e) X[e] = X[e] * f + way_x[w][E * lane + e] * fe;
    }
  }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  uint16_t* out = o + (size_t)t * a.o_token + (size_t)h * a.o_head + E * lane;
  if (E == 4)
    *reinterpret_cast<uint2*>(out) = make_uint2(pack2<DT>(X[0] * inv, X[1] * inv), pack2<DT>(X[E - 2] * inv, X[E - 1] * inv));
  else
    *reinterpret_cast<uint32_t*>(out) = pack2<DT>(X[0] * inv, X[1] * inv);
  if (lse && lane == 0) lse[id] = L == 0.0f ? -INFINITY : M * kLn2 + logf(L);
}

}  // namespace

size_t attn_shared_ws_bytes(const qre_attn& a, const qre_kv_cache& c, int n, int n_groups) {
  return space_of(a, c, n, n_groups, nullptr).bytes;
}

cudaError_t launch_attn_decode_shared(const qre_attn& a, const qre_kv_cache& c, int layer, int n, const int32_t* seqs,
                                      int n_groups, const int32_t* cu_group, const int32_t* common_len, int max_len,
                                      const void* q, void* o, float* lse, void* ws, int* status, cudaStream_t stream) {
  const Space s = space_of(a, c, n, n_groups, ws);
  // A prefix that is read again and again comes from L2, at some 11 TB/s; sharing costs launches, a join and the plan.  By
  // themselves / shared, us, for one group (8 KV heads of 128, 16 bits): 64 sequences of 612 positions 25 / 28, of 2148
  // 61 / 30; 16 of 2148 25 / 24, of 8292 63 / 31; 4 of 8292 26 / 28, of 32,868 62 / 46; 2 of 32,868 41 / 45.  In 4 bits: 16
  // of 2148 24 / 28, of 8292 45 / 30; 64 of 612 23 / 33, of 2148 43 / 32.  So it goes by the bytes that sharing can save;
  // those of 4 bits take longer.
  const long long all = 2ll * c.n_kv_heads * (long long)(kv_head_bytes(c) / c.page_size) * max_len;
  const long long saved = (c.dtype == QRE_E2M1 ? all * 3 / 2 : all) * (n > n_groups ? n - n_groups : 0);
  if (max_len > 0 && saved < kWorthBytes) return launch_attn_decode(a, c, layer, n, seqs, max_len, q, o, lse, s.decode, status, stream);
  const int g = a.n_heads / a.n_kv_heads, box = c.page_size < kN ? c.page_size : kN, grid = shared_grid();
  const bool low = c.dtype == QRE_E4M3 || c.dtype == QRE_E2M1;
  CUtensorMap tk = {}, tv = {}, tk16 = {}, tv16 = {};
  if (!low) {
    const long long rows = (long long)c.n_pages * c.n_kv_heads * c.page_size;
    const size_t skip = (size_t)layer * rows * c.head_dim * 2;
    const char *k = static_cast<const char*>(c.k) + skip, *v = static_cast<const char*>(c.v) + skip;
    // (rows beyond 31 bits, which only a pool that is larger than the memory has, cannot be addressed)
    if (rows > 0x7fffffffll || !make_tmap_bf16(&tk, k, rows, c.head_dim, box) || !make_tmap_bf16(&tv, v, rows, c.head_dim, box) ||
        !make_tmap_bf16(&tk16, k, rows, c.head_dim, 16) || !make_tmap_bf16(&tv16, v, rows, c.head_dim, 16))
      return launch_attn_decode(a, c, layer, n, seqs, max_len, q, o, lse, s.decode, status, stream);
  }
  // Queries of a launch of the own positions' kernel: chunks are counted in 32 bits (see launch_attn_decode; a hole makes one
  // more)
  const long long chunk = chunk_of(c), held = (long long)c.max_pages * c.page_size;
  const long long places = (a.window > 0 && a.window < held ? a.window : held) / chunk + 3 + kUnitCost;
  int most = 0x7fffffffll / places < n ? (int)(0x7fffffffll / places) : n;
  most = most < kPartQueries ? most : kPartQueries;
  static std::atomic<uint32_t> calls{0};
  uint32_t token = ++calls;
  if (token == 0) token = ++calls;   // what the plan sets
  const Costs costs = costs_of(c, fitting_ctas<true>(a, c, n < most ? n : most));   // (of the first: it runs beside the prefixes)
  cudaError_t e = launch_dependent(shared_plan_kernel, dim3(1), dim3(1024), 0, stream, c, n, seqs, n_groups, cu_group,
                                   common_len, a.window, g, a.n_kv_heads, kN, grid, costs, s, token, status);
  if (e != cudaSuccess) return e;
  auto prefix = [&](auto dt, auto ct, auto d) -> cudaError_t {
    constexpr int DT = decltype(dt)::value, CT = decltype(ct)::value, D = decltype(d)::value;
    using P = Shape<DT, CT, D>;
    auto kernel = shared_prefix_kernel<DT, CT, D>;
    const cudaError_t err = ensure_smem_limit(reinterpret_cast<const void*>(kernel), P::BYTES);
    if (err != cudaSuccess) return err;
    return launch_dependent(kernel, dim3(grid), dim3(P::THREADS), (size_t)P::BYTES, stream, a, c, layer, seqs, n_groups,
                            static_cast<const uint16_t*>(q), tk, tv, tk16, tv16, box, s, wait_limit_ns(), test_stall_ns(),
                            status);
  };
  using B = std::integral_constant<int, QRE_BF16>;
  using H = std::integral_constant<int, QRE_FP16>;
  using E8 = std::integral_constant<int, QRE_E4M3>;
  using E4 = std::integral_constant<int, QRE_E2M1>;
  auto by_dim = [&](auto dt, auto ct) {
    return a.head_dim == 64 ? prefix(dt, ct, std::integral_constant<int, 64>{}) : prefix(dt, ct, std::integral_constant<int, 128>{});
  };
  const bool bf = a.dtype == QRE_BF16;
  if (c.dtype == QRE_E4M3) e = bf ? by_dim(B{}, E8{}) : by_dim(H{}, E8{});
  else if (c.dtype == QRE_E2M1) e = bf ? by_dim(B{}, E4{}) : by_dim(H{}, E4{});
  else e = bf ? by_dim(B{}, B{}) : by_dim(H{}, H{});
  if (e != cudaSuccess) return e;

  // The sequences' own positions
  const bool leave = most >= n && shared_join_counts(n, places, (long long)a.n_kv_heads * ((g + kRows - 1) / kRows));
  Cuts cuts = {};
  for (int i = 0; i < n; i += most) {
    const int m = n - i < most ? n - i : most;
    const Own own{s.hole + i, s.own_o + (size_t)i * a.n_heads * a.head_dim, s.own_ml + (size_t)i * a.n_heads, i == 0,
                  token, s.start};
    e = launch_part<true>(a, c, layer, m, seqs ? seqs + i : nullptr, i, max_len, static_cast<const uint16_t*>(q) + i * a.q_token,
                          static_cast<uint16_t*>(o) + i * a.o_token, lse ? lse + (size_t)i * a.n_heads : nullptr, own, s.decode,
                          status, stream, leave ? &cuts : nullptr);
    if (e != cudaSuccess) return e;
  }
  const float* v_scale = low && c.v_scale ? c.v_scale + (size_t)layer * c.n_kv_heads : nullptr;
  const int ways = shared_join_ways(n, a.n_heads, a.n_kv_heads, n_groups, grid, kUnitRows, kAhead);
  const long long heads = (long long)n * a.n_heads;
  const dim3 ctas((unsigned)((heads * ways + 7) / 8));
  auto join = [&](auto kernel) {
    return launch_dependent(kernel, ctas, dim3(256), 0, stream, a, n, c.dtype, v_scale, static_cast<uint16_t*>(o), lse, s,
                            cuts, ways);
  };
  if (bf) return a.head_dim == 64 ? join(shared_join_kernel<QRE_BF16, 64>) : join(shared_join_kernel<QRE_BF16, 128>);
  return a.head_dim == 64 ? join(shared_join_kernel<QRE_FP16, 64>) : join(shared_join_kernel<QRE_FP16, 128>);
}

}  // namespace qre
