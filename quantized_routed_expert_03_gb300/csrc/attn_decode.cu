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
// contiguous ranges, one per CTA, whatever the lengths are; a CTA's eight warps
// take the chunks of its range in turn.  The lengths stay on the device: every
// CTA sums them up for itself.  A unit that lies inside one range is finished
// there; one that is cut leaves a part (o, m, l in fp32) per CTA in the
// workspace, and a second, dependent launch joins the parts in the order of the
// CTAs, so results do not depend on timing.
//
// A warp runs on its own between the ends of units: it fills a ring of chunks in
// shared memory with cp.async (16-byte pieces, rows that are not seen zero-filled,
// so what they hold never reaches a product) and multiplies with mma.sync
// (m16n8k16), keys and dimensions on the 16 side, heads on the 8 side:
//   S^T = K Q^T (16 keys x 8 heads), O^T += V^T P^T (16 dimensions x 8 heads);
// P turns from the first product's layout into the second's by one 8 x 8
// transpose (movmatrix).  Nothing is padding with 8 heads per KV head; tcgen05
// would want 128 rows.  More than 16 heads per KV head run as several units over
// the same keys, which then come from L2.  Two CTAs share an SM, so that one
// streams while the other joins its warps at the end of a unit.
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
constexpr int kMaxParts = 1024;       // CTAs of the main kernel at most

// What CTA b of the main kernel leaves for the join, in the workspace.
struct CutInfo {
  long long u0, u1;   // chunks of the unit that range b begins in; u0 < begin of range b iff the unit is cut there
  long long total;    // chunks of the call
  int t, block;       // query and head block of the unit
  int ctas, valid;
};

__device__ __forceinline__ long long range_begin(int c, int ctas, long long total) { return total * c / ctas; }

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
  // largest sum of a chunk's weights against a standing reference (fp16 weights end at 65504)
  static constexpr float kMost = BF ? 1.1529215e18f /* 2^60 */ : 32768.0f;

  // Byte offset of piece `col` of row `row` in a tile: pieces of a 128-byte line
  // are permuted by the row, so the eight rows that ldmatrix reads at one column
  // lie in different banks.
  static __device__ __forceinline__ uint32_t at(int row, int col) {
    return (uint32_t)(row * RB + 16 * (PR >= 8 ? col ^ (row & 7) : col ^ ((row >> 1) & 3)));
  }
};

struct Seq {
  int row, len, first;   // table row, length, chunks of the queries before
};

template <int DT, int CT, int D, int NH>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    attn_decode_kernel(const __grid_constant__ qre_attn a, const __grid_constant__ qre_kv_cache c, int layer, int n,
                       const int32_t* __restrict__ seqs, const uint16_t* __restrict__ q, uint16_t* __restrict__ o,
                       float* __restrict__ lse, CutInfo* __restrict__ cuts, float* __restrict__ parts, int stages,
                       int* status) {
  using K = Decode<DT, CT, D, NH>;
  constexpr int CK = K::CK, KS = K::KS;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem + (size_t)(threadIdx.x >> 5) * stages * 2 * kTile;   // this warp's
  float* buf = reinterpret_cast<float*>(smem + (size_t)kWarps * stages * 2 * kTile);   // [kWarps][8][64]
  float2* ml = reinterpret_cast<float2*>(buf + kWarps * 8 * 64);                       // [kWarps][kRows]
  Seq* sq = reinterpret_cast<Seq*>(ml + kWarps * kRows);                               // [n + 1]
  __shared__ int scan_part[kWarps];
  __shared__ int scan_total;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = a.n_heads / a.n_kv_heads;
  const int blocks = (g + kRows - 1) / kRows;       // head blocks of a KV head
  const int units = a.n_kv_heads * blocks;          // units of a sequence
  const int ps_shift = 31 - __clz(c.page_size);

  grid_dependency_wait();
  grid_dependents_launch();

  // ---- the plan: chunks of every query, summed up
  int before = 0;
  for (int t0 = 0; t0 < n; t0 += kThreads) {
    const int t = t0 + tid;
    int row = 0, len = 0, ch = 0;
    if (t < n) {
      row = seqs ? seqs[t] : t;
      bool bad = row < 0 || row >= c.max_seqs;
      if (!bad) {
        len = c.seq_len[row];
        bad = len < 0 || len > (long long)c.max_pages * c.page_size;
      }
      if (bad) {
        if (blockIdx.x == 0) set_status(status, QRE_DEV_BAD_INDEX);
        len = row = 0;
      }
      const int lo = a.window > 0 && len > a.window ? len - a.window : 0;
      ch = len > 0 ? (len + CK - 1) / CK - lo / CK : 0;
    }
    int inc = ch;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += u;
    }
    if (lane == 31) scan_part[warp] = inc;
    __syncthreads();
    int base = before;
    for (int w = 0; w < warp; ++w) base += scan_part[w];
    if (t < n) {
      sq[t].row = row;
      sq[t].len = len;
      sq[t].first = base + inc - ch;
    }
    if (tid == kThreads - 1) scan_total = base + inc;
    __syncthreads();
    before = scan_total;
  }
  if (tid == 0) sq[n].first = before;
  __syncthreads();
  const long long total = (long long)before * units;
  // ranges of at least one chunk per warp
  const long long want = (total + kWarps - 1) / kWarps;
  const int ctas = (int)(want < gridDim.x ? want : gridDim.x);

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
  if ((int)blockIdx.x >= ctas) {
    if (tid == 0) cuts[blockIdx.x].valid = 0;
    return;
  }
  const long long c0 = range_begin(blockIdx.x, ctas, total), c1 = range_begin(blockIdx.x + 1, ctas, total);

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

  // A place in the flat list of chunks.
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
  auto advance = [&](Place& p, int by) {   // not past the last chunk of the list
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

  // ---- loader: this warp's chunks c0 + warp, c0 + warp + kWarps, ...
  long long li = c0 + warp;          // next chunk to fetch
  Place lp = li < c1 ? place_of(li, t_first) : Place{0, 0, 0, 1};
  int pages = 0;                     // lane j: page of positions 16 j .. 16 j + 15 of that chunk, -1 missing, -2 not seen
  auto look_up = [&]() {
    pages = -2;
    if (li < c1 && lane < K::NP) {
      const int len = sq[lp.t].len;
      const int lo = a.window > 0 && len > a.window ? len - a.window : 0;
      const int pos = (lo / CK + lp.ck) * CK + 16 * lane;
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
      const int pos0 = (lo / CK + lp.ck) * CK;
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
      li += kWarps;
      if (li < c1) advance(lp, kWarps);
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
  long long next = c0 + warp;        // this warp's next chunk to compute
  while (s0 < c1) {
    const long long u0 = s0 - cp.ck, u1 = u0 + cp.nch;
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

    for (; next < s1; next += kWarps) {
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

      const int pos0 = (lo / CK + (int)(next - u0)) * CK;
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
      if (__any_sync(0xffffffffu, redo)) {   // the reference moves to the maximum so far
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < K::NP; ++i) mx = fmaxf(mx, fmaxf(s[i][nh][e], s[i][nh][e + 2]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float to = fmaxf(m[nh][e], mx * s2[nh][e]);
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

    // ---- end of the unit in this range: join the warps (the next unit's queries come meanwhile)
    Place np = cp;
    if (s1 < c1) {
      advance(np, (int)(s1 - s0));
      ask_queries(np);
    }
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nh][e] += __shfl_xor_sync(0xffffffffu, l[nh][e], d);
        if (r4 == 0) ml[warp * kRows + 8 * nh + 2 * j4 + e] = make_float2(m[nh][e], l[nh][e]);
      }
    const bool whole = s0 == u0 && s1 == u1;
    float* part = parts + ((size_t)2 * blockIdx.x + (s0 == c0 ? 0 : 1)) * kRows * (D + 2);
    // eight heads by 64 dimensions at a time
#pragma unroll
    for (int pass = 0; pass < NH * (D / 64); ++pass) {
      const int nh = pass / (D / 64), half = pass % (D / 64);
      float* b = buf + (size_t)warp * 8 * 64;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // heads are spread over the banks by permuting eights of dimensions
          const int d0 = 16 * i + (K::F8 ? 2 * r4 : r4), d1 = 16 * i + (K::F8 ? 2 * r4 + 1 : r4 + 8), x = 8 * j4;
          b[(2 * j4 + e) * 64 + (d0 ^ x)] = acc[4 * half + i][nh][e];
          b[(2 * j4 + e) * 64 + (d1 ^ x)] = acc[4 * half + i][nh][e + 2];
        }
      __syncthreads();
      {
        const int rr = tid >> 4, d = (tid & 15) * 4, r = rr + 8 * nh, dd = 64 * half + d;
        if (r < rows) {
          float M = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * kRows + r].x);
          float L = 0.0f;
          float4 sum = make_float4(0, 0, 0, 0);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 e = ml[w * kRows + r];
            // a warp that saw nothing (m = -inf, l = 0) counts nothing; a NaN in l stays one
            const float f = e.x == -INFINITY && e.y == 0.0f ? 0.0f : ex2(e.x - M);
            const float4 x = *reinterpret_cast<const float4*>(buf + (size_t)(w * 8 + rr) * 64 + (d ^ (8 * (rr >> 1))));
            L += e.y * f;
            sum.x += x.x * f;
            sum.y += x.y * f;
            sum.z += x.z * f;
            sum.w += x.w * f;
          }
          if (whole) {
            const float inv = L == 0.0f ? 0.0f : vs / L;
            *reinterpret_cast<uint2*>(o + (size_t)t * a.o_token + (size_t)(h0 + r) * a.o_head + dd) =
                make_uint2(pack2<DT>(sum.x * inv, sum.y * inv), pack2<DT>(sum.z * inv, sum.w * inv));
            if (lse && dd == 0) lse[(size_t)t * a.n_heads + h0 + r] = L == 0.0f ? -INFINITY : M * kLn2 + logf(L);
          } else {
            *reinterpret_cast<float4*>(part + r * D + dd) = sum;
            if (dd == 0) *reinterpret_cast<float2*>(part + kRows * D + 2 * r) = make_float2(M, L);
          }
        }
      }
      __syncthreads();
    }
    if (s0 == c0 && tid == 0) {
      CutInfo ci;
      ci.u0 = u0;
      ci.u1 = u1;
      ci.total = total;
      ci.t = t;
      ci.block = cp.unit;
      ci.ctas = ctas;
      ci.valid = 1;
      cuts[blockIdx.x] = ci;
    }
    s0 = s1;
    cp = np;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Joins the parts of the units that were cut: CTA b takes the unit that the begin
// of range b cuts, if no earlier begin cuts it too.
template <int DT, int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ qre_attn a,
                                                        const float* __restrict__ v_scale, uint16_t* __restrict__ o,
                                                        float* __restrict__ lse, const CutInfo* __restrict__ cuts,
                                                        const float* __restrict__ parts) {
  __shared__ float2 ml[kRows];
  grid_dependency_wait();
  grid_dependents_launch();
  const int b = blockIdx.x + 1;
  const CutInfo ci = cuts[b];
  if (!ci.valid) return;
  if (ci.u0 >= range_begin(b, ci.ctas, ci.total) || range_begin(b - 1, ci.ctas, ci.total) > ci.u0) return;
  int e = b;   // last range of the unit
  while (e + 1 < ci.ctas && range_begin(e + 1, ci.ctas, ci.total) < ci.u1) ++e;
  const int g = a.n_heads / a.n_kv_heads, blocks = (g + kRows - 1) / kRows;
  const int hk = ci.block / blocks, h0 = hk * g + (ci.block - hk * blocks) * kRows;
  const int rows = (hk + 1) * g - h0 < kRows ? (hk + 1) * g - h0 : kRows;
  // part of range c: its first slot when the unit's share begins the range, else its second
  auto part = [&](int c) {
    return parts + ((size_t)2 * c + (ci.u0 <= range_begin(c, ci.ctas, ci.total) ? 0 : 1)) * kRows * (D + 2);
  };
  const float vs = v_scale ? v_scale[hk] : 1.0f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r = warp; r < rows; r += 8) {
    float M = -INFINITY, L = 0.0f;
    for (int c = b - 1 + lane; c <= e; c += 32) M = fmaxf(M, part(c)[kRows * D + 2 * r]);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
    for (int c = b - 1 + lane; c <= e; c += 32) {
      const float2 x = *reinterpret_cast<const float2*>(part(c) + kRows * D + 2 * r);
      L += x.x == -INFINITY && x.y == 0.0f ? 0.0f : x.y * ex2(x.x - M);
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) L += __shfl_xor_sync(0xffffffffu, L, w);
    if (lane == 0) ml[r] = make_float2(M, L);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (D / 4); i += 256) {
    const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
    const float M = ml[r].x, L = ml[r].y;
    float4 sum = make_float4(0, 0, 0, 0);
#pragma unroll 4
    for (int c = b - 1; c <= e; ++c) {
      const float* p = part(c);
      const float2 x = *reinterpret_cast<const float2*>(p + kRows * D + 2 * r);
      const float4 y = *reinterpret_cast<const float4*>(p + r * D + d);
      const float f = x.x == -INFINITY && x.y == 0.0f ? 0.0f : ex2(x.x - M);
      sum.x += y.x * f;
      sum.y += y.y * f;
      sum.z += y.z * f;
      sum.w += y.w * f;
    }
    const float inv = L == 0.0f ? 0.0f : vs / L;
    *reinterpret_cast<uint2*>(o + (size_t)ci.t * a.o_token + (size_t)(h0 + r) * a.o_head + d) =
        make_uint2(pack2<DT>(sum.x * inv, sum.y * inv), pack2<DT>(sum.z * inv, sum.w * inv));
    if (lse && d == 0) lse[(size_t)ci.t * a.n_heads + h0 + r] = L == 0.0f ? -INFINITY : M * kLn2 + logf(L);
  }
}

int decode_grid() {
  const int sms = device_sm_count();
  const int n = (sms <= 0 ? 152 : sms) * kCtasPerSm;
  return n < kMaxParts ? n : kMaxParts;
}

size_t cut_bytes(int grid) { return ((size_t)grid * sizeof(CutInfo) + 255) & ~(size_t)255; }

}  // namespace

size_t attn_decode_ws_bytes(const qre_attn& a, const qre_kv_cache&, int) {
  const int grid = decode_grid();
  return cut_bytes(grid) + (size_t)2 * grid * kRows * (a.head_dim + 2) * sizeof(float);
}

cudaError_t launch_attn_decode(const qre_attn& a, const qre_kv_cache& c, int layer, int n, const int32_t* seqs,
                               int max_len, const void* q, void* o, float* lse, void* ws, int* status,
                               cudaStream_t stream) {
  const int grid = decode_grid();
  const int g = a.n_heads / a.n_kv_heads;
  const size_t fixed = (size_t)kWarps * 8 * 64 * sizeof(float) + kWarps * kRows * sizeof(float2) +
                       (size_t)(n + 1) * sizeof(Seq);
  // what the CTAs of an SM share (1 KB of each is the system's, and the kernel's static arrays)
  const long long room = ((long long)device_max_smem_optin() + 1024) / kCtasPerSm - 1024 - 128 - (long long)fixed;
  int stages = (int)(room / (kWarps * 2 * kTile));
  stages = stages < 2 ? 2 : (stages > 3 ? 3 : stages);   // a long list takes room: then one CTA has the SM
  const size_t smem = (size_t)stages * kWarps * 2 * kTile + fixed;
  CutInfo* cuts = static_cast<CutInfo*>(ws);
  float* parts = reinterpret_cast<float*>(static_cast<char*>(ws) + cut_bytes(grid));
  const float* v_scale = c.dtype == QRE_E4M3 && c.v_scale ? c.v_scale + (size_t)layer * c.n_kv_heads : nullptr;
  auto go = [&](auto kernel, auto join) -> cudaError_t {
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), (int)smem);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kernel, dim3(grid), dim3(kThreads), smem, stream, a, c, layer, n, seqs,
                         static_cast<const uint16_t*>(q), static_cast<uint16_t*>(o), lse, cuts, parts, stages, status);
    if (e != cudaSuccess || grid < 2) return e;
    return launch_dependent(join, dim3(grid - 1), dim3(256), 0, stream, a, v_scale, static_cast<uint16_t*>(o), lse,
                            const_cast<const CutInfo*>(cuts), const_cast<const float*>(parts));
  };
  auto pick = [&](auto dt, auto ct, auto d) {
    constexpr int DT = decltype(dt)::value, CT = decltype(ct)::value, D = decltype(d)::value;
    return g > 8 ? go(attn_decode_kernel<DT, CT, D, 2>, attn_join_kernel<DT, D>)
                 : go(attn_decode_kernel<DT, CT, D, 1>, attn_join_kernel<DT, D>);
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

}  // namespace qre
