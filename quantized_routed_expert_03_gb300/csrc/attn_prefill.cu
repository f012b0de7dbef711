// attn_prefill.cu -- attention over packed prompts.
//
// o_i = sum_j softmax_j(scale q_i . k_j) v_j over the keys that query i sees, in
// one pass: with the running maximum m and sum l (fp32, base 2),
//   m' = max(m, max s), l' = l 2^(m - m') + sum 2^(s - m'), o' alike.
//
// Bound: 4 D flops for each (query head, key seen).  A tile of 128 queries x 128
// keys is 1024 cycles of an SM's tensor cores at D = 128 (S and P V, 512 each) and
// 16384 exponentials, 512 cycles at the 32 a cycle that were measured: the tensor
// cores bound it if the rest runs beside them.  At D = 64 both need 512.
//
// A CTA (one per SM, 512 threads) takes pieces of work: two query tiles of one
// sequence and one group of heads, tile rows = tokens x heads of one KV head, so
// that few tokens still fill a tile and K and V are fetched once for the group.
// Warps have one job each: one finds the work (clusterlaunchcontrol hands out the
// grid's indices, so CTAs that finish early take more; three pieces ahead), one
// fetches tiles by TMA (5 x 32 KB ring), two issue the products (tcgen05, S in
// tensor memory, P over it in 16 bits, O beside it), eight weight the scores, one
// thread per row, and four bring O out while the next piece goes on.
//
// What it measured (32 heads on 8, D = 128, bf16; cuBLAS: 1901 TFLOP/s): one causal
// prompt of 8192 tokens 354 us, 1.55 PFLOP/s (82 %); 16 prompts of up to 2048, 106
// Gflop, 115 us (48 %).  A pair of query tiles takes 2620 cycles per key tile of the
// 2048 that its products need.  What short prompts lose is lost between two pieces
// of work (some 6000 cycles): the first and the last key tile of a piece, cut by the
// mask, run code that is not in the instruction cache, and O is handed over.
// Steps on the prompt of 8192: one MMA thread and plain softmax 522 us; MMA issued
// by a converged warp, three-operand maximum, paired fp32 414; persistent, weights
// against a standing reference, P V begun on the first 96 keys, tiles in turn 384;
// output and work finding on warps of their own 358.  Slower: two threads a row
// (497), first parts of 64 keys (397), a query buffer released tile by tile (380).
#include <climits>
#include <type_traits>

#include "attn.cuh"
#include "internal.h"
#include "tc.cuh"

namespace qre {
namespace {

// See launch_attn_prefill.
constexpr int kFewKeys = 512, kFewLong = 256, kFewWork = 1 << 22, kFewTotal = 1 << 26;

// For a handful of keys, for what TMA cannot address (rows that repeat: a token
// stride of 0) and for calls without any key: one warp per (query token, head); a
// lane scores one key at a time, then has two neighbouring dimensions of each 64 for
// the values.
template <int DT, int D>
__global__ void __launch_bounds__(256, 2) attn_rows_kernel(const __grid_constant__ qre_attn a, int n_seqs, int total_q,
                                                        int total_k, const int32_t* __restrict__ cu_q,
                                                        const int32_t* __restrict__ cu_k,
                                                        const uint16_t* __restrict__ q, const uint16_t* __restrict__ k,
                                                        const uint16_t* __restrict__ v, uint16_t* __restrict__ o,
                                                        float* __restrict__ lse, int* status) {
  constexpr int W = D / 64;     // 32-bit words of a row for a lane
  constexpr int kAhead = 32 / W;   // keys whose values are on their way together, the first beside the keys
  __shared__ __align__(16) float qs[8][D];
  grid_dependency_wait();
  grid_dependents_launch();
  if (blockIdx.x == gridDim.x - 1) {   // the last block has no rows: it looks over the bounds
    for (int i = threadIdx.x; i < n_seqs; i += 256) {
      const int q0 = cu_q[i], q1 = cu_q[i + 1], k0 = cu_k[i], k1 = cu_k[i + 1];
      if (q0 < 0 || q1 < q0 || q1 > total_q || k0 < 0 || k1 < k0 || k1 > total_k) set_status(status, QRE_DEV_BAD_INDEX);
    }
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * 8 + warp;
  if (unit >= (long long)total_q * a.n_heads) return;
  const int t = (int)(unit / a.n_heads), h = (int)(unit % a.n_heads), hk = h / (a.n_heads / a.n_kv_heads);
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const uint32_t x = *reinterpret_cast<const uint32_t*>(q + (size_t)t * a.q_token + (size_t)h * a.q_head + 64 * w + 2 * lane);
    qs[warp][64 * w + 2 * lane] = bits_to_float<DT>(x & 0xffffu) * a.scale * kLog2e;
    qs[warp][64 * w + 2 * lane + 1] = bits_to_float<DT>(x >> 16) * a.scale * kLog2e;
  }
  int q0 = 0, q1 = 0, k0 = 0, k1 = 0;
  bool found = false;           // the first sequence that has the token
  for (int i0 = 0; i0 < n_seqs && !found; i0 += 128) {
    int b[4][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int i = i0 + 32 * c + lane;
      b[c][0] = b[c][1] = 0;    // has no token
      if (i < n_seqs) {
        b[c][0] = cu_q[i];
        b[c][1] = cu_q[i + 1];
        b[c][2] = cu_k[i];
        b[c][3] = cu_k[i + 1];
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const unsigned has = __ballot_sync(0xffffffffu, b[c][0] <= t && t < b[c][1]);
      if (!has || found) continue;
      const int at = __ffs(has) - 1;
      q0 = __shfl_sync(0xffffffffu, b[c][0], at);
      q1 = __shfl_sync(0xffffffffu, b[c][1], at);
      k0 = __shfl_sync(0xffffffffu, b[c][2], at);
      k1 = __shfl_sync(0xffffffffu, b[c][3], at);
      found = true;
    }
  }
  if (!found) return;
  if (q0 < 0 || q1 > total_q || k0 < 0 || k1 < k0 || k1 > total_k) return;
  int lo, hi;
  visible_range(k1 - k0 - (q1 - q0) + t - q0, k1 - k0, a.causal, a.window, lo, hi);
  __syncwarp();
  float m = -INFINITY, l = 0.0f, acc[2 * W] = {};
  for (int j0 = lo; j0 < hi; j0 += 32) {
    const int j = j0 + lane, keys = hi - j0 < 32 ? hi - j0 : 32;
    uint32_t y[kAhead][W];
    auto fetch = [&](int i0) {   // rows that are not seen are not read
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
#pragma unroll
        for (int w = 0; w < W; ++w)
          y[i][w] = i0 + i < keys ? *reinterpret_cast<const uint32_t*>(v + (size_t)(k0 + j0 + i0 + i) * a.v_token +
                                                                       (size_t)hk * a.v_head + 64 * w + 2 * lane)
                                  : 0u;
    };
    fetch(0);                    // beside the keys
    float x = -INFINITY;
    if (j < hi) {
      const uint16_t* kr = k + (size_t)(k0 + j) * a.k_token + (size_t)hk * a.k_head;
      float part[2] = {0.0f, 0.0f};
#pragma unroll
      for (int d = 0; d < D; d += 8) {
        const uint4 w = *reinterpret_cast<const uint4*>(kr + d);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          part[0] = fmaf(qs[warp][d + 2 * e], bits_to_float<DT>(u[e] & 0xffffu), part[0]);
          part[1] = fmaf(qs[warp][d + 2 * e + 1], bits_to_float<DT>(u[e] >> 16), part[1]);
        }
      }
      x = part[0] + part[1];
    }
    float mx = x;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    const float m2 = fmaxf(m, mx), f = m == -INFINITY ? 0.0f : exp2f(m - m2);
    const float p = j < hi ? exp2f(x - (m2 == -INFINITY ? 0.0f : m2)) : 0.0f;   // (keys that score -infinity count 0)
    float sum = p;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    l = l * f + sum;
    m = m2;
#pragma unroll
    for (int i = 0; i < 2 * W; ++i) acc[i] *= f;
    for (int i0 = 0; i0 < keys; i0 += kAhead) {
      if (i0) fetch(i0);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float pi = __shfl_sync(0xffffffffu, p, i0 + i);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          acc[2 * w] = fmaf(pi, bits_to_float<DT>(y[i][w] & 0xffffu), acc[2 * w]);
          acc[2 * w + 1] = fmaf(pi, bits_to_float<DT>(y[i][w] >> 16), acc[2 * w + 1]);
        }
      }
    }
  }
  const bool empty = hi <= lo;
  const float inv = empty ? 0.0f : 1.0f / l;
#pragma unroll
  for (int w = 0; w < W; ++w)
    *reinterpret_cast<uint32_t*>(o + (size_t)t * a.o_token + (size_t)h * a.o_head + 64 * w + 2 * lane) =
        pack2<DT>(acc[2 * w] * inv, acc[2 * w + 1] * inv);
  if (lse && lane == 0) lse[(size_t)t * a.n_heads + h] = empty ? -INFINITY : m * kLn2 + logf(l);
}

// ---------------------------------------------------------------- tensor cores

constexpr int kM = 128;            // rows of a query tile: kM / gp tokens x gp heads of one KV head
constexpr int kN = 128;            // keys of a tile
constexpr int kPart = 96;          // keys of a tile's first part (of two): P V of it starts while the rest is weighted
constexpr int kThreads = 512;
// warps 0-3: softmax of tile 0, 4-7: of tile 1, 8-11: output of both
constexpr int kStoreWarp = 8;
constexpr int kTmaWarp = 12, kMmaWarp = 13, kFindWarp = 15;   // MMA warps 13 and 14: one per query tile
constexpr int kWorks = 3;          // pieces of work known at a time: being stored, computed, fetched
// Registers: 512 x 128 at launch = 256 x 160 + 128 x 112 + 128 x 80.
constexpr int kSoftmaxRegs = 160, kStoreRegs = 112, kOtherRegs = 80;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kS0 = 0, kS1 = 128, kO0 = 256, kO1 = 384;   // tensor-memory columns; P overwrites its S
// A row's weights are taken against a reference that stays while the sum of a part's weights is at most this:
// fp16 weights end here; and values enter the accumulators times weights of up to this, so that finite ones must
// not overflow there.
constexpr float kMostWeight = 65504.0f;
// The weight, in base 2, of the maximum that sets a row's reference.  fp16 ends at 2^-24 below: with 0, keys under
// 2^-25 of the maximum count in the sum and not in O, and many of them weigh something (60,000 keys behind one that
// is 26 ahead of them in base 2: all of their 2^-10).  With 6 prefill_chunk takes 41.4 us, not 37.2: rows that see
// few keys in their first tile set a low reference, and their sums pass kMostWeight often.  bf16 has fp32's range.
// kMove: how far ahead of the reference a maximum is when it is moved; a sum of 96 above kMostWeight has one that is.
template <int DT>
constexpr float kUp = DT == QRE_FP16 ? 4.0f : 0.0f;
template <int DT>
constexpr float kMove = DT == QRE_FP16 ? 5.0f : 8.0f;

template <int D>
struct Plan {
  static constexpr int HALF = kN * 128;              // 64 columns of a 128-row tile, 128-byte rows
  static constexpr int TILE = HALF * (D / 64);
  static constexpr int SLOTS = D == 128 ? 5 : 10;    // K and V tiles in flight
  static constexpr int BYTES = 2 * TILE + SLOTS * TILE + 2048 + 768;   // tiles; sums; barriers
};

// mbar_wait_bounded without a call: the register split (setmaxnreg) leaves no room for the calling convention.
__device__ __forceinline__ bool mbar_wait_inline(uint64_t* bar, uint32_t parity, volatile int* abort, int* status,
                                                 uint64_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t deadline = global_timer_ns() + limit_ns;
  while (!mbar_try_wait_1us(bar, parity)) {
    if (*abort) return false;
    if (global_timer_ns() > deadline) {
      *abort = 1;
      set_status(status, QRE_DEV_TIMEOUT);
      return false;
    }
  }
  return true;
}

// A count in shared memory that one thread writes and others read beside its barriers.
__device__ __forceinline__ void store_release(int* p, int n) {
  asm volatile("st.release.cta.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(p)), "r"(n) : "memory");
}
__device__ __forceinline__ int load_acquire(const int* p) {
  int n;
  asm volatile("ld.acquire.cta.shared::cta.b32 %0, [%1];" : "=r"(n) : "r"(smem_addr(p)) : "memory");
  return n;
}

__device__ __forceinline__ void prefetch_tmap(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Of two 16-bit pairs the larger magnitudes, NaN if there is one.
template <int DT>
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  if (DT == QRE_BF16) {
    const __nv_bfloat162 r = __hmax2_nan(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&a)),
                                         __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  const __half2 r = __hmax2_nan(__habs2(*reinterpret_cast<const __half2*>(&a)), __habs2(*reinterpret_cast<const __half2*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ void st_global_32(void* p, const uint32_t* z) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(z[0]), "r"(z[1]), "r"(z[2]), "r"(z[3]),
               "r"(z[4]), "r"(z[5]), "r"(z[6]), "r"(z[7])
               : "memory");
}

// One piece of work: two query tiles of one sequence and head group, with what every warp wants to
// know of it (worked out once, by the warp that finds it: between two pieces every warp's way is
// on the critical path, and cold code takes long).
struct Range {
  int jb, je;   // key tiles [jb, je) of the sequence
};
struct alignas(16) Work {
  int q0, q_len, k0, k_len;   // the sequence
  int tok0;                   // first token, in the sequence
  int h0;                     // first head
  int end;                    // no more work
  int poison;                 // a value that is not finite was taken out of a key tile
  Range r[2];                 // key tiles of the two query tiles
  int jb, je;                 // of both
  int lo_last, hi_first;      // first key of the last token, end of the keys of the first
  int lo_max[2], hi_min[2];   // the same of each query tile
  __device__ __forceinline__ void plan(const qre_attn& a, int tt) {
    const int shift = k_len - q_len;   // position of token i is i + shift
#pragma unroll
    for (int t = 0; t < 2; ++t) {      // both bounds grow with the token
      const int ta = tok0 + t * tt, tb = ta + tt < q_len ? ta + tt : q_len;
      int lo, hi;
      r[t] = Range{0, 0};
      visible_range(ta + shift, k_len, a.causal, a.window, lo, hi_min[t]);
      visible_range(tb - 1 + shift, k_len, a.causal, a.window, lo_max[t], hi);
      if (ta < tb && hi > lo) {
        r[t].jb = lo / kN;
        r[t].je = (hi + kN - 1) / kN;
      }
    }
    if (r[0].je <= r[0].jb) r[0] = r[1];   // tokens that see nothing go along, so that tile 0 has keys if the work has
    jb = r[0].jb;
    je = r[1].je > r[1].jb ? r[1].je : r[0].je;
    hi_first = hi_min[0];
    lo_last = tok0 + tt < q_len ? lo_max[1] : lo_max[0];
  }
  // some token of the work does not see all of key tile j
  __device__ __forceinline__ bool special(int j) const { return j * kN < lo_last || (j + 1) * kN > hi_first; }
};

// Finds the piece of work of an index.  The longest come first, so that the last
// CTAs to finish end together: with at most 128 sequences the tiles of all
// sequences are ordered by their last key tile, with more (then each is short
// against the whole) by sequence.
class Finder {
 public:
  __device__ __forceinline__ Finder(int n_seqs, int total_q, int total_k, const int32_t* cu_q, const int32_t* cu_k, int pair_shift)
      : n_(n_seqs), tq_(total_q), tk_(total_k), cu_q_(cu_q), cu_k_(cu_k), shift_by_(pair_shift), pair_(1 << pair_shift) {
    lane_ = threadIdx.x & 31;
    if (n_ <= 128) {
      int top = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        load(32 * c + lane_, cnt_[c], shift_[c]);
        if (cnt_[c] > 0) top = max(top, (shift_[c] + cnt_[c] * pair_ - 1) / kN);
      }
      top_ = __reduce_max_sync(0xffffffffu, top);
    }
  }
  // False: no work of that index.
  __device__ __forceinline__ bool find(int b, int& seq, int& tile) {
    if (n_ <= 128) {
      if (b >= at_least(0)) return false;
      int lo = 0, hi = top_;          // the largest level with more than b tiles at or above it
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (at_least(mid) > b) lo = mid;
        else hi = mid - 1;
      }
      int rest = b - at_least(lo + 1);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int first = lowest(c, lo), e = cnt_[c] - first - (cnt_[c] - lowest(c, lo + 1));
        const int sum = (int)__reduce_add_sync(0xffffffffu, (unsigned)e);
        if (rest < sum) {
          pick(e, rest, c, first, seq, tile);
          return true;
        }
        rest -= sum;
      }
      return false;
    }
    if (b < base_) at_ = base_ = 0;   // indices come in ascending order: go on from the last one
    for (; at_ < n_; at_ += 32) {
      int cnt, shift;
      load(at_ + lane_, cnt, shift);
      const int sum = (int)__reduce_add_sync(0xffffffffu, (unsigned)cnt);
      if (b < base_ + sum) {
        pick(cnt, b - base_, at_ / 32, 0, seq, tile);
        tile = __shfl_sync(0xffffffffu, cnt, seq & 31) - 1 - tile;   // a sequence's longest first
        return true;
      }
      base_ += sum;
    }
    return false;
  }

 private:
  __device__ __forceinline__ void load(int i, int& cnt, int& shift) const {
    cnt = shift = 0;
    if (i < n_) {
      const int q0 = cu_q_[i], q1 = cu_q_[i + 1], k0 = cu_k_[i], k1 = cu_k_[i + 1];
      if (q0 >= 0 && q1 >= q0 && q1 <= tq_ && k0 >= 0 && k1 >= k0 && k1 <= tk_) {
        cnt = (q1 - q0 + pair_ - 1) >> shift_by_;
        shift = k1 - k0 - (q1 - q0);
      }
    }
  }
  // first tile of sequence (c, lane) whose last token stands at level * kN or later
  __device__ __forceinline__ int lowest(int c, int level) const {
    const int x = level * kN + 1 - shift_[c];
    const int i = level <= 0 || x <= 0 ? 0 : ((x + pair_ - 1) >> shift_by_) - 1;
    return i < cnt_[c] ? i : cnt_[c];
  }
  __device__ __forceinline__ int at_least(int level) const {
    int s = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) s += cnt_[c] - lowest(c, level);
    return (int)__reduce_add_sync(0xffffffffu, (unsigned)s);
  }
  // the `rest`-th of the lanes' e items
  __device__ __forceinline__ void pick(int e, int rest, int c, int first, int& seq, int& tile) const {
    int inc = e;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane_ >= d) inc += u;
    }
    const int w = __ffs(__ballot_sync(0xffffffffu, rest < inc)) - 1;
    seq = 32 * c + w;
    tile = __shfl_sync(0xffffffffu, first, w) + rest - __shfl_sync(0xffffffffu, inc - e, w);
  }
  int n_, tq_, tk_;
  const int32_t *cu_q_, *cu_k_;
  int shift_by_, pair_;   // tokens of a piece of work: 1 << shift_by_
  int lane_, top_ = 0, at_ = 0, base_ = 0;
  int cnt_[4], shift_[4];
};

template <int DT, int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc_kernel(const __grid_constant__ qre_attn a, int n_seqs, int total_q, int total_k, int gp_shift, int groups,
                   const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k,
                   const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap tv, int wide_o, int q_heads_move, int k_heads_move, int v_heads_move,
                   const uint16_t* __restrict__ v, uint16_t* __restrict__ o, float* __restrict__ lse,
                   uint64_t limit_ns, int* status) {
  using P = Plan<D>;
  extern __shared__ __align__(1024) uint8_t smem[];   // the swizzle goes by addresses; no static shared memory beside it
  uint8_t* sq = smem;                       // two query tiles
  uint8_t* skv = smem + 2 * P::TILE;        // ring of key and value tiles
  uint64_t* bar = reinterpret_cast<uint64_t*>(skv + P::SLOTS * P::TILE);
  uint64_t* answer = bar;                   // [2], 16-byte aligned
  uint64_t* full = answer + 2;              // [SLOTS]
  uint64_t* empty = full + P::SLOTS;        // [SLOTS]
  uint64_t* q_full = empty + P::SLOTS;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;           // [2]
  uint64_t* p_full = s_full + 2;            // [part][2]: one phase of each per key tile
  uint64_t* o_done = p_full + 4;            // [part][2]
  uint64_t* work_full = o_done + 4;         // [kWorks]
  uint64_t* work_empty = work_full + kWorks;   // [kWorks]
  uint64_t* sums_full = work_empty + kWorks;     // [2]: a query tile's sums and maxima are there
  uint64_t* o_free = sums_full + 2;         // [2]: its output (and they) have been read
  uint64_t* answered = o_free + 2;
  uint64_t* drain = answered + 1;           // [2], and one that is not used: 28 + 2 SLOTS of 8 bytes, so
  Work* works = reinterpret_cast<Work*>(drain + 3);          // [kWorks] begin at a multiple of 16
  float2* sums = reinterpret_cast<float2*>(works + kWorks);       // [2][kM]: (l, its reference in base 2) of the rows
  uint32_t* tmem_p = reinterpret_cast<uint32_t*>(sums + 2 * kM);
  int* misc = reinterpret_cast<int*>(tmem_p + 1);
  volatile int* abort_flag = misc;          // a wait gave up
  int* issued = misc + 1;                   // ring tiles whose loads were issued
  int* q_issued = misc + 2;                 // loads of query tiles
  int* asked = misc + 3;                    // questions for the next piece of work

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gp = 1 << gp_shift, tt = kM >> gp_shift;   // heads and tokens of a query tile

  if (tid == 0) {
    for (int s = 0; s < P::SLOTS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 2);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&p_full[2 * h + t], h ? 4 : 5);   // four warps, and the other tile's MMA warp
        mbar_init(&o_done[2 * h + t], 1);
      }
      mbar_init(&sums_full[t], 4);
      mbar_init(&o_free[t], 4);
      mbar_init(&drain[t], 1);
    }
    for (int i = 0; i < kWorks; ++i) {
      mbar_init(&work_full[i], 1);
      mbar_init(&work_empty[i], kFindWarp);   // all warps but the one that finds the work
    }
    mbar_init(answered, 1);
    *abort_flag = 0;
    *issued = *q_issued = *asked = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_p, kTmemCols);
    tmem_relinquish();
  }
  if (warp == kTmaWarp && lane < 3) prefetch_tmap(lane == 0 ? &tq : lane == 1 ? &tk : &tv);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dependency_wait();
  grid_dependents_launch();
  const uint32_t tmem = *tmem_p;
  if (blockIdx.x == 0)   // bad bounds are flagged once
    for (int i = tid; i < n_seqs; i += kThreads) {
      const int q0 = cu_q[i], q1 = cu_q[i + 1], k0 = cu_k[i], k1 = cu_k[i + 1];
      if (q0 < 0 || q1 < q0 || q1 > total_q || k0 < 0 || k1 < k0 || k1 > total_k) set_status(status, QRE_DEV_BAD_INDEX);
    }
  auto wait_for = [&](uint64_t* b, int n) {   // phase n of b; the same answer in all lanes
    return __all_sync(0xffffffffu, mbar_wait_inline(b, n & 1, abort_flag, status, limit_ns) ? 1 : 0) != 0;
  };
  // The n-th piece of work; false when there is none or a wait gave up.
  auto take = [&](int n, Work& w) {
    if (!wait_for(&work_full[n % kWorks], n / kWorks)) return false;
    w = works[n % kWorks];
    return w.end == 0;
  };
  auto give_back = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&work_empty[n % kWorks]);
  };

  if (warp >= kTmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kFindWarp) {
      // ---- finds the work, and asks for the next
      Finder finder(n_seqs, total_q, total_k, cu_q, cu_k, 8 - gp_shift);
      int b = blockIdx.x;
      for (int n = 0;; ++n) {
        int seq = 0, tile = 0;
        Work w{};
        const bool have = b >= 0 && finder.find(b / groups, seq, tile);
        w.end = !have;
        if (have) {
          w.q0 = cu_q[seq];
          w.q_len = cu_q[seq + 1] - w.q0;
          w.k0 = cu_k[seq];
          w.k_len = cu_k[seq + 1] - w.k0;
          w.tok0 = tile * 2 * tt;
          w.h0 = (b % groups) * gp;
          w.plan(a, tt);
        }
        if (n >= kWorks && !wait_for(&work_empty[n % kWorks], n / kWorks - 1)) break;
        if (lane == 0) {
          works[n % kWorks] = w;
          mbar_arrive(&work_full[n % kWorks]);
        }
        __syncwarp();
        if (!have) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(answered, 16);
          ask_next_cta(answer, answered);
          *asked = n + 1;
        }
        if (!wait_for(answered, n)) break;
        b = next_cta(answer);
        fence_proxy_async_smem();   // read before the next answer is written
        __syncwarp();
      }
    } else if (warp == kTmaWarp) {
      // ---- fetches the tiles
      int i0 = 0, nq = 0;
      bool ok = true;
      Work w;
      for (int n = 0; ok && take(n, w); ++n) {
        give_back(n);
        if (w.je <= w.jb) continue;
        const int hk = w.h0 / (a.n_heads / a.n_kv_heads);
        const int qh = q_heads_move ? w.h0 : 0, kh = k_heads_move ? hk : 0, vh = v_heads_move ? hk : 0;
        ok = nq == 0 || wait_for(q_empty, nq - 1);
        if (ok && lane == 0) {
          mbar_arrive_expect_tx(q_full, 2 * P::TILE);
          for (int t = 0; t < 2; ++t)
            for (int x = 0; x < D / 64; ++x)
              tma_load_3d(sq + t * P::TILE + x * P::HALF, &tq, 64 * x, qh, w.q0 + w.tok0 + t * tt, q_full);
          *q_issued = nq + 1;
        }
        ++nq;
        const int end = i0 + 2 * (w.je - w.jb);
        for (int i = i0; ok && i < end; ++i) {
          const int s = i % P::SLOTS;
          ok = i < P::SLOTS || wait_for(&empty[s], i / P::SLOTS - 1);
          if (ok && lane == 0) {
            const bool is_v = (i - i0) & 1;
            mbar_arrive_expect_tx(&full[s], P::TILE);
            for (int x = 0; x < D / 64; ++x)
              tma_load_3d(skv + s * P::TILE + x * P::HALF, is_v ? &tv : &tk, 64 * x, is_v ? vh : kh,
                          w.k0 + (w.jb + (i - i0) / 2) * kN, &full[s]);
            store_release(issued, i + 1);
          }
        }
        i0 = end;
      }
    } else {
      // ---- MMA: the whole warp, so that the operands stay in uniform registers
      const int t = warp - kMmaWarp;
      const uint32_t lead = elect_lane();
      const uint32_t id_s = DT == QRE_BF16 ? umma_idesc_bf16(kM, kN) : umma_idesc_f16(kM, kN);
      const uint32_t id_o = (DT == QRE_BF16 ? umma_idesc_bf16(kM, D) : umma_idesc_f16(kM, D)) | kUmmaBMnMajor;
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), ts = tm + (t ? kS1 : kS0), td = tm + (t ? kO1 : kO0);
      const uint64_t qd = umma_desc_sw128(smem_addr(sq + t * P::TILE)), kd = umma_desc_sw128(smem_addr(skv));
      const uint64_t vd = umma_desc_sw128_mn(smem_addr(skv), P::HALF);
      auto scores = [&](int slot) {      // S = Q K_j^T
        const uint64_t k0d = kd + (uint32_t)slot * (P::TILE >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k / 4) * P::HALF + (k % 4) * 32) >> 4;
          umma_f16_lead(ts, qd + off, k0d + off, id_s, k ? 1u : 0u, lead);
        }
        umma_commit_lead(&s_full[t], lead);
      };
      auto values = [&](int slot, int part, bool first) {   // O += P V_j, one part of the keys
        const uint64_t v0d = vd + (uint32_t)slot * (P::TILE >> 4);
#pragma unroll
        for (int k = 0; k < kN / 16; ++k)
          if ((k < kPart / 16) == (part == 0))
            umma_f16_tmem_a_lead(td, ts + 8 * k, v0d + k * (2048 >> 4), id_o, first && k == 0 ? 0u : 1u, lead);
        umma_commit_lead(&o_done[2 * part + t], lead);
      };
      auto wait_tile = [&](int i) { return wait_for(&full[i % P::SLOTS], i / P::SLOTS); };
      // The tiles' products are issued in turn, each tile's in one go: left to themselves the two
      // softmaxes fall into step and compete for the same cycles, and the tensor cores wait.  The
      // turn is one more arrival on the barrier of the first weights: a wait of its own would
      // cost some 200 cycles, as every wait here does, next to the tensor cores' reads.  There is
      // one turn: each step hands it to the next one in the order of work, key tile, query tile,
      // so that a barrier never gets it while the phase before is open.
      auto turn_to = [&](int tile) {
        if (lead) mbar_arrive(&p_full[tile]);
        __syncwarp();
      };
      // ring tiles, query tiles, key tiles of this query tile, pieces with keys for this query tile
      int i0 = 0, nq = 0, n = 0, no = 0;
      Work w;
      bool ok = true;
      if (t == 0) turn_to(0);
      for (int nw = 0; ok && take(nw, w); ++nw) {
        give_back(nw);
        const Range r = t ? w.r[1] : w.r[0];
        // a step of key tile j hands the turn to the other query tile if j is in [give_b, give_e) or is
        // the last (of tile 0: if tile 1 has keys), else to this one; a piece begins with tile 0
        const bool two = w.r[1].je > w.r[1].jb;
        const int give_b = t ? 0 : two ? w.r[1].jb : INT_MAX, give_e = t ? w.r[0].je - 1 : INT_MAX;
        const int last = two ? r.je - 1 : INT_MAX;
        if (w.je <= w.jb) continue;
        ok = wait_for(q_full, nq);
        ++nq;
        if (ok && r.je <= r.jb && lead) mbar_arrive(q_empty);
        __syncwarp();
        for (int j = w.jb; ok && j < w.je; ++j) {
          const int i = i0 + 2 * (j - w.jb), sv = (i + 1) % P::SLOTS, sk = (i + 2) % P::SLOTS;
          const bool mine = j >= r.jb && j < r.je, more = mine && j + 1 < r.je;
          const bool pass = (j >= give_b && j < give_e) || j == last;
          if (mine && j == r.jb) {
            ok = wait_tile(i);
            if (!ok) break;
            tc_fence_after();
            scores(i % P::SLOTS);
            umma_commit_lead(&empty[i % P::SLOTS], lead);
            if (!more) umma_commit_lead(q_empty, lead);
          }
          // The waits for what is long there stand before the one for the weights.
          ok = wait_tile(i + 1) && (mine || wait_tile(i));
          if (ok && mine && j == r.jb) {   // the output of the piece before has been read
            ok = no == 0 || wait_for(&o_free[t], no - 1);
            ++no;
          }
          if (ok && mine) ok = wait_for(&p_full[t], n);
          if (!ok) break;
          if (!mine) {                     // the other query tile's keys only
            if (lead) {
              mbar_arrive(&empty[i % P::SLOTS]);
              mbar_arrive(&empty[sv]);
            }
            __syncwarp();
            continue;
          }
          tc_fence_after();
          values(sv, 0, j == r.jb);
          ok = wait_for(&p_full[2 + t], n);
          if (!ok) break;
          tc_fence_after();
          values(sv, 1, false);
          umma_commit_lead(&empty[sv], lead);
          ++n;
          if (more) {
            ok = wait_tile(i + 2);
            if (!ok) break;
            tc_fence_after();
            scores(sk);   // overwrites P: issued behind the product that reads it
          }
          if (pass) turn_to(t ^ 1);
          else turn_to(t);
          if (more) umma_commit_lead(&empty[sk], lead);
          if (more && j + 2 == r.je) umma_commit_lead(q_empty, lead);
        }
        i0 += 2 * (w.je - w.jb);
      }
    }
  } else if (warp >= kStoreWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kStoreRegs));
    // ---- output: o = O / l.  Warps of their own, because what leaves an SM leaves slowly (two tiles in
    // some 8000 cycles, by TMA through shared memory as by stores of each row's own thread): the
    // softmax goes on with the next piece of work meanwhile.
    // Loops and not unrolled: what these warps execute pushes the softmax's code out of the instruction
    // cache (unrolled, 16 prompts of up to 2048 tokens took 119.9 us, not 116.2).
    const int row = 32 * (warp & 3) + lane;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    int cnt0 = 0, cnt1 = 0, no0 = 0, no1 = 0;
    bool ok = true;
    Work w;
    for (int nw = 0; ok && take(nw, w); ++nw) {
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
        const Range r = t ? w.r[1] : w.r[0];
        const int tile0 = w.tok0 + t * tt;
        if (!ok || tile0 >= w.q_len) continue;
        const bool any = r.je > r.jb;
        float2 sum = make_float2(0.0f, 0.0f);
        if (any) {
          (t ? cnt1 : cnt0) += r.je - r.jb;
          ok = wait_for(&sums_full[t], t ? no1 : no0) && wait_for(&o_done[2 + t], (t ? cnt1 : cnt0) - 1);
          if (!ok) continue;
          tc_fence_after();
          sum = sums[t * kM + row];
        }
        const int tok = tile0 + (row >> gp_shift), head = w.h0 + (row & (gp - 1));
        const bool valid = tok < w.q_len;
        int lo, hi;
        visible_range(min(tok, w.q_len - 1) + w.k_len - w.q_len, w.k_len, a.causal, a.window, lo, hi);
        const bool empty_row = hi <= lo;
        const float inv = empty_row ? 0.0f : 1.0f / sum.x;
        if (lse && valid)
          lse[(size_t)(w.q0 + tok) * a.n_heads + head] = empty_row ? -INFINITY : sum.y * kLn2 + logf(sum.x);
        const bool poison = *reinterpret_cast<volatile int*>(&works[nw % kWorks].poison) != 0;
        uint16_t* out = o + (size_t)(w.q0 + tok) * a.o_token + (size_t)head * a.o_head;
        const uint32_t oc = lanes + (t ? kO1 : kO0);
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          uint32_t y[64];
          if (any) {
            tmem_ld_32x32b_x32(oc + 64 * c, *reinterpret_cast<uint32_t(*)[32]>(y));
            tmem_ld_32x32b_x32(oc + 64 * c + 32, *reinterpret_cast<uint32_t(*)[32]>(y + 32));
            tmem_ld_wait();
            if (c == D / 64 - 1) {       // the next piece may overwrite O and the sums
              ++(t ? no1 : no0);
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&o_free[t]);
            }
          }
#pragma unroll
          for (int i = 0; i < 64; ++i) y[i] = empty_row ? 0u : __float_as_uint(__uint_as_float(y[i]) * inv);
          if (poison && !empty_row) {
            const int hk = w.h0 / (a.n_heads / a.n_kv_heads);
            for (int j = w.jb; j < w.je; ++j) {
              if (!w.special(j)) continue;
              const int ka = j * kN > lo ? j * kN : lo, kb = (j + 1) * kN < hi ? (j + 1) * kN : hi;
              for (int key = ka; key < kb; ++key) {
                const uint16_t* vr = v + (size_t)(w.k0 + key) * a.v_token + (size_t)hk * a.v_head + 64 * c;
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                  const float z = bits_to_float<DT>(vr[i]);
                  if (!isfinite(z)) y[i] = __float_as_uint(__uint_as_float(y[i]) + z);
                }
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = pack2<DT>(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1]));
          __syncwarp();
          if (valid) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              if (wide_o) {
                st_global_32(out + 64 * c + 2 * i, y + i);
              } else {
                *reinterpret_cast<uint4*>(out + 64 * c + 2 * i) = make_uint4(y[i], y[i + 1], y[i + 2], y[i + 3]);
                *reinterpret_cast<uint4*>(out + 64 * c + 2 * i + 8) = make_uint4(y[i + 4], y[i + 5], y[i + 6], y[i + 7]);
              }
            }
          }
          __syncwarp();
        }
      }
      give_back(nw);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---- softmax: thread r of the four warps owns row r of its query tile
    const int t = warp >> 2, row = 32 * (warp & 3) + lane;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t sc = lanes + (t ? kS1 : kS0), oc = lanes + (t ? kO1 : kO0);
    const float s2 = a.scale * kLog2e;
    const uint64_t s22 = pair(s2, s2);
    int cnt = 0, no = 0;   // key tiles of this query tile so far, pieces of work with any
    int i0 = 0;            // ring tiles so far
    bool ok = true;
    for (int nw = 0; ok; ++nw) {
      Range r;
      int lo, hi, lo_max, hi_min, k_len, iv;   // iv: ring index of key tile 0's values
      {
        Work w;
        if (!take(nw, w)) break;
        give_back(nw);
        r = t ? w.r[1] : w.r[0];
        iv = i0 + 1 - 2 * w.jb;
        i0 += 2 * (w.je - w.jb);
        if (r.je <= r.jb) continue;
        k_len = w.k_len;
        const int tok = min(w.tok0 + t * tt + (row >> gp_shift), w.q_len - 1);
        visible_range(tok + w.k_len - w.q_len, w.k_len, a.causal, a.window, lo, hi);
        lo_max = t ? w.lo_max[1] : w.lo_max[0];
        hi_min = t ? w.hi_min[1] : w.hi_min[0];
      }
      float m = -INFINITY, l = 0.0f;       // reference maximum (of the raw scores) and sum
      bool started = false;                // a key tile has been through
      bool unset = true;                   // a row of the warp has no reference
      auto weights = [&](const uint32_t (&x)[32], uint32_t* p, uint64_t off2, uint64_t (&sum)[2]) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 z = unpair(fma2(pair(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), s22, off2));
          const float p0 = ex2(z.x), p1 = ex2(z.y);
          sum[i & 1] = add2(sum[i & 1], pair(p0, p1));
          p[i] = pack2<DT>(p0, p1);    // the weights of the product are rounded; the sum is not
        }
      };
      // -inf for the keys of a piece (from key k0) that the row does not see
      auto mask = [&](uint32_t (&x)[32], int k0) {
        const int a0 = min(max(lo - k0, 0), 32), a1 = min(max(hi - k0, 0), 32);
        // bits a0 .. a1 - 1 (64-bit shifts: a bound may be 32)
        const uint32_t seen = (uint32_t)((1ull << a1) - 1) & ~(uint32_t)((1ull << a0) - 1);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (!(seen & (1u << i))) x[i] = 0xff800000u;
      };
      auto offset = [&]() {
        const float off = m == -INFINITY ? 0.0f : kUp<DT> - m * s2;
        return pair(off, off);
      };
      auto add_sum = [&](const uint64_t (&sum)[2]) {
        const float2 u = unpair(add2(sum[0], sum[1]));
        l += u.x + u.y;
      };
      int unseen = -1;   // a tile whose values have yet to be looked over
      // Values that some token does not see: 0 x NaN or 0 x infinity in P V would reach its result.
      // In the key tiles that a mask cuts, rows behind the sequence's end are zeroed, and elements
      // that are not finite are zeroed and noted; the output adds them back for the tokens that see
      // them.  The softmax warps do it: a warp of its own took 8500 cycles a tile next to the tensor
      // cores' reads, and their arrival with the weights is the only one needed.
      auto look_over = [&](int j) {
        const int i = iv + 2 * j;
        const uint32_t expo = DT == QRE_BF16 ? 0x7f80u : 0x7c00u;
        uint4* tile = reinterpret_cast<uint4*>(skv + (i % P::SLOTS) * P::TILE);
        const int rows = k_len - j * kN;
        constexpr int kMine = P::TILE / 16 / kM;   // 16-byte pieces of a thread: row (e % 1024) / 8 of the tile
        bool touched = false;
        if (rows < kN) {
#pragma unroll 1
          for (int e = row; e < P::TILE / 16; e += kM)
            if ((e % (P::HALF / 16)) / 8 >= rows) {
              tile[e] = make_uint4(0, 0, 0, 0);
              touched = true;
            }
        }
        uint32_t top = 0;   // largest magnitudes of the two halves of a word: not finite iff one element is
#pragma unroll
        for (int g = 0; g < kMine; g += 8) {
          uint4 x[8];       // several loads in flight
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = tile[row + (g + i) * kM];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            top = max_abs2<DT>(max_abs2<DT>(top, x[i].x), max_abs2<DT>(x[i].y, max_abs2<DT>(x[i].z, x[i].w)));
        }
        if ((top & expo) == expo || ((top >> 16) & expo) == expo) {
          // The note first: the other query tile may see the element, multiply the zero, and look for the note.
          *reinterpret_cast<volatile int*>(&works[nw % kWorks].poison) = 1;
          __threadfence_block();
          for (int e = row; e < P::TILE / 16; e += kM) {
            uint4 x = tile[e];
            uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int y = 0; y < 4; ++y)
              u[y] &= ((u[y] & expo) == expo ? 0xffff0000u : 0xffffffffu) &
                      (((u[y] >> 16) & expo) == expo ? 0x0000ffffu : 0xffffffffu);
            tile[e] = make_uint4(u[0], u[1], u[2], u[3]);
          }
          touched = true;
        }
        if (touched) fence_proxy_async_smem();
        __syncwarp();
      };
      auto publish = [&](int part) {
        if (part == 0 && unseen >= 0) {
          const int i = iv + 2 * unseen;
          ok = wait_for(&full[i % P::SLOTS], i / P::SLOTS);
          if (!ok) return;
          look_over(unseen);
          unseen = -1;
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * part + t]);
      };
      // The 32-key pieces [b0, b1) of a tile by the book: the maximum first, the reference moved to it
      // (O and l brought along) where it is far behind, then the weights.  P of piece b lies where
      // scores of pieces up to b were, which have been read.
      auto careful = [&](bool masked, int part, int b0, int b1, int key0) {
        uint32_t y[32];
        auto piece = [&](int b) {
          tmem_ld_32x32b_x32(sc + 32 * b, y);
          tmem_ld_wait();
          if (masked) mask(y, key0 + 32 * b);
        };
        float mx = m;
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
          piece(b);
#pragma unroll
          for (int i = 0; i < 32; i += 2) mx = max3(mx, __uint_as_float(y[i]), __uint_as_float(y[i + 1]));
        }
        const bool move = mx > m && (m == -INFINITY || (mx - m) * s2 > kMove<DT>);
        if (__any_sync(0xffffffffu, move)) {
          const float f = !move ? 1.0f : m == -INFINITY ? 0.0f : ex2((m - mx) * s2);
          if (move) m = mx;
          l *= f;
          if (part || started) {         // behind the product of the part before
            ok = wait_for(&o_done[2 * (part ^ 1) + t], cnt + part - 1);
            if (!ok) return;
            tc_fence_after();
#pragma unroll 1
            for (int b = 0; b < D / 32; ++b) {
              tmem_ld_32x32b_x32(oc + 32 * b, y);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
              tmem_st_32x32b_x32(oc + 32 * b, y);
            }
          }
        }
        const uint64_t off2 = offset();
        uint64_t sum[2] = {0, 0};
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
          uint32_t p[16];
          piece(b);
          weights(y, p, off2, sum);
          tmem_st_32x32b_x16(sc + 16 * b, p);
        }
        add_sum(sum);
        publish(part);
      };
      // The weights are taken against the reference of before, with no maximum looked for (the row's
      // first keys set it).  Rounding does not depend on the reference, so it may stay behind; only
      // when the weights' sum is too large for their type the keys go by the book.  False: they have to.
      auto fits = [&](const uint64_t (&sum)[2]) {
        const float2 u = unpair(add2(sum[0], sum[1]));
        const float total = u.x + u.y;
        if (__any_sync(0xffffffffu, total > kMostWeight)) return false;
        l += total;
        return true;
      };
      // Keys that every token of the tile sees, loaded before.
      auto whole = [&](auto& x, int part, int b0, int key0) {
        constexpr int N = sizeof(x) / 4;
        uint32_t p[N / 2];
        const uint64_t off2 = offset();
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int b = 0; b < N / 32; ++b) weights(*reinterpret_cast<uint32_t(*)[32]>(x + 32 * b), p + 16 * b, off2, sum);
        if (!fits(sum)) {
          careful(false, part, b0, b0 + N / 32, key0);
          return;
        }
#pragma unroll
        for (int b = 0; b < N / 32; ++b)
          tmem_st_32x32b_x16(sc + 16 * (b0 + b), *reinterpret_cast<uint32_t(*)[16]>(p + 16 * b));
        publish(part);
      };
      // The same for a tile that a mask cuts, or with rows that have no reference yet.  (Code of its
      // own: with both branches in the loop's usual way a prompt of 8192 tokens took 392 us, not 359.)
      auto edge = [&](auto pieces, bool masked, int part, int b0, int key0) {
        constexpr int NB = decltype(pieces)::value;
        uint32_t x[32 * NB], p[16 * NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) tmem_ld_32x32b_x32(sc + 32 * (b0 + b), *reinterpret_cast<uint32_t(*)[32]>(x + 32 * b));
        tmem_ld_wait();
        if (masked)
#pragma unroll
          for (int b = 0; b < NB; ++b) mask(*reinterpret_cast<uint32_t(*)[32]>(x + 32 * b), key0 + 32 * (b0 + b));
        if (unset) {                         // rows that have seen no key: these set their references
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 32 * NB; i += 4)
#pragma unroll
            for (int e = 0; e < 2; ++e) mx[e] = max3(mx[e], __uint_as_float(x[i + e]), __uint_as_float(x[i + 2 + e]));
          if (m == -INFINITY) m = fmaxf(mx[0], mx[1]);
          unset = __any_sync(0xffffffffu, m == -INFINITY);
        }
        const uint64_t off2 = offset();
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int b = 0; b < NB; ++b) weights(*reinterpret_cast<uint32_t(*)[32]>(x + 32 * b), p + 16 * b, off2, sum);
        if (!fits(sum)) {
          careful(masked, part, b0, b0 + NB, key0);
          return;
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
          tmem_st_32x32b_x16(sc + 16 * (b0 + b), *reinterpret_cast<uint32_t(*)[16]>(p + 16 * b));
        publish(part);
      };
      for (int j = r.jb; j < r.je; ++j, ++cnt) {
        const bool masked = j * kN < lo_max || (j + 1) * kN > hi_min;
        // the values of a cut tile: before the scores are there if they have come, else before the
        // weights are published.  A parity says whether they have come only once their load is issued
        // (then the slot's tile of a lap before has come and gone): this query tile may be laps ahead of
        // the ring, because it passes by pieces that have no keys for it.
        if (masked) {
          const int i = iv + 2 * j;
          if (__all_sync(0xffffffffu, load_acquire(issued) > i && mbar_try_wait(&full[i % P::SLOTS], (i / P::SLOTS) & 1)))
            look_over(j);
          else unseen = j;
        }
        ok = wait_for(&s_full[t], cnt);
        if (!ok) break;
        tc_fence_after();
        if (masked || unset) {
          edge(std::integral_constant<int, kPart / 32>{}, masked, 0, 0, j * kN);
          if (ok) edge(std::integral_constant<int, (kN - kPart) / 32>{}, masked, 1, kPart / 32, j * kN);
          started = true;
        } else {
          uint32_t xa[kPart], xb[kN - kPart];
#pragma unroll
          for (int b = 0; b < kPart / 32; ++b)
            tmem_ld_32x32b_x32(sc + 32 * b, *reinterpret_cast<uint32_t(*)[32]>(xa + 32 * b));
          tmem_ld_wait();
          whole(xa, 0, 0, j * kN);
          if (!ok) break;
#pragma unroll
          for (int b = 0; b < (kN - kPart) / 32; ++b)
            tmem_ld_32x32b_x32(sc + kPart + 32 * b, *reinterpret_cast<uint32_t(*)[32]>(xb + 32 * b));
          tmem_ld_wait();
          whole(xb, 1, kPart / 32, j * kN);
        }
        if (!ok) break;
      }
      if (!ok) break;
      // what the output needs: for the warps that write it, once they have read the last ones
      if (no > 0) ok = wait_for(&o_free[t], no - 1);
      if (!ok) break;
      sums[t * kM + row] = make_float2(l, m * s2 - kUp<DT>);
      ++no;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sums_full[t]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag && tid == 0) {
    // a wait gave up: the loads and tensor-core work already issued complete before the CTA exits
    if (*q_issued > 0) mbar_wait_drain(q_full, (*q_issued - 1) & 1, status);
    const int n = *issued;
    for (int i = n - P::SLOTS > 0 ? n - P::SLOTS : 0; i < n; ++i)
      mbar_wait_drain(&full[i % P::SLOTS], (i / P::SLOTS) & 1, status);
    if (*asked > 0) mbar_wait_drain(answered, (*asked - 1) & 1, status);
  }
  if (*abort_flag && (warp == kMmaWarp || warp == kMmaWarp + 1)) {
    uint64_t* d = drain + (warp - kMmaWarp);
    if (elect_lane()) {   // the lane that issued them: an election of the same lanes has the same outcome
      umma_commit(d);
      mbar_wait_drain(d, 0, status);
    }
    __syncwarp();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// False when the tensor maps cannot be made.
template <int DT, int D>
bool launch_tc(const qre_attn& a, int n_seqs, int total_q, int total_k, const int32_t* cu_q, const int32_t* cu_k,
               const void* q, const void* k, const void* v, void* o, float* lse, int* status, cudaStream_t stream,
               cudaError_t* err) {
  const int g = a.n_heads / a.n_kv_heads;
  // heads that share a KV head go into one tile, as many as a power of two allows
  int gp = g & -g;
  if (gp > kM) gp = kM;
  const int qm = a.q_head > 0 || a.n_heads == 1, km = a.k_head > 0, vm = a.v_head > 0;
  if (!qm) gp = 1;   // all heads read one query row
  CUtensorMap tq, tk, tv;
  auto stride = [](long long s, long long extent) { return extent > 1 ? s : 64ll; };   // of a single row: any
  if (!make_tmap_rows16(&tq, q, total_q, stride(a.q_token, total_q), qm ? a.n_heads : 1, stride(a.q_head, qm ? a.n_heads : 1), D, gp, kM / gp) ||
      !make_tmap_rows16(&tk, k, total_k, stride(a.k_token, total_k), km ? a.n_kv_heads : 1, stride(a.k_head, km ? a.n_kv_heads : 1), D, 1, kN) ||
      !make_tmap_rows16(&tv, v, total_k, stride(a.v_token, total_k), vm ? a.n_kv_heads : 1, stride(a.v_head, vm ? a.n_kv_heads : 1), D, 1, kN))
    return false;
  const int wide_o = reinterpret_cast<uintptr_t>(o) % 32 == 0 && a.o_token % 16 == 0 && a.o_head % 16 == 0;
  const int groups = a.n_heads / gp, pair = 2 * kM / gp;
  int gp_shift = 0;
  while ((1 << gp_shift) < gp) ++gp_shift;
  const long long blocks = ((long long)total_q / pair + (n_seqs < total_q ? n_seqs : total_q)) * groups;
  auto kernel = attn_tc_kernel<DT, D>;
  *err = ensure_smem_limit(reinterpret_cast<const void*>(kernel), Plan<D>::BYTES);
  if (*err != cudaSuccess) return true;
  *err = launch_dependent(kernel, dim3((unsigned)blocks), dim3(kThreads), (size_t)Plan<D>::BYTES, stream, a, n_seqs,
                          total_q, total_k, gp_shift, groups, cu_q, cu_k, tq, tk, tv, wide_o, qm, km, vm,
                          static_cast<const uint16_t*>(v), static_cast<uint16_t*>(o), lse, wait_limit_ns(), status);
  return true;
}

}  // namespace

cudaError_t launch_attn_prefill(const qre_attn& a, int n_seqs, int total_q, int total_k, const int32_t* cu_q,
                                const int32_t* cu_k, const void* q, const void* k, const void* v, void* o, float* lse,
                                int* status, cudaStream_t stream) {
  // A tensor map wants a distance between tokens; without keys there is nothing to multiply.
  const bool maps = total_k > 0 && (total_q == 1 || a.q_token > 0) &&
                    (total_k == 1 || (a.k_token > 0 && a.v_token > 0));
  // A handful of keys is done by rows before tensor memory and barriers are set up, and a tile holds
  // one sequence's rows only.  By rows / by tiles, us: one prompt of 16 tokens 3.5 / 6.6 at 8 heads of
  // 64, 3.9 / 7.3 at 32 of 128; one of 32: 4.1 / 6.9 and 5.6 / 7.8; of 48: 5.6 / 8.1 and 11.6 / 9.3; of
  // 128: 10.7 / 7.9 and 38 / 9.8; 128 of one token: 3.9 / 11.1 and 8.3 / 37.  What counts is the rows'
  // work, by the sequences' mean length.  The host does not know the longest, so two bounds keep an uneven
  // call from rows: on the longest if none is empty (60 of one token and one of 300: 39 / 10.8 at 8 heads of
  // 64), and on the work if it were all one sequence's (512 tokens and 399 empty sequences: 375 / 81 at 32 of
  // 128).  What they cost is less: 128 of four tokens 7.3 / 11.1, 256 of one 13.5 / 68.
  const long long work = (long long)total_q * a.n_heads * a.head_dim * total_k;
  const bool few = total_k <= kFewKeys && n_seqs <= kFewKeys && total_k - n_seqs < kFewLong &&
                   work / (n_seqs > 0 ? n_seqs : 1) <= kFewWork && work <= kFewTotal;
  if (maps && !few) {
    cudaError_t err = cudaSuccess;
    const bool d64 = a.head_dim == 64;
    const bool made =
        a.dtype == QRE_BF16
            ? (d64 ? launch_tc<QRE_BF16, 64>(a, n_seqs, total_q, total_k, cu_q, cu_k, q, k, v, o, lse, status, stream, &err)
                   : launch_tc<QRE_BF16, 128>(a, n_seqs, total_q, total_k, cu_q, cu_k, q, k, v, o, lse, status, stream, &err))
            : (d64 ? launch_tc<QRE_FP16, 64>(a, n_seqs, total_q, total_k, cu_q, cu_k, q, k, v, o, lse, status, stream, &err)
                   : launch_tc<QRE_FP16, 128>(a, n_seqs, total_q, total_k, cu_q, cu_k, q, k, v, o, lse, status, stream, &err));
    if (made) return err;
  }
  const long long units = (long long)total_q * a.n_heads;
  auto go = [&](auto kernel) {
    return launch_dependent(kernel, dim3((unsigned)((units + 7) / 8 + 1)), dim3(256), 0, stream, a, n_seqs, total_q,
                            total_k, cu_q, cu_k, static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k),
                            static_cast<const uint16_t*>(v), static_cast<uint16_t*>(o), lse, status);
  };
  if (a.dtype == QRE_BF16)
    return a.head_dim == 64 ? go(attn_rows_kernel<QRE_BF16, 64>) : go(attn_rows_kernel<QRE_BF16, 128>);
  return a.head_dim == 64 ? go(attn_rows_kernel<QRE_FP16, 64>) : go(attn_rows_kernel<QRE_FP16, 128>);
}

}  // namespace qre
