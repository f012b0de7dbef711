// attn_prefill.cu -- attention over packed prompts.
//
// o_i = sum_j softmax_j(scale q_i . k_j) v_j over the keys that query i sees, in
// one pass: with the running maximum m and sum l (fp32, base 2),
//   m' = max(m, max s), l' = l 2^(m - m') + sum 2^(s - m'), o' alike.
#include "attn.cuh"
#include "internal.h"
#include "tc.cuh"

namespace qre {
namespace {

// One warp per (query token, head); a lane scores one key at a time, then the
// lanes share the head's dimensions for the values.
template <int DT, int D>
__global__ void __launch_bounds__(256) attn_rows_kernel(const __grid_constant__ qre_attn a, int n_seqs, int total_q,
                                                        int total_k, const int32_t* __restrict__ cu_q,
                                                        const int32_t* __restrict__ cu_k,
                                                        const uint16_t* __restrict__ q, const uint16_t* __restrict__ k,
                                                        const uint16_t* __restrict__ v, uint16_t* __restrict__ o,
                                                        float* __restrict__ lse, int* status) {
  __shared__ float qs[8][D];
  grid_dependency_wait();
  grid_dependents_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * 8 + warp;
  if (unit >= (long long)total_q * a.n_heads) return;
  const int t = (int)(unit / a.n_heads), h = (int)(unit % a.n_heads), hk = h / (a.n_heads / a.n_kv_heads);
  int s = -1;
  for (int i = 0; i < n_seqs; ++i)
    if (cu_q[i] <= t && t < cu_q[i + 1]) {
      s = i;
      break;
    }
  if (s < 0) return;
  const int q0 = cu_q[s], q1 = cu_q[s + 1], k0 = cu_k[s], k1 = cu_k[s + 1];
  if (q0 < 0 || q1 > total_q || k0 < 0 || k1 < k0 || k1 > total_k) {
    if (lane == 0) set_status(status, QRE_DEV_BAD_INDEX);
    return;
  }
  int lo, hi;
  visible_range(k1 - k0 - (q1 - q0) + t - q0, k1 - k0, a.causal, a.window, lo, hi);
  for (int d = lane; d < D; d += 32)
    qs[warp][d] = bits_to_float<DT>(q[(size_t)t * a.q_token + (size_t)h * a.q_head + d]) * a.scale * kLog2e;
  __syncwarp();
  float m = -INFINITY, l = 0.0f, acc[D / 32] = {};
  for (int j0 = lo; j0 < hi; j0 += 32) {
    const int j = j0 + lane;
    float x = -INFINITY;
    if (j < hi) {
      const uint16_t* kr = k + (size_t)(k0 + j) * a.k_token + (size_t)hk * a.k_head;
      x = 0.0f;
      for (int d = 0; d < D; d += 8) {
        const uint4 w = *reinterpret_cast<const uint4*>(kr + d);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x += qs[warp][d + 2 * e] * bits_to_float<DT>(u[e] & 0xffffu) +
               qs[warp][d + 2 * e + 1] * bits_to_float<DT>(u[e] >> 16);
      }
    }
    float mx = x;
    for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    const float m2 = fmaxf(m, mx), f = m == -INFINITY ? 0.0f : exp2f(m - m2);
    const float p = j < hi ? exp2f(x - m2) : 0.0f;
    float sum = p;
    for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    l = l * f + sum;
    m = m2;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] *= f;
    for (int i = 0; i < 32 && j0 + i < hi; ++i) {
      const float pi = __shfl_sync(0xffffffffu, p, i);
      const uint16_t* vr = v + (size_t)(k0 + j0 + i) * a.v_token + (size_t)hk * a.v_head;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) acc[e] += pi * bits_to_float<DT>(vr[lane + 32 * e]);
    }
  }
  const bool empty = hi <= lo;
  const float inv = empty ? 0.0f : 1.0f / l;
#pragma unroll
  for (int e = 0; e < D / 32; ++e)
    o[(size_t)t * a.o_token + (size_t)h * a.o_head + lane + 32 * e] = (uint16_t)pack2<DT>(acc[e] * inv, 0.0f);
  if (lse && lane == 0) lse[(size_t)t * a.n_heads + h] = empty ? -INFINITY : m * kLn2 + logf(l);
}

// ---------------------------------------------------------------- tensor cores

constexpr int kM = 128;            // rows of a query tile: kM / gp tokens x gp heads of one KV head
constexpr int kN = 128;            // keys of a tile
constexpr int kThreads = 384;
// warps 0-3: softmax of tile 0, 4-7: of tile 1
constexpr int kTmaWarp = 8, kMmaWarp = 9, kScanWarp = 10, kScanWarps = 2;
// Registers: 384 x 168 at launch = 256 x 208 + 128 x 88.
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kS0 = 0, kS1 = 128, kO0 = 256, kO1 = 384;   // tensor-memory columns; P overwrites its S
constexpr float kLazy = 8.0f;      // the reference maximum follows when it is 2^8 behind

template <int D>
struct Plan {
  static constexpr int HALF = kN * 128;              // 64 columns of a 128-row tile, 128-byte rows
  static constexpr int TILE = HALF * (D / 64);
  static constexpr int SLOTS = D == 128 ? 4 : 8;     // K and V tiles in flight
  static constexpr int BYTES = 1024 + 2 * TILE + SLOTS * TILE + 512;
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

// One query tile's keys: tiles [jb, je) of the sequence.
struct TileKeys {
  int jb, je;
};

template <int DT, int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc_kernel(const __grid_constant__ qre_attn a, int n_seqs, int total_q, int total_k, int gp, int groups,
                   const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k,
                   const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap tv, int q_heads_move, int k_heads_move, int v_heads_move,
                   const uint16_t* __restrict__ v, uint16_t* __restrict__ o, float* __restrict__ lse,
                   uint64_t limit_ns, int* status) {
  using P = Plan<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* sq = smem;                       // two query tiles
  uint8_t* skv = smem + 2 * P::TILE;        // ring of key and value tiles
  uint64_t* bar = reinterpret_cast<uint64_t*>(skv + P::SLOTS * P::TILE);
  uint64_t* full = bar;                     // [SLOTS]
  uint64_t* empty = full + P::SLOTS;        // [SLOTS]
  uint64_t* q_full = empty + P::SLOTS;
  uint64_t* s_full = q_full + 1;            // [2]
  uint64_t* p_full = s_full + 2;            // [2]
  uint64_t* o_done = p_full + 2;            // [2]
  uint64_t* scanned = o_done + 2;           // [SLOTS]
  uint64_t* drain = scanned + P::SLOTS;
  uint32_t* tmem_p = reinterpret_cast<uint32_t*>(drain + 1);
  int* misc = reinterpret_cast<int*>(tmem_p + 1);
  volatile int* abort_flag = misc;          // a wait gave up
  volatile int* poison = misc + 1;          // a value that is not finite was taken out of a tile
  int* issued = misc + 2;                   // ring tiles whose loads were issued
  int* where = misc + 3;                    // sequence and tile of this CTA

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = blockIdx.x % groups;
  const int tt = kM / gp;                   // tokens of a query tile

  if (tid == 0) {
    for (int s = 0; s < P::SLOTS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&scanned[s], kScanWarps);
    }
    mbar_init(q_full, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 4);
      mbar_init(&o_done[t], 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *poison = 0;
    *issued = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_p, kTmemCols);
    tmem_relinquish();
  }
  grid_dependency_wait();
  grid_dependents_launch();
  // ---- this CTA's sequence: the tile index counts the sequences' pairs of query tiles
  if (warp == 0) {
    int rest = blockIdx.x / groups, s = -1;
    for (int i0 = 0; i0 < n_seqs && s < 0; i0 += 32) {
      const int i = i0 + lane;
      int cnt = 0;
      if (i < n_seqs) {
        const int q0 = cu_q[i], q1 = cu_q[i + 1], k0 = cu_k[i], k1 = cu_k[i + 1];
        if (q0 >= 0 && q1 >= q0 && q1 <= total_q && k0 >= 0 && k1 >= k0 && k1 <= total_k)
          cnt = (q1 - q0 + 2 * tt - 1) / (2 * tt);
      }
      int inc = cnt;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += u;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, rest < inc);
      if (hit) {
        const int w = __ffs(hit) - 1;
        s = i0 + w;
        const int before = __shfl_sync(0xffffffffu, inc - cnt, w), n = __shfl_sync(0xffffffffu, cnt, w);
        rest = n - 1 - (rest - before);   // a sequence's last tiles, the longest, first
      } else {
        rest -= __shfl_sync(0xffffffffu, inc, 31);
      }
    }
    if (lane == 0) {
      where[0] = s;
      where[1] = rest;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_p;
  const int seq = where[0];
  if (blockIdx.x == 0)   // bad bounds are flagged once
    for (int i = tid; i < n_seqs; i += kThreads) {
      const int q0 = cu_q[i], q1 = cu_q[i + 1], k0 = cu_k[i], k1 = cu_k[i + 1];
      if (q0 < 0 || q1 < q0 || q1 > total_q || k0 < 0 || k1 < k0 || k1 > total_k) set_status(status, QRE_DEV_BAD_INDEX);
    }
  if (seq >= 0) {
    const int q0 = cu_q[seq], q_len = cu_q[seq + 1] - q0, k0 = cu_k[seq], k_len = cu_k[seq + 1] - k0;
    const int h0 = group * gp, hk = h0 / (a.n_heads / a.n_kv_heads);
    const int tok0 = where[1] * 2 * tt;     // first token, in the sequence
    const int shift = k_len - q_len;        // position of token i is i + shift
    // key tiles that a query tile's tokens see (both bounds grow with the token)
    auto keys_of = [&](int t) {
      TileKeys r{0, 0};
      const int ta = tok0 + t * tt, tb = ta + tt < q_len ? ta + tt : q_len;
      if (ta < tb) {
        int lo, hi, x;
        visible_range(ta + shift, k_len, a.causal, a.window, lo, x);
        visible_range(tb - 1 + shift, k_len, a.causal, a.window, x, hi);
        if (hi > lo) {
          r.jb = lo / kN;
          r.je = (hi + kN - 1) / kN;
        }
      }
      return r;
    };
    const TileKeys r0 = keys_of(0), r1 = keys_of(1);
    const bool has0 = r0.je > r0.jb, has1 = r1.je > r1.jb;
    const int jb = has0 ? r0.jb : r1.jb, je = has1 ? r1.je : r0.je;
    auto active = [&](int t, int j) { return t == 0 ? j >= r0.jb && j < r0.je : j >= r1.jb && j < r1.je; };
    // tile j is special when some token of the CTA does not see all of it
    const int last_tok = (tok0 + 2 * tt < q_len ? tok0 + 2 * tt : q_len) - 1;
    int lo_last, hi_first;
    {
      int x;
      visible_range(last_tok + shift, k_len, a.causal, a.window, lo_last, x);
      visible_range(tok0 + shift, k_len, a.causal, a.window, x, hi_first);
    }
    auto special = [&](int j) { return j * kN < lo_last || (j + 1) * kN > hi_first; };

    if (warp >= kTmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kTmaWarp) {
      if (lane == 0 && je > jb) {
        const int qh = q_heads_move ? h0 : 0, kh = k_heads_move ? hk : 0, vh = v_heads_move ? hk : 0;
        mbar_arrive_expect_tx(q_full, 2 * P::TILE);
        for (int t = 0; t < 2; ++t)
          for (int x = 0; x < D / 64; ++x)
            tma_load_3d(sq + t * P::TILE + x * P::HALF, &tq, 64 * x, qh, q0 + tok0 + t * tt, q_full);
        const int n = 2 * (je - jb);
        int i = 0;
        for (; i < n; ++i) {
          const int s = i % P::SLOTS;
          if (i >= P::SLOTS && !mbar_wait_inline(&empty[s], ((i / P::SLOTS) - 1) & 1, abort_flag, status, limit_ns)) break;
          mbar_arrive_expect_tx(&full[s], P::TILE);
          for (int x = 0; x < D / 64; ++x)
            tma_load_3d(skv + s * P::TILE + x * P::HALF, (i & 1) ? &tv : &tk, 64 * x, (i & 1) ? vh : kh,
                        k0 + (jb + i / 2) * kN, &full[s]);
        }
        *issued = i;
      }
    } else if (warp == kMmaWarp) {
      if (je > jb) {   // the whole warp, so that the operands stay in uniform registers
        const uint32_t lead = elect_lane();
        const uint32_t id_s = DT == QRE_BF16 ? umma_idesc_bf16(kM, kN) : umma_idesc_f16(kM, kN);
        const uint32_t id_o = (DT == QRE_BF16 ? umma_idesc_bf16(kM, D) : umma_idesc_f16(kM, D)) | kUmmaBMnMajor;
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t qd = umma_desc_sw128(smem_addr(sq)), kd = umma_desc_sw128(smem_addr(skv));
        const uint64_t vd = umma_desc_sw128_mn(smem_addr(skv), P::HALF);
        auto scores = [&](int t, int slot) {      // S_t = Q_t K_j^T
          const uint64_t k0d = kd + (uint32_t)slot * (P::TILE >> 4), q0d = qd + (uint32_t)t * (P::TILE >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k / 4) * P::HALF + (k % 4) * 32) >> 4;
            umma_f16_lead(tm + (t ? kS1 : kS0), q0d + off, k0d + off, id_s, k ? 1u : 0u, lead);
          }
          umma_commit_lead(&s_full[t], lead);
        };
        auto values = [&](int t, int slot, bool first) {   // O_t += P_t V_j
          const uint64_t v0d = vd + (uint32_t)slot * (P::TILE >> 4);
#pragma unroll
          for (int k = 0; k < kN / 16; ++k)
            umma_f16_tmem_a_lead(tm + (t ? kO1 : kO0), tm + (t ? kS1 : kS0) + 8 * k, v0d + k * (2048 >> 4), id_o,
                                 first && k == 0 ? 0u : 1u, lead);
          umma_commit_lead(&o_done[t], lead);
        };
        auto wait_for = [&](uint64_t* b, uint32_t parity) {
          return __all_sync(0xffffffffu, mbar_wait_inline(b, parity, abort_flag, status, limit_ns) ? 1 : 0) != 0;
        };
        auto wait_tile = [&](int i) { return wait_for(&full[i % P::SLOTS], (i / P::SLOTS) & 1); };
        bool ok = wait_for(q_full, 0) && wait_tile(0);
        tc_fence_after();
        if (ok) {
          if (active(0, jb)) scores(0, 0);
          if (active(1, jb)) scores(1, 0);
          umma_commit_lead(&empty[0], lead);
        }
        int pn[2] = {0, 0};
        for (int j = jb; ok && j < je; ++j) {
          const int i = 2 * (j - jb), sv = (i + 1) % P::SLOTS, sk = (i + 2) % P::SLOTS;
          bool have_next = j + 1 >= je;
          if (!wait_tile(i + 1) || !wait_for(&scanned[sv], ((i + 1) / P::SLOTS) & 1)) break;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (ok && active(t, j)) {
              ok = wait_for(&p_full[t], pn[t] & 1);
              tc_fence_after();
              if (ok) values(t, sv, pn[t] == 0);
              ++pn[t];
            }
            // the scores of the next tile overwrite P: issued behind the product that reads it
            if (ok && j + 1 < je && active(t, j + 1)) {
              if (!have_next) {
                ok = wait_tile(i + 2);
                have_next = true;
                tc_fence_after();
              }
              if (ok) scores(t, sk);
            }
          }
          if (!ok) break;
          umma_commit_lead(&empty[sv], lead);
          if (j + 1 < je) {
            if (!have_next && !wait_tile(i + 2)) break;
            umma_commit_lead(&empty[sk], lead);
          }
        }
      }
    } else {
      // ---- values that some token does not see: 0 x NaN or 0 x infinity in P V would reach
      // its result.  In the tiles where that can happen, rows behind the sequence's end are
      // zeroed, and elements that are not finite are zeroed and noted; the epilogue adds them
      // back for the tokens that see them.
      const int w = warp - kScanWarp;
      for (int j = jb; j < je; ++j) {
        const int i = 2 * (j - jb) + 1;
        if (!__all_sync(0xffffffffu, mbar_wait_inline(&full[i % P::SLOTS], (i / P::SLOTS) & 1, abort_flag, status,
                                                       limit_ns) ? 1 : 0))
          break;
        uint4* tile = reinterpret_cast<uint4*>(skv + (i % P::SLOTS) * P::TILE);
        const uint32_t expo = DT == QRE_BF16 ? 0x7f80u : 0x7c00u;
        bool touched = false;
        for (int e = w * 32 + lane; special(j) && e < P::TILE / 16; e += 32 * kScanWarps) {
          const int row = (e % (P::HALF / 16)) / 8;   // key of this 16-byte piece
          if (j * kN + row >= k_len) {
            tile[e] = make_uint4(0, 0, 0, 0);
            touched = true;
            continue;
          }
          uint4 x = tile[e];
          uint32_t u[4] = {x.x, x.y, x.z, x.w};
          bool bad = false;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const bool b0 = (u[y] & expo) == expo, b1 = ((u[y] >> 16) & expo) == expo;
            bad |= b0 | b1;
            u[y] &= (b0 ? 0xffff0000u : 0xffffffffu) & (b1 ? 0x0000ffffu : 0xffffffffu);
          }
          if (bad) {
            tile[e] = make_uint4(u[0], u[1], u[2], u[3]);
            *poison = 1;
            touched = true;
          }
        }
        if (touched) fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&scanned[i % P::SLOTS]);
      }
    }
    } else {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
      // ---- softmax: thread r of the four warps owns row r of its query tile
      const int t = warp >> 2, row = 32 * (warp & 3) + lane;
      const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
      const uint32_t sc = lanes + (t ? kS1 : kS0), oc = lanes + (t ? kO1 : kO0);
      const int tok = tok0 + t * tt + row / gp, head = h0 + row % gp;
      const bool valid = tok < q_len;
      const int tok_c = valid ? tok : q_len - 1;
      int lo, hi;
      visible_range(tok_c + shift, k_len, a.causal, a.window, lo, hi);
      const TileKeys r = t ? r1 : r0;
      // the tile's own tokens: the last one's first key, the first one's last
      int lo_max, hi_min;
      {
        int x;
        const int ta = tok0 + t * tt < q_len ? tok0 + t * tt : q_len - 1;
        const int tb = (tok0 + (t + 1) * tt < q_len ? tok0 + (t + 1) * tt : q_len) - 1;
        visible_range(tb + shift, k_len, a.causal, a.window, lo_max, x);
        visible_range(ta + shift, k_len, a.causal, a.window, x, hi_min);
      }
      const float s2 = a.scale * kLog2e;
      float m = -INFINITY, l = 0.0f;       // reference maximum (of the raw scores) and sum
      bool ok = true;
      for (int j = r.jb; j < r.je; ++j) {
        const int it = j - r.jb;
        ok = __all_sync(0xffffffffu, mbar_wait_inline(&s_full[t], it & 1, abort_flag, status, limit_ns) ? 1 : 0);
        if (!ok) break;
        tc_fence_after();
        uint32_t x[128];
#pragma unroll
        for (int b = 0; b < 4; ++b) tmem_ld_32x32b_x32(sc + 32 * b, *reinterpret_cast<uint32_t(*)[32]>(x + 32 * b));
        tmem_ld_wait();
        if (j * kN < lo_max || (j + 1) * kN > hi_min) {
          const int a0 = lo - j * kN, a1 = hi - j * kN;
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i < a0 || i >= a1) x[i] = 0xff800000u;   // -inf
        }
        float mx8[8];   // independent chains: a single one would be 64 dependent steps
#pragma unroll
        for (int i = 0; i < 8; ++i) mx8[i] = fmaxf(__uint_as_float(x[i]), __uint_as_float(x[i + 8]));
#pragma unroll
        for (int i = 16; i < 128; i += 16)
#pragma unroll
          for (int e = 0; e < 8; ++e) mx8[e] = max3(mx8[e], __uint_as_float(x[i + e]), __uint_as_float(x[i + 8 + e]));
        const float mx = max3(max3(mx8[0], mx8[1], mx8[2]), max3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]));
        // the reference follows the maximum only when it is far behind: weights stay below 2^8
        bool move = false;
        float f = 1.0f;
        if (mx > m && (m == -INFINITY || (mx - m) * s2 > kLazy)) {
          move = true;
          f = m == -INFINITY ? 0.0f : ex2((m - mx) * s2);
          m = mx;
        }
        if (__any_sync(0xffffffffu, move)) {
          l *= f;
          if (it > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait_inline(&o_done[t], (it - 1) & 1, abort_flag, status, limit_ns) ? 1 : 0);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < D / 16; ++b) {
              uint32_t y[16];
              tmem_ld_32x32b_x16(oc + 16 * b, y);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
              tmem_st_32x32b_x16(oc + 16 * b, y);
            }
          }
        }
        const float off = m == -INFINITY ? 0.0f : m * s2;
        const uint64_t s22 = pair(s2, s2), off2 = pair(-off, -off);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          uint32_t p[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 y = unpair(fma2(pair(__uint_as_float(x[32 * b + 2 * i]), __uint_as_float(x[32 * b + 2 * i + 1])),
                                         s22, off2));
            const float p0 = ex2(y.x), p1 = ex2(y.y);
            sum[i & 1] = add2(sum[i & 1], pair(p0, p1));
            p[i] = pack2<DT>(p0, p1);    // the weights of the product are rounded; the sum is not
          }
          tmem_st_32x32b_x16(sc + 16 * b, p);
        }
        const float2 total = unpair(add2(sum[0], sum[1]));
        l += total.x + total.y;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t]);
      }
      // ---- epilogue
      const int n = r.je - r.jb;
      if (ok && n > 0)
        ok = __all_sync(0xffffffffu, mbar_wait_inline(&o_done[t], (n - 1) & 1, abort_flag, status, limit_ns) ? 1 : 0);
      tc_fence_after();
      if (ok) {
        const bool empty_row = hi <= lo;
        const float inv = empty_row ? 0.0f : 1.0f / l;
        uint16_t* out = o + (size_t)(q0 + tok_c) * a.o_token + (size_t)head * a.o_head;
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
          uint32_t y[32];
          __syncwarp();
          if (n > 0) {
            tmem_ld_32x32b_x32(oc + 32 * b, y);
            tmem_ld_wait();
          }
          if (!valid) continue;
          if (empty_row) {
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = 0;
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * inv);
            if (*poison) {
              for (int j = jb; j < je; ++j) {
                if (!special(j)) continue;
                const int ka = j * kN > lo ? j * kN : lo, kb = (j + 1) * kN < hi ? (j + 1) * kN : hi;
                for (int key = ka; key < kb; ++key) {
                  const uint16_t* vr = v + (size_t)(k0 + key) * a.v_token + (size_t)hk * a.v_head + 32 * b;
#pragma unroll
                  for (int i = 0; i < 32; ++i) {
                    const float z = bits_to_float<DT>(vr[i]);
                    if (!isfinite(z)) y[i] = __float_as_uint(__uint_as_float(y[i]) + z);
                  }
                }
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 32; i += 8)
            *reinterpret_cast<uint4*>(out + 32 * b + i) =
                make_uint4(pack2<DT>(__uint_as_float(y[i]), __uint_as_float(y[i + 1])),
                           pack2<DT>(__uint_as_float(y[i + 2]), __uint_as_float(y[i + 3])),
                           pack2<DT>(__uint_as_float(y[i + 4]), __uint_as_float(y[i + 5])),
                           pack2<DT>(__uint_as_float(y[i + 6]), __uint_as_float(y[i + 7])));
        }
        if (lse && valid)
          lse[(size_t)(q0 + tok) * a.n_heads + head] = empty_row ? -INFINITY : m * s2 * kLn2 + logf(l);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag && tid == 0) {
    // a wait gave up: the loads and tensor-core work already issued complete before the CTA exits
    const int n = *issued;
    if (n > 0) mbar_wait_drain(q_full, 0, status);
    for (int i = n - P::SLOTS > 0 ? n - P::SLOTS : 0; i < n; ++i)
      mbar_wait_drain(&full[i % P::SLOTS], (i / P::SLOTS) & 1, status);
  }
  if (*abort_flag && warp == kMmaWarp && lane == 0) {
    umma_commit(drain);
    mbar_wait_drain(drain, 0, status);
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
  const int groups = a.n_heads / gp, pair = 2 * kM / gp;
  const long long blocks = ((long long)total_q / pair + (n_seqs < total_q ? n_seqs : total_q)) * groups;
  auto kernel = attn_tc_kernel<DT, D>;
  *err = ensure_smem_limit(reinterpret_cast<const void*>(kernel), Plan<D>::BYTES);
  if (*err != cudaSuccess) return true;
  *err = launch_dependent(kernel, dim3((unsigned)blocks), dim3(kThreads), (size_t)Plan<D>::BYTES, stream, a, n_seqs,
                          total_q, total_k, gp, groups, cu_q, cu_k, tq, tk, tv, qm, km, vm,
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
  if (maps) {
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
    return launch_dependent(kernel, dim3((unsigned)((units + 7) / 8)), dim3(256), 0, stream, a, n_seqs, total_q,
                            total_k, cu_q, cu_k, static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k),
                            static_cast<const uint16_t*>(v), static_cast<uint16_t*>(o), lse, status);
  };
  if (a.dtype == QRE_BF16)
    return a.head_dim == 64 ? go(attn_rows_kernel<QRE_BF16, 64>) : go(attn_rows_kernel<QRE_BF16, 128>);
  return a.head_dim == 64 ? go(attn_rows_kernel<QRE_FP16, 64>) : go(attn_rows_kernel<QRE_FP16, 128>);
}

}  // namespace qre
