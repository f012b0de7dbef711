// qk_rope.cu -- norms of query and key heads and the rotation by position, on
// arrays or on the way into the paged cache.
//
// Row x of a head: y = x w / sqrt(mean(x^2) + eps), then for pair i of its first
// rot_dim elements, at the angle pos * inv_freq[i]:
//   a' = a cos - b sin, b' = b cos + a sin.
//
// Bound: every row is read once and written once, some 8 flops an element, so the
// memory bounds it.
//
// A row belongs to D / 16 lanes with 16 elements each, two 16-byte pieces that are
// each other's partners in the rotation (pieces j and j + rot_dim / 16), so that the
// rotation needs no exchange between lanes; the norm's sum takes three or two
// shuffles.  A CTA has a few neighbouring tokens; their cosines and sines, the same
// for all heads, are worked out once into shared memory while the first rows are on
// their way, and each thread asks for its next row before it works on this one.  The
// queries' rows come first, then the keys', then the values', so that a lane keeps its
// weights of the norm in registers; they and its angles lie in shared memory as it reads
// them, neighbouring lanes side by side.
//
// What it measured: 11,278 tokens of 32 and 8 heads of 128 on their way into the pages, 300 MB: 55 us, 5.4 TB/s (a
// copy: 6.8).  One token a CTA and its weights from memory for each row 92; with the queries, keys and values as
// loops of their own 67 (and small calls 2 us longer); one element an instruction 56; three CTAs an SM 62, five (51
// registers) 71.  64 tokens 5.5 us, 700 of 28 heads of 64 5.0: a launch and a chain of loads.  CTAs that share a
// token's rows gain nothing there and cost 7 us on the large call.  Into E4M3 pages the large call takes 63 us, into 4 bits
// 70 (three CTAs an SM, 80 registers, 4 to 8 bytes of spills: the scales and codes); 64 tokens 5.2 either way.
#include <type_traits>

#include "internal.h"
#include "kv_rows.cuh"

namespace qre {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 4;     // of a CTA at most

// Cosine and sine of pos * f, f radians per position.  The angle in whole turns is taken modulo 1 in
// 64 bits: at position 2^31 it is still good to 2^-22 of a turn for f = 1 (in fp32 nothing would be left).
__device__ __forceinline__ float2 turn_by(int pos, float f) {
  const double turns = (double)pos * ((double)f * 0.15915494309189533577);   // 1 / (2 pi)
  float s, c;
  sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
  return make_float2(c, s);
}

enum To { kArrays = -1 };   // else the qre_dtype of the cache

template <int DT, int D, int CT>
__global__ void __launch_bounds__(kThreads, CT == QRE_E2M1 || CT == QRE_E4M3 ? 3 : 4) qk_rope_kernel(
    const __grid_constant__ qre_rope r, const __grid_constant__ qre_kv_cache c, int layer, int n_tokens, int tokens,
    uint32_t q_magic, uint32_t k_magic, const int32_t* __restrict__ token_seq, const int32_t* __restrict__ token_pos,
    const uint16_t* q, const uint16_t* k, const uint16_t* v, uint16_t* q_out, uint16_t* k_out, int* status) {
  constexpr int LR = D / 16;             // lanes of a row
  constexpr int kRowsAt = kThreads / LR; // rows of a CTA at a time
  constexpr bool kCache = CT != kArrays;
  constexpr bool kQuant = CT == QRE_E4M3 || CT == QRE_E2M1;
  __shared__ __align__(16) float turn[kTokens][D];   // a lane's angles two by two, lane beside lane
  __shared__ __align__(16) float weights[2][D];
  __shared__ int pos_of[kTokens];
  __shared__ long long page_of[kCache ? kTokens : 1];
  const int lane = threadIdx.x & 31, j = threadIdx.x % LR;
  const uint32_t mates = ((1u << LR) - 1u) << (lane & ~(LR - 1));
  const int t0 = blockIdx.x * tokens, mine = n_tokens - t0 < tokens ? n_tokens - t0 : tokens;
  const int half = r.rot_dim / 2, step = r.rot_dim / 16;
  const int ps_shift = kCache ? 31 - __clz(c.page_size) : 0;
  const bool turns = j < step;
  const int i0 = threadIdx.x / LR;

  // The CTA's rows: all queries', then all keys', then all values'.
  const int q_rows = mine * r.n_heads, k_rows = mine * r.n_kv_heads, rows = q_rows + k_rows * (kCache ? 2 : 1);
  struct Row {
    int kind, t, h;   // kind 0 q, 1 k, 2 v
    uint4 x[2];
  };
  // Pieces of a lane: a rotated pair, or two neighbours behind what is rotated; of a value row two neighbours.
  const int own0 = turns ? j : 2 * step + 2 * (j - step), own1 = turns ? j + step : own0 + 1;
  auto ask = [&](int i, Row& w) {
    if (i >= rows) return;
    w.kind = i < q_rows ? 0 : !kCache || i < q_rows + k_rows ? 1 : 2;
    const int n = w.kind == 0 ? i : w.kind == 1 ? i - q_rows : i - q_rows - k_rows;
    const int heads = w.kind == 0 ? r.n_heads : r.n_kv_heads;
    w.t = heads == 1 ? n : (int)__umulhi((uint32_t)n, w.kind == 0 ? q_magic : k_magic);
    w.h = n - w.t * heads;
    const size_t t = (size_t)(t0 + w.t);
    const uint16_t* row = w.kind == 0   ? q + t * r.q_token + (size_t)w.h * r.q_head
                          : w.kind == 1 ? k + t * r.k_token + (size_t)w.h * r.k_head
                                        : v + t * r.v_token + (size_t)w.h * r.v_head;
    const bool is_v = kCache && w.kind == 2;
    w.x[0] = *reinterpret_cast<const uint4*>(row + 8 * (is_v ? 2 * j : own0));
    w.x[1] = *reinterpret_cast<const uint4*>(row + 8 * (is_v ? 2 * j + 1 : own1));
  };
  grid_dependency_wait();
  grid_dependents_launch();
  Row next;
  ask(i0, next);
  if ((int)threadIdx.x < mine) {
    const int pos = token_pos[t0 + threadIdx.x];
    pos_of[threadIdx.x] = pos;
    if constexpr (kCache) {
      long long at = -1;
      if (pos >= 0) {
        at = kv_page_at(c, layer, token_seq[t0 + threadIdx.x], pos, ps_shift);
        if (at < 0) set_status(status, QRE_DEV_BAD_INDEX);
      }
      page_of[threadIdx.x] = at;
    }
  }
  for (int i = threadIdx.x; i < mine * half; i += kThreads) {
    const int t = i / half, f = i - t * half;
    // angle f is number e of its lane: of the pairs 8 j + e, or of the pieces j and j + step with four each
    int of, e;
    if (r.interleaved) {
      const int piece = f >> 2, second = piece >= step;
      of = piece - second * step;
      e = 4 * second + (f & 3);
    } else {
      of = f >> 3;
      e = f & 7;
    }
    const float2 z = turn_by(token_pos[t0 + t], r.inv_freq[f]);
    float* to = turn[t] + 4 * ((e >> 1) * step + of) + (e & 1);   // two cosines, two sines
    to[0] = z.x;
    to[2] = z.y;
  }
  // the norms' weights, a lane's 16 in a row: 1 without a norm
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    const int kind = i / D, at = i % D, piece = at >> 3;
    const float* norm = kind ? r.k_norm : r.q_norm;
    const int of = piece < step ? piece : piece < 2 * step ? piece - step : step + ((piece - 2 * step) >> 1);
    const int second = piece < step ? 0 : piece < 2 * step ? 1 : (piece - 2 * step) & 1;
    weights[kind][((second * 2 + ((at >> 2) & 1)) * LR + of) * 4 + (at & 3)] = norm ? norm[at] : 1.0f;
  }
  __syncthreads();

  int have = -1;                     // whose weights the registers hold
  uint64_t weight[2][4];
  for (int i = i0; i < rows; i += kRowsAt) {   // (the lanes of a row go together)
    const int kind = next.kind, t = next.t, h = next.h;
    const uint4 w0 = next.x[0], w1 = next.x[1];
    ask(i + kRowsAt, next);
    const bool is_v = kCache && kind == 2;
    const int p0 = is_v ? 2 * j : own0, p1 = is_v ? 2 * j + 1 : own1;
    const bool norm = kind == 0 ? r.q_norm != nullptr : !is_v && r.k_norm != nullptr;
    if (norm && kind != have) {
      have = kind;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 z = *reinterpret_cast<const float4*>(&weights[kind][(e * LR + j) * 4]);
        weight[e >> 1][2 * (e & 1)] = pair(z.x, z.y);
        weight[e >> 1][2 * (e & 1) + 1] = pair(z.z, z.w);
      }
    }
    const int pos = pos_of[t];
    if (pos < 0) continue;
    float x[2][8];
    uint4 y0 = w0, y1 = w1;
    if (!is_v || kQuant) {
      unpack8<DT>(w0, x[0]);
      unpack8<DT>(w1, x[1]);
    }
    if (!is_v) {
      // (two elements an instruction, neighbours: the issue slots are what this kernel runs out of next to the memory)
      uint64_t u[2][4];
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) u[b][e] = pair(x[b][2 * e], x[b][2 * e + 1]);
      if (norm) {
        uint64_t sums[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sums[0] = fma2(u[0][e], u[0][e], sums[0]);
          sums[1] = fma2(u[1][e], u[1][e], sums[1]);
        }
        const float2 two = unpair(add2(sums[0], sums[1]));
        float sum = two.x + two.y;
#pragma unroll
        for (int d = LR / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(mates, sum, d);
        const float inv = 1.0f / sqrtf(sum * (1.0f / D) + r.eps);
        const uint64_t inv2 = pair(inv, inv);
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) u[b][e] = mul2(u[b][e], mul2(inv2, weight[b][e]));
      }
      if (turns) {
        const float4* cs = reinterpret_cast<const float4*>(turn[t]) + j;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 z = cs[e * step];   // angles 2 e and 2 e + 1
          if (r.interleaved) {
            uint64_t(&w)[4] = u[e >> 1];
            const int at = 2 * (e & 1);
            const float2 a = unpair(w[at]), b = unpair(w[at + 1]);
            w[at] = fma2(pair(a.y, a.x), pair(-z.z, z.z), mul2(w[at], pair(z.x, z.x)));
            w[at + 1] = fma2(pair(b.y, b.x), pair(-z.w, z.w), mul2(w[at + 1], pair(z.y, z.y)));
          } else {
            const uint64_t a = u[0][e], b = u[1][e], c2 = pair(z.x, z.y);
            u[0][e] = fma2(b, pair(-z.z, -z.w), mul2(a, c2));
            u[1][e] = fma2(a, pair(z.z, z.w), mul2(b, c2));
          }
        }
      }
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 z = unpair(u[b][e]);
          x[b][2 * e] = z.x;
          x[b][2 * e + 1] = z.y;
        }
      y0 = pack8<DT>(x[0]);
      y1 = pack8<DT>(x[1]);
      uint16_t* dst = kind == 0 ? q_out + (size_t)(t0 + t) * r.qo_token + (size_t)h * r.qo_head
                      : k_out   ? k_out + (size_t)(t0 + t) * r.ko_token + (size_t)h * r.ko_head
                                : nullptr;
      if (dst) {
        *reinterpret_cast<uint4*>(dst + 8 * p0) = y0;
        *reinterpret_cast<uint4*>(dst + 8 * p1) = y1;
      }
    }
    if constexpr (kCache) {
      if (kind == 0) continue;
      const long long page = page_of[t];
      if (page < 0) continue;
      const size_t head = kv_head_bytes(c);
      uint8_t* base = static_cast<uint8_t*>(is_v ? c.v : c.k) + page + (size_t)h * head;
      const int row = pos & (c.page_size - 1);
      if constexpr (kQuant) {
        const float inv = kv_inverse(is_v ? c.v_scale : c.k_scale, (size_t)layer * c.n_kv_heads + h);
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[b][e] *= inv;
      }
      if constexpr (CT == QRE_E4M3) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
          *reinterpret_cast<uint2*>(base + (size_t)row * D + 8 * (b ? p1 : p0)) =
              make_uint2(to_e4m3x4(x[b][0], x[b][1], x[b][2], x[b][3]), to_e4m3x4(x[b][4], x[b][5], x[b][6], x[b][7]));
      } else if constexpr (CT == QRE_E2M1) {
        // pieces 2 i and 2 i + 1 are a block: the other piece's largest magnitude comes from the lane that has it
        const float m0 = max_magnitude8(x[0]), m1 = max_magnitude8(x[1]);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int at = b ? p1 : p0, other = at ^ 1;
          int from, second;
          if (is_v) {
            from = other >> 1;
            second = other & 1;
          } else if (other < 2 * step) {
            second = other >= step;
            from = second ? other - step : other;
          } else {
            second = other & 1;
            from = step + ((other - 2 * step) >> 1);
          }
          const float o0 = __shfl_sync(mates, m0, from, LR), o1 = __shfl_sync(mates, m1, from, LR);
          const Scale4 s(max_magnitude(b ? m1 : m0, second ? o1 : o0));
          *reinterpret_cast<uint32_t*>(base + (size_t)row * (D / 2) + 4 * at) = quantize4(x[b], s);
          if (!(at & 1)) base[(size_t)c.page_size * (D / 2) + (size_t)row * (D / 16) + at / 2] = (uint8_t)s.byte;
        }
      } else {
        uint16_t* dst = reinterpret_cast<uint16_t*>(base) + (size_t)row * D;
        *reinterpret_cast<uint4*>(dst + 8 * p0) = y0;
        *reinterpret_cast<uint4*>(dst + 8 * p1) = y1;
      }
    }
  }
}

}  // namespace

cudaError_t launch_qk_rope(const qre_rope& r, const qre_kv_cache* c, int layer, int n_tokens, const int32_t* token_seq,
                           const int32_t* token_pos, const void* q, const void* k, const void* v, void* q_out, void* k_out,
                           int* status, cudaStream_t stream) {
  // Tokens of a CTA: as many as leave every SM a few CTAs (a CTA's first rows wait for its angles).
  const int sms = device_sm_count();
  int tokens = sms > 0 ? n_tokens / (8 * sms) : 1;
  tokens = tokens > kTokens ? kTokens : tokens < 1 ? 1 : tokens;
  // floor(i / heads) = umulhi(i, magic) for the rows of a CTA (below 2^13)
  auto magic = [](int heads) { return (uint32_t)((0x100000000ull + heads - 1) / heads); };
  const dim3 grid((unsigned)((n_tokens + tokens - 1) / tokens));
  const qre_kv_cache none = {};
  auto go = [&](auto kernel) {
    return launch_dependent(kernel, grid, dim3(kThreads), 0, stream, r, c ? *c : none, layer, n_tokens, tokens,
                            magic(r.n_heads), magic(r.n_kv_heads), token_seq, token_pos, static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k),
                            static_cast<const uint16_t*>(v), static_cast<uint16_t*>(q_out), static_cast<uint16_t*>(k_out),
                            status);
  };
  auto pick = [&](auto dt, auto d) {
    constexpr int DT = decltype(dt)::value, D = decltype(d)::value;
    if (!c) return go(qk_rope_kernel<DT, D, kArrays>);
    if (c->dtype == QRE_E4M3) return go(qk_rope_kernel<DT, D, QRE_E4M3>);
    if (c->dtype == QRE_E2M1) return go(qk_rope_kernel<DT, D, QRE_E2M1>);
    return go(qk_rope_kernel<DT, D, QRE_BF16>);   // the rows' own type, either
  };
  using B = std::integral_constant<int, QRE_BF16>;
  using H = std::integral_constant<int, QRE_FP16>;
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  if (r.dtype == QRE_BF16) return r.head_dim == 64 ? pick(B{}, D64{}) : pick(B{}, D128{});
  return r.head_dim == 64 ? pick(H{}, D64{}) : pick(H{}, D128{});
}

}  // namespace qre
