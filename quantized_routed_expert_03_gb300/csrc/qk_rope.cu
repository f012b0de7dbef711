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
// their way, and each thread asks for its next row before it works on this one.
#include <type_traits>

#include "internal.h"
#include "kv_rows.cuh"

namespace qre {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 16;    // of a CTA at most

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
__global__ void __launch_bounds__(kThreads) qk_rope_kernel(
    const __grid_constant__ qre_rope r, const __grid_constant__ qre_kv_cache c, int layer, int n_tokens, int tokens,
    uint32_t magic, const int32_t* __restrict__ token_seq, const int32_t* __restrict__ token_pos, const uint16_t* q,
    const uint16_t* k, const uint16_t* v, uint16_t* q_out, uint16_t* k_out, int* status) {
  constexpr int LR = D / 16;             // lanes of a row
  constexpr int kRowsAt = kThreads / LR; // rows of a CTA at a time
  constexpr bool kCache = CT != kArrays;
  constexpr bool kQuant = CT == QRE_E4M3 || CT == QRE_E2M1;
  __shared__ __align__(16) float2 turn[kTokens][D / 2];
  __shared__ int pos_of[kTokens];
  __shared__ long long page_of[kCache ? kTokens : 1];
  const int lane = threadIdx.x & 31, j = threadIdx.x % LR;
  const uint32_t mates = ((1u << LR) - 1u) << (lane & ~(LR - 1));
  const int rows_of = r.n_heads + r.n_kv_heads * (kCache ? 2 : 1);   // of a token: q, k, v
  const int t0 = blockIdx.x * tokens, mine = n_tokens - t0 < tokens ? n_tokens - t0 : tokens;
  const int rows = mine * rows_of, half = r.rot_dim / 2, step = r.rot_dim / 16;
  const int ps_shift = kCache ? 31 - __clz(c.page_size) : 0;

  // Pieces of a lane: a rotated pair, or two neighbours behind what is rotated; of a value row two neighbours.
  const bool turns = j < step;
  const int p0 = turns ? j : 2 * step + 2 * (j - step), p1 = turns ? j + step : p0 + 1;

  struct Row {
    int t, h, kind;   // kind 0 q, 1 k, 2 v; -1 none
    uint4 x[2];
  };
  auto ask = [&](int i) {
    Row w;
    w.kind = -1;
    w.t = w.h = 0;
    if (i >= rows) return w;
    w.t = (int)__umulhi((uint32_t)i, magic);
    w.h = i - w.t * rows_of;
    const uint16_t* src;
    const size_t t = (size_t)(t0 + w.t);
    if (w.h < r.n_heads) {
      w.kind = 0;
      src = q + t * r.q_token + (size_t)w.h * r.q_head;
    } else if (!kCache || w.h < r.n_heads + r.n_kv_heads) {
      w.kind = 1;
      w.h -= r.n_heads;
      src = k + t * r.k_token + (size_t)w.h * r.k_head;
    } else {
      w.kind = 2;
      w.h -= r.n_heads + r.n_kv_heads;
      src = v + t * r.v_token + (size_t)w.h * r.v_head;
    }
    const bool is_v = kCache && w.kind == 2;
    w.x[0] = *reinterpret_cast<const uint4*>(src + 8 * (is_v ? 2 * j : p0));
    w.x[1] = *reinterpret_cast<const uint4*>(src + 8 * (is_v ? 2 * j + 1 : p1));
    return w;
  };

  grid_dependency_wait();
  grid_dependents_launch();
  const int i0 = threadIdx.x / LR;
  Row next = ask(i0);
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
    turn[t][f] = turn_by(token_pos[t0 + t], r.inv_freq[f]);
  }
  __syncthreads();

  for (int i = i0; i < rows; i += kRowsAt) {   // (the lanes of a row go together)
    const Row w = next;
    next = ask(i + kRowsAt);
    const int pos = pos_of[w.t];
    if (pos < 0) continue;
    float x[2][8];
    unpack8<DT>(w.x[0], x[0]);
    unpack8<DT>(w.x[1], x[1]);
    if (!kCache || w.kind < 2) {
      const float* weight = w.kind == 0 ? r.q_norm : r.k_norm;
      if (weight) {
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(x[0][e], x[0][e], fmaf(x[1][e], x[1][e], sum));
#pragma unroll
        for (int d = LR / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(mates, sum, d);
        const float inv = 1.0f / sqrtf(sum * (1.0f / D) + r.eps);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const float* wp = weight + 8 * (b ? p1 : p0);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[b][e] *= inv * wp[e];
        }
      }
      if (turns) {
        if (r.interleaved) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float2* cs = &turn[w.t][4 * (b ? p1 : p0)];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 z = cs[e];
              const float a = x[b][2 * e], y = x[b][2 * e + 1];
              x[b][2 * e] = a * z.x - y * z.y;
              x[b][2 * e + 1] = y * z.x + a * z.y;
            }
          }
        } else {
          const float2* cs = &turn[w.t][8 * p0];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 z = cs[e];
            const float a = x[0][e], y = x[1][e];
            x[0][e] = a * z.x - y * z.y;
            x[1][e] = y * z.x + a * z.y;
          }
        }
      }
    }
    const bool is_v = kCache && w.kind == 2;
    const int a0 = is_v ? 2 * j : p0, a1 = is_v ? 2 * j + 1 : p1;
    const uint4 y0 = is_v ? w.x[0] : pack8<DT>(x[0]), y1 = is_v ? w.x[1] : pack8<DT>(x[1]);
    const size_t t = (size_t)(t0 + w.t);
    if (w.kind == 0 || (w.kind == 1 && (!kCache || k_out))) {
      uint16_t* dst = w.kind == 0 ? q_out + t * r.qo_token + (size_t)w.h * r.qo_head : k_out + t * r.ko_token + (size_t)w.h * r.ko_head;
      *reinterpret_cast<uint4*>(dst + 8 * a0) = y0;
      *reinterpret_cast<uint4*>(dst + 8 * a1) = y1;
    }
    if constexpr (kCache) {
      if (w.kind == 0) continue;
      const long long page = page_of[w.t];
      if (page < 0) continue;
      const size_t head = kv_head_bytes(c);
      uint8_t* base = static_cast<uint8_t*>(is_v ? c.v : c.k) + page + (size_t)w.h * head;
      const int row = pos & (c.page_size - 1);
      if constexpr (kQuant) {
        const float inv = kv_inverse(is_v ? c.v_scale : c.k_scale, (size_t)layer * c.n_kv_heads + w.h);
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[b][e] *= inv;
      }
      if constexpr (CT == QRE_E4M3) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
          *reinterpret_cast<uint2*>(base + (size_t)row * D + 8 * (b ? a1 : a0)) =
              make_uint2(to_e4m3x4(x[b][0], x[b][1], x[b][2], x[b][3]), to_e4m3x4(x[b][4], x[b][5], x[b][6], x[b][7]));
      } else if constexpr (CT == QRE_E2M1) {
        // pieces 2 i and 2 i + 1 are a block: the other piece's largest magnitude comes from the lane that has it
        const float m0 = max_magnitude8(x[0]), m1 = max_magnitude8(x[1]);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int other = (b ? a1 : a0) ^ 1;
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
          const int at = b ? a1 : a0;
          *reinterpret_cast<uint32_t*>(base + (size_t)row * (D / 2) + 4 * at) = quantize4(x[b], s);
          if (!(at & 1)) base[(size_t)c.page_size * (D / 2) + (size_t)row * (D / 16) + at / 2] = (uint8_t)s.byte;
        }
      } else {
        uint16_t* dst = reinterpret_cast<uint16_t*>(base) + (size_t)row * D;
        *reinterpret_cast<uint4*>(dst + 8 * a0) = y0;
        *reinterpret_cast<uint4*>(dst + 8 * a1) = y1;
      }
    }
  }
}

}  // namespace

cudaError_t launch_qk_rope(const qre_rope& r, const qre_kv_cache* c, int layer, int n_tokens, const int32_t* token_seq,
                           const int32_t* token_pos, const void* q, const void* k, const void* v, void* q_out, void* k_out,
                           int* status, cudaStream_t stream) {
  const int rows_of = r.n_heads + r.n_kv_heads * (c ? 2 : 1);
  // tokens of a CTA: two rounds of rows if there are enough of them to fill the GPU several times over
  int tokens = 1;
  // floor(i / rows_of) = umulhi(i, magic) for the rows of a CTA (below 2^15)
  const uint32_t magic = (uint32_t)((0x100000000ull + rows_of - 1) / rows_of);
  const dim3 grid((unsigned)((n_tokens + tokens - 1) / tokens));
  const qre_kv_cache none = {};
  auto go = [&](auto kernel) {
    return launch_dependent(kernel, grid, dim3(kThreads), 0, stream, r, c ? *c : none, layer, n_tokens, tokens, magic,
                            token_seq, token_pos, static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k),
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
