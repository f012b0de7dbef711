// kv_rows.cu -- rows rounded to 4 bits on their way into the paged cache, and
// rows of any cache read back out of its pages.
//
// A QRE_E2M1 row x: every 16 neighbours get s = E4M3(max |x| / 6) and codes
// E2M1(x / s); read back, an element is code * s * (scale of layer and head).
//
// Bound: each row is read once and written once; the memory.  A thread has 16
// elements, one block: its scale needs no exchange between lanes.  As in the 8- and
// 16-bit write, a CTA has neighbouring tokens, whose pages it looks up once while the
// first rows are on their way.
//
// What it measured (8 KV heads of 128, 4 bits): 131,072 rows read back 120 us, 5.2 TB/s of which three quarters are
// written.  With several blocks of a thread on their way, and so fewer threads on an SM, it is slower (2: 2 us, 4: 38).
// 2227 rows of 4 heads of 64 written 4.3 us, read (17,997) 8.4; with as few rows as leave a CTA a quarter full 6.8.  A
// search of the bounds in shared memory gains nothing.
#include <type_traits>

#include "internal.h"
#include "kv_rows.cuh"

namespace qre {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 64;    // of a CTA at most; whole warps

template <int RT>
__global__ void __launch_bounds__(kThreads) kv_write4_kernel(
    const __grid_constant__ qre_kv_cache c, int layer, const __grid_constant__ qre_kv_rows r, int n_tokens, int tokens,
    uint32_t magic, const int32_t* __restrict__ token_seq, const int32_t* __restrict__ token_pos,
    const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, int* status) {
  __shared__ long long page_of[kTokens];   // -1: skipped
  __shared__ int pos_of[kTokens];
  __shared__ float by[2][kKvMaxHeads];     // 1 / scale of K and of V
  grid_dependency_wait();
  grid_dependents_launch();
  const int per_head_shift = c.head_dim == 64 ? 2 : 3, per_row = c.n_kv_heads << per_head_shift, per_token = 2 * per_row;
  const int t0 = blockIdx.x * tokens, mine = n_tokens - t0 < tokens ? n_tokens - t0 : tokens;
  const int blocks = mine * per_token, ps_shift = 31 - __clz(c.page_size);
  const size_t head = kv_head_bytes(c);
  for (int i0 = 0; i0 < blocks; i0 += kThreads) {
    const int i = i0 + (int)threadIdx.x;
    uint4 w[2];
    int t = 0, h = 0, b = 0;
    bool is_v = false;
    if (i < blocks) {
      t = (int)__umulhi((uint32_t)i, magic);
      const int rest = i - t * per_token;
      is_v = rest >= per_row;
      const int x = is_v ? rest - per_row : rest;
      h = x >> per_head_shift;
      b = x & ((1 << per_head_shift) - 1);
      const uint16_t* src = is_v ? v + (size_t)(t0 + t) * r.v_token + (size_t)h * r.v_head
                                 : k + (size_t)(t0 + t) * r.k_token + (size_t)h * r.k_head;
      w[0] = *reinterpret_cast<const uint4*>(src + kBlock4 * b);
      w[1] = *reinterpret_cast<const uint4*>(src + kBlock4 * b + 8);
    }
    if (i0 == 0) {
      for (int e = threadIdx.x; e < 2 * c.n_kv_heads; e += kThreads) {
        const int of_v = e >= c.n_kv_heads, hh = of_v ? e - c.n_kv_heads : e;
        by[of_v][hh] = kv_inverse(of_v ? c.v_scale : c.k_scale, (size_t)layer * c.n_kv_heads + hh);
      }
      if ((int)threadIdx.x < mine) {
        const int pos = token_pos[t0 + threadIdx.x];
        long long at = -1;
        if (pos >= 0) {
          at = kv_page_at(c, layer, token_seq[t0 + threadIdx.x], pos, ps_shift);
          if (at < 0) set_status(status, QRE_DEV_BAD_INDEX);
        }
        page_of[threadIdx.x] = at;
        pos_of[threadIdx.x] = pos;
      }
      __syncthreads();
    }
    if (i >= blocks || page_of[t] < 0) continue;
    float x[2][8];
    unpack8<RT>(w[0], x[0]);
    unpack8<RT>(w[1], x[1]);
    const float inv = by[is_v][h];
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int m = 0; m < 8; ++m) x[e][m] *= inv;
    const Scale4 s(max_magnitude(max_magnitude8(x[0]), max_magnitude8(x[1])));
    uint8_t* base = static_cast<uint8_t*>(is_v ? c.v : c.k) + page_of[t] + (size_t)h * head;
    const int row = pos_of[t] & (c.page_size - 1);
    *reinterpret_cast<uint2*>(base + (size_t)row * (c.head_dim / 2) + 8 * b) = make_uint2(quantize4(x[0], s), quantize4(x[1], s));
    base[(size_t)c.page_size * (c.head_dim / 2) + (size_t)row * (c.head_dim / kBlock4) + b] = (uint8_t)s.byte;
  }
}

// What 16 elements at element `at` of a head of a page are worth, as 16-bit pairs.
template <int RT, int CT>
__device__ __forceinline__ void load16(const uint8_t* base, int row, int b, int D, int page_size, float scale, uint32_t (&y)[8]) {
  if constexpr (CT == QRE_BF16) {   // 16 bits, the rows' own type
    const uint4* p = reinterpret_cast<const uint4*>(base + ((size_t)row * D + kBlock4 * b) * 2);
    const uint4 u = p[0], v = p[1];
    y[0] = u.x, y[1] = u.y, y[2] = u.z, y[3] = u.w, y[4] = v.x, y[5] = v.y, y[6] = v.z, y[7] = v.w;
  } else if constexpr (CT == QRE_E4M3) {
    const uint4 u = *reinterpret_cast<const uint4*>(base + (size_t)row * D + kBlock4 * b);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __half2 h(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i & 1))), __NV_E4M3));
      y[i] = pack2<RT>(__low2float(h) * scale, __high2float(h) * scale);
    }
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(base + (size_t)row * (D / 2) + 8 * b);
    const uint8_t byte = base[(size_t)page_size * (D / 2) + (size_t)row * (D / kBlock4) + b];
    const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
    e2m1x8_to_half2(u.x, *reinterpret_cast<uint32_t(*)[4]>(y));
    e2m1x8_to_half2(u.y, *reinterpret_cast<uint32_t(*)[4]>(y + 4));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __half2 h = u32_as_h2(y[i]);
      // code * s is exact in fp32 (2 + 4 bits), then one product with the head's scale, then one rounding
      y[i] = pack2<RT>(__low2float(h) * s * scale, __high2float(h) * s * scale);
    }
  }
}

// The rows of the result, 16 elements a thread; a CTA has `tokens` neighbouring rows of K and of V.
template <int RT, int CT>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(
    const __grid_constant__ qre_kv_cache c, int layer, const __grid_constant__ qre_kv_rows r, int n, int total, int tokens,
    uint32_t magic, int wide, const int32_t* __restrict__ seqs, const int32_t* __restrict__ first, const int32_t* __restrict__ cu,
    uint16_t* __restrict__ k, uint16_t* __restrict__ v, int* status) {
  __shared__ long long page_of[kTokens];   // -1: zeros, -2: nobody's row
  __shared__ int pos_of[kTokens];
  grid_dependency_wait();
  grid_dependents_launch();
  const int t0 = blockIdx.x * tokens, mine = total - t0 < tokens ? total - t0 : tokens;
  const int ps_shift = 31 - __clz(c.page_size), D = c.head_dim;
  if (blockIdx.x == 0)   // bad bounds are flagged once
    for (int i = threadIdx.x; i < n; i += kThreads)
      if (cu[i] < 0 || cu[i + 1] < cu[i] || cu[i + 1] > total) set_status(status, QRE_DEV_BAD_INDEX);
  const int t = t0 + (int)threadIdx.x;
  auto has = [&](int i) {         // sequence i row t (its bounds are asked for together)
    const int a = cu[i], b = cu[i + 1];
    return (a >= 0) & (a <= t) & (t < b) & (b <= total);
  };
  auto look_up = [&](int i) {
    const int s = seqs ? seqs[i] : i, from = first ? first[i] : 0;
    const long long p = (long long)from + (t - cu[i]);
    long long at = -1;
    int pos = 0;
    if (s >= 0 && s < c.max_seqs && from >= 0 && p < c.seq_len[s]) {
      pos = (int)p;
      at = kv_page_at(c, layer, s, pos, ps_shift);
    }
    if (at < 0) set_status(status, QRE_DEV_BAD_INDEX);
    page_of[threadIdx.x] = at;
    pos_of[threadIdx.x] = pos;
  };
  if (threadIdx.x < kTokens) {      // whole warps
    const bool row = (int)threadIdx.x < mine;
    bool lost = row;
    if (row) {
      int lo = 0, hi = n - 1;        // the last sequence that begins at or before the row
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (cu[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      if (has(lo)) {
        look_up(lo);
        lost = false;
      }
    }
    if (__any_sync(0xffffffffu, lost)) {   // nobody's row, or bounds that do not ascend have led the search astray
      int bad = 0;
#pragma unroll 8
      for (int i = threadIdx.x & 31; i < n; i += 32) bad |= (cu[i] < 0) | (cu[i + 1] < cu[i]) | (cu[i + 1] > total);
      if (__any_sync(0xffffffffu, bad))
        for (int i = 0; lost && i < n; ++i)
          if (has(i)) {
            look_up(i);
            lost = false;
          }
      if (lost) page_of[threadIdx.x] = -2;
    }
  }
  __syncthreads();
  const int per_head_shift = D == 64 ? 2 : 3, per_row = c.n_kv_heads << per_head_shift, per_token = 2 * per_row;
  const int blocks = mine * per_token;
  const size_t head = kv_head_bytes(c);
  for (int i = threadIdx.x; i < blocks; i += kThreads) {
    const int t = (int)__umulhi((uint32_t)i, magic), rest = i - t * per_token;
    const bool is_v = rest >= per_row;
    const int x = is_v ? rest - per_row : rest, h = x >> per_head_shift, b = x & ((1 << per_head_shift) - 1);
    const long long page = page_of[t];
    if (page == -2) continue;
    uint32_t y[8] = {};
    if (page >= 0) {
      const uint8_t* base = static_cast<const uint8_t*>(is_v ? c.v : c.k) + page + (size_t)h * head;
      const float* scales = is_v ? c.v_scale : c.k_scale;
      load16<RT, CT>(base, pos_of[t] & (c.page_size - 1), b, D, c.page_size,
                     CT != QRE_BF16 && scales ? scales[(size_t)layer * c.n_kv_heads + h] : 1.0f, y);
    }
    uint16_t* dst = (is_v ? v + (size_t)(t0 + t) * r.v_token + (size_t)h * r.v_head
                          : k + (size_t)(t0 + t) * r.k_token + (size_t)h * r.k_head) + kBlock4 * b;
    if (wide) {
      st_global_32(dst, y);
    } else {
      *reinterpret_cast<uint4*>(dst) = make_uint4(y[0], y[1], y[2], y[3]);
      *reinterpret_cast<uint4*>(dst + 8) = make_uint4(y[4], y[5], y[6], y[7]);
    }
  }
}

// Tokens of a CTA and the reciprocal of a token's blocks (see kv_write_kernel).
struct Cut {
  int tokens;
  uint32_t magic;
  dim3 grid;
  Cut(const qre_kv_cache& c, int n_tokens, int ctas_per_sm) {
    const int per_token = 2 * c.n_kv_heads * (c.head_dim / kBlock4);   // at most 4096
    const int ctas = device_sm_count() * ctas_per_sm;
    tokens = ctas > 0 ? (n_tokens + ctas - 1) / ctas : 1;
    const int fill = (kThreads + per_token - 1) / per_token;           // a block for every thread
    tokens = tokens < fill ? fill : tokens;
    tokens = tokens > kTokens ? kTokens : tokens < 1 ? 1 : tokens;     // at most 2^18 blocks of a CTA: the reciprocal is good to 2^20
    magic = (uint32_t)((0x100000000ull + per_token - 1) / per_token);
    grid = dim3((unsigned)((n_tokens + tokens - 1) / tokens));
  }
};

}  // namespace

cudaError_t launch_kv_write4(const qre_kv_cache& c, int layer, const qre_kv_rows& r, int n_tokens,
                             const int32_t* token_seq, const int32_t* token_pos, const void* k, const void* v,
                             int* status, cudaStream_t stream) {
  const Cut cut(c, n_tokens, 8);
  auto go = [&](auto kernel) {
    return launch_dependent(kernel, cut.grid, dim3(kThreads), 0, stream, c, layer, r, n_tokens, cut.tokens, cut.magic,
                            token_seq, token_pos, static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), status);
  };
  return r.dtype == QRE_BF16 ? go(kv_write4_kernel<QRE_BF16>) : go(kv_write4_kernel<QRE_FP16>);
}

cudaError_t launch_kv_read(const qre_kv_cache& c, int layer, const qre_kv_rows& r, int n, const int32_t* seqs,
                           const int32_t* first, const int32_t* cu, int total, void* k, void* v, int* status,
                           cudaStream_t stream) {
  // Many small CTAs: those that run write neighbouring rows (131,072 rows: 130 us with 8 per SM, 127 with 128).
  const Cut cut(c, total, 128);
  auto fits = [](const void* p, int64_t token, int64_t head) { return reinterpret_cast<uintptr_t>(p) % 32 == 0 && token % 16 == 0 && head % 16 == 0; };
  const int wide = fits(k, r.k_token, r.k_head) && fits(v, r.v_token, r.v_head);   // whole 32-byte sectors
  auto go = [&](auto kernel) {
    return launch_dependent(kernel, cut.grid, dim3(kThreads), 0, stream, c, layer, r, n, total, cut.tokens, cut.magic, wide,
                            seqs, first, cu, static_cast<uint16_t*>(k), static_cast<uint16_t*>(v), status);
  };
  if (c.dtype == QRE_E4M3) return r.dtype == QRE_BF16 ? go(kv_read_kernel<QRE_BF16, QRE_E4M3>) : go(kv_read_kernel<QRE_FP16, QRE_E4M3>);
  if (c.dtype == QRE_E2M1) return r.dtype == QRE_BF16 ? go(kv_read_kernel<QRE_BF16, QRE_E2M1>) : go(kv_read_kernel<QRE_FP16, QRE_E2M1>);
  return go(kv_read_kernel<QRE_BF16, QRE_BF16>);   // the bits as they are, either type
}

}  // namespace qre
