// attn_decode.cu -- attention of one new token per sequence over the paged cache.
//
// One pass over the sequence's positions with a running maximum and sum (base
// 2, fp32), as in attn_prefill.cu.
#include <cuda_fp8.h>

#include "attn.cuh"
#include "internal.h"

namespace qre {
namespace {

// Element e of a row of the cache.
template <int CT>
__device__ __forceinline__ float cache_value(const void* base, size_t e) {
  if (CT == QRE_E4M3) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(base)[e], __NV_E4M3);
    return __half2float(__half(h));
  }
  return bits_to_float<CT>(static_cast<const uint16_t*>(base)[e]);
}

// One warp per (sequence, head); a lane scores one key at a time, then the lanes
// share the head's dimensions for the values.
template <int DT, int CT, int D>
__global__ void __launch_bounds__(256) attn_decode_kernel(const __grid_constant__ qre_attn a,
                                                          const __grid_constant__ qre_kv_cache c, int layer, int n,
                                                          const int32_t* __restrict__ seqs,
                                                          const uint16_t* __restrict__ q, uint16_t* __restrict__ o,
                                                          float* __restrict__ lse, int* status) {
  __shared__ float qs[8][D];
  grid_dependency_wait();
  grid_dependents_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * 8 + warp;
  if (unit >= (long long)n * a.n_heads) return;
  const int t = (int)(unit / a.n_heads), h = (int)(unit % a.n_heads), hk = h / (a.n_heads / a.n_kv_heads);
  const int s = seqs ? seqs[t] : t;
  int len = 0;
  if (s >= 0 && s < c.max_seqs) len = c.seq_len[s];
  else if (lane == 0) set_status(status, QRE_DEV_BAD_INDEX);
  if (len < 0 || len > (long long)c.max_pages * c.page_size) {
    len = 0;
    if (lane == 0) set_status(status, QRE_DEV_BAD_INDEX);
  }
  int lo, hi;
  visible_range(len - 1, len, 1, a.window, lo, hi);
  const size_t si = (size_t)layer * c.n_kv_heads + hk;
  const float ks = CT == QRE_E4M3 && c.k_scale ? c.k_scale[si] : 1.0f;
  const float vs = CT == QRE_E4M3 && c.v_scale ? c.v_scale[si] : 1.0f;
  for (int d = lane; d < D; d += 32)
    qs[warp][d] = bits_to_float<DT>(q[(size_t)t * a.q_token + (size_t)h * a.q_head + d]) * a.scale * kLog2e * ks;
  __syncwarp();
  float m = -INFINITY, l = 0.0f, acc[D / 32] = {};
  for (int j0 = lo; j0 < hi; j0 += 32) {
    const int j = j0 + lane;
    float x = -INFINITY;
    int page = -1;
    if (j < hi) page = c.page_table[(size_t)s * c.max_pages + j / c.page_size];
    const bool ok = page >= 0 && page < c.n_pages;
    if (j < hi && !ok) set_status(status, QRE_DEV_BAD_INDEX);
    const size_t row =
        ok ? ((((size_t)layer * c.n_pages + page) * c.n_kv_heads + hk) * c.page_size + j % c.page_size) * D : 0;
    if (ok) {
      x = 0.0f;
      for (int d = 0; d < D; ++d) x += qs[warp][d] * cache_value<CT>(c.k, row + d);
    }
    float mx = x;
    for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    const float m2 = fmaxf(m, mx), f = m == -INFINITY ? 0.0f : exp2f(m - m2);
    const float p = ok ? exp2f(x - m2) : 0.0f;
    float sum = p;
    for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    l = l * f + sum;
    m = m2;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] *= f;
    for (int i = 0; i < 32 && j0 + i < hi; ++i) {
      const float pi = __shfl_sync(0xffffffffu, p, i);
      const size_t r = __shfl_sync(0xffffffffu, row, i);
      if (!__shfl_sync(0xffffffffu, (int)ok, i)) continue;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) acc[e] += pi * cache_value<CT>(c.v, r + lane + 32 * e);
    }
  }
  const bool empty = l == 0.0f;
  const float inv = empty ? 0.0f : vs / l;
#pragma unroll
  for (int e = 0; e < D / 32; ++e)
    o[(size_t)t * a.o_token + (size_t)h * a.o_head + lane + 32 * e] = (uint16_t)pack2<DT>(acc[e] * inv, 0.0f);
  if (lse && lane == 0) lse[(size_t)t * a.n_heads + h] = empty ? -INFINITY : m * kLn2 + logf(l);
}

}  // namespace

size_t attn_decode_ws_bytes(const qre_attn&, const qre_kv_cache&, int) { return 256; }

cudaError_t launch_attn_decode(const qre_attn& a, const qre_kv_cache& c, int layer, int n, const int32_t* seqs,
                               int max_len, const void* q, void* o, float* lse, void* ws, int* status,
                               cudaStream_t stream) {
  const long long units = (long long)n * a.n_heads;
  auto go = [&](auto kernel) {
    return launch_dependent(kernel, dim3((unsigned)((units + 7) / 8)), dim3(256), 0, stream, a, c, layer, n, seqs,
                            static_cast<const uint16_t*>(q), static_cast<uint16_t*>(o), lse, status);
  };
  const bool bf = a.dtype == QRE_BF16, d64 = a.head_dim == 64;
  if (c.dtype == QRE_E4M3) {
    if (bf) return d64 ? go(attn_decode_kernel<QRE_BF16, QRE_E4M3, 64>) : go(attn_decode_kernel<QRE_BF16, QRE_E4M3, 128>);
    return d64 ? go(attn_decode_kernel<QRE_FP16, QRE_E4M3, 64>) : go(attn_decode_kernel<QRE_FP16, QRE_E4M3, 128>);
  }
  if (bf) return d64 ? go(attn_decode_kernel<QRE_BF16, QRE_BF16, 64>) : go(attn_decode_kernel<QRE_BF16, QRE_BF16, 128>);
  return d64 ? go(attn_decode_kernel<QRE_FP16, QRE_FP16, 64>) : go(attn_decode_kernel<QRE_FP16, QRE_FP16, 128>);
}

}  // namespace qre
