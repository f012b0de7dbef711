// attn_prefill.cu -- attention over packed prompts.
//
// o_i = sum_j softmax_j(scale q_i . k_j) v_j over the keys that query i sees, in
// one pass: with the running maximum m and sum l (fp32, base 2),
//   m' = max(m, max s), l' = l 2^(m - m') + sum 2^(s - m'), o' alike.
#include "attn.cuh"
#include "internal.h"

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

}  // namespace

cudaError_t launch_attn_prefill(const qre_attn& a, int n_seqs, int total_q, int total_k, const int32_t* cu_q,
                                const int32_t* cu_k, const void* q, const void* k, const void* v, void* o, float* lse,
                                int* status, cudaStream_t stream) {
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
