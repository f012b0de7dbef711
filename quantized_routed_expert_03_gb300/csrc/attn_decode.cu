// attn_decode.cu -- attention of one new token per sequence over the paged cache: the launches (attn_decode.cuh has
// the kernels).
#include "attn_decode.cuh"

namespace qre {

size_t attn_decode_ws_bytes(const qre_attn& a, const qre_kv_cache& c, int n) { return decode_ws_bytes(a, c, n); }

cudaError_t launch_attn_decode(const qre_attn& a, const qre_kv_cache& c, int layer, int n, const int32_t* seqs,
                               int max_len, const void* q, void* o, float* lse, void* ws, int* status,
                               cudaStream_t stream) {
  // The kernel counts the places of a launch in 32 bits.  A sequence has at most as many as its table row (or the
  // window) allows, 2^27 and a few, so a launch takes at least 15; a call is split only where rows hold millions
  // of positions.
  const long long chunk = chunk_of(c), held = (long long)c.max_pages * c.page_size;
  const long long places = (a.window > 0 && a.window < held ? a.window : held) / chunk + 2 + kUnitCost;
  const int most = 0x7fffffffll / places < n ? (int)(0x7fffffffll / places) : n;
  for (int i = 0; i < n; i += most) {
    const int m = n - i < most ? n - i : most;
    const cudaError_t e =
        launch_part<false>(a, c, layer, m, seqs ? seqs + i : nullptr, i, max_len, static_cast<const uint16_t*>(q) + i * a.q_token,
                    static_cast<uint16_t*>(o) + i * a.o_token, lse ? lse + (size_t)i * a.n_heads : nullptr, Own{}, ws, status, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace qre
