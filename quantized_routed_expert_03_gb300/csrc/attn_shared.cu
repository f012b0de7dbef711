// attn_shared.cu -- attention of one new token for sequences that share the pages of a prefix.
#include "internal.h"

namespace qre {

size_t attn_shared_ws_bytes(const qre_attn& a, const qre_kv_cache& c, int n, int n_groups) {
  return attn_decode_ws_bytes(a, c, n);
}

cudaError_t launch_attn_decode_shared(const qre_attn& a, const qre_kv_cache& c, int layer, int n, const int32_t* seqs,
                                      int n_groups, const int32_t* cu_group, const int32_t* common_len, int max_len,
                                      const void* q, void* o, float* lse, void* ws, int* status, cudaStream_t stream) {
  return launch_attn_decode(a, c, layer, n, seqs, max_len, q, o, lse, ws, status, stream);
}

}  // namespace qre
