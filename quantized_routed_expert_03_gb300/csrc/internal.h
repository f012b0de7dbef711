// internal.h -- host-side declarations shared by the library's translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/qre.h"

namespace qre {

// Largest token count the bandwidth-bound decode FFN handles in one pass: the
// tokens (as E4M3 terms or fp16 parts) are the N side of its tcgen05 MMAs, at
// most 32 B-operand rows.
constexpr int kDecodeMaxTokens = 8;

// Bytes of each workspace region for a call with T tokens (each call uses its
// own region from offset 0; calls on one stream run one after the other).
size_t route_ws_bytes(const qre_layer_shape& s, int T);
size_t dispatch_ws_bytes(const qre_layer_shape& s, int T);
size_t ffn_ws_bytes(const qre_layer_shape& s, int T);
// The shared-expert-only FFN call keeps its own, smaller workspace.
size_t ffn_shared_ws_bytes(const qre_layer_shape& s, int T);
size_t ffn_prefill_shared_ws_bytes(const qre_layer_shape& s, int T);

// Which groups an expert-FFN launch computes.
enum FfnPart { kFfnAll = 0, kFfnRouted = 1, kFfnShared = 2 };

// Limit of the kernels' pipeline waits in ns (one second unless a test lowered
// it with qre_debug_wait_test), and the test hook's stall (0 = off).
uint64_t wait_limit_ns();
uint64_t test_stall_ns();
// Cost of a host-mapped unit in the decode kernels' range cut (<= 1: off).
int host_unit_cost();

// Sets the calling thread's qre_last_error() message (printf format).
void set_error_message(const char* fmt, ...);

// Device properties, cached per device.
int device_sm_count();
int device_max_smem_optin();
int* device_status_word();   // address of the current device's status word

// Raises a kernel's dynamic shared-memory limit to at least `bytes` on the
// current device (cached, so repeated launches and graph captures skip it).
cudaError_t ensure_smem_limit(const void* kernel, int bytes);

// Launches `kernel` as a programmatic dependent of the kernel before it in the
// stream (it may be scheduled while that kernel finishes).  Every kernel so
// launched executes griddepcontrol.wait before it reads or writes global
// memory that an earlier kernel touches, and lets its own dependent start
// (griddepcontrol.launch_dependents) only after that wait, so a dependent's
// early part never overlaps anything but its direct predecessor.  One kernel is
// excepted: the sequences' own positions of a decode call with shared prefixes
// (attn_decode.cuh, Own) run beside their direct predecessor, the prefixes, of
// which they need nothing.  What earlier kernels wrote they have by a token that
// the kernel before the predecessor (the plan, which has waited) releases as its
// last act and they acquire, and they wait for the predecessor before they end.
template <typename... Params, typename... Args>
cudaError_t launch_dependent_cluster(void (*kernel)(Params...), dim3 grid, dim3 block, int cluster, size_t smem,
                                     cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
  return err != cudaSuccess ? err : cudaGetLastError();
}
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                             Args... args) {
  return launch_dependent_cluster(kernel, grid, block, 1, smem, stream, args...);
}

// Kernel launchers (return the launch error, cudaSuccess otherwise).
// w2 == nullptr: plain matrix of n_rows rows.  Otherwise the gate/up pair:
// n_rows = 2I output rows interleaved in blocks of 16 from w (gate) and w2 (up).
cudaError_t launch_quantize(int n_rows, int k_dim, int group, const float* w, const float* w2, uint8_t* packed,
                            uint16_t* scales, int* status, cudaStream_t stream);

// allow_tc: the workspace has route_ws_bytes (false: the logits only, the CUDA-core kernels).
cudaError_t launch_route(const qre_layer_shape& s, int T, const uint16_t* x, const float* w_router,
                         const float* bias, int32_t* topk_idx, float* topk_w, void* ws,
                         cudaStream_t stream, bool allow_tc = true);

// Router + dispatch in two launches (GEMV, then selection and dispatch in one
// CTA) when route_dispatch_fused(s, T) (one token); the outputs of launch_route
// followed by launch_dispatch.
bool route_dispatch_fused(const qre_layer_shape& s, int T);
cudaError_t launch_route_dispatch(const qre_layer_shape& s, int T, const uint16_t* x, const float* w_router,
                                  const float* bias, int32_t* topk_idx, float* topk_w, int32_t* counts,
                                  int32_t* offsets, int32_t* perm, int32_t* inv_perm, int32_t* active,
                                  int32_t* n_active, void* ws, cudaStream_t stream);

cudaError_t launch_dispatch(const qre_layer_shape& s, int T, const int32_t* topk_idx, int32_t* counts,
                            int32_t* offsets, int32_t* perm, int32_t* inv_perm, int32_t* active,
                            int32_t* n_active, void* ws, int* status, cudaStream_t stream);

// Returns cudaErrorInvalidValue when the shape has no decode kernel instance.
cudaError_t launch_ffn_decode(const qre_layer_shape& s, int T, const uint16_t* x, const qre_slot* slots,
                              const int32_t* offsets, const int32_t* perm, const int32_t* active,
                              const int32_t* n_active, float* expert_out, void* ws, int* status,
                              cudaStream_t stream, int part = kFfnAll);
bool ffn_decode_supported(const qre_layer_shape& s);

// Grouped-GEMM expert FFN for T > kDecodeMaxTokens (tcgen05, TMEM, TMA).
size_t ffn_prefill_ws_bytes(const qre_layer_shape& s, int T);
bool ffn_prefill_supported(const qre_layer_shape& s);
cudaError_t launch_ffn_prefill(const qre_layer_shape& s, int T, const uint16_t* x, const qre_slot* slots,
                               const int32_t* offsets, const int32_t* perm, const int32_t* active,
                               const int32_t* n_active, float* expert_out, void* ws, int* status,
                               cudaStream_t stream, int part = kFfnAll);

cudaError_t launch_cache_update(int E, int S, float decay, const int32_t* active, const int32_t* n_active,
                                float* scores, int32_t* slot_expert, int32_t* expert_slot, const qre_slot* home,
                                const qre_slot* slot_mem, qre_slot* table, int32_t* copy_list, int32_t* n_copies,
                                int max_copies, int* status, cudaStream_t stream);
cudaError_t launch_cache_copy(const qre_layer_shape& s, const qre_slot* home, const qre_slot* slot_mem,
                              const int32_t* copy_list, const int32_t* n_copies, int max_copies,
                              cudaStream_t stream);

// A streaming read of `bytes` bytes (device or host-mapped memory).
cudaError_t launch_read_probe(const void* src, size_t bytes, uint32_t* sink, cudaStream_t stream);

cudaError_t launch_combine(const qre_layer_shape& s, int T, const float* expert_out, const float* topk_w,
                           const int32_t* inv_perm, float* y_f32, uint16_t* y_bf16, cudaStream_t stream);

// 2-D bf16 row-major [rows][cols] tensor map: boxes of 64 columns x box_rows
// rows, 128-byte swizzle, zero fill outside.  False when the driver refuses it
// (e.g. a base that is not 16-byte aligned).
bool make_tmap_bf16(CUtensorMap* m, const void* base, long long rows, int cols, int box_rows);

// 3-D tensor map of [token][head][cols] rows of 16-bit elements (strides in
// elements): boxes of 64 columns x box_heads heads x box_tokens tokens, 128-byte
// swizzle, zero fill outside.  False when the driver refuses it.
bool make_tmap_rows16(CUtensorMap* m, const void* base, long long tokens, long long token_stride, int heads,
                      long long head_stride, int cols, int box_heads, int box_tokens);

// Key-value cache (kv_cache.cu) and attention (attn_prefill.cu, attn_decode.cu).
// The arguments have been checked (api_attn.cu).
constexpr int kKvMaxRequests = 4096;   // sequences, requests or forks of one call
constexpr int kKvMaxHeads = 256;       // KV heads
size_t kv_ws_bytes(const qre_kv_cache& c);
cudaError_t launch_kv_reserve(const qre_kv_cache& c, int n, const int32_t* seqs, const int32_t* n_new, void* ws,
                              int* status, cudaStream_t stream);
cudaError_t launch_kv_write(const qre_kv_cache& c, int layer, const qre_kv_rows& r, int n_tokens,
                            const int32_t* token_seq, const int32_t* token_pos, const void* k, const void* v,
                            int* status, cudaStream_t stream);
// Into a QRE_E2M1 cache, and back out of any (kv_rows.cu).
cudaError_t launch_kv_write4(const qre_kv_cache& c, int layer, const qre_kv_rows& r, int n_tokens,
                             const int32_t* token_seq, const int32_t* token_pos, const void* k, const void* v,
                             int* status, cudaStream_t stream);
cudaError_t launch_kv_read(const qre_kv_cache& c, int layer, const qre_kv_rows& r, int n, const int32_t* seqs,
                           const int32_t* first, const int32_t* cu, int total, void* k, void* v, int* status,
                           cudaStream_t stream);
// Norm and rotation of queries and keys (qk_rope.cu); c: on the way into the cache, NULL: on arrays.
cudaError_t launch_qk_rope(const qre_rope& r, const qre_kv_cache* c, int layer, int n_tokens, const int32_t* token_seq,
                           const int32_t* token_pos, const void* q, const void* k, const void* v, void* q_out, void* k_out,
                           int* status, cudaStream_t stream);
cudaError_t launch_kv_fork(const qre_kv_cache& c, int n, const int32_t* src, const int32_t* dst, void* ws, int* status,
                           cudaStream_t stream);
cudaError_t launch_kv_common_len(const qre_kv_cache& c, int n, const int32_t* seqs, int n_groups, const int32_t* cu_group,
                                 int32_t* common_len, int* status, cudaStream_t stream);
cudaError_t launch_kv_free(const qre_kv_cache& c, int n, const int32_t* seqs, int* status, cudaStream_t stream);
cudaError_t launch_kv_compact(const qre_kv_cache& c, int32_t* table_out, int32_t* ref_out, int32_t* n_live, void* ws,
                              int* status, cudaStream_t stream);
cudaError_t launch_attn_prefill(const qre_attn& a, int n_seqs, int total_q, int total_k, const int32_t* cu_q,
                                const int32_t* cu_k, const void* q, const void* k, const void* v, void* o, float* lse,
                                int* status, cudaStream_t stream);
size_t attn_decode_ws_bytes(const qre_attn& a, const qre_kv_cache& c, int n);
cudaError_t launch_attn_decode(const qre_attn& a, const qre_kv_cache& c, int layer, int n, const int32_t* seqs,
                               int max_len, const void* q, void* o, float* lse, void* ws, int* status,
                               cudaStream_t stream);

// Decode attention with common prefixes read once (attn_shared.cu).
size_t attn_shared_ws_bytes(const qre_attn& a, const qre_kv_cache& c, int n, int n_groups);
cudaError_t launch_attn_decode_shared(const qre_attn& a, const qre_kv_cache& c, int layer, int n, const int32_t* seqs,
                                      int n_groups, const int32_t* cu_group, const int32_t* common_len, int max_len,
                                      const void* q, void* o, float* lse, void* ws, int* status, cudaStream_t stream);

// Router logits on the tensor cores (long token batches): whether a call of T
// tokens takes them, the workspace they need beyond the logits (the router
// weights split into three bf16 parts), and the launch (split, then GEMM).
bool route_tc_wanted(const qre_layer_shape& s, int T);     // by shape (workspace sizing)
bool route_tc_eligible(const qre_layer_shape& s, int T);   // and shared memory of this device
size_t route_tc_split_bytes(const qre_layer_shape& s);
// Returns false when the tensor maps cannot be made (nothing launched then).
bool launch_route_logits_tc(const qre_layer_shape& s, int T, const uint16_t* x, const float* w_router,
                            float* logits, void* split_ws, cudaStream_t stream, cudaError_t* err);

}  // namespace qre
