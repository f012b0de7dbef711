// kv_cache.cu -- the paged key-value cache: pages reserved, forked, freed and
// compacted on the device, and new rows written into them.
//
// State (device memory, owned by the caller): the page table, the lengths, and
// one reference count per page; a page with count 0 is free.  Which pages a
// call takes follows from that state alone: the free pages in ascending order,
// one after the other in the order of the call's list.  So every call is
// deterministic, needs no list of free pages that could fall out of step, and
// runs without the host.
//
// reserve, fork and compact begin with one CTA that scans the counts: 1024
// threads take 4 consecutive pages each, ranks within a block of 4096 pages come
// from warp scans, and the scan ends as soon as it has found what the call
// needs.  The wide part (page copies, table rows) is a second, dependent launch
// over all SMs.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace qre {
namespace {

constexpr int kThreads = 1024;        // of the one-CTA kernels
constexpr int kScan = 4 * kThreads;   // pages per scan step

// Workspace: a few counters, then two lists of page numbers.
struct KvWs {
  int32_t* head;   // [0] page copies of this call
  int32_t* a;      // [n_pages + kKvMaxRequests]
  int32_t* b;      // the same
};

size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }
size_t list_bytes(const qre_kv_cache& c) { return align256(((size_t)c.n_pages + kKvMaxRequests) * sizeof(int32_t)); }

KvWs kv_ws(const qre_kv_cache& c, void* ws) {
  char* p = static_cast<char*>(ws);
  return {reinterpret_cast<int32_t*>(p), reinterpret_cast<int32_t*>(p + 256),
          reinterpret_cast<int32_t*>(p + 256 + list_bytes(c))};
}

// Exclusive prefix sum of one value per thread over a CTA of kThreads; *total is
// the sum.  `part` is shared memory for 33 ints; the call ends with a barrier.
__device__ __forceinline__ int block_scan(int v, int* part, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int w = part[lane];
    const int own = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    part[lane] = w - own;
    if (lane == 31) part[32] = w;
  }
  __syncthreads();
  const int base = part[warp];
  *total = part[32];
  __syncthreads();
  return base + inc - v;
}

// Counts of pages p0 .. p0 + 3 (1 = in use; pages from n_pages on count as in use).
__device__ __forceinline__ int4 page_counts(const int32_t* ref, int n_pages, int p0) {
  if (p0 + 4 <= n_pages) return *reinterpret_cast<const int4*>(ref + p0);
  int4 r = make_int4(1, 1, 1, 1);
  if (p0 < n_pages) r.x = ref[p0];
  if (p0 + 1 < n_pages) r.y = ref[p0 + 1];
  if (p0 + 2 < n_pages) r.z = ref[p0 + 2];
  return r;
}

// Writes the first `want` free pages, ascending, to list; returns how many there are (at most want).
__device__ int find_free_pages(const int32_t* ref, int n_pages, int want, int32_t* list, int* part) {
  int found = 0;
  for (int p0 = 0; p0 < n_pages && found < want; p0 += kScan) {
    const int p = p0 + 4 * (int)threadIdx.x;
    const int4 r = page_counts(ref, n_pages, p);
    const int f[4] = {r.x <= 0, r.y <= 0, r.z <= 0, r.w <= 0};
    int total;
    int rank = found + block_scan(f[0] + f[1] + f[2] + f[3], part, &total);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (f[i]) {
        if (rank < want) list[rank] = p + i;
        ++rank;
      }
    found += total;
  }
  __syncthreads();
  return found < want ? found : want;
}

__device__ __forceinline__ bool page_ok(const qre_kv_cache& c, int p) { return p >= 0 && p < c.n_pages; }

// ---------------------------------------------------------------- free

// One CTA per sequence.  The length is taken by an exchange, so a sequence named
// twice gives its pages back once.
__global__ void __launch_bounds__(128) kv_free_kernel(const __grid_constant__ qre_kv_cache c,
                                                      const int32_t* __restrict__ seqs, int* status) {
  __shared__ int held;
  grid_dependency_wait();
  grid_dependents_launch();
  const int s = seqs[blockIdx.x];
  if (s < 0 || s >= c.max_seqs) {
    if (threadIdx.x == 0) set_status(status, QRE_DEV_BAD_INDEX);
    return;
  }
  if (threadIdx.x == 0) {
    const int len = atomicExch(&c.seq_len[s], 0);
    const long long pages = len > 0 ? ((long long)len + c.page_size - 1) / c.page_size : 0;
    held = pages < c.max_pages ? (int)pages : c.max_pages;
  }
  __syncthreads();
  int32_t* row = c.page_table + (size_t)s * c.max_pages;
  for (int i = threadIdx.x; i < held; i += blockDim.x) {
    const int p = row[i];
    if (!page_ok(c, p) || atomicSub(&c.ref_count[p], 1) <= 0) {
      if (page_ok(c, p)) atomicAdd(&c.ref_count[p], 1);   // a page nobody held stays free
      set_status(status, QRE_DEV_BAD_INDEX);
    }
    row[i] = -1;
  }
}

// ---------------------------------------------------------------- reserve

// One CTA.  need[i] pages of request i; first[i] = pages of the requests before
// it; the request is served iff first[i] + need[i] pages are free or it needs none.
__global__ void __launch_bounds__(kThreads) kv_reserve_kernel(const __grid_constant__ qre_kv_cache c, int n,
                                                              const int32_t* __restrict__ seqs,
                                                              const int32_t* __restrict__ n_new, KvWs ws,
                                                              int* status) {
  __shared__ int part[33];
  __shared__ int first[kKvMaxRequests + 1];
  grid_dependency_wait();
  grid_dependents_launch();
  long long sum = 0;
  for (int i0 = 0; i0 < n; i0 += kThreads) {
    const int i = i0 + (int)threadIdx.x;
    int need = 0;
    if (i < n) {
      const int s = seqs[i], add = n_new[i];
      if (s < 0 || s >= c.max_seqs || add < 0) {
        set_status(status, QRE_DEV_BAD_INDEX);
      } else {
        const long long len = c.seq_len[s] > 0 ? c.seq_len[s] : 0, ps = c.page_size;
        const long long have = (len + ps - 1) / ps, to = (len + add + ps - 1) / ps;
        if (to > c.max_pages) set_status(status, QRE_DEV_NO_PAGE);
        else need = (int)(to - have);
      }
    }
    int total;
    const int before = block_scan(need, part, &total);
    // sums beyond the pool saturate: such requests are not served
    const long long at = sum + before;
    if (i < n) first[i] = (int)(at < c.n_pages + 1 ? at : c.n_pages + 1);
    sum += total;
    if (sum > c.n_pages + 1) sum = c.n_pages + 1;
  }
  if (threadIdx.x == 0) first[n] = (int)sum;
  __syncthreads();
  const int want = first[n] < c.n_pages ? first[n] : c.n_pages;
  const int found = find_free_pages(c.ref_count, c.n_pages, want, ws.a, part);
  // the pages, spread over the threads: page number r belongs to the last request with first <= r
  for (int r = threadIdx.x; r < found; r += kThreads) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (first[mid] <= r) lo = mid;
      else hi = mid - 1;
    }
    if (first[lo + 1] > found) continue;   // its request is not served
    const int s = seqs[lo];
    const int len = c.seq_len[s] > 0 ? c.seq_len[s] : 0;
    const int col = (int)(((long long)len + c.page_size - 1) / c.page_size) + r - first[lo];
    const int p = ws.a[r];
    c.page_table[(size_t)s * c.max_pages + col] = p;
    c.ref_count[p] = 1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int s = seqs[i], add = n_new[i];
    if (s < 0 || s >= c.max_seqs || add < 0) continue;
    const long long len = c.seq_len[s] > 0 ? c.seq_len[s] : 0;
    if (len + add > (long long)c.max_pages * c.page_size) continue;
    if (first[i + 1] > first[i] && first[i + 1] > found) set_status(status, QRE_DEV_NO_PAGE);
    else c.seq_len[s] = (int)(len + add);
  }
}

// ---------------------------------------------------------------- fork

// One CTA: which requests stand, the fresh page of each one whose last page is
// not full, and the list of page copies (ws.a: from, ws.b: to).
__global__ void __launch_bounds__(kThreads) kv_fork_plan_kernel(const __grid_constant__ qre_kv_cache c, int n,
                                                                const int32_t* __restrict__ src,
                                                                const int32_t* __restrict__ dst, KvWs ws,
                                                                int32_t* fresh, int* status) {
  __shared__ int part[33];
  __shared__ int rank_of[kKvMaxRequests];   // rank of the fresh page, -1 none needed, -2 dropped
  grid_dependency_wait();
  grid_dependents_launch();
  int sum = 0;
  for (int i0 = 0; i0 < n; i0 += kThreads) {
    const int i = i0 + (int)threadIdx.x;
    int need = 0, state = -2;
    if (i < n) {
      const int s = src[i], d = dst[i];
      if (s < 0 || s >= c.max_seqs || d < 0 || d >= c.max_seqs || s == d || c.seq_len[d] != 0 || c.seq_len[s] < 0 ||
          c.seq_len[s] > (long long)c.max_pages * c.page_size) {
        set_status(status, QRE_DEV_BAD_INDEX);
      } else {
        state = -1;
        const int len = c.seq_len[s];
        if (len % c.page_size) {
          if (page_ok(c, c.page_table[(size_t)s * c.max_pages + len / c.page_size])) need = 1;
          else {
            state = -2;
            set_status(status, QRE_DEV_BAD_INDEX);
          }
        }
      }
    }
    int total;
    const int before = block_scan(need, part, &total);
    if (i < n) rank_of[i] = need ? sum + before : state;
    sum += total;
  }
  __syncthreads();
  const int want = sum < c.n_pages ? sum : c.n_pages;
  const int found = find_free_pages(c.ref_count, c.n_pages, want, ws.b, part);
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int r = rank_of[i];
    int f = r;
    if (r >= found) {
      f = -2;
      set_status(status, QRE_DEV_NO_PAGE);
    } else if (r >= 0) {
      const int s = src[i];
      f = ws.b[r];
      ws.a[r] = c.page_table[(size_t)s * c.max_pages + c.seq_len[s] / c.page_size];
      c.ref_count[f] = 1;
    }
    fresh[i] = f;
  }
  if (threadIdx.x == 0) ws.head[0] = found;
}

// Copies page from -> to of every layer, K and V: one item is one layer's page of
// one of the two, a contiguous run.
__device__ void copy_pages(const qre_kv_cache& c, const int32_t* from, const int32_t* to, int copies, int first_cta,
                           int ctas) {
  const size_t page = (size_t)c.n_kv_heads * c.page_size * c.head_dim * (c.dtype == QRE_E4M3 ? 1 : 2);
  const int vecs = (int)(page / 16);
  const long long items = (long long)copies * c.n_layers * 2;
  for (long long it = first_cta; it < items; it += ctas) {
    const int j = (int)(it / (2 * c.n_layers)), l = (int)(it % (2 * c.n_layers)) >> 1;
    const int a = from[j], b = to[j];
    if (!page_ok(c, a) || !page_ok(c, b)) continue;
    char* base = static_cast<char*>((it & 1) ? c.v : c.k) + (size_t)l * c.n_pages * page;
    const uint4* s = reinterpret_cast<const uint4*>(base + (size_t)a * page);
    uint4* d = reinterpret_cast<uint4*>(base + (size_t)b * page);
    for (int i = threadIdx.x; i < vecs; i += blockDim.x) d[i] = s[i];
  }
}

// The first n CTAs write one destination's table row each; all copy pages.
__global__ void __launch_bounds__(256) kv_fork_kernel(const __grid_constant__ qre_kv_cache c, int n,
                                                      const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
                                                      KvWs ws, const int32_t* __restrict__ fresh) {
  grid_dependency_wait();
  grid_dependents_launch();
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int f = fresh[i];
    if (f == -2) continue;
    const int s = src[i], d = dst[i], len = c.seq_len[s], full = len / c.page_size;
    const int32_t* from = c.page_table + (size_t)s * c.max_pages;
    int32_t* to = c.page_table + (size_t)d * c.max_pages;
    for (int j = threadIdx.x; j < full; j += blockDim.x) {
      const int p = from[j];
      to[j] = p;
      if (page_ok(c, p)) atomicAdd(&c.ref_count[p], 1);
    }
    if (threadIdx.x == 0) {
      if (f >= 0) to[full] = f;
      c.seq_len[d] = len;
    }
  }
  copy_pages(c, ws.a, ws.b, ws.head[0], blockIdx.x, gridDim.x);
}

// ---------------------------------------------------------------- compact

// One CTA: the number of live pages, then the holes below it and the live pages
// above it, each in ascending order (ws.b: holes, ws.a: movers), and the new counts.
__global__ void __launch_bounds__(kThreads) kv_compact_plan_kernel(const __grid_constant__ qre_kv_cache c, KvWs ws,
                                                                   int32_t* remap, int32_t* ref_out, int32_t* n_live) {
  __shared__ int part[33];
  grid_dependency_wait();
  grid_dependents_launch();
  int live = 0;
  for (int p = threadIdx.x; p < c.n_pages; p += kThreads) live += c.ref_count[p] > 0;
  int L;
  block_scan(live, part, &L);
  int holes = 0, movers = 0;
  for (int p0 = 0; p0 < c.n_pages; p0 += kScan) {
    const int p = p0 + 4 * (int)threadIdx.x;
    const int4 r = page_counts(c.ref_count, c.n_pages, p);
    const int in[4] = {r.x > 0, r.y > 0, r.z > 0, r.w > 0};
    int h = 0, m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h += p + i < L && !in[i];
      m += p + i >= L && p + i < c.n_pages && in[i];
    }
    int total;   // both ranks from one scan: at most 4096 of each in a step
    const int before = block_scan(h | (m << 16), part, &total);
    int hr = holes + (before & 0xffff), mr = movers + (before >> 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (p + i < L && !in[i]) ws.b[hr++] = p + i;
      if (p + i >= L && p + i < c.n_pages && in[i]) ws.a[mr++] = p + i;
    }
    holes += total & 0xffff;
    movers += total >> 16;
  }
  __syncthreads();
  // as many holes as movers; counts move with their pages, everything else above L is free
  for (int j = threadIdx.x; j < movers; j += kThreads) remap[ws.a[j] - L] = ws.b[j];
  if (ref_out != c.ref_count) {
    for (int p = threadIdx.x; p < L; p += kThreads)
      if (c.ref_count[p] > 0) ref_out[p] = c.ref_count[p];
  }
  for (int j = threadIdx.x; j < movers; j += kThreads) ref_out[ws.b[j]] = c.ref_count[ws.a[j]];
  __syncthreads();
  for (int p = L + threadIdx.x; p < c.n_pages; p += kThreads) ref_out[p] = 0;
  if (threadIdx.x == 0) {
    *n_live = L;
    ws.head[0] = movers;
    ws.head[1] = L;
  }
}

__global__ void __launch_bounds__(256) kv_compact_kernel(const __grid_constant__ qre_kv_cache c, KvWs ws,
                                                         const int32_t* __restrict__ remap, int32_t* table_out,
                                                         int* status) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int L = ws.head[1];
  const long long entries = (long long)c.max_seqs * c.max_pages;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < entries;
       i += (long long)gridDim.x * blockDim.x) {
    const int p = c.page_table[i];
    int to = p;
    if (p >= c.n_pages) set_status(status, QRE_DEV_BAD_INDEX);
    // an entry that names a free page (its count is 0) keeps its number
    else if (p >= L && ws.head[0] > 0) {
      int lo = 0, hi = ws.head[0] - 1;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (ws.a[mid] < p) lo = mid + 1;
        else hi = mid;
      }
      if (ws.a[lo] == p) to = remap[p - L];
      else set_status(status, QRE_DEV_BAD_INDEX);
    }
    table_out[i] = to;
  }
  copy_pages(c, ws.a, ws.b, ws.head[0], blockIdx.x, gridDim.x);
}

// ---------------------------------------------------------------- write

template <int RT>
__device__ __forceinline__ float to_float(uint16_t b) {
  return RT == QRE_BF16 ? bf16_bits_to_float(b) : __half2float(__ushort_as_half(b));
}

// One thread moves 8 elements of one row of K or V.
template <int RT, bool FP8>
__global__ void __launch_bounds__(256) kv_write_kernel(const __grid_constant__ qre_kv_cache c, int layer,
                                                       const __grid_constant__ qre_kv_rows r, int n_tokens,
                                                       const int32_t* __restrict__ token_seq,
                                                       const int32_t* __restrict__ token_pos,
                                                       const uint16_t* __restrict__ k, const uint16_t* __restrict__ v,
                                                       int* status) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int per_head = c.head_dim / 8, per_row = c.n_kv_heads * per_head;
  const long long total = 2ll * n_tokens * per_row;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (long long)gridDim.x * blockDim.x) {
    const int t = (int)(i / (2 * per_row)), rest = (int)(i - (long long)t * 2 * per_row);
    const bool is_v = rest >= per_row;
    const int w = is_v ? rest - per_row : rest, h = w / per_head, d = (w - h * per_head) * 8;
    const int pos = token_pos[t], s = token_seq[t];
    if (pos < 0) continue;
    int p = -1;
    if (s >= 0 && s < c.max_seqs && pos / c.page_size < c.max_pages)
      p = c.page_table[(size_t)s * c.max_pages + pos / c.page_size];
    if (!page_ok(c, p)) {
      set_status(status, QRE_DEV_BAD_INDEX);
      continue;
    }
    const uint16_t* src = is_v ? v + (size_t)t * r.v_token + (size_t)h * r.v_head
                               : k + (size_t)t * r.k_token + (size_t)h * r.k_head;
    const uint4 x = *reinterpret_cast<const uint4*>(src + d);
    const size_t at =
        ((((size_t)layer * c.n_pages + p) * c.n_kv_heads + h) * c.page_size + pos % c.page_size) * c.head_dim + d;
    if (!FP8) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? c.v : c.k) + at) = x;
    } else {
      // the quotient is IEEE, so a row divided elsewhere in fp32 gives the same byte; one rounding to 8 bits
      const float* scales = is_v ? c.v_scale : c.k_scale;
      const float sc = scales ? scales[(size_t)layer * c.n_kv_heads + h] : 1.0f;
      const uint32_t in[4] = {x.x, x.y, x.z, x.w};
      uint32_t out[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t b = 0;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const uint32_t u = in[2 * j + m];
          const float2 f = make_float2(__fdiv_rn(to_float<RT>((uint16_t)u), sc),
                                       __fdiv_rn(to_float<RT>((uint16_t)(u >> 16)), sc));
          b |= (uint32_t)__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3) << (16 * m);
        }
        out[j] = b;
      }
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? c.v : c.k) + at) = make_uint2(out[0], out[1]);
    }
  }
}

int wide_grid() {
  const int n = device_sm_count() * 8;
  return n > 0 ? n : 1;
}

}  // namespace

size_t kv_ws_bytes(const qre_kv_cache& c) { return 256 + 3 * list_bytes(c); }

cudaError_t launch_kv_free(const qre_kv_cache& c, int n, const int32_t* seqs, int* status, cudaStream_t stream) {
  return launch_dependent(kv_free_kernel, dim3(n), dim3(128), 0, stream, c, seqs, status);
}

cudaError_t launch_kv_reserve(const qre_kv_cache& c, int n, const int32_t* seqs, const int32_t* n_new, void* ws,
                              int* status, cudaStream_t stream) {
  return launch_dependent(kv_reserve_kernel, dim3(1), dim3(kThreads), 0, stream, c, n, seqs, n_new, kv_ws(c, ws),
                          status);
}

cudaError_t launch_kv_fork(const qre_kv_cache& c, int n, const int32_t* src, const int32_t* dst, void* ws, int* status,
                           cudaStream_t stream) {
  const KvWs w = kv_ws(c, ws);
  int32_t* fresh = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + 256 + 2 * list_bytes(c));
  const cudaError_t e = launch_dependent(kv_fork_plan_kernel, dim3(1), dim3(kThreads), 0, stream, c, n, src, dst, w,
                                         fresh, status);
  if (e != cudaSuccess) return e;
  return launch_dependent(kv_fork_kernel, dim3(wide_grid()), dim3(256), 0, stream, c, n, src, dst, w, fresh);
}

cudaError_t launch_kv_compact(const qre_kv_cache& c, int32_t* table_out, int32_t* ref_out, int32_t* n_live, void* ws,
                              int* status, cudaStream_t stream) {
  const KvWs w = kv_ws(c, ws);
  int32_t* remap = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + 256 + 2 * list_bytes(c));
  const cudaError_t e = launch_dependent(kv_compact_plan_kernel, dim3(1), dim3(kThreads), 0, stream, c, w, remap,
                                         ref_out, n_live);
  if (e != cudaSuccess) return e;
  return launch_dependent(kv_compact_kernel, dim3(wide_grid()), dim3(256), 0, stream, c, w, remap, table_out, status);
}

cudaError_t launch_kv_write(const qre_kv_cache& c, int layer, const qre_kv_rows& r, int n_tokens,
                            const int32_t* token_seq, const int32_t* token_pos, const void* k, const void* v,
                            int* status, cudaStream_t stream) {
  const long long total = 2ll * n_tokens * c.n_kv_heads * (c.head_dim / 8);
  const long long blocks = (total + 255) / 256, most = wide_grid() * 4ll;
  const dim3 grid((unsigned)(blocks < most ? blocks : most));
  auto go = [&](auto kernel) {
    return launch_dependent(kernel, grid, dim3(256), 0, stream, c, layer, r, n_tokens, token_seq, token_pos,
                            static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), status);
  };
  if (c.dtype != QRE_E4M3) return go(kv_write_kernel<QRE_BF16, false>);   // the bits as they are, either type
  return r.dtype == QRE_BF16 ? go(kv_write_kernel<QRE_BF16, true>) : go(kv_write_kernel<QRE_FP16, true>);
}

}  // namespace qre
