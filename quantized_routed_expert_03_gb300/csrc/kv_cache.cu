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

#include "internal.h"
#include "kv_rows.cuh"

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
// the sum.  `part` is shared memory for 33 values; the call ends with a barrier.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* part, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    T w = part[lane];
    const T own = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    part[lane] = w - own;
    if (lane == 31) part[32] = w;
  }
  __syncthreads();
  const T base = part[warp];
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
// first4: this thread's page_counts of the first step, asked for early.
__device__ int find_free_pages(const int32_t* ref, int n_pages, int want, int32_t* list, int* part, int4 first4) {
  int found = 0;
  for (int p0 = 0; p0 < n_pages && found < want; p0 += kScan) {
    const int p = p0 + 4 * (int)threadIdx.x;
    const int4 r = p0 == 0 ? first4 : page_counts(ref, n_pages, p);
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
  __shared__ long long part64[33];
  __shared__ int first[kKvMaxRequests + 1];
  grid_dependency_wait();
  grid_dependents_launch();
  const int4 first4 = page_counts(c.ref_count, c.n_pages, 4 * (int)threadIdx.x);
  long long sum = 0;
  for (int i0 = 0; i0 < n; i0 += kThreads) {
    const int i = i0 + (int)threadIdx.x;
    long long need = 0;   // below 2^24, but 1024 of them are summed at a time
    if (i < n) {
      const int s = seqs[i], add = n_new[i];
      if (s < 0 || s >= c.max_seqs || add < 0) {
        set_status(status, QRE_DEV_BAD_INDEX);
      } else {
        const long long len = c.seq_len[s] > 0 ? c.seq_len[s] : 0, ps = c.page_size;
        const long long have = (len + ps - 1) / ps, to = (len + add + ps - 1) / ps;
        if (to > c.max_pages) set_status(status, QRE_DEV_NO_PAGE);
        else need = to - have;
      }
    }
    long long total;
    const long long before = block_scan(need, part64, &total);
    // sums beyond the pool saturate: such requests are not served
    const long long at = sum + before;
    if (i < n) first[i] = (int)(at < c.n_pages + 1 ? at : c.n_pages + 1);
    sum += total;
    if (sum > c.n_pages + 1) sum = c.n_pages + 1;
  }
  if (threadIdx.x == 0) first[n] = (int)sum;
  __syncthreads();
  const int want = first[n] < c.n_pages ? first[n] : c.n_pages;
  const int found = find_free_pages(c.ref_count, c.n_pages, want, ws.a, part, first4);
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
    const long long len = c.seq_len[s] > 0 ? c.seq_len[s] : 0, ps = c.page_size;
    if (len + add > c.max_pages * ps) continue;
    // (the request's own need: sums that saturate do not differ)
    const bool needs = (len + add + ps - 1) / ps > (len + ps - 1) / ps;
    if (needs && first[i + 1] > found) set_status(status, QRE_DEV_NO_PAGE);
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
  __shared__ int list[kKvMaxRequests];
  constexpr int kEach = kKvMaxRequests / kThreads;
  int rank[kEach], old[kEach];   // rank of the fresh page (-1: none needed, -2: dropped), the page to copy
  grid_dependency_wait();
  grid_dependents_launch();
  const int4 first4 = page_counts(c.ref_count, c.n_pages, 4 * (int)threadIdx.x);
  int sum = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = e * kThreads + (int)threadIdx.x;
    rank[e] = -2;
    old[e] = -1;
    if (e * kThreads >= n) continue;   // the same for all threads
    int need = 0;
    if (i < n) {
      const int s = src[i], d = dst[i];
      const bool ids = s >= 0 && s < c.max_seqs && d >= 0 && d < c.max_seqs && s != d;
      const int len = ids ? c.seq_len[s] : -1, there = ids ? c.seq_len[d] : -1;
      bool ok = there == 0 && len >= 0 && len <= (long long)c.max_pages * c.page_size;
      if (ok && len % c.page_size) {
        old[e] = c.page_table[(size_t)s * c.max_pages + len / c.page_size];
        ok = page_ok(c, old[e]);
        need = ok;
      }
      if (ok) rank[e] = -1;
      else set_status(status, QRE_DEV_BAD_INDEX);
    }
    int total;
    const int before = block_scan(need, part, &total);
    if (need) rank[e] = sum + before;
    sum += total;
  }
  const int want = sum < c.n_pages ? sum : c.n_pages;
  const int found = find_free_pages(c.ref_count, c.n_pages, want, list, part, first4);
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = e * kThreads + (int)threadIdx.x, r = rank[e];
    if (i >= n) continue;
    int f = r;
    if (r >= found) {
      f = -2;
      set_status(status, QRE_DEV_NO_PAGE);
    } else if (r >= 0) {
      f = list[r];
      ws.a[r] = old[e];
      ws.b[r] = f;
      c.ref_count[f] = 1;
    }
    fresh[i] = f;
  }
  if (threadIdx.x == 0) ws.head[0] = found;
}

// Copies page from -> to of every layer, K and V: one item is 32 KB of one layer's
// page of one of the two (a contiguous run).  Bound by the memory and by how many
// bytes are on their way: with whole pages and one load of a thread at a time 64 forks
// (33 MB copied) took 20.6 us and a compaction of 1024 pages 49.6, now 14.7 and 46.9.
__device__ void copy_pages(const qre_kv_cache& c, const int32_t* from, const int32_t* to, int copies, int first_cta,
                           int ctas) {
  const size_t page = (size_t)c.n_kv_heads * kv_head_bytes(c);
  const int vecs = (int)(page / 16);
  constexpr int kEach = 8;              // 16-byte pieces of a thread on their way
  const int slices = (vecs + kEach * 256 - 1) / (kEach * 256);
  const int per_copy = 2 * c.n_layers * slices;
  const long long items = (long long)copies * per_copy;
  for (long long it = first_cta; it < items; it += ctas) {
    const int j = (int)(it / per_copy), rest = (int)(it - (long long)j * per_copy);
    const int run = rest / slices, i0 = (rest - run * slices) * kEach * 256 + (int)threadIdx.x;
    const int a = from[j], b = to[j];
    if (!page_ok(c, a) || !page_ok(c, b)) continue;
    char* base = static_cast<char*>((run & 1) ? c.v : c.k) + (size_t)(run >> 1) * c.n_pages * page;
    const uint4* s = reinterpret_cast<const uint4*>(base + (size_t)a * page);
    uint4* d = reinterpret_cast<uint4*>(base + (size_t)b * page);
    uint4 x[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (i0 + e * 256 < vecs) x[e] = s[i0 + e * 256];
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (i0 + e * 256 < vecs) d[i0 + e * 256] = x[e];
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

// ---------------------------------------------------------------- common prefix

// One CTA per group: the first column in which the rows of its sequences' tables differ.  Bound by latency (ids and
// lengths, then entries): a thread has one of 256 columns and a quarter of the sequences, 16 loads on their way; the
// first columns' entries are asked for beside the lengths.
__global__ void __launch_bounds__(kThreads) kv_common_len_kernel(const __grid_constant__ qre_kv_cache c, int n,
                                                                 const int32_t* __restrict__ seqs,
                                                                 const int32_t* __restrict__ cu_group,
                                                                 int32_t* __restrict__ common_len, int* status) {
  constexpr int kCols = 256, kParts = kThreads / kCols, kAhead = 16;
  __shared__ int ids[kKvMaxRequests];
  __shared__ int part[32];
  grid_dependency_wait();
  grid_dependents_launch();
  const int a = cu_group[blockIdx.x], b = cu_group[blockIdx.x + 1];
  if (a < 0 || b < a || b > n) {
    if (threadIdx.x == 0) {
      common_len[blockIdx.x] = 0;
      set_status(status, QRE_DEV_BAD_INDEX);
    }
    return;
  }
  if (b - a < 2) {
    if (threadIdx.x == 0) common_len[blockIdx.x] = 0;
    return;
  }
  int bad = 0;
  for (int i = threadIdx.x; i < b - a; i += kThreads) {
    const int s = seqs ? seqs[a + i] : a + i;
    ids[i] = s;
    bad |= s < 0 || s >= c.max_seqs;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) {
      common_len[blockIdx.x] = 0;
      set_status(status, QRE_DEV_BAD_INDEX);
    }
    return;
  }
  // of column col: whether the first row's page is one, and this thread's rows have it too
  const int p0 = (int)threadIdx.x / kCols;
  auto agree = [&](int col) {
    const int page = c.page_table[(size_t)ids[0] * c.max_pages + col];
    bool ok = true;
    for (int i0 = p0; i0 < b - a; i0 += kParts * kAhead) {
      int x[kAhead];
#pragma unroll
      for (int e = 0; e < kAhead; ++e)
        x[e] = i0 + e * kParts < b - a ? c.page_table[(size_t)ids[i0 + e * kParts] * c.max_pages + col] : page;
#pragma unroll
      for (int e = 0; e < kAhead; ++e) ok = ok && x[e] == page;
    }
    return ok && page_ok(c, page);
  };
  int least = 0x7fffffff;
  for (int i = threadIdx.x; i < b - a; i += kThreads) least = min(least, max(c.seq_len[ids[i]], 0));
  const int mine = (int)threadIdx.x % kCols;
  bool ok = mine < c.max_pages ? agree(mine) : false;
  least = __reduce_min_sync(0xffffffffu, least);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = least;
  __syncthreads();
  least = __reduce_min_sync(0xffffffffu, part[threadIdx.x & 31]);
  const long long held = ((long long)least + c.page_size - 1) / c.page_size;
  const int cols = held < c.max_pages ? (int)held : c.max_pages;
  int same = cols;
  for (int c0 = 0; c0 < cols; c0 += kCols) {
    const int col = c0 + mine;
    if (c0 > 0) ok = col < cols ? agree(col) : true;
    const int differ = __reduce_min_sync(0xffffffffu, !ok && col < cols ? col : 0x7fffffff);
    __syncthreads();   // the last step's values have been read
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = differ;
    __syncthreads();
    const int first = __reduce_min_sync(0xffffffffu, part[threadIdx.x & 31]);
    if (first < cols) {   // the same in all threads
      same = first;
      break;
    }
  }
  if (threadIdx.x == 0) {
    const long long positions = (long long)same * c.page_size;
    common_len[blockIdx.x] = positions < least ? (int)positions : least;
  }
}

// ---------------------------------------------------------------- write

template <int RT>
__device__ __forceinline__ float to_float(uint16_t b) {
  return RT == QRE_BF16 ? bf16_bits_to_float(b) : __half2float(__ushort_as_half(b));
}

// Memory bound: each row is read and written once.  A CTA has as many neighbouring
// tokens as let all CTAs run at once; where their rows go, and the scales'
// reciprocals, it looks up once, while the first rows' 16-byte pieces are on their
// way into registers.  No index needs a division of more than a multiply.  11,278
// tokens of 8 heads into E4M3 pages, with the free and the reservation before them:
// 22.8 us; 25.3 with CTAs of two tokens (most of their time was those look-ups), 24.3
// with four pieces of a thread on their way (fewer CTAs fit), 31 with a division for
// every element.
constexpr int kWriteThreads = 256;
constexpr int kWriteEach = 2;        // pieces of a thread on their way
constexpr int kWriteCtas = 8;        // of an SM
constexpr int kWriteTokens = 64;     // of a CTA at most

template <int RT, bool FP8>
__global__ void __launch_bounds__(kWriteThreads, kWriteCtas) kv_write_kernel(
    const __grid_constant__ qre_kv_cache c, int layer, const __grid_constant__ qre_kv_rows r, int n_tokens, int tokens,
    uint32_t magic, const int32_t* __restrict__ token_seq, const int32_t* __restrict__ token_pos,
    const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, int* status) {
  __shared__ long long to[kWriteTokens];   // element of the token's row of head 0, -1: skipped
  __shared__ float by[FP8 ? 2 : 1][FP8 ? kKvMaxHeads : 1];   // 1 / scale of K and of V
  grid_dependency_wait();
  grid_dependents_launch();
  const int per_head_shift = c.head_dim == 64 ? 3 : 4, per_row = c.n_kv_heads << per_head_shift, per_token = 2 * per_row;
  const int t0 = blockIdx.x * tokens, mine = n_tokens - t0 < tokens ? n_tokens - t0 : tokens;
  const int pieces = mine * per_token, ps_shift = 31 - __clz(c.page_size);
  for (int i0 = 0; i0 < pieces; i0 += kWriteThreads * kWriteEach) {
    uint4 x[kWriteEach];
    int at_token[kWriteEach], at_rest[kWriteEach];
#pragma unroll
    for (int e = 0; e < kWriteEach; ++e) {
      const int i = i0 + e * kWriteThreads + (int)threadIdx.x;
      if (i >= pieces) continue;
      const int t = (int)__umulhi((uint32_t)i, magic), rest = i - t * per_token;
      const bool is_v = rest >= per_row;
      const int w = is_v ? rest - per_row : rest, h = w >> per_head_shift, d = (w & ((1 << per_head_shift) - 1)) * 8;
      const uint16_t* src = is_v ? v + (size_t)(t0 + t) * r.v_token + (size_t)h * r.v_head
                                 : k + (size_t)(t0 + t) * r.k_token + (size_t)h * r.k_head;
      x[e] = *reinterpret_cast<const uint4*>(src + d);
      at_token[e] = t;
      at_rest[e] = rest;
    }
    if (i0 == 0) {
      if (FP8)
        for (int i = threadIdx.x; i < 2 * c.n_kv_heads; i += kWriteThreads) {
          const int is_v = i >= c.n_kv_heads, h = is_v ? i - c.n_kv_heads : i;
          const float* scales = is_v ? c.v_scale : c.k_scale;
          by[is_v][h] = scales ? __frcp_rn(scales[(size_t)layer * c.n_kv_heads + h]) : 1.0f;
        }
      if ((int)threadIdx.x < mine) {
        const int pos = token_pos[t0 + threadIdx.x], s = token_seq[t0 + threadIdx.x];
        long long at = -1;
        if (pos >= 0) {
          int p = -1;
          if (s >= 0 && s < c.max_seqs && (pos >> ps_shift) < c.max_pages)
            p = c.page_table[(size_t)s * c.max_pages + (pos >> ps_shift)];
          if (page_ok(c, p))
            at = ((((long long)layer * c.n_pages + p) * c.n_kv_heads << ps_shift) + (pos & (c.page_size - 1))) * c.head_dim;
          else
            set_status(status, QRE_DEV_BAD_INDEX);
        }
        to[threadIdx.x] = at;
      }
      __syncthreads();
    }
#pragma unroll
    for (int e = 0; e < kWriteEach; ++e) {
      const int i = i0 + e * kWriteThreads + (int)threadIdx.x;
      if (i >= pieces || to[at_token[e]] < 0) continue;
      const bool is_v = at_rest[e] >= per_row;
      const int w = is_v ? at_rest[e] - per_row : at_rest[e], h = w >> per_head_shift;
      const size_t at = (size_t)to[at_token[e]] + ((size_t)h << ps_shift) * c.head_dim +
                        (w & ((1 << per_head_shift) - 1)) * 8;
      if (!FP8) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? c.v : c.k) + at) = x[e];
      } else {
        // times the correctly rounded reciprocal, in fp32, then one rounding to 8 bits
        const float inv = by[is_v][h];
        const uint32_t in[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
        uint32_t out[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t b = 0;
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const uint32_t u = in[2 * j + m];
            const float2 f = make_float2(to_float<RT>((uint16_t)u) * inv, to_float<RT>((uint16_t)(u >> 16)) * inv);
            b |= (uint32_t)__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3) << (16 * m);
          }
          out[j] = b;
        }
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? c.v : c.k) + at) = make_uint2(out[0], out[1]);
      }
    }
  }
}

int wide_grid() {
  const int n = device_sm_count() * 8;
  return n > 0 ? n : 1;
}

}  // namespace

size_t kv_ws_bytes(const qre_kv_cache& c) { return 256 + 3 * list_bytes(c); }

cudaError_t launch_kv_common_len(const qre_kv_cache& c, int n, const int32_t* seqs, int n_groups, const int32_t* cu_group,
                                 int32_t* common_len, int* status, cudaStream_t stream) {
  return launch_dependent(kv_common_len_kernel, dim3(n_groups), dim3(kThreads), 0, stream, c, n, seqs, cu_group,
                          common_len, status);
}

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
  if (c.dtype == QRE_E2M1) return launch_kv_write4(c, layer, r, n_tokens, token_seq, token_pos, k, v, status, stream);
  const int per_token = 2 * c.n_kv_heads * (c.head_dim / 8);   // 16-byte pieces: at most 8192
  const int ctas = device_sm_count() * kWriteCtas;
  int tokens = ctas > 0 ? (n_tokens + ctas - 1) / ctas : 1;
  const int most = (1 << 18) / per_token < kWriteTokens ? (1 << 18) / per_token : kWriteTokens;
  tokens = tokens > most ? most : tokens < 1 ? 1 : tokens;
  // floor(i / per_token) = umulhi(i, magic) for the indices of a CTA (below 2^18): per_token is at most 2^13
  const uint32_t magic = (uint32_t)((0x100000000ull + per_token - 1) / per_token);
  const dim3 grid((unsigned)((n_tokens + tokens - 1) / tokens));
  auto go = [&](auto kernel) {
    return launch_dependent(kernel, grid, dim3(kWriteThreads), 0, stream, c, layer, r, n_tokens, tokens, magic, token_seq,
                            token_pos, static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), status);
  };
  if (c.dtype != QRE_E4M3) return go(kv_write_kernel<QRE_BF16, false>);   // the bits as they are, either type
  return r.dtype == QRE_BF16 ? go(kv_write_kernel<QRE_BF16, true>) : go(kv_write_kernel<QRE_FP16, true>);
}

}  // namespace qre
