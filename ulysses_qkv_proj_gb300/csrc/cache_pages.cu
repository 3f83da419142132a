// cache_pages.cu -- bookkeeping and copies of a paged cache: truncate / free,
// fork, reserve (allocation with copy on write), compact, copy pages.
//
// The only allocator state is page_refs: a page is free when no row holds it,
// and a reserve takes the lowest-numbered free pages.  Releases are integer
// decrements, which commute, so every table and every count is the same on
// every run, whatever order the blocks of a launch run in.
//
// Bound: the bookkeeping is launch and load latency.  Release, reserve and compact of a serving step, 64 rows and
// 8 layers: 18.8 us on the device with a warp a row in the reserve (each round a chain of four loads, done twice) and the
// lengths in a launch of their own after the moves; 14.5 with the windows as one list, a thread a block, and a
// cluster a row in the compact; 15.0 since the compact looks at the counts of the pages that it writes.  The page copies of a
// fork's reserve are HBM bandwidth (64 copies of a 2 MB page: 34.2 us with the fork and the release before it, 235 MB).
#include "../../include/qnre.h"
#include "cache.cuh"
#include "ptx.cuh"

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>

namespace {

using namespace qnre;
using namespace qnre::api;

constexpr int kReserveThreads = 1024;
constexpr int kCopyThreads = 256;

// Every launch here is a programmatic dependent launch: its blocks may start while the
// previous kernel drains, and see that kernel's writes after this.
__device__ __forceinline__ void pdl_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Releases the blocks of `row` from `first` >= 0 on (one warp).
__device__ __forceinline__ void release_from(const CacheView& c, int row, int first, int lane) {
  int32_t* table = c.table + static_cast<long long>(row) * c.max_blocks;
  for (int j = first + lane; j < c.max_blocks; j += 32) {
    const int page = table[j];
    if (page < 0) continue;
    table[j] = -1;
    if (page >= c.pages) {
      atomicOr(c.status, QNRE_CACHE_BAD_PAGE);
    } else if (atomicSub(c.refs + page, 1) < 1) {
      atomicAdd(c.refs + page, 1);
      atomicOr(c.status, QNRE_CACHE_BAD_REFS);
    }
  }
}

// One warp a row: its length becomes min(length, lens[i]).
__global__ void __launch_bounds__(128) truncate_kernel(CacheView c, const int32_t* rows, const int32_t* lens, int n) {
  pdl_wait();
  const int i = blockIdx.x * 4 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (i >= n) return;
  const int row = rows[i];
  if (!c.row_ok(row)) return;
  const int old = c.length(row);
  const int len = min(old, max(lens[i], 0));
  __syncwarp();
  if (lane == 0) c.lens[row] = len;
  const long long first = (static_cast<long long>(len) + c.page_size - 1) / c.page_size;
  if (first < c.max_blocks) release_from(c, row, static_cast<int>(first), lane);
}

// One warp a fork: the destination's table is the source's, each page held once more.
__global__ void __launch_bounds__(128) fork_kernel(CacheView c, const int32_t* src, const int32_t* dst, int n) {
  pdl_wait();
  const int i = blockIdx.x * 4 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (i >= n) return;
  const int s = src[i], d = dst[i];
  if (!c.row_ok(s) || !c.row_ok(d)) return;
  const int32_t* from = c.table + static_cast<long long>(s) * c.max_blocks;
  int32_t* to = c.table + static_cast<long long>(d) * c.max_blocks;
  const int len = c.length(s);
  const bool used = s == d || c.lens[d] != 0 || to[0] >= 0;
  __syncwarp();
  if (used) {
    if (lane == 0) atomicOr(c.status, QNRE_CACHE_BAD_ROW);
    return;
  }
  const long long touched = (static_cast<long long>(len) + c.page_size - 1) / c.page_size;
  const int blocks = static_cast<int>(min(touched, static_cast<long long>(c.max_blocks)));
  for (int j = lane; j < blocks; j += 32) {
    const int page = from[j];
    to[j] = page;
    if (page >= 0 && page < c.pages) atomicAdd(c.refs + page, 1);
  }
  if (lane == 0) c.lens[d] = len;
}

// Inclusive scan over the block's threads; `total` is the last value.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  int s = warp_sums[lane];  // kReserveThreads / 32 == 32 warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
    if (lane >= o) s += u;
  }
  total = __shfl_sync(0xFFFFFFFFu, s, 31);
  const int before = __shfl_sync(0xFFFFFFFFu, s, max(warp - 1, 0));
  return v + (warp > 0 ? before : 0);
}

// The words of `scratch`: [0] pages to copy, then free[pages], old[pages], copy
// sources[pages], copy destinations[pages].
struct Scratch {
  int32_t *count, *free, *old, *src, *dst;
  __device__ explicit Scratch(const CacheView& c)
      : count(c.scratch), free(c.scratch + 4), old(free + c.pages), src(old + c.pages), dst(src + c.pages) {}
};

// Blocks of a row that tokens [len, len + count) touch.
struct Window {
  int row, len, first, last;
  bool fits;
};

__device__ __forceinline__ Window window_of(const CacheView& c, const int32_t* rows, const int32_t* counts, int i) {
  Window w{rows[i], 0, 0, 0, true};
  if (w.row < 0 || w.row >= c.rows) return w;
  w.len = c.length(w.row);
  const int count = counts[i];
  if (count <= 0) return w;
  w.first = w.len / c.page_size;
  const long long last = (static_cast<long long>(w.len) + count + c.page_size - 1) / c.page_size;
  w.fits = last <= c.max_blocks;
  w.last = static_cast<int>(min(last, static_cast<long long>(c.max_blocks)));
  return w;
}

// true when block j needs a new page; `shared` when it replaces a page other rows hold.
__device__ __forceinline__ bool needs_page(const CacheView& c, int page, bool& shared) {
  shared = page >= 0 && page < c.pages && c.refs[page] > 1;
  return page < 0 || shared;
}

// Bit e: count at + e is 0, for 16 counts (fewer at the end).
__device__ __forceinline__ unsigned zero_counts(const CacheView& c, long long at) {
  unsigned zero = 0;
  if (at + 16 <= c.pages) {
    int4 r[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) r[q] = reinterpret_cast<const int4*>(c.refs + at)[q];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      zero |= (r[q].x == 0 ? 1u : 0u) << (4 * q) | (r[q].y == 0 ? 2u : 0u) << (4 * q) |
              (r[q].z == 0 ? 4u : 0u) << (4 * q) | (r[q].w == 0 ? 8u : 0u) << (4 * q);
  } else {
    for (int e = 0; e < 16 && at + e < c.pages; ++e) zero |= (c.refs[at + e] == 0 ? 1u : 0u) << e;
  }
  return zero;
}

// One block does a reserve's whole bookkeeping.  The rows' windows lie one after another as a list of blocks, a thread
// a block: which ones need a page (by the counts of the call's start), a scan, as many free pages from the lowest up,
// and a second round that hands them out.  A usual step is one round of 1024 blocks and one of 16384 pages, whose
// counts are fetched first.  Releases of replaced pages come last.
__global__ void __launch_bounds__(kReserveThreads) reserve_kernel(CacheView c, const int32_t* rows,
                                                                  const int32_t* counts, int n) {
  __shared__ int row_of[QNRE_MAX_CALL_ROWS], len_of[QNRE_MAX_CALL_ROWS], first_of[QNRE_MAX_CALL_ROWS];
  __shared__ int start_of[QNRE_MAX_CALL_ROWS + 1];  // of a row's window in the list
  __shared__ int sums[32];
  __shared__ int copies, refused;
  pdl_wait();
  const Scratch s(c);
  const int tid = threadIdx.x;
  const unsigned zero0 = zero_counts(c, static_cast<long long>(tid) * 16);
  if (tid == 0) copies = refused = 0;
  __syncthreads();
  int blocks = 0;
  if (tid < n) {
    const Window w = window_of(c, rows, counts, tid);
    if (w.row < 0 || w.row >= c.rows) atomicOr(c.status, QNRE_CACHE_BAD_ROW);
    if (!w.fits) refused = 1;
    blocks = w.last - w.first;
    row_of[tid] = w.row;
    len_of[tid] = w.len;
    first_of[tid] = w.first;
  }
  int items;
  {
    const int incl = block_scan(blocks, sums, items);
    if (tid < n) start_of[tid + 1] = incl;
    if (tid == 0) start_of[0] = 0;
  }
  __syncthreads();

  // block i of the list: its row (in the call), its number in the row and its page
  auto item = [&](int i, int& k, int& j, int& page, bool& shared) -> bool {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (start_of[mid] <= i) lo = mid; else hi = mid - 1;
    }
    k = lo;
    j = first_of[k] + i - start_of[k];
    page = c.table[static_cast<long long>(row_of[k]) * c.max_blocks + j];
    return needs_page(c, page, shared);
  };

  int k = 0, j = 0, page = -1;
  bool shared = false, take = false;
  int total = 0, before = 0;  // pages wanted; by the blocks of the round before this thread's
  for (int base = 0; base < items; base += kReserveThreads) {
    take = base + tid < items && item(base + tid, k, j, page, shared);
    int step;
    before = block_scan(take ? 1 : 0, sums, step) - (take ? 1 : 0);
    total += step;
  }
  int found = 0;
  if (total <= c.pages && !refused) {
    for (long long base = 0; base < c.pages && found < total; base += kReserveThreads * 16) {
      const long long at = base + tid * 16;
      unsigned zero = base == 0 ? zero0 : zero_counts(c, at);
      int step;
      int pos = found + block_scan(__popc(zero), sums, step) - __popc(zero);
      while (zero != 0 && pos < total) {
        s.free[pos++] = static_cast<int>(at) + __ffs(zero) - 1;
        zero &= zero - 1;
      }
      found += step;
    }
  }
  __syncthreads();
  if (found < total || refused) {
    if (tid == 0) {
      atomicOr(c.status, QNRE_CACHE_NO_PAGES);
      s.count[0] = 0;
    }
    return;
  }
  int done = 0;
  for (int base = 0; base < items; base += kReserveThreads) {
    if (items > kReserveThreads) {  // else the one round's findings still stand
      take = base + tid < items && item(base + tid, k, j, page, shared);
      int step;
      before = block_scan(take ? 1 : 0, sums, step) - (take ? 1 : 0);
      before += done;
      done += step;
    }
    if (take) {
      const int fresh = s.free[before];
      s.old[before] = shared ? page : -1;
      c.table[static_cast<long long>(row_of[k]) * c.max_blocks + j] = fresh;
      if (shared && static_cast<long long>(j) * c.page_size < len_of[k]) {
        const int slot = atomicAdd(&copies, 1);  // copies run in any order; at most `total` of them
        s.src[slot] = page;
        s.dst[slot] = fresh;
      }
    }
  }
  __syncthreads();
  for (int p = tid; p < total; p += kReserveThreads) {
    c.refs[s.free[p]] = 1;
    const int old = s.old[p];
    if (old >= 0) atomicSub(c.refs + old, 1);
  }
  if (tid == 0) s.count[0] = copies;
}

// Copies whole pages of every layer, K and V: item = (pair, layer, K or V, piece).
// 256 threads move 32 KiB an item, eight 16-byte loads in flight a thread.
constexpr int kPieceVecs = kCopyThreads * 8;

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(CacheView c, const int32_t* src, const int32_t* dst,
                                                                  const int32_t* count, int n) {
  pdl_wait();
  const int pairs = count != nullptr ? *count : n;
  const long long page_vecs = static_cast<long long>(c.heads) * c.page_size * c.head_dim / 8;
  const int pieces = static_cast<int>((page_vecs + kPieceVecs - 1) / kPieceVecs);
  const long long items = static_cast<long long>(pairs) * c.layers * 2 * pieces;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int piece = static_cast<int>(it % pieces);
    long long rest = it / pieces;
    const int kv = static_cast<int>(rest & 1);
    rest >>= 1;
    const int layer = static_cast<int>(rest % c.layers);
    const int p = static_cast<int>(rest / c.layers);
    const int a = src[p], b = dst[p];
    if (a < 0 || a >= c.pages || b < 0 || b >= c.pages) {
      if (threadIdx.x == 0) atomicOr(c.status, QNRE_CACHE_BAD_PAGE);
      continue;
    }
    uint4* pool = reinterpret_cast<uint4*>(kv ? c.v : c.k);
    const uint4* from = pool + (static_cast<long long>(layer) * c.pages + a) * page_vecs;
    uint4* to = pool + (static_cast<long long>(layer) * c.pages + b) * page_vecs;
    const long long at = static_cast<long long>(piece) * kPieceVecs + threadIdx.x;
    uint4 r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (at + e * kCopyThreads < page_vecs) r[e] = from[at + e * kCopyThreads];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (at + e * kCopyThreads < page_vecs) to[at + e * kCopyThreads] = r[e];
  }
}

// A compact: a cluster of CTAs takes a row, moves its accepted tokens, and when all of them have, its first CTA grows
// the length and releases the blocks past it.  Tokens are kept up to the first one that would lie in a page that is missing
// or that other rows hold too, or whose source is missing: nothing is written to a shared page, and the length never passes
// what the row's own pages hold.  Every CTA looks for itself and the first one grows by the least that any of them found.
// One thread owns 16 bytes of a head's channels for one
// (layer, K or V, head) and takes the tokens in ascending order, eight at a time: a later token's source is
// never an earlier one's destination (path ascends strictly, so path[j'] >= j' > j), so reads stay ahead of writes
// without any ordering between threads.
__global__ void __launch_bounds__(kCopyThreads) compact_kernel(CacheView c, const int32_t* rows, const int32_t* path,
                                                               const int32_t* counts, int nodes, int lanes, int ctas) {
  __shared__ long long from[QNRE_MAX_NODES], to[QNRE_MAX_NODES];  // head 0's byte offsets in layer 0, -1: skip
  __shared__ int kept, least;  // tokens; the cluster's least in its first CTA
  if (threadIdx.x == 0) kept = least = QNRE_MAX_NODES;
  __syncthreads();
  ptx::cluster_arrive();  // `least` stands
  pdl_wait();
  const int i = blockIdx.x / ctas, part = blockIdx.x % ctas;
  const int row = rows[i];
  const int listed = min(max(counts[i], 0), nodes);
  if (row < 0 || row >= c.rows) {
    if (part == 0 && threadIdx.x == 0) atomicOr(c.status, QNRE_CACHE_BAD_ROW);
    __syncwarp();
    ptx::cluster_wait();
    return;
  }
  const int len = c.length(row);
  for (int j = threadIdx.x; j < listed; j += kCopyThreads) {
    const int node = path[static_cast<long long>(i) * nodes + j];
    from[j] = to[j] = -1;
    const int pd = len <= 0x7FFFFFFF - j ? c.page_of(row, len + j) : -1;
    const int ps = node == j ? pd : (node >= 0 && len <= 0x7FFFFFFF - node ? c.page_of(row, len + node) : -1);
    if (ps < 0 || pd < 0 || c.refs[pd] > 1) {
      atomicMin(&kept, j);
      atomicOr(c.status, QNRE_CACHE_BAD_PAGE);
    } else if (node != j) {
      from[j] = c.token_offset(0, ps, 0, len + node);
      to[j] = c.token_offset(0, pd, 0, len + j);
    }
  }
  __syncthreads();
  const int count = min(kept, listed);
  const int row_vecs = c.head_dim / 8;
  const long long head_bytes = static_cast<long long>(c.page_size) * c.head_dim * 2;
  const long long layer_bytes = static_cast<long long>(c.pages) * c.heads * head_bytes;
  for (long long t = part * kCopyThreads + threadIdx.x; t < lanes; t += ctas * kCopyThreads) {
    const int vec = static_cast<int>(t % row_vecs);
    long long rest = t / row_vecs;
    const int head = static_cast<int>(rest % c.heads);
    rest /= c.heads;
    char* pool = (rest & 1) ? c.v : c.k;
    pool += (rest >> 1) * layer_bytes + head * head_bytes + vec * 16;
    for (int j0 = 0; j0 < count; j0 += 8) {
      uint4 r[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j0 + e < count && from[j0 + e] >= 0) r[e] = *reinterpret_cast<const uint4*>(pool + from[j0 + e]);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j0 + e < count && from[j0 + e] >= 0) *reinterpret_cast<uint4*>(pool + to[j0 + e]) = r[e];
    }
  }
  __syncwarp();
  ptx::cluster_wait();
  if (threadIdx.x == 0 && count < listed)
    asm volatile("red.relaxed.cluster.shared::cluster.min.s32 [%0], %1;" ::"r"(
                     ptx::mapa_shared(ptx::smem_addr(&least), 0)),
                 "r"(count)
                 : "memory");
  // every CTA of the row has read its length and table and made its moves
  __syncwarp();
  ptx::cluster_sync();
  if (part == 0 && threadIdx.x < 32) {
    const int grown = static_cast<int>(min(static_cast<long long>(len) + min(listed, least), 0x7FFFFFFFll));
    if (threadIdx.x == 0) c.lens[row] = grown;
    const long long first = (static_cast<long long>(grown) + c.page_size - 1) / c.page_size;
    if (first < c.max_blocks) release_from(c, row, static_cast<int>(first), threadIdx.x);
  }
}

template <typename K, typename... A>
qnre_status_t launch(K kernel, dim3 grid, dim3 block, unsigned cluster, qnre_stream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return from_cuda(cudaLaunchKernelEx(&cfg, kernel, args...));
}

dim3 copy_grid(const qnre_cache_t* c, int n) {
  const int64_t vecs = static_cast<int64_t>(c->heads) * c->page_size * c->head_dim / 8;
  const int64_t items = static_cast<int64_t>(n) * c->layers * 2 * ((vecs + kPieceVecs - 1) / kPieceVecs);
  return dim3(static_cast<unsigned>(std::min<int64_t>(items, 152 * 4)));
}

qnre_status_t check_call(const qnre_cache_t* cache, std::initializer_list<const void*> lists, int n) {
  const qnre_status_t st = check_cache(cache, n);
  if (st != QNRE_OK) return st;
  for (const void* p : lists) {
    if (p == nullptr && n > 0) return QNRE_ERR_INVALID_ARG;
    if (!aligned(p, 4)) return QNRE_ERR_ALIGNMENT;
  }
  return QNRE_OK;
}

}  // namespace

extern "C" {

qnre_status_t qnre_cache_truncate(const qnre_cache_t* cache, const int32_t* rows, const int32_t* lens, int n,
                                  qnre_stream_t stream) {
  const qnre_status_t st = check_call(cache, {rows, lens}, n);
  if (st != QNRE_OK || n == 0) return st;
  return launch(truncate_kernel, dim3((n + 3) / 4), dim3(128), 1, stream, view_of(cache), rows, lens, n);
}

qnre_status_t qnre_cache_fork(const qnre_cache_t* cache, const int32_t* src, const int32_t* dst, int n,
                              qnre_stream_t stream) {
  const qnre_status_t st = check_call(cache, {src, dst}, n);
  if (st != QNRE_OK || n == 0) return st;
  return launch(fork_kernel, dim3((n + 3) / 4), dim3(128), 1, stream, view_of(cache), src, dst, n);
}

qnre_status_t qnre_cache_reserve(const qnre_cache_t* cache, const int32_t* rows, const int32_t* counts, int n,
                                 qnre_stream_t stream) {
  qnre_status_t st = check_call(cache, {rows, counts}, n);
  if (st != QNRE_OK || n == 0) return st;
  const CacheView c = view_of(cache);
  st = launch(reserve_kernel, dim3(1), dim3(kReserveThreads), 1, stream, c, rows, counts, n);
  if (st != QNRE_OK) return st;
  const int32_t* src = c.scratch + 4 + 2 * static_cast<int64_t>(c.pages);
  const int32_t* count = c.scratch;
  return launch(copy_pages_kernel, copy_grid(cache, n), dim3(kCopyThreads), 1, stream, c, src, src + c.pages,
                count, n);
}

qnre_status_t qnre_cache_compact(const qnre_cache_t* cache, const int32_t* rows, const int32_t* path,
                                 const int32_t* counts, int n, int nodes, qnre_stream_t stream) {
  qnre_status_t st = check_call(cache, {rows, path, counts}, n);
  if (st != QNRE_OK) return st;
  if (nodes < 1) return QNRE_ERR_INVALID_ARG;
  if (nodes > QNRE_MAX_NODES) return QNRE_ERR_CAPACITY;
  if (n == 0) return QNRE_OK;
  const int64_t lanes = static_cast<int64_t>(cache->layers) * 2 * cache->heads * (cache->head_dim / 8);
  if (lanes > (int64_t{1} << 31) - 1) return QNRE_ERR_CAPACITY;
  // as many CTAs a row as its vectors fill, up to a cluster
  unsigned ctas = 1;
  while (ctas < 8 && lanes > static_cast<int64_t>(ctas) * kCopyThreads) ctas *= 2;
  return launch(compact_kernel, dim3(n * ctas), dim3(kCopyThreads), ctas, stream, view_of(cache), rows, path, counts,
                nodes, static_cast<int>(lanes), static_cast<int>(ctas));
}

qnre_status_t qnre_cache_copy_pages(const qnre_cache_t* cache, const int32_t* src, const int32_t* dst, int n,
                                    qnre_stream_t stream) {
  // any number of pages: the lists are read by every block, so the row limit does not apply
  const qnre_status_t st = check_call(cache, {src, dst}, std::min(n, 1));
  if (st != QNRE_OK || n == 0) return st;
  return launch(copy_pages_kernel, copy_grid(cache, n), dim3(kCopyThreads), 1, stream, view_of(cache), src, dst,
                static_cast<const int32_t*>(nullptr), n);
}

}  // extern "C"
