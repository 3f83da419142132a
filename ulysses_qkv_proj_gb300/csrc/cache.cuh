// cache.cuh -- the paged cache as kernels see it, and the argument checks the
// entry points that take one share.
#pragma once

#include "api_util.cuh"

#include <cmath>

namespace qnre {

struct CacheView {
  char* k;
  char* v;
  int32_t* table;
  int32_t* lens;
  int32_t* refs;
  uint32_t* status;
  int32_t* scratch;
  int layers, pages, heads, page_size, head_dim, rows, max_blocks;

  __device__ __forceinline__ bool row_ok(int row) const {
    if (row >= 0 && row < rows) return true;
    atomicOr(status, QNRE_CACHE_BAD_ROW);
    return false;
  }
  // Tokens of a valid row; a length below 0 counts as none, so that no block number is ever negative.
  __device__ __forceinline__ int length(int row) const { return max(lens[row], 0); }
  // Page of token `pos` of a valid row, or -1 (none, or a table entry outside the cache).
  __device__ __forceinline__ int page_of(int row, int pos) const {
    const int block = pos / page_size;
    if (pos < 0 || block >= max_blocks) return -1;
    const int page = table[static_cast<long long>(row) * max_blocks + block];
    return page >= 0 && page < pages ? page : -1;
  }
  // Bytes from the start of k or v to token `pos` of head `head` (its page given).
  __device__ __forceinline__ long long token_offset(int layer, int page, int head, int pos) const {
    return (((static_cast<long long>(layer) * pages + page) * heads + head) * page_size + pos % page_size) *
           (head_dim * 2);
  }
};

namespace api {

inline CacheView view_of(const qnre_cache_t* c) {
  return CacheView{static_cast<char*>(c->k), static_cast<char*>(c->v), c->block_table, c->seq_lens, c->page_refs,
                   c->status,  c->scratch,  c->layers,   c->pages,  c->heads,  c->page_size,
                   c->head_dim, c->rows,    c->max_blocks};
}

inline qnre_status_t check_cache(const qnre_cache_t* c, int n) {
  if (c == nullptr || c->k == nullptr || c->v == nullptr || c->block_table == nullptr || c->seq_lens == nullptr ||
      c->page_refs == nullptr || c->status == nullptr || c->scratch == nullptr)
    return QNRE_ERR_INVALID_ARG;
  if (c->layers < 1 || c->pages < 1 || c->heads < 1 || c->page_size < 1 || c->head_dim < 1 || c->rows < 1 ||
      c->max_blocks < 1 || n < 0)
    return QNRE_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return QNRE_ERR_UNSUPPORTED;
  if (c->dtype != QNRE_DTYPE_BF16 && c->dtype != QNRE_DTYPE_FP16) return QNRE_ERR_UNSUPPORTED;
  if (c->page_size % 8 != 0) return QNRE_ERR_UNSUPPORTED;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->page_refs, 16)) return QNRE_ERR_ALIGNMENT;
  if (!aligned(c->block_table, 4) || !aligned(c->seq_lens, 4) || !aligned(c->status, 4) || !aligned(c->scratch, 4))
    return QNRE_ERR_ALIGNMENT;
  const int64_t top = (int64_t{1} << 31) - 1;
  if (static_cast<int64_t>(c->layers) * c->pages > top || static_cast<int64_t>(c->rows) * c->max_blocks > top ||
      static_cast<int64_t>(c->max_blocks) * c->page_size > top - 256 || c->heads > 65535 ||
      static_cast<int64_t>(c->heads) * c->page_size > top / 256 || n > QNRE_MAX_CALL_ROWS)
    return QNRE_ERR_CAPACITY;
  return QNRE_OK;
}

// Bytes of one of the cache's two pools.
inline uint64_t pool_bytes(const qnre_cache_t* c) {
  return static_cast<uint64_t>(c->layers) * c->pages * c->heads * c->page_size * c->head_dim * 2;
}

// Bytes of the cache's scratch.
inline uint64_t scratch_bytes(const qnre_cache_t* c) { return (4 * static_cast<uint64_t>(c->pages) + 4) * 4; }

}  // namespace api
}  // namespace qnre
