// The pages of the 4-bit key/value cache: what kv_cache.hip writes and attend.hip reads.
#pragma once

#include "common.h"

namespace lvq {

// A page holds its tokens head by head, each head's in blocks of 16 tokens.  A block
// of dim channels in g groups:
//   uint8 [16][dim/2]   codes of the keys
//   uint8 [dim/2][16]   codes of the values
//   fp16 [g][16][2]     scale and low end of the keys, then of the values
constexpr int kBlockTokens = 16;

__host__ __device__ constexpr int kv_block_bytes(int dim, int groups) {
  return 16 * dim + 128 * groups;
}

// Where a token lies: the pages as the kernels see them.
struct KvPages {
  uint8_t* pool;
  const int32_t* table;
  int pages, seqs, max_pages;
  uint16_t kv_heads, dim;
  uint8_t page_shift, groups;
};

__host__ __device__ inline int64_t kv_page_size(const KvPages& c) {
  return (int64_t)(c.kv_heads << (c.page_shift - 4)) * kv_block_bytes(c.dim, c.groups);
}

// Page of token `pos` of sequence `seq`, or -1 where there is none: a sequence or
// position outside the table, a page outside the pool.
__device__ __forceinline__ int kv_page(const KvPages& c, int seq, int pos) {
  if (seq < 0 || seq >= c.seqs || pos < 0) return -1;
  const int at = pos >> c.page_shift;
  if (at >= c.max_pages) return -1;
  const int id = c.table[(int64_t)seq * c.max_pages + at];
  return id < 0 || id >= c.pages ? -1 : id;
}

// The block of 16 tokens that holds token `pos` of a page, for one head.
__device__ __forceinline__ uint8_t* kv_block(const KvPages& c, int page, int head, int pos) {
  const int blocks = 1 << (c.page_shift - 4);
  const int at = head * blocks + ((pos >> 4) & (blocks - 1));
  return c.pool + page * kv_page_size(c) + (int64_t)at * kv_block_bytes(c.dim, c.groups);
}

inline bool kv_dim_ok(int dim) { return dim == 64 || dim == 128 || dim == 256; }
inline bool kv_group_ok(int dim, int group) {
  return group == 0 || ((group == 32 || group == 64 || group == 128 || group == 256) &&
                        group <= dim);
}
inline bool kv_page_ok(int page) { return page >= 16 && page <= 1024 && (page & (page - 1)) == 0; }
constexpr int kKvMaxHeads = 1024;

// Checks the description of a cache and fills *p.
int kv_pages(const lvq_kv_cache* c, KvPages* p);

// Bytes of the pool and of the table, for checks of overlap.
inline size_t kv_pool_bytes(const KvPages& p) { return (size_t)p.pages * kv_page_size(p); }
inline size_t kv_table_bytes(const KvPages& p) { return (size_t)p.seqs * p.max_pages * 4; }

}  // namespace lvq
