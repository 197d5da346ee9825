// paged.cuh - device view of a paged bf16 cache and its ragged batch.
#pragma once
#include "common.cuh"

namespace cas {

struct PagedDev {
  uint16_t* k;
  uint16_t* v;
  int64_t n_pages, page_stride, token_stride, head_stride;
  const int32_t* row_start;
  const int32_t* kv_len;
  const int32_t* pages;
  int H, shift;  // kv heads, log2(page size)
  int batch, rows, max_pages;
};

PagedDev make_paged_dev(const cas_paged_kv* kv, const cas_paged_batch* b);
int check_paged(const cas_paged_kv* kv, const cas_paged_batch* b);

// Rows [start, end) of sequence b inside the tensor, and its length in the
// cache; row r is the token at position len - (end - r), which lies in the
// cache while it is in 0..max_pages * page_size - 1.
struct SeqSpan {
  int start, end, len;
};
__device__ __forceinline__ SeqSpan seq_span(const PagedDev& d, int b) {
  SeqSpan s;
  s.start = max(0, d.row_start[b]);
  s.end = max(s.start, min(d.rows, d.row_start[b + 1]));
  s.len = max(0, d.kv_len[b]);
  return s;
}
// Page of position p of sequence b, or -1 (no such page).
__device__ __forceinline__ int64_t page_of(const PagedDev& d, int b, int64_t p) {
  const int64_t i = p >> d.shift;
  if (p < 0 || i >= d.max_pages) return -1;
  const int32_t id = d.pages[(int64_t)b * d.max_pages + i];
  return id >= 0 && id < d.n_pages ? id : -1;
}

}  // namespace cas
