// paged.cuh -- the paged cache of keys and values as the kernels see it, and
// the checks of its descriptor.
#pragma once

#include "ops.cuh"

namespace q1 {

struct Paged {
  void* k;
  void* v;
  int64_t page_stride, slot_stride, head_stride;  // elements
  const int32_t* table;
  int64_t table_stride;
  const int32_t* kv_len;
  const int32_t* new_start;
  int pages, page_shift, kv_heads, batch;
  int table_tokens;  // tokens a row of the table covers, at most 2^30
  int total_new;
};

// Checks the descriptor and fills in the kernels' form of it.
int check_paged(const char* who, const q1_paged_kv* kv, Paged& p);

// New tokens [first, first + count) of sequence b and its cached length, held
// within what the call was given; `bad`: whether that changed them.
struct SeqSpan {
  int first, count, len;
};
__device__ __forceinline__ SeqSpan seq_span(const Paged& p, int b, bool* bad = nullptr) {
  const int begin = p.new_start[b], end = p.new_start[b + 1], length = p.kv_len[b];
  const int lo = max(0, min(begin, p.total_new));
  const int hi = max(lo, min(end, p.total_new));
  const int len = max(0, min(length, p.table_tokens));
  if (bad) *bad = lo != begin || hi != end || len != length;
  return {lo, hi - lo, len};
}

}  // namespace q1
