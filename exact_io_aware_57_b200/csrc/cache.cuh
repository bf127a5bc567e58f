// Key/value cache shared by the cache kernels: where a slot lies and which
// lengths and page numbers are accepted.
#pragma once

#include "common.cuh"

namespace attn {

// A cache of `batch` sequences: slot s of sequence b is row s % page_size of
// page table[b * max_pages + s / page_size], or row s of page b without a table.
struct CacheView {
  void *k, *v;
  const int* table;  // device [batch, max_pages] or null
  const int* lens;   // device [batch]
  int num_pages, page_size, max_pages;  // max_pages 1 without a table
};

ATTN_DEVINL long long cache_capacity(const CacheView& c) { return (long long)c.max_pages * c.page_size; }

// Slots of sequence b in use; false (and ATTN_ERR_INVALID in the status word)
// for a length that is negative or beyond `most` slots.
ATTN_DEVINL bool cache_len(const CacheView& c, int b, long long most, int* status, int& len) {
  len = c.lens[b];
  if (len < 0 || len > min(most, cache_capacity(c))) {
    atomicExch(status, ATTN_ERR_INVALID);
    return false;
  }
  return true;
}

// Rows of sequence b that count: row_lens[b], or all; false (and
// ATTN_ERR_INVALID) outside [0, most].
ATTN_DEVINL bool row_count(const int* row_lens, int b, int most, int* status, int& n) {
  n = row_lens ? row_lens[b] : most;
  if (n < 0 || n > most) {
    atomicExch(status, ATTN_ERR_INVALID);
    return false;
  }
  return true;
}

// Row of the page pools (a row holds h_kv * d elements) of slot s; -1 (and
// ATTN_ERR_INVALID) when the table names a page outside the pool.
ATTN_DEVINL long long cache_row(const CacheView& c, int b, int s, int* status) {
  if (!c.table) return (long long)b * c.page_size + s;
  const int page = __ldg(c.table + (long long)b * c.max_pages + s / c.page_size);
  if (page < 0 || page >= c.num_pages) {
    atomicExch(status, ATTN_ERR_INVALID);
    return -1;
  }
  return (long long)page * c.page_size + s % c.page_size;
}

}  // namespace attn
