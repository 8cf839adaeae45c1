// Index arithmetic of the paged KV cache.  Every value from device memory that the kernels form an
// address of (a length, a page number, a slot, a chosen page) is checked by one of these functions,
// which return false, -1 or a clamped length for anything out of range.  Plain C++ as well, so that
// the bounds are tested on the CPU.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define PG_HD __host__ __device__ __forceinline__
#else
#define PG_HD inline
#endif

namespace rtvla {

// What an index needs to know of a cache.  Pages hold 1 << shift tokens.
struct PageGeom {
  int shift;        // log2(page_size)
  int n_pages;      // pages in the pool
  int width;        // block-table entries per request
  int n_kv_heads;
  int head_dim;
};

// A request's length, clamped to what its table row can hold.
PG_HD int pg_len(int len, const PageGeom &g, bool *bad) {
  const int cap = g.width << g.shift;
  if (len < 0 || len > cap) {
    *bad = true;
    return len < 0 ? 0 : cap;
  }
  return len;
}

// Pages that hold `n` tokens (0 <= n <= 2^24).
PG_HD int pg_pages(int n, const PageGeom &g) { return (n + (1 << g.shift) - 1) >> g.shift; }

// Is `page` a page of the pool?
PG_HD bool pg_in_pool(int page, const PageGeom &g) { return page >= 0 && page < g.n_pages; }

// Physical page of entry `e` of a table row, -1 when the entry or its content is out of range.
PG_HD int pg_page(const int32_t *row, int e, const PageGeom &g) {
  if (e < 0 || e >= g.width) return -1;
  const int p = row[e];
  return pg_in_pool(p, g) ? p : -1;
}

// Keys that a request's `len` tokens give when it attends to `n_sel` of its pages (no list: all).
// With a list, every entry counts a whole page; the kernel masks what lies past `len`.
PG_HD int pg_list_len(int len, int n_sel, bool listed, const PageGeom &g) {
  if (!listed) return len;
  const int held = pg_pages(len, g);
  return (held < n_sel ? held : n_sel) << g.shift;
}

// Row (page * page_size + offset) of the j-th key a request attends to, -1 when it attends to
// none there: past its length, a listed page it does not hold, a page outside the pool.  `sel`
// is the request's list of logical pages for this KV head, or null.  Sets *bad where the caller's
// table or list is at fault (a key merely past the length is not).
PG_HD int pg_key_row(const int32_t *row, const int32_t *sel, int j, int n_keys, int len, const PageGeom &g,
                     bool *bad) {
  if (j < 0 || j >= n_keys) return -1;
  const int off = j & ((1 << g.shift) - 1);
  int e = j >> g.shift;
  if (sel) {
    e = sel[e];
    if (e < 0 || e >= pg_pages(len, g)) {
      *bad = true;
      return -1;
    }
  }
  if ((e << g.shift) + off >= len) return -1;
  const int p = pg_page(row, e, g);
  if (p < 0) {
    *bad = true;
    return -1;
  }
  return (p << g.shift) + off;
}

// A slot the caller gave: -1 skips the row, anything else must lie in the pool.
PG_HD int pg_slot(int slot, const PageGeom &g, bool *bad) {
  if (slot == -1) return -1;
  if (slot < 0 || (slot >> g.shift) >= g.n_pages) {
    *bad = true;
    return -1;
  }
  return slot;
}

// First element of token row `row` of KV head `h` in layer `layer`.
PG_HD size_t pg_elem(int layer, int row, int h, const PageGeom &g) {
  const size_t page = (size_t)layer * g.n_pages + (size_t)(row >> g.shift);
  const size_t off = (size_t)(row & ((1 << g.shift) - 1));
  return (((page * g.n_kv_heads + h) << g.shift) + off) * g.head_dim;
}

// First element of the mean key of physical page `p`.
PG_HD size_t pg_mean_elem(int layer, int p, int h, const PageGeom &g) {
  return (((size_t)layer * g.n_pages + p) * g.n_kv_heads + h) * g.head_dim;
}

}  // namespace rtvla
