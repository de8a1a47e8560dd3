// fg_paged.cuh -- what the paged KV cache's kernels share: host checks and page lookup.
#pragma once

#include "fg_internal.cuh"

struct PagedArgs {
  uint8_t *kc, *vc;
  __half *km, *ks, *vm, *vs;
  float *weights;
  int32_t *tokens;
  const int32_t *table;
  int num_pages, ps, ps_shift, max_pages, H;  // ps_shift: log2(ps), -1 if ps is no power of two
  unsigned int *err;
};

// Shape and pointer rules of fg_paged_kv (fg.h); no CUDA call.
fg_status fg_paged_validate(const fg_paged_kv *kv);
// Fills the kernels' view of a valid cache; false if the device's error word has no address.
bool fg_paged_args(const fg_paged_kv *kv, PagedArgs *a);

static inline int fg_paged_capacity(const fg_paged_kv *kv) { return kv->max_pages * kv->page_size; }

// Page of a sequence that slot `p` lies in.
__device__ __forceinline__ int paged_index(const PagedArgs &a, int p) {
  return a.ps_shift >= 0 ? p >> a.ps_shift : p / a.ps;
}

// Pool index of slot `p` (inside the table's pages) of sequence `s`, head `h`; -1: a bad page.
__device__ __forceinline__ int64_t paged_slot(const PagedArgs &a, int s, int h, int p) {
  const int pi = paged_index(a, p);
  const int page = a.table[static_cast<int64_t>(s) * a.max_pages + pi];
  if (page < 0 || page >= a.num_pages) return -1;
  return (static_cast<int64_t>(page) * a.H + h) * a.ps + (p - pi * a.ps);
}
