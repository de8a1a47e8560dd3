// fg_paged.cu -- the paged 4-bit KV cache: host checks and the append of new k, v rows.
//
// "FlexGen Guide: High-Throughput LLM Offloading on One GPU", section 3: the KV cache is held as
// 4-bit groups; the format and its fp32 steps are those of fg.h, the group quantiser is the one
// that the contiguous cache's append uses, so both caches receive the same bits.
#include "fg_paged.cuh"

fg_status fg_paged_validate(const fg_paged_kv *kv) {
  if (!kv) return FG_ERR_INVALID;
  if (kv->num_seqs < 0 || kv->num_pages < 1 || kv->max_pages < 1 || kv->num_heads < 1 || kv->page_size < 1)
    return FG_ERR_INVALID;
  const int G = fg_kv_group(kv->group);
  if (G == 0 || (kv->head_dim != 64 && kv->head_dim != 128 && kv->head_dim != 256)) return FG_ERR_UNSUPPORTED;
  if (kv->head_dim % G || kv->page_size % 16) return FG_ERR_SHAPE;
  if (static_cast<int64_t>(kv->max_pages) * kv->page_size > INT32_MAX) return FG_ERR_SHAPE;
  if (!kv->k_codes || !kv->v_codes || !kv->k_mins || !kv->k_scales || !kv->v_mins || !kv->v_scales || !kv->page_table)
    return FG_ERR_INVALID;
  if (!fg_aligned16(kv->k_codes) || !fg_aligned16(kv->v_codes) || !fg_aligned16(kv->k_mins) ||
      !fg_aligned16(kv->k_scales) || !fg_aligned16(kv->v_mins) || !fg_aligned16(kv->v_scales) ||
      !fg_aligned16(kv->weights) || !fg_aligned16(kv->tokens))
    return FG_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(kv->page_table) & 3u) return FG_ERR_INVALID;
  return FG_OK;
}

bool fg_paged_args(const fg_paged_kv *kv, PagedArgs *a) {
  a->kc = kv->k_codes;
  a->vc = kv->v_codes;
  a->km = reinterpret_cast<__half *>(kv->k_mins);
  a->ks = reinterpret_cast<__half *>(kv->k_scales);
  a->vm = reinterpret_cast<__half *>(kv->v_mins);
  a->vs = reinterpret_cast<__half *>(kv->v_scales);
  a->weights = kv->weights;
  a->tokens = kv->tokens;
  a->table = kv->page_table;
  a->num_pages = kv->num_pages;
  a->ps = kv->page_size;
  a->ps_shift = (kv->page_size & (kv->page_size - 1)) ? -1 : __builtin_ctz(kv->page_size);
  a->max_pages = kv->max_pages;
  a->H = kv->num_heads;
  a->err = fg_error_word_ptr();
  return a->err != nullptr;
}

namespace {

struct AppendArgs {
  PagedArgs kv;
  const __half *k, *v;
  int64_t ld;
  int rows, rows_per_seq, ng;  // ng: groups per head (head_dim / G)
  const int32_t *positions, *counts, *first;
};

// One warp per (row, head): its 2 * ng groups (k and v), G/8 lanes each, 32 / (G/8) groups a step.
template <int G>
__global__ void __launch_bounds__(256) paged_append_kernel(const AppendArgs a) {
  constexpr int L = G / 8, USTEP = 32 / L;
  const int lane = threadIdx.x & 31, unit = lane / L, j = lane % L;
  const int64_t items = static_cast<int64_t>(a.rows) * a.kv.H;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t nwarps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
  const int64_t capacity = static_cast<int64_t>(a.kv.max_pages) * a.kv.ps;
  for (int64_t item = warp; item < items; item += nwarps) {
    const int r = static_cast<int>(item / a.kv.H), h = static_cast<int>(item - static_cast<int64_t>(r) * a.kv.H);
    const int s = r / a.rows_per_seq, i = r - s * a.rows_per_seq;
    const int pos = a.positions[s], count = a.counts ? a.counts[s] : a.rows_per_seq;
    if (pos < -1 || count < 0 || count > a.rows_per_seq) {
      if (lane == 0) atomicOr(a.kv.err, FG_DEVERR_RANGE);
      continue;
    }
    if (pos == -1 || i >= count) continue;
    const int64_t p = static_cast<int64_t>(pos) + i;
    const int64_t slot = p < capacity ? paged_slot(a.kv, s, h, static_cast<int>(p)) : -1;
    if (slot < 0) {
      if (lane == 0) atomicOr(a.kv.err, FG_DEVERR_RANGE);
      continue;
    }
    if (lane == 0) {
      if (a.kv.weights) a.kv.weights[slot] = 0.f;
      if (a.kv.tokens) a.kv.tokens[slot] = (a.first ? a.first[s] : pos) + i;
    }
    for (int u0 = 0; u0 < 2 * a.ng; u0 += USTEP) {  // warp-uniform
      const int u = u0 + unit, g = u >> 1;          // unit u: group u / 2 of k (even u) or v
      const bool live = u < 2 * a.ng;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (live)
        x = *reinterpret_cast<const uint4 *>(((u & 1) ? a.v : a.k) + static_cast<int64_t>(r) * a.ld +
                                             (static_cast<int64_t>(h) * a.ng + g) * G + j * 8);
      __half mn, sc;
      const uint32_t w = quant_group8<L>(x, mn, sc);
      if (!live) continue;
      reinterpret_cast<uint32_t *>((u & 1) ? a.kv.vc : a.kv.kc)[(slot * a.ng + g) * L + j] = w;
      if (j == 0) {
        ((u & 1) ? a.kv.vm : a.kv.km)[slot * a.ng + g] = mn;
        ((u & 1) ? a.kv.vs : a.kv.ks)[slot * a.ng + g] = sc;
      }
    }
  }
}

}  // namespace

extern "C" fg_status fg_paged_kv_bytes(int num_pages, int num_heads, int head_dim, int page_size, int group,
                                       size_t *codes_bytes, size_t *meta_bytes, size_t *track_bytes) {
  if (num_pages < 1 || num_heads < 1 || page_size < 1) return FG_ERR_INVALID;
  const int G = fg_kv_group(group);
  if (G == 0 || (head_dim != 64 && head_dim != 128 && head_dim != 256)) return FG_ERR_UNSUPPORTED;
  if (head_dim % G || page_size % 16) return FG_ERR_SHAPE;
  const size_t slots = static_cast<size_t>(num_pages) * num_heads * page_size;
  if (codes_bytes) *codes_bytes = slots * (head_dim / 2);
  if (meta_bytes) *meta_bytes = slots * (head_dim / G) * 2;
  if (track_bytes) *track_bytes = slots * 4;
  return FG_OK;
}

extern "C" fg_status fg_paged_kv_append(const fg_paged_kv *kv, const fg_half *k, const fg_half *v, int64_t ld,
                                        int rows, int rows_per_seq, const int32_t *positions,
                                        const int32_t *row_counts, const int32_t *first_tokens, void *stream) {
  fg_status rc = fg_paged_validate(kv);
  if (rc != FG_OK) return rc;
  if (rows < 0 || rows_per_seq < 1 || rows % rows_per_seq || rows / rows_per_seq > kv->num_seqs) return FG_ERR_SHAPE;
  if (rows == 0) return FG_OK;
  if (!k || !v || !positions || !fg_aligned16(k) || !fg_aligned16(v)) return FG_ERR_INVALID;
  if (ld < static_cast<int64_t>(kv->num_heads) * kv->head_dim || ld % 8) return FG_ERR_SHAPE;
  AppendArgs a;
  if (!fg_paged_args(kv, &a.kv)) return FG_ERR_CUDA;
  const int G = fg_kv_group(kv->group);
  a.k = reinterpret_cast<const __half *>(k);
  a.v = reinterpret_cast<const __half *>(v);
  a.ld = ld;
  a.rows = rows;
  a.rows_per_seq = rows_per_seq;
  a.ng = kv->head_dim / G;
  a.positions = positions;
  a.counts = row_counts;
  a.first = first_tokens;
  const int64_t blocks = (static_cast<int64_t>(rows) * kv->num_heads + 7) / 8, most = 8LL * fg_sm_count();
  const unsigned grid = static_cast<unsigned>(blocks < most ? blocks : most);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (G == 64) paged_append_kernel<64><<<grid, 256, 0, st>>>(a);
  else paged_append_kernel<128><<<grid, 256, 0, st>>>(a);
  return fg_launch_check();
}
