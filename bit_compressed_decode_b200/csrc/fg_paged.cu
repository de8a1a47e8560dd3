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
  if (static_cast<int64_t>(kv->max_pages) * kv->page_size > (1 << 30)) return FG_ERR_SHAPE;
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
  int rows, rows_per_seq;
  const int32_t *positions, *counts, *first;
};

// A warp takes R consecutive rows of one head: a row's k and v are D/4 lanes of 8 values, all R rows
// are loaded before the first is quantised, and the codes of consecutive slots of a page are
// consecutive in the pool.  The group numbers (2 to 8 bytes of a row and array) go through shared
// memory, so that a lane stores a row's of one array and the warp stores whole sectors where the
// rows are a prompt's.  Bound: 4 D bytes read and D + 8 D/G written per row and head; what it spends
// is instructions, 83 % of the issue slots: the quantiser's fp32 steps, which alone run at 0.77 of a
// copy's rate, and its own slots, shuffles and divisions, with no next tile's loads in flight behind
// them.  32 prompts of up to 512 tokens, 56 heads of 128, 315 MB in 95 to 103 us, 3.3 to 3.0 TB/s (a
// warp per row and head: 217 us).
template <int D>
struct Append {
  static constexpr int R = D == 256 ? 4 : 8;       // rows per warp
  static constexpr int STEPS = R * (D / 4) / 32;   // 32 lanes of 8 values each
};

template <int D, int G>
__global__ void __launch_bounds__(256) paged_append_kernel(const AppendArgs a) {
  constexpr int L = G / 8, NG = D / G, R = Append<D>::R, STEPS = Append<D>::STEPS, ROW = D / 4;  // ROW: lanes of a row
  __shared__ __align__(8) __half nums[8][4][R][NG];  // [warp][k min, k scale, v min, v scale]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t tile = static_cast<int64_t>(blockIdx.x) * 8 + warp;
  const int64_t block = tile / a.kv.H;  // heads of the same rows are neighbours
  const int h = static_cast<int>(tile - block * a.kv.H);
  if (block * R >= a.rows) return;
  const int r0 = static_cast<int>(block) * R;
  // lane i < R: where row r0 + i goes (-1: nowhere)
  int64_t slot = -1;
  int token = 0;
  if (lane < R && r0 + lane < a.rows) {
    const int r = r0 + lane, s = r / a.rows_per_seq, i = r - s * a.rows_per_seq;
    const int pos = a.positions[s], count = a.counts ? a.counts[s] : a.rows_per_seq;
    const bool range = pos < -1 || count < 0 || count > a.rows_per_seq;
    if (!range && pos >= 0 && i < count) {
      const int64_t p = static_cast<int64_t>(pos) + i;
      if (p < static_cast<int64_t>(a.kv.max_pages) * a.kv.ps) slot = paged_slot(a.kv, s, h, static_cast<int>(p));
      if (slot < 0) atomicOr(a.kv.err, FG_DEVERR_RANGE);
      token = (a.first ? a.first[s] : pos) + i;
    }
    if (range) atomicOr(a.kv.err, FG_DEVERR_RANGE);
  }
  if (__ballot_sync(0xffffffffu, slot >= 0) == 0) return;
  if (slot >= 0) {
    if (a.kv.weights) a.kv.weights[slot] = 0.f;
    if (a.kv.tokens) a.kv.tokens[slot] = token;
  }
  // step st, lane: value vector e = (32 st + lane) % ROW of row (32 st + lane) / ROW; k, then v
  constexpr int PER = STEPS > R ? STEPS / R : 1;  // steps of a row
  uint4 x[STEPS];
  int64_t to[STEPS / PER];
  const int e0 = lane % ROW;
  const __half *const ksrc = a.k + static_cast<int64_t>(r0) * a.ld + static_cast<int64_t>(h) * D;
  const __half *const vsrc = a.v + static_cast<int64_t>(r0) * a.ld + static_cast<int64_t>(h) * D;
#pragma unroll
  for (int st = 0; st < STEPS; st++) {
    const int row = (32 * st + lane) / ROW, e = PER == 1 ? e0 : (32 * st + lane) % ROW;
    if (st % PER == 0) to[st / PER] = __shfl_sync(0xffffffffu, slot, row);
    x[st] = make_uint4(0, 0, 0, 0);
    if (to[st / PER] >= 0)
      x[st] = __ldcs(reinterpret_cast<const uint4 *>((e < D / 8 ? ksrc : vsrc) + row * a.ld + (e % (D / 8)) * 8));
  }
#pragma unroll
  for (int st = 0; st < STEPS; st++) {
    const int row = (32 * st + lane) / ROW, e = PER == 1 ? e0 : (32 * st + lane) % ROW, w8 = e % (D / 8);
    const bool of_v = e >= D / 8;
    __half mn, sc;
    const uint32_t w = quant_group8<L>(x[st], mn, sc);
    if (to[st / PER] >= 0)
      reinterpret_cast<uint32_t *>(of_v ? a.kv.vc : a.kv.kc)[to[st / PER] * (D / 8) + w8] = w;
    if (w8 % L == 0) {
      nums[warp][of_v ? 2 : 0][row][w8 / L] = mn;
      nums[warp][of_v ? 3 : 1][row][w8 / L] = sc;
    }
  }
  __syncwarp();
  const int arr = lane / R, row = lane % R;
  const int64_t mine = __shfl_sync(0xffffffffu, slot, row);
  if (arr < 4 && mine >= 0) {
    __half *const pool = arr == 0 ? a.kv.km : arr == 1 ? a.kv.ks : arr == 2 ? a.kv.vm : a.kv.vs;
    const __half *const src = nums[warp][arr][row];
    if constexpr (NG == 1) pool[mine] = src[0];
    else if constexpr (NG == 2) reinterpret_cast<uint32_t *>(pool)[mine] = *reinterpret_cast<const uint32_t *>(src);
    else reinterpret_cast<uint2 *>(pool)[mine] = *reinterpret_cast<const uint2 *>(src);
  }
}

template <int D, int G>
fg_status append(const AppendArgs &a, cudaStream_t st) {
  constexpr int R = Append<D>::R;
  const int64_t tiles = (static_cast<int64_t>(a.rows) + R - 1) / R * a.kv.H, grid = (tiles + 7) / 8;
  if (grid > INT32_MAX) return FG_ERR_SHAPE;
  paged_append_kernel<D, G><<<static_cast<unsigned>(grid), 256, 0, st>>>(a);
  return fg_launch_check();
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
  a.positions = positions;
  a.counts = row_counts;
  a.first = first_tokens;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (G == 64) {
    switch (kv->head_dim) {
      case 64: return append<64, 64>(a, st);
      case 128: return append<128, 64>(a, st);
      case 256: return append<256, 64>(a, st);
    }
  } else {
    switch (kv->head_dim) {
      case 128: return append<128, 128>(a, st);
      case 256: return append<256, 128>(a, st);
    }
  }
  return FG_ERR_UNSUPPORTED;
}
