// fg_paged_evict.cu -- eviction from the paged 4-bit KV cache by accumulated attention weight.
//
// Every (sequence, head) ranks its slots by a 32-bit key: the largest for a protected slot (one of
// the last `recent` tokens), else the weight's bits in an order-preserving form.  The budget-th
// largest key splits the slots into kept ones (above it), evicted ones (below) and ties, of which
// the lowest slots are kept.  Evicted slots below the budget are holes, kept ones at or above it
// movers; there are as many of the ones as of the others, and mover i goes into hole i.  Sources
// and destinations are disjoint, so the moves need no order and no second buffer.
//
// One CTA per (sequence, head).  Its slots' weights and tokens are read from memory once, 16 bytes
// of each at a time; the keys stay in shared memory (the `Wide` form, for more slots than fit
// there, reads them again instead).  The budget-th key is found by a radix selection of 11, 11 and
// 10 bits; the ranks of ties, holes and movers come from a bit per slot (ballots) and prefix sums over
// the words.  What moves is read and written by 16 lanes
// per slot, 16 bytes of codes a lane.
#include "fg_paged.cuh"

namespace {

constexpr uint32_t kProtected = 0xFFFFFFFFu;
constexpr int kBins = 2048;
#ifndef FG_EVICT_SMEM
#define FG_EVICT_SMEM (200 * 1024)
#endif
#ifndef FG_EVICT_LONG
#define FG_EVICT_LONG 4096
#endif

struct EvictArgs {
  PagedArgs kv;
  const int32_t *lengths, *next;
  int32_t *new_lengths;
  float *wout;
  int32_t *tout;
  int *lists;  // Wide: [items][2 * list + 2 * words]
  int budget, recent, limit;
  int keys, pages, list, words;  // capacities: slots (a multiple of 4), pages, holes or movers, 32 slots
  int code_vecs, meta;    // 16-byte vectors of a slot's codes; bytes of its mins (or scales): 2, 4 or 8
};

// Unsigned order of the keys = order of the weights; NaN below everything, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint32_t slot_key(float w, int token, int64_t since) {
  return token >= since ? kProtected : weight_key(w);
}

// Sum of the first `warp` of W numbers in shared memory, and of all of them; a whole warp calls it.
template <int W>
__device__ __forceinline__ int sum_before(const int *red, int warp, int lane, int *all) {
  const int v = lane < W ? red[lane] : 0;
  int before = lane < warp ? v : 0, sum = v;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  *all = sum;
  return before;
}

template <int T, bool Wide>
__global__ void __launch_bounds__(T) paged_evict_kernel(const EvictArgs a) {
  constexpr int W = T / 32;
  extern __shared__ __align__(16) int sm[];
  int *const hist = sm;
  uint32_t *const skeys = reinterpret_cast<uint32_t *>(sm + kBins);
  int *const spages = sm + kBins + (Wide ? 0 : a.keys);
  int *const holes = Wide ? a.lists + static_cast<int64_t>(blockIdx.x) * 2 * (a.list + a.words) : spages + a.pages;
  int *const movers = holes + a.list;
  uint32_t *const above = reinterpret_cast<uint32_t *>(movers + a.list);  // a bit per slot
  uint32_t *const equal = above + a.words;
  __shared__ int red[W];
  __shared__ int pick[2];  // the bin that the budget-th key lies in; keys still wanted from it

  const int s = blockIdx.x / a.kv.H, h = blockIdx.x % a.kv.H;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = a.lengths[s];
  const bool range = n < -1 || n > a.limit;
  const int32_t *const table = a.kv.table + static_cast<int64_t>(s) * a.kv.max_pages;
  bool bad = false;
  if (!range && n > 0)
    for (int i = tid; i < (n + a.kv.ps - 1) / a.kv.ps; i += T) {
      const int page = table[i];
      bad |= page < 0 || page >= a.kv.num_pages;
      if (!Wide) spages[i] = page;
    }
  for (int i = tid; i < kBins; i += T) hist[i] = 0;
  bad = __syncthreads_or(bad);
  if ((range || bad) && tid == 0) atomicOr(a.kv.err, FG_DEVERR_RANGE);
  const bool evicts = !range && !bad && n > a.budget;
  if (h == 0 && tid == 0 && a.new_lengths != a.lengths) a.new_lengths[s] = evicts ? a.budget : n;
  if (range || bad || n < 1) return;

  auto pool_slot = [&](int p) -> int64_t {
    const int i = paged_index(a.kv, p);
    const int page = Wide ? table[i] : spages[i];
    return (static_cast<int64_t>(page) * a.kv.H + h) * a.kv.ps + (p - i * a.kv.ps);
  };
  const int64_t since = static_cast<int64_t>(a.next[s]) - a.recent;
  const int keep = evicts ? a.budget : n;
  const bool wcopy = a.wout != a.kv.weights, tcopy = a.tout != a.kv.tokens;
  if (!evicts && !wcopy && !tcopy) return;

  // ---- every slot once: its key, the selection's first histogram, and the numbers of the slots
  //      below the budget into their new pools (the holes' are written over below) ----
  constexpr int U = 4;  // loads in flight: four slots each
  for (int q = 4 * tid; q < n; q += 4 * U * T) {
    int64_t slots[U];
    float4 ws[U];
    int4 ts[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int p = q + 4 * u * T;
      if (p < n) {
        slots[u] = pool_slot(p);  // four slots of one page
        ws[u] = *reinterpret_cast<const float4 *>(a.kv.weights + slots[u]);
        ts[u] = *reinterpret_cast<const int4 *>(a.kv.tokens + slots[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int p = q + 4 * u * T;
      if (p >= n) break;
      const int64_t slot = slots[u];
      const float4 w = ws[u];
      const int4 t = ts[u];
      if (evicts) {
        const uint32_t k[4] = {slot_key(w.x, t.x, since), slot_key(w.y, t.y, since), slot_key(w.z, t.z, since),
                               slot_key(w.w, t.w, since)};
        if (!Wide) *reinterpret_cast<uint4 *>(skeys + p) = make_uint4(k[0], k[1], k[2], k[3]);
#pragma unroll
        for (int e = 0; e < 4; e++)
          if (p + e < n) atomicAdd(&hist[k[e] >> 21], 1);
      }
      if (p + 3 < keep) {
        if (wcopy) *reinterpret_cast<float4 *>(a.wout + slot) = w;
        if (tcopy) *reinterpret_cast<int4 *>(a.tout + slot) = t;
      } else if (p < keep) {
        if (wcopy) {
          a.wout[slot] = w.x;
          if (p + 1 < keep) a.wout[slot + 1] = w.y;
          if (p + 2 < keep) a.wout[slot + 2] = w.z;
        }
        if (tcopy) {
          a.tout[slot] = t.x;
          if (p + 1 < keep) a.tout[slot + 1] = t.y;
          if (p + 2 < keep) a.tout[slot + 2] = t.z;
        }
      }
    }
  }
  if (!evicts) return;
  __syncthreads();

  auto key_of = [&](int p) -> uint32_t {
    if (!Wide) return skeys[p];
    const int64_t slot = pool_slot(p);
    return slot_key(a.kv.weights[slot], a.kv.tokens[slot], since);
  };
  // The bin of `bins` from the top that holds the want-th key, into pick; all threads.
  auto select = [&](int bins, int want) {
    const int per = bins / T > 0 ? bins / T : 1;  // bins of a thread, from the top
    int sum = 0;
    if (tid * per < bins)
      for (int i = 0; i < per; i++) sum += hist[bins - 1 - tid * per - i];
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) red[warp] = incl;
    __syncthreads();
    int all;
    int before = incl - sum + sum_before<W>(red, warp, lane, &all);
    if (before < want && before + sum >= want) {  // (one thread)
      for (int i = 0; i < per; i++) {
        const int b = bins - 1 - tid * per - i, c = hist[b];
        if (before + c >= want) {
          pick[0] = b;
          pick[1] = want - before;
          break;
        }
        before += c;
      }
    }
    __syncthreads();
  };
  uint32_t prefix = 0;
  int want = a.budget;
  select(kBins, want);
  prefix = static_cast<uint32_t>(pick[0]);
  want = pick[1];
#pragma unroll
  for (int pass = 1; pass < 3; pass++) {
    const int low = pass == 1 ? 10 : 0, bits = pass == 1 ? 11 : 10;
    for (int i = tid; i < (1 << bits); i += T) hist[i] = 0;
    __syncthreads();
    for (int p = tid; p < n; p += T) {
      const uint32_t k = key_of(p);
      if (k >> (low + bits) == prefix) atomicAdd(&hist[(k >> low) & ((1u << bits) - 1u)], 1);
    }
    __syncthreads();
    select(1 << bits, want);
    prefix = prefix << bits | static_cast<uint32_t>(pick[0]);
    want = pick[1];
  }
  const uint32_t key = prefix;  // of the slots with this key, the first `want` are kept

  const bool all_ties = hist[key & 1023u] == want;

  // ---- the slots as bits, a word for 32: above the key, and with it ----
  const int words = (n + 31) / 32;
  for (int p = tid; p < words * 32; p += T) {
    const uint32_t k = p < n ? key_of(p) : 0u;
    const uint32_t over = __ballot_sync(0xffffffffu, p < n && k > key), same = __ballot_sync(0xffffffffu, p < n && k == key);
    if (lane == 0) {
      above[p / 32] = over;
      equal[p / 32] = same;
    }
  }
  __syncthreads();
  // the kept ones: ties in order until enough
  auto scan = [&](int v, int *total) -> int {  // exclusive prefix sum over the CTA's threads
    int incl = v, sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) red[warp] = incl;
    __syncthreads();
    const int before = sum_before<W>(red, warp, lane, &sum);
    __syncthreads();
    *total = sum;
    return before + incl - v;
  };
  int tie0 = 0, hole0 = 0, mover0 = 0;
  for (int w0 = 0; w0 < words; w0 += T) {
    const int w = w0 + tid;
    uint32_t kept = 0, hole = 0, mover = 0;
    if (w < words) kept = above[w] | (all_ties ? equal[w] : 0u);
    if (!all_ties) {  // (block-uniform)
      const uint32_t same = w < words ? equal[w] : 0u;
      int total;
      int left = want - tie0 - scan(__popc(same), &total);  // ties this word may still keep
      for (uint32_t b = same; b && left > 0; b &= b - 1, left--) kept |= b & (0u - b);
      tie0 += total;
    }
    if (w < words) {
      const int low = a.budget - 32 * w;  // bits of the word below the budget
      const uint32_t mask = low >= 32 ? 0xFFFFFFFFu : low <= 0 ? 0u : (1u << low) - 1u;
      hole = ~kept & mask;  // (the budget is below n: all of these are slots)
      mover = kept & ~mask;
    }
    int th, tm;
    int hi = hole0 + scan(__popc(hole), &th), mi = mover0 + scan(__popc(mover), &tm);
    for (; hole; hole &= hole - 1, hi++)
      if (hi < a.list) holes[hi] = 32 * w + __ffs(hole) - 1;
    for (; mover; mover &= mover - 1, mi++)
      if (mi < a.list) movers[mi] = 32 * w + __ffs(mover) - 1;
    hole0 += th;
    mover0 += tm;
  }
  const int moves = min(min(hole0, mover0), a.list);  // (as many of the ones as of the others)
  __syncthreads();

  // ---- the moves: 16 lanes per slot, M slots of each in flight.  Lanes 0 .. 7 (0 .. 3 for head dim
  //      64) take 16 bytes of codes, half of them k's (twice for head dim 256), lanes 8 .. 11 the
  //      group numbers, 12 the weight, 13 the token ----
  constexpr int M = 4;
  const int l16 = tid & 15, cv = a.code_vecs;
  const bool codes = l16 < 8 && l16 < 2 * cv, second = codes && cv == 8;
  const bool of_v = l16 >= (cv == 8 ? 4 : cv);
  uint4 *const cpool = reinterpret_cast<uint4 *>(of_v ? a.kv.vc : a.kv.kc) + (of_v ? l16 - (cv == 8 ? 4 : cv) : l16);
  __half *const mpool = l16 == 8 ? a.kv.km : l16 == 9 ? a.kv.ks : l16 == 10 ? a.kv.vm : a.kv.vs;
  const bool nums = l16 >= 8 && l16 < 12, track = l16 == 12 || l16 == 13;
  const uint32_t *const tsrc = l16 == 12 ? reinterpret_cast<const uint32_t *>(a.kv.weights)
                                         : reinterpret_cast<const uint32_t *>(a.kv.tokens);
  uint32_t *const tdst = l16 == 12 ? reinterpret_cast<uint32_t *>(a.wout) : reinterpret_cast<uint32_t *>(a.tout);
  for (int i0 = tid / 16; i0 < moves; i0 += M * (T / 16)) {
    int64_t dst[M];
    uint4 x[M], y[M];
#pragma unroll
    for (int u = 0; u < M; u++) {
      const int i = i0 + u * (T / 16);
      if (i >= moves) break;
      const int64_t src = pool_slot(movers[i]);
      dst[u] = pool_slot(holes[i]);
      if (codes) x[u] = cpool[src * cv];
      if (second) y[u] = cpool[src * cv + 4];
      if (nums) {
        if (a.meta == 4) x[u].x = reinterpret_cast<const uint32_t *>(mpool)[src];
        else if (a.meta == 2) x[u].x = reinterpret_cast<const uint16_t *>(mpool)[src];
        else *reinterpret_cast<uint2 *>(&x[u]) = reinterpret_cast<const uint2 *>(mpool)[src];
      }
      if (track) x[u].x = tsrc[src];
    }
#pragma unroll
    for (int u = 0; u < M; u++) {
      if (i0 + u * (T / 16) >= moves) break;
      if (codes) cpool[dst[u] * cv] = x[u];
      if (second) cpool[dst[u] * cv + 4] = y[u];
      if (nums) {
        if (a.meta == 4) reinterpret_cast<uint32_t *>(mpool)[dst[u]] = x[u].x;
        else if (a.meta == 2) reinterpret_cast<uint16_t *>(mpool)[dst[u]] = static_cast<uint16_t>(x[u].x);
        else reinterpret_cast<uint2 *>(mpool)[dst[u]] = *reinterpret_cast<const uint2 *>(&x[u]);
      }
      if (track) tdst[dst[u]] = x[u].x;
    }
  }
}

// new_lengths given as lengths itself: written once every CTA has read its length.
__global__ void paged_new_lengths_kernel(int32_t *lengths, int seqs, const EvictArgs a) {
  const int s = blockIdx.x, n = lengths[s];
  bool bad = n <= a.budget || n > a.limit;
  for (int p = threadIdx.x * a.kv.ps; !bad && p < n; p += blockDim.x * a.kv.ps) bad = paged_slot(a.kv, s, 0, p) < 0;
  if (!__syncthreads_or(bad) && threadIdx.x == 0) lengths[s] = a.budget;
}

struct EvictPlan {
  bool wide;
  int threads, keys, pages, list, words;
  size_t smem, lists;
};

EvictPlan evict_plan(const fg_paged_kv *kv, int budget, int max_len) {
  EvictPlan p;
  const int cap = fg_paged_capacity(kv), limit = max_len && max_len < cap ? max_len : cap;
  p.keys = (limit + 3) / 4 * 4;
  p.pages = (limit + kv->page_size - 1) / kv->page_size;
  const int over = limit > budget ? limit - budget : 0;
  p.list = over < budget ? over : budget;
  p.words = (limit + 31) / 32;
  const size_t lists = 2 * (static_cast<size_t>(p.list) + p.words) * 4;
  const size_t need = (static_cast<size_t>(kBins) + p.keys + p.pages) * 4 + lists;
  p.wide = need > FG_EVICT_SMEM;
  p.smem = p.wide ? kBins * 4 : need;
  p.lists = p.wide ? static_cast<size_t>(kv->num_seqs) * kv->num_heads * lists : 0;
  p.threads = limit > FG_EVICT_LONG ? 1024 : 256;
  return p;
}

template <int T, bool Wide>
fg_status launch(const EvictArgs &a, const EvictPlan &p, unsigned grid, cudaStream_t st) {
  static bool done[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (!Wide && dev >= 0 && dev < 64 && !done[dev]) {
    const fg_status rc = fg_cuda_check(cudaFuncSetAttribute(paged_evict_kernel<T, Wide>,
                                                            cudaFuncAttributeMaxDynamicSharedMemorySize, FG_EVICT_SMEM));
    if (rc != FG_OK) return rc;
    done[dev] = true;
  }
  paged_evict_kernel<T, Wide><<<grid, T, p.smem, st>>>(a);
  return fg_launch_check();
}

}  // namespace

extern "C" size_t fg_paged_kv_evict_workspace_bytes(const fg_paged_kv *kv, int budget, int max_len) {
  if (fg_paged_validate(kv) != FG_OK || budget < 1 || max_len < 0) return 0;
  return evict_plan(kv, budget, max_len).lists;
}

extern "C" fg_status fg_paged_kv_evict(const fg_paged_kv *kv, const int32_t *lengths, const int32_t *next_tokens,
                                       int budget, int recent, int max_len, int32_t *new_lengths, float *weights_out,
                                       int32_t *tokens_out, void *workspace, size_t workspace_bytes, void *stream) {
  fg_status rc = fg_paged_validate(kv);
  if (rc != FG_OK) return rc;
  if (!kv->weights || !kv->tokens) return FG_ERR_INVALID;
  if (budget < 1 || recent < 0 || recent > budget || max_len < 0) return FG_ERR_INVALID;
  if (kv->num_seqs == 0) return FG_OK;
  if (!lengths || !next_tokens || !new_lengths || !fg_aligned16(workspace)) return FG_ERR_INVALID;
  if (!fg_aligned16(weights_out) || !fg_aligned16(tokens_out)) return FG_ERR_INVALID;
  if (static_cast<int64_t>(kv->num_seqs) * kv->num_heads > INT32_MAX) return FG_ERR_SHAPE;
  const EvictPlan p = evict_plan(kv, budget, max_len);
  if (p.lists > (workspace ? workspace_bytes : 0)) return FG_ERR_WORKSPACE;
  EvictArgs a;
  if (!fg_paged_args(kv, &a.kv)) return FG_ERR_CUDA;
  a.lengths = lengths;
  a.next = next_tokens;
  a.new_lengths = new_lengths;
  a.wout = weights_out ? weights_out : kv->weights;
  a.tout = tokens_out ? tokens_out : kv->tokens;
  a.lists = static_cast<int *>(workspace);
  a.budget = budget;
  a.recent = recent;
  a.limit = fg_paged_capacity(kv);
  if (max_len && max_len < a.limit) a.limit = max_len;
  a.keys = p.keys;
  a.pages = p.pages;
  a.list = p.list;
  a.words = p.words;
  a.code_vecs = kv->head_dim / 32;
  a.meta = kv->head_dim / fg_kv_group(kv->group) * 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(kv->num_seqs) * kv->num_heads;
  if (p.wide) rc = launch<1024, true>(a, p, grid, st);
  else if (p.threads == 1024) rc = launch<1024, false>(a, p, grid, st);
  else rc = launch<256, false>(a, p, grid, st);
  if (rc != FG_OK || new_lengths != lengths) return rc;
  paged_new_lengths_kernel<<<kv->num_seqs, 128, 0, st>>>(new_lengths, kv->num_seqs, a);
  return fg_launch_check();
}
