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
// 10 bits; then every warp takes a run of consecutive slots and the ranks of ties, holes and movers
// come from ballots and one prefix sum over the warps.  What moves is read and written by 16 lanes
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
  int *lists;  // Wide: [items][2][list]
  int budget, recent, limit;
  int keys, pages, list;  // capacities: slots (a multiple of 4), pages, holes or movers
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

template <int T, bool Wide>
__global__ void __launch_bounds__(T) paged_evict_kernel(const EvictArgs a) {
  constexpr int W = T / 32;
  extern __shared__ __align__(16) int sm[];
  int *const hist = sm;
  uint32_t *const skeys = reinterpret_cast<uint32_t *>(sm + kBins);
  int *const spages = sm + kBins + (Wide ? 0 : a.keys);
  int *const holes = Wide ? a.lists + static_cast<int64_t>(blockIdx.x) * 2 * a.list : spages + a.pages;
  int *const movers = holes + a.list;
  __shared__ int red[2][W];
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
    const int i = p / a.kv.ps;
    const int page = Wide ? table[i] : spages[i];
    return (static_cast<int64_t>(page) * a.kv.H + h) * a.kv.ps + (p - i * a.kv.ps);
  };
  const int64_t since = static_cast<int64_t>(a.next[s]) - a.recent;
  const int keep = evicts ? a.budget : n;
  const bool wcopy = a.wout != a.kv.weights, tcopy = a.tout != a.kv.tokens;
  if (!evicts && !wcopy && !tcopy) return;

  // ---- every slot once: its key, the selection's first histogram, and the numbers of the slots
  //      below the budget into their new pools (the holes' are written over below) ----
  for (int p = 4 * tid; p < n; p += 4 * T) {
    const int64_t slot = pool_slot(p);  // four slots of one page
    const float4 w = *reinterpret_cast<const float4 *>(a.kv.weights + slot);
    const int4 t = *reinterpret_cast<const int4 *>(a.kv.tokens + slot);
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
    if (lane == 31) red[0][warp] = incl;
    __syncthreads();
    int before = incl - sum;
    for (int w = 0; w < warp; w++) before += red[0][w];
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

  // ---- ranks: warp w has the slots w * run .. (w + 1) * run - 1 ----
  const int run = ((n + W - 1) / W + 31) / 32 * 32;
  const int p0 = min(n, warp * run), p1 = min(n, p0 + run);
  const uint32_t below = (1u << lane) - 1u;
  int ties = 0;
  for (int p = p0 + lane; p - lane < p1; p += 32)
    ties += __popc(__ballot_sync(0xffffffffu, p < p1 && key_of(p) == key));
  if (lane == 0) red[0][warp] = ties;
  __syncthreads();
  int tie0 = 0;
  for (int w = 0; w < warp; w++) tie0 += red[0][w];
  __syncthreads();
  auto walk = [&](bool write, int hole, int mover, int *holes_found, int *movers_found) {
    int tie = tie0;
    for (int p = p0 + lane; p - lane < p1; p += 32) {
      const uint32_t k = p < p1 ? key_of(p) : 0u;
      const bool eq = p < p1 && k == key;
      const uint32_t eqs = __ballot_sync(0xffffffffu, eq);
      const bool kept = p < p1 && (k > key || (eq && tie + __popc(eqs & below) < want));
      tie += __popc(eqs);
      const uint32_t hs = __ballot_sync(0xffffffffu, p < p1 && !kept && p < a.budget);
      const uint32_t ms = __ballot_sync(0xffffffffu, kept && p >= a.budget);
      if (write) {
        const int hi = hole + __popc(hs & below), mi = mover + __popc(ms & below);
        if (hs >> lane & 1u && hi < a.list) holes[hi] = p;
        if (ms >> lane & 1u && mi < a.list) movers[mi] = p;
      }
      hole += __popc(hs);
      mover += __popc(ms);
    }
    *holes_found = hole;
    *movers_found = mover;
  };
  int hn, mn;
  walk(false, 0, 0, &hn, &mn);
  if (lane == 0) {
    red[0][warp] = hn;
    red[1][warp] = mn;
  }
  __syncthreads();
  int h0 = 0, m0 = 0, moves = 0;
  for (int w = 0; w < W; w++) {
    h0 += w < warp ? red[0][w] : 0;
    m0 += w < warp ? red[1][w] : 0;
    moves += red[0][w];
  }
  moves = min(moves, a.list);  // (as many movers as holes)
  if (moves == 0) return;
  walk(true, h0, m0, &hn, &mn);
  __syncthreads();

  // ---- the moves: 16 lanes per slot; lane 0 .. 2 code_vecs - 1 a vector of codes of k or v (twice
  //      16 of them for head dim 256 in turn), then the four group numbers, the weight, the token ----
  const int l16 = tid & 15;
  for (int i = tid / 16; i < moves; i += T / 16) {
    const int64_t dst = pool_slot(holes[i]), src = pool_slot(movers[i]);
    const int units = 2 * a.code_vecs + 6;
    for (int u = l16; u < units; u += 16) {
      if (u < 2 * a.code_vecs) {
        const bool v = u >= a.code_vecs;
        uint4 *const pool = reinterpret_cast<uint4 *>(v ? a.kv.vc : a.kv.kc);
        const int x = v ? u - a.code_vecs : u;
        pool[dst * a.code_vecs + x] = pool[src * a.code_vecs + x];
      } else {
        const int x = u - 2 * a.code_vecs;
        if (x < 4) {
          __half *const pool = x == 0 ? a.kv.km : x == 1 ? a.kv.ks : x == 2 ? a.kv.vm : a.kv.vs;
          uint8_t *const b = reinterpret_cast<uint8_t *>(pool);
          if (a.meta == 4) {
            *reinterpret_cast<uint32_t *>(b + dst * 4) = *reinterpret_cast<const uint32_t *>(b + src * 4);
          } else if (a.meta == 2) {
            *reinterpret_cast<uint16_t *>(b + dst * 2) = *reinterpret_cast<const uint16_t *>(b + src * 2);
          } else {
            *reinterpret_cast<uint2 *>(b + dst * 8) = *reinterpret_cast<const uint2 *>(b + src * 8);
          }
        } else if (x == 4) {
          a.wout[dst] = a.kv.weights[src];
        } else {
          a.tout[dst] = a.kv.tokens[src];
        }
      }
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
  int threads, keys, pages, list;
  size_t smem, lists;
};

EvictPlan evict_plan(const fg_paged_kv *kv, int budget, int max_len) {
  EvictPlan p;
  const int cap = fg_paged_capacity(kv), limit = max_len && max_len < cap ? max_len : cap;
  p.keys = (limit + 3) / 4 * 4;
  p.pages = (limit + kv->page_size - 1) / kv->page_size;
  const int over = limit > budget ? limit - budget : 0;
  p.list = over < budget ? over : budget;
  const size_t need = (static_cast<size_t>(kBins) + p.keys + p.pages + 2 * static_cast<size_t>(p.list)) * 4;
  p.wide = need > FG_EVICT_SMEM;
  p.smem = p.wide ? kBins * 4 : need;
  p.lists = p.wide ? static_cast<size_t>(kv->num_seqs) * kv->num_heads * 2 * p.list * 4 : 0;
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
