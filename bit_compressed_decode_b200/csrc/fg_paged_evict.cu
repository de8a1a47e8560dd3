// fg_paged_evict.cu -- eviction from the paged 4-bit KV cache by accumulated attention weight.
//
// Every (sequence, head) ranks its slots by a 32-bit key: the largest for a protected slot (one of
// the last `recent` tokens), else the weight's bits in an order-preserving form.  The budget-th
// largest key splits the slots into kept ones (above it), evicted ones (below) and ties, of which
// the lowest slots are kept.  Evicted slots below the budget are holes, kept ones at or above it
// movers; there are as many of the ones as of the others, and mover i goes into hole i.  Sources
// and destinations are disjoint, so the moves need no order and no second buffer.
//
// Bound: 8 bytes read per slot (and 8 written per kept one where the numbers go to other pools), and
// what moves, read and written once (144 + 8 bytes for heads of 128 in groups of 64).
//
// One CTA per (sequence, head).  Its slots' weights and tokens are read from memory once, 16 bytes
// of each at a time and several a thread in flight; the keys stay in shared memory (the `Wide` form,
// for more slots than fit there, reads them again instead).  A histogram of the keys' 11 leading bits
// names the bin of the budget-th; its few keys are ranked against one another, key then slot (a bin
// with more than kRanked keys is told apart by further bits first; equal keys beyond that are taken
// in slot order from a bit per slot).  Kept or not is a bit per slot, holes and movers are listed by
// prefix sums over the words.  What moves is read and written 16 bytes of codes at a time, several a
// thread in flight: the moves, a dependent load after a store, were half of the time before.
// Measured: 2048 items of 2049 to 2112 slots to 2048 in 38 us (87 MB, 2.3 TB/s: the latencies of
// the phases, one after the other); 128 items of 700 to 16384 slots to 1024 in 26 us; the Wide form,
// 16 items of 100000 slots to 4096, in 164 us (13 MB a pass over the numbers, several passes, an SM an
// item).
#include "fg_paged.cuh"

namespace {

constexpr uint32_t kProtected = 0xFFFFFFFFu;
constexpr int kBins = 2048;
constexpr int kRanked = 128;
constexpr size_t kSmem = 200 * 1024;  // shared memory of a CTA; more: the Wide form

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

// T threads, U vectors of 4 slots a thread in flight, B CTAs per SM.
template <int T, int U, int B, bool Wide>
__global__ void __launch_bounds__(T, B) paged_evict_kernel(const EvictArgs a) {
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
  __shared__ uint64_t cand[kRanked];  // the keys that are ranked one by one, with their slots
  __shared__ int cands;
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
  if (tid == 0) cands = 0;
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
  for (int q = 4 * tid; q < n; q += 4 * U * T) {
    float4 ws[U];
    int4 ts[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int p = q + 4 * u * T;
      if (p < n) {
        const int64_t slot = pool_slot(p);  // four slots of one page
        ws[u] = *reinterpret_cast<const float4 *>(a.kv.weights + slot);
        ts[u] = *reinterpret_cast<const int4 *>(a.kv.tokens + slot);
      }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int p = q + 4 * u * T;
      if (p >= n) break;
      const int64_t slot = wcopy || tcopy ? pool_slot(p) : 0;
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
  auto keys4 = [&](int p, uint32_t (&k)[4]) {  // of slots p .. p + 3 (p < n; those behind n: anything)
    if (!Wide) {
      const uint4 v = *reinterpret_cast<const uint4 *>(skeys + p);
      k[0] = v.x, k[1] = v.y, k[2] = v.z, k[3] = v.w;
    } else {
      const int64_t slot = pool_slot(p);
      const float4 w = *reinterpret_cast<const float4 *>(a.kv.weights + slot);
      const int4 t = *reinterpret_cast<const int4 *>(a.kv.tokens + slot);
      k[0] = slot_key(w.x, t.x, since), k[1] = slot_key(w.y, t.y, since);
      k[2] = slot_key(w.z, t.z, since), k[3] = slot_key(w.w, t.w, since);
    }
  };
  // The bin of `bins` from the top that holds the want-th key, into pick; all threads.
  auto select = [&](int bins, int want) {
    const int per = (bins + T - 1) / T, top = bins - 1 - tid * per;  // a thread's bins, from the top
    int sum = 0;
    for (int i = 0; i < per && top - i >= 0; i++) sum += hist[top - i];
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
        const int c = hist[top - i];
        if (before + c >= want) {
          pick[0] = top - i;
          pick[1] = want - before;
          break;
        }
        before += c;
      }
    }
    __syncthreads();
  };
  uint32_t prefix = 0;  // of the budget-th key: its leading bits so far
  int want = a.budget;   // which of the keys with them it is, from the largest
  select(kBins, want);
  prefix = static_cast<uint32_t>(pick[0]);
  want = pick[1];
  int left = hist[prefix], low = 21;  // keys with these leading bits; bits behind them
  // Few keys left are ranked against one another; more (a bin of near or equal weights) are told
  // apart by further bits first.
  const int words = (n + 31) / 32;
#pragma unroll 1
  while (left > kRanked && left > want && low > 0) {
    const int bits = low == 21 ? 11 : 10;
    low -= bits;
    __syncthreads();
    for (int i = tid; i < (1 << bits); i += T) hist[i] = 0;
    __syncthreads();
    for (int p = tid; p < n; p += T) {
      const uint32_t k = key_of(p);
      if (k >> (low + bits) == prefix) atomicAdd(&hist[(k >> low) & ((1u << bits) - 1u)], 1);
    }
    __syncthreads();
    select(1 << bits, want);
    left = hist[pick[0]];
    prefix = prefix << bits | static_cast<uint32_t>(pick[0]);
    want = pick[1];
  }

  // ---- the slots as bits, a word for 32: above the leading bits, and with them ----
  const bool all_ties = left == want;                      // all of the latter are kept
  const bool ranked = !all_ties && left <= kRanked;        // the first `want` by key, then slot
  const bool plain = all_ties || ranked;
  for (int p = 4 * tid; p - 4 * lane < words * 32; p += 4 * T) {  // four slots a lane, eight lanes a word
    uint32_t k[4] = {0u, 0u, 0u, 0u};
    if (p < n) keys4(p, k);
    uint32_t up = 0, same = 0;
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const uint32_t lead = k[e] >> low;
      const bool in = p + e < n;
      up |= in && lead > prefix ? 1u << e : 0u;
      same |= in && lead == prefix ? 1u << e : 0u;
    }
    if (ranked)
      for (uint32_t b = same; b; b &= b - 1) {  // (their order among themselves is of no matter)
        const int e = __ffs(b) - 1;
        const uint32_t key = e == 0 ? k[0] : e == 1 ? k[1] : e == 2 ? k[2] : k[3];
        cand[atomicAdd(&cands, 1)] = static_cast<uint64_t>(key) << 32 | ~static_cast<uint32_t>(p + e);
      }
    if (all_ties) up |= same;
    const uint32_t at = 4 * (lane & 7);
    up <<= at, same <<= at;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) up |= __shfl_xor_sync(0xffffffffu, up, o);
    if (!plain)
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) same |= __shfl_xor_sync(0xffffffffu, same, o);
    if ((lane & 7) == 0 && p < words * 32) {
      above[p / 32] = up;
      if (!plain) equal[p / 32] = same;
    }
  }
  __syncthreads();
  if (ranked) {
    if (tid < left) {
      const uint64_t mine = cand[tid];  // larger: a larger key, or the same and a lower slot
      int rank = 0;
#pragma unroll 8
      for (int i = 0; i < left; i++) rank += cand[i] > mine;
      const uint32_t p = ~static_cast<uint32_t>(mine);
      if (rank < want) atomicOr(&above[p / 32], 1u << (p & 31));
    }
    __syncthreads();
  }
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
    if (w < words) kept = above[w];
    if (!plain) {  // (block-uniform) equal keys: the lowest slots
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
    static_assert(32 * T < 65536, "holes and movers of T words in 16 bits each");
    int total;
    const int v = scan(__popc(hole) | __popc(mover) << 16, &total);  // both counts in one scan
    // the lists: the words in turn to the warps, a lane a bit (the histogram's place is free)
    if (w < words) {
      above[w] = mover;
      equal[w] = hole;
      hist[tid] = v;
    }
    __syncthreads();
    const uint32_t below = (1u << lane) - 1u;
    for (int i = warp; i < min(T, words - w0); i += W) {
      const uint32_t hw = equal[w0 + i], mw = above[w0 + i];
      if ((hw | mw) == 0) continue;
      const int p = 32 * (w0 + i) + lane;
      const unsigned at = hist[i];
      const int hx = hole0 + (at & 0xFFFF) + __popc(hw & below), mx = mover0 + (at >> 16) + __popc(mw & below);
      if (hw >> lane & 1u && hx < a.list) holes[hx] = p;
      if (mw >> lane & 1u && mx < a.list) movers[mx] = p;
    }
    __syncthreads();
    hole0 += total & 0xFFFF;
    mover0 += static_cast<unsigned>(total) >> 16;
  }
  const int moves = min(min(hole0, mover0), a.list);  // (as many of the ones as of the others)
  __syncthreads();

  // ---- the moves: 16 bytes of codes at a time, and one number at a time (array by array, so that
  //      neighbouring moves' numbers are neighbours); V and N of them in flight per thread ----
  constexpr int V = B > 1 ? 2 : 4, N = B > 1 ? 2 : 3;  // (many CTAs per SM: fewer registers)
  // kMoves of them at a time, so that their vectors and numbers are counted in 32 bits (what fits in
  // shared memory is less)
  constexpr int kMoves = 1 << 24;
  static_assert(kMoves * 16LL + 2 * V * T <= INT32_MAX && kMoves * 6LL + 2 * N * T <= INT32_MAX, "32-bit counters");
  const int cv = a.code_vecs;
  const int cs = cv == 2 ? 1 : cv == 4 ? 2 : 3;  // log2(cv)
  int m0 = 0;
  do {
    const int count = Wide ? min(moves - m0, kMoves) : moves, vecs = count * 2 * cv, nums = count * 6;
    const int *const hole = holes + m0, *const mover = movers + m0;
    for (int v0 = tid, n0 = tid; v0 < vecs || n0 < nums; v0 += V * T, n0 += N * T) {
      uint4 x[V];
      uint4 *to[V];
#pragma unroll
      for (int u = 0; u < V; u++) {
        const int v = v0 + u * T;
        if (v < vecs) {
          const int i = v >> (cs + 1), part = v & (2 * cv - 1);
          uint4 *const pool = reinterpret_cast<uint4 *>(part >= cv ? a.kv.vc : a.kv.kc) + (part & (cv - 1));
          to[u] = pool + pool_slot(hole[i]) * cv;
          x[u] = pool[pool_slot(mover[i]) * cv];
        }
      }
      uint2 y[N];
      void *dst[N];
#pragma unroll
      for (int u = 0; u < N; u++) {
        const int k = n0 + u * T;
        if (k < nums) {
          const int arr = k / count, i = k - arr * count;
          const int64_t src = pool_slot(mover[i]), d = pool_slot(hole[i]);
          if (arr < 4) {
            uint8_t *const b = reinterpret_cast<uint8_t *>(arr == 0   ? a.kv.km
                                                           : arr == 1 ? a.kv.ks
                                                           : arr == 2 ? a.kv.vm
                                                                      : a.kv.vs);
            dst[u] = b + d * a.meta;
            if (a.meta == 4) y[u].x = *reinterpret_cast<const uint32_t *>(b + src * 4);
            else if (a.meta == 2) y[u].x = *reinterpret_cast<const uint16_t *>(b + src * 2);
            else y[u] = *reinterpret_cast<const uint2 *>(b + src * 8);
          } else if (arr == 4) {
            dst[u] = a.wout + d;
            y[u].x = __float_as_uint(a.kv.weights[src]);
          } else {
            dst[u] = a.tout + d;
            y[u].x = static_cast<uint32_t>(a.kv.tokens[src]);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < V; u++)
        if (v0 + u * T < vecs) *to[u] = x[u];
#pragma unroll
      for (int u = 0; u < N; u++) {
        const int k = n0 + u * T;
        if (k < nums) {
          const int meta = k < 4 * count ? a.meta : 4;
          if (meta == 4) *static_cast<uint32_t *>(dst[u]) = y[u].x;
          else if (meta == 2) *static_cast<uint16_t *>(dst[u]) = static_cast<uint16_t>(y[u].x);
          else *static_cast<uint2 *>(dst[u]) = y[u];
        }
      }
    }
    m0 += kMoves;
  } while (Wide && m0 < moves);
}

// new_lengths given as lengths itself: written once every CTA has read its length.
__global__ void paged_new_lengths_kernel(int32_t *lengths, int seqs, const EvictArgs a) {
  const int s = blockIdx.x, n = lengths[s];
  bool bad = n <= a.budget || n > a.limit;
  // (page by page, not slot by slot: a page may have 2^30 slots)
  const int pages = bad ? 0 : (n + a.kv.ps - 1) / a.kv.ps;
  for (int i = threadIdx.x; i < pages; i += blockDim.x) {
    const int page = a.kv.table[static_cast<int64_t>(s) * a.kv.max_pages + i];
    bad |= page < 0 || page >= a.kv.num_pages;
  }
  if (!__syncthreads_or(bad) && threadIdx.x == 0) lengths[s] = a.budget;
}

// Two arrays of n numbers have memory in common.
bool overlap(const int32_t *a, const int32_t *b, int n) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b), size = 4 * static_cast<uintptr_t>(n);
  return x < y + size && y < x + size;
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
  p.wide = need > kSmem;
  p.smem = p.wide ? kBins * 4 : need;
  p.lists = p.wide ? static_cast<size_t>(kv->num_seqs) * kv->num_heads * lists : 0;
  const int64_t items = static_cast<int64_t>(kv->num_seqs) * kv->num_heads;
  // long items have an SM each (16384 slots: 27 us, 45 with 192 threads); many items are throughput:
  // 192 threads, eight CTAs per SM (2048 items of 2100 slots: 38 us; 41 with six, whose third wave is
  // a third full, 58 with 256 threads)
  p.threads = limit > 4096 ? 1024 : items >= 8LL * fg_sm_count() ? 192 : 256;
  return p;
}

template <int T, int U, int B, bool Wide>
fg_status launch(const EvictArgs &a, const EvictPlan &p, unsigned grid, cudaStream_t st) {
  static bool done[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (!Wide && dev >= 0 && dev < 64 && !done[dev]) {
    const fg_status rc = fg_cuda_check(cudaFuncSetAttribute(
        paged_evict_kernel<T, U, B, Wide>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem)));
    if (rc != FG_OK) return rc;
    done[dev] = true;
  }
  paged_evict_kernel<T, U, B, Wide><<<grid, T, p.smem, st>>>(a);
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
  // (one head's CTA writes a sequence's new length while the others may not have read their inputs)
  if (new_lengths != lengths && (overlap(new_lengths, lengths, kv->num_seqs) || overlap(new_lengths, next_tokens, kv->num_seqs)))
    return FG_ERR_INVALID;
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
  if (p.wide) rc = launch<1024, 4, 1, true>(a, p, grid, st);
  else if (p.threads == 1024) rc = launch<1024, 4, 1, false>(a, p, grid, st);
  else if (p.threads == 192) rc = launch<192, 3, 8, false>(a, p, grid, st);
  else rc = launch<256, 4, 1, false>(a, p, grid, st);
  if (rc != FG_OK || new_lengths != lengths) return rc;
  paged_new_lengths_kernel<<<kv->num_seqs, 128, 0, st>>>(new_lengths, kv->num_seqs, a);
  return fg_launch_check();
}
