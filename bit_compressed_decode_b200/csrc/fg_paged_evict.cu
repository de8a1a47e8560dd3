// fg_paged_evict.cu -- eviction from the paged 4-bit KV cache by accumulated attention weight.
//
// Every (sequence, head) ranks its slots by a 32-bit key: the largest for a protected slot (one of
// the last `recent` tokens), else the weight's bits in an order-preserving form.  The budget-th
// largest key splits the slots into kept ones (above it), evicted ones (below) and ties, of which
// the lowest slots are kept.
#include "fg_paged.cuh"

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kProtected = 0xFFFFFFFFu;

struct EvictArgs {
  PagedArgs kv;
  const int32_t *lengths, *next;
  int32_t *new_lengths;
  float *wout;
  int32_t *tout;
  int budget, recent, limit, rb, mb;  // rb, mb: bytes of a slot's codes and of its mins (or scales)
};

// Unsigned order of the keys = order of the weights; NaN below everything, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint32_t slot_key(const EvictArgs &a, int64_t slot, int64_t since) {
  return a.kv.tokens[slot] >= since ? kProtected : weight_key(a.kv.weights[slot]);
}

__device__ __forceinline__ int block_sum(int v, int *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  int t = 0;
  for (int w = 0; w < kThreads / 32; w++) t += red[w];
  return t;
}

// Exclusive prefix count of `flag` over the block; *total: the count.
__device__ __forceinline__ int block_rank(bool flag, int *red, int *total) {
  const uint32_t b = __ballot_sync(0xffffffffu, flag);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 0) red[warp] = __popc(b);
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kThreads / 32; w++) {
    before += w < warp ? red[w] : 0;
    all += red[w];
  }
  *total = all;
  return before + __popc(b & ((1u << lane) - 1u));
}

__device__ __forceinline__ void copy_bytes(uint8_t *pool, int64_t dst, int64_t src, int bytes) {
  for (int i = 0; i < bytes; i += 2)
    *reinterpret_cast<uint16_t *>(pool + dst * bytes + i) = *reinterpret_cast<const uint16_t *>(pool + src * bytes + i);
}

// One CTA per (sequence, head).  The budget-th largest key by bisection on its 32 bits; then the
// holes below the budget and the kept slots at or above it are walked together, hole by hole.
__global__ void __launch_bounds__(kThreads) paged_evict_kernel(const EvictArgs a) {
  __shared__ int red[kThreads / 32];
  const int s = blockIdx.x / a.kv.H, h = blockIdx.x % a.kv.H, tid = threadIdx.x;
  const int n = a.lengths[s];
  const bool range = n < -1 || n > a.limit;
  int bad = 0;
  for (int p = tid * a.kv.ps; !range && p < n; p += kThreads * a.kv.ps) bad |= paged_slot(a.kv, s, h, p) < 0;
  bad = block_sum(bad, red);
  if ((range || bad) && tid == 0) atomicOr(a.kv.err, FG_DEVERR_RANGE);
  const bool skip = range || bad || n <= a.budget;
  if (h == 0 && tid == 0 && a.new_lengths != a.lengths) a.new_lengths[s] = skip ? n : a.budget;
  if (range || bad || n < 1) return;
  if (skip) {
    if (a.wout != a.kv.weights)
      for (int p = tid; p < n; p += kThreads) {
        const int64_t slot = paged_slot(a.kv, s, h, p);
        a.wout[slot] = a.kv.weights[slot];
      }
    if (a.tout != a.kv.tokens)
      for (int p = tid; p < n; p += kThreads) {
        const int64_t slot = paged_slot(a.kv, s, h, p);
        a.tout[slot] = a.kv.tokens[slot];
      }
    return;
  }
  const int64_t since = static_cast<int64_t>(a.next[s]) - a.recent;
  // the largest `key` that at least `budget` slots reach
  uint32_t key = 0;
  for (int bit = 31; bit >= 0; bit--) {
    const uint32_t trial = key | (1u << bit);
    int c = 0;
    for (int p = tid; p < n; p += kThreads) c += slot_key(a, paged_slot(a.kv, s, h, p), since) >= trial;
    if (block_sum(c, red) >= a.budget) key = trial;
  }
  int c = 0;
  for (int p = tid; p < n; p += kThreads) c += slot_key(a, paged_slot(a.kv, s, h, p), since) > key;
  const int ties = a.budget - block_sum(c, red);  // of the slots with this key, the first `ties` are kept
  int tie_base = 0;
  __shared__ int mover[kThreads], hole[kThreads];
  int next_mover = a.budget, movers = 0, used = 0;  // movers found in [budget, next_mover), not yet placed: movers - used
  int mover_ties = 0;
  // ties below the budget, needed to know which ties above it are kept
  for (int p0 = 0; p0 < a.budget; p0 += kThreads) {
    const int p = p0 + tid;
    mover_ties += block_sum(p < a.budget && slot_key(a, paged_slot(a.kv, s, h, p), since) == key, red);
  }
  for (int p0 = 0; p0 < a.budget; p0 += kThreads) {
    const int p = p0 + tid;
    const bool in = p < a.budget;
    const int64_t slot = in ? paged_slot(a.kv, s, h, p) : 0;
    const uint32_t k = in ? slot_key(a, slot, since) : 0u;
    int total;
    const int rank = tie_base + block_rank(in && k == key, red, &total);
    tie_base += total;
    const bool kept = in && (k > key || (k == key && rank < ties));
    const float w = in ? a.kv.weights[slot] : 0.f;
    const int32_t tk = in ? a.kv.tokens[slot] : 0;
    const int hr = block_rank(in && !kept, red, &total);
    __syncthreads();
    if (in && !kept) hole[hr] = p;
    const int holes = total;
    if (kept) {
      if (a.wout != a.kv.weights) a.wout[slot] = w;
      if (a.tout != a.kv.tokens) a.tout[slot] = tk;
    }
    // fill the chunk's holes with the next kept slots above the budget
    int filled = 0;
    while (filled < holes) {
      if (used == movers) {  // look through the next chunk above the budget
        if (next_mover >= n) break;  // (as many kept slots above the budget as holes below it)
        const int q = next_mover + tid;
        const bool qin = q < n;
        const uint32_t qk = qin ? slot_key(a, paged_slot(a.kv, s, h, q), since) : 0u;
        const int qrank = mover_ties + block_rank(qin && qk == key, red, &total);
        mover_ties += total;
        const bool qkept = qin && (qk > key || (qk == key && qrank < ties));
        const int mr = block_rank(qkept, red, &total);
        __syncthreads();
        if (qkept) mover[mr] = q;
        movers = total;
        used = 0;
        next_mover += kThreads;
        __syncthreads();
        continue;
      }
      const int take = min(holes - filled, movers - used);
      __syncthreads();
      if (tid < take) {
        const int64_t dst = paged_slot(a.kv, s, h, hole[filled + tid]), src = paged_slot(a.kv, s, h, mover[used + tid]);
        copy_bytes(a.kv.kc, dst, src, a.rb);
        copy_bytes(a.kv.vc, dst, src, a.rb);
        copy_bytes(reinterpret_cast<uint8_t *>(a.kv.km), dst, src, a.mb);
        copy_bytes(reinterpret_cast<uint8_t *>(a.kv.ks), dst, src, a.mb);
        copy_bytes(reinterpret_cast<uint8_t *>(a.kv.vm), dst, src, a.mb);
        copy_bytes(reinterpret_cast<uint8_t *>(a.kv.vs), dst, src, a.mb);
        a.wout[dst] = a.kv.weights[src];
        a.tout[dst] = a.kv.tokens[src];
      }
      filled += take;
      used += take;
    }
  }
}

// new_lengths given as lengths itself: written once every CTA has read its length.
__global__ void paged_new_lengths_kernel(int32_t *lengths, int seqs, const EvictArgs a) {
  const int s = blockIdx.x * blockDim.x + threadIdx.x;
  if (s >= seqs) return;
  const int n = lengths[s];
  if (n <= a.budget || n > a.limit) return;
  for (int p = 0; p < n; p += a.kv.ps)
    if (paged_slot(a.kv, s, 0, p) < 0) return;
  lengths[s] = a.budget;
}

}  // namespace

extern "C" size_t fg_paged_kv_evict_workspace_bytes(const fg_paged_kv *kv, int budget, int max_len) { return 0; }

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
  EvictArgs a;
  if (!fg_paged_args(kv, &a.kv)) return FG_ERR_CUDA;
  a.lengths = lengths;
  a.next = next_tokens;
  a.new_lengths = new_lengths;
  a.wout = weights_out ? weights_out : kv->weights;
  a.tout = tokens_out ? tokens_out : kv->tokens;
  a.budget = budget;
  a.recent = recent;
  a.limit = fg_paged_capacity(kv);
  if (max_len && max_len < a.limit) a.limit = max_len;
  a.rb = kv->head_dim / 2;
  a.mb = kv->head_dim / fg_kv_group(kv->group) * 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  paged_evict_kernel<<<static_cast<unsigned>(kv->num_seqs) * kv->num_heads, kThreads, 0, st>>>(a);
  if ((rc = fg_launch_check()) != FG_OK) return rc;
  if (new_lengths == lengths)
    paged_new_lengths_kernel<<<(kv->num_seqs + 127) / 128, 128, 0, st>>>(new_lengths, kv->num_seqs, a);
  return fg_launch_check();
}
