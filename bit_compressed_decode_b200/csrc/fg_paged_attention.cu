// fg_paged_attention.cu -- softmax attention of query rows over the paged 4-bit KV cache, and the
// accumulation of its probabilities in the slots' weights.
#include <math.h>

#include "fg_paged.cuh"

namespace {

constexpr int kThreads = 128;

struct PagedAttnArgs {
  PagedArgs kv;
  const __half *q;
  int64_t ldq;
  __half *out;
  int64_t ldo;
  int R, rows_per_seq, limit, accumulate;
  const int32_t *positions, *counts;
};

__device__ __forceinline__ float block_max(float v, float *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = red[0];
  for (int w = 1; w < kThreads / 32; w++) t = fmaxf(t, red[w]);
  return t;
}

__device__ __forceinline__ float block_sum(float v, float *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = red[0];
  for (int w = 1; w < kThreads / 32; w++) t += red[w];
  return t;
}

// One CTA per (sequence, key-value head); its rows and query heads one after the other.  A thread
// takes a slot's score, then a head dim's sum; the running maximum and sum follow 128-slot chunks.
template <int D, int G>
__global__ void __launch_bounds__(kThreads) paged_attn_kernel(const PagedAttnArgs a) {
  constexpr int NG = D / G;
  __shared__ float q[D], p[kThreads], red[kThreads / 32];
  __shared__ int64_t slots[kThreads];
  __shared__ int bad;
  const int s = blockIdx.x / a.kv.H, h = blockIdx.x % a.kv.H, tid = threadIdx.x;
  const int pos = a.positions[s], count = a.counts ? a.counts[s] : a.rows_per_seq;
  const bool range = pos < -1 || count < 0 || count > a.rows_per_seq ||
                     (pos >= 0 && static_cast<int64_t>(pos) + count > a.limit);
  if (range && tid == 0) atomicOr(a.kv.err, FG_DEVERR_RANGE);
  const int live = range || pos < 0 ? 0 : count;

  auto score = [&](int64_t slot) {
    float t = 0.f;
    for (int g = 0; g < NG; g++) {
      float dot = 0.f, sum = 0.f;
      for (int i = 0; i < G / 2; i++) {
        const uint32_t b = a.kv.kc[slot * (D / 2) + g * (G / 2) + i];
        dot += q[g * G + 2 * i] * static_cast<float>(b & 15u) + q[g * G + 2 * i + 1] * static_cast<float>(b >> 4);
        sum += q[g * G + 2 * i] + q[g * G + 2 * i + 1];
      }
      t += __half2float(a.kv.km[slot * NG + g]) * sum + __half2float(a.kv.ks[slot * NG + g]) * dot;
    }
    return t;
  };

  for (int i = 0; i < a.rows_per_seq; i++) {
    for (int j = 0; j < a.R; j++) {
      const int64_t r = static_cast<int64_t>(s) * a.rows_per_seq + i;
      const int hq = h * a.R + j;
      __half *out = a.out + r * a.ldo + hq * D;
      __syncthreads();
      if (tid == 0) bad = 0;
      for (int d = tid; d < D; d += kThreads) q[d] = __half2float(a.q[r * a.ldq + hq * D + d]);
      __syncthreads();
      const int L = i < live ? pos + i + 1 : 0;
      float m = -INFINITY, l = 0.f, o[(D + kThreads - 1) / kThreads] = {0.f};
      for (int t0 = 0; t0 < L; t0 += kThreads) {
        const int t = t0 + tid, n = min(kThreads, L - t0);
        float sc = -INFINITY;
        if (t < L) {
          slots[tid] = paged_slot(a.kv, s, h, t);
          if (slots[tid] < 0) bad = 1;
          else sc = score(slots[tid]);
        }
        const float mc = block_max(sc, red);  // (its barriers also publish slots and bad)
        if (bad) break;
        const float mn = fmaxf(m, mc), alpha = expf(m - mn);
        p[tid] = t < L ? expf(sc - mn) : 0.f;
        l = l * alpha + block_sum(p[tid], red);
        m = mn;
        for (int e = 0; e * kThreads + tid < D; e++) {
          const int d = e * kThreads + tid;
          float acc = o[e] * alpha;
          for (int x = 0; x < n; x++) {
            const uint32_t b = a.kv.vc[slots[x] * (D / 2) + d / 2];
            const float c = static_cast<float>(d & 1 ? b >> 4 : b & 15u);
            acc += p[x] * (__half2float(a.kv.vm[slots[x] * NG + d / G]) + c * __half2float(a.kv.vs[slots[x] * NG + d / G]));
          }
          o[e] = acc;
        }
        __syncthreads();
      }
      if (bad && tid == 0) atomicOr(a.kv.err, FG_DEVERR_RANGE);
      for (int e = 0; e * kThreads + tid < D; e++)
        out[e * kThreads + tid] = __float2half_rn(L > 0 && !bad ? o[e] / l : 0.f);
      if (a.accumulate && !bad)
        for (int t = tid; t < L; t += kThreads) {
          const int64_t slot = paged_slot(a.kv, s, h, t);
          a.kv.weights[slot] += expf(score(slot) - m) / l;
        }
    }
  }
}

template <int D, int G>
fg_status launch(const PagedAttnArgs &a, int seqs, cudaStream_t st) {
  paged_attn_kernel<D, G><<<static_cast<unsigned>(seqs) * a.kv.H, kThreads, 0, st>>>(a);
  return fg_launch_check();
}

}  // namespace

extern "C" size_t fg_paged_attention_workspace_bytes(const fg_paged_kv *kv, int num_q_heads, int rows, int rows_per_seq,
                                                     int max_len, int accumulate) {
  return 0;
}

extern "C" fg_status fg_paged_attention(const fg_paged_kv *kv, const fg_half *q, int64_t ldq, int num_q_heads,
                                        fg_half *out, int64_t ldo, int rows, int rows_per_seq,
                                        const int32_t *positions, const int32_t *row_counts, int max_len,
                                        int accumulate, void *workspace, size_t workspace_bytes, void *stream) {
  fg_status rc = fg_paged_validate(kv);
  if (rc != FG_OK) return rc;
  if (num_q_heads < 1 || num_q_heads % kv->num_heads) return FG_ERR_SHAPE;
  if (rows < 0 || rows_per_seq < 1 || rows % rows_per_seq || rows / rows_per_seq > kv->num_seqs) return FG_ERR_SHAPE;
  if (max_len < 0 || (accumulate != 0 && accumulate != 1)) return FG_ERR_INVALID;
  if (accumulate && !kv->weights) return FG_ERR_INVALID;
  if (rows == 0) return FG_OK;
  if (!q || !out || !positions || !fg_aligned16(q) || !fg_aligned16(out) || !fg_aligned16(workspace))
    return FG_ERR_INVALID;
  const int64_t hD = static_cast<int64_t>(num_q_heads) * kv->head_dim;
  if (ldq < hD || ldo < hD || ldq % 8 || ldo % 8) return FG_ERR_SHAPE;
  const int seqs = rows / rows_per_seq;
  if (static_cast<int64_t>(seqs) * kv->num_heads > INT32_MAX) return FG_ERR_SHAPE;
  PagedAttnArgs a;
  if (!fg_paged_args(kv, &a.kv)) return FG_ERR_CUDA;
  a.q = reinterpret_cast<const __half *>(q);
  a.ldq = ldq;
  a.out = reinterpret_cast<__half *>(out);
  a.ldo = ldo;
  a.R = num_q_heads / kv->num_heads;
  a.rows_per_seq = rows_per_seq;
  a.limit = fg_paged_capacity(kv);
  if (max_len && max_len < a.limit) a.limit = max_len;
  a.accumulate = accumulate;
  a.positions = positions;
  a.counts = row_counts;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (fg_kv_group(kv->group) == 64) {
    switch (kv->head_dim) {
      case 64: return launch<64, 64>(a, seqs, st);
      case 128: return launch<128, 64>(a, seqs, st);
      case 256: return launch<256, 64>(a, seqs, st);
    }
  } else {
    switch (kv->head_dim) {
      case 128: return launch<128, 128>(a, seqs, st);
      case 256: return launch<256, 128>(a, seqs, st);
    }
  }
  return FG_ERR_UNSUPPORTED;
}
