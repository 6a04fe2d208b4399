// cache_evict.cu -- eviction from the paged latent cache by accumulated weight.
//
// A sequence of L > budget keys keeps its last `recent` keys and the budget -
// recent others with the largest weights (equal weights: the lowest index),
// compacted in place into logical slots [0, budget) in their old order.
//
// evict_select_kernel: one CTA per sequence.  Four 8-bit radix passes over
// the order-preserving image of the weights give the smallest kept image T
// and how many keys equal to T are kept; a pass in index order then writes the
// kept list by prefix sums.
// evict_move_kernel: a kept key never moves up (list entry i is >= i), so
// walking the list upwards in batches, each read before it is written, is safe
// in place.  Keys depend on each other only through their own bytes, so a CTA
// takes one 128-byte column of every key of a sequence.
#include "latent.h"

namespace dsa {

namespace {
constexpr int ES_THREADS = 1024;
constexpr int EM_THREADS = 256;
constexpr int EM_UNROLL = 8;
constexpr int EM_BATCH = EM_THREADS / 8 * EM_UNROLL;  // keys per batch: 8 lanes x 16 bytes per key

// Order-preserving image; every NaN counts as the largest weight.
__device__ __forceinline__ uint32_t weight_key(float w) {
  return w != w ? 0xffffffffu : ordered_key(w);
}

// Exclusive prefix sum of x over the CTA and the total (tmp: 33 ints).
__device__ __forceinline__ int block_scan(int x, int* tmp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();
  if (lane == 31) tmp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int s = tmp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    tmp[lane] = s;
  }
  __syncthreads();
  *total = tmp[31];
  return v - x + (warp ? tmp[warp - 1] : 0);
}
}  // namespace

__global__ void __launch_bounds__(ES_THREADS) evict_select_kernel(const EvictParams p) {
  pdl_enter();
  __shared__ int hist[256], pick[3], tmp[32];
  const int b = blockIdx.x, tid = threadIdx.x;
  int L = p.seq_lens[b];
  if (L < 0 || L > (int64_t)p.max_pages * PAGE) {
    if (tid == 0) atomicOr(&p.status->now, ST_RANGE);
    L = 0;
  }
  __syncthreads();  // every thread has its length: new_lens may be seq_lens
  if (L > p.budget)  // the pages the move reads and writes
    for (int i = tid; i < ceil_div(L, PAGE); i += ES_THREADS) {
      const int page = p.block_table[(int64_t)b * p.max_pages + i];
      if (page < 0 || page >= p.num_pages) atomicOr(&p.status->now, ST_RANGE);
    }
  const int n = min(L, p.budget);
  int32_t* kept = p.kept + (int64_t)b * p.budget;
  for (int i = n + tid; i < p.budget; i += ES_THREADS) kept[i] = -1;
  if (L <= p.budget) {
    for (int i = tid; i < n; i += ES_THREADS) kept[i] = i;
  } else {
    const float* w = p.weights + (int64_t)b * p.ld_weights;
    const int need = p.budget - p.recent, cand = L - p.recent;
    for (int i = tid; i < p.recent; i += ES_THREADS) kept[need + i] = cand + i;
    if (need > 0) {
      uint32_t prefix = 0;
      int rem = need;  // rank of the last kept key among those that share the prefix
      for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int i = tid; i < cand; i += ES_THREADS) {
          const uint32_t k = weight_key(w[i]);
          if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid < 32) radix_pick_digit(hist, rem, pick);
        __syncthreads();
        prefix |= (uint32_t)pick[0] << shift;
        rem = pick[1];
        __syncthreads();
      }
      int base = 0, ties = 0;  // kept so far, equal keys so far
      for (int i0 = 0; i0 < cand; i0 += ES_THREADS) {
        const int i = i0 + tid;
        const uint32_t k = i < cand ? weight_key(w[i]) : 0;
        const bool eq = i < cand && k == prefix;
        int n_eq, n_keep;
        const int before = block_scan(eq, tmp, &n_eq);
        const bool keep = i < cand && (k > prefix || (eq && ties + before < rem));
        const int at = block_scan(keep, tmp, &n_keep);
        if (keep) kept[base + at] = i;
        base += n_keep;
        ties += n_eq;
      }
    }
  }
  if (tid == 0) {
    p.old_lens[b] = L;
    p.new_lens[b] = n;
  }
}

// blockIdx.x: column of 128 bytes: 0-7 ckv, 8 kpe, 9 weights (and key scales), 10 indexer keys.
__global__ void __launch_bounds__(EM_THREADS) evict_move_kernel(const EvictParams p) {
  pdl_enter();
  const int b = blockIdx.y, col = blockIdx.x, tid = threadIdx.x;
  if (b == 0 && col == 0 && tid == 0) {  // the call's last kernel
    p.status->last = p.status->now;
    p.status->now = 0;
  }
  const int L = p.old_lens[b], n = min(L, p.budget);
  if (L <= p.budget) return;
  const int32_t* kept = p.kept + (int64_t)b * p.budget;
  const int32_t* table = p.block_table + (int64_t)b * p.max_pages;
  auto slot = [&](int s) -> int64_t {
    const int page = table[s / PAGE];
    return page >= 0 && page < p.num_pages ? (int64_t)page * PAGE + s % PAGE : -1;  // (reported by the selection)
  };
  if (col == 9) {
    float* w = p.weights + (int64_t)b * p.ld_weights;
    for (int i0 = 0; i0 < n; i0 += EM_THREADS) {
      const int i = i0 + tid;
      float x = 0.f, y = 0.f;
      int64_t to = -1, from = -1;
      if (i < n) {
        const int k = kept[i];
        x = w[k];
        if (p.k_scale) {
          to = slot(i);
          from = slot(k);
          if (to >= 0 && from >= 0) y = p.k_scale[from];
        }
      }
      __syncthreads();
      if (i < n) w[i] = x;
      if (to >= 0 && from >= 0) p.k_scale[to] = y;
    }
    __syncthreads();
    for (int i = n + tid; i < L; i += EM_THREADS) w[i] = 0.f;
    return;
  }
  uint8_t* base = col < 8 ? p.ckv + 128 * col : col == 8 ? p.kpe : p.k_cache;
  const int64_t stride = col < 8 ? p.ckv_stride : col == 8 ? p.kpe_stride : 128;
  const int lane8 = tid & 7;
  for (int i0 = 0; i0 < n; i0 += EM_BATCH) {
    uint4 v[EM_UNROLL];
    int64_t to[EM_UNROLL];
#pragma unroll
    for (int j = 0; j < EM_UNROLL; ++j) {
      const int i = i0 + j * (EM_THREADS / 8) + (tid >> 3);
      to[j] = -1;
      if (i < n) {
        const int k = kept[i];
        if (k != i) {
          const int64_t from = slot(k);
          to[j] = slot(i);
          if (from < 0) to[j] = -1;
          if (to[j] >= 0) v[j] = *reinterpret_cast<const uint4*>(base + from * stride + 16 * lane8);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < EM_UNROLL; ++j)
      if (to[j] >= 0) *reinterpret_cast<uint4*>(base + to[j] * stride + 16 * lane8) = v[j];
  }
}

cudaError_t launch_evict(const EvictParams& p, cudaStream_t s) {
  count_launch();
  cudaError_t e = launch_pdl(evict_select_kernel, dim3(p.B), dim3(ES_THREADS), 0, s, p);
  if (e != cudaSuccess) return e;
  count_launch();
  return launch_pdl(evict_move_kernel, dim3(p.k_cache ? 11 : 10, p.B), dim3(EM_THREADS), 0, s, p);
}

}  // namespace dsa
