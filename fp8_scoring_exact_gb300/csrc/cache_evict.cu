// cache_evict.cu -- eviction from the paged latent cache by accumulated weight.
//
// A sequence of L > budget keys keeps its last `recent` keys and the budget -
// recent others with the largest weights (equal weights: the lowest index),
// compacted in place into logical slots [0, budget) in their old order.
//
// evict_select_kernel: one to eight CTAs per sequence (a cluster), each with a
// contiguous slice of its weights in shared memory as order-preserving 32-bit
// images.  The CTAs double while each would have more than 16K keys: the
// cluster's barriers cost more than they save below (eviction of 64 sequences of
// up to 32K keys: 154 us with 1 CTA each, 148 with 2, 156 with 4, 193 with 8; of
// five of up to 128K: 195, 122, 80, 70).
// Four 8-bit radix passes (histograms summed over the cluster) give the
// smallest kept image T and how many keys equal to T are kept; a last pass
// counts kept keys per warp segment, and the prefix sums over warps and CTAs
// place the kept list in index order.
//
// evict_move_kernel: bound by the moved bytes, 2 x 1152 per kept key (2 x 132
// more with the indexer's cache).  A CTA takes 64 entries of a kept list, reads
// their keys into registers, says so in a flag, and writes them to slots [64
// c, 64 c + 64) once the entries that live in those slots have been read.  A
// kept key never moves up (entry i is >= i), so those belong to this chunk or
// lower ones: their flags, found by two searches in the list.  Chunks are
// handed out in order and each reads before it waits, so the wait ends.  One that
// runs out all the same leaves its slots alone and is reported.
//
// With every kept key moving: 64 sequences of up to 32768 keys to 4096, the
// indexer's keys along (656 MB): 148 us, 25 of them the selection; the move's 122
// are 5.3 TB/s, 332 MB read from DRAM and 279 written.  Five of up to 131072 to
// 16384 (191 MB): 70 us, 28 of them the selection on 40 SMs: four passes over 16K
// images per CTA, and the cluster's barriers between them; 42 the move.  One of
// 3000 keys to 2048: 12 + 8 us, all latency.  Where hardly a key changes its place
// (the same weights and lengths again: some 13% and 6% of them) 77 and 45 us: the move
// then takes 57 and 24, for the most part the dependent loads that a chunk
// starts with (its number, the old length, two searches in the list).
#include "latent.h"

namespace dsa {

namespace {
constexpr int ES_THREADS = 1024;
constexpr int ES_WARPS = ES_THREADS / 32;
constexpr int ES_COPIES = 32;              // histogram copies, one per lane: most weights share a few exponents
constexpr int EM_THREADS = 256;
constexpr int EM_KEYS = EVICT_CHUNK;       // kept keys per CTA

// Order-preserving image; every NaN counts as the largest weight.
__device__ __forceinline__ uint32_t weight_key(float w) { return w != w ? 0xffffffffu : ordered_key(w); }

template <int CS>
__device__ __forceinline__ void cluster_barrier() {
  if constexpr (CS > 1) cluster_sync_all();
  else __syncthreads();
}
template <int CS>
__device__ __forceinline__ int cluster_read(const int* p, int rank) {
  if constexpr (CS > 1) return ld_dsmem(p, rank);
  else return *p;
}
}  // namespace

template <int CS>
__global__ void __launch_bounds__(ES_THREADS) evict_select_kernel(const EvictParams p) {
  pdl_enter();
  extern __shared__ uint32_t s_key[];      // [p.cached] images of the slice
  __shared__ int s_copy[ES_COPIES][256 + 1], s_hist[2][256], s_all[256], pick[3];
  __shared__ int s_gt[ES_WARPS], s_eq[ES_WARPS], s_tot[2];
  const int b = blockIdx.x / CS, rank = CS > 1 ? (int)cluster_ctarank() : 0;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int L = p.seq_lens[b];
  if (L < 0 || L > (int64_t)p.max_pages * PAGE) {
    if (tid == 0) atomicOr(&p.status->now, ST_RANGE);
    L = 0;
  }
  // (new_lens may be seq_lens: it is written where every thread has its length,
  // or with the same length)
  if constexpr (CS == 1) __syncthreads();
  const int n = min(L, p.budget), all = CS * ES_THREADS, me = rank * ES_THREADS + tid;
  int32_t* kept = p.kept + (int64_t)b * p.budget;
  float* new_w = p.new_w + (int64_t)b * p.budget;
  const float* w = p.weights + (int64_t)b * p.ld_weights;
  for (int i = n + me; i < p.budget; i += all) kept[i] = -1;
  for (int i = me; i < p.chunks; i += all) p.flags[(int64_t)b * p.chunks + i] = 0;
  if (me == 0) {
    p.old_lens[b] = L;
    if (b == 0) {
      *p.ticket = 0;
      p.status->last = 0;  // the move kernel's CTAs add to it in any order
    }
  }
  if (L <= p.budget) {  // (the same in the whole cluster)
    for (int i = me; i < n; i += all) kept[i] = i;
    if (me == 0) p.new_lens[b] = n;
    return;
  }
  // the pages that the move reads and writes
  for (int i = me; i < ceil_div(L, PAGE); i += all) {
    const int page = p.block_table[(int64_t)b * p.max_pages + i];
    if (page < 0 || page >= p.num_pages) atomicOr(&p.status->now, ST_RANGE);
  }
  const int need = p.budget - p.recent, cand = L - p.recent;
  for (int i = me; i < p.recent; i += all) {
    kept[need + i] = cand + i;
    new_w[need + i] = w[cand + i];
  }
  if (need == 0) {
    cluster_barrier<CS>();
    if (me == 0) p.new_lens[b] = n;
    return;
  }
  // this CTA's slice [lo, hi); what exceeds the cached part is read again
  const int per = ceil_div(ceil_div(cand, CS), 32) * 32;
  const int lo = min(cand, rank * per), hi = min(cand, lo + per), cached = min(hi, lo + p.cached);
  auto key = [&](int i) { return i < cached ? s_key[i - lo] : weight_key(w[i]); };
  uint32_t prefix = 0;
  int rem = need;  // rank of the last kept key among those that share the prefix
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    for (int i = tid; i < ES_COPIES * 257; i += ES_THREADS) (&s_copy[0][0])[i] = 0;
    __syncthreads();
    for (int i = lo + tid; i < hi; i += ES_THREADS) {
      uint32_t k;
      if (pass == 0) {
        k = weight_key(w[i]);
        if (i < cached) s_key[i - lo] = k;
      } else {
        k = key(i);
      }
      if (pass == 0 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&s_copy[lane][(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid < 256) {
      int x = 0;
#pragma unroll
      for (int c = 0; c < ES_COPIES; ++c) x += s_copy[c][tid];
      s_hist[pass & 1][tid] = x;
    }
    cluster_barrier<CS>();  // (two buffers: the pass after the next is behind another barrier)
    if (tid < 256) {
      int x = 0;
#pragma unroll
      for (int r = 0; r < CS; ++r) x += cluster_read<CS>(&s_hist[pass & 1][tid], r);
      s_all[tid] = x;
    }
    __syncthreads();
    if (warp == 0) radix_pick_digit(s_all, rem, pick);
    __syncthreads();
    prefix |= (uint32_t)pick[0] << shift;
    rem = pick[1];
  }
  // keys above and equal to the threshold per warp segment, warp and CTA
  const int seg = ceil_div(ceil_div(max(0, hi - lo), ES_WARPS), 32) * 32;
  const int s0 = min(hi, lo + warp * seg), s1 = min(hi, s0 + seg);
  int gt = 0, eq = 0;
  for (int i0 = s0; i0 < s1; i0 += 32) {
    const uint32_t k = i0 + lane < s1 ? key(i0 + lane) : 0;
    gt += __popc(__ballot_sync(0xffffffffu, i0 + lane < s1 && k > prefix));
    eq += __popc(__ballot_sync(0xffffffffu, i0 + lane < s1 && k == prefix));
  }
  if (lane == 0) {
    s_gt[warp] = gt;
    s_eq[warp] = eq;
  }
  __syncthreads();
  int gt0 = 0, eq0 = 0, gt1 = 0, eq1 = 0;  // before this warp in the CTA, and in the CTA
#pragma unroll
  for (int i = 0; i < ES_WARPS; ++i) {
    gt0 += i < warp ? s_gt[i] : 0;
    eq0 += i < warp ? s_eq[i] : 0;
    gt1 += s_gt[i];
    eq1 += s_eq[i];
  }
  if (tid == 0) {
    s_tot[0] = gt1;
    s_tot[1] = eq1;
  }
  cluster_barrier<CS>();
  for (int r = 0; r < rank; ++r) {
    gt0 += cluster_read<CS>(&s_tot[0], r);
    eq0 += cluster_read<CS>(&s_tot[1], r);
  }
  const uint32_t lt = lanemask_lt();
  for (int i0 = s0; i0 < s1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < s1 ? key(i) : 0;
    const bool is_gt = i < s1 && k > prefix, is_eq = i < s1 && k == prefix;
    const uint32_t mg = __ballot_sync(0xffffffffu, is_gt), me_ = __ballot_sync(0xffffffffu, is_eq);
    const int e = eq0 + __popc(me_ & lt);  // equal keys before this one
    if (is_gt || (is_eq && e < rem)) {
      const int at = gt0 + __popc(mg & lt) + min(e, rem);
      kept[at] = i;
      new_w[at] = w[i];
    }
    gt0 += __popc(mg);
    eq0 += __popc(me_);
  }
  cluster_barrier<CS>();  // nobody leaves while its counts may be read
  if (me == 0) p.new_lens[b] = n;
}

__global__ void __launch_bounds__(EM_THREADS) evict_move_kernel(const EvictParams p) {
  pdl_enter();
  __shared__ int s_from[EM_KEYS], s_to[EM_KEYS], s_job[3];  // slots (-1: stays, or a page outside the cache)
  const int tid = threadIdx.x;
  if (tid == 0) s_job[0] = atomicAdd(p.ticket, 1);
  __syncthreads();
  const int b = s_job[0] / p.chunks, c = s_job[0] % p.chunks;
  // the call's last kernel: what the selection found, beside what the waits below report
  if (s_job[0] == 0 && tid == 0) atomicOr(&p.status->last, atomicExch(&p.status->now, 0));
  const int L = p.old_lens[b], n = p.budget;
  if (L <= n) return;
  const int i0 = c * EM_KEYS, i1 = min(n, i0 + EM_KEYS);
  const int32_t* kept = p.kept + (int64_t)b * p.budget;
  const int32_t* table = p.block_table + (int64_t)b * p.max_pages;
  auto slot = [&](int s) {
    const int page = table[s / PAGE];
    return page >= 0 && page < p.num_pages ? page * PAGE + s % PAGE : -1;
  };
  bool moves = false;
  if (tid < EM_KEYS) {
    int from = -1, to = -1;
    if (i0 + tid < i1) {
      const int k = kept[i0 + tid];
      if (k != i0 + tid) {
        from = slot(k);
        to = slot(i0 + tid);
      }
    }
    moves = from >= 0 && to >= 0;
    s_from[tid] = moves ? from : -1;
    s_to[tid] = to;
  } else if (tid >= EM_THREADS - 2) {
    // entries of the list that live in the slots written here: [s_job[1], s_job[2])
    const int limit = tid == EM_THREADS - 2 ? i0 : i1;
    int x = 0, y = i1;  // kept[i] >= i, so none of them lies past i1
    while (x < y) {
      const int mid = (x + y) >> 1;
      if (kept[mid] < limit) x = mid + 1;
      else y = mid;
    }
    s_job[1 + (tid - (EM_THREADS - 2))] = x;
  }
  // the weights: compacted by the selection, the rest of the old length 0
  float* w = p.weights + (int64_t)b * p.ld_weights;
  const float* new_w = p.new_w + (int64_t)b * p.budget;
  if (i0 + tid < i1) w[i0 + tid] = new_w[i0 + tid];
  const int strip = ceil_div(L - n, p.chunks);
  for (int i = n + c * strip + tid; i < min(L, n + (c + 1) * strip); i += EM_THREADS) w[i] = 0.f;
  const bool any = __syncthreads_or(moves);
  uint4 v[EM_KEYS * 64 / EM_THREADS], e[EM_KEYS * 8 / EM_THREADS], x[EM_KEYS * 8 / EM_THREADS];
  float scale = 0.f;
  if (any) {
#pragma unroll
    for (int j = 0; j < EM_KEYS * 64 / EM_THREADS; ++j) {
      const int k = (j * EM_THREADS + tid) >> 6;
      if (s_from[k] >= 0) v[j] = *reinterpret_cast<const uint4*>(p.ckv + (int64_t)s_from[k] * p.ckv_stride + 16 * (tid & 63));
    }
#pragma unroll
    for (int j = 0; j < EM_KEYS * 8 / EM_THREADS; ++j) {
      const int k = (j * EM_THREADS + tid) >> 3;
      if (s_from[k] >= 0) {
        e[j] = *reinterpret_cast<const uint4*>(p.kpe + (int64_t)s_from[k] * p.kpe_stride + 16 * (tid & 7));
        if (p.k_cache) x[j] = *reinterpret_cast<const uint4*>(p.k_cache + (int64_t)s_from[k] * 128 + 16 * (tid & 7));
      }
    }
    if (p.k_cache && tid < EM_KEYS && s_from[tid] >= 0) scale = p.k_scale[s_from[tid]];
  }
  // read: publish, then wait for the lower chunks whose keys live in the
  // slots written here (this chunk's own are behind the barrier)
  __syncthreads();
  int* flags = p.flags + (int64_t)b * p.chunks;
  if (tid == 0 && !(p.withhold && c == 0)) {
    __threadfence();
    atomicExch(&flags[c], 1);
  }
  if (!any) return;
  if (tid == 0) {
    const uint64_t t0 = globaltimer_ns();
    bool ok = true;
    for (int d = s_job[1] / EM_KEYS; ok && d < c && d * EM_KEYS < s_job[2]; ++d)
      for (uint32_t spin = 1; *(volatile int*)&flags[d] == 0; ++spin)
        if ((spin & 255u) == 0u && globaltimer_ns() - t0 > p.wait_ns) {
          ok = false;
          break;
        }
    __threadfence();
    if (!ok) atomicOr(&p.status->last, ST_TIMEOUT);
    s_job[0] = ok;
  }
  __syncthreads();
  if (!s_job[0]) return;  // these slots hold keys that may not have been read: they stay
#pragma unroll
  for (int j = 0; j < EM_KEYS * 64 / EM_THREADS; ++j) {
    const int k = (j * EM_THREADS + tid) >> 6;
    if (s_from[k] >= 0) *reinterpret_cast<uint4*>(p.ckv + (int64_t)s_to[k] * p.ckv_stride + 16 * (tid & 63)) = v[j];
  }
#pragma unroll
  for (int j = 0; j < EM_KEYS * 8 / EM_THREADS; ++j) {
    const int k = (j * EM_THREADS + tid) >> 3;
    if (s_from[k] >= 0) {
      *reinterpret_cast<uint4*>(p.kpe + (int64_t)s_to[k] * p.kpe_stride + 16 * (tid & 7)) = e[j];
      if (p.k_cache) *reinterpret_cast<uint4*>(p.k_cache + (int64_t)s_to[k] * 128 + 16 * (tid & 7)) = x[j];
    }
  }
  if (p.k_cache && tid < EM_KEYS && s_from[tid] >= 0) p.k_scale[s_to[tid]] = scale;
}

template <int CS>
static cudaError_t launch_select_cs(const EvictParams& p, cudaStream_t s) {
  static DeviceFlags attr_set;
  cudaError_t e = set_smem_attr_once(evict_select_kernel<CS>, EVICT_CACHED_MAX * 4, attr_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.B * CS);
  cfg.blockDim = dim3(ES_THREADS);
  cfg.dynamicSmemBytes = 4 * (size_t)p.cached;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CS;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CS > 1 ? 2 : 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<CS>, p);
}

cudaError_t launch_evict(const EvictParams& p, cudaStream_t s) {
  const cudaError_t e = p.cluster == 8   ? launch_select_cs<8>(p, s)
                        : p.cluster == 4 ? launch_select_cs<4>(p, s)
                        : p.cluster == 2 ? launch_select_cs<2>(p, s)
                                         : launch_select_cs<1>(p, s);
  if (e != cudaSuccess) return e;
  count_launch();
  return launch_pdl(evict_move_kernel, dim3((unsigned)((int64_t)p.B * p.chunks)), dim3(EM_THREADS), 0, s, p);
}

}  // namespace dsa
