// cache_accept.cu -- keeps the accepted path of a tree of drafted tokens in the
// paged latent cache.
//
// A sequence's drafted nodes lie in logical slots [ctx, ctx + n) behind its ctx =
// seq_len - n settled keys.  Node path[j] moves to slot ctx + j.  A path ascends
// (a node comes after its parent), so path[j] >= j: whatever a move overwrites
// has been read, if the keys of a step are read before any of them is written:
// slot ctx + j is the source of an entry j at most, and the sources of later
// steps lie behind all targets of this one.
//
// A few keys of 1284 bytes per sequence: one CTA per sequence, one warp per key,
// all of a step's loads in flight at once.  Bound by latency, some five dependent
// accesses: 4 us for one sequence, 5 for 64 with trees of 64 nodes (0.8 MB).
#include "latent.h"

namespace dsa {

namespace {
constexpr int AC_THREADS = 512;
constexpr int AC_KEYS = AC_THREADS / 32;  // keys per step: few paths are longer
}  // namespace

__global__ void __launch_bounds__(AC_THREADS) accept_kernel(const AcceptParams p) {
  pdl_enter();
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int len = p.seq_lens[b], n = p.draft_lens[b], m = p.path_lens[b];
  const int32_t* path = p.path + (int64_t)b * p.max_path;
  bool bad = len < 0 || len > (int64_t)p.max_pages * PAGE || n < 0 || n > len || m < 0 || m > n || m > p.max_path;
  if (!bad)
    for (int j = tid; j < m; j += AC_THREADS) bad |= path[j] <= (j ? path[j - 1] : -1) || path[j] >= n;
  // (a path that is not one leaves its sequence as it is)
  const bool whole = !__syncthreads_or(bad);
  const int32_t* table = p.block_table + (int64_t)b * p.max_pages;
  const int ctx = len - n;
  if (whole) {
    for (int j0 = 0; j0 < m; j0 += AC_KEYS) {
      const int j = j0 + warp;
      int64_t src = -1, dst = -1;
      if (j < m) {
        const int from = ctx + path[j], to = ctx + j;
        const int pf = table[from / PAGE], pt = table[to / PAGE];
        if (pf < 0 || pf >= p.num_pages || pt < 0 || pt >= p.num_pages) bad = true;
        else if (from != to) {
          src = (int64_t)pf * PAGE + from % PAGE;
          dst = (int64_t)pt * PAGE + to % PAGE;
        }
      }
      uint4 c[2], e;
      float scale = 0.f;
      const bool pe = lane < 8, key = lane >= 8 && lane < 16 && p.k_cache;
      if (src >= 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) c[i] = *reinterpret_cast<const uint4*>(p.ckv + src * p.ckv_stride + 512 * i + 16 * lane);
        if (pe) e = *reinterpret_cast<const uint4*>(p.kpe + src * p.kpe_stride + 16 * lane);
        if (key) e = *reinterpret_cast<const uint4*>(p.k_cache + src * 128 + 16 * (lane - 8));
        if (lane == 16 && p.k_cache) scale = p.k_scale[src];
      }
      __syncthreads();  // every key of the step has been read
      if (src >= 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) *reinterpret_cast<uint4*>(p.ckv + dst * p.ckv_stride + 512 * i + 16 * lane) = c[i];
        if (pe) *reinterpret_cast<uint4*>(p.kpe + dst * p.kpe_stride + 16 * lane) = e;
        if (key) *reinterpret_cast<uint4*>(p.k_cache + dst * 128 + 16 * (lane - 8)) = e;
        if (lane == 16 && p.k_cache) p.k_scale[dst] = scale;
      }
    }
  }
  if (tid == 0) p.new_lens[b] = whole ? ctx + m : len;  // (new_lens may be seq_lens: every thread has its length)
  last_cta(p.status, bad);
}

cudaError_t launch_accept(const AcceptParams& p, cudaStream_t s) {
  count_launch();
  return launch_pdl(accept_kernel, dim3(p.B), dim3(AC_THREADS), 0, s, p);
}

}  // namespace dsa
