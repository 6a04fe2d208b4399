// latent_items.cuh -- the work of attention over the paged latent cache, as its
// kernels divide it: items (a block of rows and the keys they see) cut into
// equal runs of key tiles.
#pragma once

#include "latent.h"

namespace dsa {

namespace {

__device__ __forceinline__ float neg_inf() { return -__int_as_float(0x7f800000); }
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Length of sequence b, and of the prefix; an invalid one counts as 0.
__device__ __forceinline__ int valid_len(int len, int pages, bool& bad) {
  bad = len < 0 || len > (int64_t)pages * PAGE;
  return bad ? 0 : len;
}

// Drafted nodes of sequence b, its last keys; a sequence of an invalid number of them counts as empty.
__device__ __forceinline__ int tree_nodes(const LatentAttnParams& p, int b, int& len, bool& bad) {
  if (!p.draft_lens) return min(p.next_n, len);
  const int n = p.draft_lens[b];
  if (n >= 0 && n <= p.next_n && n <= len) return n;
  bad = true;
  return len = 0;
}

// One item: a block of rows and the keys they see.
struct Item {
  int row0, nrows;         // flat query rows
  int len;                 // keys behind `table`
  int lim0;                // keys that the block's first row sees; later tokens see one more each
  int r0;                  // first row within its sequence (-1: a prefix, every row sees all)
  const int32_t* table;
  // a tree: the sequence, its nodes, and the keys before them, which every row of a node sees
  int b, nodes, ctx;
};
template <bool TREE>
__device__ __forceinline__ Item load_item(const LatentAttnParams& p, int w) {
  Item it;
  bool bad;
  if (w < p.prefix_items) {
    it.row0 = w * p.n;
    it.nrows = min(p.n, p.B * p.next_n * p.H - it.row0);
    it.len = it.lim0 = valid_len(*p.prefix_len, p.prefix_pages, bad);
    it.r0 = -1;
    it.table = p.prefix_table;
    return it;
  }
  const int v = w - p.prefix_items, b = v / p.blocks, j = v % p.blocks, R = p.next_n * p.H;
  it.r0 = j * p.n;
  it.row0 = b * R + it.r0;
  it.nrows = min(p.n, R - it.r0);
  it.len = valid_len(p.seq_lens[b], p.max_pages, bad);
  it.lim0 = max(0, it.len - p.next_n + 1 + it.r0 / p.H);
  it.table = p.block_table + (int64_t)b * p.max_pages;
  if constexpr (TREE) {
    it.b = b;
    it.nodes = tree_nodes(p, b, it.len, bad);
    it.ctx = it.len - it.nodes;
    it.lim0 = it.r0 + p.n > it.nodes * p.H ? 0 : it.ctx;  // (rows that see nothing are masked in every tile)
  }
  return it;
}

// Which keys of page k a tree's row sees, one bit per key.
__device__ __forceinline__ uint64_t tree_bits(const LatentAttnParams& p, const Item& it, int row, int k) {
  const int node = row / p.H, d0 = k * PAGE - it.ctx;  // place of the page's first key among the drafted
  if (row >= p.next_n * p.H || node >= it.nodes) return 0;
  const uint64_t* mask = p.tree_mask + ((int64_t)it.b * p.next_n + node) * p.mask_words;
  auto word = [&](int w) {
    const int left = it.nodes - 64 * w;
    if (left <= 0) return (uint64_t)0;
    return left >= 64 ? mask[w] : mask[w] & (((uint64_t)1 << left) - 1);
  };
  if (d0 >= 0) {
    const int w = d0 >> 6, s = d0 & 63;
    return s ? word(w) >> s | word(w + 1) << (64 - s) : word(w);
  }
  if (d0 <= -PAGE) return ~(uint64_t)0;
  return word(0) << -d0 | (((uint64_t)1 << -d0) - 1);
}

// The pieces of one CTA: next() gives item w and its tiles [k0, k1).
struct Runs {
  const int32_t* start;
  int t, t1, w, extra;
  __device__ __forceinline__ bool next(int& item, int& k0, int& k1, bool& whole) {
    for (;;) {
      if (t >= t1) return false;
      int s0 = start[w], s1 = start[w + 1];
      while (s1 <= t) {
        ++w;
        s0 = s1;
        s1 = start[w + 1];
      }
      const int u1 = min(t1, s1) - s0;
      item = w;
      k0 = max(0, t - s0 - extra);
      k1 = max(0, u1 - extra);
      whole = k0 == 0 && u1 == s1 - s0;
      t = s0 + u1;
      if (k1 > k0) return true;  // (a run may end before an item's first tile)
    }
  }
};

// Numbers the items' units (start[]), the same in every CTA; returns the
// units and the first item of a run (of a CTA, or of a pair).  tmp: 34 ints of shared memory.
template <int THREADS, bool TREE, int KEYS>
__device__ __forceinline__ Runs plan_runs(const LatentAttnParams& p, int* tmp, int* status, int run) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* start = p.start + (int64_t)blockIdx.x * (p.items + 1);
  bool bad = false;
  const int pre = p.prefix_items ? valid_len(*p.prefix_len, p.prefix_pages, bad) : 0;
  if (bad) atomicOr(status, ST_RANGE);
  int base = 0, mine = 0, mine_end = 0;  // this thread's last item
  for (int i0 = 0; i0 < p.items; i0 += THREADS) {
    const int w = i0 + tid;
    int units = 0;
    if (w < p.items) {
      int len = pre;
      if (w >= p.prefix_items) {
        len = valid_len(p.seq_lens[(w - p.prefix_items) / p.blocks], p.max_pages, bad);
        // (a block without a node has nothing to do)
        if (TREE && w % p.blocks * p.n >= tree_nodes(p, w / p.blocks, len, bad) * p.H) len = 0;
        if (bad) atomicOr(status, ST_RANGE);
      }
      units = len ? ceil_div(len, KEYS) + p.item_units : 0;
    }
    int x = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) tmp[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
      const int v = tmp[i];
      before += i < warp ? v : 0;
      all += v;
    }
    mine = base + before + x - units;
    mine_end = mine + units;
    if (w < p.items) start[w] = mine;
    base += all;
  }
  const int per = max(p.item_units + 2, ceil_div(base, p.grid));
  const int t = min((int64_t)base, (int64_t)run * per);
  if (tid == 0) {
    start[p.items] = base;
    tmp[33] = 0;
    if (blockIdx.x == 0) *p.per = per;
  }
  __syncthreads();
  if (p.items <= THREADS) {  // (start[] need not be read back)
    if (tid < p.items && mine <= t && t < mine_end) tmp[33] = tid;
  } else {
    for (int w = tid; w < p.items; w += THREADS)
      if (start[w] <= t && t < start[w + 1]) tmp[33] = w;  // one item at most
  }
  __syncthreads();
  return Runs{start, t, (int)min((int64_t)base, (int64_t)t + per), tmp[33], p.item_units};
}

}  // namespace

}  // namespace dsa
