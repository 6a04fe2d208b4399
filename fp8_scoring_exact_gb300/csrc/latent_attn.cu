// latent_attn.cu -- attention over the paged latent cache in the absorbed form.
//
// Row (b, i, h), the query of head h at token i of sequence b, sees the
// prefix keys (if any) and then the logical keys [0, seq_lens[b] - next_n + i
// + 1) of its sequence; with u_s = scale_log2 * (q_nope . ckv[s] + q_pe .
// kpe[s]) its output is sum_s 2^(u_s - lse) ckv[s], lse = log2(sum_s 2^u_s).
// A row that sees no key gets zeros and lse = -inf.
//
// A key is 1152 bytes and costs a row 2176 operations, so up to about 128
// rows a sequence the cache's bandwidth bounds the call, beyond that (a
// prefix shared by the batch) the tensor cores.  One kernel serves both:
// blocks of N = 16, 32 or 64 rows against tiles of one page (64 keys), with
// the products transposed so that the key data, not the few rows, fill the
// MMA's M side:
//     S^T [64 keys x N rows]  = K [64 x 576] . Q^T         (36 steps of M = 64)
//     O^T [512 dims x N rows] += V^T [512 x 64] . P^T      (16 steps of M = 128)
// K and V are the same shared-memory tile, copied once by TMA: the first
// product reads it with the dims contiguous, the second with M = dims (the
// contiguous axis) and K = keys.  O^T (4 x N columns) and two S^T buffers stay
// in TMEM; nothing but the result leaves the SM.
//
// Warps: 0 copies (a ring of 16 KB slots of 128 dims of a page, and 8 KB
// slots of the rope dims), 1 issues S^T, the last O^T (a warp of its own: a
// tile's weights are ready while the next tile's data are on their way, and
// its slots should come free then), those between do the softmax: the 16 x
// 256b TMEM load leaves a thread two keys and some rows; the weights go to
// shared memory as bf16 by stmatrix.  The reference maximum of a row only
// moves when a logit passes it by 8 (a factor of 2^8: fp32 sums and bf16
// weights have the range for that), which a vote over the warps finds out; only
// then are maxima exchanged and O^T is rescaled (finding the maximum of every
// tile instead took 7% longer for 64 sequences behind 32768 shared keys).
//
// Every CTA takes an equal run of the call's tiles, whatever item they
// belong to; an item cut by a run's border is joined by the finish kernel in
// the order of its pieces, so results do not depend on timing.
//
// Rows per block: the least that holds a sequence's rows, as every block reads
// the keys anew.  16 sequences of 32768 keys, in us, against the copy rate's 89:
//     rows      N = 16   N = 32   N = 64
//     16          102      106      109
//     32          187      106      110
//     64          356        -      114
// 64 sequences of up to 131072 keys with two tokens of 16 heads (4.6 GB): 662 to
// 682 us, 6.8 to 7.0 TB/s, the measured copy rate.  N = 64 is bound by its chain:
// the query block leaves room for two tiles, a tile's copy, S^T, softmax and
// O^T take some 4200 cycles one after the other, and 1650 of the 2100 per tile
// are the tensor cores' (the M = 64 steps of S^T run at half their rate): 64
// sequences of two tokens of 16 heads behind 32768 shared keys 160 us, 0.94
// PFLOP/s; seven sequences of 128 heads 70 us, which read 282 MB from DRAM for their
// 193, as a sequence's two blocks come to its keys at different times.  The MMAs
// take shared memory's whole bandwidth, so the softmax keeps what it can in
// registers (references read from shared memory for every tile: 5 us more).
// (Prefetching the pages of tiles 2, 3, 5 or 8 ahead into L2 made all of these
// slower: 16 sequences of 64 rows 122, 129, 164, 173 us.)
#include "latent.h"

namespace dsa {

namespace {

constexpr int LT = PAGE;                       // keys per tile
constexpr uint32_t CHUNK = LT * 128;           // 64 keys x 64 dims, bf16
constexpr uint32_t PAIR = 2 * CHUNK;           // 64 keys x 128 dims
constexpr float NO_REF = -3.402823466e38f;     // the reference of a row that has seen no key: any logit passes it
constexpr float RESCALE_AT = 8.f;              // a row's reference moves when its maximum passes it by this

template <int N>
struct LA {
  // Softmax warps: four (a quarter of the TMEM lanes each), for 64 rows eight
  // (half the rows each), as there the softmax of a tile takes as long as its products.
  static constexpr int SW = N == 64 ? 8 : 4, ST = 32 * SW;
  static constexpr int NC = N * 4 / SW;                    // rows per softmax warp
  static constexpr int W_PV = 2 + SW;                      // the last warp issues the second product
  static constexpr int THREADS = 32 * (W_PV + 1);
  // Ring depths: what 227 KB leave next to the query block.  64 rows keep
  // two tiles of ckv and one of the rope part, and one weight buffer.
  static constexpr int PAIRS = N == 64 ? 8 : N == 32 ? 10 : 11;
  static constexpr int KPES = N == 64 ? 1 : 2;
  static constexpr int PBUFS = N == 64 ? 1 : 2;
  static constexpr uint32_t P_BYTES = N * 128;  // weights of a tile: N rows x 64 keys bf16
  static constexpr uint32_t OFF_Q = 0;          // 9 chunks of N rows x 64 dims
  static constexpr uint32_t OFF_P = OFF_Q + 9 * N * 128;
  static constexpr uint32_t OFF_PAIR = (OFF_P + PBUFS * P_BYTES + 1023) / 1024 * 1024;
  static constexpr uint32_t OFF_KPE = OFF_PAIR + PAIRS * PAIR;
  static constexpr uint32_t OFF_MISC = OFF_KPE + KPES * CHUNK;
  // barriers: pair full/empty, kpe full/empty, q full/empty, S full/empty x 2, P full x 2, PV done x 2, O empty, drain x 2
  static constexpr int B_PF = 0, B_PE = PAIRS, B_KF = 2 * PAIRS, B_KE = B_KF + KPES, B_QF = B_KE + KPES, B_QE = B_QF + 1,
                       B_SF = B_QE + 1, B_SE = B_SF + 2, B_WF = B_SE + 2, B_VD = B_WF + 2, B_OE = B_VD + 2,
                       B_DRAIN = B_OE + 1, N_BARS = B_DRAIN + 2;
  static constexpr uint32_t OFF_BAR = OFF_MISC;
  static constexpr uint32_t OFF_RED = OFF_BAR + (N_BARS * 8 + 127) / 128 * 128;  // [4][N] floats
  static constexpr uint32_t OFF_REF = OFF_RED + 4 * N * 4;                       // [N] reference maxima
  static constexpr uint32_t OFF_ALPHA = OFF_REF + N * 4;                         // [N] factors
  static constexpr uint32_t OFF_LIM = OFF_ALPHA + N * 4;                         // [N] visible keys per row
  static constexpr uint32_t OFF_FLAG = OFF_LIM + N * 4;                          // abort, tmem base
  static constexpr uint32_t OFF_STAT = OFF_FLAG + 128;                           // Stats: this CTA's status and wait limit
  static constexpr uint32_t SMEM = OFF_STAT + 128 + 1024;                        // + alignment
  static constexpr uint32_t TMEM_S = 4 * N;                                      // column of the first S^T buffer (2 N each)
  static constexpr uint32_t TMEM_COLS = N == 64 ? 512 : N == 32 ? 256 : 128;     // 8 N
  static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
};

__device__ __forceinline__ float neg_inf() { return -__int_as_float(0x7f800000); }
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void stsm_x4_t(uint32_t addr, const uint32_t* r) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}

// Length of sequence b, and of the prefix; an invalid one counts as 0.
__device__ __forceinline__ int valid_len(int len, int pages, bool& bad) {
  bad = len < 0 || len > (int64_t)pages * PAGE;
  return bad ? 0 : len;
}

// Reduces a[i] over the lanes that differ in bits 2..4 (the keys of a warp):
// each step halves what a lane holds and the lanes a row is spread over.  A
// lane ends with the row own_row() of its warp's, in a[0].
template <int n, class Op>
__device__ __forceinline__ void over_keys(float (&a)[n], int lane, Op op) {
  int h = n;
#pragma unroll
  for (int o = 16; o >= 4; o >>= 1) {
    if (h > 1) {
      h >>= 1;
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < h; ++i) {
        const float keep = up ? a[i + h] : a[i], send = up ? a[i] : a[i + h];
        a[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
      }
    } else {
      a[0] = op(a[0], __shfl_xor_sync(0xffffffffu, a[0], o));
    }
  }
}
template <int n>
__device__ __forceinline__ int own_row(int lane) {
  static_assert(n == 8 || n == 4, "NC = 32 or 16");
  const int i = n == 8 ? (lane >> 4 & 1) * 4 + (lane >> 3 & 1) * 2 + (lane >> 2 & 1) : (lane >> 4 & 1) * 2 + (lane >> 3 & 1);
  return 8 * (i >> 1) + 2 * (lane & 3) + (i & 1);
}

// One item: a block of rows and the keys they see.
struct Item {
  int row0, nrows;         // flat query rows
  int len;                 // keys behind `table`
  int lim0;                // keys that the block's first row sees; later tokens see one more each
  int r0;                  // first row within its sequence (-1: a prefix, every row sees all)
  const int32_t* table;
};
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
  return it;
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

// Numbers the items' units (start[]), the same in every CTA; returns this
// CTA's units and first item.  tmp: 34 ints of shared memory.
template <int THREADS>
__device__ __forceinline__ Runs plan_runs(const LatentAttnParams& p, int* tmp, int* status) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* start = p.start + (int64_t)blockIdx.x * (p.items + 1);
  bool bad = false;
  const int pre = p.prefix_items ? valid_len(*p.prefix_len, p.prefix_pages, bad) : 0;
  if (bad) atomicOr(status, ST_RANGE);
  int base = 0;
  for (int i0 = 0; i0 < p.items; i0 += THREADS) {
    const int w = i0 + tid;
    int units = 0;
    if (w < p.items) {
      int len = pre;
      if (w >= p.prefix_items) {
        len = valid_len(p.seq_lens[(w - p.prefix_items) / p.blocks], p.max_pages, bad);
        if (bad) atomicOr(status, ST_RANGE);
      }
      units = len ? ceil_div(len, LT) + p.item_units : 0;
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
    if (w < p.items) start[w] = base + before + x - units;
    base += all;
  }
  const int per = max(p.item_units + 2, ceil_div(base, p.grid));
  const int t = min((int64_t)base, (int64_t)blockIdx.x * per);
  if (tid == 0) {
    start[p.items] = base;
    tmp[33] = 0;
    if (blockIdx.x == 0) *p.per = per;
  }
  __syncthreads();
  for (int w = tid; w < p.items; w += THREADS)
    if (start[w] <= t && t < start[w + 1]) tmp[33] = w;  // one item at most
  __syncthreads();
  return Runs{start, t, (int)min((int64_t)base, (int64_t)t + per), tmp[33], p.item_units};
}

}  // namespace

template <int N>
__global__ void __launch_bounds__(LA<N>::THREADS, 1)
    latent_attn_kernel(const __grid_constant__ LatentMaps maps, const LatentAttnParams p) {
  using C = LA<N>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + C::OFF_BAR + 8u * i; };
  float* s_red = reinterpret_cast<float*>(smem + C::OFF_RED);
  float* s_ref = reinterpret_cast<float*>(smem + C::OFF_REF);
  float* s_alpha = reinterpret_cast<float*>(smem + C::OFF_ALPHA);
  int* s_lim = reinterpret_cast<int*>(smem + C::OFF_LIM);
  volatile int* abort_flag = reinterpret_cast<int*>(smem + C::OFF_FLAG);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::OFF_FLAG + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Stats* stats = reinterpret_cast<Stats*>(smem + C::OFF_STAT);

  // before the wait for the previous kernel of the stream: barriers, TMEM
  // and the tensor maps (the call's own inputs are read after it)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    stats->status = 0;
    stats->wait_ns = p.wait_ns;
    tma_prefetch_desc(&maps.q_nope);
    tma_prefetch_desc(&maps.q_pe);
    tma_prefetch_desc(&maps.ckv);
    tma_prefetch_desc(&maps.kpe);
    for (int i = 0; i < 2 * C::PAIRS + 2 * C::KPES + 2; ++i) mbar_init(bar(i), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::B_SF + i), 1);
      mbar_init(bar(C::B_SE + i), C::SW);
      mbar_init(bar(C::B_WF + i), C::SW);
      mbar_init(bar(C::B_VD + i), 1);
    }
    mbar_init(bar(C::B_OE), C::SW);
    mbar_init(bar(C::B_DRAIN), 1);
    mbar_init(bar(C::B_DRAIN + 1), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  // (the scan's scratch lies in the exchange buffer of the softmax)
  Runs runs = plan_runs<C::THREADS>(p, reinterpret_cast<int*>(smem + C::OFF_RED), &stats->status);
  __syncthreads();
  uint32_t it = 0;       // this CTA's tiles so far
  uint32_t seg = 0;      // and its pieces
  uint32_t n_pair = 0, n_kpe = 0, n_q = 0;  // producer: copies armed
  int w, k0, k1;
  bool whole;

  if (warp == 0) {
    // ------------------------------------------------------- TMA producer --
    bool ok = true;
    while (ok && runs.next(w, k0, k1, whole)) {
      const Item im = load_item(p, w);
      if (!(ok = mbar_wait_warp(bar(C::B_QE), (seg & 1) ^ 1, abort_flag, stats))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(C::B_QF), 9 * N * 128);
        tma_load_3d(sbase + C::OFF_Q, &maps.q_nope, 0, im.row0, 0, bar(C::B_QF));
        tma_load_2d(sbase + C::OFF_Q + 8 * N * 128, &maps.q_pe, 0, im.row0, bar(C::B_QF));
      }
      ++n_q;
      ++seg;
      int pages = 0;  // lane j: page of tile (k & ~31) + j, the page past the cache for an invalid one
      for (int k = k0; ok && k < k1; ++k) {
        if (k == k0 || (k & 31) == 0) {
          const int j = (k & ~31) + lane;
          bool bad = false;
          if (j >= k && j < k1) {
            pages = im.table[j];
            bad = pages < 0 || pages >= p.num_pages;
            if (bad) pages = p.num_pages;
          }
          if (__ballot_sync(0xffffffffu, bad) && lane == 0) atomicOr(&stats->status, ST_RANGE);
        }
        const int slot = __shfl_sync(0xffffffffu, pages, k & 31) * PAGE;
        const int ks = n_kpe % C::KPES;
        if (!(ok = mbar_wait_warp(bar(C::B_KE + ks), ((n_kpe / C::KPES) & 1) ^ 1, abort_flag, stats))) break;
        if (lane == 0 && !(p.withhold && n_kpe == 0)) {
          mbar_arrive_expect_tx(bar(C::B_KF + ks), CHUNK);
          tma_load_2d(sbase + C::OFF_KPE + ks * CHUNK, &maps.kpe, 0, slot, bar(C::B_KF + ks));
        }
        ++n_kpe;
        for (int c = 0; c < 4; ++c, ++n_pair) {
          const int st = n_pair % C::PAIRS;
          if (!(ok = mbar_wait_warp(bar(C::B_PE + st), ((n_pair / C::PAIRS) & 1) ^ 1, abort_flag, stats))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(C::B_PF + st), PAIR);
            tma_load_3d(sbase + C::OFF_PAIR + st * PAIR, &maps.ckv, 0, slot, 2 * c, bar(C::B_PF + st));
          }
        }
      }
    }
  } else if (warp == 1) {
    // --------------------------------------------------------- S^T issuer --
    constexpr uint32_t ID_S = idesc_bf16_f32(64, N, false, false);
    const uint32_t leader = elect_one();
    const uint32_t q_lo = desc_lo_kmajor(sbase + C::OFF_Q);
    // Each step's addition to the accumulator truncates.  Where the logits
    // themselves are wanted (key weights come back in fp32) their 36 steps are
    // split over two accumulators, which halves that error.
    const uint32_t split = p.logits ? 2 : 4;
    bool ok = true;
    while (ok && runs.next(w, k0, k1, whole)) {
      if (!(ok = mbar_wait_warp(bar(C::B_QF), seg & 1, abort_flag, stats))) break;
      for (int k = k0; ok && k < k1; ++k, ++it) {
        const uint32_t sb = it & 1;
        if (!(ok = mbar_wait_warp(bar(C::B_SE + sb), ((it >> 1) & 1) ^ 1, abort_flag, stats))) break;
        tc_fence_after();
        const uint32_t d = tmem + C::TMEM_S + sb * 2 * N;
        // the rope part first, so that its slot comes free first
        const uint32_t ks = it % C::KPES;
        if (!(ok = mbar_wait_warp(bar(C::B_KF + ks), (it / C::KPES) & 1, abort_flag, stats))) break;
        const uint32_t e_lo = desc_lo_kmajor(sbase + C::OFF_KPE + ks * CHUNK);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma_bf16_ss(leader, d, e_lo + 2 * j, q_lo + 8 * (N * 128 >> 4) + 2 * j, ID_S, j > 0);
        mma_commit_warp(leader, bar(C::B_KE + ks));
        for (uint32_t c = 0; c < 4; ++c) {
          const uint32_t i = 4 * it + c, st = i % C::PAIRS;
          if (!(ok = mbar_wait_warp(bar(C::B_PF + st), (i / C::PAIRS) & 1, abort_flag, stats))) break;
          const uint32_t k_lo = desc_lo_kmajor(sbase + C::OFF_PAIR + st * PAIR);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            mma_bf16_ss(leader, d + (c >= split ? N : 0), k_lo + (j >> 2) * (CHUNK >> 4) + 2 * (j & 3),
                        q_lo + (2 * c + (j >> 2)) * (N * 128 >> 4) + 2 * (j & 3), ID_S, c != split || j > 0);
        }
        if (!ok) break;
        mma_commit_warp(leader, bar(C::B_SF + sb));
        if (k == k1 - 1) mma_commit_warp(leader, bar(C::B_QE));
      }
      ++seg;
    }
  } else if (warp == C::W_PV) {
    // --------------------------------------------------------- O^T issuer --
    // A warp of its own: a tile's weights are ready while the next tile's data
    // are still on their way, and its slots should come free then.
    constexpr uint32_t ID_O = idesc_bf16_f32(128, N, true, false);
    const uint32_t leader = elect_one();
    bool ok = true;
    while (ok && runs.next(w, k0, k1, whole)) {
      // the previous piece's O^T has been read out
      if (!(ok = mbar_wait_warp(bar(C::B_OE), (seg & 1) ^ 1, abort_flag, stats))) break;
      for (int k = k0; k < k1; ++k, ++it) {
        if (!(ok = mbar_wait_warp(bar(C::B_WF + (it & 1)), (it >> 1) & 1, abort_flag, stats))) break;
        tc_fence_after();
        const uint32_t p_lo = desc_lo_kmajor(sbase + C::OFF_P + (it % C::PBUFS) * C::P_BYTES);
        for (uint32_t c = 0; c < 4; ++c) {
          const uint32_t st = (4 * it + c) % C::PAIRS;
          const uint32_t v_lo = desc_lo_mnmajor(sbase + C::OFF_PAIR + st * PAIR, CHUNK);
#pragma unroll
          for (int j = 0; j < 4; ++j)  // 16 keys: 2 KB of V, 32 bytes of a P row
            mma_bf16_ss(leader, tmem + c * N, v_lo + 128 * j, p_lo + 2 * j, ID_O, k > k0 || j > 0);
          mma_commit_warp(leader, bar(C::B_PE + st));
        }
        mma_commit_warp(leader, bar(C::B_VD + (it & 1)));
      }
      ++seg;
    }
  } else {
    // ----------------------------------------------------- softmax warps --
    // A wait that gives up does not leave the loop (the other warps of the
    // exchange would wait for ever): with the abort flag set every later
    // wait returns at once, and the result is undefined but complete.
    const int q = warp & 3;                  // TMEM lane quarter: keys [16 q, + 16)
    const int half = (warp - 2) >> 2;        // rows [NC half, + NC)
    const int st_id = threadIdx.x - 64;      // 0 .. ST - 1
    const int g = lane >> 2, cb = half * C::NC, cc = cb + 2 * (lane & 3);
    constexpr int M8 = C::NC / 8;            // blocks of 8 rows
    constexpr int HALVES = C::SW / 4;
    float ref = neg_inf();                   // threads st_id < N: the reference maximum of row st_id
    while (runs.next(w, k0, k1, whole)) {
      const Item im = load_item(p, w);
      for (int c = st_id; c < N; c += C::ST)
        s_lim[c] = c >= im.nrows ? 0 : im.r0 < 0 ? im.len : max(0, im.len - p.next_n + 1 + (im.r0 + c) / p.H);
      float2 f[M8];                          // the references of this thread's rows
      float l[2 * M8];                       // its part of each row's sum
#pragma unroll
      for (int i = 0; i < 2 * M8; ++i) l[i] = 0.f;
      ref = neg_inf();
      for (int k = k0; k < k1; ++k, ++it) {
        const uint32_t sb = it & 1;
        mbar_wait_warp(bar(C::B_SF + sb), (it >> 1) & 1, abort_flag, stats);
        tc_fence_after();
        uint32_t s[4 * M8];
        const uint32_t sa = tmem + C::TMEM_S + sb * 2 * N + cb + ((uint32_t)(32 * q) << 16);
        if constexpr (M8 == 4) tmem_ld16x256b_x4(sa, s);
        if constexpr (M8 == 2) tmem_ld16x256b_x2(sa, s);
        tmem_wait_ld();
        if (p.logits) {
          uint32_t s2[4 * M8];
          if constexpr (M8 == 4) tmem_ld16x256b_x4(sa + N, s2);
          if constexpr (M8 == 2) tmem_ld16x256b_x2(sa + N, s2);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 4 * M8; ++i) s[i] = __float_as_uint(__uint_as_float(s[i]) + __uint_as_float(s2[i]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::B_SE + sb));
        // slots past the sequence may hold anything: their values become 0
        // in the tile itself (a weight of 0 does not silence a NaN)
        const int valid = im.len - k * LT;
        if (valid < LT) {
          for (int i = st_id; i < (LT - valid) * 64; i += C::ST) {
            const int row = valid + (i >> 6), ch = (i >> 3) & 7, x = i & 7;  // row, chunk of 64 dims, 16 bytes
            const uint32_t ps = (4 * it + (ch >> 1)) % C::PAIRS;
            *reinterpret_cast<uint4*>(smem + C::OFF_PAIR + ps * PAIR + (ch & 1) * CHUNK + row * 128 + 16 * x) =
                make_uint4(0, 0, 0, 0);
          }
        }
        // logits of rows 8 m + cc + {0, 1}, keys 16 q + g and + 8
        float u[M8][4];
#pragma unroll
        for (int i = 0; i < 4 * M8; ++i) u[i >> 2][i & 3] = __uint_as_float(s[i]);
        const int key = k * LT + 16 * q + g;
        if ((k + 1) * LT > im.lim0 || im.nrows < N) {
          named_bar_sync(1, C::ST);  // s_lim
#pragma unroll
          for (int m = 0; m < M8; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int lim = s_lim[8 * m + cc + e];
              if (key >= lim) u[m][e] = neg_inf();
              if (key + 8 >= lim) u[m][2 + e] = neg_inf();
            }
        }
        if (p.logits) {
          float* dst = p.logits + (((int64_t)w * p.max_pages + k) * LT + 16 * q + g) * N + cc;
#pragma unroll
          for (int m = 0; m < M8; ++m) {
            *reinterpret_cast<float2*>(dst + 8 * m) = make_float2(u[m][0], u[m][1]);
            *reinterpret_cast<float2*>(dst + 8 * N + 8 * m) = make_float2(u[m][2], u[m][3]);
          }
        }
        // does a logit lie so far above its row's reference that the row's
        // maximum has to be found?  (always in a piece's first tile)
        bool rescale = true;
        if (k > k0) {
          float over = neg_inf();
#pragma unroll
          for (int m = 0; m < M8; ++m) {
            over = fmaxf(over, fmaf(fmaxf(u[m][0], u[m][2]), p.scale_log2, -f[m].x));
            over = fmaxf(over, fmaf(fmaxf(u[m][1], u[m][3]), p.scale_log2, -f[m].y));
          }
          rescale = named_bar_or(1, C::ST, over > RESCALE_AT);
        }
        if (rescale) {
          float mx[2 * M8];
#pragma unroll
          for (int i = 0; i < 2 * M8; ++i) mx[i] = fmaxf(u[i >> 1][i & 1], u[i >> 1][2 + (i & 1)]);
          over_keys<2 * M8>(mx, lane, [](float a, float b) { return fmaxf(a, b); });
          s_red[q * N + own_row<2 * M8>(lane) + cb] = mx[0];
          named_bar_sync(1, C::ST);
          if (st_id < N) {
            const float top = p.scale_log2 * fmaxf(fmaxf(s_red[st_id], s_red[N + st_id]),
                                                   fmaxf(s_red[2 * N + st_id], s_red[3 * N + st_id]));
            float a = 1.f;
            if (top > ref + RESCALE_AT || (ref == neg_inf() && top > ref)) {
              a = ex2(ref - top);  // 0 from a reference of -inf
              ref = top;
            }
            s_alpha[st_id] = a;
            s_ref[st_id] = fmaxf(ref, NO_REF);
          }
          named_bar_sync(1, C::ST);
#pragma unroll
          for (int i = 0; i < 2 * M8; ++i) l[i] *= s_alpha[8 * (i >> 1) + cc + (i & 1)];
#pragma unroll
          for (int m = 0; m < M8; ++m) f[m] = *reinterpret_cast<const float2*>(&s_ref[8 * m + cc]);
        }
        // weights: fp32 into the sums, rounded to bf16 (the type of V, which
        // the MMA wants of both operands) for P
        uint32_t r[M8][2];
#pragma unroll
        for (int m = 0; m < M8; ++m) {
          const float a0 = ex2(fmaf(u[m][0], p.scale_log2, -f[m].x)), a1 = ex2(fmaf(u[m][1], p.scale_log2, -f[m].y));
          const float b0 = ex2(fmaf(u[m][2], p.scale_log2, -f[m].x)), b1 = ex2(fmaf(u[m][3], p.scale_log2, -f[m].y));
          l[2 * m] += a0 + b0;
          l[2 * m + 1] += a1 + b1;
          const __nv_bfloat162 pa = __floats2bfloat162_rn(a0, a1), pc = __floats2bfloat162_rn(b0, b1);
          r[m][0] = *reinterpret_cast<const uint32_t*>(&pa);
          r[m][1] = *reinterpret_cast<const uint32_t*>(&pc);
        }
        // the weight buffer is free once the product that read it last is done
        if (C::PBUFS == 1) {
          if (it > 0) mbar_wait_warp(bar(C::B_VD + (sb ^ 1)), ((it - 1) >> 1) & 1, abort_flag, stats);
        } else if (it > 1) {
          mbar_wait_warp(bar(C::B_VD + sb), ((it - 2) >> 1) & 1, abort_flag, stats);
        }
        if (rescale && k > k0) {  // O^T: four blocks of 128 dims, 32 lanes of each
          mbar_wait_warp(bar(C::B_VD + (sb ^ 1)), ((it - 1) >> 1) & 1, abort_flag, stats);
          tc_fence_after();
#pragma unroll 1
          for (int j = half; j < 4 * N / 16; j += HALVES) {
            uint32_t o[16];
            const uint32_t oa = tmem + 16 * j + ((uint32_t)(32 * q) << 16);
            tmem_ld16(oa, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o[i] = __float_as_uint(__uint_as_float(o[i]) * s_alpha[(16 * j + i) % N]);
            tmem_st16(oa, o);
          }
          tmem_wait_st();
        }
        const uint32_t pb = sbase + C::OFF_P + (it % C::PBUFS) * C::P_BYTES;
#pragma unroll
        for (int m = 0; m < M8; m += 2) {
          // matrix lane / 8: rows 8 (m + lane / 16), keys 16 q + 8 (lane / 8 % 2)
          const int row = cb + 8 * (m + (lane >> 4)) + (lane & 7);
          const int ch = 2 * q + ((lane >> 3) & 1);
          const uint32_t x[4] = {r[m][0], r[m][1], r[m + 1][0], r[m + 1][1]};
          stsm_x4_t(pb + row * 128 + ((ch ^ (row & 7)) << 4), x);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::B_WF + sb));
      }
      // ---- the piece's result: sums over the warps, then O^T out of TMEM
      over_keys<2 * M8>(l, lane, [](float a, float b) { return a + b; });
      named_bar_sync(1, C::ST);  // s_red, s_alpha and s_lim are free
      s_red[q * N + own_row<2 * M8>(lane) + cb] = l[0];
      named_bar_sync(1, C::ST);
      const bool direct = whole && !p.prefix_items;
      const int64_t piece = (int64_t)w + blockIdx.x;
      const int64_t part = p.prefix_items ? piece : 2 * (int64_t)blockIdx.x + (k0 == 0 ? 1 : 0);
      if (st_id < N) {
        const float sum = (s_red[st_id] + s_red[N + st_id]) + (s_red[2 * N + st_id] + s_red[3 * N + st_id]);
        if (direct) {
          s_alpha[st_id] = sum == 0.f ? 0.f : 1.f / sum;
          if (st_id < im.nrows) p.lse[im.row0 + st_id] = sum == 0.f ? neg_inf() : s_ref[st_id] + log2f(sum);
        }
        if (!direct || p.logits) p.part_ml[piece * N + st_id] = make_float2(ref, sum);
      }
      named_bar_sync(1, C::ST);
      mbar_wait_warp(bar(C::B_VD + ((it - 1) & 1)), ((it - 1) >> 1) & 1, abort_flag, stats);
      tc_fence_after();
#pragma unroll 1
      for (int j = half; j < 4 * N / 16; j += HALVES) {
        uint32_t o[16];
        tmem_ld16(tmem + 16 * j + ((uint32_t)(32 * q) << 16), o);
        tmem_wait_ld();
        const int dim = 128 * (16 * j / N) + 32 * q + lane, c0 = 16 * j % N;
        if (direct) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c0 + i < im.nrows)
              p.out[(int64_t)(im.row0 + c0 + i) * LA_DC + dim] = __float2bfloat16(__uint_as_float(o[i]) * s_alpha[c0 + i]);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c0 + i < im.nrows) p.part_o[(part * N + c0 + i) * LA_DC + dim] = __uint_as_float(o[i]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::B_OE));
      named_bar_sync(1, C::ST);  // s_alpha has been read
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // before shared memory and TMEM are released, the copies and MMAs
    // already issued land: the last phase armed on each slot, a last commit
    const uint64_t until = globaltimer_ns() + DRAIN_ALL_NS;
    if (warp == 0 && lane == 0) {
      for (uint32_t s = 0; s < C::PAIRS; ++s)
        if (n_pair > s) mbar_drain_until(bar(C::B_PF + s), ((n_pair - 1 - s) / C::PAIRS) & 1, until);
      for (uint32_t s = 0; s < C::KPES; ++s)
        if (n_kpe > s) mbar_drain_until(bar(C::B_KF + s), ((n_kpe - 1 - s) / C::KPES) & 1, until);
      if (n_q) mbar_drain_until(bar(C::B_QF), (n_q - 1) & 1, until);
    } else if (warp == 1 || warp == C::W_PV) {
      const uint32_t db = bar(C::B_DRAIN + (warp == C::W_PV));
      mma_commit_warp(elect_one(), db);  // (elect.sync picks the lane that issued: it is deterministic)
      mbar_drain_until(db, 0, until);
    }
    __syncthreads();
  }
  if (threadIdx.x == 0 && stats->status) atomicOr(&p.status->now, stats->status);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// The pieces of a row: two runs of ids (prefix, own keys) and its place in their blocks.
struct RowPieces {
  int id0[2], cnt[2], col[2], n, cta0;
  __device__ __forceinline__ RowPieces(const LatentAttnParams& p, int64_t row) {
    const int R = p.next_n * p.H, b = (int)(row / R), r = (int)(row % R), per = *p.per;
    n = cta0 = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int w = k ? p.prefix_items + b * p.blocks + r / p.n : (int)(row / p.n);
      cnt[k] = id0[k] = 0;
      col[k] = k ? r % p.n : (int)(row % p.n);
      if (k == 0 && !p.prefix_items) continue;
      const int s0 = p.start[w], s1 = p.start[w + 1];
      if (s0 == s1) continue;
      cta0 = (s0 + p.item_units) / per;  // the CTA of its first tile
      id0[k] = w + cta0;
      cnt[k] = w + (s1 - 1) / per - id0[k] + 1;
      n += cnt[k];
    }
  }
  // the only piece of a row without a prefix wrote its result itself
  __device__ __forceinline__ bool done(const LatentAttnParams& p) const { return n == 1 && !p.prefix_items; }
  __device__ __forceinline__ int64_t at(const LatentAttnParams& p, int i) const {
    return i < cnt[0] ? (int64_t)(id0[0] + i) * p.n + col[0] : (int64_t)(id0[1] + i - cnt[0]) * p.n + col[1];
  }
};

// A row's pieces joined in their order, dims [d0, d0 + DIMS) of it: THREADS / (DIMS / 4)
// parts take every so manieth piece, 4 dims per thread.
constexpr int FIN_MAX = 2 * 1024;  // pieces of a row at most: the grid's CTAs, twice with a prefix
template <int THREADS, int DIMS>
__device__ __forceinline__ void join_row(const LatentAttnParams& p, int64_t row, int d0) {
  constexpr int PER = DIMS / 4, PARTS = THREADS / PER, WARPS = THREADS / 32;
  __shared__ float s_w[FIN_MAX];
  __shared__ __align__(16) float s_part[PARTS > 1 ? PARTS - 1 : 1][DIMS];
  __shared__ float s_tmp[WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const RowPieces rp(p, row);
  const int n = rp.n;
  if (rp.done(p)) return;
  float m = neg_inf();
  for (int i = tid; i < n; i += THREADS) m = fmaxf(m, p.part_ml[rp.at(p, i)].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) s_tmp[warp] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < WARPS; ++i) m = fmaxf(m, s_tmp[i]);
  const float mm = m == neg_inf() ? 0.f : m;
  float sum = 0.f;
  for (int i = tid; i < n; i += THREADS) {
    const float2 ml = p.part_ml[rp.at(p, i)];
    const float x = ex2(ml.x - mm);
    s_w[i] = x;
    sum += x * ml.y;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  __syncthreads();
  if (lane == 0) s_tmp[warp] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) sum += s_tmp[i];
  // rows of part_o: two runs with a prefix; without one the first piece's, then every second from there
  const bool own = !p.prefix_items;
  const int split = own ? 1 : rp.cnt[0], step = own ? 2 * p.n : p.n;
  const int64_t row_a = own ? (int64_t)(2 * rp.cta0 + 1) * p.n + rp.col[1] : (int64_t)rp.id0[0] * p.n + rp.col[0];
  const int64_t row_b = own ? (int64_t)(2 * rp.cta0) * p.n + rp.col[1] : (int64_t)(rp.id0[1] - split) * p.n + rp.col[1];
  const int part = tid / PER, d = 4 * (tid % PER);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = part; i < n; i += PARTS) {
    const float x = s_w[i];
    const int64_t at = (i < split ? row_a : row_b) + (int64_t)i * step;
    const float4 v = __ldcs(reinterpret_cast<const float4*>(p.part_o + at * LA_DC + d0 + d));
    if (x != 0.f) {  // a piece without a visible key adds nothing
      o.x += x * v.x;
      o.y += x * v.y;
      o.z += x * v.z;
      o.w += x * v.w;
    }
  }
  if (PARTS > 1) {
    if (part) *reinterpret_cast<float4*>(&s_part[part - 1][d]) = o;
    __syncthreads();
    if (part) return;
#pragma unroll
    for (int i = 0; i < PARTS - 1; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(&s_part[i][d]);
      o.x += v.x;
      o.y += v.y;
      o.z += v.z;
      o.w += v.w;
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(p.out + row * LA_DC + d0 + d);
  dst[0] = __floats2bfloat162_rn(o.x * inv, o.y * inv);
  dst[1] = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  if (tid == 0 && d0 == 0) p.lse[row] = sum == 0.f ? neg_inf() : mm + log2f(sum);
}

// The call's last kernel: CTA (row, chunk of dims).
template <int THREADS, int DIMS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) latent_join_kernel(const LatentAttnParams p) {
  pdl_enter();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    p.status->last = p.status->now;
    p.status->now = 0;
  }
  join_row<THREADS, DIMS>(p, blockIdx.x, DIMS * blockIdx.y);
}

// The same with key weights.  CTAs [0, rows) join a row each; of those after
// them `spread` per sequence add to weights[b, s] the sum over the rows that see key s
// of 2^(u - m) / l, from the logits that the main kernel left, N / 4 lanes per key
// and 4 rows per lane; they work the rows' maxima m and sums l out of the pieces
// themselves rather than wait (and than use lse = m + log2 l, which as one
// number has lost bits).  Bound by latency, a handful of dependent loads: 15 us for
// 32 sequences of up to 16384 keys and 16 rows (17 MB of logits).  Summing in
// the main kernel would need every row's final maximum and sum before its last tile.
constexpr int FIN_THREADS = 256;
constexpr int FIN_BATCH = 4;    // loads in flight per thread (one: 17 us instead of 15)
template <int N>
__global__ void __launch_bounds__(FIN_THREADS) latent_finish_kernel(const LatentAttnParams p, int spread) {
  pdl_enter();
  extern __shared__ float2 s_ml[];  // [rows of a sequence] (-m, 1 / l)
  const int64_t row = blockIdx.x, rows = (int64_t)p.B * p.next_n * p.H;
  const int tid = threadIdx.x;
  if (row == 0 && tid == 0) {
    p.status->last = p.status->now;
    p.status->now = 0;
  }
  if (row < rows) {
    join_row<FIN_THREADS, LA_DC>(p, row, 0);
    return;
  }
  const int R = p.next_n * p.H, b = (int)(row - rows) / spread;
  for (int i = tid; i < R; i += FIN_THREADS) {
    const RowPieces rp(p, (int64_t)b * R + i);
    float m = neg_inf(), sum = 0.f;
    for (int j = 0; j < rp.n; ++j) m = fmaxf(m, p.part_ml[rp.at(p, j)].x);
    const float mm = m == neg_inf() ? 0.f : m;
    for (int j = 0; j < rp.n; ++j) {
      const float2 ml = p.part_ml[rp.at(p, j)];
      sum += ex2(ml.x - mm) * ml.y;
    }
    s_ml[i] = make_float2(-mm, sum == 0.f ? 0.f : 1.f / sum);
  }
  constexpr int LPK = N / 4, KEYS = FIN_THREADS / LPK, STEPS = LT / KEYS;  // lanes per key, keys per step, steps per tile
  bool bad;
  const int len = valid_len(p.seq_lens[b], p.max_pages, bad), tiles = ceil_div(len, LT);
  const int sub = tid % LPK, kk = tid / LPK;
  // FIN_BATCH steps at a time, their loads together: one after the other
  // they were the kernel's time
  const int t0 = (int)(row - rows) % spread, steps = tiles > t0 ? ceil_div(tiles - t0, spread) * STEPS : 0;
  for (int i0 = 0; i0 < steps; i0 += FIN_BATCH) {
    float old[FIN_BATCH], sum[FIN_BATCH];
    int key[FIN_BATCH];
#pragma unroll
    for (int x = 0; x < FIN_BATCH; ++x) {
      const int i = i0 + x;
      key[x] = (t0 + i / STEPS * spread) * LT + i % STEPS * KEYS + kk;
      if (i >= steps || key[x] >= len) key[x] = -1;
      old[x] = sub == 0 && key[x] >= 0 ? p.weights[b * p.ld_weights + key[x]] : 0.f;
      sum[x] = 0.f;
    }
    for (int j = 0; j < p.blocks; ++j) {
      const float* base = p.logits + (int64_t)(b * p.blocks + j) * p.max_pages * LT * N + 4 * sub;
      float4 u[FIN_BATCH];
#pragma unroll
      for (int x = 0; x < FIN_BATCH; ++x)
        u[x] = key[x] >= 0 ? __ldcs(reinterpret_cast<const float4*>(base + (int64_t)key[x] * N))
                           : make_float4(neg_inf(), neg_inf(), neg_inf(), neg_inf());
      if (i0 == 0 && j == 0) __syncthreads();  // s_ml, behind the first loads
#pragma unroll
      for (int x = 0; x < FIN_BATCH; ++x) {
        const int r = j * N + 4 * sub;
        const float v[4] = {u[x].x, u[x].y, u[x].z, u[x].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (r + e < R && v[e] != neg_inf()) sum[x] += ex2(fmaf(v[e], p.scale_log2, s_ml[r + e].x)) * s_ml[r + e].y;
      }
    }
#pragma unroll
    for (int x = 0; x < FIN_BATCH; ++x) {
#pragma unroll
      for (int o = 1; o < LPK; o <<= 1) sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], o);
      if (sub == 0 && key[x] >= 0) p.weights[b * p.ld_weights + key[x]] = old[x] + sum[x];
    }
  }
}

template <int N>
static cudaError_t launch_n(const LatentMaps& m, const LatentAttnParams& p, cudaStream_t s) {
  static DeviceFlags attr_set;
  cudaError_t e = set_smem_attr_once(latent_attn_kernel<N>, LA<N>::SMEM, attr_set);
  if (e != cudaSuccess) return e;
  count_launch();
  e = launch_pdl(latent_attn_kernel<N>, dim3(p.grid), dim3(LA<N>::THREADS), LA<N>::SMEM, s, m, p);
  if (e != cudaSuccess) return e;
  count_launch();
  const int R = p.next_n * p.H, spread = min(p.max_pages, ceil_div(8 * p.grid, p.B));
  if (p.weights)
    return launch_pdl(latent_finish_kernel<N>, dim3((unsigned)(p.B * (R + spread))), dim3(FIN_THREADS), 8 * (size_t)R, s,
                      p, spread);
  // few items, so rows of many pieces: more threads take fewer dims (a sequence of 131072 keys and 16 rows:
  // 37 us, 41 the other way; two of 64 rows 63 and 70).  Else two parts of 256 dims (seven sequences of 128
  // rows, 11 pieces each, 70 us and 79 the first way; 64 sequences behind 32768 shared keys 159 and 183).  128
  // threads for all 512 dims are the best for even lengths (156), but a long sequence among short ones has
  // as many pieces as one alone (the sequence of 131072 keys: 48 us).
  if (p.grid > 32 * (p.prefix_items ? p.prefix_items : p.items))
    return launch_pdl(latent_join_kernel<256, 128, 4>, dim3(p.B * R, LA_DC / 128), dim3(256), 0, s, p);
  return launch_pdl(latent_join_kernel<128, 256, 8>, dim3(p.B * R, LA_DC / 256), dim3(128), 0, s, p);
}

cudaError_t launch_latent_attn(const LatentMaps& m, const LatentAttnParams& p, cudaStream_t s) {
  return p.n == 16 ? launch_n<16>(m, p, s) : p.n == 32 ? launch_n<32>(m, p, s) : launch_n<64>(m, p, s);
}

}  // namespace dsa
