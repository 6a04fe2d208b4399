// latent_prefill.cu -- causal attention of a ragged batch in the expanded form.
//
// Sequence z has queries [cu_q[z], cu_q[z+1]) and keys [cu_k[z], cu_k[z+1]).
// Query i of n sees keys [0, m - n + i + 1) of the sequence's m (all m without
// the causal mask); a key of head h is (k_nope[s, h] | k_pe[s]), 192 dims,
// its value v[s, h], 128 dims.  Softmax in base 2 as in latent_attn.cu.
//
// 640 operations per (query, key, head): bound by the tensor cores.  A pair of
// CTAs (cta_group::2) takes blocks of 256 queries of one head, 128 per CTA,
// against tiles of 128 keys:
//     S [256 x 128] = Q [256 x 192] . K^T    12 steps
//     O [256 x 128] += P [256 x 128] . V      8 steps
// The pair's MMA splits the B operand: each CTA holds 64 of a tile's keys and
// 64 of the value dims, so a key tile costs 40 KB of shared memory and of copies
// per CTA and three of them fit beside the queries and the output.  S has three
// buffers of 128 columns in TMEM, O the fourth; the weights go back over their
// logits as bf16 and are the second product's A operand there: the logits of the
// next tiles are made while this one's softmax runs, two threads per row.  As in
// latent_attn.cu a row's reference moves only when a logit passes it by 8.
// (One CTA per block with two 128-query tiles and one S buffer each ran at 56%
// tensor time: a tile's next S had to wait for its softmax and its product.  One
// thread per row: 211 us where two take 206, in short runs of the first case below; four 216.
// Loading the next tile's logits while this one's become weights: 215.  Two
// buffers of logits and two of weights instead of three shared ones: 218.)
//
// 2048 queries on 16384 keys of 16 heads: 236 us in long runs, which meet the power
// limit, 1.37 PFLOP/s of the 1.71 that a library product sustains; 206 us in short
// ones, 1.56 of 1.94.  A tile takes some 1620 cycles, 1280 of them the
// tensor cores'; the softmax spends 360 on loading the logits and their maximum,
// 920 on the weights (without the exponentials the call took as long) and 320 on
// waits.  Nine prompts
// of up to 2500 tokens: 91 us, 0.83 PFLOP/s of unmasked work; 38% more is done
// than that in the tiles that the diagonal and the prompts' ends cut, and a
// block's start and end and its two masked tiles cost about three tiles' time.
//
// Every pair takes an equal run of the call's units (a unit: a key tile of a
// block, and PF_BLOCK_UNITS more per block); a block cut by a run's border is
// joined by the merge kernel in the order of its pieces.
#include "latent.h"

namespace dsa {

namespace {

constexpr int PF_ROWS = 256;           // queries per block: 128 per CTA of a pair
constexpr int PF_KEYS = 128;           // keys per tile
// What starting and ending a block costs, in key tiles: nine prompts of up to
// 2500 tokens took 101, 93.1, 90.7 and 92.8 us with 1, 2, 3 and 4.
constexpr int PF_BLOCK_UNITS = 3;
constexpr uint32_t PF_QCHUNK = 128 * 128;  // 128 queries x 64 dims, bf16
constexpr uint32_t PF_SLOT = 64 * 128;     // 64 keys x 64 dims, bf16
constexpr int PF_PER_TILE = 5;         // slots of a key tile: 3 of its 64 keys (192 dims), 2 of 64 value dims
constexpr int PF_SLOTS = 17;
constexpr int PF_BUFS = 3;             // S buffers: with O they fill the 512 TMEM columns
constexpr int PF_WARPS = 16;           // 0 copies, 1 and 2 issue (even CTA), 4-11 softmax, 12-15 output
constexpr int PF_THREADS = 32 * PF_WARPS;
constexpr int PF_ROW_THREADS = 384;    // of the softmax and output warps
constexpr float PF_NO_REF = -3.402823466e38f;  // the reference of a row that has seen no key: any logit passes it
constexpr float PF_RESCALE_AT = 8.f;

constexpr uint32_t PF_OFF_Q = 0;
constexpr uint32_t PF_OFF_RING = PF_OFF_Q + 3 * PF_QCHUNK;
constexpr uint32_t PF_OFF_OUT = PF_OFF_RING + PF_SLOTS * PF_SLOT;  // 128 output rows of 256 bytes
constexpr uint32_t PF_OFF_MISC = PF_OFF_OUT + 128 * 2 * LA_DV;
// Barriers of the even CTA: slot full, q full, P full (per buffer and half), O empty; of both: slot empty, q empty, S
// full, product done (per buffer), values of a sequence's last tile there; drain
constexpr int B_FULL = 0, B_EMPTY = PF_SLOTS, B_QF = 2 * PF_SLOTS, B_QE = B_QF + 1, B_S = B_QE + 1,
              B_P = B_S + PF_BUFS, B_V = B_P + 2 * PF_BUFS, B_O = B_V + PF_BUFS, B_Z = B_O + 1, B_DRAIN = B_Z + PF_BUFS, PF_BARS = B_DRAIN + 2;
constexpr uint32_t PF_OFF_STAT = PF_OFF_MISC + PF_BARS * 8;
constexpr uint32_t PF_OFF_FLAG = PF_OFF_STAT + 128;  // abort, TMEM base
constexpr uint32_t PF_OFF_SCAN = PF_OFF_FLAG + 16;   // PF_WARPS + 1 int64
constexpr uint32_t PF_OFF_ROW = PF_OFF_SCAN + 8 * (PF_WARPS + 2);  // [parity][half][row] reference and sum of a piece
constexpr uint32_t PF_OFF_MAX = PF_OFF_ROW + 4 * 128 * 8;          // [half][row] a tile's maximum
constexpr uint32_t PF_SMEM = PF_OFF_MAX + 2 * 128 * 4 + 1024;      // + alignment
static_assert(PF_SMEM <= 227 * 1024 && sizeof(Stats) <= 128, "shared memory per CTA");

__device__ __forceinline__ float neg_inf() { return -__int_as_float(0x7f800000); }
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

struct Seq {
  int q0, n, k0, m;  // first query and queries, first key and keys
};
// A sequence outside the arrays counts as empty and is reported.
__device__ __forceinline__ Seq load_seq(const PrefillParams& p, int z, bool& bad) {
  const int q0 = p.cu_q[z], q1 = p.cu_q[z + 1], k0 = p.cu_k[z], k1 = p.cu_k[z + 1];
  bad = q0 < 0 || q1 < q0 || q1 > p.Tq || k0 < 0 || k1 < k0 || k1 > p.Tk;
  return bad ? Seq{0, 0, 0, 0} : Seq{q0, q1 - q0, k0, k1 - k0};
}
// Keys that the first `i` queries of a sequence see at most.
__device__ __forceinline__ int keys_seen(const PrefillParams& p, const Seq& s, int i) {
  return p.causal ? max(0, s.m - s.n + min(i, s.n)) : s.m;
}
__device__ __forceinline__ int block_tiles(const PrefillParams& p, const Seq& s, int blk) {
  return ceil_div(keys_seen(p, s, (blk + 1) * PF_ROWS), PF_KEYS);
}

// One pair's pieces: next() gives sequence, head, block and key tiles [k0, k1).
struct Pieces {
  int64_t t, t1, s0;  // next unit, end, first unit of the current block
  int z, h, blk;
  Seq seq;

  __device__ __forceinline__ bool next(const PrefillParams& p, int& k0, int& k1, int& tiles) {
    for (;;) {
      if (t >= t1) return false;
      bool bad;
      while (blk * PF_ROWS >= seq.n) {  // past the last block: next head or sequence
        blk = 0;
        if (++h == p.H) {
          h = 0;
          seq = load_seq(p, ++z, bad);
          if (seq.n == 0) {
            h = p.H - 1;  // an empty sequence has no units
            blk = 1;
          }
        }
      }
      tiles = block_tiles(p, seq, blk);
      const int units = tiles + PF_BLOCK_UNITS;
      if (s0 + units <= t) {  // (only on the way to the first block)
        s0 += units;
        ++blk;
        continue;
      }
      const int u0 = (int)(t - s0), u1 = (int)(min(t1, s0 + units) - s0);
      k0 = max(0, u0 - PF_BLOCK_UNITS);
      k1 = max(0, u1 - PF_BLOCK_UNITS);
      t = s0 + u1;
      if (k1 > k0 || (tiles == 0 && u0 == 0)) return true;  // (an empty block: its rows are written once)
      if (u1 < units) return false;                          // the run ends before the block's first tile
    }
  }
  // what next() left: block `blk` of head h; step past it once its end has been reached
  __device__ __forceinline__ void step(int tiles) {
    if (t == s0 + tiles + PF_BLOCK_UNITS) {
      s0 = t;
      ++blk;
    }
  }
};

// Numbers the units of all sequences (start[], the same in every CTA); the
// pieces of units [c per, (c + 1) per) for c = `pair`.
template <int THREADS>
__device__ __forceinline__ Pieces plan_pieces(const PrefillParams& p, int64_t* start, int pair, int64_t* tmp, int* status) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t base = 0;
  for (int z0 = 0; z0 < p.S; z0 += THREADS) {
    const int z = z0 + tid;
    int64_t units = 0;
    if (z < p.S) {
      bool bad;
      const Seq s = load_seq(p, z, bad);
      if (bad && status) atomicOr(status, ST_RANGE);
      for (int blk = 0; blk * PF_ROWS < s.n; ++blk) units += block_tiles(p, s, blk) + PF_BLOCK_UNITS;
      units *= p.H;
    }
    int64_t x = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) tmp[warp] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
      before += i < warp ? tmp[i] : 0;
      all += tmp[i];
    }
    if (z < p.S) start[z] = base + before + x - units;
    base += all;
  }
  const int64_t per = max((int64_t)(PF_BLOCK_UNITS + 1), (base + p.grid - 1) / p.grid);
  const int64_t t = min(base, pair * per);
  if (tid == 0) {
    start[p.S] = base;
    tmp[THREADS / 32] = 0;
    if (blockIdx.x == 0) *p.per = per;
  }
  __syncthreads();
  for (int z = tid; z < p.S; z += THREADS)
    if (start[z] <= t && t < start[z + 1]) tmp[THREADS / 32] = z;
  __syncthreads();
  Pieces r;
  r.t = t;
  r.t1 = min(base, t + per);
  r.z = (int)tmp[THREADS / 32];
  r.s0 = start[r.z];
  bool bad;
  r.seq = load_seq(p, r.z, bad);
  r.h = 0;
  r.blk = 0;
  if (r.t < r.t1) {  // the head, then (in next) the block
    const int64_t head = (start[r.z + 1] - start[r.z]) / p.H;
    r.h = (int)((t - r.s0) / head);
    r.s0 += r.h * head;
  }
  return r;
}

}  // namespace

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PF_THREADS, 1)
    prefill_kernel(const __grid_constant__ PrefillMaps maps, const PrefillParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + PF_OFF_MISC + 8u * i; };
  volatile int* abort_flag = reinterpret_cast<int*>(smem + PF_OFF_FLAG);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + PF_OFF_FLAG + 4);
  Stats* stats = reinterpret_cast<Stats*>(smem + PF_OFF_STAT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  auto lead_bar = [&](int i) { return cluster_addr(bar(i), 0); };  // in the even CTA

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    stats->status = 0;
    stats->wait_ns = p.wait_ns;
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k_nope);
    tma_prefetch_desc(&maps.k_pe);
    tma_prefetch_desc(&maps.v);
    for (int i = 0; i < 2 * PF_SLOTS + 2; ++i) mbar_init(bar(i), 1);
    for (int i = 0; i < PF_BUFS; ++i) {
      mbar_init(bar(B_S + i), 1);
      mbar_init(bar(B_P + 2 * i), 8);  // four softmax warps of each CTA
      mbar_init(bar(B_P + 2 * i + 1), 8);
      mbar_init(bar(B_V + i), 1);
    }
    mbar_init(bar(B_DRAIN), 1);
    mbar_init(bar(B_DRAIN + 1), 1);
    mbar_init(bar(B_O), 8);
    for (int i = 0; i < PF_BUFS; ++i) mbar_init(bar(B_Z + i), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(s_tmem), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers are ready
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  Pieces pc = plan_pieces<PF_THREADS>(p, p.start + (int64_t)blockIdx.x * (p.S + 1), blockIdx.x >> 1,
                                      reinterpret_cast<int64_t*>(smem + PF_OFF_SCAN), &stats->status);
  uint32_t n_slot = 0, n_q = 0;  // producer: copies armed
  int k0, k1, tiles;
  const uint32_t d_o = tmem + 128 * PF_BUFS;

  if (warp == 0) {
    // ------------------------------------------------------- TMA producer --
    // Each CTA loads its part; both report to the even CTA's barriers, whose
    // producer expects the bytes of both.
    bool ok = true;
    for (; ok && pc.next(p, k0, k1, tiles); pc.step(tiles)) {
      if (k1 <= k0) continue;
      if (!(ok = mbar_wait_warp(bar(B_QE), (n_q & 1) ^ 1, abort_flag, stats))) break;
      if (lane == 0) {
        if (rank == 0) mbar_arrive_expect_tx(bar(B_QF), 2 * 3 * PF_QCHUNK);
        for (int c = 0; c < 3; ++c)
          tma_load_3d_pair(sbase + PF_OFF_Q + c * PF_QCHUNK, &maps.q, 64 * c, pc.h,
                           pc.seq.q0 + pc.blk * PF_ROWS + 128 * rank, lead_bar(B_QF));
      }
      ++n_q;
      for (int k = k0; ok && k < k1; ++k) {
        const int key = pc.seq.k0 + k * PF_KEYS;
        for (int c = 0; c < PF_PER_TILE; ++c, ++n_slot) {
          const int st = n_slot % PF_SLOTS;
          if (!(ok = mbar_wait_warp(bar(B_EMPTY + st), ((n_slot / PF_SLOTS) & 1) ^ 1, abort_flag, stats))) break;
          if (lane == 0 && !(p.withhold && n_slot == 0)) {
            const uint32_t dst = sbase + PF_OFF_RING + st * PF_SLOT, full = lead_bar(B_FULL + st);
            if (rank == 0) mbar_arrive_expect_tx(bar(B_FULL + st), 2 * PF_SLOT);
            if (c < 2)
              tma_load_3d_pair(dst, &maps.k_nope, 64 * c, pc.h, key + 64 * rank, full);
            else if (c == 2)
              tma_load_2d_pair(dst, &maps.k_pe, 0, key + 64 * rank, full);
            else
              tma_load_3d_pair(dst, &maps.v, 64 * rank, pc.h, key + 64 * (c - 3), full);
          }
        }
      }
    }
  } else if (warp == 1 && rank == 0) {
    // ----------------------------------------------------------- S issuer --
    constexpr uint32_t ID_S = idesc_bf16_f32(256, PF_KEYS, false, false);
    const uint32_t leader = elect_one();
    const uint32_t q_lo = desc_lo_kmajor(sbase + PF_OFF_Q);
    uint32_t seg = 0, it = 0;
    bool ok = true;
    for (; ok && pc.next(p, k0, k1, tiles); pc.step(tiles)) {
      if (k1 <= k0) continue;
      if (!(ok = mbar_wait_one(leader, bar(B_QF), seg & 1, abort_flag, stats))) break;
      for (int k = k0; k < k1; ++k, ++it) {
        const uint32_t sb = it % PF_BUFS, sp = it / PF_BUFS & 1;
        // the weights that were in the buffer have been multiplied
        if (!(ok = mbar_wait_warp(bar(B_V + sb), sp ^ 1, abort_flag, stats))) break;
        for (uint32_t c = 0; c < 3; ++c) {
          const uint32_t n = PF_PER_TILE * it + c, st = n % PF_SLOTS;
          if (!(ok = mbar_wait_one(leader, bar(B_FULL + st), (n / PF_SLOTS) & 1, abort_flag, stats))) break;
          tc_fence_after();
          const uint32_t k_lo = desc_lo_kmajor(sbase + PF_OFF_RING + st * PF_SLOT);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_bf16_ss_pair(leader, tmem + 128 * sb, q_lo + c * (PF_QCHUNK >> 4) + 2 * j, k_lo + 2 * j, ID_S,
                             c > 0 || j > 0);
          mma_commit_pair(leader, bar(B_EMPTY + st));
        }
        if (!ok) break;
        mma_commit_pair(leader, bar(B_S + sb));
        if (k == k1 - 1) mma_commit_pair(leader, bar(B_QE));
        if (pc.seq.m - k * PF_KEYS < PF_KEYS) {
          // the sequence ends in this tile: once its values are there, both
          // CTAs' softmax warps may clear what follows (a barrier per S buffer:
          // with blocks of one tile this warp is up to three ends ahead)
          for (uint32_t c = 3; ok && c < 5; ++c) {
            const uint32_t n = PF_PER_TILE * it + c;
            ok = mbar_wait_one(leader, bar(B_FULL + n % PF_SLOTS), (n / PF_SLOTS) & 1, abort_flag, stats);
          }
          if (!ok) break;
          if (leader) {  // (the lane that acquired them)
            mbar_arrive(bar(B_Z + sb));
            mbar_arrive_cluster<true>(cluster_addr(bar(B_Z + sb), 1));
          }
        }
      }
      ++seg;
    }
  } else if (warp == 2 && rank == 0) {
    // ----------------------------------------------------------- O issuer --
    constexpr uint32_t ID_O = idesc_bf16_f32(256, LA_DV, false, true);
    const uint32_t leader = elect_one();
    uint32_t seg = 0, it = 0;
    bool ok = true;
    for (; ok && pc.next(p, k0, k1, tiles); pc.step(tiles)) {
      if (k1 <= k0) continue;
      // the previous piece's O has been read out
      if (!(ok = mbar_wait_one(leader, bar(B_O), (seg & 1) ^ 1, abort_flag, stats))) break;
      for (int k = k0; ok && k < k1; ++k, ++it) {
        const uint32_t sb = it % PF_BUFS, sp = it / PF_BUFS & 1;
        for (uint32_t half = 0; half < 2; ++half) {  // 64 keys: the weights' halves and the values' slots
          const uint32_t n = PF_PER_TILE * it + 3 + half, st = n % PF_SLOTS;
          if (!(ok = mbar_wait_one(leader, bar(B_FULL + st), (n / PF_SLOTS) & 1, abort_flag, stats))) break;
          if (!(ok = mbar_wait_one(leader, bar(B_P + 2 * sb + half), sp, abort_flag, stats))) break;
          tc_fence_after();
          const uint32_t v_lo = desc_lo_mnmajor(sbase + PF_OFF_RING + st * PF_SLOT, PF_SLOT);
#pragma unroll
          for (int j = 0; j < 4; ++j)  // 16 keys: 8 columns of P, 2 KB of V
            mma_bf16_ts_pair(leader, d_o, tmem + 128 * sb + 32 * half + 8 * j, v_lo + 128 * j, ID_O,
                             k > k0 || half > 0 || j > 0);
          mma_commit_pair(leader, bar(B_EMPTY + st));
        }
        if (!ok) break;
        mma_commit_pair(leader, bar(B_V + sb));
      }
      ++seg;
    }
  } else if (warp >= 4 && warp < 12) {
    // ----------------------------------------------------- softmax warps --
    // Two threads per row, 64 keys of a tile each, in two warps that meet at
    // a barrier of their own.  (A wait that gives up leaves the result
    // undefined; the loops still end.)
    const int q = warp & 3, half = (warp - 4) >> 2, r = 32 * q + lane;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    const uint32_t lead_p = lead_bar(B_P) + 8 * half;
    float2* s_row = reinterpret_cast<float2*>(smem + PF_OFF_ROW) + 128 * half + r;
    float* s_max = reinterpret_cast<float*>(smem + PF_OFF_MAX) + r;
    uint32_t it = 0, tails = 0, seg = 0;  // tails: the phase of each buffer's B_Z
    const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2);
    for (; pc.next(p, k0, k1, tiles); pc.step(tiles)) {
      const int first = pc.blk * PF_ROWS + 128 * (int)rank, i = first + r;  // this row's query within its sequence
      const int lim = i < pc.seq.n ? keys_seen(p, pc.seq, i + 1) : 0;
      // what the CTA's first row sees, the least (without rows here nothing matters)
      const int lim0 = first < pc.seq.n ? keys_seen(p, pc.seq, first + 1) : 0x7fffffff;
      float ref = PF_NO_REF;
      uint64_t l[2] = {0, 0};                // this half's sum so far, in four parts
      for (int k = k0; k < k1; ++k, ++it) {
        const uint32_t sb = it % PF_BUFS, sp = it / PF_BUFS & 1;
        const uint32_t d_s = tmem + 128 * sb + lanes;  // the row's logits, then its weights
        mbar_wait_warp(bar(B_S + sb), sp, abort_flag, stats);
        tc_fence_after();
        uint32_t s[64];
        tmem_ld32(d_s + 64 * half, s);
        tmem_ld32(d_s + 64 * half + 32, s + 32);
        tmem_wait_ld32(s);
        tmem_wait_ld32(s + 32);
        if ((k + 1) * PF_KEYS > lim0) {
          const int left = lim - k * PF_KEYS - 64 * half;
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c >= left) s[c] = 0xff800000u;  // -inf
        }
        float mx[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
        for (int c = 0; c < 64; c += 2)
          mx[(c >> 1) & 3] = fmax3(mx[(c >> 1) & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
        float top = p.scale_log2 * fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        // the next sequence's values share its last tile: they become 0 (a
        // weight of 0 does not silence a NaN), in the 64 keys that this half's
        // arrival releases; a CTA's slots hold its value dims of all 128 keys
        const int valid = pc.seq.m - k * PF_KEYS;
        if (valid < PF_KEYS) {
          mbar_wait_one(lane == 0, bar(B_Z + sb), tails >> sb & 1, abort_flag, stats);
          __syncwarp();
          tails ^= 1u << sb;
          uint4* v = reinterpret_cast<uint4*>(smem + PF_OFF_RING + ((PF_PER_TILE * it + 3 + half) % PF_SLOTS) * PF_SLOT);
          for (int x = max(0, valid - 64 * half) * 8 + r; x < 64 * 8; x += 128) v[x] = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          // for the issuer in the other CTA (the arrivals below are relaxed)
          __syncwarp();
          asm volatile("fence.acq_rel.cluster;" ::: "memory");
        }
        // A vote of the two warps: only where a logit passes some row's reference
        // (always in a piece's first tile) are the maxima exchanged.  It also
        // comes between the other half's last read of its logits and the weights
        // that go over them.
        tc_fence_before();
        if (named_bar_or(2 + q, 64, k == k0 || top > ref + PF_RESCALE_AT)) {
          s_max[128 * half] = top;
          named_bar_sync(2 + q, 64);
          top = fmaxf(top, s_max[128 * (half ^ 1)]);
          const bool moves = top > ref + PF_RESCALE_AT;
          const float a = moves ? ex2(ref - top) : 1.f;  // 0 from no reference
          if (moves) ref = top;
#pragma unroll
          for (int j = 0; j < 2; ++j) l[j] = fmul2(l[j], pack2(a, a));
          if (k > k0 && __any_sync(0xffffffffu, moves)) {
            mbar_wait_warp(bar(B_V + (it - 1) % PF_BUFS), (it - 1) / PF_BUFS & 1, abort_flag, stats);
            tc_fence_after();
#pragma unroll 1
            for (int c = 4 * half; c < 4 * half + 4; ++c) {
              uint32_t o[16];
              const uint32_t oa = d_o + lanes + 16 * c;
              tmem_ld16(oa, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * a);
              tmem_st16(oa, o);
            }
            tmem_wait_st();
            tc_fence_before();
          }
          // (either half's arrival may start the product: all of O is ready by
          // then, and s_max has been read)
          named_bar_sync(2 + q, 64);
        }
        tc_fence_after();
        // weights: fp32 into the sums, rounded to bf16 (the type of V, which
        // the MMA wants of both operands) over the logits in TMEM
        const uint64_t nr2 = pack2(-ref, -ref);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int e = 32 * h + 2 * j;
            const float2 x =
                unpack2(fma2(pack2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), scale2, nr2));
            const float e0 = ex2(x.x), e1 = ex2(x.y);
            l[j & 1] = fadd2(l[j & 1], pack2(e0, e1));
            const __nv_bfloat162 b = __floats2bfloat162_rn(e0, e1);
            w[j] = *reinterpret_cast<const uint32_t*>(&b);
          }
          tmem_st16(d_s + 32 * half + 16 * h, w);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster<false>(lead_p + 16 * sb);
      }
      const float2 la = unpack2(l[0]), lb = unpack2(l[1]);
      s_row[256 * (seg++ & 1)] = make_float2(ref == PF_NO_REF ? neg_inf() : ref, (la.x + la.y) + (lb.x + lb.y));
      __syncwarp();
      bar_sync_all<1, PF_ROW_THREADS>();  // (the output warps are done with the piece before)
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------ output warps --
    // Each piece's result, while the softmax warps are at the next piece.
    const int q = warp & 3, r = 32 * q + lane;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    const float2* s_row = reinterpret_cast<const float2*>(smem + PF_OFF_ROW) + r;
    uint32_t it = 0, seg = 0;
    for (; pc.next(p, k0, k1, tiles); pc.step(tiles)) {
      const bool cut = k0 > 0 || k1 < tiles, any = k1 > k0;
      const int64_t piece = 2 * (int64_t)(blockIdx.x >> 1) + (k0 == 0 ? 1 : 0);
      const int first = pc.blk * PF_ROWS + 128 * (int)rank;
      if (any) it += k1 - k0;
      __syncwarp();
      bar_sync_all<1, PF_ROW_THREADS>();
      const float2 rs = s_row[256 * (seg & 1)];
      const float ref = rs.x, sum = rs.y + s_row[256 * (seg & 1) + 128].y;
      ++seg;
      if (cut) {
        p.part_ml[piece * PF_ROWS + 128 * rank + r] = make_float2(ref, sum);
      } else if (first + r < pc.seq.n) {
        p.lse[(int64_t)(pc.seq.q0 + first + r) * p.H + pc.h] =
            sum == 0.f ? neg_inf() : (ref == neg_inf() ? 0.f : ref) + log2f(sum);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      if (any) {
        mbar_wait_warp(bar(B_V + (it - 1) % PF_BUFS), (it - 1) / PF_BUFS & 1, abort_flag, stats);
        tc_fence_after();
      }
      // O out of TMEM, 64 dims at a time; the next piece's may begin once the
      // last are in registers.  Whole blocks go through shared memory, so that a
      // warp writes whole rows (a thread writing its own: 32 lines per
      // instruction, 3000 cycles a block).
      uint4* out = reinterpret_cast<uint4*>(smem + PF_OFF_OUT) + 16 * 32 * q;  // this warp's 32 rows of 16 x 16 bytes
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t o[64];
        if (any) {
          tmem_ld32(d_o + lanes + 64 * h, o);
          tmem_ld32(d_o + lanes + 64 * h + 32, o + 32);
          tmem_wait_ld32(o);
          tmem_wait_ld32(o + 32);
          if (h == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster<false>(lead_bar(B_O));
          }
        } else {
#pragma unroll
          for (int c = 0; c < 64; ++c) o[c] = 0;
        }
        if (cut) {
          // [piece][dim / 4][row][4]: lanes are rows
          float4* dst = reinterpret_cast<float4*>(p.part_o) + (piece * 32 + 16 * h) * PF_ROWS + 128 * rank + r;
#pragma unroll
          for (int c = 0; c < 16; ++c)
            dst[c * PF_ROWS] = make_float4(__uint_as_float(o[4 * c]), __uint_as_float(o[4 * c + 1]),
                                           __uint_as_float(o[4 * c + 2]), __uint_as_float(o[4 * c + 3]));
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(o[8 * c + 2 * j]) * inv,
                                                             __uint_as_float(o[8 * c + 2 * j + 1]) * inv);
              w[j] = *reinterpret_cast<const uint32_t*>(&b);
            }
            out[16 * lane + ((8 * h + c) ^ (lane & 15))] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (!cut) {
        __syncwarp();
        const int left = pc.seq.n - (first + 32 * q);  // rows of this warp that exist
        uint4* dst = reinterpret_cast<uint4*>(p.out + ((int64_t)(pc.seq.q0 + first + 32 * q) * p.H + pc.h) * LA_DV);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const int x = 2 * c + (lane >> 4);
          if (x < left) dst[(int64_t)x * p.H * 16 + (lane & 15)] = out[16 * x + ((lane & 15) ^ (x & 15))];
        }
        __syncwarp();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // before shared memory and TMEM are released, the copies and MMAs
    // already issued land: a last commit, and the last phase armed on each
    // slot.  Those count both CTAs' bytes, and a phase of which the other CTA
    // issued no copy never completes, nor can the odd CTA wait for its own:
    // both give copies in flight a fixed time as well.
    const uint64_t until = globaltimer_ns() + DRAIN_ALL_NS;
    if (rank == 0) {
      if (warp == 0 && lane == 0) {
        for (uint32_t s = 0; s < PF_SLOTS; ++s)
          if (n_slot > s) mbar_drain_until(bar(B_FULL + s), ((n_slot - 1 - s) / PF_SLOTS) & 1, until);
        if (n_q) mbar_drain_until(bar(B_QF), (n_q - 1) & 1, until);
      } else if (warp == 1 || warp == 2) {
        mma_commit_pair(elect_one(), bar(B_DRAIN + warp - 1));
        mbar_drain_until(bar(B_DRAIN + warp - 1), 0, until);
      }
    }
    while (globaltimer_ns() < until) __nanosleep(1000);
    __syncthreads();
  }
  if (threadIdx.x == 0 && stats->status) atomicOr(&p.status->now, stats->status);
  cluster_sync_all();  // nothing of the pair is in flight any more
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// Joins the pieces of cut blocks.  CTA (c, y): if the border between the runs
// of c and c + 1 is the first inside some block, rows [32 y, + 32) of it; a
// lane per row, 16 dims per warp.
constexpr int PM_THREADS = 256;
__global__ void __launch_bounds__(PM_THREADS) prefill_merge_kernel(const PrefillParams p) {
  pdl_enter();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {  // the call's last kernel
    p.status->last = p.status->now;
    p.status->now = 0;
  }
  const int64_t per = *p.per, total = p.start[p.S], t = (blockIdx.x + 1) * per;  // the unit after the border
  if (t >= total) return;
  int lo = 0, hi = p.S - 1;  // the last sequence that starts at or before t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.start[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  bool bad;
  const Seq seq = load_seq(p, lo, bad);
  int64_t s0 = p.start[lo];
  const int64_t head = (p.start[lo + 1] - s0) / p.H;
  const int h = (int)((t - s0) / head);
  s0 += h * head;
  int blk = 0, tiles = block_tiles(p, seq, 0);
  while (s0 + tiles + PF_BLOCK_UNITS <= t) {
    s0 += tiles + PF_BLOCK_UNITS;
    tiles = block_tiles(p, seq, ++blk);
  }
  // pieces: the CTA of the block's first tile, then every one up to that of its last
  const int64_t c0 = (s0 + PF_BLOCK_UNITS) / per, c1 = (s0 + PF_BLOCK_UNITS + tiles - 1) / per;
  if (tiles == 0 || c0 != blockIdx.x || c1 == c0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = 32 * blockIdx.y + lane, i = blk * PF_ROWS + r;
  if (blk * PF_ROWS + 32 * (int)blockIdx.y >= seq.n) return;
  auto at = [&](int64_t c) { return 2 * c + (c == c0 ? 1 : 0); };
  float m = neg_inf();
  for (int64_t c = c0; c <= c1; ++c) m = fmaxf(m, p.part_ml[at(c) * PF_ROWS + r].x);
  const float mm = m == neg_inf() ? 0.f : m;
  float sum = 0.f, o[16];
#pragma unroll
  for (int d = 0; d < 16; ++d) o[d] = 0.f;
  for (int64_t c = c0; c <= c1; ++c) {
    const float2 ml = p.part_ml[at(c) * PF_ROWS + r];
    const float x = ex2(ml.x - mm);
    sum += x * ml.y;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const float4 v = __ldcs(reinterpret_cast<const float4*>(p.part_o) + (at(c) * 32 + 4 * warp + d) * PF_ROWS + r);
      if (x != 0.f) {
        o[4 * d] += x * v.x;
        o[4 * d + 1] += x * v.y;
        o[4 * d + 2] += x * v.z;
        o[4 * d + 3] += x * v.w;
      }
    }
  }
  if (i >= seq.n) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t row = (int64_t)(seq.q0 + i) * p.H + h;
  uint32_t w[8];
#pragma unroll
  for (int d = 0; d < 8; ++d) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(o[2 * d] * inv, o[2 * d + 1] * inv);
    w[d] = *reinterpret_cast<const uint32_t*>(&v);
  }
  uint4* dst = reinterpret_cast<uint4*>(p.out + row * LA_DV + 16 * warp);
  dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
  dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  if (warp == 0) p.lse[row] = sum == 0.f ? neg_inf() : mm + log2f(sum);
}

cudaError_t launch_prefill(const PrefillMaps& m, const PrefillParams& p, cudaStream_t s) {
  static DeviceFlags attr_set;
  cudaError_t e = set_smem_attr_once(prefill_kernel, PF_SMEM, attr_set);
  if (e != cudaSuccess) return e;
  count_launch();
  e = launch_pdl(prefill_kernel, dim3(2 * p.grid), dim3(PF_THREADS), PF_SMEM, s, m, p);
  if (e != cudaSuccess) return e;
  count_launch();
  return launch_pdl(prefill_merge_kernel, dim3(p.grid, PF_ROWS / 32), dim3(PM_THREADS), 0, s, p);
}

}  // namespace dsa
