// latent_tree.cu -- attention of a tree of drafted tokens over the paged latent
// cache, more than 64 rows (nodes x heads) a sequence.
//
// Formulas, masks and the division into items are latent_attn.cu's.  A row costs
// a key 2176 operations, so from some 256 rows a key on the tensor cores bound the
// call.  There the transposed products of latent_attn.cu run at half rate (M = 64)
// and read shared memory faster than it delivers; here a pair of CTAs
// (cta_group::2, M = 128: 64 rows per CTA) takes blocks of 128 rows against
// tiles of two pages:
//     S [128 x 128 keys] = Q [128 x 576] . K^T     36 steps of 32 cycles
//     O [128 x 512 dims] += P [128 x 128] . V      8 x 2 steps (256 dims) of 64 cycles
// (measured rates; 2193 cycles a tile).  The pair's MMA takes half of its B operand
// from each CTA: a page of keys with all dims for S, half the dims of both
// pages for O.  So a CTA copies a tile's keys in two ways, K and V, into
// rings of their own that give a slot back as soon as its one product is done: two
// tiles kept for both products would not fit beside the queries (74 KB), and
// the L2 delivers the 139 KB a tile in some 1700 cycles (measured: 84 bytes a cycle
// and SM, all SMs at once).  O takes 256 TMEM columns, S two buffers of 64: in both
// lane r and lane 64 + r are row r, with the first and the second half of the columns.
//
// Warps: 0 copies K, 3 copies V (a copy takes a warp some 225 cycles to issue),
// 1 and 2 issue S and O (even CTA), 4-11 softmax, four threads per row.  As in
// latent_attn.cu a row's reference moves only when a logit passes it by 8, which
// a vote of the row's four warps finds out.  Weights are handed over and multiplied 32 keys at
// a time, so that one buffer serves: with a barrier per tile the next tile's
// weights waited for the product (3310 cycles a tile).  The odd CTA announces its
// weights by a copy of 16 bytes that counts on the even one's barrier; an arrival with
// release at cluster scope took 1500 to 4000 cycles (3300 to 4500 a tile; 2490
// this way).
//
// Four sequences of up to 16384 keys, 16 nodes of 128 heads (194 GFLOP): 113 us,
// the tensor cores 76% busy, and 10 to join the pieces; in long runs, which meet
// the power limit, 132 in all, 1.47 PFLOP/s of the 1.70 that a library product
// sustains.  64 sequences of up to 32768 keys, 8 nodes of 16 heads (1.31 GB, read from
// DRAM once): 230 us, 5.7 TB/s, and 9; in long runs 253 to 265.  Prefetching the keys of the tiles
// 1, 2, 3 or 4 ahead into the L2 made both slower (268, 275, 281, 313 for 264).
// Seven sequences with up to 64 nodes of 16 heads (46 GFLOP): 42 and 8 us; the 17
// tiles of a pair of CTAs take 2200 cycles each, the way to the first logits 12000, a
// piece's end 13000 (its masked tiles wait for values to be cleared, then the
// last product, then 4300 for O's way out).  In all of them the blocks of 64 rows of latent_attn.cu took 1.5
// times as long (208, 411 and 77 us).
#include "latent_items.cuh"

namespace dsa {

namespace {

constexpr int TP_ROWS = 128;               // rows per block: 64 per CTA of a pair
constexpr int TP_KEYS = 2 * PAGE;          // keys per tile
constexpr uint32_t TP_CHUNK = 64 * 128;    // 64 rows or keys x 64 dims, bf16
constexpr uint32_t TP_SLOT = 2 * TP_CHUNK;
constexpr int TP_SLOTS = 4;                // of each ring: one tile's
constexpr int TP_WARPS = 12;
constexpr int TP_THREADS = 32 * TP_WARPS;
constexpr int TP_SOFTMAX = 256;            // threads
constexpr float TP_NO_REF = -3.402823466e38f;  // the reference of a row that has seen no key: any logit passes it
constexpr float TP_RESCALE_AT = 8.f;

constexpr uint32_t TP_OFF_Q = 0;
constexpr uint32_t TP_OFF_P = TP_OFF_Q + 9 * TP_CHUNK;   // weights: two chunks of 64 rows x 64 keys
constexpr uint32_t TP_OFF_K = TP_OFF_P + 2 * TP_CHUNK;
constexpr uint32_t TP_OFF_R = TP_OFF_K + TP_SLOTS * TP_SLOT;  // the page's rope parts
constexpr uint32_t TP_OFF_V = TP_OFF_R + TP_CHUNK;
constexpr uint32_t TP_OFF_MISC = TP_OFF_V + TP_SLOTS * TP_SLOT;
// Barriers of the even CTA: K, rope, V and Q full, S empty (per buffer), P full (per 32 keys), O read out; of both: K,
// rope and Q empty, S full (per buffer), product of 32 keys done, a masked tile's values there; drain
constexpr int T_KF = 0, T_KE = T_KF + TP_SLOTS, T_VF = T_KE + TP_SLOTS, T_RF = T_VF + TP_SLOTS, T_RE = T_RF + 1,
              T_QF = T_RE + 1, T_QE = T_QF + 1, T_SF = T_QE + 1, T_SE = T_SF + 2, T_PF = T_SE + 2, T_PD = T_PF + 4,
              T_OE = T_PD + 4, T_Z = T_OE + 1, T_DRAIN = T_Z + 1, T_BARS = T_DRAIN + 2;
constexpr uint32_t TP_OFF_STAT = TP_OFF_MISC + (T_BARS * 8 + 127) / 128 * 128;
constexpr uint32_t TP_OFF_FLAG = TP_OFF_STAT + 128;  // abort, TMEM base
constexpr uint32_t TP_OFF_SEEN = TP_OFF_FLAG + 16;   // [parity][warp] keys that some row of the block sees
constexpr uint32_t TP_OFF_NOTE = TP_OFF_SEEN + 2 * 8 * 8;  // [softmax warp, O issuer] 16 bytes that note_cluster copies
// per group of 32 rows: a masked tile's bits [row][page], then [part][row] maxima or sums
constexpr uint32_t TP_OFF_ROW = (TP_OFF_NOTE + 9 * 16 + 127) / 128 * 128;
constexpr uint32_t TP_SMEM = TP_OFF_ROW + 2 * 512 + 1024;  // + alignment
static_assert(TP_SMEM <= 227 * 1024 && sizeof(Stats) <= 128 && TP_OFF_ROW % 128 == 0, "shared memory per CTA");

constexpr uint32_t TP_D_S = 256;           // TMEM columns: O 0 .. 255, S buffers of 64 from here

// Pages of tiles from k on, a lane each: the page past the cache (whose keys read as zeros) for one that is invalid or
// behind the sequence.
__device__ __forceinline__ int load_pages(const LatentAttnParams& p, const Item& im, int k, int lane, bool& bad) {
  const int j = 2 * k + lane;
  int page = p.num_pages;
  if (j < ceil_div(im.len, PAGE)) {
    page = im.table[j];
    if (page < 0 || page >= p.num_pages) {
      bad = true;
      page = p.num_pages;
    }
  }
  return page;
}

// Tells a barrier of another CTA what this warp has done: a copy of 16 bytes
// that counts on the barrier there.  (An arrival with release at cluster scope
// waits on all of the SM's traffic: 1500 to 4000 cycles beside the copies of keys.)
// What orders a warp's writes before the product that the other CTA issues:
//   1. each lane's fence.proxy.async behind its own writes to shared memory: from
//      here on they are there for the async proxy, through which the copy and the
//      MMA read; tcgen05.wait::st and tcgen05.fence::before_thread_sync behind
//      writes to TMEM, which have then been done
//   2. __syncwarp: every lane's fences come before lane 0 issues the copy
//   3. the copy's bytes land in the other CTA and count on its barrier, whose phase ends
//   4. the lane there that issues the MMA waits for that phase (acquire), then
//      tcgen05.fence::after_thread_sync, and issues
// Steps 1, 2 and 4 are the PTX model's own.  The one between 2 and 3 is a reading: the
// model does not spell out whether writes of other lanes, before a bulk copy was
// issued, are among what its completion releases.  It rests on those writes having
// been done when the copy is issued, in the SM whose shared memory and TMEM the MMA reads
// them from; 35000 random trees, 16 runs each, gave the same bits.  The other way, from
// the issuer that has seen both CTAs' values arrive to the odd CTA's warps, which clear
// some, is alike, with the arrival of the values (their copies' completion, acquired)
// as step 1.
__device__ __forceinline__ void note_cluster(uint32_t dst, uint32_t src, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], 16, [%2];" ::"r"(dst),
               "r"(src), "r"(bar)
               : "memory");
}

}  // namespace

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(TP_THREADS, 1)
    tree_pair_kernel(const __grid_constant__ LatentMaps maps, const LatentAttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + TP_OFF_MISC + 8u * i; };
  volatile int* abort_flag = reinterpret_cast<int*>(smem + TP_OFF_FLAG);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + TP_OFF_FLAG + 4);
  Stats* stats = reinterpret_cast<Stats*>(smem + TP_OFF_STAT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank(), pair = blockIdx.x >> 1;
  auto lead_bar = [&](int i) { return cluster_addr(bar(i), 0); };  // in the even CTA

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    stats->status = 0;
    stats->wait_ns = p.wait_ns;
    tma_prefetch_desc(&maps.q_nope);
    tma_prefetch_desc(&maps.q_pe);
    tma_prefetch_desc(&maps.ckv);
    tma_prefetch_desc(&maps.kpe);
    for (int i = 0; i < T_BARS; ++i)
      mbar_init(bar(i), i == T_SE || i == T_SE + 1 || i == T_OE ? 16 : i >= T_PF && i < T_PD ? 2 : 1);
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
  Runs runs = plan_runs<TP_THREADS, true, TP_KEYS>(p, reinterpret_cast<int*>(smem + TP_OFF_ROW), &stats->status, pair);
  __syncthreads();
  uint32_t it = 0, seg = 0;  // tiles and pieces so far
  int w, k0, k1;
  bool whole;

  if (warp == 0) {
    // --------------------------------------------------- queries and keys --
    // Each CTA copies its part; both report to the even CTA's barriers, whose
    // producer expects the bytes of both.
    bool ok = true;
    while (ok && runs.next(w, k0, k1, whole)) {
      const Item im = load_item<true>(p, w);
      bool bad = false;
      int pages = load_pages(p, im, k0 & ~15, lane, bad);  // (on their way while the queries' copies are issued)
      if (!(ok = mbar_wait_warp(bar(T_QE), (seg & 1) ^ 1, abort_flag, stats))) break;
      if (lane == 0) {
        if (rank == 0) mbar_arrive_expect_tx(bar(T_QF), 2 * 9 * TP_CHUNK);
        tma_load_3d_pair(sbase + TP_OFF_Q, &maps.q_nope, 0, im.row0 + 64 * rank, 0, lead_bar(T_QF));
        tma_load_2d_pair(sbase + TP_OFF_Q + 8 * TP_CHUNK, &maps.q_pe, 0, im.row0 + 64 * rank, lead_bar(T_QF));
      }
      ++seg;
      for (int k = k0; ok && k < k1; ++k, ++it) {
        if (k > k0 && (k & 15) == 0) pages = load_pages(p, im, k, lane, bad);
        const int slot = __shfl_sync(0xffffffffu, pages, 2 * (k & 15) + rank) * PAGE;
        if (!(ok = mbar_wait_warp(bar(T_RE), (it & 1) ^ 1, abort_flag, stats))) break;
        if (lane == 0 && !(p.withhold && it == 0)) {
          if (rank == 0) mbar_arrive_expect_tx(bar(T_RF), 2 * TP_CHUNK);
          tma_load_2d_pair(sbase + TP_OFF_R, &maps.kpe, 0, slot, lead_bar(T_RF));
        }
        for (int c = 0; c < TP_SLOTS; ++c) {
          if (!(ok = mbar_wait_warp(bar(T_KE + c), (it & 1) ^ 1, abort_flag, stats))) break;
          if (lane == 0) {
            if (rank == 0) mbar_arrive_expect_tx(bar(T_KF + c), 2 * TP_SLOT);
            tma_load_3d_pair(sbase + TP_OFF_K + c * TP_SLOT, &maps.ckv, 0, slot, 2 * c, lead_bar(T_KF + c));
          }
        }
      }
      if (__ballot_sync(0xffffffffu, bad) && lane == 0) atomicOr(&stats->status, ST_RANGE);
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------- values --
    // Slot 2 h + n: page h of the tile, dims [256 n + 128 rank, + 128).
    bool ok = true;
    while (ok && runs.next(w, k0, k1, whole)) {
      const Item im = load_item<true>(p, w);
      int pages = 0;
      for (int k = k0; ok && k < k1; ++k, ++it) {
        bool bad;
        if (k == k0 || (k & 15) == 0) pages = load_pages(p, im, k & ~15, lane, bad);
        for (int c = 0; c < TP_SLOTS; ++c) {
          const int slot = __shfl_sync(0xffffffffu, pages, 2 * (k & 15) + (c >> 1)) * PAGE;
          // the products of page h's second half end the use of its slots
          if (!(ok = mbar_wait_warp(bar(T_PD + (c | 1)), (it & 1) ^ 1, abort_flag, stats))) break;
          if (lane == 0) {
            if (rank == 0) mbar_arrive_expect_tx(bar(T_VF + c), 2 * TP_SLOT);
            tma_load_3d_pair(sbase + TP_OFF_V + c * TP_SLOT, &maps.ckv, 0, slot, 4 * (c & 1) + 2 * rank, lead_bar(T_VF + c));
          }
        }
      }
    }
  } else if (warp == 1 && rank == 0) {
    // ----------------------------------------------------------- S issuer --
    constexpr uint32_t ID_S = idesc_bf16_f32(TP_ROWS, TP_KEYS, false, false);
    const uint32_t leader = elect_one();
    const uint32_t q_lo = desc_lo_kmajor(sbase + TP_OFF_Q), r_lo = desc_lo_kmajor(sbase + TP_OFF_R);
    bool ok = true;
    while (ok && runs.next(w, k0, k1, whole)) {
      if (!(ok = mbar_wait_one(leader, bar(T_QF), seg & 1, abort_flag, stats))) break;
      for (int k = k0; k < k1; ++k, ++it) {
        const uint32_t sb = it & 1, d = tmem + TP_D_S + 64 * sb;
        // the softmax has read what was in the buffer
        if (!(ok = mbar_wait_one(leader, bar(T_SE + sb), ((it >> 1) & 1) ^ 1, abort_flag, stats))) break;
        // the rope part first, so that its slot comes free first
        if (!(ok = mbar_wait_one(leader, bar(T_RF), it & 1, abort_flag, stats))) break;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma_bf16_ss_pair(leader, d, q_lo + 8 * (TP_CHUNK >> 4) + 2 * j, r_lo + 2 * j, ID_S, j > 0);
        mma_commit_pair(leader, bar(T_RE));
        for (uint32_t c = 0; c < TP_SLOTS; ++c) {
          if (!(ok = mbar_wait_one(leader, bar(T_KF + c), it & 1, abort_flag, stats))) break;
          tc_fence_after();
          const uint32_t k_lo = desc_lo_kmajor(sbase + TP_OFF_K + c * TP_SLOT);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t at = (j >> 2) * (TP_CHUNK >> 4) + 2 * (j & 3);
            mma_bf16_ss_pair(leader, d, q_lo + 2 * c * (TP_CHUNK >> 4) + at, k_lo + at, ID_S, 1);
          }
          mma_commit_pair(leader, bar(T_KE + c));
        }
        if (!ok) break;
        mma_commit_pair(leader, bar(T_SF + sb));
        if (k == k1 - 1) mma_commit_pair(leader, bar(T_QE));
      }
      ++seg;
    }
  } else if (warp == 2 && rank == 0) {
    // ----------------------------------------------------------- O issuer --
    constexpr uint32_t ID_O = idesc_bf16_f32(TP_ROWS, 256, false, true);
    const uint32_t leader = elect_one();
    const uint32_t p_lo = desc_lo_kmajor(sbase + TP_OFF_P);
    bool ok = true;
    while (ok && runs.next(w, k0, k1, whole)) {
      const Item im = load_item<true>(p, w);
      // the previous piece's O has been read out
      if (!(ok = mbar_wait_one(leader, bar(T_OE), (seg & 1) ^ 1, abort_flag, stats))) break;
      for (int k = k0; ok && k < k1; ++k, ++it) {
        if ((k + 1) * TP_KEYS > im.ctx) {
          // a masked tile: once its values are there, both CTAs' softmax warps may clear those that nobody sees
          for (uint32_t c = 0; ok && c < TP_SLOTS; ++c)
            ok = mbar_wait_one(leader, bar(T_VF + c), it & 1, abort_flag, stats);
          if (!ok) break;
          if (leader) {  // (the lane that acquired them)
            mbar_arrive(bar(T_Z));
            const uint32_t note = sbase + TP_OFF_NOTE + 16 * 8;
            note_cluster(cluster_addr(note, 1), note, cluster_addr(bar(T_Z), 1));
          }
          __syncwarp();
        }
        // 32 keys at a time: their weights' arrival from the other CTA takes some 1500 cycles, in which the buffer of
        // the others is used
        for (uint32_t c = 0; c < 4; ++c) {
          if (!(ok = mbar_wait_one(leader, bar(T_PF + c), it & 1, abort_flag, stats))) break;
          const uint32_t h = c >> 1;
          if (!(c & 1)) {
            ok = mbar_wait_one(leader, bar(T_VF + c), it & 1, abort_flag, stats) &&
                 mbar_wait_one(leader, bar(T_VF + c + 1), it & 1, abort_flag, stats);
            if (!ok) break;
          }
          tc_fence_after();
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const uint32_t v_lo = desc_lo_mnmajor(sbase + TP_OFF_V + (2 * h + n) * TP_SLOT, TP_CHUNK);
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // 16 keys: 32 bytes of a P row, 2 KB of V
              const uint32_t j = 2 * (c & 1) + i;
              mma_bf16_ss_pair(leader, tmem + 128 * n, p_lo + h * (TP_CHUNK >> 4) + 2 * j, v_lo + 128 * j, ID_O,
                               k > k0 || c > 0 || i > 0);
            }
          }
          mma_commit_pair(leader, bar(T_PD + c));
        }
        if (!ok) break;
      }
      ++seg;
    }
  } else if (warp >= 4) {
    // ----------------------------------------------------- softmax warps --
    // Row r = 32 (q & 1) + lane of the CTA in four warps: page q >> 1 of the
    // tile and keys [32 ch, + 32) of it, which meet at a barrier of their group of 32 rows.
    // A wait that gives up leaves the result undefined; the loops still end.
    // From then on the warp's weights are not announced any more (`ok`): the
    // announcement counts on a barrier whose phases end only with the other CTA's
    // bytes, and a second arrival in one phase is an error.
    const int q = warp & 3, ch = (warp - 4) >> 2, g = q & 1, h = q >> 1, r = 32 * g + lane, part = 2 * h + ch;
    const int tid = threadIdx.x - 128, sw = warp - 4;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    uint64_t* s_seen = reinterpret_cast<uint64_t*>(smem + TP_OFF_SEEN);
    uint64_t* s_bits = reinterpret_cast<uint64_t*>(smem + TP_OFF_ROW + 512 * g);  // [lane][page]
    float* s_red = reinterpret_cast<float*>(smem + TP_OFF_ROW + 512 * g);         // [part][lane]
    const uint32_t lead_s = lead_bar(T_SE), lead_p = lead_bar(T_PF + part), lead_o = lead_bar(T_OE);
    const uint32_t note = sbase + TP_OFF_NOTE + 16 * sw, lead_note = cluster_addr(note, 0);
    const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2);
    uint32_t masked = 0;  // masked tiles so far
    bool ok = true;
    while (runs.next(w, k0, k1, whole)) {
      const Item im = load_item<true>(p, w);
      float ref = TP_NO_REF;
      uint64_t l[2] = {0, 0};  // this thread's part of the row's sum, in four parts
      for (int k = k0; k < k1; ++k, ++it) {
        const uint32_t sb = it & 1;
        const bool cut = (k + 1) * TP_KEYS > im.ctx;  // some of the tile's keys are nodes, or behind the last
        uint64_t* seen = s_seen + 8 * (masked & 1);
        if (cut) {
          // Bits of the block's 128 rows, two pages, on their way while the logits are made: this CTA's are kept (a
          // row's by a warp of the group that reads them), and all of them added up, since both CTAs' rows read the
          // values that are cleared.
          const int i = tid & 127, page = tid >> 7;
          const uint64_t bits = tree_bits(p, im, im.r0 + i, 2 * k + page);
          if (i >> 6 == rank) s_bits[2 * lane + page] = bits;
          const uint32_t lo = __reduce_or_sync(0xffffffffu, (uint32_t)bits);
          const uint32_t hi = __reduce_or_sync(0xffffffffu, (uint32_t)(bits >> 32));
          // (two parities: a group may come here for the next masked tile while the other still reads)
          if (lane == 0) seen[sw] = (uint64_t)hi << 32 | lo;
          if (rank == 1 && sw == 0 && lane == 0 && ok) mbar_arrive_expect_tx(bar(T_Z), 16);
        }
        ok &= mbar_wait_warp(bar(T_SF + sb), (it >> 1) & 1, abort_flag, stats);
        tc_fence_after();
        uint32_t s[32];
        tmem_ld32(tmem + TP_D_S + 64 * sb + 32 * ch + lanes, s);
        tmem_wait_ld32(s);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster<false>(lead_s + 8 * sb);
        if (cut) {
          named_bar_sync(1, TP_SOFTMAX);
          const uint32_t mine = (uint32_t)(s_bits[2 * lane + h] >> (32 * ch));
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (!(mine >> c & 1)) s[c] = 0xff800000u;  // -inf
          // keys that no row of the block sees may hold anything, as those past the end: their values become 0 (a
          // weight of 0 does not silence a NaN)
          ok &= mbar_wait_one(lane == 0, bar(T_Z), masked & 1, abort_flag, stats);
          __syncwarp();
          ++masked;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint64_t hidden = ~(seen[4 * x] | seen[4 * x + 1] | seen[4 * x + 2] | seen[4 * x + 3]);
            if (!hidden) continue;
            uint4* v = reinterpret_cast<uint4*>(smem + TP_OFF_V + 2 * x * TP_SLOT);  // four chunks of 64 keys
            for (int e = tid; e < 4 * 64 * 8; e += TP_SOFTMAX)
              if (hidden >> (e >> 3 & 63) & 1) v[e] = make_uint4(0, 0, 0, 0);
          }
          // (any 32 keys' product may start once their own warps have arrived: the others' writes are ready for it at
          // the vote, which comes before every arrival)
          fence_proxy_async_smem();
        }
        float mx[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
        for (int c = 0; c < 32; c += 2)
          mx[(c >> 1) & 3] = fmax3(mx[(c >> 1) & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
        float top = p.scale_log2 * fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (named_bar_or(2 + g, 128, k == k0 || top > ref + TP_RESCALE_AT)) {
          s_red[32 * part + lane] = top;
          named_bar_sync(2 + g, 128);
          top = fmaxf(fmaxf(s_red[lane], s_red[32 + lane]), fmaxf(s_red[64 + lane], s_red[96 + lane]));
          const bool moves = top > ref + TP_RESCALE_AT;
          const float a = moves ? ex2(ref - top) : 1.f;  // 0 from no reference
          if (moves) ref = top;
#pragma unroll
          for (int j = 0; j < 2; ++j) l[j] = fmul2(l[j], pack2(a, a));
          if (k > k0 && __any_sync(0xffffffffu, moves)) {
            ok &= mbar_wait_warp(bar(T_PD + 3), (it - 1) & 1, abort_flag, stats);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t o[16];
              const uint32_t oa = tmem + 128 * ch + 16 * c + lanes;
              tmem_ld16(oa, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * a);
              tmem_st16(oa, o);
            }
            tmem_wait_st();
            tc_fence_before();
          }
          // s_red has been read, and all of the rows' O is ready: any quarter's arrival may start its product
          named_bar_sync(2 + g, 128);
          tc_fence_after();
        }
        // weights: fp32 into the sums, rounded to bf16 (the type of V, which
        // the MMA wants of both operands) for P
        const uint64_t nr2 = pack2(-ref, -ref);
        uint32_t x[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float2 u = unpack2(fma2(pack2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), scale2, nr2));
          const float e0 = ex2(u.x), e1 = ex2(u.y);
          l[j & 1] = fadd2(l[j & 1], pack2(e0, e1));
          const __nv_bfloat162 b = __floats2bfloat162_rn(e0, e1);
          x[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
        // this part of the weight buffer is free once the product that read it last is done
        if (it > 0) ok &= mbar_wait_warp(bar(T_PD + part), (it - 1) & 1, abort_flag, stats);
        uint8_t* row = smem + TP_OFF_P + h * TP_CHUNK + r * 128;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(row + (((4 * ch + j) ^ (r & 7)) << 4)) =
              make_uint4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) {
          if (rank == 0) mbar_arrive_expect_tx(bar(T_PF + part), 16);
          else note_cluster(lead_note, note, lead_p);
        }
      }
      // ---- the piece's result: the row's sum, then O out of TMEM
      const float2 la = unpack2(l[0]), lb = unpack2(l[1]);
      s_red[32 * part + lane] = (la.x + la.y) + (lb.x + lb.y);
      named_bar_sync(2 + g, 128);
      float sum = (s_red[lane] + s_red[32 + lane]) + (s_red[64 + lane] + s_red[96 + lane]);
      const int i = 64 * rank + r;  // row of the block
      const bool row = i < im.nrows, node = row && im.r0 + i < im.nodes * p.H;
      if (!node) sum = 0.f;
      const int64_t piece = (int64_t)w + pair, part_at = 2 * (int64_t)pair + (k0 == 0 ? 1 : 0);
      if (part == 0) {
        if (!whole) p.part_ml[piece * TP_ROWS + i] = make_float2(sum == 0.f ? neg_inf() : ref, sum);
        else if (row) p.lse[im.row0 + i] = sum == 0.f ? neg_inf() : ref + log2f(sum);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      ok &= mbar_wait_warp(bar(T_PD + 3), (it - 1) & 1, abort_flag, stats);
      tc_fence_after();
      const int dim = 256 * ch + 128 * h;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        tmem_ld32(tmem + 128 * ch + 32 * c + lanes, o);
        tmem_wait_ld32(o);
        if (whole) {
          if (row) {
            uint4* dst = reinterpret_cast<uint4*>(p.out + (int64_t)(im.row0 + i) * LA_DC + dim + 32 * c);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t y[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                // (a row that is no node's may hold anything)
                const float a = node ? __uint_as_float(o[8 * j + 2 * e]) * inv : 0.f;
                const float b = node ? __uint_as_float(o[8 * j + 2 * e + 1]) * inv : 0.f;
                const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
                y[e] = *reinterpret_cast<const uint32_t*>(&v);
              }
              dst[j] = make_uint4(y[0], y[1], y[2], y[3]);
            }
          }
        } else if (row) {
          // [piece][dim / 4][row][4]: lanes are rows
          float4* dst = reinterpret_cast<float4*>(p.part_o) + (part_at * (LA_DC / 4) + (dim + 32 * c) / 4) * TP_ROWS + i;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            dst[j * TP_ROWS] = make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]), __uint_as_float(o[4 * j + 2]),
                                 __uint_as_float(o[4 * j + 3]));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster<false>(lead_o);
      named_bar_sync(2 + g, 128);  // s_red has been read
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // before shared memory and TMEM are released, the copies and MMAs
    // already issued land: a last commit of each issuer, and a fixed time for
    // the copies (a barrier of the even CTA counts both CTAs' bytes, of which
    // the other may have issued none)
    const uint64_t until = globaltimer_ns() + DRAIN_ALL_NS;
    if (rank == 0 && (warp == 1 || warp == 2)) {
      mma_commit_pair(elect_one(), bar(T_DRAIN + warp - 1));
      mbar_drain_until(bar(T_DRAIN + warp - 1), 0, until);
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

// The call's last kernel: joins the pieces of cut items, in a fixed order, and
// gives the rows of items without a key their zeros.  CTA (item, 32 rows, 8 /
// PARTS strips of 16 dims): a lane per row, a strip per warp, or, with PARTS = 8, one
// strip of which each warp takes every eighth piece.  A warp takes its pieces in
// turn, rescaling as the maximum moves, so that their values are on the way together
// with their maxima (four at a time).
constexpr int TJ_THREADS = 256;
template <int PARTS>
__global__ void __launch_bounds__(TJ_THREADS) tree_join_kernel(const LatentAttnParams p) {
  pdl_enter();
  __shared__ float s_part[PARTS > 1 ? PARTS - 1 : 1][18][32];  // maximum, sum and 16 dims
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) {
    p.status->last = p.status->now;
    p.status->now = 0;
  }
  const int w = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s0 = p.start[w], s1 = p.start[w + 1], per = *p.per;
  const int b = w / p.blocks, R = p.next_n * p.H, r0 = w % p.blocks * TP_ROWS;
  const int i = 32 * blockIdx.y + lane, part = PARTS > 1 ? warp : 0;
  const int d0 = 16 * (PARTS > 1 ? blockIdx.z : 8 * blockIdx.z + warp);
  const bool row = r0 + i < R;
  // the runs of its first and its last tile
  const int c0 = s1 > s0 ? (s0 + p.item_units) / per : 0, n = s1 > s0 ? (s1 - 1) / per - c0 + 1 : 0;
  if (n == 1) return;  // (its only piece wrote the result)
  float m = neg_inf(), sum = 0.f, o[16];
#pragma unroll
  for (int d = 0; d < 16; ++d) o[d] = 0.f;
  // adds what a piece (or another warp's pieces) has; nothing with a sum of 0, whatever its values
  auto add = [&](float pm, float ps, const float* v) {
    if (ps == 0.f) return;
    const float top = fmaxf(m, pm), a = ex2(m - top), x = ex2(pm - top);  // (a = 0 from no piece)
    m = top;
    sum = sum * a + x * ps;
#pragma unroll
    for (int d = 0; d < 16; ++d) o[d] = o[d] * a + x * v[d];
  };
  constexpr int BATCH = PARTS > 1 ? 4 : 2;
  for (int j0 = part; j0 < n; j0 += BATCH * PARTS) {
    float2 ml[BATCH];
    float4 v[BATCH][4];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int j = j0 + k * PARTS;
      if (j < n && row) {
        const int64_t piece = 2 * (int64_t)(c0 + j) + (j == 0 ? 1 : 0);
        const float4* src = reinterpret_cast<const float4*>(p.part_o) + (piece * (LA_DC / 4) + d0 / 4) * TP_ROWS + i;
        ml[k] = p.part_ml[(int64_t)(w + c0 + j) * TP_ROWS + i];
#pragma unroll
        for (int d = 0; d < 4; ++d) v[k][d] = __ldcs(src + d * TP_ROWS);
      } else {
        ml[k] = make_float2(neg_inf(), 0.f);
      }
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) add(ml[k].x, ml[k].y, &v[k][0].x);
  }
  if constexpr (PARTS > 1) {
    if (part) {
      s_part[part - 1][0][lane] = m;
      s_part[part - 1][1][lane] = sum;
#pragma unroll
      for (int d = 0; d < 16; ++d) s_part[part - 1][2 + d][lane] = o[d];
    }
    __syncthreads();
    if (part) return;
#pragma unroll 1
    for (int k = 0; k < PARTS - 1; ++k) {
      float v[16];
#pragma unroll
      for (int d = 0; d < 16; ++d) v[d] = s_part[k][2 + d][lane];
      add(s_part[k][0][lane], s_part[k][1][lane], v);
    }
  }
  if (!row) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t at = (int64_t)b * R + r0 + i;
  uint32_t y[8];
#pragma unroll
  for (int d = 0; d < 8; ++d) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(o[2 * d] * inv, o[2 * d + 1] * inv);
    y[d] = *reinterpret_cast<const uint32_t*>(&v);
  }
  uint4* dst = reinterpret_cast<uint4*>(p.out + at * LA_DC + d0);
  dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
  dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
  if (d0 == 0) p.lse[at] = sum == 0.f ? neg_inf() : m + log2f(sum);
}

cudaError_t launch_tree_pair(const LatentMaps& m, const LatentAttnParams& p, cudaStream_t s) {
  static DeviceFlags attr_set;
  cudaError_t e = set_smem_attr_once(tree_pair_kernel, TP_SMEM, attr_set);
  if (e != cudaSuccess) return e;
  count_launch();
  e = launch_pdl(tree_pair_kernel, dim3(2 * p.grid), dim3(TP_THREADS), TP_SMEM, s, m, p);
  if (e != cudaSuccess) return e;
  count_launch();
  // Eight warps a strip where rows have many pieces.  The whole call, us in a graph by eight warps and by one, 76 pairs:
  //     blocks      1           2           4           5           6           7           8           16
  //     keys 4096                       21  22      22  22      23  23      24  23
  //         16384                       28  36      36  38      41  43      45  45
  //         32768   21  50      24  43      46  53                  60  62                  78  75      130 120
  // (40 pairs, 16384 keys: 2 blocks 25  28, 3 28  28, 4 32  32, 5 41  39.)
  if (p.grid > 12 * p.items)
    return launch_pdl(tree_join_kernel<8>, dim3(p.items, 4, 32), dim3(TJ_THREADS), 0, s, p);
  return launch_pdl(tree_join_kernel<1>, dim3(p.items, 4, 4), dim3(TJ_THREADS), 0, s, p);
}

}  // namespace dsa
