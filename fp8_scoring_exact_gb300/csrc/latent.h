// latent.h -- parameters and host launchers of the latent-attention operators:
// dense attention over the paged latent cache (latent_attn.cu), eviction from
// that cache (cache_evict.cu), prefill in the expanded form (latent_prefill.cu),
// new tokens encoded and appended (token_encode.cu) and the accepted path of
// drafted ones (cache_accept.cu).  Their entry points are in latent_api.cu.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"

namespace dsa {

constexpr int LA_DC = 512;             // compressed dims of a latent key (keys and values)
constexpr int LA_DP = 64;              // its rope dims (keys only)
constexpr int LA_DN = 128, LA_DV = 128;  // expanded form: no-rope key dims and value dims of a head

// Status of a latent operator's call: its kernels OR into `now`; the last one
// moves it to `last` and leaves `now` zero for the next call (also when the
// call is replayed from a graph).  An eviction's last kernel can itself give up
// waiting: its CTAs OR into `last`, which the selection has cleared.
// A call of one kernel collects its status in the CTA that ends last, which `ticket` finds out: the CTAs of a call add
// up to 2^32, each a share, and the last one brings the count back to 0.  So it is 0 again behind any calls that have
// ended, those too that ran beside each other where they must not (a count of CTAs would be left out of step with every
// later call).  (A kernel behind each call instead: 0.7 us less on the device, 3 to 6 us more for the host.)
struct LatentStatus {
  int now, last;
  unsigned ticket;
};
#ifdef __CUDACC__
// Ends a call of one kernel: the CTA that is the last to come here collects the call's status, and gets true; what
// every CTA read and wrote before is behind it.
__device__ __forceinline__ bool last_cta(LatentStatus* st, bool bad) {
  __shared__ int s_last;
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) {
    if (any) atomicOr(&st->now, ST_RANGE);
    __threadfence();
    s_last = gridDim.x == 1;
    if (gridDim.x > 1) {
      unsigned share = 0xffffffffu / gridDim.x;
      if (blockIdx.x == 0) share -= share * gridDim.x;  // and what the others' shares leave of 2^32
      s_last = atomicAdd(&st->ticket, share) + share == 0;
    }
    if (s_last) {
      __threadfence();
      st->last = atomicExch(&st->now, 0);
    }
  }
  __syncthreads();
  return s_last;
}
#endif

// Row blocks of cached attention: an item is a block of up to n rows with the keys
// its rows see, cut into tiles: 16, 32 or 64 rows and tiles of one page, or, of
// trees with more rows a sequence, 128 rows and tiles of two pages.  An item with
// tiles counts item_units units and one per tile; the items' units are
// numbered through, and run c takes units [c per, (c + 1) per): its tiles in one item
// are a piece, whose id is item + c.  A run is a CTA's, or, with 128 rows, that of a
// pair of CTAs (cta_group::2).
// What starting and ending a piece costs, in tiles: 2 without a prefix (128 rows of seven sequences: 70.2 us; 70.7 with
// 4); 4 with one, where most of a sequence's own items are short and their pages cold (64 sequences behind 32768 shared
// keys: 171 us with 2, 163 with 3, 159 with 4, 163 with 8).
constexpr int LA_ITEM_UNITS = 2, LA_PREFIX_ITEM_UNITS = 4;
constexpr int LA_MAX_WEIGHT_ROWS = 4096;  // rows of a sequence with key weights (their sums lie in shared memory)

// Process-wide options and the launch counter (api.cu).
uint64_t option_wait_ns();
int option_withhold();
int option_grid();  // CTAs of the persistent kernels: the option, else the SM count
void count_launch();
// Frees the scratch of the latent operators (latent_api.cu); called by dsa_indexer_release.
void release_latent_scratch();

// Attention of every sequence's next_n query tokens over its cached keys, in
// the absorbed form; with a prefix, over the prefix keys and then its own.
struct LatentAttnParams {
  const __nv_bfloat16* q_nope;  // [B, next_n, H, 512]
  const __nv_bfloat16* q_pe;    // [B, next_n, H, 64]
  const __nv_bfloat16* ckv;     // slot-major, ckv_stride elements per slot
  const __nv_bfloat16* kpe;
  int64_t ckv_stride, kpe_stride;
  const int32_t* prefix_table;  // [prefix_pages] (null: no prefix)
  const int32_t* prefix_len;    // [1]
  int prefix_pages;
  const int32_t* block_table;   // [B, max_pages]
  const int32_t* seq_lens;      // [B]
  int B, next_n, H, max_pages, num_pages;
  float scale_log2;             // sm_scale * log2(e)
  __nv_bfloat16* out;           // [B, next_n, H, 512]
  float* lse;                   // [B, next_n, H]
  float* weights;               // [B, ld_weights] or null: += the softmax weight of every key
  int64_t ld_weights;
  LatentStatus* status;
  // a tree of drafted tokens: the sequence's last keys (null tree_mask: next_n tokens in a row)
  const uint64_t* tree_mask;    // [B, next_n, mask_words]: node i sees node j where bit j % 64 of word j / 64 is set
  const int32_t* draft_lens;    // [B] nodes of a sequence, or null: next_n, or all its keys if it has fewer
  int mask_words;
  // the call's row blocks and scratch
  int n;                        // rows per block (128: of a pair of CTAs; grid then counts pairs)
  int prefix_items, blocks;     // row blocks over the prefix (all sequences' rows), and per sequence
  int items, grid, item_units;
  uint64_t wait_ns;
  int withhold;                 // test option: the first keys are never loaded (a wait must run out)
  int32_t* per;                 // [1] units per CTA
  // [grid, items + 1] ([2 grid, items + 1] for pairs of CTAs) first unit of each item, worked out by every CTA for itself
  int32_t* start;
  // unnormalised outputs of the pieces: with a prefix all of them, [items + grid, n, 512]; without one those of cut items,
  // of which a run has two at most, [2 grid, n, 512] (1: the one that starts with its item's first tile); a pair's pieces
  // are [512 / 4 dims, 128 rows, 4] each
  float* part_o;
  float2* part_ml;              // [items + grid, n]: reference maximum (base-2 units) and sum
  float* logits;                // [B, blocks, max_pages, 64, n] unscaled logits (-inf: not seen), for the key weights
};

constexpr int EVICT_CLUSTER = 8;           // CTAs per sequence of the selection at most
constexpr int EVICT_KEYS_PER_CTA = 16384;  // a sequence's CTAs double while each has more than that
constexpr int EVICT_CACHED_MAX = 32768;  // weights a CTA of the selection holds at most (128 KB)
constexpr int EVICT_CHUNK = 64;

// Eviction in place: every sequence of more than `budget` keys keeps its last
// `recent` keys and the budget - recent others with the largest weights.
struct EvictParams {
  uint8_t* ckv;                 // slot-major rows of 1024 bytes, ckv_stride bytes apart
  uint8_t* kpe;                 // rows of 128 bytes
  int64_t ckv_stride, kpe_stride;
  uint8_t* k_cache;             // indexer keys [P, 64, 128] or null
  float* k_scale;               // [P, 64] or null
  float* weights;               // [B, ld_weights]
  int64_t ld_weights;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int B, max_pages, num_pages, budget, recent;
  int32_t* kept;                // [B, budget]
  int32_t* new_lens;            // [B]
  int cluster, cached;          // CTAs per sequence of the selection; weights each holds in shared memory
  int chunks;                   // of EVICT_CHUNK kept keys, per sequence
  uint64_t wait_ns;
  int withhold;                 // test option: a sequence's first chunk never says that it has been read
  int32_t* old_lens;            // [B] scratch: the validated lengths (new_lens may be seq_lens itself)
  float* new_w;                 // [B, budget] the kept keys' weights
  int* flags;                   // [B, chunks] 1: the chunk's keys have been read
  int* ticket;                  // [1] chunks handed out
  LatentStatus* status;
};

// Causal attention of a ragged batch in the expanded form (a key of a head:
// 128 dims of its own and 64 rope dims shared by the heads).
struct PrefillParams {
  const int32_t *cu_q, *cu_k;   // [S + 1]
  int S, Tq, Tk, H, causal;
  float scale_log2;
  __nv_bfloat16* out;           // [Tq, H, 128]
  float* lse;                   // [Tq, H]
  int grid;                     // pairs of CTAs
  uint64_t wait_ns;
  int withhold;                 // test option: the first keys are never loaded (a wait must run out)
  int64_t* per;                 // [1] units per pair
  int64_t* start;               // [2 grid, S + 1] first unit of each sequence, worked out by every CTA for itself
  float* part_o;                // [2 grid, 128 / 4, 256, 4] unnormalised outputs of the pieces of cut blocks
  float2* part_ml;              // [2 grid, 256]: reference maximum (base-2 units) and sum
  LatentStatus* status;
};

// How rows of 128 dims are encoded for the indexer.
struct RowEncoding {
  const float *norm_w, *norm_b;  // [128] LayerNorm, or null
  float eps;
  bool pairs, hadamard;          // rotated pairs (2 i, 2 i + 1), else (i, i + 32); Hadamard transform behind
};

// Rows of T tokens encoded for the indexer, and rope parts of the same tokens rotated.
struct EncodeParams {
  const __nv_bfloat16* x;        // [T, G, 128] or null
  int64_t x_token, x_head;       // strides in elements
  int G;                         // 64 or 1
  RowEncoding enc;
  const __nv_bfloat16* pe;       // [T, H, 64] or null
  int64_t pe_token, pe_head;
  int H;
  bool pe_pairs;
  const float* cos_sin;          // [max_positions, 64]: 32 cosines, 32 sines
  int max_positions;
  const int32_t* positions;      // [T]; negative: padding
  int T;
  uint8_t* codes;                // [T, G, 128]
  float* scale;                  // [T]
  __nv_bfloat16* pe_out;         // [T, H, 64], may be pe
  int64_t po_token, po_head;
  int index_ctas;                // CTAs that encode; the rest rotate
  LatentStatus* status;
};

// New tokens into the paged cache: sequence b's tokens [cu_new[b], cu_new[b + 1]) behind its seq_lens[b] keys.
struct AppendParams {
  const __nv_bfloat16 *c, *k_pe, *index_k;  // [T, 512], [T, 64], [T, 128] or null
  int64_t c_stride, kp_stride, ik_stride;
  const float* c_norm;           // [512] RMSNorm, or null
  float c_eps;
  RowEncoding enc;
  bool pe_pairs;
  const float* cos_sin;
  int max_positions;
  const int32_t* positions;      // [T], or null: a token's logical slot
  const int32_t *cu_new, *block_table, *seq_lens;
  int B, T, max_pages, num_pages;
  __nv_bfloat16 *ckv, *kpe;
  int64_t ckv_stride, kpe_stride;
  uint8_t* k_cache;              // [P, 64, 128] or null
  float* k_scale;
  __nv_bfloat16 *c_out, *k_pe_out;  // [T, 512], [T, 64]: what the cache gets, or null
  int64_t c_out_stride, kp_out_stride;
  int32_t* new_lens;             // [B], may be seq_lens
  int row_ctas;                  // CTAs that rotate and encode; the rest normalise latents
  LatentStatus* status;
};

// The accepted path of every sequence's drafted nodes, moved together behind its settled keys.
struct AcceptParams {
  uint8_t *ckv, *kpe;            // rows of 1024 and 128 bytes
  int64_t ckv_stride, kpe_stride;  // bytes
  uint8_t* k_cache;              // [P, 64, 128] or null
  float* k_scale;
  const int32_t *block_table, *seq_lens, *draft_lens;
  const int32_t* path;           // [B, max_path] nodes, ascending
  const int32_t* path_lens;      // [B]
  int B, max_pages, num_pages, max_path;
  int32_t* new_lens;             // [B], may be seq_lens
  LatentStatus* status;
};

// Tensor maps of cached attention: queries [rows, 512] and [rows, 64], caches
// [slots, 512] and [slots, 64], all bf16 in 128-byte swizzled boxes of 64 dims.
struct LatentMaps {
  CUtensorMap q_nope, q_pe, ckv, kpe;
};
cudaError_t launch_latent_attn(const LatentMaps& m, const LatentAttnParams& p, cudaStream_t s);
// Trees of more than 64 rows a sequence (p.n = 128): runs of pairs of CTAs.
cudaError_t launch_tree_pair(const LatentMaps& m, const LatentAttnParams& p, cudaStream_t s);
cudaError_t launch_evict(const EvictParams& p, cudaStream_t s);
cudaError_t launch_encode(const EncodeParams& p, cudaStream_t s);
cudaError_t launch_append(AppendParams p, cudaStream_t s);
cudaError_t launch_accept(const AcceptParams& p, cudaStream_t s);
// Tensor maps of the expanded form: q [Tq, H, 192], k_nope and v [Tk, H, 128],
// boxes of 64 dims x 1 head x 128 queries or 64 keys; k_pe [Tk, 64].
struct PrefillMaps {
  CUtensorMap q, k_nope, k_pe, v;
};
cudaError_t launch_prefill(const PrefillMaps& m, const PrefillParams& p, cudaStream_t s);

}  // namespace dsa
