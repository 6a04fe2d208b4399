// latent_api.cu -- C ABI of the latent-attention operators
// (include/dsa_indexer.h): argument validation, per-(device, stream) scratch
// with the status word, and the launches.
#include <cudaTypedefs.h>

#include <algorithm>
#include <map>
#include <mutex>
#include <utility>
#include <vector>

#include "dsa_indexer.h"
#include "latent.h"

using namespace dsa;

namespace {

// Scratch of one (device, stream), and the status of the calls on it.  A buffer that has become too small is kept
// until dsa_indexer_release: a captured graph may still hold its address, and
// growing by half at least bounds what is kept to twice the last size.  The
// status has an allocation of its own that never moves, so that a graph
// captured before the scratch grew reports where the others do.
struct Scratch {
  LatentStatus* status = nullptr;
  uint8_t* base = nullptr;
  size_t cap = 0;
  std::vector<uint8_t*> outgrown;
};
std::mutex g_mu;
std::map<std::pair<int, cudaStream_t>, Scratch> g_scratch;

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Scratch with room for `need` bytes.  Null on an error, and where it would have
// to grow in a capture: an allocation there ends the capture with an error,
// or, where the capture's mode allows it, the clearing of the status would only
// be recorded.
const Scratch* get_scratch(cudaStream_t stream, size_t need) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
  Scratch& a = g_scratch[{dev, stream}];
  if (!a.status || a.cap < need) {
    cudaStreamCaptureStatus capturing;
    if (cudaStreamIsCapturing(stream, &capturing) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    if (capturing != cudaStreamCaptureStatusNone) return nullptr;
  }
  if (!a.status) {
    LatentStatus* p = nullptr;
    if (cudaMalloc(&p, sizeof(*p)) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    if (cudaMemsetAsync(p, 0, sizeof(*p), stream) != cudaSuccess) {
      cudaFree(p);
      return nullptr;
    }
    a.status = p;
  }
  if (a.cap < need) {
    const size_t want = align_up(std::max(need, a.cap + a.cap / 2), 1 << 20);
    uint8_t* p = nullptr;
    if (cudaMalloc(&p, want) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    if (a.base) a.outgrown.push_back(a.base);
    a.base = p;
    a.cap = want;
  }
  return &a;
}

// sm_scale * log2(e) has to be a positive finite number
bool usable_scale(float s) { return s > 0.f && s <= 3.4e38f; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
template <class T>
const __nv_bfloat16* bf(const T* p) {
  return reinterpret_cast<const __nv_bfloat16*>(p);
}

// Arguments shared by the two forms of cached attention.
int check_cached(const LatentAttnParams& p) {
  if (!p.q_nope || !p.q_pe || !p.ckv || !p.kpe || !p.block_table || !p.seq_lens || !p.out || !p.lse) return DSA_ERR_ARG;
  if (p.B <= 0 || p.next_n <= 0 || p.H <= 0 || p.max_pages <= 0 || p.num_pages <= 0) return DSA_ERR_ARG;
  if (!usable_scale(p.scale_log2) || p.ckv_stride < LA_DC || p.kpe_stride < LA_DP || (p.ckv_stride & 7) || (p.kpe_stride & 7))
    return DSA_ERR_ARG;
  if (!aligned16(p.q_nope) || !aligned16(p.q_pe) || !aligned16(p.ckv) || !aligned16(p.kpe) || !aligned16(p.out))
    return DSA_ERR_ARG;
  if (p.weights && p.ld_weights < (int64_t)p.max_pages * PAGE) return DSA_ERR_ARG;
  if (p.weights && (int64_t)p.next_n * p.H > LA_MAX_WEIGHT_ROWS) return DSA_ERR_UNSUPPORTED;
  if ((int64_t)p.B * p.next_n * p.H >= (1ll << 31) / 64 || p.next_n > 65535 || (int64_t)p.max_pages * PAGE >= (1ll << 30) ||
      (int64_t)p.prefix_pages * PAGE >= (1ll << 30) || (int64_t)p.num_pages * PAGE >= (1ll << 31) || p.B > 65535)
    return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// bf16 rows `stride` elements apart, `chunks` of 64 dims each: dims (64, rows,
// chunks), boxes of 64 dims x box_rows x box_chunks in the 128-byte swizzle.
bool tmap_rows(CUtensorMap* m, const void* base, int64_t rows, int64_t stride, int chunks, int box_rows,
               int box_chunks) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)chunks};
  const cuuint64_t strides[2] = {(cuuint64_t)stride * 2, 128};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_chunks};
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, chunks > 1 ? 3 : 2, const_cast<void*>(base), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16 [tokens, heads, dims], boxes of 64 dims x 1 head x box_tokens.
bool tmap_heads(CUtensorMap* m, const void* base, int64_t tokens, int heads, int dims_, int64_t token_stride,
                int64_t head_stride, int box_tokens) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)dims_, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)token_stride * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)box_tokens}, one[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int run_cached(LatentAttnParams& p, cudaStream_t stream) {
  const int rc = check_cached(p);
  if (rc != DSA_OK) return rc;
  const int R = p.next_n * p.H;
  const int64_t rows = (int64_t)p.B * R;
  // the rows of a block: a prefix gathers the rows of the whole batch, so its
  // blocks are full; else the smallest block that holds a sequence's rows
  p.n = p.prefix_table || R > 32 ? 64 : R > 16 ? 32 : 16;
  p.blocks = ceil_div(R, p.n);
  p.prefix_items = p.prefix_table ? (int)((rows + p.n - 1) / p.n) : 0;
  p.items = p.prefix_items + p.B * p.blocks;
  p.grid = std::min(option_grid(), 1024);
  p.item_units = p.prefix_table ? LA_PREFIX_ITEM_UNITS : LA_ITEM_UNITS;
  if ((int64_t)p.items * (std::max(p.max_pages, p.prefix_pages) + p.item_units) >= (1ll << 31) - (1 << 20))
    return DSA_ERR_UNSUPPORTED;
  p.wait_ns = option_wait_ns();
  p.withhold = option_withhold();
  LatentMaps m;
  const int64_t slots = (int64_t)p.num_pages * PAGE;
  if (!tmap_rows(&m.q_nope, p.q_nope, rows, LA_DC, 8, p.n, 8) || !tmap_rows(&m.q_pe, p.q_pe, rows, LA_DP, 1, p.n, 1) ||
      !tmap_rows(&m.ckv, p.ckv, slots, p.ckv_stride, 8, PAGE, 2) ||
      !tmap_rows(&m.kpe, p.kpe, slots, p.kpe_stride, 1, PAGE, 1))
    return DSA_ERR_CUDA;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  const size_t pieces = (size_t)p.items + p.grid;
  const size_t o_per = take(4), o_start = take(4 * ((size_t)p.items + 1) * p.grid), o_ml = take(8 * pieces * p.n),
               o_po = take(4 * (p.prefix_items ? pieces : 2 * (size_t)p.grid) * p.n * LA_DC),
               o_log = p.weights ? take(4 * (size_t)p.B * p.blocks * p.max_pages * PAGE * p.n) : 0;
  std::lock_guard<std::mutex> lk(g_mu);
  const Scratch* scratch = get_scratch(stream, off);
  if (!scratch) return DSA_ERR_CUDA;
  uint8_t* base = scratch->base;
  p.status = scratch->status;
  p.per = reinterpret_cast<int32_t*>(base + o_per);
  p.start = reinterpret_cast<int32_t*>(base + o_start);
  p.part_ml = reinterpret_cast<float2*>(base + o_ml);
  p.part_o = reinterpret_cast<float*>(base + o_po);
  p.logits = p.weights ? reinterpret_cast<float*>(base + o_log) : nullptr;
  return launch_latent_attn(m, p, stream) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace

namespace dsa {
void release_latent_scratch() {
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_scratch.empty()) cudaDeviceSynchronize();
  for (auto& kv : g_scratch) {
    int cur = 0;
    cudaGetDevice(&cur);
    cudaSetDevice(kv.first.first);
    if (kv.second.base) cudaFree(kv.second.base);
    if (kv.second.status) cudaFree(kv.second.status);
    for (uint8_t* q : kv.second.outgrown) cudaFree(q);
    cudaSetDevice(cur);
  }
  g_scratch.clear();
}
}  // namespace dsa

// (an entry lets no C++ exception out: the table of scratch buffers may fail to grow)
extern "C" {

int dsa_latent_attention_paged(const uint16_t* q_nope, const uint16_t* q_pe, const uint16_t* ckv, int64_t ckv_stride,
                               const uint16_t* kpe, int64_t kpe_stride, const int32_t* block_table,
                               const int32_t* seq_lens, int B, int next_n, int H, int max_pages, int num_pages,
                               float sm_scale, uint16_t* out, float* lse, float* weights, int64_t ld_weights,
                               dsa_stream_t stream) try {
  LatentAttnParams p{};
  p.q_nope = bf(q_nope);
  p.q_pe = bf(q_pe);
  p.ckv = bf(ckv);
  p.kpe = bf(kpe);
  p.ckv_stride = ckv_stride;
  p.kpe_stride = kpe_stride;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.B = B;
  p.next_n = next_n;
  p.H = H;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.weights = weights;
  p.ld_weights = ld_weights;
  return run_cached(p, reinterpret_cast<cudaStream_t>(stream));
} catch (...) {
  return DSA_ERR_CUDA;
}

int dsa_latent_attention_shared_prefix(const uint16_t* q_nope, const uint16_t* q_pe, const uint16_t* ckv,
                                       int64_t ckv_stride, const uint16_t* kpe, int64_t kpe_stride,
                                       const int32_t* prefix_table, const int32_t* prefix_len, int prefix_pages,
                                       const int32_t* block_table, const int32_t* seq_lens, int B, int next_n, int H,
                                       int max_pages, int num_pages, float sm_scale, uint16_t* out, float* lse,
                                       dsa_stream_t stream) try {
  if (!prefix_table || !prefix_len || prefix_pages <= 0) return DSA_ERR_ARG;
  LatentAttnParams p{};
  p.q_nope = bf(q_nope);
  p.q_pe = bf(q_pe);
  p.ckv = bf(ckv);
  p.kpe = bf(kpe);
  p.ckv_stride = ckv_stride;
  p.kpe_stride = kpe_stride;
  p.prefix_table = prefix_table;
  p.prefix_len = prefix_len;
  p.prefix_pages = prefix_pages;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.B = B;
  p.next_n = next_n;
  p.H = H;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  return run_cached(p, reinterpret_cast<cudaStream_t>(stream));
} catch (...) {
  return DSA_ERR_CUDA;
}

int dsa_latent_cache_evict(uint16_t* ckv, int64_t ckv_stride, uint16_t* kpe, int64_t kpe_stride, uint8_t* k_cache,
                           float* k_cache_scale, float* weights, int64_t ld_weights, const int32_t* block_table,
                           const int32_t* seq_lens, int B, int max_pages, int num_pages, int budget, int recent,
                           int32_t* kept, int32_t* new_lens, dsa_stream_t stream_) try {
  if (!ckv || !kpe || !weights || !block_table || !seq_lens || !kept || !new_lens || !k_cache != !k_cache_scale)
    return DSA_ERR_ARG;
  if (B <= 0 || max_pages <= 0 || num_pages <= 0 || budget <= 0 || recent < 0 || recent > budget) return DSA_ERR_ARG;
  if (ckv_stride < LA_DC || kpe_stride < LA_DP || (ckv_stride & 7) || (kpe_stride & 7) ||
      ld_weights < (int64_t)max_pages * PAGE)
    return DSA_ERR_ARG;
  if (!aligned16(ckv) || !aligned16(kpe) || !aligned16(k_cache)) return DSA_ERR_ARG;
  // (lengths and the kept list's entries are stepped through with 32-bit indices)
  if ((int64_t)max_pages * PAGE >= (1ll << 30) || (int64_t)num_pages * PAGE >= (1ll << 31) || B > 65535 ||
      budget >= (1 << 30))
    return DSA_ERR_UNSUPPORTED;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  EvictParams p{};
  p.ckv = reinterpret_cast<uint8_t*>(ckv);
  p.kpe = reinterpret_cast<uint8_t*>(kpe);
  p.ckv_stride = 2 * ckv_stride;
  p.kpe_stride = 2 * kpe_stride;
  p.k_cache = k_cache;
  p.k_scale = k_cache_scale;
  p.weights = weights;
  p.ld_weights = ld_weights;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.B = B;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.budget = budget;
  p.recent = recent;
  p.kept = kept;
  p.new_lens = new_lens;
  // CTAs per sequence of the selection
  const int64_t keys = (int64_t)max_pages * PAGE;
  p.cluster = 1;
  while (p.cluster < EVICT_CLUSTER && keys > (int64_t)EVICT_KEYS_PER_CTA * p.cluster) p.cluster *= 2;
  p.cached = (int)std::min<int64_t>(EVICT_CACHED_MAX, keys / p.cluster + 32);
  p.chunks = ceil_div(budget, EVICT_CHUNK);
  if ((int64_t)B * p.chunks >= (1ll << 31) - 1) return DSA_ERR_UNSUPPORTED;
  p.wait_ns = option_wait_ns();
  p.withhold = option_withhold();
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  const size_t o_len = take(4 * (size_t)B), o_w = take(4 * (size_t)B * budget), o_fl = take(4 * (size_t)B * p.chunks),
               o_ti = take(4);
  std::lock_guard<std::mutex> lk(g_mu);
  const Scratch* scratch = get_scratch(stream, off);
  if (!scratch) return DSA_ERR_CUDA;
  uint8_t* base = scratch->base;
  p.old_lens = reinterpret_cast<int32_t*>(base + o_len);
  p.new_w = reinterpret_cast<float*>(base + o_w);
  p.flags = reinterpret_cast<int*>(base + o_fl);
  p.ticket = reinterpret_cast<int*>(base + o_ti);
  p.status = scratch->status;
  return launch_evict(p, stream) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
} catch (...) {
  return DSA_ERR_CUDA;
}

int dsa_latent_attention_prefill(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride,
                                 const uint16_t* k_nope, int64_t kn_token_stride, int64_t kn_head_stride,
                                 const uint16_t* k_pe, int64_t kp_token_stride, const uint16_t* v,
                                 int64_t v_token_stride, int64_t v_head_stride, const int32_t* cu_q,
                                 const int32_t* cu_k, int S, int Tq, int Tk, int H, int causal, float sm_scale,
                                 uint16_t* out, float* lse, dsa_stream_t stream_) try {
  if (!q || !k_nope || !k_pe || !v || !cu_q || !cu_k || !out || !lse) return DSA_ERR_ARG;
  if (S <= 0 || Tq <= 0 || Tk <= 0 || H <= 0 || !usable_scale(sm_scale * 1.4426950408889634f)) return DSA_ERR_ARG;
  // the stride of an axis of one element is never taken, and may be anything
  if (H == 1) q_head_stride = kn_head_stride = v_head_stride = LA_DN + LA_DP;
  if (Tq == 1) q_token_stride = LA_DN + LA_DP;
  if (Tk == 1) kn_token_stride = kp_token_stride = v_token_stride = LA_DN + LA_DP;
  const int64_t strides[] = {q_token_stride, q_head_stride, kn_token_stride, kn_head_stride,
                             kp_token_stride, v_token_stride, v_head_stride};
  for (int64_t x : strides)
    if (x <= 0 || (x & 7) || x >= (1ll << 38)) return DSA_ERR_ARG;
  if (!aligned16(q) || !aligned16(k_nope) || !aligned16(k_pe) || !aligned16(v) || !aligned16(out)) return DSA_ERR_ARG;
  if (H > 65535 || S > 65535 || (int64_t)Tq * H >= (1ll << 31) || Tq >= (1 << 30) || Tk >= (1 << 30))
    return DSA_ERR_UNSUPPORTED;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  PrefillParams p{};
  p.cu_q = cu_q;
  p.cu_k = cu_k;
  p.S = S;
  p.Tq = Tq;
  p.Tk = Tk;
  p.H = H;
  p.causal = causal ? 1 : 0;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.grid = std::max(1, std::min(option_grid(), 1024) / 2);
  p.wait_ns = option_wait_ns();
  p.withhold = option_withhold();
  PrefillMaps m;
  if (!tmap_heads(&m.q, q, Tq, H, LA_DN + LA_DP, q_token_stride, q_head_stride, 128) ||
      !tmap_heads(&m.k_nope, k_nope, Tk, H, LA_DN, kn_token_stride, kn_head_stride, 64) ||
      !tmap_heads(&m.v, v, Tk, H, LA_DV, v_token_stride, v_head_stride, 64) ||
      !tmap_rows(&m.k_pe, k_pe, Tk, kp_token_stride, 1, 64, 1))
    return DSA_ERR_CUDA;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  const size_t o_per = take(8), o_start = take(8 * ((size_t)S + 1) * 2 * p.grid), o_ml = take(8 * 512 * (size_t)p.grid),
               o_po = take(4 * 512 * (size_t)p.grid * LA_DV);
  std::lock_guard<std::mutex> lk(g_mu);
  const Scratch* scratch = get_scratch(stream, off);
  if (!scratch) return DSA_ERR_CUDA;
  uint8_t* base = scratch->base;
  p.status = scratch->status;
  p.per = reinterpret_cast<int64_t*>(base + o_per);
  p.start = reinterpret_cast<int64_t*>(base + o_start);
  p.part_ml = reinterpret_cast<float2*>(base + o_ml);
  p.part_o = reinterpret_cast<float*>(base + o_po);
  return launch_prefill(m, p, stream) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
} catch (...) {
  return DSA_ERR_CUDA;
}

int dsa_latent_last_status(dsa_stream_t stream_) try {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (cudaStreamSynchronize(stream) != cudaSuccess) return DSA_ERR_CUDA;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSA_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_mu);
  auto it = g_scratch.find({dev, stream});
  if (it == g_scratch.end() || !it->second.status) return DSA_OK;
  LatentStatus s;
  if (cudaMemcpy(&s, it->second.status, sizeof(s), cudaMemcpyDeviceToHost) != cudaSuccess) return DSA_ERR_CUDA;
  const int st = s.last;
  if (st & ST_TIMEOUT) return DSA_ERR_TIMEOUT;
  return (st & ST_RANGE) ? DSA_ERR_RANGE : DSA_OK;
} catch (...) {
  return DSA_ERR_CUDA;
}

}  // extern "C"
