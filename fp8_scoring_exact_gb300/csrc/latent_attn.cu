// latent_attn.cu -- attention over the paged latent cache in the absorbed form.
//
// Row (b, i, h), the query of head h at token i of sequence b, sees the
// prefix keys (if any) and then the logical keys [0, seq_lens[b] - next_n + i
// + 1) of its sequence; with u_s = scale_log2 * (q_nope . ckv[s] + q_pe .
// kpe[s]) its output is sum_s 2^(u_s - lse) ckv[s], lse = log2(sum_s 2^u_s).
// A row that sees no key gets zeros and lse = -inf.
//
// One CTA per row, one warp per key at a time: lane l holds dims [16 l, + 16)
// of the query, of the running output and of the key, and 2 rope dims; running
// maximum and sum in base 2 per warp, joined at the end.
#include "latent.h"

namespace dsa {

namespace {
constexpr int LR_WARPS = 8;
__device__ __forceinline__ float neg_inf() { return -__int_as_float(0x7f800000); }

__device__ __forceinline__ void load16(const __nv_bfloat16* src, float* f) {
  const uint4* p = reinterpret_cast<const uint4*>(src);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 v = p[i];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
      f[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ float2 load2(const __nv_bfloat16* src) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(src));
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Validated length of sequence b (an invalid one counts as empty and is reported).
__device__ __forceinline__ int seq_len(const LatentAttnParams& p, int b) {
  const int len = p.seq_lens[b];
  if (len >= 0 && len <= (int64_t)p.max_pages * PAGE) return len;
  atomicOr(p.status, ST_RANGE);
  return 0;
}
__device__ __forceinline__ int prefix_len(const LatentAttnParams& p) {
  if (!p.prefix_table) return 0;
  const int len = *p.prefix_len;
  if (len >= 0 && len <= (int64_t)p.prefix_pages * PAGE) return len;
  atomicOr(p.status, ST_RANGE);
  return 0;
}
// Slot of logical key s of a table, -1 for a page outside the cache (reported; its keys read as zeros).
__device__ __forceinline__ int64_t slot_of(const LatentAttnParams& p, const int32_t* table, int s) {
  const int page = table[s / PAGE];
  if (page >= 0 && page < p.num_pages) return (int64_t)page * PAGE + s % PAGE;
  atomicOr(p.status, ST_RANGE);
  return -1;
}

struct Key {
  float c[16];
  float2 e;
};
__device__ __forceinline__ void load_key(const LatentAttnParams& p, int64_t slot, int lane, Key& k) {
  if (slot < 0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) k.c[i] = 0.f;
    k.e = make_float2(0.f, 0.f);
    return;
  }
  load16(p.ckv + slot * p.ckv_stride + 16 * lane, k.c);
  k.e = load2(p.kpe + slot * p.kpe_stride + 2 * lane);
}
__device__ __forceinline__ float dot(const Key& a, const Key& b) {
  float x = a.e.x * b.e.x + a.e.y * b.e.y;
#pragma unroll
  for (int i = 0; i < 16; ++i) x += a.c[i] * b.c[i];
  return warp_sum(x);
}
}  // namespace

__global__ void __launch_bounds__(32 * LR_WARPS) latent_rows_kernel(const LatentAttnParams p) {
  pdl_enter();
  __shared__ float s_m[LR_WARPS], s_l[LR_WARPS], s_o[LR_WARPS][LA_DC];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  const int tok = (int)(row / p.H), b = tok / p.next_n, i = tok % p.next_n;
  const int32_t* table = p.block_table + (int64_t)b * p.max_pages;
  const int pre = prefix_len(p);
  const int own = max(0, seq_len(p, b) - p.next_n + i + 1);
  Key q, k;
  load16(p.q_nope + row * LA_DC + 16 * lane, q.c);
  q.e = load2(p.q_pe + row * LA_DP + 2 * lane);
  float m = neg_inf(), l = 0.f, c = 0.f, o[16];
#pragma unroll
  for (int d = 0; d < 16; ++d) o[d] = 0.f;
  for (int64_t s = warp; s < (int64_t)pre + own; s += LR_WARPS) {
    load_key(p, s < pre ? slot_of(p, p.prefix_table, (int)s) : slot_of(p, table, (int)(s - pre)), lane, k);
    const float u = dot(q, k) * p.scale_log2;
    const float m_new = fmaxf(m, u);
    const float mm = m_new == neg_inf() ? 0.f : m_new;
    const float a = exp2f(m - mm), w = exp2f(u - mm);
    m = m_new;
    // compensated: over many keys of nearly equal weight a plain sum would
    // lose the weights' differences
    l *= a;
    const float y = w - c * a, sum = l + y;
    c = (sum - l) - y;
    l = sum;
#pragma unroll
    for (int d = 0; d < 16; ++d) o[d] = o[d] * a + w * k.c[d];
  }
#pragma unroll
  for (int d = 0; d < 16; ++d) s_o[warp][16 * lane + d] = o[d];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  float M = neg_inf(), L = 0.f;
  for (int w = 0; w < LR_WARPS; ++w) M = fmaxf(M, s_m[w]);
  const float mm = M == neg_inf() ? 0.f : M;
  for (int w = 0; w < LR_WARPS; ++w) L += exp2f(s_m[w] - mm) * s_l[w];
  const float inv = L > 0.f ? 1.f / L : 0.f;
  for (int d = threadIdx.x; d < LA_DC; d += blockDim.x) {
    float x = 0.f;
    for (int w = 0; w < LR_WARPS; ++w) x += exp2f(s_m[w] - mm) * s_o[w][d];
    p.out[row * LA_DC + d] = __float2bfloat16(x * inv);
  }
  if (threadIdx.x == 0) p.lse[row] = L > 0.f ? M + log2f(L) : neg_inf();
}

// weights[b, s] += sum over the rows that see key s of 2^(u - lse): one warp per key.
__global__ void __launch_bounds__(32 * LR_WARPS) latent_weights_kernel(const LatentAttnParams p) {
  pdl_enter();
  const int b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = seq_len(p, b);
  const int32_t* table = p.block_table + (int64_t)b * p.max_pages;
  for (int s = blockIdx.x * LR_WARPS + warp; s < len; s += gridDim.x * LR_WARPS) {
    Key k, q;
    load_key(p, slot_of(p, table, s), lane, k);
    float sum = 0.f;
    for (int r = 0; r < p.next_n * p.H; ++r) {
      if (s >= len - p.next_n + r / p.H + 1) continue;
      const int64_t row = (int64_t)b * p.next_n * p.H + r;
      load16(p.q_nope + row * LA_DC + 16 * lane, q.c);
      q.e = load2(p.q_pe + row * LA_DP + 2 * lane);
      sum += exp2f(dot(q, k) * p.scale_log2 - p.lse[row]);
    }
    if (lane == 0) p.weights[b * p.ld_weights + s] += sum;
  }
}

cudaError_t launch_latent_attn(const LatentAttnParams& p, cudaStream_t s) {
  count_launch();
  cudaError_t e = launch_pdl(latent_rows_kernel, dim3((unsigned)(p.B * p.next_n * p.H)), dim3(32 * LR_WARPS), 0, s, p);
  if (e != cudaSuccess || !p.weights) return e;
  count_launch();
  return launch_pdl(latent_weights_kernel, dim3(p.max_pages, p.B), dim3(32 * LR_WARPS), 0, s, p);
}

}  // namespace dsa
