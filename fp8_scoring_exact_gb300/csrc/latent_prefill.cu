// latent_prefill.cu -- causal attention of a ragged batch in the expanded form.
//
// Sequence z has queries [cu_q[z], cu_q[z+1]) and keys [cu_k[z], cu_k[z+1]).
// Query i of n sees keys [0, m - n + i + 1) of the sequence's m (all m without
// the causal mask); a key of head h is (k_nope[s, h] | k_pe[s]), 192 dims,
// its value v[s, h], 128 dims.  Softmax in base 2 as in latent_attn.cu.
//
// One warp per (query, head): lane l holds 4 key dims, 2 rope dims and 4
// value dims.
#include "latent.h"

namespace dsa {

namespace {
constexpr int PR_WARPS = 8;
__device__ __forceinline__ float4 load4(const __nv_bfloat16* src) {
  const uint2 v = *reinterpret_cast<const uint2*>(src);
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                     __uint_as_float(v.y & 0xffff0000u));
}
}  // namespace

__global__ void __launch_bounds__(32 * PR_WARPS) prefill_rows_kernel(const PrefillParams p) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * PR_WARPS + (threadIdx.x >> 5);
  if (row >= (int64_t)p.Tq * p.H) return;
  const int t = (int)(row / p.H), h = (int)(row % p.H);
  int z = 0;
  while (z < p.S && p.cu_q[z + 1] <= t) ++z;
  if (z >= p.S) return;
  const int q0 = p.cu_q[z], q1 = p.cu_q[z + 1], k0 = p.cu_k[z], k1 = p.cu_k[z + 1];
  if (q0 < 0 || q1 > p.Tq || k0 < 0 || k1 > p.Tk || k0 > k1) {
    atomicOr(&p.status->now, ST_RANGE);
    return;
  }
  const int n = p.causal ? max(0, (k1 - k0) - (q1 - q0) + (t - q0) + 1) : k1 - k0;
  const float4 q = load4(p.q + t * p.q_st + h * p.q_sh + 4 * lane);
  const float2 qe = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p.q + t * p.q_st + h * p.q_sh + 128 + 2 * lane));
  float m = -__int_as_float(0x7f800000), l = 0.f, c = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int64_t s = k0; s < k0 + n; ++s) {
    const float4 k = load4(p.k_nope + s * p.kn_st + h * p.kn_sh + 4 * lane);
    const float4 v = load4(p.v + s * p.v_st + h * p.v_sh + 4 * lane);
    const float2 ke = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p.k_pe + s * p.kp_st + 2 * lane));
    float x = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w + qe.x * ke.x + qe.y * ke.y;
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    const float u = x * p.scale_log2, m_new = fmaxf(m, u);
    const float a = exp2f(m - m_new), w = exp2f(u - m_new);
    m = m_new;
    // compensated: over many keys of nearly equal weight a plain sum would
    // lose the weights' differences
    l *= a;
    const float y = w - c * a, sum = l + y;
    c = (sum - l) - y;
    l = sum;
    o = make_float4(o.x * a + w * v.x, o.y * a + w * v.y, o.z * a + w * v.z, o.w * a + w * v.w);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(p.out + row * LA_DV + 4 * lane);
  dst[0] = __floats2bfloat162_rn(o.x * inv, o.y * inv);
  dst[1] = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  if (lane == 0) p.lse[row] = l > 0.f ? m + log2f(l) : -__int_as_float(0x7f800000);
}

__global__ void prefill_status_kernel(LatentStatus* s) {
  pdl_enter();
  s->last = s->now;
  s->now = 0;
}

cudaError_t launch_prefill(const PrefillParams& p, cudaStream_t s) {
  count_launch();
  const int64_t rows = (int64_t)p.Tq * p.H;
  cudaError_t e = launch_pdl(prefill_rows_kernel, dim3((unsigned)((rows + PR_WARPS - 1) / PR_WARPS)), dim3(32 * PR_WARPS), 0, s, p);
  if (e != cudaSuccess) return e;
  count_launch();
  return launch_pdl(prefill_status_kernel, dim3(1), dim3(1), 0, s, p.status);
}

}  // namespace dsa
