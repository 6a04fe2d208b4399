// token_encode.cu -- rows of new tokens made ready for the indexer and the
// latent cache: norm, rotation by position, Hadamard transform, FP8 codes.
//
// encode_kernel: rows x[t, g] (64 query heads, or the one key of a token)
//     y = LayerNorm(x) (optional);  y[0:64] rotated by the token's angles;
//     y = H y / sqrt(128) (optional, H the Hadamard matrix in Sylvester's order)
//     scale[t] = max over g, d of |y| / 448 (1 where all are 0);  codes = e4m3(y / scale)
// and, in CTAs of their own, rope parts pe[t, h] rotated to bf16.
// append_kernel: a token's latent (RMSNorm), rope part (rotated) and index key (as above) to its
// cache slot, behind the block table.
//
// All of it is bound by bytes: a query token reads 16 KB and writes 8 KB.  A
// row of 128 dims lies in four lanes, lane j with dims 8 j + 32 c + e: 16-byte
// loads whose four lanes fill two sectors, both halves of every rotated pair in
// one lane (pairs (2 i, 2 i + 1) in e, pairs (i, i + 32) in c), and five of the
// seven Hadamard stages as well; two are shuffles.  Values stay fp32 between the
// loads and the one rounding at the end.
#include <cuda_fp8.h>

#include "latent.h"

namespace dsa {

namespace {
constexpr int TE_THREADS = 256;
constexpr int TE_ROWS = TE_THREADS / 4;  // rows of four lanes per CTA

__device__ __forceinline__ void unpack8(const uint4& v, float (&y)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = __uint_as_float(u[i] << 16);
    y[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&y)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ float sum4(float x) {  // over the four lanes of a row
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// cos and sin of lane j's eight rotated pairs: with `pairs` pair 4 j + i of
// dims 8 j.. and pair 16 + 4 j + i of dims 32 + 8 j..; else pair 8 j + e.
struct Angles {
  float c[8], s[8];
  __device__ __forceinline__ void load(const float* cs, int j, bool pairs) {
    const int a = pairs ? 4 * j : 8 * j, b = pairs ? 16 + 4 * j : 8 * j + 4;
    const float4 c0 = *reinterpret_cast<const float4*>(cs + a), c1 = *reinterpret_cast<const float4*>(cs + b);
    const float4 s0 = *reinterpret_cast<const float4*>(cs + 32 + a), s1 = *reinterpret_cast<const float4*>(cs + 32 + b);
    c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
    s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w, s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
  }
};
// Rotates dims 8 j + e (y0) and 32 + 8 j + e (y1) of a row's 64.
__device__ __forceinline__ void rotate(float (&y0)[8], float (&y1)[8], const Angles& a, bool pairs) {
  if (pairs) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p = y0[2 * i], q = y0[2 * i + 1], r = y1[2 * i], s = y1[2 * i + 1];
      y0[2 * i] = p * a.c[i] - q * a.s[i];
      y0[2 * i + 1] = p * a.s[i] + q * a.c[i];
      y1[2 * i] = r * a.c[4 + i] - s * a.s[4 + i];
      y1[2 * i + 1] = r * a.s[4 + i] + s * a.c[4 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = y0[i], q = y1[i];
      y0[i] = p * a.c[i] - q * a.s[i];
      y1[i] = p * a.s[i] + q * a.c[i];
    }
  }
}

// One row's values in place; returns the lane's largest magnitude, without the Hadamard transform's factor.
__device__ __forceinline__ float encode_values(float (&y)[4][8], const RowEncoding& o, const Angles& a, int j) {
  if (o.norm_w) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += y[i >> 3][i & 7];
    const float mean = sum4(s) * (1.f / 128);
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float d = y[i >> 3][i & 7] - mean;
      y[i >> 3][i & 7] = d;
      s = fmaf(d, d, s);
    }
    const float r = rsqrtf(sum4(s) * (1.f / 128) + o.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = i >> 1, d = 8 * j + 32 * c + 4 * (i & 1);
      const float4 w = *reinterpret_cast<const float4*>(o.norm_w + d), b = *reinterpret_cast<const float4*>(o.norm_b + d);
      float* v = &y[c][4 * (i & 1)];
      v[0] = fmaf(v[0] * r, w.x, b.x);
      v[1] = fmaf(v[1] * r, w.y, b.y);
      v[2] = fmaf(v[2] * r, w.z, b.z);
      v[3] = fmaf(v[3] * r, w.w, b.w);
    }
  }
  rotate(y[0], y[1], a, o.pairs);
  if (o.hadamard) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int h = 1; h < 8; h <<= 1)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!(e & h)) {
            const float p = y[c][e], q = y[c][e | h];
            y[c][e] = p + q;
            y[c][e | h] = p - q;
          }
#pragma unroll
    for (int h = 1; h < 4; h <<= 1)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (!(c & h))
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float p = y[c][e], q = y[c | h][e];
            y[c][e] = p + q;
            y[c | h][e] = p - q;
          }
#pragma unroll
    for (int h = 1; h < 4; h <<= 1) {
      const float sign = j & h ? -1.f : 1.f;  // the lane of the lower dims gets the sum, the other the difference
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float other = __shfl_xor_sync(0xffffffffu, y[i >> 3][i & 7], h);
        y[i >> 3][i & 7] = fmaf(sign, y[i >> 3][i & 7], other);
      }
    }
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) m = fmaxf(m, fabsf(y[i >> 3][i & 7]));
  return m;
}

// The scale of a token whose largest magnitude is `amax` (before the Hadamard transform's factor).
__device__ __forceinline__ float encode_scale(float amax, const RowEncoding& o) {
  const float s = (o.hadamard ? amax * 0.08838834764831845f : amax) * (1.f / 448);
  return s > 0.f ? s : 1.f;
}

// Rounds a row's values to codes, eight bytes for each of the lane's four runs of dims.
__device__ __forceinline__ void store_codes(uint8_t* row, const float (&y)[4][8], float amax, int j) {
  // y / (amax / 448); where the reciprocal would leave the range, by a division
  const bool far = amax < 1e-30f;
  const float top = amax > 0.f ? amax * (1.f / 448) : 1.f, inv = far ? 0.f : 448.f / amax;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t u[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t x[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float2 v = make_float2(y[c][4 * h + 2 * e], y[c][4 * h + 2 * e + 1]);
        v = far ? make_float2(v.x / top, v.y / top) : make_float2(v.x * inv, v.y * inv);
        x[e] = __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
      }
      u[h] = x[0] | x[1] << 16;
    }
    *reinterpret_cast<uint2*>(row + 8 * j + 32 * c) = make_uint2(u[0], u[1]);
  }
}

// Rope part of one row: lane j of four reads 16 bytes at dims 8 j and 32 + 8 j, and writes them rotated.
__device__ __forceinline__ void load_pe(const __nv_bfloat16* row, int j, uint4 (&v)[2]) {
  v[0] = *reinterpret_cast<const uint4*>(row + 8 * j);
  v[1] = *reinterpret_cast<const uint4*>(row + 32 + 8 * j);
}
__device__ __forceinline__ void rotate_pe(const uint4 (&v)[2], const Angles& a, bool pairs, uint4 (&r)[2]) {
  float y0[8], y1[8];
  unpack8(v[0], y0);
  unpack8(v[1], y1);
  rotate(y0, y1, a, pairs);
  r[0] = pack8(y0);
  r[1] = pack8(y1);
}
__device__ __forceinline__ void store_pe(__nv_bfloat16* row, int j, const uint4 (&v)[2]) {
  *reinterpret_cast<uint4*>(row + 8 * j) = v[0];
  *reinterpret_cast<uint4*>(row + 32 + 8 * j) = v[1];
}
}  // namespace

// CTAs [0, index_ctas) encode 64 rows each: with 64 rows a token one token, else 64
// tokens.  The others rotate 64 rope rows each.
template <int G>
__global__ void __launch_bounds__(TE_THREADS) encode_kernel(const EncodeParams p) {
  pdl_enter();
  __shared__ float s_max[TE_THREADS / 32];
  const int tid = threadIdx.x, j = tid & 3, lane = tid & 31;
  bool bad = false;
  if (blockIdx.x < (unsigned)p.index_ctas) {
    const int64_t row = (int64_t)blockIdx.x * TE_ROWS + (tid >> 2);
    const int64_t t = G == 1 ? row : blockIdx.x;
    const int g = G == 1 ? 0 : tid >> 2;
    int pos = t < p.T ? p.positions[t] : -1;
    if (pos >= p.max_positions) bad = true, pos = -1;
    float y[4][8] = {};
    Angles a = {};
    if (pos >= 0) {
      const __nv_bfloat16* x = p.x + t * p.x_token + g * p.x_head + 8 * j;
      uint4 v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = *reinterpret_cast<const uint4*>(x + 32 * c);
      a.load(p.cos_sin + (int64_t)pos * 64, j, p.enc.pairs);
#pragma unroll
      for (int c = 0; c < 4; ++c) unpack8(v[c], y[c]);
    }
    float m = encode_values(y, p.enc, a, j);
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if constexpr (G > 1) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (lane == 0) s_max[tid >> 5] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < TE_THREADS / 32; ++i) m = fmaxf(m, s_max[i]);
    }
    if (pos >= 0) {
      store_codes(p.codes + (t * G + g) * 128, y, m, j);
      if (G == 1 ? j == 0 : tid == 0) p.scale[t] = encode_scale(m, p.enc);
    }
  } else {
    const int64_t row = ((int64_t)blockIdx.x - p.index_ctas) * TE_ROWS + (tid >> 2);
    const int64_t t = row / p.H;
    const int h = (int)(row % p.H);
    int pos = t < p.T ? p.positions[t] : -1;
    if (pos >= p.max_positions) bad = true, pos = -1;
    if (pos >= 0) {
      uint4 v[2], r[2];
      load_pe(p.pe + t * p.pe_token + h * p.pe_head, j, v);
      Angles a;
      a.load(p.cos_sin + (int64_t)pos * 64, j, p.pe_pairs);
      rotate_pe(v, a, p.pe_pairs, r);
      store_pe(p.pe_out + t * p.po_token + h * p.po_head, j, r);
    }
  }
  last_cta(p.status, bad);
}

cudaError_t launch_encode(EncodeParams p, cudaStream_t s) {
  p.index_ctas = !p.x ? 0 : p.G == 1 ? (p.T + TE_ROWS - 1) / TE_ROWS : p.T;
  const int64_t pe_rows = p.pe ? (int64_t)p.T * p.H : 0;
  const unsigned ctas = (unsigned)(p.index_ctas + (pe_rows + TE_ROWS - 1) / TE_ROWS);
  count_launch();
  return p.G == 1 ? launch_pdl(encode_kernel<1>, dim3(ctas), dim3(TE_THREADS), 0, s, p)
                  : launch_pdl(encode_kernel<64>, dim3(ctas), dim3(TE_THREADS), 0, s, p);
}

// ---------------------------------------------------------------- append --
namespace {
// Where token t goes: its slot (-1: nowhere) and its position.
struct Place {
  int64_t slot;
  int pos;
};
__device__ __forceinline__ bool valid_sequence(const AppendParams& p, int b, int& first, int& n, int& len) {
  first = p.cu_new[b];
  const int64_t end = p.cu_new[b + 1];
  len = p.seq_lens[b];
  if (first < 0 || end < first || end > p.T || len < 0) return false;
  n = (int)end - first;
  return (int64_t)len + n <= (int64_t)p.max_pages * PAGE;
}
__device__ __forceinline__ Place place_token(const AppendParams& p, int t, bool& bad) {
  Place r{-1, 0};
  if (t >= p.T) return r;
  int lo = 0, hi = p.B;  // the first sequence that ends behind t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (p.cu_new[mid + 1] > t) hi = mid;
    else lo = mid + 1;
  }
  int first, n, len;
  if (lo == p.B || !valid_sequence(p, lo, first, n, len) || first > t) return r;
  const int s = len + t - first;
  const int page = p.block_table[(int64_t)lo * p.max_pages + s / PAGE];
  r.pos = p.positions ? p.positions[t] : s;
  if (page < 0 || page >= p.num_pages || r.pos < 0 || r.pos >= p.max_positions) bad = true;
  else r.slot = (int64_t)page * PAGE + s % PAGE;
  return r;
}
}  // namespace

// CTAs [0, latent_ctas): a warp per token normalises its latent, 16 dims per
// lane.  The others: four lanes per token rotate the rope part and encode the
// index key.
__global__ void __launch_bounds__(TE_THREADS) append_kernel(const AppendParams p) {
  pdl_enter();
  const int tid = threadIdx.x, lane = tid & 31;
  bool bad = false;
  if (blockIdx.x < (unsigned)p.latent_ctas) {
    const int64_t t = (int64_t)blockIdx.x * (TE_THREADS / 32) + (tid >> 5);
    if (t < p.T) {
      uint4 v[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) v[k] = *reinterpret_cast<const uint4*>(p.c + t * p.c_stride + 256 * k + 8 * lane);
      const Place at = place_token(p, (int)t, bad);
      if (p.c_norm) {
        float y[2][8];
        unpack8(v[0], y[0]);
        unpack8(v[1], y[1]);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) s = fmaf(y[i >> 3][i & 7], y[i >> 3][i & 7], s);
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const float r = rsqrtf(s * (1.f / LA_DC) + p.c_eps);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            const float4 g = *reinterpret_cast<const float4*>(p.c_norm + 256 * k + 8 * lane + e);
            y[k][e] *= r * g.x;
            y[k][e + 1] *= r * g.y;
            y[k][e + 2] *= r * g.z;
            y[k][e + 3] *= r * g.w;
          }
          v[k] = pack8(y[k]);
        }
      }
      if (at.slot >= 0) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          *reinterpret_cast<uint4*>(p.ckv + at.slot * p.ckv_stride + 256 * k + 8 * lane) = v[k];
          if (p.c_out) *reinterpret_cast<uint4*>(p.c_out + t * p.c_out_stride + 256 * k + 8 * lane) = v[k];
        }
      }
    }
  } else {
    const int64_t t = ((int64_t)blockIdx.x - p.latent_ctas) * TE_ROWS + (tid >> 2);
    const int j = tid & 3;
    float y[4][8] = {};
    Angles a = {};
    uint4 e[2] = {};
    Place at{-1, 0};
    if (t < p.T) {
      load_pe(p.k_pe + t * p.kp_stride, j, e);
      uint4 v[4];
      if (p.index_k) {
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = *reinterpret_cast<const uint4*>(p.index_k + t * p.ik_stride + 32 * c + 8 * j);
      }
      at = place_token(p, (int)t, bad);
      if (p.index_k) {
#pragma unroll
        for (int c = 0; c < 4; ++c) unpack8(v[c], y[c]);
      }
    }
    const float* cs = p.cos_sin + (int64_t)at.pos * 64;
    if (at.slot >= 0) {
      uint4 r[2];
      a.load(cs, j, p.pe_pairs);
      rotate_pe(e, a, p.pe_pairs, r);
      store_pe(p.kpe + at.slot * p.kpe_stride, j, r);
      if (p.k_pe_out) store_pe(p.k_pe_out + t * p.kp_out_stride, j, r);
    }
    if (p.index_k) {
      if (at.slot >= 0 && p.enc.pairs != p.pe_pairs) a.load(cs, j, p.enc.pairs);
      float m = encode_values(y, p.enc, a, j);
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      if (at.slot >= 0) {
        store_codes(p.k_cache + at.slot * 128, y, m, j);
        if (j == 0) p.k_scale[at.slot] = encode_scale(m, p.enc);
      }
    }
  }
  // new_lens may be seq_lens itself: it is written where every CTA has read what it needs
  if (last_cta(p.status, bad)) {
    bool wrong = false;
    for (int b = tid; b < p.B; b += TE_THREADS) {
      int first, n, len;
      const bool ok = valid_sequence(p, b, first, n, len);
      wrong |= !ok;
      p.new_lens[b] = ok ? len + n : len;
    }
    if (wrong) atomicOr(&p.status->last, ST_RANGE);
  }
}

cudaError_t launch_append(AppendParams p, cudaStream_t s) {
  p.latent_ctas = (p.T + TE_THREADS / 32 - 1) / (TE_THREADS / 32);
  const unsigned ctas = (unsigned)(p.latent_ctas + (p.T + TE_ROWS - 1) / TE_ROWS);
  count_launch();
  return launch_pdl(append_kernel, dim3(ctas), dim3(TE_THREADS), 0, s, p);
}

}  // namespace dsa
