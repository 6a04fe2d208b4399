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
// What it cannot do without are bytes: a query token reads 16 KB and writes 8 KB.  A
// row of 128 dims lies in L lanes, lane j with dims 32 / L j + 32 c + e: 16-byte
// loads that fill whole sectors, both halves of every rotated pair in one lane
// (pairs (2 i, 2 i + 1) in e, pairs (i, i + 32) in c), and all Hadamard stages
// but log2 L, which are shuffles.  The 64 rows of a query token take two lanes
// each, which halves the shuffles (4096 tokens 30.3 us, 32.0 with four), single
// rows four (131072 keys 28.6 us, and 42 with two, whose norm and rope part spill;
// with four 8 or 22 bytes of a norm's builds do, or none).
// Values stay fp32, two to a register pair for the packed arithmetic, between
// the loads and the one rounding at the end.  CTAs stay and take every so manieth
// token: with a CTA for each, what starting and ending it costs (the status among
// it) was a third of the time.
//
// On the device, in a graph: 4096 query tokens with 16 rope rows each (118 MB)
// 30.4 us, 3.9 TB/s, of which a start of 4; the index rows alone 27.1, without the
// Hadamard transform 22.0, with a norm 36.6 (40.8 with the rope rows; a row's weights
// are 16 loads a lane); the rope rows alone 7.7.  The shared-memory path is 58%
// busy, issue 31%.  CTAs per SM: three 33.7, five 32.3.  Slower were also
// the next token's rows in registers (33.8), rows fetched ahead by cp.async, and
// the exchange of the last stages through shared memory; those stages on mma.sync
// with values in three bf16 parts gained 3%, rows copied ahead by TMA 4% (with a
// norm they lost 5%): neither was worth its code.
// 131072 keys with norm and rope part (118 MB): 28.0 us; the index rows alone 21.8,
// 16.5 without the norm, 13.7 without both.  16384 tokens appended (48 MB): 16.2 us.
#include <cuda_fp8.h>

#include <limits.h>

#include <algorithm>

#include "latent.h"

namespace dsa {

namespace {
constexpr int TE_ROWS = 64;  // per CTA
// Lanes of a row of encode_kernel, the threads of a CTA and the CTAs per SM.
template <int G>
constexpr int LANES = G > 1 ? 2 : 4;
template <int G>
constexpr int THREADS = TE_ROWS * LANES<G>;
template <int G>
constexpr int CTAS = G > 1 ? 4 : 3;

// A lane's values of a row, of L lanes: element (16 / L) c + i holds dims (32 / L) j + 32 c + 2 i and the next.
template <int L>
using Row = uint64_t[64 / L];

// Where a lane's `n`-th 16 bytes of bf16 begin.
template <int L>
__device__ __forceinline__ int dim8(int n, int j) {
  return 32 * (n / (4 / L)) + 8 * (n % (4 / L)) + 32 / L * j;
}
template <int L, int N>
__device__ __forceinline__ void load_row(const __nv_bfloat16* row, int j, uint4 (&v)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = *reinterpret_cast<const uint4*>(row + dim8<L>(n, j));
}
template <int L, int N>
__device__ __forceinline__ void store_row(__nv_bfloat16* row, int j, const uint4 (&v)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) *reinterpret_cast<uint4*>(row + dim8<L>(n, j)) = v[n];
}

__device__ __forceinline__ void unpack8(const uint4& v, uint64_t* y) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = pack2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
}
__device__ __forceinline__ uint4 pack8(const uint64_t* y) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2(y[i]);
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}
template <int L>
__device__ __forceinline__ float sum_row(float x) {
#pragma unroll
  for (int h = 1; h < L; h <<= 1) x += __shfl_xor_sync(0xffffffffu, x, h);
  return x;
}
__device__ __forceinline__ float sum_warp(float2 v) {
  float x = v.x + v.y;
#pragma unroll
  for (int h = 16; h; h >>= 1) x += __shfl_xor_sync(0xffffffffu, x, h);
  return x;
}
template <int N>
__device__ __forceinline__ float max_lanes(float x) {  // over every N lanes
#pragma unroll
  for (int h = 1; h < N; h <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, h));
  return x;
}

// cos and sin of lane j's 32 / L rotated pairs: with `pairs` those from 16 / L j on,
// of its dims below 32, and from 16 + 16 / L j on, of the others; else those from 32 / L j on.
template <int L>
struct Angles {
  static constexpr int HALF = 4 / L;  // of them, in fours, in dims below 32
  float4 c[2 * HALF], s[2 * HALF];
  __device__ __forceinline__ void load(const float* cs, int j, bool pairs) {
#pragma unroll
    for (int i = 0; i < 2 * HALF; ++i) {
      const int at = 4 * i + (pairs ? 4 * HALF * j + (i < HALF ? 0 : 16 - 4 * HALF) : 8 * HALF * j);
      c[i] = *reinterpret_cast<const float4*>(cs + at);
      s[i] = *reinterpret_cast<const float4*>(cs + 32 + at);
    }
  }
};
__device__ __forceinline__ uint64_t turn_pair(uint64_t y, float c, float s) {
  const float2 v = unpack2(y);
  return pack2(v.x * c - v.y * s, v.x * s + v.y * c);
}
// Rotates a lane's dims below 64.
template <int L>
__device__ __forceinline__ void rotate(uint64_t* y, const Angles<L>& a, bool pairs) {
  if (pairs) {
#pragma unroll
    for (int h = 0; h < 8 / L; ++h, y += 4) {
      y[0] = turn_pair(y[0], a.c[h].x, a.s[h].x);
      y[1] = turn_pair(y[1], a.c[h].y, a.s[h].y);
      y[2] = turn_pair(y[2], a.c[h].z, a.s[h].z);
      y[3] = turn_pair(y[3], a.c[h].w, a.s[h].w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16 / L; ++i) {
      const float4 cc = a.c[i >> 1], ss = a.s[i >> 1];
      const uint64_t c = i & 1 ? pack2(cc.z, cc.w) : pack2(cc.x, cc.y), s = i & 1 ? pack2(ss.z, ss.w) : pack2(ss.x, ss.y);
      const uint64_t n = i & 1 ? pack2(-ss.z, -ss.w) : pack2(-ss.x, -ss.y);
      const uint64_t p = y[i], q = y[16 / L + i];
      y[i] = fma2(p, c, fmul2(q, n));
      y[16 / L + i] = fma2(p, s, fmul2(q, c));
    }
  }
}

// max(|a|, |b|, |c|); a NaN is passed over
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// (p, q) -> (p + q, p - q)
__device__ __forceinline__ void butterfly(uint64_t& p, uint64_t& q) {
  const uint64_t minus = pack2(-1.f, -1.f), sum = fadd2(p, q);
  q = fma2(q, minus, p);
  p = sum;
}

// A power of two that brings `top`, the largest magnitude of what is squared, to [1, 4) (and what is below fp32's normal
// range as far up as it can).
__device__ __forceinline__ float unit_scale(float top) {
  const int e = (int)(__float_as_uint(top) >> 23) - 127;
  return __uint_as_float((uint32_t)(127 - min(max(e, -126), 126)) << 23);
}
// Whether a mean square (with eps) was formed without overflow, and is large enough that no square has lost bits that it
// still has: 2^-90 is 2^59 steps of fp32's lower end.
__device__ __forceinline__ bool sound_square(float t) { return t >= 0x1p-90f && t <= 3.402823466e38f; }

// One row's norm and rotation in place.  False: the row is too large (from 2e18 on) or too small to be squared, and
// has to be taken SCALED: times a power of two, with eps times its square.
template <int L, bool NORM, bool SCALED>
__device__ __forceinline__ bool norm_rotate(Row<L>& y, const RowEncoding& o, const Angles<L>& a, int j) {
  bool sound = true;
  if constexpr (NORM) {
    float k = 1.f;
    if constexpr (SCALED) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 64 / L; ++i) {
        const float2 x = unpack2(y[i]);
        m = max_abs3(m, x.x, x.y);
      }
      k = unit_scale(fmaxf(max_lanes<L>(m), sqrtf(o.eps)));
#pragma unroll
      for (int i = 0; i < 64 / L; ++i) y[i] = fmul2(y[i], pack2(k, k));
    }
    uint64_t s2 = 0;
#pragma unroll
    for (int i = 0; i < 64 / L; ++i) s2 = fadd2(s2, y[i]);
    const float2 s = unpack2(s2);
    const float mean = sum_row<L>(s.x + s.y) * (1.f / 128);
    const uint64_t minus = pack2(-mean, -mean);
    uint64_t q2 = 0;
#pragma unroll
    for (int i = 0; i < 64 / L; ++i) {
      y[i] = fadd2(y[i], minus);
      q2 = fma2(y[i], y[i], q2);
    }
    const float2 q = unpack2(q2);
    const float t = sum_row<L>(q.x + q.y) * (1.f / 128) + (SCALED ? o.eps * k * k : o.eps);
    sound = SCALED || sound_square(t);
    const float r = rsqrtf(t);
    const uint64_t r2 = pack2(r, r);
#pragma unroll
    for (int i = 0; i < 32 / L; ++i) {
      const int d = dim8<L>(i >> 1, j) + 4 * (i & 1);
      const float4 w = *reinterpret_cast<const float4*>(o.norm_w + d), b = *reinterpret_cast<const float4*>(o.norm_b + d);
      y[2 * i] = fma2(fmul2(y[2 * i], r2), pack2(w.x, w.y), pack2(b.x, b.y));
      y[2 * i + 1] = fma2(fmul2(y[2 * i + 1], r2), pack2(w.z, w.w), pack2(b.z, b.w));
    }
  }
  rotate<L>(y, a, o.pairs);
  return sound;
}
// Its Hadamard transform, without the factor; returns the lane's largest magnitude.
template <int L, bool HAD>
__device__ __forceinline__ float transform(Row<L>& y, int j) {
  if constexpr (HAD) {
#pragma unroll
    for (int i = 0; i < 64 / L; ++i) {
      const float2 v = unpack2(y[i]);
      y[i] = pack2(v.x + v.y, v.x - v.y);
    }
#pragma unroll
    for (int h = 1; h < 64 / L; h <<= 1)
#pragma unroll
      for (int i = 0; i < 64 / L; ++i)
        if (!(i & h)) butterfly(y[i], y[i | h]);
#pragma unroll
    for (int h = 1; h < L; h <<= 1) {
      // the lane of the lower dims gets the sum, the other the difference
      const float sign = j & h ? -1.f : 1.f;
      const uint64_t sign2 = pack2(sign, sign);
#pragma unroll
      for (int i = 0; i < 64 / L; ++i) {
        const float2 v = unpack2(y[i]);
        const uint64_t other = pack2(__shfl_xor_sync(0xffffffffu, v.x, h), __shfl_xor_sync(0xffffffffu, v.y, h));
        y[i] = fma2(sign2, y[i], other);
      }
    }
  }
  float m[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 64 / L; ++i) {
    const float2 v = unpack2(y[i]);
    m[i & 1] = max_abs3(m[i & 1], v.x, v.y);
  }
  return fmaxf(m[0], m[1]);
}

// The Hadamard transform's factor, 1 / sqrt(128).
template <bool HAD>
constexpr float FACTOR = HAD ? 0.08838834764831845f : 1.f;

// The scale of a token whose largest magnitude is `amax` (before the factor); 1 where it is 0, or rounds to it.
template <bool HAD>
__device__ __forceinline__ float encode_scale(float amax) {
  const float s = amax * FACTOR<HAD> * (1.f / 448);
  return s > 0.f ? s : 1.f;
}

// Rounds a row's values to codes, 32 / L bytes for each of the lane's four runs of dims.
template <int L, bool HAD>
__device__ __forceinline__ void store_codes(uint8_t* row, Row<L>& y, float amax, int j) {
  if (!(amax >= 1e-30f && amax <= 1e30f)) {
    // 448 / amax would leave the range, or __fdividef's; and below it a scale has few bits, or is 1
    const float top = encode_scale<HAD>(amax);
#pragma unroll
    for (int i = 0; i < 64 / L; ++i) {
      const float2 v = unpack2(y[i]);
      y[i] = pack2(v.x * FACTOR<HAD> / top, v.y * FACTOR<HAD> / top);
    }
  } else {
    const float inv = __fdividef(448.f, amax);
#pragma unroll
    for (int i = 0; i < 64 / L; ++i) y[i] = fmul2(y[i], pack2(inv, inv));
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t x[8 / L];
#pragma unroll
    for (int i = 0; i < 8 / L; ++i) {
      const uint64_t* p = y + 16 / L * c + 2 * i;
      x[i] = __nv_cvt_float2_to_fp8x2(unpack2(p[0]), __NV_SATFINITE, __NV_E4M3) |
             (uint32_t)__nv_cvt_float2_to_fp8x2(unpack2(p[1]), __NV_SATFINITE, __NV_E4M3) << 16;
    }
    uint8_t* to = row + 32 * c + 32 / L * j;
    if constexpr (L == 4) *reinterpret_cast<uint2*>(to) = make_uint2(x[0], x[1]);
    else *reinterpret_cast<uint4*>(to) = make_uint4(x[0], x[1], x[2], x[3]);
  }
}

// A lane's share of a rope part, rotated.
template <int L>
__device__ __forceinline__ void rotate_pe(uint4 (&v)[8 / L], const Angles<L>& a, bool pairs) {
  uint64_t y[32 / L];
#pragma unroll
  for (int i = 0; i < 8 / L; ++i) unpack8(v[i], y + 4 * i);
  rotate<L>(y, a, pairs);
#pragma unroll
  for (int i = 0; i < 8 / L; ++i) v[i] = pack8(y + 4 * i);
}

// The position of token t; -1: padding, or nothing.
__device__ __forceinline__ int token_position(const EncodeParams& p, int64_t t, bool& bad) {
  const int pos = t < p.T ? p.positions[t] : -1;
  if (pos < p.max_positions) return pos;
  bad = true;
  return -1;
}

// The index rows of a CTA's tokens, and with JOINT their rope parts: a step is one token of 64 rows (G = 64) or 64 tokens
// of one (G = 1).  s_unsound (in shared memory: a register more made 4096 query tokens with a norm 41.6 us instead of
// 40.8): some row has to be taken SCALED.
template <int G, bool NORM, bool HAD, bool JOINT, bool SCALED>
__device__ __forceinline__ void encode_rows(const EncodeParams& p, float (*s_max)[THREADS<G> / 32], int& s_unsound, bool& bad) {
  constexpr int L = LANES<G>, WARPS = THREADS<G> / 32, TOKENS = TE_ROWS / G;  // per step
  const int tid = threadIdx.x, j = tid % L, lane = tid & 31, group = tid / L, g = G == 1 ? 0 : group;
  const int64_t step = (int64_t)p.index_ctas * TOKENS;
  int64_t t = (int64_t)blockIdx.x * TOKENS + (G == 1 ? group : 0);
  int pos = token_position(p, t, bad);
  for (int64_t t0 = (int64_t)blockIdx.x * TOKENS, n = 0; t0 < p.T; t0 += step, t += step, ++n) {
    uint4 v[16 / L] = {};
    Angles<L> a = {};
    if (pos >= 0) {
      load_row<L>(p.x + t * p.x_token + g * p.x_head, j, v);
      a.load(p.cos_sin + (int64_t)pos * 64, j, p.enc.pairs);
    }
    uint4 e[8 / L] = {};
    if (JOINT && pos >= 0) load_row<L>(p.pe + t * p.pe_token, j, e);
    const int next = token_position(p, t + step, bad);
    Row<L> y;
#pragma unroll
    for (int c = 0; c < 16 / L; ++c) unpack8(v[c], y + 4 * c);
    if (!norm_rotate<L, NORM, SCALED>(y, p.enc, a, j) && pos >= 0) s_unsound = 1;
    float m = max_lanes<G == 1 ? L : 32>(transform<L, HAD>(y, j));
    if constexpr (G > 1) {
      if (lane == 0) s_max[n & 1][tid >> 5] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < WARPS; ++i) m = fmaxf(m, s_max[n & 1][i]);
    }
    if (JOINT && pos >= 0) {
      if (p.pe_pairs != p.enc.pairs) a.load(p.cos_sin + (int64_t)pos * 64, j, p.pe_pairs);
      rotate_pe<L>(e, a, p.pe_pairs);
      store_row<L>(p.pe_out + t * p.po_token, j, e);
    }
    if (pos >= 0) {
      store_codes<L, HAD>(p.codes + (t * G + g) * 128, y, m, j);
      if (G == 1 ? j == 0 : tid == 0) p.scale[t] = encode_scale<HAD>(m);
    }
    pos = next;
  }
}
}  // namespace

// CTAs [0, index_ctas) encode rows, the others rotate rope rows, 64 a step.
template <int G, bool NORM, bool HAD, bool JOINT>
__global__ void __launch_bounds__(THREADS<G>, CTAS<G>) encode_kernel(const EncodeParams p) {
  pdl_enter();
  constexpr int L = LANES<G>;
  __shared__ float s_max[2][THREADS<G> / 32];
  __shared__ int s_unsound;
  bool bad = false;
  if (blockIdx.x < (unsigned)p.index_ctas) {
    if constexpr (NORM) {
      if (threadIdx.x == 0) s_unsound = 0;
      __syncthreads();
    }
    encode_rows<G, NORM, HAD, JOINT, false>(p, s_max, s_unsound, bad);
    // a CTA that has met a row too large or too small to be squared takes its tokens once more, whose rope parts are done
    // (a vote on every row instead made 131072 keys 31.7 us)
    if constexpr (NORM) {
      __syncthreads();
      if (s_unsound) encode_rows<G, NORM, HAD, false, true>(p, s_max, s_unsound, bad);
    }
  } else {
    const int j = threadIdx.x % L, group = threadIdx.x / L;
    const int64_t rows = (int64_t)p.T * p.H, step = (int64_t)(gridDim.x - p.index_ctas) * TE_ROWS;
    for (int64_t row = (int64_t)(blockIdx.x - p.index_ctas) * TE_ROWS + group; row < rows; row += step) {
      const int64_t t = rows < (1ll << 31) ? (int)row / p.H : row / p.H;
      const int h = (int)(row - t * p.H), pos = token_position(p, t, bad);
      uint4 v[8 / L];
      load_row<L>(p.pe + t * p.pe_token + h * p.pe_head, j, v);
      if (pos < 0) continue;
      Angles<L> a;
      a.load(p.cos_sin + (int64_t)pos * 64, j, p.pe_pairs);
      rotate_pe<L>(v, a, p.pe_pairs);
      store_row<L>(p.pe_out + t * p.po_token + h * p.po_head, j, v);
    }
  }
  last_cta(p.status, bad);
}

template <int G, bool NORM, bool HAD, bool JOINT>
static cudaError_t launch_encode_as(EncodeParams p, cudaStream_t s) {
  // Both kinds of CTAs at once; a rope row counts 3 quarters of an index row.  us in a graph with 1, 2, 3, 4 and 6:
  //     tokens    16 heads                        5 heads                         64 heads
  //     1000      15.1  11.4  11.0  12.5  13.1    15.1  10.9  10.7  10.6  10.7    17.4  14.1  13.9  15.8  17.3
  //     2500      30.0  21.7  20.4  22.4  23.1    30.0  20.5  20.0  20.2  20.2    35.0  27.5  28.5  29.2  36.1
  //     4096      46.2  32.0  30.4  32.8  34.7    45.6  30.2  28.1  29.4  29.6    54.2  41.2  42.2  44.6  54.7
  //     6000      65.4  43.9  42.8  45.1  48.1    65.2  42.4  39.4  39.6  40.1    77.4  57.4  59.5  61.8  78.3
  // (128 heads: 2 is faster by 3 to 7%)
  const int all = CTAS<G> * option_grid(), steps = !p.x ? 0 : G == 1 ? ceil_div(p.T, TE_ROWS) : p.T;
  const int64_t pe_rows = p.pe && !JOINT ? (int64_t)p.T * p.H : 0, pe_steps = (pe_rows + TE_ROWS - 1) / TE_ROWS;
  const int64_t share = 4 * (int64_t)steps + 3 * pe_steps;
  const int pe_ctas = (int)std::min<int64_t>(pe_steps, std::max<int64_t>(pe_steps > 0, all * 3 * pe_steps / share));
  p.index_ctas = min(steps, max(1, all - pe_ctas));
  count_launch();
  return launch_pdl(encode_kernel<G, NORM, HAD, JOINT>, dim3(p.index_ctas + pe_ctas), dim3(THREADS<G>), 0, s, p);
}
template <int G, bool JOINT>
static cudaError_t launch_encode_g(const EncodeParams& p, cudaStream_t s) {
  if (p.enc.norm_w)
    return p.enc.hadamard ? launch_encode_as<G, true, true, JOINT>(p, s) : launch_encode_as<G, true, false, JOINT>(p, s);
  return p.enc.hadamard ? launch_encode_as<G, false, true, JOINT>(p, s) : launch_encode_as<G, false, false, JOINT>(p, s);
}
cudaError_t launch_encode(const EncodeParams& p, cudaStream_t s) {
  if (p.G > 1) return launch_encode_g<64, false>(p, s);
  return p.x && p.pe && p.H == 1 ? launch_encode_g<1, true>(p, s) : launch_encode_g<1, false>(p, s);
}

// ---------------------------------------------------------------- append --
namespace {
// Where token t goes: its slot (-1: nowhere) and its position.
struct Place {
  int64_t slot;
  int pos;
};
// Searches the sequences' ends, down to one of them; the borders it passes are kept.
struct Search {
  int lo, hi, before, behind;  // the sequences left; the last border that lies before them, the first behind
  __device__ __forceinline__ explicit Search(int B) : lo(0), hi(B), before(INT_MIN), behind(INT_MAX) {}
  template <class Left>
  __device__ __forceinline__ void run(const AppendParams& p, Left left) {
    while (lo < hi) {
      const int mid = (lo + hi) >> 1, end = p.cu_new[mid + 1];
      if (left(mid, end)) {
        hi = mid;
        behind = min(behind, end);
      } else {
        lo = mid + 1;
        before = max(before, end);
      }
    }
  }
};
// The sequence that a search ended at.  It is whole if the search for each of its tokens ends there: with borders that
// ascend always; else where it lies behind every border that the search passes on the left and before those on the right.
// So no token is placed for two sequences, and a valid one has all of its tokens.
__device__ __forceinline__ bool valid_sequence(const AppendParams& p, const Search& at, int& first, int& n, int& len) {
  first = p.cu_new[at.lo];
  const int64_t end = p.cu_new[at.lo + 1];
  len = p.seq_lens[at.lo];
  if (first < 0 || end < first || end > p.T || at.before > first || at.behind < end || len < 0) return false;
  n = (int)end - first;
  return (int64_t)len + n <= (int64_t)p.max_pages * PAGE;
}
__device__ __forceinline__ Place place_token(const AppendParams& p, int64_t t, bool& bad) {
  Place r{-1, 0};
  if (t >= p.T) return r;
  Search at(p.B);  // the first sequence that ends behind t
  at.run(p, [&](int, int end) { return end > t; });
  int first, n, len;
  if (at.lo == p.B || !valid_sequence(p, at, first, n, len) || first > t) return r;
  const int s = len + (int)t - first;
  const int page = p.block_table[(int64_t)at.lo * p.max_pages + s / PAGE];
  r.pos = p.positions ? p.positions[t] : s;
  if (page < 0 || page >= p.num_pages || r.pos < 0 || r.pos >= p.max_positions) bad = true;
  else r.slot = (int64_t)page * PAGE + s % PAGE;
  return r;
}
constexpr int AP_TOKENS = 4, AP_LANES = LANES<1>, AP_THREADS = THREADS<1>, AP_CTAS = CTAS<1>;

// The rope parts (but for SCALED, where they are done) and index keys of a CTA's tokens, four lanes each.  True: some key
// of this thread has to be taken SCALED.
template <bool NORM, bool HAD, bool SCALED>
__device__ __forceinline__ bool append_rows(const AppendParams& p, bool& bad) {
  constexpr int L = AP_LANES;
  const int tid = threadIdx.x, j = tid % L;
  bool unsound = false;
  // (every lane takes part in the shuffles)
  for (int64_t t0 = (int64_t)blockIdx.x * TE_ROWS; t0 < p.T; t0 += (int64_t)p.row_ctas * TE_ROWS) {
    const int64_t t = t0 + tid / L;
    uint4 e[8 / L] = {}, v[16 / L] = {};
    if (t < p.T) {
      if (!SCALED) load_row<L>(p.k_pe + t * p.kp_stride, j, e);
      if (p.index_k) load_row<L>(p.index_k + t * p.ik_stride, j, v);
    }
    const Place at = place_token(p, t, bad);
    const float* cs = p.cos_sin + (int64_t)at.pos * 64;
    Angles<L> a = {};
    if (at.slot >= 0) {
      a.load(cs, j, p.pe_pairs);
      if (!SCALED) {
        rotate_pe<L>(e, a, p.pe_pairs);
        store_row<L>(p.kpe + at.slot * p.kpe_stride, j, e);
        if (p.k_pe_out) store_row<L>(p.k_pe_out + t * p.kp_out_stride, j, e);
      }
    }
    if (p.index_k) {
      if (at.slot >= 0 && p.enc.pairs != p.pe_pairs) a.load(cs, j, p.enc.pairs);
      Row<L> y;
#pragma unroll
      for (int c = 0; c < 16 / L; ++c) unpack8(v[c], y + 4 * c);
      const bool sound = norm_rotate<L, NORM, SCALED>(y, p.enc, a, j);
      unsound |= at.slot >= 0 && !sound;
      const float m = max_lanes<L>(transform<L, HAD>(y, j));
      if (at.slot >= 0) {
        store_codes<L, HAD>(p.k_cache + at.slot * 128, y, m, j);
        if (j == 0) p.k_scale[at.slot] = encode_scale<HAD>(m);
      }
    }
  }
  return unsound;
}
}  // namespace

// CTAs [0, row_ctas): four lanes per token rotate the rope part and encode the
// index key.  The others: a warp normalises the latents of AP_TOKENS tokens at a time, 16 dims
// per lane, so that enough loads are in flight.
template <bool NORM, bool HAD>
__global__ void __launch_bounds__(AP_THREADS, AP_CTAS) append_kernel(const AppendParams p) {
  pdl_enter();
  const int tid = threadIdx.x, lane = tid & 31;
  bool bad = false;
  if (blockIdx.x >= (unsigned)p.row_ctas) {
    const int64_t step = (int64_t)(gridDim.x - p.row_ctas) * (AP_THREADS / 32) * AP_TOKENS;
    const int64_t first = ((int64_t)(blockIdx.x - p.row_ctas) * (AP_THREADS / 32) + (tid >> 5)) * AP_TOKENS;
    for (int64_t t0 = first; t0 < p.T; t0 += step) {
      uint4 v[AP_TOKENS][2];
#pragma unroll
      for (int i = 0; i < AP_TOKENS; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (t0 + i < p.T) v[i][k] = *reinterpret_cast<const uint4*>(p.c + (t0 + i) * p.c_stride + 256 * k + 8 * lane);
      int64_t slot = lane < AP_TOKENS ? place_token(p, t0 + lane, bad).slot : -1;
#pragma unroll
      for (int i = 0; i < AP_TOKENS; ++i) {
        const int64_t at = __shfl_sync(0xffffffffu, slot, i);
        if (at < 0) continue;  // (the same in the whole warp)
        if (p.c_norm) {
          uint64_t y[8], s2 = 0;
          unpack8(v[i][0], y);
          unpack8(v[i][1], y + 4);
#pragma unroll
          for (int x = 0; x < 8; ++x) s2 = fma2(y[x], y[x], s2);
          float t = sum_warp(unpack2(s2)) * (1.f / LA_DC) + p.c_eps;
          if (!sound_square(t)) {  // (the same in the whole warp) too large or too small to be squared
            float m = 0.f;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const float2 u = unpack2(y[x]);
              m = max_abs3(m, u.x, u.y);
            }
            const float k = unit_scale(fmaxf(max_lanes<32>(m), sqrtf(p.c_eps)));
            s2 = 0;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              y[x] = fmul2(y[x], pack2(k, k));
              s2 = fma2(y[x], y[x], s2);
            }
            t = sum_warp(unpack2(s2)) * (1.f / LA_DC) + p.c_eps * k * k;
          }
          const float r = rsqrtf(t);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float4 g = *reinterpret_cast<const float4*>(p.c_norm + 256 * (x >> 1) + 8 * lane + 4 * (x & 1));
            y[2 * x] = fmul2(y[2 * x], fmul2(pack2(r, r), pack2(g.x, g.y)));
            y[2 * x + 1] = fmul2(y[2 * x + 1], fmul2(pack2(r, r), pack2(g.z, g.w)));
          }
          v[i][0] = pack8(y);
          v[i][1] = pack8(y + 4);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          *reinterpret_cast<uint4*>(p.ckv + at * p.ckv_stride + 256 * k + 8 * lane) = v[i][k];
          if (p.c_out) *reinterpret_cast<uint4*>(p.c_out + (t0 + i) * p.c_out_stride + 256 * k + 8 * lane) = v[i][k];
        }
      }
    }
  } else {
    const bool unsound = append_rows<NORM, HAD, false>(p, bad);
    if (NORM && __syncthreads_or(unsound)) append_rows<NORM, HAD, true>(p, bad);
  }
  // new_lens may be seq_lens itself: it is written where every CTA has read what it needs
  if (last_cta(p.status, bad)) {
    bool wrong = false, falls = false;
    for (int b = tid; b < p.B; b += AP_THREADS) falls |= (p.cu_new[b + 1] < p.cu_new[b]) | (p.seq_lens[b] < 0);
    falls = __syncthreads_or(falls);  // (where borders ascend no search need be made: 64 sequences 6.9 us, 7.6 with it)
    for (int b = tid; b < p.B; b += AP_THREADS) {
      Search at(p.B);
      if (falls) at.run(p, [&](int mid, int) { return mid >= b; });
      else at.lo = b;
      int first, n, len;
      const bool ok = valid_sequence(p, at, first, n, len);  // (from the L1: a length has been read above, too)
      wrong |= !ok;
      p.new_lens[b] = ok ? len + n : len;
    }
    if (wrong) atomicOr(&p.status->last, ST_RANGE);
  }
}

cudaError_t launch_append(AppendParams p, cudaStream_t s) {
  // Both kinds of CTAs at once.  us in a graph, CTAs for rope parts and index keys a sixth, a quarter, a third, 10/24 and
  // a half of all:
  //     tokens    with an index key               without
  //     7000      12.7  10.0  10.0  10.0  10.0     9.0   8.9   8.7   8.8   8.8
  //     16384     21.1  18.2  15.8  15.5  16.5    14.5  13.5  14.1  14.0  15.1
  //     20000     24.7  19.8  18.5  18.4  18.2    16.2  14.6  16.2  16.6  16.2
  //     30000     32.7  26.6  24.1  22.9  24.1    22.3  19.9  20.9  20.9  20.7
  // (between 9000 and 60000 tokens without a key a quarter and a third are within 3%, either way)
  const int all = AP_CTAS * option_grid(), rows = ceil_div(p.T, TE_ROWS);
  const int latents = ceil_div(p.T, AP_THREADS / 32 * AP_TOKENS);
  p.row_ctas = min(rows, max(1, all / 3));
  const dim3 ctas(p.row_ctas + min(latents, max(1, all - p.row_ctas))), threads(AP_THREADS);
  count_launch();
  if (p.enc.norm_w)
    return p.enc.hadamard ? launch_pdl(append_kernel<true, true>, ctas, threads, 0, s, p)
                          : launch_pdl(append_kernel<true, false>, ctas, threads, 0, s, p);
  return p.enc.hadamard ? launch_pdl(append_kernel<false, true>, ctas, threads, 0, s, p)
                        : launch_pdl(append_kernel<false, false>, ctas, threads, 0, s, p);
}

}  // namespace dsa
