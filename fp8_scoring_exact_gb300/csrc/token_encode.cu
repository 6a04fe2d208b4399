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
// row of 128 dims lies in four lanes, lane j with dims 8 j + 32 c + e: 16-byte
// loads whose four lanes fill two sectors, both halves of every rotated pair in
// one lane (pairs (2 i, 2 i + 1) in e, pairs (i, i + 32) in c), and five of the
// seven Hadamard stages as well; two are shuffles.  Values stay fp32, two to a
// register pair for the packed arithmetic, between the loads and the one rounding
// at the end.  CTAs stay and take every so manieth token: with a CTA for each, what
// starting and ending it costs (the status among it) was a third of the time.
//
// 4096 query tokens with 16 rope rows each (118 MB): 32 us, 3.7 TB/s; the index
// rows alone 28, without the Hadamard transform 21, which is the memory's pace and a start of
// 4 us.  The transform's 470 instructions per warp and token do not hide behind
// it: the issue slots are 38% used, the shared-memory path (shuffles) 54%, and a
// fourth CTA per SM changed nothing.  Slower or no faster were: rows fetched ahead by
// cp.async (30.8 us), the exchange of the last two stages through shared memory
// (32.3), those stages on mma.sync with values in three bf16 parts (27.3).
// 131072 keys with norm and rope part (118 MB): 31 us; 16384 tokens appended (48
// MB): 14 us.
#include <cuda_fp8.h>

#include <algorithm>

#include "latent.h"

namespace dsa {

namespace {
constexpr int TE_THREADS = 256;
constexpr int TE_ROWS = TE_THREADS / 4;  // rows of four lanes per CTA
constexpr int TE_CTAS = 3;               // per SM

// A lane's 32 values of a row: element 4 c + i holds dims 8 j + 32 c + 2 i and the next.
using Row = uint64_t[16];

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
__device__ __forceinline__ float sum4(float x) {  // over the four lanes of a row
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// cos and sin of lane j's eight rotated pairs: with `pairs` pair 4 j + i of
// dims 8 j.. and pair 16 + 4 j + i of dims 32 + 8 j..; else pair 8 j + e.
struct Angles {
  float4 c[2], s[2];
  // where c[0], c[1], s[0] and s[1] (i = 0 .. 3) begin
  __device__ __forceinline__ static int at(int i, int j, bool pairs) {
    return (i & 2 ? 32 : 0) + (pairs ? 4 * j + (i & 1 ? 16 : 0) : 8 * j + (i & 1 ? 4 : 0));
  }
  __device__ __forceinline__ void load(const float* cs, int j, bool pairs) {
#pragma unroll
    for (int i = 0; i < 4; ++i) (i & 2 ? s : c)[i & 1] = *reinterpret_cast<const float4*>(cs + at(i, j, pairs));
  }
};
__device__ __forceinline__ uint64_t turn_pair(uint64_t y, float c, float s) {
  const float2 v = unpack2(y);
  return pack2(v.x * c - v.y * s, v.x * s + v.y * c);
}
// Rotates dims 8 j + e (y0) and 32 + 8 j + e (y1) of a row's 64.
__device__ __forceinline__ void rotate(uint64_t* y0, uint64_t* y1, const Angles& a, bool pairs) {
  if (pairs) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint64_t* y = h ? y1 : y0;
      y[0] = turn_pair(y[0], a.c[h].x, a.s[h].x);
      y[1] = turn_pair(y[1], a.c[h].y, a.s[h].y);
      y[2] = turn_pair(y[2], a.c[h].z, a.s[h].z);
      y[3] = turn_pair(y[3], a.c[h].w, a.s[h].w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 cc = a.c[i >> 1], ss = a.s[i >> 1];
      const uint64_t c = i & 1 ? pack2(cc.z, cc.w) : pack2(cc.x, cc.y), s = i & 1 ? pack2(ss.z, ss.w) : pack2(ss.x, ss.y);
      const uint64_t n = i & 1 ? pack2(-ss.z, -ss.w) : pack2(-ss.x, -ss.y);
      const uint64_t p = y0[i], q = y1[i];
      y0[i] = fma2(p, c, fmul2(q, n));
      y1[i] = fma2(p, s, fmul2(q, c));
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

// One row's norm and rotation in place.
template <bool NORM>
__device__ __forceinline__ void norm_rotate(Row& y, const RowEncoding& o, const Angles& a, int j) {
  if constexpr (NORM) {
    uint64_t s2 = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) s2 = fadd2(s2, y[i]);
    const float2 s = unpack2(s2);
    const float mean = sum4(s.x + s.y) * (1.f / 128);
    const uint64_t minus = pack2(-mean, -mean);
    uint64_t q2 = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      y[i] = fadd2(y[i], minus);
      q2 = fma2(y[i], y[i], q2);
    }
    const float2 q = unpack2(q2);
    const float r = rsqrtf(sum4(q.x + q.y) * (1.f / 128) + o.eps);
    const uint64_t r2 = pack2(r, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = 8 * j + 32 * (i >> 1) + 4 * (i & 1);
      const float4 w = *reinterpret_cast<const float4*>(o.norm_w + d), b = *reinterpret_cast<const float4*>(o.norm_b + d);
      y[2 * i] = fma2(fmul2(y[2 * i], r2), pack2(w.x, w.y), pack2(b.x, b.y));
      y[2 * i + 1] = fma2(fmul2(y[2 * i + 1], r2), pack2(w.z, w.w), pack2(b.z, b.w));
    }
  }
  rotate(y, y + 4, a, o.pairs);
}
// Its Hadamard transform, without the factor; returns the lane's largest magnitude.
template <bool HAD>
__device__ __forceinline__ float transform(Row& y, int j) {
  if constexpr (HAD) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 v = unpack2(y[i]);
      y[i] = pack2(v.x + v.y, v.x - v.y);
    }
#pragma unroll
    for (int h = 1; h < 16; h <<= 1)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (!(i & h)) butterfly(y[i], y[i | h]);
#pragma unroll
    for (int h = 1; h < 4; h <<= 1) {
      // the lane of the lower dims gets the sum, the other the difference
      const float sign = j & h ? -1.f : 1.f;
      const uint64_t sign2 = pack2(sign, sign);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 v = unpack2(y[i]);
        const uint64_t other = pack2(__shfl_xor_sync(0xffffffffu, v.x, h), __shfl_xor_sync(0xffffffffu, v.y, h));
        y[i] = fma2(sign2, y[i], other);
      }
    }
  }
  float m[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
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

// Rounds a row's values to codes, eight bytes for each of the lane's four runs of dims.
template <bool HAD>
__device__ __forceinline__ void store_codes(uint8_t* row, Row& y, float amax, int j) {
  if (!(amax >= 1e-30f && amax <= 1e30f)) {
    // 448 / amax would leave the range, or __fdividef's; and below it a scale has few bits, or is 1
    const float top = encode_scale<HAD>(amax);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 v = unpack2(y[i]);
      y[i] = pack2(v.x * FACTOR<HAD> / top, v.y * FACTOR<HAD> / top);
    }
  } else {
    const float inv = __fdividef(448.f, amax);
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = fmul2(y[i], pack2(inv, inv));
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __nv_cvt_float2_to_fp8x2(unpack2(y[4 * c + i]), __NV_SATFINITE, __NV_E4M3);
    *reinterpret_cast<uint2*>(row + 8 * j + 32 * c) = make_uint2(x[0] | x[1] << 16, x[2] | x[3] << 16);
  }
}

// Rope part of one row: lane j of four reads 16 bytes at dims 8 j and 32 + 8 j, and writes them rotated.
__device__ __forceinline__ void load_pe(const __nv_bfloat16* row, int j, uint4 (&v)[2]) {
  v[0] = *reinterpret_cast<const uint4*>(row + 8 * j);
  v[1] = *reinterpret_cast<const uint4*>(row + 32 + 8 * j);
}
__device__ __forceinline__ void rotate_pe(const uint4 (&v)[2], const Angles& a, bool pairs, uint4 (&r)[2]) {
  uint64_t y0[4], y1[4];
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

// CTAs [0, index_ctas): a step is one token of 64 rows (G = 64) or 64 tokens of
// one (G = 1).  The others rotate rope rows, 64 a step.
template <int G, bool NORM, bool HAD, bool JOINT>
__global__ void __launch_bounds__(TE_THREADS, TE_CTAS) encode_kernel(const EncodeParams p) {
  pdl_enter();
  __shared__ float s_max[2][TE_THREADS / 32];
  constexpr int TOKENS = TE_ROWS / G;  // per step
  const int tid = threadIdx.x, j = tid & 3, lane = tid & 31, group = tid >> 2;
  bool bad = false;
  auto position = [&](int64_t t) {  // -1: padding, or nothing
    const int pos = t < p.T ? p.positions[t] : -1;
    if (pos < p.max_positions) return pos;
    bad = true;
    return -1;
  };
  if (blockIdx.x < (unsigned)p.index_ctas) {
    const int g = G == 1 ? 0 : group;
    const int64_t step = (int64_t)p.index_ctas * TOKENS;
    int64_t t = (int64_t)blockIdx.x * TOKENS + (G == 1 ? group : 0);
    int pos = position(t);
    for (int64_t t0 = (int64_t)blockIdx.x * TOKENS, n = 0; t0 < p.T; t0 += step, t += step, ++n) {
      uint4 v[4] = {};
      Angles a = {};
      if (pos >= 0) {
        const __nv_bfloat16* x = p.x + t * p.x_token + g * p.x_head + 8 * j;
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = *reinterpret_cast<const uint4*>(x + 32 * c);
        a.load(p.cos_sin + (int64_t)pos * 64, j, p.enc.pairs);
      }
      uint4 e[2] = {};
      if (JOINT && pos >= 0) load_pe(p.pe + t * p.pe_token, j, e);
      const int next = position(t + step);
      Row y;
#pragma unroll
      for (int c = 0; c < 4; ++c) unpack8(v[c], y + 4 * c);
      norm_rotate<NORM>(y, p.enc, a, j);
      float m = transform<HAD>(y, j);
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      if constexpr (G > 1) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) s_max[n & 1][tid >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TE_THREADS / 32; ++i) m = fmaxf(m, s_max[n & 1][i]);
      }
      if (JOINT && pos >= 0) {
        if (p.pe_pairs != p.enc.pairs) a.load(p.cos_sin + (int64_t)pos * 64, j, p.pe_pairs);
        uint4 r[2];
        rotate_pe(e, a, p.pe_pairs, r);
        store_pe(p.pe_out + t * p.po_token, j, r);
      }
      if (pos >= 0) {
        store_codes<HAD>(p.codes + (t * G + g) * 128, y, m, j);
        if (G == 1 ? j == 0 : tid == 0) p.scale[t] = encode_scale<HAD>(m);
      }
      pos = next;
    }
  } else {
    const int64_t rows = (int64_t)p.T * p.H, step = (int64_t)(gridDim.x - p.index_ctas) * TE_ROWS;
    for (int64_t row = (int64_t)(blockIdx.x - p.index_ctas) * TE_ROWS + group; row < rows; row += step) {
      const int64_t t = rows < (1ll << 31) ? (int)row / p.H : row / p.H;
      const int h = (int)(row - t * p.H), pos = position(t);
      uint4 v[2], r[2];
      load_pe(p.pe + t * p.pe_token + h * p.pe_head, j, v);
      if (pos < 0) continue;
      Angles a;
      a.load(p.cos_sin + (int64_t)pos * 64, j, p.pe_pairs);
      rotate_pe(v, a, p.pe_pairs, r);
      store_pe(p.pe_out + t * p.po_token + h * p.po_head, j, r);
    }
  }
  last_cta(p.status, bad);
}

template <int G, bool NORM, bool HAD, bool JOINT>
static cudaError_t launch_encode_as(EncodeParams p, cudaStream_t s) {
  // both kinds of CTAs at once, in shares that end together
  const int all = TE_CTAS * option_grid(), steps = !p.x ? 0 : G == 1 ? ceil_div(p.T, TE_ROWS) : p.T;
  const int64_t pe_rows = p.pe && !JOINT ? (int64_t)p.T * p.H : 0, pe_steps = (pe_rows + TE_ROWS - 1) / TE_ROWS;
  const int64_t share = 4 * (int64_t)steps + 3 * pe_steps;
  const int pe_ctas = (int)std::min<int64_t>(pe_steps, std::max<int64_t>(pe_steps > 0, all * 3 * pe_steps / share));
  p.index_ctas = min(steps, max(1, all - pe_ctas));
  count_launch();
  return launch_pdl(encode_kernel<G, NORM, HAD, JOINT>, dim3(p.index_ctas + pe_ctas), dim3(TE_THREADS), 0, s, p);
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
__device__ __forceinline__ bool valid_sequence(const AppendParams& p, int b, int& first, int& n, int& len) {
  first = p.cu_new[b];
  const int64_t end = p.cu_new[b + 1];
  len = p.seq_lens[b];
  if (first < 0 || end < first || end > p.T || len < 0) return false;
  n = (int)end - first;
  return (int64_t)len + n <= (int64_t)p.max_pages * PAGE;
}
__device__ __forceinline__ Place place_token(const AppendParams& p, int64_t t, bool& bad) {
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
  const int s = len + (int)t - first;
  const int page = p.block_table[(int64_t)lo * p.max_pages + s / PAGE];
  r.pos = p.positions ? p.positions[t] : s;
  if (page < 0 || page >= p.num_pages || r.pos < 0 || r.pos >= p.max_positions) bad = true;
  else r.slot = (int64_t)page * PAGE + s % PAGE;
  return r;
}
}  // namespace

// CTAs [0, row_ctas): four lanes per token rotate the rope part and encode the
// index key.  The others: a warp normalises the latents of AP_TOKENS tokens at a time, 16 dims
// per lane, so that enough loads are in flight.
constexpr int AP_TOKENS = 4;
template <bool NORM, bool HAD>
__global__ void __launch_bounds__(TE_THREADS, TE_CTAS) append_kernel(const AppendParams p) {
  pdl_enter();
  const int tid = threadIdx.x, lane = tid & 31;
  bool bad = false;
  if (blockIdx.x >= (unsigned)p.row_ctas) {
    const int64_t step = (int64_t)(gridDim.x - p.row_ctas) * (TE_THREADS / 32) * AP_TOKENS;
    const int64_t first = ((int64_t)(blockIdx.x - p.row_ctas) * (TE_THREADS / 32) + (tid >> 5)) * AP_TOKENS;
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
          const float2 ss = unpack2(s2);
          float s = ss.x + ss.y;
#pragma unroll
          for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          const float r = rsqrtf(s * (1.f / LA_DC) + p.c_eps);
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
    const int j = tid & 3;
    // (every lane takes part in the shuffles)
    for (int64_t t0 = (int64_t)blockIdx.x * TE_ROWS; t0 < p.T; t0 += (int64_t)p.row_ctas * TE_ROWS) {
      const int64_t t = t0 + (tid >> 2);
      uint4 e[2] = {}, v[4] = {};
      if (t < p.T) {
        load_pe(p.k_pe + t * p.kp_stride, j, e);
        if (p.index_k) {
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] = *reinterpret_cast<const uint4*>(p.index_k + t * p.ik_stride + 32 * c + 8 * j);
        }
      }
      const Place at = place_token(p, t, bad);
      const float* cs = p.cos_sin + (int64_t)at.pos * 64;
      Angles a = {};
      if (at.slot >= 0) {
        uint4 r[2];
        a.load(cs, j, p.pe_pairs);
        rotate_pe(e, a, p.pe_pairs, r);
        store_pe(p.kpe + at.slot * p.kpe_stride, j, r);
        if (p.k_pe_out) store_pe(p.k_pe_out + t * p.kp_out_stride, j, r);
      }
      if (p.index_k) {
        if (at.slot >= 0 && p.enc.pairs != p.pe_pairs) a.load(cs, j, p.enc.pairs);
        Row y;
#pragma unroll
        for (int c = 0; c < 4; ++c) unpack8(v[c], y + 4 * c);
        norm_rotate<NORM>(y, p.enc, a, j);
        float m = transform<HAD>(y, j);
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        if (at.slot >= 0) {
          store_codes<HAD>(p.k_cache + at.slot * 128, y, m, j);
          if (j == 0) p.k_scale[at.slot] = encode_scale<HAD>(m);
        }
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
  // both kinds of CTAs at once, in shares that end together
  const int all = TE_CTAS * option_grid(), rows = ceil_div(p.T, TE_ROWS);
  const int latents = ceil_div(p.T, TE_THREADS / 32 * AP_TOKENS);
  p.row_ctas = min(rows, max(1, all / 3));
  const dim3 ctas(p.row_ctas + min(latents, max(1, all - p.row_ctas))), threads(TE_THREADS);
  count_launch();
  if (p.enc.norm_w)
    return p.enc.hadamard ? launch_pdl(append_kernel<true, true>, ctas, threads, 0, s, p)
                          : launch_pdl(append_kernel<true, false>, ctas, threads, 0, s, p);
  return p.enc.hadamard ? launch_pdl(append_kernel<false, true>, ctas, threads, 0, s, p)
                        : launch_pdl(append_kernel<false, false>, ctas, threads, 0, s, p);
}

}  // namespace dsa
