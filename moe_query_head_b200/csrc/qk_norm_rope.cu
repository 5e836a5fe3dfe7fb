// RMS norm of every query and key head with the position rotation in the same pass: forward,
// backward, and the serving form that writes one new token per sequence into its KV caches.
//
// For a head's row x of d_h values at position p, with weight w and r = 1 / sqrt(mean(x^2) +
// eps): h = w * x * r, and every pair (a, b) of the first rot_dim values at angle p f_i turns
// to (a cos - b sin, a sin + b cos). Backward, with g the upstream gradient turned back by
// the same angle and xh = x r: dw = sum over rows of g * xh, dx = r (w g - xh mean(w g xh)).
//
// The work is bound by memory (two bytes moved per bf16 value and direction, about ten
// operations on it), so each value is read once and written once and everything between
// stays in registers. Lanes: a row is d_h / 16 lanes (rounded up to a power of two for the
// shuffles, see RowCfg) of 16 values each, in two 16-byte-aligned pieces of 8. The pieces are chosen so
// that a lane holds both members of its eight pairs in either pairing: values 8 l .. 8 l + 7
// and the same of the second half of the rotated part (half pairing), or 16 neighbours
// (interleaved pairing); so the rotation needs no exchange. In registers the members are x[8]
// and y[8] in both pairings, and the arithmetic runs on packed pairs of floats. A thread keeps
// one token for all the heads of its chunk: the eight angles are formed once per token and
// chunk, in 64 bits (position times frequency in turns, whole turns dropped: a float32 angle
// at position 10^6 is off by 0.03 rad), and the sine and cosine of the remainder in 32; they
// are then multiplied by the weights, so that a value costs one product, one fma and the
// row's factor. What bounds the kernel beside the memory is the instruction issue: forming
// the angles costs as much as two heads, so the chunks are as long as the grid allows.
//
// Weight gradients: a thread sums its own 16 columns over its tokens and heads, the block
// joins its warps in a fixed order and writes one row of partial sums, and a second kernel
// adds the rows in a fixed order: no atomics, the same bits from run to run.
#include <string.h>

#include "gqe_common.cuh"
#include "qk_norm_rope.cuh"
#include "tc_ptx.cuh"

namespace gqe {
namespace {

using tc::fma2;
using tc::mul2;

constexpr int THREADS = 128;
constexpr int WARPS = THREADS / 32;

template <int DH>
struct RowCfg {
  static constexpr int LANES = DH / 16;  // lanes that hold values
  // Lanes of a row: exactly those for 3, 5 and 6 (10, 6 and 5 rows a warp; their sums go over
  // the row's lanes one by one), else the next power of two (the sum by halves). 
  static constexpr bool EXACT = LANES == 3 || LANES == 5 || LANES == 6;
  static constexpr int LPR = EXACT ? LANES : LANES <= 1 ? 1 : LANES <= 2 ? 2 : LANES <= 4 ? 4 : 8;
  static constexpr int RPW = 32 / LPR;     // rows of a warp
  static constexpr int TPB = WARPS * RPW;  // tokens of a block
};
// A thread's row in its block, its lane in the row, and whether it holds values.
template <int DH>
struct Place {
  using C = RowCfg<DH>;
  int row, l;
  bool holds;
  __device__ __forceinline__ Place() {
    const int lane = threadIdx.x % 32;
    l = lane % C::LPR;
    row = threadIdx.x / 32 * C::RPW + lane / C::LPR;
    holds = l < C::LANES && lane / C::LPR < C::RPW;
    if (lane / C::LPR >= C::RPW) row = 1 << 30;  // no token
  }
};

// Sixteen values of a row as they come from memory: two pieces of 8.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const __nv_bfloat16* a, const __nv_bfloat16* b) {
    const uint4 u = *reinterpret_cast<const uint4*>(a), v = *reinterpret_cast<const uint4*>(b);
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    w[4] = v.x; w[5] = v.y; w[6] = v.z; w[7] = v.w;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0u;
  }
  // pair members 2 i and 2 i + 1 as packed floats
  template <bool INTER>
  __device__ __forceinline__ void pair2(int i, float2& x, float2& y) const {
    if constexpr (INTER) {
      x = make_float2(lo(w[2 * i]), lo(w[2 * i + 1]));
      y = make_float2(hi(w[2 * i]), hi(w[2 * i + 1]));
    } else {
      x = make_float2(lo(w[i]), hi(w[i]));
      y = make_float2(lo(w[4 + i]), hi(w[4 + i]));
    }
  }
  template <bool INTER>
  __device__ __forceinline__ void set2(int i, float2 x, float2 y) {
    if constexpr (INTER) {
      w[2 * i] = tc::pack_bf16x2(x.x, y.x);
      w[2 * i + 1] = tc::pack_bf16x2(x.y, y.y);
    } else {
      w[i] = tc::pack_bf16x2(x.x, x.y);
      w[4 + i] = tc::pack_bf16x2(y.x, y.y);
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16* a, __nv_bfloat16* b) const {
    *reinterpret_cast<uint4*>(a) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(b) = make_uint4(w[4], w[5], w[6], w[7]);
  }
  static __device__ __forceinline__ float lo(uint32_t v) { return __uint_as_float(v << 16); }
  static __device__ __forceinline__ float hi(uint32_t v) {
    return __uint_as_float(v & 0xffff0000u);
  }
};
template <>
struct Raw<float> {
  float v[16];
  __device__ __forceinline__ void load(const float* a, const float* b) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4* p = reinterpret_cast<const float4*>(h ? b : a);
      const float4 s = p[0], t = p[1];
      v[8 * h] = s.x; v[8 * h + 1] = s.y; v[8 * h + 2] = s.z; v[8 * h + 3] = s.w;
      v[8 * h + 4] = t.x; v[8 * h + 5] = t.y; v[8 * h + 6] = t.z; v[8 * h + 7] = t.w;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
  }
  template <bool INTER>
  __device__ __forceinline__ void pair2(int i, float2& x, float2& y) const {
    if constexpr (INTER) {
      x = make_float2(v[4 * i], v[4 * i + 2]);
      y = make_float2(v[4 * i + 1], v[4 * i + 3]);
    } else {
      x = make_float2(v[2 * i], v[2 * i + 1]);
      y = make_float2(v[8 + 2 * i], v[8 + 2 * i + 1]);
    }
  }
  template <bool INTER>
  __device__ __forceinline__ void set2(int i, float2 x, float2 y) {
    if constexpr (INTER) {
      v[4 * i] = x.x; v[4 * i + 2] = x.y;
      v[4 * i + 1] = y.x; v[4 * i + 3] = y.y;
    } else {
      v[2 * i] = x.x; v[2 * i + 1] = x.y;
      v[8 + 2 * i] = y.x; v[8 + 2 * i + 1] = y.y;
    }
  }
  __device__ __forceinline__ void store(float* a, float* b) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float4* p = reinterpret_cast<float4*>(h ? b : a);
      p[0] = make_float4(v[8 * h], v[8 * h + 1], v[8 * h + 2], v[8 * h + 3]);
      p[1] = make_float4(v[8 * h + 4], v[8 * h + 5], v[8 * h + 6], v[8 * h + 7]);
    }
  }
};

// Offsets of the two pieces of lane l's 16 values in a row.
template <bool INTER>
__device__ __forceinline__ void pieces(const QkArgs& A, int l, int& pa, int& pb) {
  if (!INTER && l < A.rot_dim / 16) {
    pa = 8 * l;
    pb = A.rot_dim / 2 + 8 * l;
  } else {
    pa = 16 * l;
    pb = 16 * l + 8;
  }
}

// Weights of the members of lane pair i (ones without weights).
template <bool INTER>
__device__ __forceinline__ void weights2(const float* w, bool use, int pa, int pb, int i, float2& wx,
                                         float2& wy) {
  wx = wy = make_float2(1.f, 1.f);
  if (!use || !w) return;
  if constexpr (INTER) {
    const int p = i < 2 ? pa + 4 * i : pb + 4 * (i - 2);
    wx = make_float2(w[p], w[p + 2]);
    wy = make_float2(w[p + 1], w[p + 3]);
  } else {
    wx = make_float2(w[pa + 2 * i], w[pa + 2 * i + 1]);
    wy = make_float2(w[pb + 2 * i], w[pb + 2 * i + 1]);
  }
}

// cos and sin of the lane's pairs 2 i, 2 i + 1 at position pos; 1 and 0 where the lane is not
// rotated. float32 rows take the full functions; for bf16 rows, rounded at 2^-8, the fast ones
// (absolute error 2^-21) cost a tenth of the instructions.
template <typename T>
__device__ __forceinline__ void angles(const QkArgs& A, int l, int pos, bool rot, float2 (&c)[4],
                                       float2 (&s)[4]) {
  constexpr double kInvTurn = 0.15915494309189533577;  // 1 / (2 pi)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = make_float2(1.f, 1.f);
    s[i] = make_float2(0.f, 0.f);
    if (!rot) continue;
    const double* f = A.inv_freq + 8 * l + 2 * i;
    float cc[2], ss[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      double t = (double)pos * (f[e] * kInvTurn);
      t -= rint(t);
      if constexpr (sizeof(T) == 4) sincospif((float)(t + t), &ss[e], &cc[e]);
      else __sincosf((float)t * 6.2831853071795865f, &ss[e], &cc[e]);
    }
    c[i] = make_float2(cc[0], cc[1]);
    s[i] = make_float2(ss[0], ss[1]);
  }
}

__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }

// Sum over a row's lanes, the same bits in each.
template <int DH>
__device__ __forceinline__ float row_sum(float v) {
  using C = RowCfg<DH>;
  if constexpr (C::EXACT) {
    const int first = threadIdx.x % 32 / C::LPR * C::LPR;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < C::LPR; ++j) sum += __shfl_sync(0xffffffffu, v, first + j);
    return sum;
  } else {
#pragma unroll
    for (int o = C::LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
}

// Chunk y of the heads: tensor (0 q, 1 k, 2 v) and its heads [h0, h1). Chunks do not cross
// tensors, so a block's weight sums belong to one of them.
__device__ __forceinline__ int chunk_of(const QkArgs& A, int y, int& h0, int& h1) {
  int which = 0;
  if (y >= A.chunks_q) {
    y -= A.chunks_q;
    which = 1;
    if (y >= A.chunks_k) {
      y -= A.chunks_k;
      which = 2;
    }
  }
  const int H = which == 0 ? A.q.heads : A.k.heads;
  h0 = y * A.heads_per_chunk;
  h1 = min(H, h0 + A.heads_per_chunk);
  return which;
}

// Heads whose loads are in flight per thread.
// (32768 tokens of 17 heads of 128, sixteen warps an SM: forward 52.8 us at four, 59.1 at two, 53.1
// at six; backward 87.7 at two, 95.9 at one, 100 at three. More warps spill.)
template <typename T>
constexpr int kUnrollF = sizeof(T) == 2 ? 4 : 2;
template <typename T>
constexpr int kUnrollB = sizeof(T) == 2 ? 2 : 1;

// APPEND: one token per sequence; k and v rows go to row positions[t] of the caches.
template <typename T, int DH, bool INTER, bool APPEND>
__global__ void __launch_bounds__(THREADS, 4) qk_forward_kernel(const __grid_constant__ QkArgs A) {
  using C = RowCfg<DH>;
  constexpr int U = kUnrollF<T>;
  pdl_wait();
  pdl_allow_next();
  const Place<DH> at;
  const int l = at.l;
  const int64_t t = (int64_t)blockIdx.x * C::TPB + at.row;
  bool on = t < A.M && at.holds;
  int h0, h1;
  const int which = chunk_of(A, blockIdx.y, h0, h1);
  int pos = 0;
  if (t < A.M) pos = A.positions ? A.positions[t] : (int)(t % A.period);
  if constexpr (APPEND) {
    // -1: an idle slot; other positions outside the cache are reported. Nothing is written.
    if (t < A.M && (pos < 0 || pos >= A.L_max)) {
      if ((pos != -1 || !A.idle_ok) && l == 0) atomicCAS(A.status, kStatusOk, kStatusBadInput);
      on = false;
    }
  }
  int pa, pb;
  pieces<INTER>(A, l, pa, pb);
  const QkTensor& in = which == 0 ? A.q : which == 1 ? A.k : A.v;
  const QkTensor& out = which == 0 ? A.q_out : which == 1 ? A.k_out : A.v_out;
  const int64_t in_step = in.head_stride, out_step = out.head_stride;
  const T* src = static_cast<const T*>(in.data) + t * in.token_stride + h0 * in_step;
  T* dst = static_cast<T*>(out.data) + t * out.token_stride + h0 * out_step;
  if (APPEND && which > 0) dst += (int64_t)pos * DH;
  Raw<T> raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) raw[u].zero();  // lanes without values stay zero
  auto fetch = [&](int hb) {
    if (!on) return;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (hb + u < h1) raw[u].load(src + pa, src + pb);
      src += in_step;
    }
  };
  fetch(h0);  // the first heads are on their way while the angles are formed
  const bool norm = A.norm && which < 2;
  const bool rot = l < A.rot_dim / 16 && which < 2;
  // cos and sin times the weights of the members they meet
  float2 cx[4], cy[4], sx[4], sy[4];
  if (which < 2) {
    float2 c[4], s[4];
    angles<T>(A, l, pos, on && rot, c, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 wx, wy;
      weights2<INTER>(which == 0 ? A.q_weight : A.k_weight, norm && at.holds, pa, pb, i, wx, wy);
      cx[i] = mul2(c[i], wx);
      sx[i] = mul2(s[i], wx);
      cy[i] = mul2(c[i], wy);
      sy[i] = neg2(mul2(s[i], wy));
    }
  }
  for (int hb = h0; hb < h1; hb += U) {
    if (hb > h0) fetch(hb);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (hb + u >= h1) break;  // the same for every thread of the block
      if (which < 2) {
        float2 x[4], y[4];
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          raw[u].template pair2<INTER>(i, x[i], y[i]);
          ss = fma2(x[i], x[i], fma2(y[i], y[i], ss));
        }
        if (norm) {
          const float f = rsqrtf(row_sum<DH>(ss.x + ss.y) * (1.f / DH) + A.eps);
          const float2 f2 = make_float2(f, f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = mul2(x[i], f2);
            y[i] = mul2(y[i], f2);
          }
        }
        Raw<T> r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (rot)
            r.template set2<INTER>(i, fma2(x[i], cx[i], mul2(y[i], sy[i])),
                                   fma2(x[i], sx[i], mul2(y[i], cy[i])));
          else
            r.template set2<INTER>(i, mul2(x[i], cx[i]), mul2(y[i], cy[i]));
        }
        if (on) r.store(dst + pa, dst + pb);
      } else {
        if (on) raw[u].store(dst + pa, dst + pb);
      }
      dst += out_step;
    }
  }
}

// Blocks stride over the tokens, so that the partial weight sums stay few.
template <typename T, int DH, bool INTER>
__global__ void __launch_bounds__(THREADS, 4) qk_backward_kernel(const __grid_constant__ QkArgs A) {
  using C = RowCfg<DH>;
  constexpr int U = kUnrollB<T>;
  __shared__ float sw[THREADS][17];
  pdl_wait();
  pdl_allow_next();
  const Place<DH> at;
  const int l = at.l;
  int h0, h1;
  const int which = chunk_of(A, blockIdx.y, h0, h1);
  int pa, pb;
  pieces<INTER>(A, l, pa, pb);
  const bool rot = l < A.rot_dim / 16;
  const bool lane_on = at.holds;
  float2 wx[4], wy[4], dx[4], dy[4];  // weights, and the sums of their gradients
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    weights2<INTER>(which == 0 ? A.q_weight : A.k_weight, A.norm && lane_on, pa, pb, i, wx[i], wy[i]);
    dx[i] = dy[i] = make_float2(0.f, 0.f);
  }
  const QkTensor& in = which == 0 ? A.q : A.k;
  const QkTensor& gin = which == 0 ? A.q_out : A.k_out;
  const QkTensor& gout = which == 0 ? A.dq : A.dk;
  const int64_t x_step = in.head_stride, g_step = gin.head_stride;
  const int64_t step = (int64_t)gridDim.x * C::TPB;
  // the loop bound is the block's, so the shuffles below are met by whole warps
  for (int64_t t0 = (int64_t)blockIdx.x * C::TPB; t0 < A.M; t0 += step) {
    const int64_t t = t0 + at.row;
    const bool on = t < A.M && lane_on;
    const T* xp = static_cast<const T*>(in.data) + t * in.token_stride + h0 * x_step;
    const T* gp = static_cast<const T*>(gin.data) + t * gin.token_stride + h0 * g_step;
    Raw<T> xr[U], gr[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {  // rows without values add nothing
      xr[u].zero();
      gr[u].zero();
    }
    auto fetch = [&](int hb) {
      if (!on) return;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (hb + u < h1) {
          if (A.norm) xr[u].load(xp + pa, xp + pb);
          gr[u].load(gp + pa, gp + pb);
        }
        xp += x_step;
        gp += g_step;
      }
    };
    fetch(h0);
    float2 c[4], s[4];
    {
      const int pos = t < A.M ? (A.positions ? A.positions[t] : (int)(t % A.period)) : 0;
      angles<T>(A, l, pos, on && rot, c, s);
    }
    for (int hb = h0; hb < h1; hb += U) {
      if (hb > h0) fetch(hb);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = hb + u;
        if (h >= h1) break;  // the same for every thread of the block
        float2 gx[4], gy[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          gr[u].template pair2<INTER>(i, gx[i], gy[i]);
          if (rot) {
            const float2 a = gx[i], b = gy[i];
            gx[i] = fma2(a, c[i], mul2(b, s[i]));
            gy[i] = fma2(b, c[i], neg2(mul2(a, s[i])));
          }
        }
        Raw<T> r;
        if (A.norm) {
          float2 x[4], y[4], ss = make_float2(0.f, 0.f), dot = make_float2(0.f, 0.f);
          float2 ux[4], uy[4];  // weighted gradients
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            xr[u].template pair2<INTER>(i, x[i], y[i]);
            ss = fma2(x[i], x[i], fma2(y[i], y[i], ss));
            ux[i] = mul2(gx[i], wx[i]);
            uy[i] = mul2(gy[i], wy[i]);
            dot = fma2(ux[i], x[i], fma2(uy[i], y[i], dot));
          }
          // places without a token (zeros, whose factor is infinite without an epsilon) add nothing
          const float mean = row_sum<DH>(ss.x + ss.y) * (1.f / DH);
          const float f = on ? rsqrtf(mean + A.eps) : 0.f;
          // dx = f (w g - xh mean(w g xh)), the mean being f dot / d_h
          const float m = -f * f * (1.f / DH) * row_sum<DH>(dot.x + dot.y);
          const float2 f2 = make_float2(f, f), m2 = make_float2(m, m);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = mul2(x[i], f2);  // xh
            y[i] = mul2(y[i], f2);
            dx[i] = fma2(gx[i], x[i], dx[i]);
            dy[i] = fma2(gy[i], y[i], dy[i]);
            r.template set2<INTER>(i, fma2(x[i], m2, mul2(ux[i], f2)),
                                   fma2(y[i], m2, mul2(uy[i], f2)));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) r.template set2<INTER>(i, gx[i], gy[i]);
        }
        if (on) {
          T* d = static_cast<T*>(gout.data) + t * gout.token_stride;
          if (which == 0 && A.sel && h < A.routed) {
            // a routed stream's gradient goes to the block of the expert it was projected by
            d += (int64_t)((h / A.top_k) * A.experts + A.sel[t * A.sel_stride + A.sel_off + h]) * DH;
          } else if (which == 0 && A.sel) {
            d = static_cast<T*>(A.dq_shared) + t * DH;
          } else {
            d += (int64_t)h * gout.head_stride;
          }
          r.store(d + pa, d + pb);
        }
      }
    }
  }
  if (!A.partial) return;
  // the block's weight sums: the rows of every warp, in order
  Raw<float> v;  // in the row's order
#pragma unroll
  for (int i = 0; i < 4; ++i) v.template set2<INTER>(i, dx[i], dy[i]);
#pragma unroll
  for (int i = 0; i < 16; ++i) sw[threadIdx.x][i] = v.v[i];
  __syncthreads();
  if (threadIdx.x < DH) {
    const int ll = threadIdx.x / 16, e = threadIdx.x % 16;
    float sum = 0.f;
    for (int w = 0; w < WARPS; ++w)
#pragma unroll
      for (int i = 0; i < C::RPW; ++i) sum += sw[w * 32 + i * C::LPR + ll][e];
    int qa, qb;
    pieces<INTER>(A, ll, qa, qb);
    A.partial[((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * DH + (e < 8 ? qa + e : qb + e - 8)] =
        sum;
  }
}

// Adds the blocks' rows of partial weight sums: blockIdx.y 0 for q, 1 for k, and 16 columns a
// block. Thread (r, d) sums rows r, r + 64, ... of column d; a column's 64 sums are added in
// order.
__global__ void __launch_bounds__(1024) qk_weight_sum_kernel(const __grid_constant__ QkArgs A,
                                                             int blocks_x) {
  __shared__ float sm[64][17];
  pdl_wait();
  pdl_allow_next();
  const int which = blockIdx.y;
  float* out = which == 0 ? A.dq_weight : A.dk_weight;
  if (!out) return;
  const int64_t first = which == 0 ? 0 : (int64_t)A.chunks_q * blocks_x;
  const int rows = (which == 0 ? A.chunks_q : A.chunks_k) * blocks_x;
  const int r = threadIdx.x / 16, d = threadIdx.x % 16;
  const float* p = A.partial + first * A.d_h + blockIdx.x * 16 + d;
  float v = 0.f;
#pragma unroll 4
  for (int i = r; i < rows; i += 64) v += p[(int64_t)i * A.d_h];
  sm[r][d] = v;
  __syncthreads();
  if (threadIdx.x < 16) {
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < 64; ++i) total += sm[i][threadIdx.x];
    out[blockIdx.x * 16 + threadIdx.x] = total;
  }
}

// Splits the heads into chunks of equal length: as many as give the grid eight blocks per SM
// (four of them resident), up to one per head for the smallest calls. (16384 tokens of 17 heads
// of 48: 15.6 us at eight and at four, 17.6 at sixteen; 5001 float32 tokens of 25 heads of 64:
// 14.9, 15.8, 16.0. Blocks of 256 threads: 16.1 and 15.9.)
void split_heads(QkArgs& A, int64_t token_blocks, int num_sms, bool v_heads) {
  const int H = A.q.heads + A.k.heads * (v_heads ? 2 : 1);
  int64_t want = (8 * (int64_t)num_sms + token_blocks - 1) / token_blocks;
  if (want > H) want = H;
  if (want < 1) want = 1;
  const int per = (int)((H + want - 1) / want);
  A.heads_per_chunk = per;
  A.chunks_q = (A.q.heads + per - 1) / per;
  A.chunks_k = (A.k.heads + per - 1) / per;
}

template <typename T, int DH, bool INTER>
int forward_dh(QkArgs& A, int num_sms, bool append, cudaStream_t st) {
  using C = RowCfg<DH>;
  const int tb = (int)((A.M + C::TPB - 1) / C::TPB);
  split_heads(A, tb, num_sms, append);
  const dim3 grid(tb, A.chunks_q + A.chunks_k * (append ? 2 : 1));
  const cudaError_t e =
      append ? launch_pdl(qk_forward_kernel<T, DH, INTER, true>, grid, dim3(THREADS), 0, st, A)
             : launch_pdl(qk_forward_kernel<T, DH, INTER, false>, grid, dim3(THREADS), 0, st, A);
  return e == cudaSuccess ? 1 : -1;
}

template <typename T, int DH, bool INTER>
int backward_dh(QkArgs& A, int num_sms, cudaStream_t st) {
  using C = RowCfg<DH>;
  const int64_t tb = (A.M + C::TPB - 1) / C::TPB;
  split_heads(A, tb, num_sms, false);
  const int ny = A.chunks_q + A.chunks_k;
  int bx = kQkPartialRows / ny;
  if (bx < 1) bx = 1;
  if (bx > tb) bx = (int)tb;
  if (launch_pdl(qk_backward_kernel<T, DH, INTER>, dim3(bx, ny), dim3(THREADS), 0, st, A) !=
      cudaSuccess)
    return -1;
  if (!A.partial) return 1;
  return launch_pdl(qk_weight_sum_kernel, dim3(DH / 16, 2), dim3(1024), 0, st, A, bx) == cudaSuccess
             ? 2
             : -1;
}

template <typename T, int DH>
int forward_dh(QkArgs& A, int num_sms, bool append, cudaStream_t st) {
  return A.interleaved ? forward_dh<T, DH, true>(A, num_sms, append, st)
                       : forward_dh<T, DH, false>(A, num_sms, append, st);
}
template <typename T, int DH>
int backward_dh(QkArgs& A, int num_sms, cudaStream_t st) {
  return A.interleaved ? backward_dh<T, DH, true>(A, num_sms, st)
                       : backward_dh<T, DH, false>(A, num_sms, st);
}

template <typename T>
int forward_t(QkArgs& A, int num_sms, bool append, cudaStream_t st) {
  switch (A.d_h) {
    case 16: return forward_dh<T, 16>(A, num_sms, append, st);
    case 32: return forward_dh<T, 32>(A, num_sms, append, st);
    case 48: return forward_dh<T, 48>(A, num_sms, append, st);
    case 64: return forward_dh<T, 64>(A, num_sms, append, st);
    case 80: return forward_dh<T, 80>(A, num_sms, append, st);
    case 96: return forward_dh<T, 96>(A, num_sms, append, st);
    case 112: return forward_dh<T, 112>(A, num_sms, append, st);
    case 128: return forward_dh<T, 128>(A, num_sms, append, st);
    default: return -1;
  }
}

template <typename T>
int backward_t(QkArgs& A, int num_sms, cudaStream_t st) {
  switch (A.d_h) {
    case 16: return backward_dh<T, 16>(A, num_sms, st);
    case 32: return backward_dh<T, 32>(A, num_sms, st);
    case 48: return backward_dh<T, 48>(A, num_sms, st);
    case 64: return backward_dh<T, 64>(A, num_sms, st);
    case 80: return backward_dh<T, 80>(A, num_sms, st);
    case 96: return backward_dh<T, 96>(A, num_sms, st);
    case 112: return backward_dh<T, 112>(A, num_sms, st);
    case 128: return backward_dh<T, 128>(A, num_sms, st);
    default: return -1;
  }
}

}  // namespace

int launch_qk_forward(QkArgs& A, int num_sms, bool append, cudaStream_t st) {
  return A.dtype == GQE_BF16 ? forward_t<__nv_bfloat16>(A, num_sms, append, st)
                             : forward_t<float>(A, num_sms, append, st);
}

int launch_qk_backward(QkArgs& A, int num_sms, cudaStream_t st) {
  return A.dtype == GQE_BF16 ? backward_t<__nv_bfloat16>(A, num_sms, st)
                             : backward_t<float>(A, num_sms, st);
}

}  // namespace gqe
