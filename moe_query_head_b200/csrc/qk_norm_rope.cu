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
// shuffles) of 16 values each, in two 16-byte-aligned pieces of 8. The pieces are chosen so
// that a lane holds both members of its eight pairs in either pairing: values 8 l .. 8 l + 7
// and the same of the second half of the rotated part (half pairing), or 16 neighbours
// (interleaved pairing); so the rotation needs no exchange. A thread keeps one token for all
// the heads of its chunk: the eight angles are formed once per token and chunk, in 64 bits
// (position times frequency in turns, whole turns dropped: a float32 angle at position 10^6
// is off by 0.03 rad), and the sine and cosine of the remainder in 32.
//
// Weight gradients: a thread sums its own 16 columns over its tokens and heads, the block
// joins its warps in a fixed order and writes one row of partial sums, and a second kernel
// adds the rows in a fixed order: no atomics, the same bits from run to run.
#include <string.h>

#include "gqe_common.cuh"
#include "qk_norm_rope.cuh"

namespace gqe {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;

template <int DH>
struct RowCfg {
  static constexpr int LANES = DH / 16;  // lanes that hold values
  // lanes of a row, a power of two
  static constexpr int LPR = LANES <= 1 ? 1 : LANES <= 2 ? 2 : LANES <= 4 ? 4 : 8;
  static constexpr int TPB = THREADS / LPR;  // tokens of a block
};

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0];
  const float4 b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Offsets of the two pieces of lane l's 16 values in a row.
__device__ __forceinline__ void pieces(const QkArgs& A, int l, int& pa, int& pb) {
  if (!A.interleaved && l < A.rot_dim / 16) {
    pa = 8 * l;
    pb = A.rot_dim / 2 + 8 * l;
  } else {
    pa = 16 * l;
    pb = 16 * l + 8;
  }
}

// cos and sin of pairs 8 l .. 8 l + 7 at position pos (lanes of the rotated part).
__device__ __forceinline__ void angles(const QkArgs& A, int l, int pos, float (&c)[8],
                                       float (&s)[8]) {
  constexpr double kInvTurn = 0.15915494309189533577;  // 1 / (2 pi)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    double t = (double)pos * (A.inv_freq[8 * l + i] * kInvTurn);
    t -= rint(t);
    sincospif((float)(t + t), &s[i], &c[i]);
  }
}

// Turns a lane's pairs by their angles (sign 1) or back (sign -1).
__device__ __forceinline__ void turn(bool interleaved, float (&a)[8], float (&b)[8],
                                     const float (&c)[8], const float (&s)[8], float sign) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x0 = a[2 * i], y0 = a[2 * i + 1], s0 = sign * s[i];
      a[2 * i] = x0 * c[i] - y0 * s0;
      a[2 * i + 1] = x0 * s0 + y0 * c[i];
      const float x1 = b[2 * i], y1 = b[2 * i + 1], s1 = sign * s[4 + i];
      b[2 * i] = x1 * c[4 + i] - y1 * s1;
      b[2 * i + 1] = x1 * s1 + y1 * c[4 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = a[i], y = b[i], si = sign * s[i];
      a[i] = x * c[i] - y * si;
      b[i] = x * si + y * c[i];
    }
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
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

// Loads of four heads are in flight per thread.
constexpr int UNROLL = 4;

// APPEND: one token per sequence; k and v rows go to row positions[t] of the caches.
template <typename T, int DH, bool APPEND>
__global__ void __launch_bounds__(THREADS) qk_forward_kernel(const __grid_constant__ QkArgs A) {
  using C = RowCfg<DH>;
  pdl_wait();
  pdl_allow_next();
  const int l = threadIdx.x % C::LPR;
  const int64_t t = (int64_t)blockIdx.x * C::TPB + threadIdx.x / C::LPR;
  bool on = t < A.M && l < C::LANES;
  int h0, h1;
  const int which = chunk_of(A, blockIdx.y, h0, h1);
  int pos = 0;
  if (t < A.M) pos = A.positions ? A.positions[t] : (int)(t % A.period);
  if constexpr (APPEND) {
    // -1: an idle slot; other positions outside the cache are reported. Nothing is written.
    if (t < A.M && (pos < 0 || pos >= A.L_max)) {
      if ((pos != -1 || !A.idle_ok) && l == 0) atomicExch(A.status, kStatusBadInput);
      on = false;
    }
  }
  int pa, pb;
  pieces(A, l, pa, pb);
  const bool rot = l < A.rot_dim / 16;
  const bool norm = A.norm && which < 2;
  float c[8], s[8], wa[8], wb[8];
  if (on && rot && which < 2) angles(A, l, pos, c, s);
  const float* w = which == 0 ? A.q_weight : A.k_weight;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    wa[i] = norm && w && l < C::LANES ? w[pa + i] : 1.f;
    wb[i] = norm && w && l < C::LANES ? w[pb + i] : 1.f;
  }
  const QkTensor& in = which == 0 ? A.q : which == 1 ? A.k : A.v;
  const QkTensor& out = which == 0 ? A.q_out : which == 1 ? A.k_out : A.v_out;
  const T* src = static_cast<const T*>(in.data) + t * in.token_stride;
  T* dst = static_cast<T*>(out.data) + t * out.token_stride;
  if (APPEND && which > 0) dst += (int64_t)pos * DH;
  for (int hb = h0; hb < h1; hb += UNROLL) {
    float a[UNROLL][8], b[UNROLL][8];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const bool live = on && hb + u < h1;
#pragma unroll
      for (int i = 0; i < 8; ++i) a[u][i] = b[u][i] = 0.f;
      if (live) {
        load8(src + (int64_t)(hb + u) * in.head_stride + pa, a[u]);
        load8(src + (int64_t)(hb + u) * in.head_stride + pb, b[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (hb + u >= h1) break;  // the same for every thread of the block
      if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(a[u][i], a[u][i], fmaf(b[u][i], b[u][i], ss));
        ss = row_sum<C::LPR>(ss);
        const float r = rsqrtf(ss * (1.f / DH) + A.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[u][i] *= r * wa[i];
          b[u][i] *= r * wb[i];
        }
      }
      if (rot && which < 2) turn(A.interleaved, a[u], b[u], c, s, 1.f);
      if (on) {
        store8(dst + (int64_t)(hb + u) * out.head_stride + pa, a[u]);
        store8(dst + (int64_t)(hb + u) * out.head_stride + pb, b[u]);
      }
    }
  }
}

// Blocks stride over the tokens, so that the partial weight sums stay few.
template <typename T, int DH>
__global__ void __launch_bounds__(THREADS) qk_backward_kernel(const __grid_constant__ QkArgs A) {
  using C = RowCfg<DH>;
  __shared__ float sw[WARPS][C::LPR][16];
  pdl_wait();
  pdl_allow_next();
  const int l = threadIdx.x % C::LPR;
  int h0, h1;
  const int which = chunk_of(A, blockIdx.y, h0, h1);
  int pa, pb;
  pieces(A, l, pa, pb);
  const bool rot = l < A.rot_dim / 16;
  const bool lane_on = l < C::LANES;
  float wa[8], wb[8], da[8], db[8];
  const float* w = which == 0 ? A.q_weight : A.k_weight;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    wa[i] = w && lane_on ? w[pa + i] : 1.f;
    wb[i] = w && lane_on ? w[pb + i] : 1.f;
    da[i] = db[i] = 0.f;
  }
  const QkTensor& in = which == 0 ? A.q : A.k;
  const QkTensor& gin = which == 0 ? A.q_out : A.k_out;
  const QkTensor& gout = which == 0 ? A.dq : A.dk;
  const int64_t step = (int64_t)gridDim.x * C::TPB;
  // the loop bound is the block's, so the shuffles below are met by whole warps
  for (int64_t t0 = (int64_t)blockIdx.x * C::TPB; t0 < A.M; t0 += step) {
    const int64_t t = t0 + threadIdx.x / C::LPR;
    const bool on = t < A.M && lane_on;
    float c[8], s[8];
    if (on && rot) angles(A, l, A.positions ? A.positions[t] : (int)(t % A.period), c, s);
    const T* x = static_cast<const T*>(in.data) + t * in.token_stride;
    const T* gy = static_cast<const T*>(gin.data) + t * gin.token_stride;
    for (int hb = h0; hb < h1; hb += 2) {
      float xa[2][8], xb[2][8], ga[2][8], gb[2][8];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bool live = on && hb + u < h1;
#pragma unroll
        for (int i = 0; i < 8; ++i) xa[u][i] = xb[u][i] = ga[u][i] = gb[u][i] = 0.f;
        if (live) {
          if (A.norm) {
            load8(x + (int64_t)(hb + u) * in.head_stride + pa, xa[u]);
            load8(x + (int64_t)(hb + u) * in.head_stride + pb, xb[u]);
          }
          load8(gy + (int64_t)(hb + u) * gin.head_stride + pa, ga[u]);
          load8(gy + (int64_t)(hb + u) * gin.head_stride + pb, gb[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int h = hb + u;
        if (h >= h1) break;  // the same for every thread of the block
        if (on && rot) turn(A.interleaved, ga[u], gb[u], c, s, -1.f);
        if (A.norm) {
          float ss = 0.f;
          float dot = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            ss = fmaf(xa[u][i], xa[u][i], fmaf(xb[u][i], xb[u][i], ss));
            dot = fmaf(ga[u][i] * wa[i], xa[u][i], fmaf(gb[u][i] * wb[i], xb[u][i], dot));
          }
          ss = row_sum<C::LPR>(ss);
          dot = row_sum<C::LPR>(dot);
          const float r = rsqrtf(ss * (1.f / DH) + A.eps);
          // mean(w g xh) r = (r^2 / d_h) dot, the factor of x in dx / r
          const float m = r * r * dot * (1.f / DH);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            da[i] = fmaf(ga[u][i] * r, xa[u][i], da[i]);
            db[i] = fmaf(gb[u][i] * r, xb[u][i], db[i]);
            ga[u][i] = r * (ga[u][i] * wa[i] - xa[u][i] * m);
            gb[u][i] = r * (gb[u][i] * wb[i] - xb[u][i] * m);
          }
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
          store8(d + pa, ga[u]);
          store8(d + pb, gb[u]);
        }
      }
    }
  }
  if (!A.partial) return;
  // the block's weight sums: lanes of a warp that hold the same columns, then the warps
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int o = C::LPR; o < 32; o <<= 1) {
      da[i] += __shfl_xor_sync(0xffffffffu, da[i], o);
      db[i] += __shfl_xor_sync(0xffffffffu, db[i], o);
    }
  }
  if (threadIdx.x % 32 < C::LPR) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sw[threadIdx.x / 32][l][i] = da[i];
      sw[threadIdx.x / 32][l][8 + i] = db[i];
    }
  }
  __syncthreads();
  if (threadIdx.x < C::LANES * 16) {
    const int ll = threadIdx.x / 16, e = threadIdx.x % 16;
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) v += sw[i][ll][e];
    int qa, qb;
    pieces(A, ll, qa, qb);
    A.partial[((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * DH + (e < 8 ? qa + e : qb + e - 8)] = v;
  }
}

// Adds the blocks' rows of partial weight sums: block 0 for q, 1 for k; a warp per column
// group would read strided, so thread (r, d) sums rows r, r + R, ... of column d, and column
// d's R sums are added in order.
__global__ void __launch_bounds__(1024) qk_weight_sum_kernel(const __grid_constant__ QkArgs A,
                                                             int blocks_x) {
  __shared__ float sm[1024];
  pdl_wait();
  pdl_allow_next();
  const int DH = A.d_h;
  const int which = blockIdx.x;
  float* out = which == 0 ? A.dq_weight : A.dk_weight;
  if (!out) return;
  const int64_t first = which == 0 ? 0 : (int64_t)A.chunks_q * blocks_x;
  const int64_t rows = (int64_t)(which == 0 ? A.chunks_q : A.chunks_k) * blocks_x;
  const int R = 1024 / DH;
  const int r = threadIdx.x / DH, d = threadIdx.x % DH;
  float v = 0.f;
  if (r < R)
    for (int64_t i = r; i < rows; i += R) v += A.partial[(first + i) * DH + d];
  sm[threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.x < DH) {
    float total = 0.f;
    for (int i = 0; i < R; ++i) total += sm[i * DH + threadIdx.x];
    out[threadIdx.x] = total;
  }
}

// Splits the heads into chunks so that the grid has about eight blocks of eight warps per SM
// (what the SMs hold; at 16384 tokens of 17 heads of 48: one chunk 20 us, this split 12 us);
// the smallest calls get a chunk per head.
void split_heads(QkArgs& A, int token_blocks, int num_sms, bool v_heads) {
  const int H = A.q.heads + A.k.heads * (v_heads ? 2 : 1);
  int want = (8 * num_sms + token_blocks - 1) / token_blocks;
  if (want < 1) want = 1;
  int per = (H + want - 1) / want;
  if (per < 1) per = 1;
  A.heads_per_chunk = per;
  A.chunks_q = (A.q.heads + per - 1) / per;
  A.chunks_k = (A.k.heads + per - 1) / per;
}

template <typename T, int DH>
int forward_dh(QkArgs& A, int num_sms, bool append, cudaStream_t st) {
  using C = RowCfg<DH>;
  const int tb = (int)((A.M + C::TPB - 1) / C::TPB);
  split_heads(A, tb, num_sms, append);
  const dim3 grid(tb, A.chunks_q + A.chunks_k * (append ? 2 : 1));
  const cudaError_t e = append ? launch_pdl(qk_forward_kernel<T, DH, true>, grid, dim3(THREADS), 0, st, A)
                               : launch_pdl(qk_forward_kernel<T, DH, false>, grid, dim3(THREADS), 0, st, A);
  return e == cudaSuccess ? 1 : -1;
}

template <typename T, int DH>
int backward_dh(QkArgs& A, int num_sms, cudaStream_t st) {
  using C = RowCfg<DH>;
  const int64_t tb = (A.M + C::TPB - 1) / C::TPB;
  split_heads(A, tb > num_sms ? num_sms : (int)tb, num_sms, false);
  const int ny = A.chunks_q + A.chunks_k;
  int bx = kQkPartialRows / ny;
  if (bx < 1) bx = 1;
  if (bx > tb) bx = (int)tb;
  if (launch_pdl(qk_backward_kernel<T, DH>, dim3(bx, ny), dim3(THREADS), 0, st, A) != cudaSuccess)
    return -1;
  if (!A.partial) return 1;
  return launch_pdl(qk_weight_sum_kernel, dim3(2), dim3(1024), 0, st, A, bx) == cudaSuccess ? 2 : -1;
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
