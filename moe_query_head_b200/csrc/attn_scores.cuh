// Arguments and device helpers shared by the kernels of the attention with capped, biased and
// masked scores (attn_scores.cu, attn_scores_bwd.cu, attn_scores_decode.cu).
//
// Query stream s of token t (position t of its sequence) sees the keys u of its KV head with
// begin_t <= u < end_t. Its scores are
//   z = scale <q, k_u>;  z = softcap tanh(z / softcap) if softcap > 0;  z -= slope_s |t - u|,
// its weights the softmax of z over those keys; a row without keys gives zeros.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "gqe_common.cuh"
#include "qk_norm_rope.cuh"
#include "tc_ptx.cuh"

namespace gqe {

struct AttnArgs {
  int B = 0, T = 0;           // sequences and tokens of each (prefill and backward)
  int S = 0, G = 0, k = 0;    // query streams, KV heads, streams per KV head (S = G k, G k + 1)
  int d_h = 0;
  int causal = 0;
  float scale = 0.f;          // of <q, k>
  float softcap = 0.f;        // 0: none
  const float* slopes = nullptr;        // [S] or none
  const int32_t* key_begin = nullptr;   // [B T] or none (0)
  const int32_t* key_end = nullptr;     // [B T] or none (T)
  QkTensor q, kk, v, out;               // bf16, [heads, B T, d_h] by strides
  // inside the layer: the shared stream's column of Z differs from S - 1 blocks, and routed
  // streams may be scaled by their router probability
  int64_t last_off = -1;                // offset of stream S - 1 in `out` (-1: by the stride)
  const float* psel = nullptr;          // [B T, psel_stride] at column psel_off + s
  int psel_stride = 0, psel_off = 0;
  float* lse = nullptr;                 // [S, B T] log2-sum-exp2 of the scores, -inf without keys
  // backward
  QkTensor dout, dq, dk, dv;
  float* dsum = nullptr;                // [S, B T] rowsum(dout * out)
  int dsum_given = 0;                   // dsum holds them already (the layer's combine does)
  int2* blocks = nullptr;               // [B, ceil(T / 128)] (first key, end of keys) of 128 rows
  const int32_t* sel = nullptr;         // inside the layer: dq goes to its expert's block
  void* dq_shared = nullptr;
  int64_t sel_stride = 0;
  int sel_off = 0, experts = 0;
  int32_t* status = nullptr;
  int64_t spin = 0;
};

// Each returns the number of kernels launched, or -1.
int launch_attn_scores(const AttnArgs& a, cudaStream_t st);
int launch_attn_scores_backward(const AttnArgs& a, cudaStream_t st);

// Tensor map of [heads, B T, d_h] rows cut into chunks of cw columns: coordinates (column in
// the chunk, position, chunk, head, sequence). Positions past a sequence read zeros.
bool tmap_heads(CUtensorMap* m, const QkTensor& t, int B, int T, int d_h, int cw, int box_rows,
                CUtensorMapSwizzle sw);

constexpr float kLog2e = 1.4426950408889634f;

// The caps that are served. tc::tanh_from_2log2 is off by 1e-7, so a capped score by 1e-7 of the
// cap: 8e-4 at 2^13, a fifth of a weight's bf16 half step; far larger caps would lose the score
// itself. (The polynomial below serves only scores it gives to 5e-4.) At the lower end and for
// scales below 2^60 the tanh's argument stays finite.
inline bool cap_in_range(float scale, float softcap) {
  return softcap == 0.f || (softcap >= 0x1p-13f && softcap <= 0x1p13f && scale <= 0x1p60f);
}

// The scales that are served with a distance bias: the uncapped forward forms slope / scale, which
// must neither overflow nor lose its third bf16 piece.
inline bool bias_in_range(float scale, const float* slopes) {
  return !slopes || scale == 0.f || (scale >= 0x1p-60f && scale <= 0x1p60f);
}

namespace tc {

__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, int c0, int c1,
                                            int c2, int c3, int c4, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4),
      "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(x) = 1 - 2 / (e^(2x) + 1): absolute error about 1e-7 over the whole range, saturating
// to +-1 where the exponential overflows or vanishes; NaN stays NaN. x2 is 2 log2(e) x.
__device__ __forceinline__ float tanh_from_2log2(float x2) {
  return fmaf(-2.f, rcp_approx(ex2(x2) + 1.f), 1.f);
}

// The cap's tanh of a pair of scores. An odd polynomial of degree 7 on the FMA pipe serves
// scores up to three quarters of the cap (the ordinary case: caps are chosen above the scores),
// but none above kPolyScore; a warp that meets larger ones takes the exponential and a reciprocal
// for its tile, 16 cycles of the MUFU unit per score and warp against the polynomial's 5 of the
// FMA pipe. x Q(x^2) was fitted for minimal largest relative error on [0, 3/4] (iteratively
// reweighted least squares): 1.1e-5. A score of 44 is so off by 2^-11 at most, an eighth of its
// weight's bf16 half step; tiles of a row, and the forward and its backward, may therefore
// differ in the form they take. At a cap of 50 three quarters of the cap, 37, is the lower bound
// of the two: 3.5e-4. (Degree 9 up to the cap itself: one more FMA per score, no faster where
// scores are large.) The host folds the scores' factor into the coefficients, so the raw score
// is the polynomial's argument.
constexpr float kPolyScore = 44.f;
struct CapForm {
  float2 c[4];   // Q's coefficients times factor^(2 i + 1), each twice
  float limit;   // largest |score| the polynomial serves
  float t2;      // factor 2 log2(e): the argument of tanh_from_2log2
  float log2;    // softcap log2(e)
  int on;
};
inline CapForm cap_form(float scale, float softcap) {
  CapForm f = {};
  if (!(softcap > 0.f)) return f;
  const double q[4] = {0.9999889837677725, -0.3326967088343551, 0.12742696990927016,
                       -0.03545278562805266};
  const double x = (double)scale / softcap;
  double power = x;
  for (int i = 0; i < 4; ++i) {
    f.c[i] = make_float2((float)(q[i] * power), (float)(q[i] * power));
    power *= x * x;
  }
  f.limit = (float)(0.75 / x);
  // beyond float32's range for the coefficients nothing is served by the polynomial
  if (!(f.limit < 1e4f && f.limit > 1e-4f)) f.limit = 0.f;
  f.limit = fminf(f.limit, kPolyScore / scale);
  f.t2 = (float)(x * 2.8853900817779268);
  f.log2 = softcap * 1.4426950408889634f;
  f.on = 1;
  return f;
}
template <bool POLY>
__device__ __forceinline__ float2 cap_tanh(const CapForm& f, float2 s) {
  if constexpr (POLY) {
    const float2 y = mul2(s, s);
    float2 p = fma2(f.c[3], y, f.c[2]);
    p = fma2(p, y, f.c[1]);
    p = fma2(p, y, f.c[0]);
    return mul2(p, s);
  } else {
    return make_float2(tanh_from_2log2(s.x * f.t2), tanh_from_2log2(s.y * f.t2));
  }
}
// Largest |s| of N scores (NaN aside).
template <int N>
__device__ __forceinline__ float abs_max(const float* s) {
  float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < N; i += 2) m[(i >> 1) & 3] = fmax3(m[(i >> 1) & 3], fabsf(s[i]), fabsf(s[i + 1]));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// Runs f with the compile-time flags of the score's form (the same for the whole grid).
template <typename F>
__device__ __forceinline__ void by_form(bool cap, bool bias, F&& f) {
  using Yes = std::integral_constant<bool, true>;
  using No = std::integral_constant<bool, false>;
  if (cap) {
    if (bias) f(Yes{}, Yes{});
    else f(Yes{}, No{});
  } else {
    if (bias) f(No{}, Yes{});
    else f(No{}, No{});
  }
}
// Runs f with a warp-uniform flag as a compile-time one.
template <typename F>
__device__ __forceinline__ void by_flag(bool flag, F&& f) {
  if (flag) f(std::integral_constant<bool, true>{});
  else f(std::integral_constant<bool, false>{});
}

// 2^x of a pair on the FMA pipe, as exp2_fma.cuh's exp2_fma2 (nearest integer n of x by adding
// and subtracting 1.5 * 2^23, then the degree-2 polynomial of 2^(x - n) fitted there, 1.9e-3,
// the size of the bf16 rounding that follows), with two differences. The clamp is at -127: there
// n is exact, the polynomial is 1 + 4.7e-4 and the exponent field becomes 0, which leaves 5e-42,
// a zero in bf16, so a masked score (-inf) has no weight at all however large the finite value
// beside it (below -126 what is left of a weight is denormal or nothing). And NaN is kept: the
// clamp passes it on and the exponent addition turns it into the largest float (infinity in
// bf16), so that a row that sees a NaN score does not just lose that key; what sums such
// weights says NaN.
__device__ __forceinline__ float2 exp2_fma2_nan(float2 x) {
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(x.x));  // -127
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(x.y));
  const float2 j = add2(x, make_float2(kMagic, kMagic));
  const float2 n = add2(j, make_float2(-kMagic, -kMagic));
  const float2 f = fma2(n, make_float2(-1.0f, -1.0f), x);
  float2 p = fma2(make_float2(0.23876238f, 0.23876238f), f, make_float2(0.70411982f, 0.70411982f));
  p = fma2(p, f, make_float2(1.00047162f, 1.00047162f));
  const uint32_t bx = __float_as_uint(p.x) + (__float_as_uint(j.x) << 23);
  const uint32_t by = __float_as_uint(p.y) + (__float_as_uint(j.y) << 23);
  return make_float2(__uint_as_float(bx), __uint_as_float(by));
}

}  // namespace tc

// After a wait gave up: waits (with a limit of its own) for the `issued` tile loads of a ring that
// are still on their way, so that none lands in shared memory the CTA has left. Where all
// loads were consumed this returns at once.
__device__ __forceinline__ void drain_ring(uint64_t* full, int stages, int issued) {
  constexpr int64_t kLimit = int64_t(1) << 22;
  for (int i = issued > stages ? issued - stages : 0; i < issued; ++i)
    tc::mbar_wait(&full[i % stages], (uint32_t)(i / stages) & 1u, kLimit);
}

// The keys [b0, e0) that token q of sequence b sees; e0 <= b0 for a row without keys and
// for rows past the sequence.
struct SpanArgs {
  const int32_t* key_begin;
  const int32_t* key_end;
  int T, causal;
};
__device__ __forceinline__ void span_of(const SpanArgs& P, int b, int q, int& b0, int& e0) {
  b0 = 0;
  e0 = 0;
  if (q >= P.T) return;
  const int64_t i = (int64_t)b * P.T + q;
  if (P.key_begin) b0 = max(0, P.key_begin[i]);
  e0 = P.causal ? q + 1 : P.T;
  if (P.key_end) e0 = min(e0, P.key_end[i]);
}

// Sets every infinity and NaN of a tile of bf16 values in shared memory to zero; true if there
// was one. Warp-collective. A masked weight is zero, and zero times a NaN would reach the row
// through the tensor cores, so tiles that some row sees only in part are cleaned first.
// The first pass multiplies every value by zero and adds it up (a NaN says that one was not
// finite); only then the second looks for them.
__device__ __forceinline__ bool clean_tile(uint8_t* tile, int bytes) {
  const int lane = threadIdx.x & 31;
  const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
  __nv_bfloat162 acc[4] = {zero, zero, zero, zero};
#pragma unroll 4
  for (int i = lane * 16; i < bytes; i += 512) {
    const uint4 v = *reinterpret_cast<const uint4*>(tile + i);
    acc[0] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.x), zero, acc[0]);
    acc[1] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.y), zero, acc[1]);
    acc[2] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.z), zero, acc[2]);
    acc[3] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.w), zero, acc[3]);
  }
  const __nv_bfloat162 all = __hadd2(__hadd2(acc[0], acc[1]), __hadd2(acc[2], acc[3]));
  if (!__any_sync(0xffffffffu, (*reinterpret_cast<const uint32_t*>(&all) & 0x7fff7fffu) != 0u))
    return false;
#pragma unroll 1
  for (int i = lane * 16; i < bytes; i += 512) {
    uint32_t* w = reinterpret_cast<uint32_t*>(tile + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t x = w[e];
      if ((x & 0x00007f80u) == 0x00007f80u) x &= 0xffff0000u;
      if ((x & 0x7f800000u) == 0x7f800000u) x &= 0x0000ffffu;
      w[e] = x;
    }
  }
  return true;
}

}  // namespace gqe
