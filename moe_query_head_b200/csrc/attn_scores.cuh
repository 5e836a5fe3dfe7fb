// Arguments and device helpers shared by the kernels of the attention with capped, biased and
// masked scores (attn_scores.cu, attn_scores_bwd.cu, attn_scores_decode.cu).
//
// Query stream s of token t (position t of its sequence) sees the keys u of its KV head with
// begin_t <= u < end_t. Its scores are
//   z = scale <q, k_u>;  z = softcap tanh(z / softcap) if softcap > 0;  z -= slope_s |t - u|,
// its weights the softmax of z over those keys; a row without keys gives zeros.
#pragma once

#include <cuda.h>

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

// 2^x of a pair on the FMA pipe, as exp2_fma.cuh's exp2_fma2 (nearest integer n of x by adding
// and subtracting 1.5 * 2^23, then the degree-2 polynomial of 2^(x - n) fitted there, 1.9e-3,
// the size of the bf16 rounding that follows), with NaN kept: the clamp passes a NaN on and
// the exponent addition turns it into a value of the largest magnitudes, so that a row that
// sees a NaN score ends as NaN instead of losing that key.
__device__ __forceinline__ float2 exp2_fma2_nan(float2 x) {
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
  asm("max.NaN.f32 %0, %0, 0fC2FA0000;" : "+f"(x.x));  // -125
  asm("max.NaN.f32 %0, %0, 0fC2FA0000;" : "+f"(x.y));
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
__device__ __forceinline__ bool clean_tile(uint8_t* tile, int bytes) {
  bool bad = false;
  const int lane = threadIdx.x & 31;
#pragma unroll 4
  for (int i = lane * 16; i < bytes; i += 512) {
    uint4 v = *reinterpret_cast<const uint4*>(tile + i);
    // exponent field all ones: adding one unit of it carries into (or past) the sign bit
    const uint32_t c = ((v.x & 0x7f807f80u) + 0x00800080u) | ((v.y & 0x7f807f80u) + 0x00800080u) |
                       ((v.z & 0x7f807f80u) + 0x00800080u) | ((v.w & 0x7f807f80u) + 0x00800080u);
    if (c & 0x80008000u) {
      bad = true;
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if ((w[e] & 0x00007f80u) == 0x00007f80u) w[e] &= 0xffff0000u;
        if ((w[e] & 0x7f800000u) == 0x7f800000u) w[e] &= 0x0000ffffu;
      }
      *reinterpret_cast<uint4*>(tile + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  return __any_sync(0xffffffffu, bad);
}

}  // namespace gqe
