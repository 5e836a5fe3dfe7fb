// Attention of one new token per sequence over its KV cache, with capped and biased scores
// and a first visible key per sequence (the mathematics is in attn_scores.cuh).
//
// The work is bound by the cache's bytes (every visible K and V row is read once, for all the
// query streams of its head), so it runs on CUDA cores. CTA (chunk, KV head, sequence): the
// sequence's own visible keys are cut into equal chunks, so ragged lengths and windows leave
// no CTA with more than its share. A chunk streams in tiles of 64 rows through a two-stage
// cp.async ring in shared memory; each of the four warps takes 16 keys of every tile for all
// the head's queries: a score per (key, half of the head dims) lane pair, an online softmax
// over the warp's keys with shuffles, P V with each lane owning pairs of head dimensions. The
// warps' states are merged in shared memory; with more than one chunk a second kernel, one
// CTA per (stream, sequence), merges the chunks' states in a fixed order. Rows outside the
// visible keys are not read: they enter the ring as zeros, so a cache may hold anything there.
#include <string.h>

#include "attn_scores.cuh"
#include "attn_scores_decode.cuh"

namespace gqe {
namespace {

using namespace tc;

constexpr int THREADS = 128;
constexpr int WARPS = THREADS / 32;
constexpr int TKD = 64;  // keys per tile
constexpr int STAGES = 2;
constexpr int MAXQ = kMaxTopK + 1;
constexpr int KPW = TKD / WARPS;

template <int DH>
struct Cfg {
  // Dense rows where two lanes per key read them without bank conflicts (d_h an odd multiple
  // of 16), else rows padded by 16 bytes with a lane per key and half.
  static constexpr bool DENSE = DH % 32 == 16;
  static constexpr int ROWB = DENSE ? DH * 2 : DH * 2 + 16;
  static constexpr int TILE = TKD * ROWB;
  static constexpr int CHUNKS = DH / 8;
  static constexpr int NP = (DH / 2 + 31) / 32;  // dim pairs per lane
  static constexpr int SMEM = STAGES * 2 * TILE + MAXQ * DH * 4;
  static_assert(STAGES * 2 * TILE >= WARPS * MAXQ * (DH + 2) * 4,
                "the ring holds the warps' states for the merge");
};

__device__ __forceinline__ int stream_of(const DecodeArgs& P, int g, int i) {
  return i < P.k ? g * P.k + i : P.G * P.k;
}
__device__ __forceinline__ __nv_bfloat16* out_row(const DecodeArgs& P, int s, int b) {
  const int64_t head = s == P.S - 1 && P.last_off >= 0 ? P.last_off : (int64_t)s * P.out.head_stride;
  return static_cast<__nv_bfloat16*>(P.out.data) + head + (int64_t)b * P.out.token_stride;
}
__device__ __forceinline__ float out_scale(const DecodeArgs& P, int s, int b, float l) {
  float sc = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // no key: zeros; NaN stays
  if (P.psel && s < P.G * P.k) sc *= P.psel[(int64_t)b * P.psel_stride + P.psel_off + s];
  return sc;
}
// Sequence b's visible keys [first, end); false for a position outside the cache (reported).
__device__ __forceinline__ bool visible(const DecodeArgs& P, int b, int& first, int& end) {
  const int L = P.lengths[b];
  first = P.key_begin ? max(0, P.key_begin[b]) : 0;
  end = L + 1;
  return L >= -1 && L < P.L_max;
}

// QMAX: the most queries of a KV head in this launch (2, 4 or 9), a compile-time count so
// that the per-query state stays in registers; at two queries and d_h <= 48 it fits 64
// registers and eight CTAs share an SM (more CTAs, more bytes in flight).
template <int DH, int QMAX>
__global__ void __launch_bounds__(THREADS, (DH <= 48 && QMAX <= 2) ? 8 : 1)
attn_decode_kernel(const __grid_constant__ DecodeArgs P) {
  using C = Cfg<DH>;
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* sK = smem;
  uint8_t* sV = smem + STAGES * C::TILE;
  float* sQ = reinterpret_cast<float*>(smem + 2 * STAGES * C::TILE);  // [MAXQ][DH]
  const int c = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  pdl_wait();
  pdl_allow_next();
  int first, end;
  if (!visible(P, b, first, end)) {
    if (tid == 0 && c == 0 && g == 0) atomicExch(P.status, kStatusBadInput);
    return;
  }
  const int nq = P.k + (g == 0 && P.S > P.G * P.k ? 1 : 0);
  // this chunk's keys: the visible ones in nc equal parts, rounded up to whole tiles
  const int n = max(0, end - first);
  const int per = (n + P.nc * TKD - 1) / (P.nc * TKD) * TKD;
  const int k0 = first + min(n, c * per);
  const int k1 = first + min(n, c * per + per);
  const __nv_bfloat16* kc = static_cast<const __nv_bfloat16*>(P.kc.data) +
                            g * P.kc.head_stride + (int64_t)b * P.kc.token_stride;
  const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(P.vc.data) +
                            g * P.vc.head_stride + (int64_t)b * P.vc.token_stride;
  const int ntiles = (k1 - k0 + TKD - 1) / TKD;
  auto load_tile = [&](int t, int st) {
    const int base = k0 + t * TKD;
    for (int e = tid; e < TKD * C::CHUNKS; e += THREADS) {
      const int r = e / C::CHUNKS, ch = e % C::CHUNKS;
      const int u = base + r;
      const int64_t off = (int64_t)min(u, k1 - 1) * DH + ch * 8;
      const uint32_t bytes = u < k1 ? 16 : 0;
      cp_async_16(smem_u32(sK + st * C::TILE + r * C::ROWB + ch * 16), kc + off, bytes);
      cp_async_16(smem_u32(sV + st * C::TILE + r * C::ROWB + ch * 16), vc + off, bytes);
    }
  };
  for (int t = 0; t < STAGES - 1; ++t) {
    if (t < ntiles) load_tile(t, t);
    cp_async_commit();
  }
  // queries of this head, prescaled to log2 units
  for (int e = tid; e < nq * DH; e += THREADS) {
    const int i = e / DH, d = e % DH;
    sQ[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(
                P.q.data)[stream_of(P, g, i) * P.q.head_stride + (int64_t)b * P.q.token_stride + d]) *
            P.scale_log2;
  }
  const int kq = C::DENSE ? lane >> 1 : lane & 15, half = C::DENSE ? lane & 1 : lane >> 4;
  constexpr int kHalfXor = C::DENSE ? 1 : 16;  // the lane holding the key's other half
  constexpr int kKeyLane = C::DENSE ? 2 : 1;   // lane stride between keys
  const int krow = warp * KPW + kq;
  float m[QMAX], l[QMAX], slope2[QMAX];
  float2 o[QMAX][C::NP];
#pragma unroll
  for (int a = 0; a < QMAX; ++a) {
    m[a] = -INFINITY;
    l[a] = 0.f;
    slope2[a] = P.slopes && a < nq ? P.slopes[stream_of(P, g, a)] * kLog2e : 0.f;
#pragma unroll
    for (int p = 0; p < C::NP; ++p) o[a][p] = make_float2(0.f, 0.f);
  }
  __syncthreads();  // sQ written
  for (int t = 0; t < ntiles; ++t) {
    if (t + STAGES - 1 < ntiles) load_tile(t + STAGES - 1, (t + STAGES - 1) % STAGES);
    cp_async_commit();
    cp_async_wait<STAGES - 1>();
    __syncthreads();  // tile t is in shared memory for every thread
    const int st = t % STAGES;
    const uint8_t* kt = sK + st * C::TILE;
    const uint8_t* vt = sV + st * C::TILE;
    const int u = k0 + t * TKD + krow;
    const bool key_ok = u < k1;
    const float dist = (float)(end - 1 - u);  // the new token's position minus the key's
    float kf[DH / 2];
    {
      const uint8_t* row = kt + krow * C::ROWB + half * DH;
#pragma unroll
      for (int ch = 0; ch < DH / 16; ++ch) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + ch * 16);
        const __nv_bfloat162* p2 = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = __bfloat1622float2(p2[e]);
          kf[ch * 8 + 2 * e] = f.x;
          kf[ch * 8 + 2 * e + 1] = f.y;
        }
      }
    }
#pragma unroll
    for (int a = 0; a < QMAX; ++a) {
      if (a >= nq) break;  // uniform over the CTA
      const float* q = sQ + a * DH + half * (DH / 2);
      float acc = 0.f;
#pragma unroll
      for (int d = 0; d < DH / 2; ++d) acc = fmaf(q[d], kf[d], acc);
      acc += __shfl_xor_sync(0xffffffffu, acc, kHalfXor);
      if (P.cap_log2 != 0.f) acc = tanh_from_2log2(acc * P.cap_in) * P.cap_log2;
      acc = fmaf(-slope2[a], dist, acc);
      const float sc = key_ok ? acc : -INFINITY;
      float mt = sc;
#pragma unroll
      for (int off = 8 * kKeyLane; off >= kKeyLane; off >>= 1)
        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, off));
      const float m_new = fmaxf(m[a], mt);
      // a warp whose keys are all masked so far keeps m = -inf, l = 0, O = 0
      const float m_ref = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = ex2(m[a] - m_ref);  // 0 while m is -inf
      const float pk = ex2(sc - m_ref);       // 0 for a masked key
      float ps = pk;
#pragma unroll
      for (int off = 8 * kKeyLane; off >= kKeyLane; off >>= 1)
        ps += __shfl_xor_sync(0xffffffffu, ps, off);
      l[a] = l[a] * alpha + ps;
      m[a] = m_new;
#pragma unroll
      for (int p = 0; p < C::NP; ++p) {
        o[a][p].x *= alpha;
        o[a][p].y *= alpha;
      }
#pragma unroll
      for (int j = 0; j < KPW; ++j) {
        const float pj = __shfl_sync(0xffffffffu, pk, j * kKeyLane);
        const uint8_t* row = vt + (warp * KPW + j) * C::ROWB;
#pragma unroll
        for (int p = 0; p < C::NP; ++p) {
          const int d2 = lane + 32 * p;
          if (2 * d2 < DH) {
            const float2 f =
                __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(row + 4 * d2));
            o[a][p].x = fmaf(pj, f.x, o[a][p].x);
            o[a][p].y = fmaf(pj, f.y, o[a][p].y);
          }
        }
      }
    }
    __syncthreads();  // every warp is done with stage st before it is refilled
  }
  cp_async_wait<0>();
  __syncthreads();  // the ring is free: it holds the warps' states for the merge
  float* sM = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int a = 0; a < QMAX; ++a) {
    if (a >= nq) break;
    float* st = sM + (warp * MAXQ + a) * (DH + 2);
    if (lane == 0) {
      st[0] = m[a];
      st[1] = l[a];
    }
#pragma unroll
    for (int p = 0; p < C::NP; ++p) {
      const int d2 = lane + 32 * p;
      if (2 * d2 < DH) {
        st[2 + 2 * d2] = o[a][p].x;
        st[2 + 2 * d2 + 1] = o[a][p].y;
      }
    }
  }
  __syncthreads();
  for (int e = tid; e < nq * DH; e += THREADS) {
    const int i = e / DH, d = e % DH;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) mx = fmaxf(mx, sM[(w * MAXQ + i) * (DH + 2)]);
    const float mref = mx == -INFINITY ? 0.f : mx;
    float lt = 0.f, ot = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float* st = sM + (w * MAXQ + i) * (DH + 2);
      const float f = ex2(st[0] - mref);  // 0 for a warp that saw no key
      lt += f * st[1];
      ot += f * st[2 + d];
    }
    const int s = stream_of(P, g, i);
    if (P.nc == 1) {
      out_row(P, s, b)[d] = __float2bfloat16_rn(ot * out_scale(P, s, b, lt));
    } else {
      float* slot = P.part + (((int64_t)s * P.B + b) * P.nc + c) * (DH + 2);
      if (d == 0) {
        slot[0] = mx;
        slot[1] = lt;
      }
      slot[2 + d] = ot;
    }
  }
}

// Merges the chunks' states of (stream, sequence) in chunk order.
__global__ void __launch_bounds__(128) attn_decode_merge_kernel(const __grid_constant__ DecodeArgs P) {
  const int s = blockIdx.x, b = blockIdx.y, d = threadIdx.x;
  pdl_wait();
  pdl_allow_next();
  int first, end;
  if (!visible(P, b, first, end)) return;
  const int row = P.d_h + 2;
  const float* base = P.part + ((int64_t)s * P.B + b) * P.nc * row;
  float mx = -INFINITY;
  for (int c = 0; c < P.nc; ++c) mx = fmaxf(mx, base[c * row]);
  const float mref = mx == -INFINITY ? 0.f : mx;
  float l = 0.f, o = 0.f;
  for (int c = 0; c < P.nc; ++c) {
    const float w = ex2(base[c * row] - mref);  // 0 for a chunk without keys
    l += w * base[c * row + 1];
    o += w * base[c * row + 2 + d];
  }
  out_row(P, s, b)[d] = __float2bfloat16_rn(o * out_scale(P, s, b, l));
}

template <int DH, int QMAX>
int launch_attn(const DecodeArgs& P, cudaStream_t st) {
  using C = Cfg<DH>;
  if (!set_smem_limit_once<attn_decode_kernel<DH, QMAX>>(C::SMEM)) return -1;
  if (launch_pdl(attn_decode_kernel<DH, QMAX>, dim3(P.nc, P.G, P.B), dim3(THREADS), C::SMEM, st,
                 P) != cudaSuccess)
    return -1;
  if (P.nc == 1) return 1;
  return launch_pdl(attn_decode_merge_kernel, dim3(P.S, P.B), dim3(DH), 0, st, P) == cudaSuccess
             ? 2
             : -1;
}

template <int DH>
int launch_dh(const DecodeArgs& P, cudaStream_t st) {
  const int nq_max = P.k + (P.S > P.G * P.k ? 1 : 0);
  return nq_max <= 2   ? launch_attn<DH, 2>(P, st)
         : nq_max <= 4 ? launch_attn<DH, 4>(P, st)
                       : launch_attn<DH, MAXQ>(P, st);
}

}  // namespace

// Chunks per (sequence, KV head): enough CTAs for sixteen per SM, at least one tile each.
int attn_decode_chunks(int B, int G, int L_max, int num_sms) {
  const int64_t bg = (int64_t)B * G;
  int64_t nc = (16 * (int64_t)num_sms + bg - 1) / bg;
  const int64_t tiles = ((int64_t)L_max + TKD - 1) / TKD;
  if (nc > tiles) nc = tiles;
  return nc < 1 ? 1 : (int)nc;
}

int launch_attn_decode(const DecodeArgs& P, cudaStream_t st) {
  switch (P.d_h) {
    case 16: return launch_dh<16>(P, st);
    case 32: return launch_dh<32>(P, st);
    case 48: return launch_dh<48>(P, st);
    case 64: return launch_dh<64>(P, st);
    case 80: return launch_dh<80>(P, st);
    case 96: return launch_dh<96>(P, st);
    case 112: return launch_dh<112>(P, st);
    case 128: return launch_dh<128>(P, st);
    default: return -1;
  }
}

}  // namespace gqe
