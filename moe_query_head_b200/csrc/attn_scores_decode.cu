// Attention of one new token per sequence over its KV cache, with capped and biased scores
// and a first visible key per sequence (the mathematics is in attn_scores.cuh).
//
// The work is bound by the cache's bytes (every visible K and V row is read once, for all the
// query streams of its head), with the instruction issue close behind: a score and its part of
// P V are few operations on few bytes, so it runs on CUDA cores and counts instructions. CTA
// (chunk, KV head, sequence): the sequence's own visible keys are cut into equal chunks, so
// ragged lengths and windows leave no CTA with more than its share. A chunk streams in tiles
// of 64 rows through a three-stage cp.async ring in shared memory (a tile is one contiguous run
// of memory: thread addresses are constants away from a moving pointer); each of the four
// warps takes 16 keys of every tile for all the head's queries:
//   scores  a (key, half of the head dims) pair per lane, packed products in 32 bits;
//   softmax one warp-wide maximum (redux); the sums stay in the lanes and O is rescaled only
//           when the maximum grows by more than 2^8;
//   P V     eight dims per lane, so a key's row takes d_h / 8 lanes and the warp works on
//           several keys at once; those partial sums are added after the last tile.
// The warps' states are merged in shared memory. The chunks' are merged by a second kernel,
// or, where few (sequence, KV head) pairs leave SMs free, by up to eight CTAs of a cluster in
// the first one's shared memory in the same launch. All merges run in a fixed order. Rows outside the visible keys are not read: they enter the ring as zeros,
// so a cache may hold anything there.
#include <string.h>

#include "attn_scores.cuh"
#include "attn_scores_decode.cuh"

namespace gqe {
namespace {

using namespace tc;

constexpr int THREADS = 128;
constexpr int WARPS = THREADS / 32;
constexpr int TKD = 64;  // keys per tile
constexpr int STAGES = 3;
constexpr int MAXQ = kMaxTopK + 1;
constexpr int KPW = TKD / WARPS;
constexpr int kMaxCluster = 8;  // chunks merged in shared memory

template <int DH>
struct Cfg {
  // Dense rows where two lanes per key read them without bank conflicts (d_h an odd multiple
  // of 16), else rows padded by 16 bytes with a lane per key and half.
  static constexpr bool DENSE = DH % 32 == 16;
  static constexpr int ROWB = DENSE ? DH * 2 : DH * 2 + 16;
  static constexpr int TILE = TKD * ROWB;
  static constexpr int CHUNKS = DH / 8;                       // 16-byte pieces per row
  static constexpr int PIECES = TKD * CHUNKS / THREADS;       // of a tile, per thread
  static constexpr int LK = DH / 8;                           // lanes of a key in P V
  static constexpr int NG = DH == 16 ? 16 : DH == 32 ? 8 : DH <= 64 ? 4 : 2;  // keys at once
  static constexpr int SMEM = STAGES * 2 * TILE + MAXQ * DH * 4;
  static_assert(STAGES * 2 * TILE >= (WARPS + kMaxCluster) * MAXQ * (DH + 2) * 4,
                "the ring holds the warps' and the chunks' states for the merges");
  static_assert(NG * LK <= 32 && KPW % NG == 0, "lanes of P V");
};

__device__ __forceinline__ float warp_max(float v) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}
__device__ __forceinline__ float2 bf2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ int stream_of(const DecodeArgs& P, int g, int i) {
  return i < P.k ? g * P.k + i : P.G * P.k;
}
__device__ __forceinline__ __nv_bfloat16* out_row(const DecodeArgs& P, int s, int b) {
  const int64_t head = s == P.S - 1 && P.last_off >= 0 ? P.last_off : (int64_t)s * P.out.head_stride;
  return static_cast<__nv_bfloat16*>(P.out.data) + head + (int64_t)b * P.out.token_stride;
}
// The factor of a row with the sum l: 0 without keys (`any`). With keys whose scores are all
// -infinity l and O are 0, which gives NaN.
__device__ __forceinline__ float out_scale(const DecodeArgs& P, int s, int b, float l, bool any) {
  float sc = any ? 1.f / l : 0.f;
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

// (m, l, O[d]) of query i over the keys of one cluster: the output, or the cluster's state.
__device__ __forceinline__ void finish_row(const DecodeArgs& P, int g, int i, int b, int part, int d,
                                           float mx, float lt, float ot, bool any) {
  const int s = stream_of(P, g, i);
  if (P.np == 1) {
    out_row(P, s, b)[d] = __float2bfloat16_rn(ot * out_scale(P, s, b, lt, any));
    return;
  }
  float* slot = P.part + (((int64_t)s * P.B + b) * P.np + part) * (P.d_h + 2);
  if (d == 0) {
    slot[0] = mx;
    slot[1] = lt;
  }
  slot[2 + d] = ot;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The address of a shared-memory location of this CTA in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_shared(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// QMAX: the most queries of a KV head in this launch (2, 4 or 9), a compile-time count so
// that the per-query state stays in registers. Four CTAs an SM at two queries and d_h <= 48
// leave it 128 (64 sequences of 8192 cached tokens, 805 MB: 128 us; six CTAs of 85 registers
// 167 us, eight of 64 218 us, both spilling; two ring stages instead of three 134 us).
template <int DH, int QMAX>
__global__ void __launch_bounds__(THREADS, (DH <= 48 && QMAX <= 2) ? 4 : 1)
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
    if (tid == 0 && c == 0 && g == 0) atomicCAS(P.status, kStatusOk, kStatusBadInput);
    return;
  }
  const int nq = P.k + (g == 0 && P.S > P.G * P.k ? 1 : 0);
  // this chunk's keys: the visible ones in equal parts, rounded up to whole tiles
  const int n = max(0, end - first), parts = P.nc * P.np;
  const int per = (int)(((int64_t)n + parts * TKD - 1) / (parts * TKD)) * TKD;
  const int k0 = first + (int)min((int64_t)n, (int64_t)c * per);
  const int k1 = first + (int)min((int64_t)n, (int64_t)c * per + per);
  const __nv_bfloat16* kc = static_cast<const __nv_bfloat16*>(P.kc.data) +
                            g * P.kc.head_stride + (int64_t)b * P.kc.token_stride;
  const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(P.vc.data) +
                            g * P.vc.head_stride + (int64_t)b * P.vc.token_stride;
  const int ntiles = (k1 - k0 + TKD - 1) / TKD;
  // piece i of a tile: 16 bytes at element 8 (tid + 128 i) of the tile's rows
  kc += (int64_t)k0 * DH + tid * 8;
  vc += (int64_t)k0 * DH + tid * 8;
  uint32_t dst[C::PIECES];
#pragma unroll
  for (int i = 0; i < C::PIECES; ++i) {
    const int e = tid + i * THREADS;
    dst[i] = smem_u32(sK) + (C::DENSE ? e * 16 : e / C::CHUNKS * C::ROWB + e % C::CHUNKS * 16);
  }
  auto load_tile = [&](int t, int st) {
    const __nv_bfloat16* ks = kc + (int64_t)t * TKD * DH;
    const __nv_bfloat16* vs = vc + (int64_t)t * TKD * DH;
    const uint32_t ring = st * C::TILE;
    if ((t + 1) * TKD <= k1 - k0) {
#pragma unroll
      for (int i = 0; i < C::PIECES; ++i) {
        cp_async_16(dst[i] + ring, ks + i * THREADS * 8, 16);
        cp_async_16(dst[i] + ring + STAGES * C::TILE, vs + i * THREADS * 8, 16);
      }
    } else {
      // the last tile: rows past the chunk become zeros (their addresses stay inside)
      const int rows = k1 - k0 - t * TKD;
#pragma unroll
      for (int i = 0; i < C::PIECES; ++i) {
        const bool in = tid + i * THREADS < rows * C::CHUNKS;
        const int off = in ? i * THREADS * 8 : -tid * 8;
        cp_async_16(dst[i] + ring, ks + off, in ? 16 : 0);
        cp_async_16(dst[i] + ring + STAGES * C::TILE, vs + off, in ? 16 : 0);
      }
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
  // P V: this lane's key of every NG and its eight dims (lanes without a key repeat key 0's)
  const int pg = lane / C::LK < C::NG ? lane / C::LK : 0;
  const uint32_t v_off = (warp * KPW + pg) * C::ROWB + lane % C::LK * 16;
  float m[QMAX], l[QMAX], slope2[QMAX];
  float2 o[QMAX][4];
#pragma unroll
  for (int a = 0; a < QMAX; ++a) {
    m[a] = -INFINITY;
    l[a] = 0.f;
    slope2[a] = P.slopes && a < nq ? P.slopes[stream_of(P, g, a)] * kLog2e : 0.f;
#pragma unroll
    for (int p = 0; p < 4; ++p) o[a][p] = make_float2(0.f, 0.f);
  }
  __syncthreads();  // sQ written
  for (int t = 0; t < ntiles; ++t) {
    if (t + STAGES - 1 < ntiles) load_tile(t + STAGES - 1, (t + STAGES - 1) % STAGES);
    cp_async_commit();
    cp_async_wait<STAGES - 1>();
    __syncthreads();  // tile t is in shared memory for every thread
    const uint8_t* kt = sK + t % STAGES * C::TILE + krow * C::ROWB + half * DH;
    const uint8_t* vt = sV + t % STAGES * C::TILE + v_off;
    const int u = k0 + t * TKD + krow;
    const bool key_ok = u < k1;
    const float dist = (float)(end - 1 - u);  // the new token's position minus the key's
    float2 kf[DH / 4];
#pragma unroll
    for (int ch = 0; ch < DH / 16; ++ch) {
      const uint4 v = *reinterpret_cast<const uint4*>(kt + ch * 16);
      kf[4 * ch] = bf2(v.x);
      kf[4 * ch + 1] = bf2(v.y);
      kf[4 * ch + 2] = bf2(v.z);
      kf[4 * ch + 3] = bf2(v.w);
    }
#pragma unroll
    for (int a = 0; a < QMAX; ++a) {
      if (a >= nq) break;  // uniform over the CTA
      const float4* q = reinterpret_cast<const float4*>(sQ + a * DH + half * (DH / 2));
      float2 acc2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int d = 0; d < DH / 8; ++d) {
        const float4 qv = q[d];
        acc2[0] = fma2(make_float2(qv.x, qv.y), kf[2 * d], acc2[0]);
        acc2[1] = fma2(make_float2(qv.z, qv.w), kf[2 * d + 1], acc2[1]);
      }
      acc2[0] = add2(acc2[0], acc2[1]);
      float acc = acc2[0].x + acc2[0].y;
      acc += __shfl_xor_sync(0xffffffffu, acc, kHalfXor);
      if (P.cap_log2 != 0.f) acc = tanh_from_2log2(acc * P.cap_in) * P.cap_log2;
      acc = fmaf(-slope2[a], dist, acc);
      const float sc = key_ok ? acc : -INFINITY;
      const float mt = warp_max(sc);
      if (mt > m[a] + 8.f) {
        const float alpha = ex2(m[a] - mt);  // 0 from a reference of -inf
        l[a] *= alpha;
#pragma unroll
        for (int p = 0; p < 4; ++p) o[a][p] = mul2(o[a][p], make_float2(alpha, alpha));
        m[a] = mt;
      }
      // a warp whose keys are all masked so far keeps m = -inf, l = 0, O = 0
      const float pk = ex2(sc - (m[a] == -INFINITY ? 0.f : m[a]));  // 0 for a masked key
      l[a] += pk;
#pragma unroll
      for (int j = 0; j < KPW / C::NG; ++j) {
        const float pj = __shfl_sync(0xffffffffu, pk, (j * C::NG + pg) * kKeyLane);
        const uint4 v = *reinterpret_cast<const uint4*>(vt + j * C::NG * C::ROWB);
        const float2 p2 = make_float2(pj, pj);
        o[a][0] = fma2(p2, bf2(v.x), o[a][0]);
        o[a][1] = fma2(p2, bf2(v.y), o[a][1]);
        o[a][2] = fma2(p2, bf2(v.z), o[a][2]);
        o[a][3] = fma2(p2, bf2(v.w), o[a][3]);
      }
    }
    __syncthreads();  // every warp is done with the stage before it is refilled
  }
  cp_async_wait<0>();
  __syncthreads();  // the ring is free: it holds the warps' states for the merge
  float* sM = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int a = 0; a < QMAX; ++a) {
    if (a >= nq) break;
    float* st = sM + (warp * MAXQ + a) * (DH + 2);
    // a key's two lanes hold the same weight: half the sum over the lanes
    float lw = l[a];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, off);
    if (lane == 0) {
      st[0] = m[a];
      st[1] = 0.5f * lw;
    }
    // P V of the NG keys at a time, in their order
    float v[8];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      v[2 * p] = o[a][p].x;
      v[2 * p + 1] = o[a][p].y;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float sum = v[i];
#pragma unroll
      for (int gi = 1; gi < C::NG; ++gi) sum += __shfl_sync(0xffffffffu, v[i], lane + gi * C::LK);
      if (lane < C::LK) st[2 + lane * 8 + i] = sum;
    }
  }
  // the states of n_states states at `from` (`stride` floats apart) of query i, dim d, merged
  auto merge = [&](const float* from, int stride, int n_states, int d, float& mx, float& lt,
                   float& ot) {
    mx = -INFINITY;
    for (int w = 0; w < n_states; ++w) mx = fmaxf(mx, from[w * stride]);
    const float mref = mx == -INFINITY ? 0.f : mx;
    lt = ot = 0.f;
    for (int w = 0; w < n_states; ++w) {
      const float f = ex2(from[w * stride] - mref);  // 0 for one that saw no key
      lt += f * from[w * stride + 1];
      ot += f * from[w * stride + 2 + d];
    }
  };
  const int rank = c % P.nc, part = c / P.nc;
  float* sC = sM + WARPS * MAXQ * (DH + 2);  // in the first CTA: [nc][MAXQ][DH + 2]
  if (P.nc > 1) cluster_sync();  // the first CTA is done with its ring
  else __syncthreads();
  for (int e = tid; e < nq * DH; e += THREADS) {
    const int i = e / DH, d = e % DH;
    float mx, lt, ot;
    merge(sM + i * (DH + 2), MAXQ * (DH + 2), WARPS, d, mx, lt, ot);
    if (P.nc > 1) {
      const uint32_t to = map_shared(smem_u32(sC + (rank * MAXQ + i) * (DH + 2)), 0);
      if (d == 0) {
        st_cluster(to, mx);
        st_cluster(to + 4, lt);
      }
      st_cluster(to + 8 + d * 4, ot);
    } else {
      finish_row(P, g, i, b, part, d, mx, lt, ot, n > 0);
    }
  }
  if (P.nc > 1) {
    cluster_sync();  // every chunk's states have arrived
    if (rank == 0) {
      for (int e = tid; e < nq * DH; e += THREADS) {
        const int i = e / DH, d = e % DH;
        float mx, lt, ot;
        merge(sC + i * (DH + 2), MAXQ * (DH + 2), P.nc, d, mx, lt, ot);
        finish_row(P, g, i, b, part, d, mx, lt, ot, n > 0);
      }
    }
  }
}

// Merges the clusters' states of (stream, sequence) in order.
__global__ void __launch_bounds__(128) attn_decode_merge_kernel(const __grid_constant__ DecodeArgs P) {
  const int s = blockIdx.x, b = blockIdx.y, d = threadIdx.x;
  pdl_wait();
  pdl_allow_next();
  int first, end;
  if (!visible(P, b, first, end)) return;
  const int row = P.d_h + 2;
  const float* base = P.part + ((int64_t)s * P.B + b) * P.np * row;
  float mx = -INFINITY;
  for (int c = 0; c < P.np; ++c) mx = fmaxf(mx, base[c * row]);
  const float mref = mx == -INFINITY ? 0.f : mx;
  float l = 0.f, o = 0.f;
  for (int c = 0; c < P.np; ++c) {
    const float w = ex2(base[c * row] - mref);  // 0 for a cluster without keys
    l += w * base[c * row + 1];
    o += w * base[c * row + 2 + d];
  }
  out_row(P, s, b)[d] = __float2bfloat16_rn(o * out_scale(P, s, b, l, first < end));
}

template <int DH, int QMAX>
int launch_attn(const DecodeArgs& P, cudaStream_t st) {
  using C = Cfg<DH>;
  if (!set_smem_limit_once<attn_decode_kernel<DH, QMAX>>(C::SMEM)) return -1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(P.nc * P.np, P.G, P.B);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)P.nc;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = P.nc > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, attn_decode_kernel<DH, QMAX>, P) != cudaSuccess) return -1;
  if (P.np == 1) return 1;
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

// Chunks of a (sequence, KV head): enough CTAs for sixteen per SM, at least a tile each. With
// fewer pairs than SMs the latency counts: clusters of up to eight chunks, and several of them
// only where each chunk would have more than eight tiles (one sequence of 8192 tokens: 15 us
// against 22 with single CTAs and the second kernel). With more pairs the clusters' common
// start costs more than the second kernel (32 sequences of 8192 tokens at d_h 128: 212 us
// against 172).
void attn_decode_plan(int B, int G, int L_max, int num_sms, int& nc, int& np) {
  const int64_t bg = (int64_t)B * G;
  const int64_t tiles = ((int64_t)L_max + TKD - 1) / TKD;
  int64_t want = (16 * (int64_t)num_sms + bg - 1) / bg;
  if (want > tiles) want = tiles;
  if (bg >= num_sms) {
    nc = 1;
    np = (int)want;
    return;
  }
  nc = (int)(want < kMaxCluster ? want : kMaxCluster);
  int64_t more = (tiles + 8 * kMaxCluster - 1) / (8 * kMaxCluster);
  const int64_t most = (want + kMaxCluster - 1) / kMaxCluster;
  if (more > most) more = most;
  np = (int)(more < 1 ? 1 : more);
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
