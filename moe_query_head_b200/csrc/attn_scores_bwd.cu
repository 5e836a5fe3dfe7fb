// Tensor-core (tcgen05) backward pass of the attention with capped, biased and masked scores
// (the forward's mathematics is in attn_scores.cuh). With p = softmax(z) over a row's keys,
// D = <dout, out>, dP = dout v^T:
//   dz = p (dP - D),  times 1 - tanh^2 where the scores are capped,
//   dq = scale dz k,  dk = scale sum over the head's streams of dz^T q,
//   dv = sum over the head's streams of p^T dout.
//
// Two kernels, none with atomics (every output value is written by one CTA, so results are
// the same from run to run):
//   attn_scores_dq_kernel    CTA, or a cluster that shares the steps = (sequence, stream,
//                            128-query tile); D of its rows, then per 64-key step S = Q K^T and
//                            dP into TMEM, dz in bf16 back to TMEM, dQ += dz K. It leaves D and
//                            the union of its rows' intervals for the second kernel (a kernel
//                            of its own for them took 7 us).
//   attn_scores_dkdv_kernel  CTA = (sequence, KV head, 128-key tile); per job (a stream of the
//                            head, a tile of queries) S^T and dP^T, then dV += p^T dout and
//                            dK += dz^T Q, accumulated in TMEM over all the head's streams.
// Scores and weights are formed again from the saved log-sum-exp rather than read: T^2 values
// per stream would be the largest traffic by far. p and dz are rounded to bf16, the type of
// the products' operands; D, the sums and the accumulators stay in 32 bits. Steps and jobs
// outside the rows' intervals are never loaded; those that some row sees only in part are
// masked, and their key (or query and dout) tiles are cleaned of infinities and NaN, which a
// weight of zero would not keep out of a product.
#include <cudaTypedefs.h>
#include <limits.h>
#include <string.h>

#include <type_traits>

#include "attn_scores.cuh"
#include "scores_api.cuh"

namespace gqe {
namespace {

using namespace tc;

constexpr int THREADS = 256;
constexpr int TQ = 128, TK = 128;
// Registers of the two warpgroups, by setmaxnreg. 9 streams of 64, 5 documents in 8192 tokens, at
// 48 / 208: 228 us, 64 / 192: 222, 80 / 176: 213; 8192 causal of 48: 442, 433, 430 (96 / 160 gains
// on some and loses 4 % on documents of 48).
constexpr int kSmallRegs = 80, kLargeRegs = 176;
static_assert(kSmallRegs * 128 + kLargeRegs * 128 == THREADS * (65536 / (2 * THREADS)),
              "register split must equal the launch allocation");

template <int DH>
struct BCfg {
  static constexpr int CW = (DH % 64 == 0) ? 64 : 16;  // 128- or 32-byte swizzle
  static constexpr uint32_t LAYOUT = CW == 64 ? kSwizzle128B : kSwizzle32B;
  static constexpr int ROW_BYTES = CW * 2;
  static constexpr int TILE_BYTES = 128 * DH * 2;
  static constexpr int CTAS = DH <= 64 ? 2 : 1;
  static constexpr int TMEM_COLS = CTAS == 2 ? 256 : 512;
  static constexpr int STAGES = 3;
};

struct Params {
  CUtensorMap tm_q, tm_do, tm_k, tm_v;  // dQ: 128-row q, dout; 64-row k, v. dK / dV: job-row
                                        // q, dout; 128-row k, v
  SpanArgs span;
  const float* lse;
  float* dsum;
  const __nv_bfloat16* dout;  // with out: rows for D; null where dsum holds it already
  const __nv_bfloat16* out;
  int64_t dout_hs, dout_ts, out_hs, out_ts;
  const __nv_bfloat16* keys;  // for the rare rows that see an infinity or NaN
  int64_t key_hs, key_ts;
  const float* slopes;
  int2* blocks;  // [B, nq] intervals of 128 rows; null without masks
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  int64_t dq_hs, dq_ts, dk_hs, dk_ts, dv_hs, dv_ts;
  const int32_t* sel;
  __nv_bfloat16* dq_shared;
  int64_t sel_stride;
  int sel_off, experts;
  int T, B, S, Sr, k, G, nq;
  int split;  // CTAs (a cluster) that share a query tile's steps or a key tile's jobs
  float scale, scale_log2;
  CapForm cap;
  int32_t* status;
  int64_t spin;
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const Params& P) {
  const bool ok = !__any_sync(0xffffffffu, !mbar_wait(bar, parity, P.spin));
  if (!ok && (threadIdx.x & 31) == 0) atomicExch(P.status, kStatusTimeout);
  return ok;
}
__device__ __forceinline__ bool lane_wait(uint64_t* bar, uint32_t parity, const Params& P) {
  if (mbar_wait(bar, parity, P.spin)) return true;
  atomicExch(P.status, kStatusTimeout);
  return false;
}

template <int DH, int ROWS>
__device__ __forceinline__ uint32_t kmajor_off(int kk) {
  using C = BCfg<DH>;
  return (((kk * 16) / C::CW) * ROWS * C::ROW_BYTES + ((kk * 16) % C::CW) * 2) >> 4;
}

// TMEM -> registers, N consecutive 32-bit columns per lane (N = 32, 48 or 64).
template <int N>
__device__ __forceinline__ void tmem_ldN_wait(uint32_t taddr, uint32_t (&r)[N]) {
  static_assert(N == 32 || N == 48 || N == 64, "TMEM row widths of a job");
  if constexpr (N == 64) {
    tmem_ld64_wait(taddr, r);
  } else {
    uint32_t a[32];
    tmem_ld32(taddr, a);
    uint32_t b[16];
    if constexpr (N == 48) tmem_ld16(taddr + 32, b);
    // the wait names the registers it completes, so no use of them can move above it
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]),
                   "+r"(a[6]), "+r"(a[7]), "+r"(a[8]), "+r"(a[9]), "+r"(a[10]), "+r"(a[11]),
                   "+r"(a[12]), "+r"(a[13]), "+r"(a[14]), "+r"(a[15])
                 :
                 : "memory");
    asm volatile("" : "+r"(a[16]), "+r"(a[17]), "+r"(a[18]), "+r"(a[19]), "+r"(a[20]),
                      "+r"(a[21]), "+r"(a[22]), "+r"(a[23]), "+r"(a[24]), "+r"(a[25]),
                      "+r"(a[26]), "+r"(a[27]), "+r"(a[28]), "+r"(a[29]), "+r"(a[30]),
                      "+r"(a[31]));
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = a[i];
    if constexpr (N == 48) {
      asm volatile("" : "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]), "+r"(b[4]), "+r"(b[5]),
                        "+r"(b[6]), "+r"(b[7]), "+r"(b[8]), "+r"(b[9]), "+r"(b[10]),
                        "+r"(b[11]), "+r"(b[12]), "+r"(b[13]), "+r"(b[14]), "+r"(b[15]));
#pragma unroll
      for (int i = 0; i < 16; ++i) r[32 + i] = b[i];
    }
  }
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// Of every 8 pairs of scores, this many take the FMA-pipe exponential and the rest MUFU's: none
// where the cap's polynomial keeps the FMA pipe busy.
template <bool CAP, bool BIAS>
constexpr int kBwdFma = CAP ? 0 : 2;

// A product that takes denormals for zeros: what the FMA-pipe exponential leaves of a score of
// -infinity (5e-42) is then no factor of dz.
__device__ __forceinline__ float2 mul2_ftz(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.ftz.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}

// Writes a TMEM accumulator row (DH columns, scaled) as bf16.
template <int DH>
__device__ __forceinline__ void store_row(uint32_t taddr, __nv_bfloat16* dst, float sc, bool write,
                                          bool zero) {
#pragma unroll
  for (int c0 = 0; c0 < DH; c0 += 16) {
    uint32_t r[16];
    tmem_ld16_wait(taddr + c0, r);
    if (write) {
      uint32_t w[8];
#pragma unroll
      for (int x = 0; x < 8; ++x)
        w[x] = zero ? 0u
                    : pack_bf16x2(__uint_as_float(r[2 * x]) * sc, __uint_as_float(r[2 * x + 1]) * sc);
      *reinterpret_cast<uint4*>(dst + c0) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(dst + c0 + 8) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}
template <int DH>
__device__ __forceinline__ void zero_row(__nv_bfloat16* dst) {
#pragma unroll
  for (int c0 = 0; c0 < DH; c0 += 8) *reinterpret_cast<uint4*>(dst + c0) = make_uint4(0, 0, 0, 0);
}

constexpr int kMaxSplit = 4;  // CTAs of a cluster that share a tile's steps or jobs

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The address of a shared-memory location of this CTA in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_shared(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, const uint32_t* v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}
__device__ __forceinline__ void tmem_ld4_wait(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld8_wait(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

// ---------------------------------------------------------------------------------------
// dQ
// ---------------------------------------------------------------------------------------
template <int DH>
struct QCfg {
  using C = BCfg<DH>;
  static constexpr int TKD = 64;                 // keys per step
  static constexpr int KT_BYTES = TKD * DH * 2;  // one 64-row K or V tile
  static constexpr int STAGES = C::STAGES;
  static constexpr int SMEM = 2 * C::TILE_BYTES + STAGES * 2 * KT_BYTES + 1024 + 512;
  static constexpr int S_COL = 0, DP_COL = 64, DS_COL = 128, DQ_COL = 160;
  static_assert(DQ_COL + DH <= C::TMEM_COLS, "TMEM budget");
  static_assert((kMaxSplit - 1) * 128 * (DH / kMaxSplit) * 4 <= 2 * C::TILE_BYTES,
                "the Q and dO tiles' memory holds the other CTAs' parts");
  static_assert(DH / kMaxSplit % 4 == 0, "parts of whole 16-byte stores");
  static_assert(C::CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory per SM");
};

template <int DH>
__global__ void __launch_bounds__(THREADS, BCfg<DH>::CTAS)
attn_scores_dq_kernel(const __grid_constant__ Params P) {
  using C = BCfg<DH>;
  using Q = QCfg<DH>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sdO = sQ + C::TILE_BYTES;
  uint8_t* sK = sdO + C::TILE_BYTES;
  uint8_t* sV = sK + Q::STAGES * Q::KT_BYTES;
  uint64_t* bar = reinterpret_cast<uint64_t*>(sV + Q::STAGES * Q::KT_BYTES);
  uint64_t* q_full = bar;
  uint64_t* r_full = bar + 1;
  uint64_t* r_empty = r_full + Q::STAGES;
  uint64_t* r_clean = r_empty + Q::STAGES;
  uint64_t* sdp_full = r_clean + Q::STAGES;
  uint64_t* s_free = sdp_full + 1;
  uint64_t* d_ready = s_free + 1;
  uint64_t* d_free = d_ready + 1;
  uint64_t* acc_full = d_free + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile int* bad_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* sp = reinterpret_cast<int*>(tmem_holder + 4);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int bs = P.B * P.S;
  const int item = blockIdx.x / P.split, part = blockIdx.x % P.split;  // part: rank in the cluster
  const int qt = P.nq - 1 - item / bs;
  const int s_idx = item % bs % P.S, b_idx = item % bs / P.S;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < Q::STAGES; ++s) {
      mbar_init(&r_full[s], 1);
      mbar_init(&r_empty[s], 2);  // the product that read it last, and the cleaning warp
      mbar_init(&r_clean[s], 1);
    }
    mbar_init(sdp_full, 1);
    mbar_init(s_free, 4);
    mbar_init(d_ready, 4);
    mbar_init(d_free, 1);
    mbar_init(acc_full, 1);
    *bad_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, C::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&P.tm_q);
    prefetch_tmap(&P.tm_do);
    prefetch_tmap(&P.tm_k);
    prefetch_tmap(&P.tm_v);
  }
  pdl_wait();
  pdl_allow_next();
  const int row = threadIdx.x & 127;
  const int q = qt * TQ + row;
  int b0 = 0, e0 = 0;
  if (warp >= 4) {
    span_of(P.span, b_idx, q, b0, e0);
    const bool live = b0 < e0;
    const int lo = __reduce_min_sync(0xffffffffu, live ? b0 : INT_MAX);
    const int hi = __reduce_max_sync(0xffffffffu, live ? e0 : 0);
    const int blo = __reduce_max_sync(0xffffffffu, live ? b0 : 0);
    const int ehi = __reduce_min_sync(0xffffffffu, live ? e0 : INT_MAX);
    if (lane == 0) {
      int* d = sp + (warp & 3) * 4;
      d[0] = lo;
      d[1] = hi;
      d[2] = blo;
      d[3] = ehi;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int lo = min(min(sp[0], sp[4]), min(sp[8], sp[12]));
  const int hi = max(max(sp[1], sp[5]), max(sp[9], sp[13]));
  const int full_lo = max(max(sp[2], sp[6]), max(sp[10], sp[14]));
  const int full_hi = min(min(sp[3], sp[7]), min(sp[11], sp[15]));
  // this CTA's steps j0 .. j0 + nk - 1: its share of the tile's
  const int tile_j0 = lo < hi ? lo / Q::TKD : 0;
  const int tile_nk = lo < hi ? (hi + Q::TKD - 1) / Q::TKD - tile_j0 : 0;
  const int share = (tile_nk + P.split - 1) / P.split;
  const int j0 = tile_j0 + part * share;
  const int nk = max(0, min(share, tile_nk - part * share));
  auto whole = [&](int j) { return j * Q::TKD >= full_lo && (j + 1) * Q::TKD <= full_hi; };
  if (P.blocks && s_idx == 0 && part == 0 && threadIdx.x == 0)
    P.blocks[(int64_t)b_idx * P.nq + qt] = make_int2(lo, hi);
  const int kvh = s_idx < P.Sr ? s_idx / P.k : 0;
  // the output row of this thread's query (softmax warps)
  auto dq_row = [&]() -> __nv_bfloat16* {
    const int64_t tok = (int64_t)b_idx * P.T + q;
    if (!P.sel) return P.dq + (int64_t)s_idx * P.dq_hs + tok * P.dq_ts;
    if (s_idx >= P.Sr) return P.dq_shared + tok * DH;
    const int e = (s_idx / P.k) * P.experts + P.sel[tok * P.sel_stride + P.sel_off + s_idx];
    return P.dq + tok * P.dq_ts + (int64_t)e * DH;
  };

  bool nan_row = false;
  if (warp < 4) {
    if constexpr (C::CTAS == 2) setmaxnreg_dec<kSmallRegs>();
    if (warp == 0) {
      // ---------------------------------------------------------------- loads
      if (lane == 0 && nk > 0) {
        mbar_arrive_expect_tx(q_full, 2 * C::TILE_BYTES);
        tma_load_5d(sQ, &P.tm_q, 0, qt * TQ, 0, s_idx, b_idx, q_full);
        tma_load_5d(sdO, &P.tm_do, 0, qt * TQ, 0, s_idx, b_idx, q_full);
        int st = 0, j = 0;
        uint32_t ph = 0;
        for (; j < nk; ++j) {
          if (!lane_wait(&r_empty[st], ph ^ 1, P)) break;
          mbar_arrive_expect_tx(&r_full[st], 2 * Q::KT_BYTES);
          tma_load_5d(sK + st * Q::KT_BYTES, &P.tm_k, 0, (j0 + j) * Q::TKD, 0, kvh, b_idx,
                      &r_full[st]);
          tma_load_5d(sV + st * Q::KT_BYTES, &P.tm_v, 0, (j0 + j) * Q::TKD, 0, kvh, b_idx,
                      &r_full[st]);
          if (++st == Q::STAGES) {
            st = 0;
            ph ^= 1;
          }
        }
        drain_ring(q_full, 1, 1);
        drain_ring(r_full, Q::STAGES, j);
      }
    } else if (warp == 3) {
      // ---------------------------------------------------------------- cleaning of K tiles
      int st = 0;
      uint32_t ph = 0;
      for (int j = 0; j < nk; ++j) {
        if (!warp_wait(&r_full[st], ph, P)) break;
        if (!whole(j0 + j)) {
          if (clean_tile(sK + st * Q::KT_BYTES, Q::KT_BYTES)) {
            fence_async_shared();
            if (lane == 0) *bad_flag = 1;
            __threadfence_block();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&r_clean[st]);
        }
        // every tile passes here, so this warp is never a phase of a stage behind or ahead
        if (lane == 0) mbar_arrive(&r_empty[st]);
        if (++st == Q::STAGES) {
          st = 0;
          ph ^= 1;
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA issue
      const uint32_t idesc_s = idesc_bf16_f32(TQ, Q::TKD);
      const uint32_t idesc_dq = idesc_bf16_f32(TQ, DH) | (1u << 16);  // B (K) MN-major
      const uint64_t q_desc = smem_desc(smem_u32(sQ), 8 * C::ROW_BYTES, C::LAYOUT);
      const uint64_t do_desc = smem_desc(smem_u32(sdO), 8 * C::ROW_BYTES, C::LAYOUT);
      const uint64_t k_desc = smem_desc(smem_u32(sK), 8 * C::ROW_BYTES, C::LAYOUT);
      const uint64_t v_desc = smem_desc(smem_u32(sV), 8 * C::ROW_BYTES, C::LAYOUT);
      const uint64_t kmn_desc =
          smem_desc_mn(smem_u32(sK), Q::TKD * C::ROW_BYTES, 8 * C::ROW_BYTES, C::LAYOUT);
      constexpr uint32_t kStep = Q::KT_BYTES >> 4;
      int st_next = 0;
      uint32_t ph = 0, clean_phase = 0;
      // S = Q K^T and dP = dO V^T of step j
      auto issue_sdp = [&](int j) -> bool {
        if (!warp_wait(&r_full[st_next], ph, P)) return false;
        if (!whole(j0 + j)) {
          if (!warp_wait(&r_clean[st_next], (clean_phase >> st_next) & 1, P)) return false;
          clean_phase ^= 1u << st_next;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint64_t kd = k_desc + (uint64_t)(st_next * kStep);
          const uint64_t vd = v_desc + (uint64_t)(st_next * kStep);
#pragma unroll
          for (int kk = 0; kk < DH / 16; ++kk)
            mma_ss(tmem + Q::S_COL, q_desc + kmajor_off<DH, 128>(kk),
                   kd + kmajor_off<DH, Q::TKD>(kk), idesc_s, kk > 0 ? 1u : 0u);
#pragma unroll
          for (int kk = 0; kk < DH / 16; ++kk)
            mma_ss(tmem + Q::DP_COL, do_desc + kmajor_off<DH, 128>(kk),
                   vd + kmajor_off<DH, Q::TKD>(kk), idesc_s, kk > 0 ? 1u : 0u);
          mma_commit(sdp_full);
        }
        __syncwarp();
        if (++st_next == Q::STAGES) {
          st_next = 0;
          ph ^= 1;
        }
        return true;
      };
      bool ok = nk > 0 && warp_wait(q_full, 0, P) && issue_sdp(0);
      int st = 0;
      for (int j = 0; ok && j < nk; ++j) {
        if (j + 1 < nk) {
          // the softmax warps hold S(j), dP(j) in registers: the next pair may be written
          if (!warp_wait(s_free, j & 1, P) || !issue_sdp(j + 1)) break;
        }
        if (!warp_wait(d_ready, j & 1, P)) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t kd = kmn_desc + (uint64_t)(st * kStep);
#pragma unroll
          for (int kk = 0; kk < Q::TKD / 16; ++kk)
            mma_ts(tmem + Q::DQ_COL, tmem + Q::DS_COL + kk * 8,
                   kd + (uint64_t)((kk * 16 * C::ROW_BYTES) >> 4), idesc_dq,
                   (j == 0 && kk == 0) ? 0u : 1u);
          mma_commit(&r_empty[st]);
          mma_commit(d_free);
          if (j + 1 == nk) mma_commit(acc_full);
        }
        __syncwarp();
        if (++st == Q::STAGES) st = 0;
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax + epilogue
    if constexpr (C::CTAS == 2) setmaxnreg_inc<kLargeRegs>();
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_base = tmem + lane_off;
    const bool valid = q < P.T, live = b0 < e0;
    const int64_t tok = (int64_t)b_idx * P.T + q;
    const int64_t srow = (int64_t)s_idx * P.B * P.T + tok;
    const float lse = live ? P.lse[srow] : 0.f;
    float dsum = 0.f;
    if (!P.dout) {
      dsum = live ? P.dsum[srow] : 0.f;
    } else if (valid) {
      // D = <dout, out> in 32 bits; out is the bf16 output
      const __nv_bfloat16* x = P.dout + (int64_t)s_idx * P.dout_hs + tok * P.dout_ts;
      const __nv_bfloat16* y = P.out + (int64_t)s_idx * P.out_hs + tok * P.out_ts;
#pragma unroll
      for (int c0 = 0; c0 < DH; c0 += 8) {
        const uint4 a = *reinterpret_cast<const uint4*>(x + c0);
        const uint4 b = *reinterpret_cast<const uint4*>(y + c0);
        const uint32_t as[4] = {a.x, a.y, a.z, a.w}, bs4[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dsum = fmaf(__uint_as_float(as[i] << 16), __uint_as_float(bs4[i] << 16), dsum);
          dsum = fmaf(__uint_as_float(as[i] & 0xffff0000u),
                      __uint_as_float(bs4[i] & 0xffff0000u), dsum);
        }
      }
      if (part == 0) P.dsum[srow] = dsum;
    }
    const float slope2 = P.slopes ? P.slopes[s_idx] * kLog2e : 0.f;
    const int q0 = qt * TQ;
    bool ok = true;
    by_form(P.cap.on, P.slopes != nullptr, [&](auto cap, auto bias) {
      constexpr bool CAP = decltype(cap)::value, BIAS = decltype(bias)::value;
      for (int j = 0; j < nk; ++j) {
        if (!warp_wait(sdp_full, j & 1, P)) { ok = false; break; }
        tc_fence_after();
        const int kv0 = (j0 + j) * Q::TKD;
        uint32_t pk[32];
        {
          float sr[64];
          uint32_t dr[64];
          {
            uint32_t r[64];
            tmem_ld64_wait(t_base + Q::S_COL, r);
#pragma unroll
            for (int c = 0; c < 64; ++c) sr[c] = __uint_as_float(r[c]);
          }
          tmem_ld64_wait(t_base + Q::DP_COL, dr);
          if (j + 1 < nk) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_free);
          }
          const bool poly = !CAP || !__any_sync(0xffffffffu, !(abs_max<64>(sr) < P.cap.limit));
          const float in = CAP ? P.cap.log2 : P.scale_log2;
          const float2 in2 = make_float2(in, in), nl2 = make_float2(-lse, -lse);
          const float Ds = CAP ? dsum : -dsum;
          const float2 nD2 = make_float2(Ds, Ds), m1 = make_float2(-1.f, -1.f);
          // dz of the scores' columns 2x, 2x + 1, their bias and -lse in b
          auto pair = [&](int x, float2 b, auto pl) {
            float2 v = make_float2(sr[2 * x], sr[2 * x + 1]);
            if constexpr (CAP) v = cap_tanh<decltype(pl)::value>(P.cap, v);
            const float2 t = fma2(v, in2, b);
            const float2 p = (x & 7) >= 8 - kBwdFma<CAP, BIAS>
                                 ? exp2_fma2_nan(t)
                                 : make_float2(ex2(t.x), ex2(t.y));
            const float2 dp = make_float2(__uint_as_float(dr[2 * x]), __uint_as_float(dr[2 * x + 1]));
            if constexpr (CAP)  // (1 - tanh^2) (dP - D) = (tanh^2 - 1) (D - dP)
              return mul2(mul2(p, fma2(dp, m1, nD2)), fma2(v, v, m1));
            else
              return mul2_ftz(p, add2(dp, nD2));
          };
          const float d0 = (float)(kv0 - q);
          auto all = [&](auto pl) {
            if (!BIAS || kv0 + Q::TKD - 1 <= q0) {
              // no bias, or every key at or before every query: the distance is linear (four
              // chains of additions, eight columns a step: packed constants would be moved in)
              const float base = fmaf(d0, slope2, -lse);
              const float2 step = make_float2(8.f * slope2, 8.f * slope2);
              float2 chain[4];
  #pragma unroll
              for (int i = 0; i < 4; ++i)
                chain[i] = make_float2(fmaf(slope2, (float)(2 * i), base),
                                       fmaf(slope2, (float)(2 * i + 1), base));
  #pragma unroll
              for (int x = 0; x < 32; ++x) {
                const float2 d = pair(x, BIAS ? chain[x & 3] : nl2, pl);
                if constexpr (BIAS) chain[x & 3] = add2(chain[x & 3], step);
                sr[2 * x] = d.x;
                sr[2 * x + 1] = d.y;
              }
            } else {
  #pragma unroll
              for (int x = 0; x < 32; ++x) {
                const float2 d =
                    pair(x, make_float2(fmaf(-slope2, fabsf(d0 + (float)(2 * x)), -lse),
                                        fmaf(-slope2, fabsf(d0 + (float)(2 * x + 1)), -lse)), pl);
                sr[2 * x] = d.x;
                sr[2 * x + 1] = d.y;
              }
            }
          };
          if (CAP && !poly) all(std::integral_constant<bool, false>{});
          else all(std::integral_constant<bool, true>{});
          // masks, each side only where some row has it inside the step
          if (kv0 < full_lo) {
            const int first = live ? b0 - kv0 : 64;
#pragma unroll
            for (int c = 0; c < 64; ++c) sr[c] = c < first ? 0.f : sr[c];
          }
          if (kv0 + Q::TKD > full_hi) {
            const int last = live ? e0 - kv0 : 0;
#pragma unroll
            for (int c = 0; c < 64; ++c) sr[c] = c >= last ? 0.f : sr[c];
          }
#pragma unroll
          for (int x = 0; x < 32; ++x) pk[x] = pack_bf16x2(sr[2 * x], sr[2 * x + 1]);
        }
        // the previous dQ product has read dz: it may be overwritten
        if (j > 0 && !warp_wait(d_free, (j - 1) & 1, P)) { ok = false; break; }
#pragma unroll
        for (int c0 = 0; c0 < 32; c0 += 8) tmem_st8(t_base + Q::DS_COL + c0, pk + c0);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(d_ready);
      }
    });
    if (ok && nk > 0) ok = warp_wait(acc_full, 0, P);
    if (ok) tc_fence_after();
    // A cleaned K tile hides the infinities and NaN that a row does see, and its scores of -inf
    // were formed without them: the row becomes NaN (rare; whole tiles are not cleaned and carry
    // theirs themselves).
    if (ok && nk > 0 && *bad_flag && valid && live) {
      for (int j = j0; j < j0 + nk; ++j) {
        if (whole(j)) continue;
        const int u1 = min(e0, (j + 1) * Q::TKD);
        for (int u = max(b0, j * Q::TKD); u < u1; ++u) {
          const uint32_t* kr = reinterpret_cast<const uint32_t*>(
              P.keys + (int64_t)kvh * P.key_hs + ((int64_t)b_idx * P.T + u) * P.key_ts);
          for (int c = 0; c < DH / 2; ++c)
            if ((kr[c] & 0x7f80u) == 0x7f80u || (kr[c] & 0x7f800000u) == 0x7f800000u) nan_row = true;
        }
      }
    }
    if (ok && P.split == 1) {
      __nv_bfloat16* dst = valid ? dq_row() : nullptr;
      const float sc = nan_row ? __int_as_float(0x7fffffff) : P.scale;
      if (nk > 0) store_row<DH>(t_base + Q::DQ_COL, dst, sc, valid, !live);
      else if (valid) zero_row<DH>(dst);
    }
  }
  if (P.split > 1) {
    // The cluster's CTAs hold partial sums of the same rows. Each takes one part of the columns:
    // it receives the others' values of them in its own shared memory (the tiles there have been
    // read) and adds the parts in rank order.
    cluster_sync();  // every CTA's products are done
    const int cols = DH / P.split;  // columns of a part, a multiple of 4
    const uint32_t t_acc = tmem + ((uint32_t)((warp & 3) * 32) << 16) + Q::DQ_COL;
    if (warp >= 4) {
      for (int p = 0; p < P.split; ++p) {
        if (p == part) continue;
        const int slot = part < p ? part : part - 1;
        const uint32_t dst = map_shared(smem_u32(smem) + (slot * cols / 4 * 128 + row) * 16, p);
        for (int c = 0; c < cols; c += 4) {
          uint32_t v[4];
          tmem_ld4_wait(t_acc + p * cols + c, v);
          if (nk == 0) v[0] = v[1] = v[2] = v[3] = 0u;
          if (nan_row) v[0] = v[1] = v[2] = v[3] = 0x7fffffffu;
          st_cluster_v4(dst + c / 4 * 2048, v);
        }
      }
    }
    cluster_sync();  // all parts have arrived
    if (warp >= 4) {
      const bool valid = q < P.T, live = b0 < e0;
      __nv_bfloat16* dst = valid ? dq_row() : nullptr;
      const float4* got = reinterpret_cast<const float4*>(smem);
      for (int c = 0; c < cols; c += 4) {
        uint32_t v[4];
        tmem_ld4_wait(t_acc + part * cols + c, v);
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        for (int p = 0; p < P.split; ++p) {
          if (p == part) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              sum[i] += nan_row ? __int_as_float(0x7fffffff) : nk == 0 ? 0.f : __uint_as_float(v[i]);
          } else {
            const int slot = p < part ? p : p - 1;
            const float4 x = got[(slot * cols + c) / 4 * 128 + row];
            sum[0] += x.x; sum[1] += x.y; sum[2] += x.z; sum[3] += x.w;
          }
        }
        if (valid)
          *reinterpret_cast<uint2*>(dst + part * cols + c) =
              live ? make_uint2(pack_bf16x2(sum[0] * P.scale, sum[1] * P.scale),
                                pack_bf16x2(sum[2] * P.scale, sum[3] * P.scale))
                   : make_uint2(0u, 0u);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------------------
// dK, dV. Jobs of TQJ queries, small enough that S^T, dP^T, p^T, dz^T, dV and dK all have TMEM
// columns of their own: at two CTAs per SM (256 columns) 48 queries for head dims up to 48
// and 32 for 64; at one CTA per SM (512 columns) 64.
// ---------------------------------------------------------------------------------------
template <int DH>
struct KCfg {
  using C = BCfg<DH>;
  static constexpr int TQJ = DH <= 48 ? 48 : (DH <= 64 ? 32 : 64);
  static constexpr int QT_BYTES = TQJ * DH * 2;
  static constexpr int STAGES = C::STAGES;
  // per stage a job's -lse, -D, first keys, ends of keys, and whether it is seen whole
  static constexpr int STAT_BYTES = (4 * TQJ + 4) * 4;
  static constexpr int SMEM =
      2 * C::TILE_BYTES + STAGES * (2 * QT_BYTES + STAT_BYTES) + 1024 + 512;
  static constexpr int S_COL = 0, DP_COL = TQJ, P_COL = 2 * TQJ, DS_COL = 2 * TQJ + TQJ / 2;
  static constexpr int DV_COL = 3 * TQJ, DK_COL = 3 * TQJ + DH;
  static_assert(TQJ % 16 == 0 && TQJ <= 64, "a job's queries: two per lane at most");
  static_assert(DK_COL + DH <= C::TMEM_COLS, "TMEM budget");
  static_assert(DK_COL == DV_COL + DH, "the cluster's sum takes [dV | dK] as one row");
  static_assert((kMaxSplit - 1) * 128 * (2 * DH / kMaxSplit) * 4 <=
                    2 * C::TILE_BYTES + STAGES * 2 * QT_BYTES,
                "the tiles' memory holds the other CTAs' parts");
  static_assert(2 * DH / kMaxSplit % 8 == 0, "parts of whole 16-byte stores");
  static_assert(C::CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory per SM");
};

template <int DH>
__global__ void __launch_bounds__(THREADS, BCfg<DH>::CTAS)
attn_scores_dkdv_kernel(const __grid_constant__ Params P) {
  using C = BCfg<DH>;
  using K = KCfg<DH>;
  constexpr int TQJ = K::TQJ;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sK = smem;
  uint8_t* sV = sK + C::TILE_BYTES;
  uint8_t* sQ = sV + C::TILE_BYTES;
  uint8_t* sdO = sQ + K::STAGES * K::QT_BYTES;
  uint8_t* sStat = sdO + K::STAGES * K::QT_BYTES;
  uint64_t* bar = reinterpret_cast<uint64_t*>(sStat + K::STAGES * K::STAT_BYTES);
  uint64_t* kv_full = bar;
  uint64_t* r_full = bar + 1;
  uint64_t* r_empty = r_full + K::STAGES;
  uint64_t* r_clean = r_empty + K::STAGES;
  uint64_t* sdp_full = r_clean + K::STAGES;
  uint64_t* s_free = sdp_full + 1;
  uint64_t* d_ready = s_free + 1;
  uint64_t* d_free = d_ready + 1;
  uint64_t* acc_full = d_free + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(acc_full + 1);
  int* sp = reinterpret_cast<int*>(tmem_holder + 4);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // first key tiles first: under a causal mask the most queries see them
  const int bg = P.B * P.G;
  const int item = blockIdx.x / P.split, part = blockIdx.x % P.split;  // part: rank in the cluster
  const int kt = item / bg, g = item % bg % P.G, b_idx = item % bg / P.G;
  const int u0 = kt * TK, u1 = min(u0 + TK, P.T);
  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int s = 0; s < K::STAGES; ++s) {
      mbar_init(&r_full[s], 1);
      mbar_init(&r_empty[s], 1);
      mbar_init(&r_clean[s], 1);
    }
    mbar_init(sdp_full, 1);
    mbar_init(s_free, 4);
    mbar_init(d_ready, 4);
    mbar_init(d_free, 1);
    mbar_init(acc_full, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, C::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&P.tm_q);
    prefetch_tmap(&P.tm_do);
    prefetch_tmap(&P.tm_k);
    prefetch_tmap(&P.tm_v);
  }
  pdl_wait();
  pdl_allow_next();
  // the 128-row blocks of queries that may see a key of this tile: first .. last
  int first = INT_MAX, last = -1;
  if (P.blocks) {
    for (int i = threadIdx.x; i < P.nq; i += THREADS) {
      const int2 v = P.blocks[(int64_t)b_idx * P.nq + i];
      if (v.x < u1 && v.y > u0) {
        first = min(first, i);
        last = max(last, i);
      }
    }
    first = __reduce_min_sync(0xffffffffu, first);
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0) {
      sp[2 * warp] = first;
      sp[2 * warp + 1] = last;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  int q_lo = P.span.causal ? u0 : 0, q_hi = P.T;  // queries q_lo .. q_hi - 1
  if (P.blocks) {
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      first = min(first, sp[2 * w]);
      last = max(last, sp[2 * w + 1]);
    }
    q_lo = last >= 0 ? first * TQ : 0;
    q_hi = last >= 0 ? min(P.T, (last + 1) * TQ) : 0;
  }
  const int qt0 = q_lo / TQJ;
  const int per = q_lo < q_hi ? (q_hi + TQJ - 1) / TQJ - qt0 : 0;  // query tiles of a stream
  const int ns = P.k + (g == 0 && P.S > P.Sr ? 1 : 0);             // streams of the head
  // this CTA's share of the item's jobs: nj from job (si0, r0) on
  const int nj_all = ns * per;
  const int j_first = (int)((int64_t)nj_all * part / P.split);
  const int nj = (int)((int64_t)nj_all * (part + 1) / P.split) - j_first;
  const int si0 = per > 0 ? j_first / per : 0, r0 = per > 0 ? j_first % per : 0;
  auto stream_of = [&](int si) { return si < P.k ? g * P.k + si : P.Sr; };
  if (warp < 4) {
    if constexpr (C::CTAS == 2) setmaxnreg_dec<kSmallRegs>();
    if (warp == 0) {
      // ---------------------------------------------------------------- loads
      if (lane == 0 && nj > 0) {
        mbar_arrive_expect_tx(kv_full, 2 * C::TILE_BYTES);
        tma_load_5d(sK, &P.tm_k, 0, u0, 0, g, b_idx, kv_full);
        tma_load_5d(sV, &P.tm_v, 0, u0, 0, g, b_idx, kv_full);
        int st = 0, si = si0, r = r0, j = 0;
        uint32_t ph = 0;
        for (; j < nj; ++j) {
          if (!lane_wait(&r_empty[st], ph ^ 1, P)) break;
          mbar_arrive_expect_tx(&r_full[st], 2 * K::QT_BYTES);
          const int s = stream_of(si), qrow = (qt0 + r) * TQJ;
          tma_load_5d(sQ + st * K::QT_BYTES, &P.tm_q, 0, qrow, 0, s, b_idx, &r_full[st]);
          tma_load_5d(sdO + st * K::QT_BYTES, &P.tm_do, 0, qrow, 0, s, b_idx, &r_full[st]);
          if (++r == per) {
            r = 0;
            ++si;
          }
          if (++st == K::STAGES) {
            st = 0;
            ph ^= 1;
          }
        }
        drain_ring(kv_full, 1, 1);
        drain_ring(r_full, K::STAGES, j);
      }
    } else if (warp == 3) {
      // ------------------------------------------ per job: the rows' lse, D and intervals
      // for the softmax warps, and the cleaning of q and dout tiles that are seen in part
      int st = 0, si = si0, r = r0;
      uint32_t ph = 0;
      // lane l holds queries l and l + 32 of a job, loaded a job ahead
      int jb[2], je[2];
      float nl[2], nd[2];
      auto fetch = [&]() {
        const int64_t base = (int64_t)stream_of(si) * P.B * P.T + (int64_t)b_idx * P.T;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int qq = (qt0 + r) * TQJ + lane + 32 * h;
          jb[h] = je[h] = 0;
          nl[h] = nd[h] = 0.f;
          if (lane + 32 * h < TQJ) {
            span_of(P.span, b_idx, qq, jb[h], je[h]);
            if (qq < P.T) {
              nl[h] = -P.lse[base + qq];
              nd[h] = -P.dsum[base + qq];
            }
          }
        }
        if (++r == per) {
          r = 0;
          ++si;
        }
      };
      if (nj > 0) fetch();
      for (int j = 0; j < nj; ++j) {
        // the stage's statistics were read before its products ended
        if (!warp_wait(&r_empty[st], ph ^ 1, P)) break;
        float* f = reinterpret_cast<float*>(sStat + st * K::STAT_BYTES);
        int* fi = reinterpret_cast<int*>(f + 2 * TQJ);
        bool w = true;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = lane + 32 * h;
          if (c < TQJ) {
            const bool live = jb[h] < je[h];  // false for queries past the sequence
            f[c] = live ? nl[h] : 0.f;
            f[TQJ + c] = live ? nd[h] : 0.f;
            fi[c] = jb[h];
            fi[TQJ + c] = je[h];
            w = w && jb[h] <= u0 && je[h] >= u1;
          }
        }
        w = __all_sync(0xffffffffu, w) != 0;
        if (lane == 0) fi[2 * TQJ] = w;
        if (j + 1 < nj) fetch();
        if (!warp_wait(&r_full[st], ph, P)) break;
        if (!w) {
          const bool bq = clean_tile(sQ + st * K::QT_BYTES, K::QT_BYTES);
          const bool bd = clean_tile(sdO + st * K::QT_BYTES, K::QT_BYTES);
          if (bq || bd) fence_async_shared();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&r_clean[st]);
        if (++st == K::STAGES) {
          st = 0;
          ph ^= 1;
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA issue
      const uint32_t idesc_s = idesc_bf16_f32(TK, TQJ);
      const uint32_t idesc_kv = idesc_bf16_f32(TK, DH) | (1u << 16);  // B (Q, dO) MN-major
      const uint64_t k_desc = smem_desc(smem_u32(sK), 8 * C::ROW_BYTES, C::LAYOUT);
      const uint64_t v_desc = smem_desc(smem_u32(sV), 8 * C::ROW_BYTES, C::LAYOUT);
      const uint64_t q_desc = smem_desc(smem_u32(sQ), 8 * C::ROW_BYTES, C::LAYOUT);
      const uint64_t do_desc = smem_desc(smem_u32(sdO), 8 * C::ROW_BYTES, C::LAYOUT);
      const uint64_t qmn_desc =
          smem_desc_mn(smem_u32(sQ), TQJ * C::ROW_BYTES, 8 * C::ROW_BYTES, C::LAYOUT);
      const uint64_t domn_desc =
          smem_desc_mn(smem_u32(sdO), TQJ * C::ROW_BYTES, 8 * C::ROW_BYTES, C::LAYOUT);
      constexpr uint32_t kStep = K::QT_BYTES >> 4;
      int st_next = 0;
      uint32_t ph = 0;
      // S^T = K Q^T and dP^T = V dO^T of the next job
      auto issue_sdp = [&]() -> bool {
        if (!warp_wait(&r_full[st_next], ph, P) || !warp_wait(&r_clean[st_next], ph, P))
          return false;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t qd = q_desc + (uint64_t)(st_next * kStep);
          const uint64_t dd = do_desc + (uint64_t)(st_next * kStep);
#pragma unroll
          for (int kk = 0; kk < DH / 16; ++kk)
            mma_ss(tmem + K::S_COL, k_desc + kmajor_off<DH, 128>(kk), qd + kmajor_off<DH, TQJ>(kk),
                   idesc_s, kk > 0 ? 1u : 0u);
#pragma unroll
          for (int kk = 0; kk < DH / 16; ++kk)
            mma_ss(tmem + K::DP_COL, v_desc + kmajor_off<DH, 128>(kk),
                   dd + kmajor_off<DH, TQJ>(kk), idesc_s, kk > 0 ? 1u : 0u);
          mma_commit(sdp_full);
        }
        __syncwarp();
        if (++st_next == K::STAGES) {
          st_next = 0;
          ph ^= 1;
        }
        return true;
      };
      bool ok = nj > 0 && warp_wait(kv_full, 0, P) && issue_sdp();
      int st = 0;
      for (int j = 0; ok && j < nj; ++j) {
        if (j + 1 < nj) {
          if (!warp_wait(s_free, j & 1, P) || !issue_sdp()) break;
        }
        if (!warp_wait(d_ready, j & 1, P)) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t dmn = domn_desc + (uint64_t)(st * kStep);
          const uint64_t qmn = qmn_desc + (uint64_t)(st * kStep);
#pragma unroll
          for (int kk = 0; kk < TQJ / 16; ++kk)
            mma_ts(tmem + K::DV_COL, tmem + K::P_COL + kk * 8,
                   dmn + (uint64_t)((kk * 16 * C::ROW_BYTES) >> 4), idesc_kv,
                   (j == 0 && kk == 0) ? 0u : 1u);
#pragma unroll
          for (int kk = 0; kk < TQJ / 16; ++kk)
            mma_ts(tmem + K::DK_COL, tmem + K::DS_COL + kk * 8,
                   qmn + (uint64_t)((kk * 16 * C::ROW_BYTES) >> 4), idesc_kv,
                   (j == 0 && kk == 0) ? 0u : 1u);
          mma_commit(&r_empty[st]);
          mma_commit(d_free);
          if (j + 1 == nj) mma_commit(acc_full);
        }
        __syncwarp();
        if (++st == K::STAGES) st = 0;
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax + epilogue
    if constexpr (C::CTAS == 2) setmaxnreg_inc<kLargeRegs>();
    const int row = (warp & 3) * 32 + lane;  // key row of the tile
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_base = tmem + lane_off;
    const int u = u0 + row;
    const bool key_ok = u < P.T;
    bool ok = true;
    by_form(P.cap.on, P.slopes != nullptr, [&](auto cap, auto bias) {
      constexpr bool CAP = decltype(cap)::value, BIAS = decltype(bias)::value;
      int si = si0, r = r0, st = 0;
      uint32_t ph = 0;
      for (int j = 0; j < nj; ++j) {
        const float* sL = reinterpret_cast<const float*>(sStat + st * K::STAT_BYTES);
        const float* sD = sL + TQJ;
        const int* sB = reinterpret_cast<const int*>(sD + TQJ);
        const int* sE = sB + TQJ;
        const float slope2 = BIAS ? P.slopes[stream_of(si)] * kLog2e : 0.f;
        const int qa = (qt0 + r) * TQJ;  // the job's first query
        const float d0 = (float)(qa - u);
        if (++r == per) {
          r = 0;
          ++si;
        }
        if (!warp_wait(&r_clean[st], ph, P)) { ok = false; break; }
        const bool all_live = sE[TQJ] != 0;
        if (++st == K::STAGES) {
          st = 0;
          ph ^= 1;
        }
        if (!warp_wait(sdp_full, j & 1, P)) { ok = false; break; }
        tc_fence_after();
        uint32_t pp[TQJ / 2], pd[TQJ / 2];
        {
          float sr[TQJ];
          uint32_t dr[TQJ];
          {
            uint32_t r[TQJ];
            tmem_ldN_wait<TQJ>(t_base + K::S_COL, r);
#pragma unroll
            for (int c = 0; c < TQJ; ++c) sr[c] = __uint_as_float(r[c]);
          }
          tmem_ldN_wait<TQJ>(t_base + K::DP_COL, dr);
          if (j + 1 < nj) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_free);
          }
          const bool poly = !CAP || !__any_sync(0xffffffffu, !(abs_max<TQJ>(sr) < P.cap.limit));
          const float in = CAP ? P.cap.log2 : P.scale_log2;
          const float2 in2 = make_float2(in, in);
          // Plain jobs: every query sees every key and lies at or behind it, so there is nothing
          // to mask and the bias is linear. The loop has no branches: one in it would keep the
          // pairs' chains of operations from overlapping (31 cycles a score instead of 12).
          const bool plain = all_live && (!BIAS || qa >= u1 - 1);
          const float2 step = make_float2(-8.f * slope2, -8.f * slope2);
          float2 chain[4];  // the linear bias of four pairs, eight queries a step
#pragma unroll
          for (int i = 0; i < 4; ++i)
            chain[i] = make_float2(-slope2 * (d0 + (float)(2 * i)), -slope2 * (d0 + (float)(2 * i + 1)));
          auto all = [&](auto pl, auto pn) {
            constexpr bool PLAIN = decltype(pn)::value;
  #pragma unroll
            for (int x4 = 0; x4 < TQJ / 4; ++x4) {
              const float4 L4 = reinterpret_cast<const float4*>(sL)[x4];  // -lse
              const float4 D4 = reinterpret_cast<const float4*>(sD)[x4];  // -D
              const float2 nL[2] = {make_float2(L4.x, L4.y), make_float2(L4.z, L4.w)};
              const float2 nD[2] = {make_float2(D4.x, D4.y), make_float2(D4.z, D4.w)};
              float2 p[2], d[2];
  #pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int c = 4 * x4 + 2 * h;
                float2 v = make_float2(sr[c], sr[c + 1]);
                if constexpr (CAP) v = cap_tanh<decltype(pl)::value>(P.cap, v);
                float2 b = nL[h];
                if constexpr (BIAS) {
                  if constexpr (PLAIN) {
                    b = add2(b, chain[(c >> 1) & 3]);
                    chain[(c >> 1) & 3] = add2(chain[(c >> 1) & 3], step);
                  } else {
                    b.x = fmaf(-slope2, fabsf(d0 + (float)c), b.x);
                    b.y = fmaf(-slope2, fabsf(d0 + (float)(c + 1)), b.y);
                  }
                }
                const float2 t = fma2(v, in2, b);
                p[h] = ((c >> 1) & 7) >= 8 - kBwdFma<CAP, BIAS> ? exp2_fma2_nan(t)
                                                                : make_float2(ex2(t.x), ex2(t.y));
                const float2 g = add2(make_float2(__uint_as_float(dr[c]), __uint_as_float(dr[c + 1])),
                                      nD[h]);
                if constexpr (CAP)  // (1 - tanh^2) g, the sign in the factor -p
                  d[h] = mul2(mul2(g, mul2(p[h], make_float2(-1.f, -1.f))),
                              fma2(v, v, make_float2(-1.f, -1.f)));
                else
                  d[h] = mul2_ftz(p[h], g);
              }
              if constexpr (!PLAIN) {
                const int4 B4 = reinterpret_cast<const int4*>(sB)[x4];
                const int4 E4 = reinterpret_cast<const int4*>(sE)[x4];
                const bool in0 = u >= B4.x && u < E4.x, in1 = u >= B4.y && u < E4.y;
                const bool in2b = u >= B4.z && u < E4.z, in3 = u >= B4.w && u < E4.w;
                // a row whose dout was cleaned has an infinite or NaN D, which p takes on
                p[0].x = in0 ? fmaf(0.f, nD[0].x, p[0].x) : 0.f;
                p[0].y = in1 ? fmaf(0.f, nD[0].y, p[0].y) : 0.f;
                p[1].x = in2b ? fmaf(0.f, nD[1].x, p[1].x) : 0.f;
                p[1].y = in3 ? fmaf(0.f, nD[1].y, p[1].y) : 0.f;
                d[0].x = in0 ? d[0].x : 0.f;
                d[0].y = in1 ? d[0].y : 0.f;
                d[1].x = in2b ? d[1].x : 0.f;
                d[1].y = in3 ? d[1].y : 0.f;
              }
              pp[2 * x4] = pack_bf16x2(p[0].x, p[0].y);
              pp[2 * x4 + 1] = pack_bf16x2(p[1].x, p[1].y);
              pd[2 * x4] = pack_bf16x2(d[0].x, d[0].y);
              pd[2 * x4 + 1] = pack_bf16x2(d[1].x, d[1].y);
            }
          };
          by_flag(plain, [&](auto pn) {
            if (CAP && !poly) all(std::integral_constant<bool, false>{}, pn);
            else all(std::integral_constant<bool, true>{}, pn);
          });
        }
        // the previous job's products have read p^T and dz^T
        if (j > 0 && !warp_wait(d_free, (j - 1) & 1, P)) { ok = false; break; }
#pragma unroll
        for (int c0 = 0; c0 < TQJ / 2; c0 += 8) {
          tmem_st8(t_base + K::P_COL + c0, pp + c0);
          tmem_st8(t_base + K::DS_COL + c0, pd + c0);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(d_ready);
      }
    });
    if (ok && nj > 0) ok = warp_wait(acc_full, 0, P);
    tc_fence_after();
    const int64_t tok = (int64_t)b_idx * P.T + u;
    if (P.split == 1 && ok) {
      __nv_bfloat16* dk = P.dk + (int64_t)g * P.dk_hs + tok * P.dk_ts;
      __nv_bfloat16* dv = P.dv + (int64_t)g * P.dv_hs + tok * P.dv_ts;
      if (nj > 0) {
        store_row<DH>(t_base + K::DK_COL, dk, P.scale, key_ok, false);
        store_row<DH>(t_base + K::DV_COL, dv, 1.f, key_ok, false);
      } else if (key_ok) {
        zero_row<DH>(dk);
        zero_row<DH>(dv);
      }
    }
  }
  if (P.split > 1) {
    // The cluster's CTAs hold partial sums of the same rows of [dV | dK]. Each takes one part
    // of the columns: it receives the others' values of them in its own shared memory (the
    // tiles there have been read) and adds the parts in rank order.
    cluster_sync();  // every CTA's products are done
    const int cols = 2 * DH / P.split;  // columns of a part, a multiple of 8
    const int row = (warp & 3) * 32 + lane;
    const uint32_t t_acc = tmem + ((uint32_t)((warp & 3) * 32) << 16) + K::DV_COL;
    if (warp >= 4) {
      for (int p = 0; p < P.split; ++p) {
        if (p == part) continue;
        const int slot = part < p ? part : part - 1;
        const uint32_t dst = map_shared(smem_u32(smem) + (slot * cols / 4 * 128 + row) * 16, p);
        for (int c = 0; c < cols; c += 8) {
          uint32_t v[8];
          tmem_ld8_wait(t_acc + p * cols + c, v);
          if (nj == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0u;
          }
          st_cluster_v4(dst + c / 4 * 2048, v);
          st_cluster_v4(dst + (c / 4 + 1) * 2048, v + 4);
        }
      }
    }
    cluster_sync();  // all parts have arrived
    if (warp >= 4) {
      const int u = u0 + row;
      const bool key_ok = u < P.T;
      const int64_t tok = (int64_t)b_idx * P.T + u;
      const float4* got = reinterpret_cast<const float4*>(smem);
      for (int c = 0; c < cols; c += 8) {
        uint32_t v[8];
        tmem_ld8_wait(t_acc + part * cols + c, v);
        float sum[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = 0.f;
        for (int p = 0; p < P.split; ++p) {
          if (p == part) {
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += nj == 0 ? 0.f : __uint_as_float(v[i]);
          } else {
            const int slot = p < part ? p : p - 1;
            const float4 x = got[(slot * cols + c) / 4 * 128 + row];
            const float4 y = got[((slot * cols + c) / 4 + 1) * 128 + row];
            sum[0] += x.x; sum[1] += x.y; sum[2] += x.z; sum[3] += x.w;
            sum[4] += y.x; sum[5] += y.y; sum[6] += y.z; sum[7] += y.w;
          }
        }
        const int col = part * cols + c;
        const bool is_k = col >= DH;
        const float sc = is_k ? P.scale : 1.f;
        __nv_bfloat16* dst = is_k ? P.dk + (int64_t)g * P.dk_hs + tok * P.dk_ts + (col - DH)
                                  : P.dv + (int64_t)g * P.dv_hs + tok * P.dv_ts + col;
        if (key_ok)
          *reinterpret_cast<uint4*>(dst) =
              make_uint4(pack_bf16x2(sum[0] * sc, sum[1] * sc), pack_bf16x2(sum[2] * sc, sum[3] * sc),
                         pack_bf16x2(sum[4] * sc, sum[5] * sc), pack_bf16x2(sum[6] * sc, sum[7] * sc));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// items * P.split CTAs in clusters of P.split, as a programmatic dependent launch.
bool launch_cluster(void (*kernel)(const Params), int64_t items, int smem, cudaStream_t st,
                    const Params& P) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * P.split));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)P.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = P.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, P) == cudaSuccess;
}

template <int DH>
int launch_dh(const AttnArgs& a, cudaStream_t st) {
  using C = BCfg<DH>;
  using Q = QCfg<DH>;
  using K = KCfg<DH>;
  if (!set_smem_limit_once<attn_scores_dq_kernel<DH>>(Q::SMEM)) return -1;
  if (!set_smem_limit_once<attn_scores_dkdv_kernel<DH>>(K::SMEM)) return -1;
  const CUtensorMapSwizzle sw = C::CW == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_32B;
  Params P;
  memset(&P, 0, sizeof(P));
  P.span = SpanArgs{a.key_begin, a.key_end, a.T, a.causal};
  P.lse = a.lse;
  P.dsum = a.dsum;
  P.slopes = a.slopes;
  const bool masked = a.key_begin || a.key_end;
  P.blocks = masked ? a.blocks : nullptr;
  P.dq = static_cast<__nv_bfloat16*>(a.dq.data);
  P.dk = static_cast<__nv_bfloat16*>(a.dk.data);
  P.dv = static_cast<__nv_bfloat16*>(a.dv.data);
  P.dq_hs = a.dq.head_stride;
  P.dq_ts = a.dq.token_stride;
  P.dk_hs = a.dk.head_stride;
  P.dk_ts = a.dk.token_stride;
  P.dv_hs = a.dv.head_stride;
  P.dv_ts = a.dv.token_stride;
  P.sel = a.sel;
  P.dq_shared = static_cast<__nv_bfloat16*>(a.dq_shared);
  P.sel_stride = a.sel_stride;
  P.sel_off = a.sel_off;
  P.experts = a.experts;
  P.T = a.T;
  P.B = a.B;
  P.S = a.S;
  P.Sr = a.G * a.k;
  P.k = a.k;
  P.keys = static_cast<const __nv_bfloat16*>(a.kk.data);
  P.key_hs = a.kk.head_stride;
  P.key_ts = a.kk.token_stride;
  P.G = a.G;
  P.nq = (a.T + TQ - 1) / TQ;
  P.scale = a.scale;
  P.scale_log2 = a.scale * kLog2e;
  P.cap = cap_form(a.scale, a.softcap);
  P.status = a.status;
  P.spin = a.spin > 0 ? a.spin : (int64_t)1 << 22;
  const int num_sms = current_num_sms();
  if (num_sms < 0) return -1;
  if (!a.dsum_given) {
    P.dout = static_cast<const __nv_bfloat16*>(a.dout.data);
    P.dout_hs = a.dout.head_stride;
    P.dout_ts = a.dout.token_stride;
    P.out = static_cast<const __nv_bfloat16*>(a.out.data);
    P.out_hs = a.out.head_stride;
    P.out_ts = a.out.token_stride;
  }
  if (!tmap_heads(&P.tm_q, a.q, a.B, a.T, DH, C::CW, TQ, sw) ||
      !tmap_heads(&P.tm_do, a.dout, a.B, a.T, DH, C::CW, TQ, sw) ||
      !tmap_heads(&P.tm_k, a.kk, a.B, a.T, DH, C::CW, Q::TKD, sw) ||
      !tmap_heads(&P.tm_v, a.v, a.B, a.T, DH, C::CW, Q::TKD, sw))
    return -1;
  const int64_t q_items = (int64_t)a.B * a.S * P.nq;
  P.split = 1;
  // A query tile's steps are split over a cluster while the grid leaves an SM's second CTA empty
  // and every CTA keeps 16 steps of the longest row. Under a plain causal mask the last tiles have
  // the most steps, so there also a grid below one CTA per place is split if it keeps 32. Backward
  // of 9 streams of 48, without and with: 4096 causal tokens 175, 157 us; 2 x 2048 133, 124; 2 x
  // 1024 55, 52. Not split, for what it would cost: 4 x 1024 causal 84, 88; all of 4096 keys 256,
  // 263; 5 documents 106, 109. With one CTA per SM (1024 tokens of 128) it costs more: 61, 74.
  if (C::CTAS == 2) {
    const bool triangle = a.causal && !a.key_begin && !a.key_end;
    auto splits = [&](int n) {
      return (q_items * n < num_sms && a.T >= 1024 * n) ||
             (triangle && q_items * n < 2 * (int64_t)num_sms && a.T >= 2048 * n);
    };
    while (P.split < kMaxSplit && splits(P.split)) P.split *= 2;
  }
  if (!launch_cluster(attn_scores_dq_kernel<DH>, q_items, Q::SMEM, st, P)) return -1;
  if (!tmap_heads(&P.tm_q, a.q, a.B, a.T, DH, C::CW, K::TQJ, sw) ||
      !tmap_heads(&P.tm_do, a.dout, a.B, a.T, DH, C::CW, K::TQJ, sw) ||
      !tmap_heads(&P.tm_k, a.kk, a.B, a.T, DH, C::CW, TK, sw) ||
      !tmap_heads(&P.tm_v, a.v, a.B, a.T, DH, C::CW, TK, sw))
    return -1;
  // Under a causal mask the first key tiles have by far the most jobs, and head 0 has the
  // shared stream's too: one CTA per tile would leave most of the grid waiting for a few. Tiles
  // are split over clusters while the grid holds fewer than two items per resident CTA (one
  // where an SM holds a single CTA: nothing then hides a CTA's start and the cluster's sum)
  // and every CTA keeps at least four jobs. 8192 causal tokens at d_h 48: 592 us of backward
  // without the split, 443 with this rule, 472 at twice as much; at d_h 128, 2 x 2048 tokens
  // in a window: 110, 110, 193.
  const int64_t items = (int64_t)a.B * a.G * P.nq;
  const int64_t jobs = (int64_t)(a.k + (a.S > a.G * a.k ? 1 : 0)) * ((a.T + K::TQJ - 1) / K::TQJ);
  P.split = 1;
  while (P.split < kMaxSplit && items * P.split < (C::CTAS == 2 ? 4 : 1) * (int64_t)num_sms &&
         jobs >= 8 * P.split)
    P.split *= 2;
  if (!launch_cluster(attn_scores_dkdv_kernel<DH>, items, K::SMEM, st, P)) return -1;
  return 2;
}

}  // namespace

int launch_attn_scores_backward(const AttnArgs& a, cudaStream_t st) {
  switch (a.d_h) {
    case 16: return launch_dh<16>(a, st);
    case 32: return launch_dh<32>(a, st);
    case 48: return launch_dh<48>(a, st);
    case 64: return launch_dh<64>(a, st);
    case 80: return launch_dh<80>(a, st);
    case 96: return launch_dh<96>(a, st);
    case 112: return launch_dh<112>(a, st);
    case 128: return launch_dh<128>(a, st);
    default: return -1;
  }
}

}  // namespace gqe
