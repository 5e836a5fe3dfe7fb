// Tensor-core (tcgen05) attention of the GQE query streams whose scores may be capped by a
// tanh, biased by the distance of query and key, and masked by an interval of keys per query
// (documents packed in a sequence, bidirectional prefixes, sliding windows, padding); the
// mathematics is in attn_scores.cuh.
//
// One CTA per 128-query tile of a stream, two CTAs per SM for head dims up to 64: while one
// computes exponentials the other's products run. The CTA first reduces its rows' intervals:
// the key tiles outside their union are never loaded, and tiles that every row sees whole
// skip the masks. Per CTA:
//   warp 0     TMA: the Q tile, then K tiles into their own ring;
//   warp 1     owns the TMEM columns; one elected lane issues S = Q K^T (both operands in
//              shared memory) and O += P V with P from TMEM and V as an MN-major operand;
//   warp 2     TMA: V tiles into a second ring;
//   warp 3     cleans the V tiles that some row sees only in part: infinities and NaN in
//              masked places become zeros before the product (0 x NaN would be NaN);
//   warps 4-7  softmax: one query row per thread, 128 scores per tile in registers. Cap and
//              bias are applied to the registers, then exp2 against the running row
//              reference; P goes to TMEM in bf16 (the type of the second product), the row
//              sums stay in 32 bits. O is rescaled in TMEM only when a row's reference moves
//              by more than 2^8.
// The bias of uncapped scores costs the softmax nothing: -slope (t - u) is slope c plus a number
// of the row and the tile (c: the key's place in its tile), and slope c comes from the tensor
// cores as sixteen more columns of the first product: (slope / scale) in three bf16 pieces on
// the query side, (c, c, c) on the key side, exact to 24 bits. Only tiles that hold visible
// keys behind their queries (not under a causal mask) correct the sign in registers.
// A row's reference is -inf until it meets its first key, so rows whose first tiles are
// masked lose nothing when their scores are far below zero.
#include <cudaTypedefs.h>
#include <limits.h>
#include <string.h>

#include "attn_scores.cuh"

namespace gqe {
namespace {

using namespace tc;

constexpr int THREADS = 256;
constexpr int kSmallRegs = 48;   // warpgroup 0 after setmaxnreg.dec (two CTAs per SM)
constexpr int kLargeRegs = 208;  // softmax warpgroup after setmaxnreg.inc
static_assert(kSmallRegs * 128 + kLargeRegs * 128 == THREADS * (65536 / (2 * THREADS)),
              "register split must equal the launch allocation");
constexpr int TQ = 128, TK = 128;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

template <int DH, bool BIAS>
struct Cfg {
  // Chunk width (columns of a swizzle atom); 16-column chunks where the row sums come from
  // the tensor cores, so that the 16 columns of ones after a V tile are one chunk.
  static constexpr int CW = (DH % 64 == 0) ? 64 : (DH % 32 == 0 && DH > 48) ? 32 : 16;
  static constexpr uint32_t LAYOUT =
      CW == 64 ? kSwizzle128B : (CW == 32 ? kSwizzle64B : kSwizzle32B);
  static constexpr int ROW_BYTES = CW * 2;
  static constexpr int CHUNK_BYTES = 128 * ROW_BYTES;
  static constexpr int TILE_BYTES = 128 * DH * 2;
  // Head dims up to 48: a chunk of ones after every V tile makes the product leave sum_j P
  // (32-bit accumulation of the same bf16 weights) in the columns after the head dim.
  static constexpr bool SUM_MMA = DH <= 48;
  static constexpr int ONES_BYTES = SUM_MMA ? CHUNK_BYTES : 0;
  static constexpr int N_PV = DH + (SUM_MMA ? 16 : 0);
  static constexpr int V_BYTES = TILE_BYTES + ONES_BYTES;
  static constexpr int CTAS = DH <= 64 ? 2 : 1;
  static constexpr int TMEM_COLS = CTAS == 2 ? 256 : 512;
  // With a bias its columns of the first product take the place of one K stage where shared
  // memory is short.
  static constexpr int AUG_BYTES = BIAS ? 2 * 128 * 32 : 0;
  static constexpr int K_STAGES = (DH <= 48 ? 4 : 3) - (BIAS && (DH == 48 || DH == 128) ? 1 : 0);
  static constexpr int V_STAGES = DH == 64 ? 2 : 3;
  static constexpr int SMEM =
      TILE_BYTES * (1 + K_STAGES) + V_STAGES * V_BYTES + AUG_BYTES + 1024 + 512;
  static constexpr int P_COL = 128, O_COL = 192;
  static_assert(O_COL + N_PV <= TMEM_COLS, "TMEM budget");
  static_assert(!SUM_MMA || CW == 16, "the ones chunk must be one 16-column chunk");
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory budget");
  static_assert(SMEM <= 227 * 1024, "shared memory of a CTA");
};

// Of every 8 pairs of scores, this many take the FMA-pipe exponential and the rest MUFU's.
constexpr int kFmaPairsOf8 = 3;

struct Params {
  CUtensorMap tm_q, tm_k, tm_v;
  SpanArgs span;
  __nv_bfloat16* out;
  int64_t out_hs, out_ts, last_off;
  const __nv_bfloat16* v;  // for the rare rows that see an infinity or NaN
  int64_t v_hs, v_ts;
  float* lse;
  const float* psel;
  int psel_stride, psel_off;
  const float* slopes;
  int T, B, S, Sr, k, nq;
  float scale_log2;  // scale log2(e), of uncapped scores
  float inv_scale;
  CapForm cap;
  int32_t* status;
  int64_t spin;
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const Params& P,
                                          volatile int* abort_flag) {
  const bool ok = !__any_sync(0xffffffffu, !mbar_wait(bar, parity, P.spin));
  if (!ok && (threadIdx.x & 31) == 0) {
    *abort_flag = 1;
    atomicExch(P.status, kStatusTimeout);
  }
  return ok;
}
__device__ __forceinline__ bool lane_wait(uint64_t* bar, uint32_t parity, const Params& P,
                                          volatile int* abort_flag) {
  if (mbar_wait(bar, parity, P.spin)) return true;
  *abort_flag = 1;
  atomicExch(P.status, kStatusTimeout);
  return false;
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Largest of 64 scores s[0..63]; NaN if one of them is.
__device__ __forceinline__ float max64(const float* s) {
  float mp[8];
#pragma unroll
  for (int x = 0; x < 8; ++x) mp[x] = max3_nan(s[x], s[8 + x], s[16 + x]);
#pragma unroll
  for (int c = 24; c < 56; c += 16)
#pragma unroll
    for (int x = 0; x < 8; ++x) mp[x] = max3_nan(mp[x], s[c + x], s[c + 8 + x]);
#pragma unroll
  for (int x = 0; x < 8; ++x) mp[x] = max_nan(mp[x], s[56 + x]);
  return max_nan(max3_nan(mp[0], mp[1], mp[2]),
                 max3_nan(max3_nan(mp[3], mp[4], mp[5]), mp[6], mp[7]));
}

template <int DH, bool BIAS>
__global__ void __launch_bounds__(THREADS, Cfg<DH, BIAS>::CTAS)
attn_scores_kernel(const __grid_constant__ Params P) {
  using C = Cfg<DH, BIAS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = smem + C::TILE_BYTES;
  uint8_t* sV = sK + C::K_STAGES * C::TILE_BYTES;
  uint8_t* sAug = sV + C::V_STAGES * C::V_BYTES;  // bias columns: query side, key side
  uint64_t* bar = reinterpret_cast<uint64_t*>(sAug + C::AUG_BYTES);
  uint64_t* q_full = bar;
  uint64_t* k_full = bar + 1;
  uint64_t* k_empty = k_full + C::K_STAGES;
  uint64_t* v_full = k_empty + C::K_STAGES;
  uint64_t* v_empty = v_full + C::V_STAGES;
  uint64_t* v_clean = v_empty + C::V_STAGES;
  uint64_t* s_full = v_clean + C::V_STAGES;
  uint64_t* s_free = s_full + 1;
  uint64_t* p_ready = s_free + 1;
  uint64_t* pv_done = p_ready + 1;
  uint64_t* o_full = pv_done + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(o_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile int* bad_flag = abort_flag + 1;
  int* sp = reinterpret_cast<int*>(tmem_holder + 4);  // [4][4] the warps' interval bounds

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int bs = P.B * P.S;
  // last query tiles first: under a causal mask they have the most keys
  const int qt = P.nq - 1 - blockIdx.x / bs;
  const int s_idx = blockIdx.x % bs % P.S, b_idx = blockIdx.x % bs / P.S;
  if constexpr (C::SUM_MMA) {
    for (int st = 0; st < C::V_STAGES; ++st) {
      uint4* o = reinterpret_cast<uint4*>(sV + st * C::V_BYTES + C::TILE_BYTES);
      for (int i = threadIdx.x; i < C::ONES_BYTES / 16; i += THREADS)
        o[i] = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
    }
    fence_async_shared();
  }
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < C::K_STAGES; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < C::V_STAGES; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 2);  // the product that read it, and the cleaning warp
      mbar_init(&v_clean[s], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_free, 4);
    mbar_init(p_ready, 4);
    mbar_init(pv_done, 1);
    mbar_init(o_full, 1);
    *abort_flag = 0;
    *bad_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, C::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&P.tm_q);
    prefetch_tmap(&P.tm_k);
    prefetch_tmap(&P.tm_v);
  }
  pdl_wait();  // the inputs are complete from here on
  pdl_allow_next();
  const float slope = BIAS ? P.slopes[s_idx] : 0.f;
  if constexpr (BIAS) {
    // rows of 32 bytes in the 32-byte swizzle: the halves of rows 4..7 of every 8 change places
    if (!P.cap.on) {
      const bool keys = threadIdx.x >= 128;
      const int rr = threadIdx.x & 127;
      const float a = keys ? (float)rr : slope * P.inv_scale;
      const float hi = __bfloat162float(__float2bfloat16_rn(a));
      const float mid = keys ? a : __bfloat162float(__float2bfloat16_rn(a - hi));
      const float lo = keys ? a : a - hi - mid;
      uint8_t* at = sAug + (keys ? 4096 : 0) + rr * 32;
      const int first = (rr >> 2) & 1;
      *reinterpret_cast<uint4*>(at + first * 16) =
          make_uint4(pack_bf16x2(hi, mid), pack_bf16x2(lo, 0.f), 0u, 0u);
      *reinterpret_cast<uint4*>(at + (first ^ 1) * 16) = make_uint4(0u, 0u, 0u, 0u);
      fence_async_shared();
    }
  }
  const int row = threadIdx.x & 127;
  const int q = qt * TQ + row;  // a softmax thread's query
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
  // tiles inside [full_lo, full_hi) are seen whole by every row that sees anything
  const int full_lo = max(max(sp[2], sp[6]), max(sp[10], sp[14]));
  const int full_hi = min(min(sp[3], sp[7]), min(sp[11], sp[15]));
  const int j0 = lo < hi ? lo / TK : 0;
  const int nk = lo < hi ? (hi + TK - 1) / TK - j0 : 0;  // key tiles j0 .. j0 + nk - 1
  // The order of the key tiles: with a bias from the nearest on, since weights fall with the
  // distance and the row references then hardly move after the first tile.
  auto tile = [&](int j) { return BIAS ? j0 + nk - 1 - j : j0 + j; };
  auto whole = [&](int j) { return j * TK >= full_lo && (j + 1) * TK <= full_hi; };
  const int kvh = s_idx < P.Sr ? s_idx / P.k : 0;

  if (warp < 4) {
    if constexpr (C::CTAS == 2) setmaxnreg_dec<kSmallRegs>();
    if (warp == 0) {
      // -------------------------------------------------------------- Q and K loads
      if (lane == 0 && nk > 0) {
        mbar_arrive_expect_tx(q_full, C::TILE_BYTES);
        tma_load_5d(sQ, &P.tm_q, 0, qt * TQ, 0, s_idx, b_idx, q_full);
        int st = 0, j = 0;
        uint32_t ph = 0;
        for (; j < nk; ++j) {
          if (!lane_wait(&k_empty[st], ph ^ 1, P, abort_flag)) break;
          mbar_arrive_expect_tx(&k_full[st], C::TILE_BYTES);
          tma_load_5d(sK + st * C::TILE_BYTES, &P.tm_k, 0, tile(j) * TK, 0, kvh, b_idx,
                      &k_full[st]);
          if (++st == C::K_STAGES) {
            st = 0;
            ph ^= 1;
          }
        }
        drain_ring(q_full, 1, 1);
        drain_ring(k_full, C::K_STAGES, j);
      }
    } else if (warp == 2) {
      // -------------------------------------------------------------- V loads
      if (lane == 0) {
        int st = 0, j = 0;
        uint32_t ph = 0;
        for (; j < nk; ++j) {
          if (!lane_wait(&v_empty[st], ph ^ 1, P, abort_flag)) break;
          mbar_arrive_expect_tx(&v_full[st], C::TILE_BYTES);
          tma_load_5d(sV + st * C::V_BYTES, &P.tm_v, 0, tile(j) * TK, 0, kvh, b_idx,
                      &v_full[st]);
          if (++st == C::V_STAGES) {
            st = 0;
            ph ^= 1;
          }
        }
        drain_ring(v_full, C::V_STAGES, j);
      }
    } else if (warp == 3) {
      // -------------------------------------------------------------- cleaning of V tiles
      int st = 0;
      uint32_t ph = 0;
      for (int j = 0; j < nk; ++j) {
        if (!warp_wait(&v_full[st], ph, P, abort_flag)) break;
        if (!whole(tile(j))) {
          if (clean_tile(sV + st * C::V_BYTES, C::TILE_BYTES)) {
            fence_async_shared();
            if (lane == 0) *bad_flag = 1;
            __threadfence_block();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_clean[st]);
        }
        // every tile passes here, so this warp is never a phase of a stage behind or ahead
        if (lane == 0) mbar_arrive(&v_empty[st]);
        if (++st == C::V_STAGES) {
          st = 0;
          ph ^= 1;
        }
      }
    } else {
      // -------------------------------------------------------------- MMA issue
      const uint32_t idesc_s = idesc_bf16_f32(TQ, TK);
      const uint32_t idesc_pv = idesc_bf16_f32(TQ, C::N_PV) | (1u << 16);  // B (V) MN-major
      const uint64_t q_desc = smem_desc(smem_u32(sQ), 8 * C::ROW_BYTES, C::LAYOUT);
      const uint64_t k_desc = smem_desc(smem_u32(sK), 8 * C::ROW_BYTES, C::LAYOUT);
      const uint64_t v_desc =
          smem_desc_mn(smem_u32(sV), C::CHUNK_BYTES, 8 * C::ROW_BYTES, C::LAYOUT);
      constexpr uint32_t kKStep = C::TILE_BYTES >> 4;
      constexpr uint32_t kVStep = C::V_BYTES >> 4;
      int kst = 0, vst = 0;
      uint32_t k_phase = 0, v_phase = 0, clean_phase = 0;  // clean_phase: a bit per stage
      uint32_t n_sf = 0;
      auto issue_s = [&]() -> bool {
        if (!warp_wait(&k_full[kst], k_phase, P, abort_flag)) return false;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t kd = k_desc + (uint64_t)(kst * kKStep);
#pragma unroll
          for (int kk = 0; kk < DH / 16; ++kk) {
            const uint32_t o =
                (((kk * 16) / C::CW) * C::CHUNK_BYTES + ((kk * 16) % C::CW) * 2) >> 4;
            mma_ss(tmem, q_desc + o, kd + o, idesc_s, kk > 0 ? 1u : 0u);
          }
          if constexpr (BIAS)
            if (!P.cap.on)
              mma_ss(tmem, smem_desc(smem_u32(sAug), 256, kSwizzle32B),
                     smem_desc(smem_u32(sAug + 4096), 256, kSwizzle32B), idesc_s, 1u);
          mma_commit(s_full);
          mma_commit(&k_empty[kst]);
        }
        __syncwarp();
        if (++kst == C::K_STAGES) {
          kst = 0;
          k_phase ^= 1;
        }
        return true;
      };
      bool ok = nk > 0 && warp_wait(q_full, 0, P, abort_flag) && issue_s();  // S(0)
      if (ok && nk > 1) {
        ok = warp_wait(s_free, n_sf & 1, P, abort_flag) && issue_s();  // S(1)
        ++n_sf;
      }
      // then for every tile j, once P(j) is ready, P(j) V and S(j + 2)
      for (int j = 0; ok && j < nk; ++j) {
        if (!warp_wait(p_ready, j & 1, P, abort_flag)) break;
        if (!warp_wait(&v_full[vst], v_phase, P, abort_flag)) break;
        if (!whole(tile(j))) {
          if (!warp_wait(&v_clean[vst], (clean_phase >> vst) & 1, P, abort_flag)) break;
          clean_phase ^= 1u << vst;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint64_t vd = v_desc + (uint64_t)(vst * kVStep);
#pragma unroll
          for (int kk = 0; kk < TK / 16; ++kk)
            mma_ts(tmem + C::O_COL, tmem + C::P_COL + kk * 8,
                   vd + (uint64_t)((kk * 16 * C::ROW_BYTES) >> 4), idesc_pv,
                   (j == 0 && kk == 0) ? 0u : 1u);
          mma_commit(pv_done);
          if (j + 1 == nk) mma_commit(o_full);
          mma_commit(&v_empty[vst]);
        }
        __syncwarp();
        if (j + 2 < nk) {
          if (!warp_wait(s_free, n_sf & 1, P, abort_flag)) break;
          ++n_sf;
          if (!issue_s()) break;
        }
        if (++vst == C::V_STAGES) {
          vst = 0;
          v_phase ^= 1;
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax + epilogue
    if constexpr (C::CTAS == 2) setmaxnreg_inc<kLargeRegs>();
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_off;
    const uint32_t t_p = tmem + lane_off + C::P_COL;
    const uint32_t t_o = tmem + lane_off + C::O_COL;
    const float slope2 = slope * kLog2e;
    const int q0 = qt * TQ;
    const bool live = b0 < e0;
    float m_used = -INFINITY, l = 0.f;
    bool ok = true;
    by_flag(P.cap.on, [&](auto cap) {
      constexpr bool CAP = decltype(cap)::value;
      // a score in log2 units is (tanh of) the product times in, plus the bias
      const float in = CAP ? P.cap.log2 : P.scale_log2;
      // what is still to be multiplied after the registers' pass
      const float cs = CAP && BIAS ? 1.f : in;
      for (int j = 0; j < nk; ++j) {
        if (!warp_wait(s_full, j & 1, P, abort_flag)) { ok = false; break; }
        tc_fence_after();
        float s[TK];
        {
          uint32_t r[TK];
          tmem_ld128_wait(t_s, r);
#pragma unroll
          for (int c = 0; c < TK; ++c) s[c] = __uint_as_float(r[c]);
        }
        if (j + 1 < nk) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_free);
        }
        const int kv0 = tile(j) * TK;
        if constexpr (CAP) {
          by_flag(!__any_sync(0xffffffffu, !(abs_max<TK>(s) < P.cap.limit)), [&](auto poly) {
#pragma unroll
            for (int c = 0; c < TK; c += 2) {
              const float2 th =
                  cap_tanh<decltype(poly)::value>(P.cap, make_float2(s[c], s[c + 1]));
              s[c] = th.x;
              s[c + 1] = th.y;
            }
          });
        }
        if constexpr (CAP && BIAS) {
          if (kv0 + TK - 1 <= q0) {
            // every key at or before every query: the distance is linear (four chains of
            // additions, eight columns a step: packed constants would have to be moved in)
            const float base = (float)(kv0 - q) * slope2;
            const float2 in2 = make_float2(in, in), step = make_float2(8.f * slope2, 8.f * slope2);
            float2 chain[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              chain[i] = make_float2(fmaf(slope2, (float)(2 * i), base),
                                     fmaf(slope2, (float)(2 * i + 1), base));
#pragma unroll
            for (int c = 0; c < TK; c += 2) {
              const float2 z = fma2(make_float2(s[c], s[c + 1]), in2, chain[(c >> 1) & 3]);
              chain[(c >> 1) & 3] = add2(chain[(c >> 1) & 3], step);
              s[c] = z.x;
              s[c + 1] = z.y;
            }
          } else {
            const float d0 = (float)(kv0 - q);
#pragma unroll
            for (int c = 0; c < TK; ++c) s[c] = fmaf(s[c], in, -slope2 * fabsf(d0 + (float)c));
          }
        }
        // uncapped: the products hold slope c; keys behind the query turn its sign
        const float base = BIAS && !CAP ? (float)(kv0 - q) * slope2 : 0.f;
        if constexpr (BIAS && !CAP) {
          if (!P.span.causal && kv0 + TK - 1 > q0) {
            const float d0 = (float)(kv0 - q), a2 = -2.f * slope * P.inv_scale;
#pragma unroll
            for (int c = 0; c < TK; ++c) s[c] = fmaf(a2, fmaxf(d0 + (float)c, 0.f), s[c]);
          }
        }
        // masks, each side only where some row has it inside the tile
        if (kv0 < full_lo) {
          const int first = live ? b0 - kv0 : TK;
#pragma unroll
          for (int c = 0; c < TK; ++c) s[c] = c < first ? -INFINITY : s[c];
        }
        if (kv0 + TK > full_hi) {
          const int last = live ? e0 - kv0 : 0;
#pragma unroll
          for (int c = 0; c < TK; ++c) s[c] = c >= last ? -INFINITY : s[c];
        }
        // Row maximum in two halves: the exponentials of the first need only its own maximum
        // and the running reference, so the second half's maximum is formed while they run. A
        // reference moves only when a maximum passes it by more than the threshold; if the
        // second half's does, the first half's P is rescaled.
        const float m_old = m_used;
        uint32_t pk[TK / 2];
        float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        auto half = [&](auto hc) {
          constexpr int H = decltype(hc)::value, C0 = 64 * H;
          const float m = fmaf(max64(s + C0), cs, base);
          // A NaN score moves the reference too: the half's weights become NaN, and with them the
          // row's sum, before a larger reference could scale a mark of it away.
          if (!(m <= m_used + kRescaleThreshold)) {
            if constexpr (H == 1) {
              // a first half without keys holds only zeros: the factor is then 0
              const float a2 = ex2(m_used - m);
#pragma unroll
              for (int x = 0; x < TK / 4; ++x)
                pk[x] = pack_bf16x2(__uint_as_float(pk[x] << 16) * a2,
                                    __uint_as_float(pk[x] & 0xffff0000u) * a2);
              if constexpr (!C::SUM_MMA) {
                ls[0] = mul2(ls[0], make_float2(a2, a2));
                ls[1] = mul2(ls[1], make_float2(a2, a2));
              }
            }
            m_used = m;
          }
          const float ref = m_used == -INFINITY ? 0.f : m_used;
          const float2 cs2 = make_float2(cs, cs), nm2 = make_float2(base - ref, base - ref);
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            const float2 v = make_float2(s[C0 + 2 * x], s[C0 + 2 * x + 1]);
            const float2 t = CAP && BIAS ? add2(v, nm2) : fma2(v, cs2, nm2);
            const float2 p = (x & 7) >= 8 - kFmaPairsOf8 ? exp2_fma2_nan(t)
                                                         : make_float2(ex2(t.x), ex2(t.y));
            if constexpr (!C::SUM_MMA) ls[x & 1] = add2(ls[x & 1], p);
            pk[32 * H + x] = pack_bf16x2(p.x, p.y);
          }
        };
        half(std::integral_constant<int, 0>{});
        half(std::integral_constant<int, 1>{});
        const bool need = j > 0 && m_used != m_old;
        const float alpha = need ? ex2(m_old - m_used) : 1.f;  // 0 from a reference of -inf
        if constexpr (!C::SUM_MMA) {
          const float2 a = add2(ls[0], ls[1]);
          l = l * alpha + (a.x + a.y);
        }
        if (j > 0 && !warp_wait(pv_done, (j - 1) & 1, P, abort_flag)) { ok = false; break; }
        if (__any_sync(0xffffffffu, need)) {
          tc_fence_after();
#pragma unroll
          for (int c0 = 0; c0 < C::N_PV; c0 += 16) {
            uint32_t r[16];
            tmem_ld16_wait(t_o + c0, r);
#pragma unroll
            for (int x = 0; x < 16; ++x) r[x] = __float_as_uint(__uint_as_float(r[x]) * alpha);
            tmem_st16(t_o + c0, r);
          }
        }
#pragma unroll
        for (int c0 = 0; c0 < TK / 2; c0 += 16) {
          uint32_t r[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) r[x] = pk[c0 + x];
          tmem_st16(t_p + c0, r);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready);
      }
    });
    // ---- epilogue: O / l into the output row
    if (ok && nk > 0) ok = warp_wait(o_full, 0, P, abort_flag);
    if (ok) {
      tc_fence_after();
      const bool valid = q < P.T;
      const int64_t tok = (int64_t)b_idx * P.T + q;
      if constexpr (C::SUM_MMA) {
        if (nk > 0) {
          uint32_t r[16];
          tmem_ld16_wait(t_o + DH, r);
          l = __uint_as_float(r[0]);
        }
      }
      // The largest score's weight is near 1 (as near as its float32 is to the reference) and none
      // is far above 2^8. A sum of 1e30 comes from NaN weights through the FMA-pipe exponential
      // (the largest float, infinity in bf16), one below 1e-30 from scores that are all -infinity
      // (5e-42 each): the whole row and its log-sum-exp are NaN.
      if (!(l > 1e-30f && l < 1e30f)) l = __int_as_float(0x7fffffff);
      float scale = live ? 1.f / l : 0.f;
      if (valid && P.lse)
        P.lse[(int64_t)s_idx * P.B * P.T + tok] = live ? m_used + __log2f(l) : -INFINITY;
      if (P.psel && live && s_idx < P.Sr)
        scale *= P.psel[tok * P.psel_stride + P.psel_off + s_idx];
      // A cleaned V tile hides the infinities and NaN that a row does see: those columns of
      // the row become NaN (rare; whole tiles are not cleaned and carry theirs themselves).
      uint32_t nan_cols[4] = {0u, 0u, 0u, 0u};
      if (*bad_flag && valid && live) {
        for (int j = 0; j < nk; ++j) {
          if (whole(j0 + j)) continue;
          const int u1 = min(e0, (j0 + j + 1) * TK);
          for (int u = max(b0, (j0 + j) * TK); u < u1; ++u) {
            const uint32_t* vr = reinterpret_cast<const uint32_t*>(
                P.v + (int64_t)kvh * P.v_hs + ((int64_t)b_idx * P.T + u) * P.v_ts);
#pragma unroll
            for (int c = 0; c < DH / 2; ++c) {
              const uint32_t w = vr[c];
              if ((w & 0x7f80u) == 0x7f80u) nan_cols[c / 16] |= 1u << (2 * c % 32);
              if ((w & 0x7f800000u) == 0x7f800000u) nan_cols[c / 16] |= 2u << (2 * c % 32);
            }
          }
        }
      }
      const bool any_nan = (nan_cols[0] | nan_cols[1] | nan_cols[2] | nan_cols[3]) != 0u;
      const int64_t head =
          s_idx == P.S - 1 && P.last_off >= 0 ? P.last_off : (int64_t)s_idx * P.out_hs;
      __nv_bfloat16* dst = P.out + head + tok * P.out_ts;
#pragma unroll
      for (int c0 = 0; c0 < DH; c0 += 16) {
        uint32_t r[16];
        if (nk > 0) {
          tmem_ld16_wait(t_o + c0, r);
        }
        if (valid) {
          uint32_t w[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            float lo_v = live ? __uint_as_float(r[2 * x]) * scale : 0.f;
            float hi_v = live ? __uint_as_float(r[2 * x + 1]) * scale : 0.f;
            if (any_nan) {
              const uint32_t bits = nan_cols[(c0 + 2 * x) / 32] >> ((c0 + 2 * x) % 32);
              if (bits & 1u) lo_v = __int_as_float(0x7fffffff);
              if (bits & 2u) hi_v = __int_as_float(0x7fffffff);
            }
            w[x] = pack_bf16x2(lo_v, hi_v);
          }
          *reinterpret_cast<uint4*>(dst + c0) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(dst + c0 + 8) = make_uint4(w[4], w[5], w[6], w[7]);
        }
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

template <int DH, bool BIAS>
int launch_form(const AttnArgs& a, cudaStream_t st) {
  using C = Cfg<DH, BIAS>;
  if (!set_smem_limit_once<attn_scores_kernel<DH, BIAS>>(C::SMEM)) return -1;
  Params P;
  memset(&P, 0, sizeof(P));
  const CUtensorMapSwizzle sw = C::CW == 64 ? CU_TENSOR_MAP_SWIZZLE_128B
                                : C::CW == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                              : CU_TENSOR_MAP_SWIZZLE_32B;
  if (!tmap_heads(&P.tm_q, a.q, a.B, a.T, DH, C::CW, TQ, sw) ||
      !tmap_heads(&P.tm_k, a.kk, a.B, a.T, DH, C::CW, TK, sw) ||
      !tmap_heads(&P.tm_v, a.v, a.B, a.T, DH, C::CW, TK, sw))
    return -1;
  P.span = SpanArgs{a.key_begin, a.key_end, a.T, a.causal};
  P.out = static_cast<__nv_bfloat16*>(a.out.data);
  P.out_hs = a.out.head_stride;
  P.out_ts = a.out.token_stride;
  P.last_off = a.last_off;
  P.v = static_cast<const __nv_bfloat16*>(a.v.data);
  P.v_hs = a.v.head_stride;
  P.v_ts = a.v.token_stride;
  P.lse = a.lse;
  P.psel = a.psel;
  P.psel_stride = a.psel_stride;
  P.psel_off = a.psel_off;
  P.slopes = a.slopes;
  P.T = a.T;
  P.B = a.B;
  P.S = a.S;
  P.Sr = a.G * a.k;
  P.k = a.k;
  P.nq = (a.T + TQ - 1) / TQ;
  P.scale_log2 = a.scale * kLog2e;
  P.inv_scale = 1.f / a.scale;
  P.cap = cap_form(a.scale, a.softcap);
  P.status = a.status;
  P.spin = a.spin > 0 ? a.spin : (int64_t)1 << 22;
  const int64_t items = (int64_t)a.B * a.S * P.nq;
  return launch_pdl(attn_scores_kernel<DH, BIAS>, dim3((unsigned)items), dim3(THREADS), C::SMEM,
                    st, P) == cudaSuccess
             ? 1
             : -1;
}

template <int DH>
int launch_dh(const AttnArgs& a, cudaStream_t st) {
  return a.slopes ? launch_form<DH, true>(a, st) : launch_form<DH, false>(a, st);
}

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

bool encoder() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    cudaGetLastError();
  });
  return g_encode != nullptr;
}

}  // namespace

bool tmap_heads(CUtensorMap* m, const QkTensor& t, int B, int T, int d_h, int cw, int box_rows,
                CUtensorMapSwizzle sw) {
  if (!encoder()) return false;
  const cuuint64_t row = (cuuint64_t)t.token_stride * 2;
  cuuint64_t dims[5] = {(cuuint64_t)cw, (cuuint64_t)T, (cuuint64_t)(d_h / cw),
                        (cuuint64_t)t.heads, (cuuint64_t)B};
  cuuint64_t strides[4] = {row, (cuuint64_t)cw * 2, (cuuint64_t)t.head_stride * 2,
                           row * (cuuint64_t)T};
  cuuint32_t box[5] = {(cuuint32_t)cw, (cuuint32_t)box_rows, (cuuint32_t)(d_h / cw), 1, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, t.data, dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int launch_attn_scores(const AttnArgs& a, cudaStream_t st) {
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
