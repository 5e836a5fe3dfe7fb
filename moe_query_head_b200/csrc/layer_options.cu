// The layer with options: the norm and rotation of its queries and keys between the
// projections and the attention, and capped, biased and masked scores in the attention, its
// backward pass and its decode step. The kernels are the operators' (qk_norm_rope.cu,
// attn_scores*.cu), here on the handle's buffers: outputs go to their blocks of Z, query
// gradients to the column blocks of the experts that projected them.
#include <string.h>

#include "attn_scores.cuh"
#include "attn_scores_decode.cuh"
#include "layer_options.cuh"
#include "scores_api.cuh"

namespace gqe {
namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

QkTensor tensor(void* data, int heads, int64_t head_stride, int64_t token_stride) {
  QkTensor t;
  t.data = data;
  t.heads = heads;
  t.head_stride = head_stride;
  t.token_stride = token_stride;
  return t;
}

// The handle's sizes, scores and stream tensors; q and k as the attention reads them.
AttnArgs attn_args(gqe_ctx* h, int B, int T, int S, int causal) {
  const LayerOptions& o = options(h);
  const int64_t M = (int64_t)B * T;
  const int d = h->d_h, Gl = h->g1 - h->g0;
  AttnArgs a;
  a.B = B;
  a.T = T;
  a.S = S;
  a.G = Gl;
  a.k = h->k;
  a.d_h = d;
  a.causal = causal;
  a.scale = o.scale > 0.f ? o.scale : 1.f / sqrtf((float)d);
  if (o.scores) {
    a.softcap = o.softcap;
    a.slopes = o.slopes;
    a.key_begin = o.key_begin;
    a.key_end = o.key_end;
  }
  a.q = tensor(o.transform ? o.q_t : h->ws.Q, S, M * d, d);
  a.kk = tensor(o.transform ? o.k_t : h->ws.K, Gl, M * d, d);
  a.v = tensor(h->ws.V, Gl, M * d, d);
  a.lse = h->ws.lse;
  a.status = h->ws.status;
  a.spin = h->spin_limit;
  return a;
}

QkArgs transform_of(gqe_ctx* h, int64_t M, int period, int S) {
  const LayerOptions& o = options(h);
  QkArgs A = transform_args(o.tr);
  const int d = h->d_h, Gl = h->g1 - h->g0;
  A.q = tensor(h->ws.Q, S, M * d, d);
  A.k = tensor(h->ws.K, Gl, M * d, d);
  A.positions = o.positions;
  A.period = period;
  A.M = M;
  return A;
}

}  // namespace

gqe_status layer_options_alloc(gqe_ctx* h) {
  LayerOptions& o = options(h);
  const size_t rows = (size_t)h->max_tokens * h->d_h * h->esz;
  const size_t q_bytes = align_up(((size_t)h->G * h->k + 1) * rows);
  const size_t k_bytes = align_up((size_t)h->G * rows);
  if (o.transform && !o.fwd_base) {
    if (cudaMalloc(&o.fwd_base, q_bytes + k_bytes) != cudaSuccess) {
      cudaGetLastError();
      o.fwd_base = nullptr;
      return GQE_ERR_CUDA;
    }
    o.q_t = o.fwd_base;
    o.k_t = static_cast<char*>(o.fwd_base) + q_bytes;
  }
  if (h->bwd_base && (o.transform || o.scores) && !o.bwd_base) {
    const size_t part = align_up((size_t)kQkPartialRows * h->d_h * 4);
    const size_t blocks = align_up((size_t)h->max_tokens * sizeof(int2));
    if (cudaMalloc(&o.bwd_base, q_bytes + k_bytes + part + blocks) != cudaSuccess) {
      cudaGetLastError();
      o.bwd_base = nullptr;
      return GQE_ERR_CUDA;
    }
    char* p = static_cast<char*>(o.bwd_base);
    o.dq_t = p;
    o.dk_t = p + q_bytes;
    o.partial = reinterpret_cast<float*>(p + q_bytes + k_bytes);
    o.blocks = reinterpret_cast<int2*>(p + q_bytes + k_bytes + part);
  }
  return GQE_OK;
}

void layer_options_release(gqe_ctx* h) {
  LayerOptions& o = options(h);
  if (o.fwd_base) cudaFree(o.fwd_base);
  if (o.bwd_base) cudaFree(o.bwd_base);
  o.fwd_base = o.bwd_base = nullptr;
}

int launch_layer_attention(gqe_ctx* h, int B, int T, int S, int has_shared, int variant,
                           int causal, int Do, cudaStream_t st) {
  const LayerOptions& o = options(h);
  const int d = h->d_h;
  int n = 0;
  if (o.transform) {
    QkArgs A = transform_of(h, (int64_t)B * T, T, S);
    A.q_out = A.q;
    A.k_out = A.k;
    if (h->dtype == GQE_BF16) {  // float32 handles have no backward: in place
      A.q_out.data = o.q_t;
      A.k_out.data = o.k_t;
    }
    n = launch_qk_forward(A, h->num_sms, false, st);
    if (n < 0) return -1;
  }
  if (h->dtype != GQE_BF16) {
    const int m = launch_simt_attention(h, B, T, S, has_shared, variant, causal, Do, st);
    return m < 0 ? -1 : n + m;
  }
  AttnArgs a = attn_args(h, B, T, S, causal);
  const int Sr = a.G * h->k;
  a.out = tensor(h->ws.Z, S, d, Do);
  if (has_shared) a.last_off = (int64_t)(Sr + (variant == GQE_VARIANT_GQE ? 1 : 0)) * d;
  if (variant == GQE_VARIANT_WEIGHTED_CONCAT) {
    a.psel = h->ws.psel;
    a.psel_stride = h->G * h->k;
    a.psel_off = h->g0 * h->k;
  }
  const int m = launch_attn_scores(a, st);
  return m < 0 ? -1 : n + m;
}

int launch_layer_decode(gqe_ctx* h, int B, int S, int has_shared, int variant, int Do,
                        void* k_cache, void* v_cache, int L_max, const int32_t* lengths,
                        cudaStream_t st) {
  const LayerOptions& o = options(h);
  const int d = h->d_h, Gl = h->g1 - h->g0, Sr = Gl * h->k;
  const int64_t seq = (int64_t)L_max * d;
  // the new tokens: queries turned in place, keys and values into the caches
  QkArgs A = transform_of(h, B, 1, S);
  if (!o.transform) {
    A.d_h = d;
    A.dtype = h->dtype;
  }
  A.v = tensor(h->ws.V, Gl, (int64_t)B * d, d);
  A.q_out = A.q;
  A.k_out = tensor(k_cache, Gl, B * seq, seq);
  A.v_out = tensor(v_cache, Gl, B * seq, seq);
  A.positions = lengths;
  A.L_max = L_max;
  A.status = h->ws.status;
  A.idle_ok = 0;
  const int n = launch_qk_forward(A, h->num_sms, true, st);
  if (n < 0) return -1;
  DecodeArgs P;
  P.q = A.q;
  P.out = tensor(h->ws.Z, S, d, Do);
  P.kc = A.k_out;
  P.vc = A.v_out;
  P.lengths = lengths;
  P.key_begin = o.scores ? o.key_begin : nullptr;
  P.slopes = o.scores ? o.slopes : nullptr;
  if (variant == GQE_VARIANT_WEIGHTED_CONCAT) {
    P.psel = h->ws.psel;
    P.psel_stride = h->G * h->k;
    P.psel_off = h->g0 * h->k;
  }
  if (has_shared) P.last_off = (int64_t)(Sr + (variant == GQE_VARIANT_GQE ? 1 : 0)) * d;
  P.part = h->ws.dec_part;
  P.status = h->ws.status;
  P.B = B;
  P.S = S;
  P.G = Gl;
  P.k = h->k;
  P.d_h = d;
  P.L_max = L_max;
  attn_decode_plan(B, Gl, L_max, h->num_sms, P.nc, P.np);
  while (P.np > 1 && (int64_t)B * Gl * P.np > kDecodeSlots) --P.np;  // the handle's slots
  set_decode_scores(P, o.scale, o.scores ? o.softcap : 0.f);
  const int m = launch_attn_decode(P, st);
  return m < 0 ? -1 : n + m;
}

int launch_layer_attention_backward(gqe_ctx* h, const BwdBuffers& bb, int B, int T, int S,
                                    int has_shared, int causal, cudaStream_t st) {
  (void)has_shared;
  const LayerOptions& o = options(h);
  if (!o.bwd_base) return -1;  // gqe_enable_backward could not allocate it
  const int64_t M = (int64_t)B * T;
  const int d = h->d_h, Gl = h->g1 - h->g0;
  AttnArgs a = attn_args(h, B, T, S, causal);
  a.dout = tensor(bb.dO, S, M * d, d);
  a.out = a.dout;  // not read: D is given
  a.dsum = bb.dsum;
  a.dsum_given = 1;
  a.blocks = o.blocks;
  const QkTensor dk = tensor(bb.dk, Gl, d, (int64_t)Gl * d);
  a.dv = tensor(bb.dv, Gl, d, (int64_t)Gl * d);
  const int64_t dq_row = (int64_t)Gl * h->E * d;
  if (o.transform) {
    a.dq = tensor(o.dq_t, S, M * d, d);
    a.dk = tensor(o.dk_t, Gl, M * d, d);
  } else {
    a.dq = tensor(bb.dq_exp, S, 0, dq_row);
    a.dk = dk;
    a.sel = h->ws.sel;
    a.dq_shared = bb.dq_sh;
    a.sel_stride = h->G * h->k;
    a.sel_off = h->g0 * h->k;
    a.experts = h->E;
  }
  const int n = launch_attn_scores_backward(a, st);
  if (n < 0 || !o.transform) return n;
  QkArgs A = transform_of(h, M, T, S);
  A.q_out = a.dq;
  A.k_out = a.dk;
  A.dq = tensor(bb.dq_exp, S, 0, dq_row);
  A.dk = dk;
  A.sel = h->ws.sel;
  A.dq_shared = bb.dq_sh;
  A.sel_stride = h->G * h->k;
  A.sel_off = h->g0 * h->k;
  A.routed = Gl * h->k;
  A.top_k = h->k;
  A.experts = h->E;
  if (o.tr.norm && (o.dq_weight || o.dk_weight)) {
    A.partial = o.partial;
    A.dq_weight = o.dq_weight;
    A.dk_weight = o.dk_weight;
  } else {
    float* w[] = {o.dq_weight, o.dk_weight};  // no norm, no gradient
    for (float* p : w)
      if (p && cudaMemsetAsync(p, 0, (size_t)d * 4, st) != cudaSuccess) return -1;
  }
  const int m = launch_qk_backward(A, h->num_sms, st);
  return m < 0 ? -1 : n + m;
}

}  // namespace gqe

using namespace gqe;

extern "C" {

gqe_status gqe_set_qk_transform(gqe_handle h, const gqe_qk_transform* tr,
                                const int32_t* positions, float* dq_weight, float* dk_weight) {
  if (!h) return GQE_ERR_INVALID_ARG;
  LayerOptions& o = options(h);
  if (!tr) {
    if (o.transform) ++o.generation;
    o.transform = false;
    o.tr = {};
    o.positions = nullptr;
    o.dq_weight = o.dk_weight = nullptr;
    return GQE_OK;
  }
  const gqe_status r = check_transform(tr);
  if (r != GQE_OK) return r;
  if (tr->d_h != h->d_h || tr->dtype != h->dtype) return GQE_ERR_INVALID_ARG;
  const void* ptrs[] = {positions, dq_weight, dk_weight};
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return GQE_ERR_INVALID_ARG;
  if (dq_weight && dq_weight == dk_weight) return GQE_ERR_INVALID_ARG;  // two sums, one place
  const gqe_qk_transform& t = o.tr;
  const bool same = o.transform && t.norm == tr->norm && t.eps == tr->eps &&
                    t.q_weight == tr->q_weight && t.k_weight == tr->k_weight &&
                    t.rot_dim == tr->rot_dim && t.interleaved == tr->interleaved &&
                    t.inv_freq == tr->inv_freq && o.positions == positions;
  const bool before = o.transform;
  o.transform = true;
  const gqe_status s = layer_options_alloc(h);
  if (s != GQE_OK) {
    o.transform = before;
    return s;
  }
  if (!same) ++o.generation;
  o.tr = *tr;
  o.positions = positions;
  o.dq_weight = dq_weight;
  o.dk_weight = dk_weight;
  return GQE_OK;
}

gqe_status gqe_set_scores(gqe_handle h, float scale, float softcap, const float* slopes,
                          const int32_t* key_begin, const int32_t* key_end) {
  if (!h) return GQE_ERR_INVALID_ARG;
  if (!(scale >= 0.f && scale < INFINITY) || !(softcap >= 0.f && softcap < INFINITY))
    return GQE_ERR_INVALID_ARG;
  const void* ptrs[] = {slopes, key_begin, key_end};
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return GQE_ERR_INVALID_ARG;
  if (!cap_in_range(scale, softcap) || !bias_in_range(scale, slopes)) return GQE_ERR_UNSUPPORTED;
  const bool on = scale > 0.f || softcap > 0.f || slopes || key_begin || key_end;
  if (on && h->dtype != GQE_BF16) return GQE_ERR_UNSUPPORTED;
  LayerOptions& o = options(h);
  const bool same = o.scores == on && o.scale == scale && o.softcap == softcap &&
                    o.slopes == slopes && o.key_begin == key_begin && o.key_end == key_end;
  const bool before = o.scores;
  o.scores = on;
  const gqe_status s = layer_options_alloc(h);
  if (s != GQE_OK) {
    o.scores = before;
    return s;
  }
  if (!same) ++o.generation;
  o.scale = scale;
  o.softcap = softcap;
  o.slopes = slopes;
  o.key_begin = key_begin;
  o.key_end = key_end;
  return GQE_OK;
}

}  // extern "C"
