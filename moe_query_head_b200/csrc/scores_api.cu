// Entry points of the operators without a handle (include/gqe.h): the norm and rotation of
// queries and keys, and the attention with capped, biased and masked scores. Argument checks
// and launches; the kernels are in qk_norm_rope.cu and attn_scores*.cu.
#include <math.h>
#include <string.h>

#include <atomic>

#include "attn_scores.cuh"
#include "attn_scores_decode.cuh"
#include "scores_api.cuh"

namespace gqe {

// The device's status word: what the operators' kernels report (gqe_check_op_status reads it).
__device__ int32_t g_op_status;

namespace {
// Clears the word if it still holds what was read: a report that came in between stays.
__global__ void clear_status_kernel(int32_t* word, int32_t seen) { atomicCAS(word, seen, 0); }

constexpr int kMaxDevices = 64;
std::atomic<int32_t*> g_status_words[kMaxDevices];  // looked up once per device
std::atomic<int> g_num_sms[kMaxDevices];
}  // namespace

int32_t* op_status_word() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
  const bool known = dev >= 0 && dev < kMaxDevices;
  if (known)
    if (int32_t* p = g_status_words[dev].load(std::memory_order_relaxed)) return p;
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, g_op_status) != cudaSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  if (known) g_status_words[dev].store(static_cast<int32_t*>(p), std::memory_order_relaxed);
  return static_cast<int32_t*>(p);
}

int current_num_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  const bool known = dev >= 0 && dev < kMaxDevices;
  if (known && (n = g_num_sms[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
  if (known) g_num_sms[dev].store(n, std::memory_order_relaxed);
  return n;
}

gqe_status check_transform(const gqe_qk_transform* tr) {
  if (!tr) return GQE_ERR_INVALID_ARG;
  if (tr->dtype != GQE_BF16 && tr->dtype != GQE_F32) return GQE_ERR_INVALID_ARG;
  if (tr->norm != 0 && tr->norm != 1) return GQE_ERR_INVALID_ARG;
  if (tr->interleaved != 0 && tr->interleaved != 1) return GQE_ERR_INVALID_ARG;
  if (tr->norm && !(tr->eps >= 0.f && tr->eps < INFINITY)) return GQE_ERR_INVALID_ARG;
  if (tr->rot_dim < 0 || tr->rot_dim > tr->d_h || tr->rot_dim % 16 != 0)
    return GQE_ERR_INVALID_ARG;
  if (tr->rot_dim && (!tr->inv_freq || (reinterpret_cast<uintptr_t>(tr->inv_freq) & 7u)))
    return GQE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(tr->q_weight) & 3u) ||
      (reinterpret_cast<uintptr_t>(tr->k_weight) & 3u))
    return GQE_ERR_INVALID_ARG;
  if (tr->d_h < 16 || tr->d_h > 128 || tr->d_h % 16 != 0) return GQE_ERR_UNSUPPORTED;
  return GQE_OK;
}

QkArgs transform_args(const gqe_qk_transform& tr) {
  QkArgs A;
  A.d_h = tr.d_h;
  A.dtype = tr.dtype;
  A.norm = tr.norm;
  A.eps = tr.eps;
  A.q_weight = tr.norm ? tr.q_weight : nullptr;
  A.k_weight = tr.norm ? tr.k_weight : nullptr;
  A.rot_dim = tr.rot_dim;
  A.interleaved = tr.interleaved;
  A.inv_freq = tr.inv_freq;
  return A;
}

namespace {

constexpr int kMaxHeads = 512;                 // of one tensor of the norm and rotation
constexpr int64_t kMaxStride = int64_t(1) << 38;  // elements (tensor maps take 2^40 bytes)

// A gqe_heads of `heads` heads and `tokens` tokens (rows of row_min elements at least between
// tokens), with the strides of dimensions of one element set to something harmless.
bool take(const gqe_heads* t, int heads, int64_t tokens, int d_h, int esz, int64_t row_min,
          QkTensor& out) {
  if (!t || t->heads != heads) return false;
  out = QkTensor();
  out.heads = heads;
  if (heads == 0 || tokens == 0) return true;
  if (!t->data || (reinterpret_cast<uintptr_t>(t->data) & 15u)) return false;
  out.data = t->data;
  out.head_stride = heads > 1 ? t->head_stride : d_h;
  out.token_stride = tokens > 1 ? t->token_stride : row_min;
  const int64_t unit = 16 / esz;
  return out.head_stride >= d_h && out.token_stride >= row_min &&
         out.head_stride % unit == 0 && out.token_stride % unit == 0 &&
         out.head_stride < kMaxStride && out.token_stride < kMaxStride;
}

size_t align_up(size_t v) { return (v + 255) / 256 * 256; }

// The sizes and options of a gqe_scores; `decode`: T and the intervals of rows do not matter.
gqe_status check_scores(const gqe_scores* a, bool decode) {
  if (!a) return GQE_ERR_INVALID_ARG;
  if (a->B < 0 || (!decode && a->T < 0) || a->G < 1 || a->k < 1) return GQE_ERR_INVALID_ARG;
  if (a->G > 65535 || a->k > 65535) return GQE_ERR_UNSUPPORTED;
  const int64_t gk = (int64_t)a->G * a->k;
  if (a->S != gk && a->S != gk + 1) return GQE_ERR_INVALID_ARG;
  if (!decode && a->causal != 0 && a->causal != 1) return GQE_ERR_INVALID_ARG;
  if (!(a->scale >= 0.f && a->scale < INFINITY)) return GQE_ERR_INVALID_ARG;
  if (!(a->softcap >= 0.f && a->softcap < INFINITY)) return GQE_ERR_INVALID_ARG;
  if (!cap_in_range(a->scale, a->softcap)) return GQE_ERR_UNSUPPORTED;
  if (!bias_in_range(a->scale, a->slopes)) return GQE_ERR_UNSUPPORTED;
  const void* ptrs[] = {a->slopes, a->key_begin, decode ? nullptr : a->key_end};
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return GQE_ERR_INVALID_ARG;
  if (a->d_h < 16 || a->d_h > 128 || a->d_h % 16 != 0) return GQE_ERR_UNSUPPORTED;
  if (decode) {
    if (a->k > kMaxTopK || a->B > 65535) return GQE_ERR_UNSUPPORTED;
    return GQE_OK;
  }
  const int64_t M = (int64_t)a->B * a->T;
  if (M > (int64_t(1) << 27)) return GQE_ERR_UNSUPPORTED;
  if ((int64_t)a->B * (((int64_t)a->T + 127) / 128) * a->S > INT32_MAX)
    return GQE_ERR_UNSUPPORTED;
  if (a->S > 65535) return GQE_ERR_UNSUPPORTED;
  return GQE_OK;
}

AttnArgs attn_args(const gqe_scores& s) {
  AttnArgs a;
  a.B = s.B;
  a.T = s.T;
  a.S = s.S;
  a.G = s.G;
  a.k = s.k;
  a.d_h = s.d_h;
  a.causal = s.causal;
  a.scale = s.scale > 0.f ? s.scale : 1.f / sqrtf((float)s.d_h);
  a.softcap = s.softcap;
  a.slopes = s.slopes;
  a.key_begin = s.key_begin;
  a.key_end = s.key_end;
  return a;
}

}  // namespace
}  // namespace gqe

using namespace gqe;

extern "C" {

gqe_status gqe_qk_norm_rope(const gqe_qk_transform* tr, int M, const gqe_heads* q,
                            const gqe_heads* k, const int32_t* positions, int T,
                            const gqe_heads* q_out, const gqe_heads* k_out, void* stream) {
  const gqe_status r = check_transform(tr);
  if (r != GQE_OK) return r;
  if (M < 0 || !q || !k || q->heads < 0 || k->heads < 0) return GQE_ERR_INVALID_ARG;
  if (q->heads > kMaxHeads || k->heads > kMaxHeads) return GQE_ERR_UNSUPPORTED;
  if (positions ? (reinterpret_cast<uintptr_t>(positions) & 3u) != 0 : T < 1)
    return GQE_ERR_INVALID_ARG;
  const int esz = tr->dtype == GQE_F32 ? 4 : 2, d = tr->d_h;
  QkArgs A = transform_args(*tr);
  if (!take(q, q->heads, M, d, esz, d, A.q) || !take(k, k->heads, M, d, esz, d, A.k) ||
      !take(q_out, q->heads, M, d, esz, d, A.q_out) || !take(k_out, k->heads, M, d, esz, d, A.k_out))
    return GQE_ERR_INVALID_ARG;
  if (M == 0 || q->heads + k->heads == 0) return GQE_OK;
  A.positions = positions;
  A.M = M;
  A.period = positions ? 1 : T;
  const int sms = current_num_sms();
  if (sms < 0) return GQE_ERR_CUDA;
  return launch_qk_forward(A, sms, false, static_cast<cudaStream_t>(stream)) < 0 ? GQE_ERR_CUDA
                                                                                 : GQE_OK;
}

int64_t gqe_qk_norm_rope_workspace_bytes(int d_h) {
  if (d_h < 16 || d_h > 128 || d_h % 16 != 0) return -1;
  return (int64_t)kQkPartialRows * d_h * 4;
}

gqe_status gqe_qk_norm_rope_backward(const gqe_qk_transform* tr, int M, const gqe_heads* q,
                                     const gqe_heads* k, const int32_t* positions, int T,
                                     const gqe_heads* dq_out, const gqe_heads* dk_out,
                                     const gqe_heads* dq, const gqe_heads* dk, float* dq_weight,
                                     float* dk_weight, void* workspace, size_t bytes,
                                     void* stream) {
  const gqe_status r = check_transform(tr);
  if (r != GQE_OK) return r;
  if (M < 0 || !q || !k || q->heads < 0 || k->heads < 0) return GQE_ERR_INVALID_ARG;
  if (q->heads > kMaxHeads || k->heads > kMaxHeads) return GQE_ERR_UNSUPPORTED;
  if (positions ? (reinterpret_cast<uintptr_t>(positions) & 3u) != 0 : T < 1)
    return GQE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(dq_weight) & 3u) || (reinterpret_cast<uintptr_t>(dk_weight) & 3u))
    return GQE_ERR_INVALID_ARG;
  if (dq_weight && dq_weight == dk_weight) return GQE_ERR_INVALID_ARG;  // two sums, one place
  const int esz = tr->dtype == GQE_F32 ? 4 : 2, d = tr->d_h;
  QkArgs A = transform_args(*tr);
  if (!take(q, q->heads, M, d, esz, d, A.q) || !take(k, k->heads, M, d, esz, d, A.k) ||
      !take(dq_out, q->heads, M, d, esz, d, A.q_out) ||
      !take(dk_out, k->heads, M, d, esz, d, A.k_out) || !take(dq, q->heads, M, d, esz, d, A.dq) ||
      !take(dk, k->heads, M, d, esz, d, A.dk))
    return GQE_ERR_INVALID_ARG;
  const bool sums = tr->norm && (dq_weight || dk_weight);
  if (sums) {
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u)) return GQE_ERR_INVALID_ARG;
    if (bytes < (size_t)gqe_qk_norm_rope_workspace_bytes(d)) return GQE_ERR_WORKSPACE;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // without rows or without a norm the weights have no gradient
  if (!tr->norm || M == 0 || q->heads + k->heads == 0) {
    float* w[] = {dq_weight, dk_weight};
    for (float* p : w)
      if (p && cudaMemsetAsync(p, 0, (size_t)d * 4, st) != cudaSuccess) return GQE_ERR_CUDA;
  }
  if (M == 0 || q->heads + k->heads == 0) return GQE_OK;
  A.positions = positions;
  A.M = M;
  A.period = positions ? 1 : T;
  if (sums) {
    A.partial = static_cast<float*>(workspace);
    A.dq_weight = dq_weight;
    A.dk_weight = dk_weight;
  }
  const int sms = current_num_sms();
  if (sms < 0) return GQE_ERR_CUDA;
  return launch_qk_backward(A, sms, st) < 0 ? GQE_ERR_CUDA : GQE_OK;
}

gqe_status gqe_qk_norm_rope_append(const gqe_qk_transform* tr, int B, const gqe_heads* q,
                                   const gqe_heads* k, const gqe_heads* v,
                                   const int32_t* lengths, int L_max, const gqe_heads* q_out,
                                   const gqe_heads* k_cache, const gqe_heads* v_cache,
                                   void* stream) {
  const gqe_status r = check_transform(tr);
  if (r != GQE_OK) return r;
  if (B < 0 || L_max < 1 || !q || !k || q->heads < 0 || k->heads < 0) return GQE_ERR_INVALID_ARG;
  if (q->heads > kMaxHeads || k->heads > kMaxHeads) return GQE_ERR_UNSUPPORTED;
  if (!lengths || (reinterpret_cast<uintptr_t>(lengths) & 3u)) return GQE_ERR_INVALID_ARG;
  const int esz = tr->dtype == GQE_F32 ? 4 : 2, d = tr->d_h;
  const int64_t rows = (int64_t)L_max * d;
  QkArgs A = transform_args(*tr);
  if (!take(q, q->heads, B, d, esz, d, A.q) || !take(k, k->heads, B, d, esz, d, A.k) ||
      !take(v, k->heads, B, d, esz, d, A.v) || !take(q_out, q->heads, B, d, esz, d, A.q_out) ||
      !take(k_cache, k->heads, B, d, esz, rows, A.k_out) ||
      !take(v_cache, k->heads, B, d, esz, rows, A.v_out))
    return GQE_ERR_INVALID_ARG;
  if (B == 0 || q->heads + k->heads == 0) return GQE_OK;
  A.positions = lengths;
  A.M = B;
  A.L_max = L_max;
  A.status = op_status_word();
  const int sms = current_num_sms();
  if (sms < 0 || !A.status) return GQE_ERR_CUDA;
  return launch_qk_forward(A, sms, true, static_cast<cudaStream_t>(stream)) < 0 ? GQE_ERR_CUDA
                                                                                : GQE_OK;
}

gqe_status gqe_attention_forward(const gqe_scores* s, const gqe_heads* q, const gqe_heads* k,
                                 const gqe_heads* v, const gqe_heads* out, float* lse,
                                 void* stream) {
  const gqe_status r = check_scores(s, false);
  if (r != GQE_OK) return r;
  AttnArgs a = attn_args(*s);
  const int64_t M = (int64_t)s->B * s->T;
  const int d = s->d_h;
  if (!take(q, s->S, M, d, 2, d, a.q) || !take(k, s->G, M, d, 2, d, a.kk) ||
      !take(v, s->G, M, d, 2, d, a.v) || !take(out, s->S, M, d, 2, d, a.out))
    return GQE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(lse) & 3u) return GQE_ERR_INVALID_ARG;
  if (M == 0) return GQE_OK;
  a.lse = lse;
  a.status = op_status_word();
  if (!a.status) return GQE_ERR_CUDA;
  return launch_attn_scores(a, static_cast<cudaStream_t>(stream)) < 0 ? GQE_ERR_CUDA : GQE_OK;
}

int64_t gqe_attention_workspace_bytes(const gqe_scores* s) {
  if (check_scores(s, false) != GQE_OK) return -1;
  const size_t dsum = align_up((size_t)s->S * s->B * s->T * 4);
  return (int64_t)(dsum + align_up((size_t)s->B * (((size_t)s->T + 127) / 128) * 8));
}

gqe_status gqe_attention_backward(const gqe_scores* s, const gqe_heads* q, const gqe_heads* k,
                                  const gqe_heads* v, const gqe_heads* out, const float* lse,
                                  const gqe_heads* dout, const gqe_heads* dq,
                                  const gqe_heads* dk, const gqe_heads* dv, void* workspace,
                                  size_t bytes, void* stream) {
  const gqe_status r = check_scores(s, false);
  if (r != GQE_OK) return r;
  AttnArgs a = attn_args(*s);
  const int64_t M = (int64_t)s->B * s->T;
  const int d = s->d_h;
  if (!take(q, s->S, M, d, 2, d, a.q) || !take(k, s->G, M, d, 2, d, a.kk) ||
      !take(v, s->G, M, d, 2, d, a.v) || !take(out, s->S, M, d, 2, d, a.out) ||
      !take(dout, s->S, M, d, 2, d, a.dout) || !take(dq, s->S, M, d, 2, d, a.dq) ||
      !take(dk, s->G, M, d, 2, d, a.dk) || !take(dv, s->G, M, d, 2, d, a.dv))
    return GQE_ERR_INVALID_ARG;
  if (M == 0) return GQE_OK;
  if (!lse || (reinterpret_cast<uintptr_t>(lse) & 3u)) return GQE_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u)) return GQE_ERR_INVALID_ARG;
  if (bytes < (size_t)gqe_attention_workspace_bytes(s)) return GQE_ERR_WORKSPACE;
  a.lse = const_cast<float*>(lse);
  a.dsum = static_cast<float*>(workspace);
  a.blocks = reinterpret_cast<int2*>(static_cast<char*>(workspace) + align_up((size_t)s->S * M * 4));
  a.status = op_status_word();
  if (!a.status) return GQE_ERR_CUDA;
  return launch_attn_scores_backward(a, static_cast<cudaStream_t>(stream)) < 0 ? GQE_ERR_CUDA
                                                                               : GQE_OK;
}

int64_t gqe_attention_decode_workspace_bytes(const gqe_scores* s, int L_max) {
  if (check_scores(s, true) != GQE_OK || L_max < 1 || L_max > (1 << 30)) return -1;
  const int sms = current_num_sms();
  if (sms < 0) return -1;
  if (s->B == 0) return 0;
  int nc, np;
  attn_decode_plan(s->B, s->G, L_max, sms, nc, np);
  return np > 1 ? (int64_t)s->S * s->B * np * (s->d_h + 2) * 4 : 0;
}

gqe_status gqe_attention_decode(const gqe_scores* s, const gqe_heads* q,
                                const gqe_heads* k_cache, const gqe_heads* v_cache, int L_max,
                                const int32_t* lengths, const gqe_heads* out, void* workspace,
                                size_t bytes, void* stream) {
  const gqe_status r = check_scores(s, true);
  if (r != GQE_OK) return r;
  if (L_max < 1) return GQE_ERR_INVALID_ARG;
  if (L_max > (1 << 30)) return GQE_ERR_UNSUPPORTED;
  if (!lengths || (reinterpret_cast<uintptr_t>(lengths) & 3u)) return GQE_ERR_INVALID_ARG;
  const int d = s->d_h;
  const int64_t rows = (int64_t)L_max * d;
  DecodeArgs P;
  if (!take(q, s->S, s->B, d, 2, d, P.q) || !take(out, s->S, s->B, d, 2, d, P.out) ||
      !take(k_cache, s->G, s->B, d, 2, rows, P.kc) || !take(v_cache, s->G, s->B, d, 2, rows, P.vc))
    return GQE_ERR_INVALID_ARG;
  if (s->B == 0) return GQE_OK;
  const int sms = current_num_sms();
  P.status = op_status_word();
  if (sms < 0 || !P.status) return GQE_ERR_CUDA;
  attn_decode_plan(s->B, s->G, L_max, sms, P.nc, P.np);
  if (P.np > 1) {
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u)) return GQE_ERR_INVALID_ARG;
    if (bytes < (size_t)s->S * s->B * P.np * (d + 2) * 4) return GQE_ERR_WORKSPACE;
    P.part = static_cast<float*>(workspace);
  }
  P.lengths = lengths;
  P.key_begin = s->key_begin;
  P.slopes = s->slopes;
  P.B = s->B;
  P.S = s->S;
  P.G = s->G;
  P.k = s->k;
  P.d_h = d;
  P.L_max = L_max;
  set_decode_scores(P, s->scale, s->softcap);
  return launch_attn_decode(P, static_cast<cudaStream_t>(stream)) < 0 ? GQE_ERR_CUDA : GQE_OK;
}

gqe_status gqe_check_op_status(void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t* word = op_status_word();
  if (!word || cudaStreamSynchronize(st) != cudaSuccess) return GQE_ERR_CUDA;
  int32_t v = 0;
  if (cudaMemcpy(&v, word, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return GQE_ERR_CUDA;
  if (v == kStatusOk) return GQE_OK;
  clear_status_kernel<<<1, 1, 0, st>>>(word, v);
  if (cudaGetLastError() != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess)
    return GQE_ERR_CUDA;
  return v == kStatusBadInput ? GQE_ERR_INVALID_ARG : GQE_ERR_TIMEOUT;
}

}  // extern "C"
