// Arguments of the query / key norm and rotation kernels (qk_norm_rope.cu), shared with the
// entry points and the layer's calls.
#pragma once

#include "gqe_common.cuh"

namespace gqe {

// Rows of partial weight sums of a backward call at most (blocks of four warps: eight per SM).
constexpr int kQkPartialRows = 1184;

struct QkTensor {
  void* data = nullptr;
  int64_t head_stride = 0, token_stride = 0;  // elements
  int heads = 0;
};

struct QkArgs {
  QkTensor q, k, v;              // inputs (v: append only)
  QkTensor q_out, k_out, v_out;  // outputs; for the backward their gradients (inputs)
  QkTensor dq, dk;               // backward: gradients of q and k
  const float* q_weight = nullptr;  // [d_h] or none
  const float* k_weight = nullptr;
  const double* inv_freq = nullptr;    // [rot_dim / 2] radians per position
  const int32_t* positions = nullptr;  // [M]; none: token index modulo period
  int64_t M = 0;
  int period = 1;
  int d_h = 0, dtype = 0, norm = 0, rot_dim = 0, interleaved = 0;
  float eps = 0.f;
  int L_max = 0;              // append: rows per sequence of the caches
  int32_t* status = nullptr;  // append: device status word
  int idle_ok = 1;            // append: position -1 marks an idle slot (0: it is reported too)
  // backward
  float* partial = nullptr;  // [kQkPartialRows, d_h] or none (no weight gradient asked for)
  float* dq_weight = nullptr;
  float* dk_weight = nullptr;
  // backward inside the layer: a routed stream's gradient goes to the column block of its
  // expert (dq rows of experts-major blocks), the shared stream's to dq_shared
  const int32_t* sel = nullptr;
  void* dq_shared = nullptr;
  int64_t sel_stride = 0;
  int sel_off = 0, routed = 0, top_k = 1, experts = 0;
  // set by the launcher
  int heads_per_chunk = 1, chunks_q = 0, chunks_k = 0;
};

// Each returns the number of kernels launched, or -1.
int launch_qk_forward(QkArgs& A, int num_sms, bool append, cudaStream_t st);
int launch_qk_backward(QkArgs& A, int num_sms, cudaStream_t st);

}  // namespace gqe
