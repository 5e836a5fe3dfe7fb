// Arguments of the decode attention with capped, biased and windowed scores
// (attn_scores_decode.cu), shared with the entry points and the layer's calls.
#pragma once

#include "qk_norm_rope.cuh"

namespace gqe {

struct DecodeArgs {
  QkTensor q, out;   // [S, B, d_h]
  QkTensor kc, vc;   // [G, B, L_max, d_h]: token_stride is the sequences' stride, rows dense
  const int32_t* lengths = nullptr;    // [B] positions of the new tokens (-1: no keys)
  const int32_t* key_begin = nullptr;  // [B] first visible keys, or none
  const float* slopes = nullptr;       // [S] or none
  const float* psel = nullptr;         // inside the layer, as the prefill's
  int64_t last_off = -1;
  int psel_stride = 0, psel_off = 0;
  float* part = nullptr;               // [S, B, np, d_h + 2] clusters' states (m, l, O)
  int32_t* status = nullptr;
  int B = 0, S = 0, G = 0, k = 0, d_h = 0, L_max = 0;
  int nc = 1, np = 1;      // chunks of a cluster (up to 8), clusters, per (sequence, KV head)
  float scale_log2 = 0.f;  // scale log2(e)
  float cap_in = 0.f;      // 2 / softcap: the tanh's argument from a score in log2 units
  float cap_log2 = 0.f;    // softcap log2(e), 0: none
};

void attn_decode_plan(int B, int G, int L_max, int num_sms, int& nc, int& np);
// Returns the number of kernels launched, or -1.
int launch_attn_decode(const DecodeArgs& P, cudaStream_t st);

}  // namespace gqe
