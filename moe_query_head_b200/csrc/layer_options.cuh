// What a handle carries beyond gqe_ctx: the norm and rotation of its queries and keys and the
// form of its scores (gqe_set_qk_transform, gqe_set_scores), with their buffers, and the
// layer's stages that run with them (layer_options.cu). Every handle is a LayerCtx.
#pragma once

#include "gqe_common.cuh"

namespace gqe {

struct LayerOptions {
  bool transform = false;
  gqe_qk_transform tr = {};
  const int32_t* positions = nullptr;  // [B T] or none
  float* dq_weight = nullptr;
  float* dk_weight = nullptr;
  bool scores = false;
  float scale = 0.f, softcap = 0.f;
  const float* slopes = nullptr;
  const int32_t* key_begin = nullptr;
  const int32_t* key_end = nullptr;
  // counts changes of what a forward computes; a backward needs its forward's
  uint64_t generation = 0;
  uint64_t last_forward = 0;
  // buffers: transformed queries and keys; for the backward their gradients, the weight
  // gradients' partial sums and the intervals of row blocks
  void* fwd_base = nullptr;
  void* q_t = nullptr;  // [S, M, d_h]
  void* k_t = nullptr;  // [G, M, d_h]
  void* bwd_base = nullptr;
  void* dq_t = nullptr;  // [S, M, d_h]
  void* dk_t = nullptr;  // [G, M, d_h]
  float* partial = nullptr;
  int2* blocks = nullptr;
};

}  // namespace gqe

struct LayerCtx : gqe_ctx {
  gqe::LayerOptions opt;
};

namespace gqe {

inline LayerOptions& options(gqe_ctx* h) { return static_cast<LayerCtx*>(h)->opt; }
inline const LayerOptions& options(const gqe_ctx* h) {
  return static_cast<const LayerCtx*>(h)->opt;
}
inline bool has_options(const gqe_ctx* h) { return options(h).transform || options(h).scores; }

// Allocates the buffers that the options need and that are missing (those of the backward
// once the handle has one). Frees: layer_options_release.
gqe_status layer_options_alloc(gqe_ctx* h);
void layer_options_release(gqe_ctx* h);

// The attention stages of a handle with options. Each returns the number of kernels
// launched, or -1.
int launch_layer_attention(gqe_ctx* h, int B, int T, int S, int has_shared, int variant,
                           int causal, int Do, cudaStream_t st);
int launch_layer_decode(gqe_ctx* h, int B, int S, int has_shared, int variant, int Do,
                        void* k_cache, void* v_cache, int L_max, const int32_t* lengths,
                        cudaStream_t st);
int launch_layer_attention_backward(gqe_ctx* h, const BwdBuffers& bb, int B, int T, int S,
                                    int has_shared, int causal, cudaStream_t st);

}  // namespace gqe
