// What the layer's entry points share with the operators' (scores_api.cu).
#pragma once

#include <math.h>

#include "attn_scores.cuh"
#include "attn_scores_decode.cuh"

namespace gqe {

int32_t* op_status_word();  // the current device's status word of the operators, or NULL
int current_num_sms();      // of the current device, or -1
gqe_status check_transform(const gqe_qk_transform* tr);
QkArgs transform_args(const gqe_qk_transform& tr);

inline void set_decode_scores(DecodeArgs& P, float scale, float softcap) {
  P.scale_log2 = (scale > 0.f ? scale : 1.f / sqrtf((float)P.d_h)) * kLog2e;
  P.cap_in = softcap > 0.f ? 2.f / softcap : 0.f;
  P.cap_log2 = softcap * kLog2e;
}

}  // namespace gqe
