// packed_attend.h -- host-side declarations of the attention over the 4-bit cache.
#pragma once

#include "internal.h"

namespace mla {

struct AttendPackedParams : AttendParams {
  const uint16_t *q_tilde;    // [B, Q, H, R]
  int window, sinks;          // window 0: every row up to the query's own
  float unit;                 // c = unit * scale * code
  float score_factor;         // softmax scale * log2(e) * unit
};

// The attend kernel, then the combine that writes o_latent / lse.
cudaError_t launch_attend_packed(const CUtensorMap &tm_codes, const CUtensorMap &tm_scales, const AttendPackedParams &p,
                                 cudaStream_t stream);

}  // namespace mla
