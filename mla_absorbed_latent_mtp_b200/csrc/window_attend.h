// window_attend.h -- host-side declarations of the attention with a sliding window and sinks.
#pragma once

#include "internal.h"

namespace mla {

struct WindowParams : AttendParams {
  int window, sinks;  // rows j <= t with t - j < window or j < sinks are seen
};

// The attend kernel, then the combine that writes o_latent / lse.
cudaError_t launch_attend_window(bool paged, const CUtensorMap &tm_cache, const CUtensorMap &tm_qt, const WindowParams &p,
                                 cudaStream_t stream);

}  // namespace mla
