// seq_gates.cuh -- log alpha of the sequence kernels.
#pragma once

#include "gates.cuh"
#include "seq_internal.h"

namespace gdn {

// log alpha in 64 bits, from `floor` up; not a number where alpha is not or is negative (seq_alpha).
__device__ __forceinline__ double seq_log_gate(float a, float floor) {
    return a >= 0.f ? fmax(log_gate<double>(a), (double)floor) : (double)seq_alpha(a);
}

}  // namespace gdn
