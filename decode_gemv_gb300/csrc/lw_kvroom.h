// Stretches of the numbers that a cluster chooses from (lw_kvselect.cuh), and
// the room for them.  Plain C++ apart from the __host__ __device__ marks, so
// that it also builds (and is tested) without the CUDA compiler.
#pragma once

#include "lw_tcplan.h"

namespace lw {

// Numbers of a CTA's stretch, where `ranks` CTAs share `count`: whole warps'.
LW_TC_HD int kv_select_stretch(long long count, int ranks) { return (int)(((count + ranks - 1) / ranks + 31) / 32 * 32); }

// Numbers that a CTA gets room for, where there may be `count`.  In steps: the launcher keeps an answer of the
// driver's for every size that it met, and a program's lengths grow number by number.
constexpr long long kSelectStep = 1024;
inline long long kv_select_room(long long count, int ranks) {
  return (kv_select_stretch(count, ranks) + kSelectStep - 1) / kSelectStep * kSelectStep;
}

}  // namespace lw
