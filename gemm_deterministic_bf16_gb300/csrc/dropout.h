// dropout.h -- launcher of dropout from a counter-based generator.
#pragma once

#include "block.h"

namespace detffn {

struct DropoutArgs {
  long long M = 0, H = 0;
  int dtype = 0;
  Rows x, residual, out;
  uint32_t limit = 0;        // an element is kept where its word is at least this
  float scale = 1.0f;        // 1 / (1 - p); with p = 1 nothing is kept
  bool none = false;         // p = 1
  unsigned long long seed = 0, offset = 0;
  const unsigned long long* state = nullptr;   // device: {seed, offset}, the seed instead of `seed`, the offset added
};

cudaError_t launch_dropout(const DropoutArgs& a, int sm_count, cudaStream_t st);

}  // namespace detffn
