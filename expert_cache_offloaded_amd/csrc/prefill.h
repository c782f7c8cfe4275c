// Steps of a prefill layer that its two forms share (prefill.hip, prefill_act.hip).
#pragma once

#include "mc_common.h"

namespace mc {

constexpr int kP_MaxE = 1024;      // experts of a layer

// Device buffers of the token sort; tile_e and status may be null.
struct SortBuffers {
  int32_t* counts;      // [E]
  int32_t* counts4;     // [E][4]
  int32_t* offsets;     // [E+1]
  int32_t* mtile_off;   // [E+1]
  int32_t* perm;        // [T*k]
  int32_t* tile_e;
  uint32_t* status;
};

int sort_routes_launch(const int32_t* ids, int T, int k, const int32_t* n_tok, int E, const SortBuffers& b,
                       hipStream_t s);
// y[t] = bf16 of the sum of token t's valid routes' rows of yr [T*k][H], in route order
int combine_launch(const int32_t* ids, int T, int k, int E, int H, const int32_t* n_tok, const float* yr,
                   uint16_t* y_bf16, hipStream_t s);
// checks and enqueues the next layer's whole-pool copy (mc_prefetch)
int prefetch_launch(const char* fn, const mc_prefetch* next, int E);

}  // namespace mc
