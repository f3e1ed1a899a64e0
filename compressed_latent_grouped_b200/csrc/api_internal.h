// What the translation units of the C ABI share: the validated geometry of a
// configuration, argument checks and the CUDA error record.
#pragma once

#include <stddef.h>

#include "kernels.h"

namespace ccgqa {

struct Geo {
  int E, C, Hq, Hkv, d, G, N, K;
  int qk_mean, value_shift, causal, rope_on, channel_conv;
  double rope_log2_base;
  int dtype;
  size_t es;  // element size
};

// Validate cfg and fill g.
ccgqa_status derive(const ccgqa_config* cfg, Geo* g);
// Validate a cache descriptor (need_state: the conv histories and v_prev too).
ccgqa_status check_cache(const Geo& g, const ccgqa_kvcache* c, bool need_state);
PageMap page_map(const ccgqa_kvcache* c);
// theta_i / (2 pi) as a 0.64 fixed-point fraction of a turn.
uint64_t rope_turn_fraction(double log2_base, int i, int d);
// Keep the error for ccgqa_last_error_string and return CCGQA_ERR_CUDA.
ccgqa_status cuda_fail(cudaError_t e);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace ccgqa
