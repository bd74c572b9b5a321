// Host half of spec_sample_tokens: argument checks.  Plain C++ with no HIP
// types, like sv_host.h.
#pragma once

#include "sv_host_quant.h"

namespace sv {

// A request setting: one value per row, or one for all.
template <typename T>
struct Setting {
  const T* rows;  // [R] or null
  T all;          // where rows is null
};

struct SampleSettings {
  Setting<float> temperature;
  Setting<int32_t> top_k;
  Setting<float> top_p, min_p;
};

constexpr int kSampleThreads = 1024;  // a row's block at most
// Up to so many rows, one per CU, the blocks have 16 waves, else eight: top-p on 64 and 256 rows of 128256 bf16 42 and
// 45 us, with eight 48 and 52; on 300 rows 81 with sixteen and 72 with eight.
constexpr int kSampleWideRows = 256;

inline spec_status_t validate_sample(const void* logits, const float* uniforms, int32_t R, int32_t V,
                                     spec_dtype_t dtype, const SampleSettings& set, const int32_t* tokens,
                                     bool* empty) {
  if (!valid_dtype(dtype) || R < 0 || V < 1) return SPEC_ERR_INVALID_ARG;
  if (!set.temperature.rows && !(set.temperature.all >= 0.0f && isfinite(set.temperature.all)))
    return SPEC_ERR_INVALID_ARG;
  if (!set.top_p.rows && set.top_p.all != set.top_p.all) return SPEC_ERR_INVALID_ARG;
  if (!set.min_p.rows && set.min_p.all != set.min_p.all) return SPEC_ERR_INVALID_ARG;
  if (V > (1 << 30) || (size_t)R > max_blocks(kSampleThreads)) return SPEC_ERR_UNSUPPORTED;
  *empty = R == 0;
  if (*empty) return SPEC_OK;
  if (!logits || !uniforms || !tokens) return SPEC_ERR_INVALID_ARG;
  if ((uintptr_t)logits % elem_size(dtype) || (uintptr_t)uniforms % 4 || (uintptr_t)tokens % 4 ||
      (uintptr_t)set.temperature.rows % 4 || (uintptr_t)set.top_k.rows % 4 || (uintptr_t)set.top_p.rows % 4 ||
      (uintptr_t)set.min_p.rows % 4)
    return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}

// The tokens share a byte with what the call reads: a row's block would write where another reads its logits or settings.
// Of a call that validate_sample took.
inline bool sample_overlaps(const void* logits, const float* uniforms, int32_t R, int32_t V, spec_dtype_t dtype,
                            const SampleSettings& set, const int32_t* tokens) {
  const size_t rows = (size_t)R * 4;
  const void* const per_row[] = {uniforms, set.temperature.rows, set.top_k.rows, set.top_p.rows, set.min_p.rows};
  for (const void* p : per_row)
    if (p && overlap(tokens, rows, p, rows)) return true;
  return overlap(tokens, rows, logits, (size_t)R * (size_t)V * elem_size(dtype));
}

}  // namespace sv
