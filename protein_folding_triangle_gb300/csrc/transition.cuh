// Activations and tensor maps of the transition, shared by its kernels.
#pragma once
#include <cudaTypedefs.h>

#include <type_traits>

#include "kernels.cuh"
#include "triattn.h"

namespace triattn {
namespace {

// act(a) and act'(a).  Each takes one hardware tanh (absolute error about
// 2^-11, below the BF16 rounding of h): sigmoid(a) = (1 + tanh(a / 2)) / 2.
template <int ACT>
__device__ __forceinline__ float act_fwd(float a) {
  if constexpr (ACT == TRIATTN_ACT_GELU) {
    const float u = a * fmaf(0.0356774081f * a, a, 0.7978845608f);  // sqrt(2/pi) (a + 0.044715 a^3)
    const float ha = 0.5f * a;
    return fmaf(ha, tanh_approx(u), ha);
  } else {
    const float s = fmaf(0.5f, tanh_approx(0.5f * a), 0.5f);
    return ACT == TRIATTN_ACT_SILU ? a * s : s;
  }
}
template <int ACT>
__device__ __forceinline__ void act_both(float a, float& f, float& df) {
  if constexpr (ACT == TRIATTN_ACT_GELU) {
    const float a2 = a * a;
    const float t = tanh_approx(a * fmaf(0.0356774081f, a2, 0.7978845608f));
    const float ht = fmaf(0.5f, t, 0.5f);
    f = a * ht;
    df = fmaf(0.5f * a * fmaf(-t, t, 1.f), fmaf(0.1070322243f, a2, 0.7978845608f), ht);
  } else {
    const float s = fmaf(0.5f, tanh_approx(0.5f * a), 0.5f);
    if constexpr (ACT == TRIATTN_ACT_SILU) {
      f = a * s;
      df = fmaf(f, 1.f - s, s);
    } else {
      f = s;
      df = s * (1.f - s);
    }
  }
}

// f(std::integral_constant<int, ACT>) for the activations.
template <typename F>
cudaError_t by_act(int act, F&& f) {
  switch (act) {
    case TRIATTN_ACT_SILU: return f(std::integral_constant<int, TRIATTN_ACT_SILU>{});
    case TRIATTN_ACT_SIGMOID: return f(std::integral_constant<int, TRIATTN_ACT_SIGMOID>{});
    case TRIATTN_ACT_GELU: return f(std::integral_constant<int, TRIATTN_ACT_GELU>{});
  }
  return cudaErrorInvalidValue;
}

// 3-D BF16 map in boxes of 64 (inner) x box1 x box2, 128-byte swizzle.
inline bool tf_map(CUtensorMap* m, const void* base, const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2],
                   cuuint32_t box1, cuuint32_t box2) {
  const auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (enc == nullptr) return false;
  const cuuint32_t box[3] = {64u, box1, box2}, es[3] = {1u, 1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace triattn
