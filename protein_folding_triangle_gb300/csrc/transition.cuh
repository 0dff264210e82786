// Activations and tensor maps of the transition, shared by its kernels.
#pragma once
#include <cudaTypedefs.h>

#include <type_traits>

#include "kernels.cuh"
#include "triattn.h"

namespace triattn {
namespace {

// The gates, two features at once on packed FP32 pairs.  All three activations
// are sigmoids: SiLU a sigmoid(a), GELU (tanh form) a sigmoid(2 u), u = sqrt(2/pi)
// (a + 0.044715 a^3).  A sigmoid is 1 / (1 + 2^t), t = -a log2(e), one hardware
// exponential and one reciprocal, right to a few 2^-22 of its own value (and what FP32
// leaves of t) however closed the gate is.  (1 + tanh(a / 2)) / 2 with the
// hardware's tanh takes the special-function unit once instead of twice (768 x 768 rows,
// C = 128, H = 512: nothing of the forward's 0.17 ms, 50 of 990 us forward and backward), but
// is right relative to 1 only: gates below a = -18 were 0.
__device__ __forceinline__ float2 sigmoid2(float2 t) {
  const float2 d = fadd2(make_float2(ex2_approx(t.x), ex2_approx(t.y)), make_float2(1.f, 1.f));
  return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}
// t of the activation's sigmoid.
template <int ACT>
__device__ __forceinline__ float2 gate_arg2(float2 a) {
  if constexpr (ACT == TRIATTN_ACT_GELU)
    return fmul2(a, ffma2(fmul2(a, a), make_float2(-0.10294323f, -0.10294323f), make_float2(-2.3022082f, -2.3022082f)));
  return fmul2(a, make_float2(-1.442695041f, -1.442695041f));
}
// h = act(a) b
template <int ACT>
__device__ __forceinline__ float2 gate_fwd2(float2 a, float2 b) {
  const float2 s = sigmoid2(gate_arg2<ACT>(a));
  return fmul2(ACT == TRIATTN_ACT_SIGMOID ? b : fmul2(a, b), s);
}
// ... and h, da = d b act'(a), db = d act(a).
template <int ACT>
__device__ __forceinline__ void gate_bwd2(float2 a, float2 b, float2 d, float2& h, float2& da, float2& db) {
  const float2 one = make_float2(1.f, 1.f);
  float2 t = gate_arg2<ACT>(a), f, df;
  if constexpr (ACT == TRIATTN_ACT_SIGMOID) {
    // s (1 - s) with 1 - s = 2^t s: taken from 1 it would lose an open gate's digits.
    // 2^126 at most, so that the product is not infinity times 0
    t = make_float2(fmin_nan(t.x, 126.f), fmin_nan(t.y, 126.f));
    const float2 e = make_float2(ex2_approx(t.x), ex2_approx(t.y)), w = fadd2(e, one);
    f = make_float2(rcp_approx(w.x), rcp_approx(w.y));
    df = fmul2(fmul2(e, f), f);
  } else {
    // s + f (1 - s) (t's slope): where 1 - s loses digits s is near 1 beside it
    const float2 s = sigmoid2(t);
    f = fmul2(a, s);
    float2 c = ffma2(make_float2(-f.x, -f.y), s, f);
    if constexpr (ACT == TRIATTN_ACT_GELU)
      c = fmul2(c, ffma2(fmul2(a, a), make_float2(0.21406448f, 0.21406448f), make_float2(1.5957691f, 1.5957691f)));
    df = fadd2(c, s);
  }
  h = fmul2(f, b);
  db = fmul2(d, f);
  da = fmul2(fmul2(d, b), df);
}
__device__ __forceinline__ float2 bf16x2_to_f32x2(uint32_t w) {
  return make_float2(bf16lo_to_f32(w), bf16hi_to_f32(w));
}

// Mean and 1 / sqrt(variance + eps) of a row of C features held as C / 8
// chunks of 16 bytes at z16(c), in one pass about the mean k of its first 8
// features: |k - mean| is at most sqrt((C - 8) / 8) < 6 standard deviations
// whatever the row holds, so that the difference below loses less than a
// factor of 37 of the FP32 precision.
template <int C, typename F>
__device__ __forceinline__ float2 row_stats(F&& z16) {
  float k;
  {
    const uint4 w = *z16(0);
    const float2 k2 = fadd2(fadd2(bf16x2_to_f32x2(w.x), bf16x2_to_f32x2(w.y)),
                            fadd2(bf16x2_to_f32x2(w.z), bf16x2_to_f32x2(w.w)));
    k = (k2.x + k2.y) * 0.125f;
  }
  const float2 nk = make_float2(-k, -k);
  float2 s2[2], q2[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) s2[e] = q2[e] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int c = 0; c < C / 8; ++c) {
    const uint4 w = *z16(c);
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 d = fadd2(bf16x2_to_f32x2(ws[e]), nk);
      s2[e & 1] = fadd2(s2[e & 1], d);
      q2[e & 1] = ffma2(d, d, q2[e & 1]);
    }
  }
  const float2 ss = fadd2(s2[0], s2[1]), qq = fadd2(q2[0], q2[1]);
  const float ds = (ss.x + ss.y) * (1.f / C);  // mean - k
  return make_float2(k + ds, rsqrtf(fmaxf(fmaf(-ds, ds, (qq.x + qq.y) * (1.f / C)), 0.f) + 1e-5f));
}

// Allows a kernel `bytes` of dynamic shared memory: the most that any launch of it
// takes, the same in every call, so that a thread that sets it never takes away
// what another one is about to launch with.  `regs` is what its warpgroups'
// register split adds up to: a split above what the launch of `warpgroups` has
// would wait for ever.  One query per call, and a setting only where it is
// missing (the first call on a device, or after its reset).
template <typename K>
cudaError_t tf_allow(K* kernel, int bytes, int warpgroups = 0, int regs = 0) {
  cudaFuncAttributes at;
  const cudaError_t e = cudaFuncGetAttributes(&at, kernel);
  if (e != cudaSuccess) return e;
  if (at.numRegs * warpgroups < regs) return cudaErrorInvalidConfiguration;
  if (at.maxDynamicSharedSizeBytes >= bytes) return cudaSuccess;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
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

// 3-D BF16 maps: boxes of 64 (inner) x box1 x box2 with the 128-byte swizzle,
// and (tf_map32) boxes of 32 x 32 with the 64-byte swizzle.
inline bool tf_map_box(CUtensorMap* m, const void* base, const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2],
                       cuuint32_t box0, cuuint32_t box1, cuuint32_t box2, CUtensorMapSwizzle swizzle) {
  const auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (enc == nullptr) return false;
  const cuuint32_t box[3] = {box0, box1, box2}, es[3] = {1u, 1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
inline bool tf_map(CUtensorMap* m, const void* base, const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2],
                   cuuint32_t box1, cuuint32_t box2) {
  return tf_map_box(m, base, dims, strides, 64u, box1, box2, CU_TENSOR_MAP_SWIZZLE_128B);
}
inline bool tf_map32(CUtensorMap* m, void* base, const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2]) {
  return tf_map_box(m, base, dims, strides, 32u, 32u, 1u, CU_TENSOR_MAP_SWIZZLE_64B);
}

}  // namespace
}  // namespace triattn
