// Transition: the gated feed-forward block of the pair stack over M rows of C
// features, forward and backward.
//
//   x = LayerNorm(z; ln_w, ln_b)                    eps 1e-5
//   [a | b] = x W_in      W_in [C, 2H]              h = act(a) b
//   out = m (h W_o)       W_o [H, C]                m: optional row mask
//
// backward from d_out, with g = m d_out (nothing is kept from the forward:
// x, a and b are computed again):
//
//   dW_o = h^T g    dh = g W_o^T    da = dh b act'(a)    db = dh act(a)
//   dW_in = x^T [da | db]    dx = [da | db] W_in^T    dz, d_ln_w, d_ln_b from dx
//
// A row whose mask is 0 is left out: out and dz are 0 and no gradient takes a
// part of it, whatever z and d_out hold there (padding may be NaN).
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "kernels.cuh"
#include "pairops.cuh"
#include "transition.cuh"
#include "triattn.h"

namespace triattn {
namespace {

using namespace pairops;

constexpr int kMaxH = 4096;

__device__ __forceinline__ void unpack8(const uint4 w, float (&f)[8]) {
  f[0] = bf16lo_to_f32(w.x); f[1] = bf16hi_to_f32(w.x);
  f[2] = bf16lo_to_f32(w.y); f[3] = bf16hi_to_f32(w.y);
  f[4] = bf16lo_to_f32(w.z); f[5] = bf16hi_to_f32(w.z);
  f[6] = bf16lo_to_f32(w.w); f[7] = bf16hi_to_f32(w.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ uint4 ld16(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void st16(uint16_t* p, uint4 v) { *reinterpret_cast<uint4*>(p) = v; }

// g = m d_out, exactly 0 where m is 0 (8 features per thread).
__global__ void __launch_bounds__(256) mask_rows_kernel(const uint16_t* __restrict__ d_out,
                                                        const uint16_t* __restrict__ mask, uint16_t* __restrict__ g,
                                                        int C, size_t M) {
  const size_t chunks = C / 8;
  for (size_t t = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x; t < M * chunks;
       t += static_cast<size_t>(gridDim.x) * blockDim.x) {
    const size_t m = t / chunks;
    const float mk = bf16lo_to_f32(mask[m]);
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (mk != 0.f) {
      float v[8];
      unpack8(ld16(d_out + 8 * t), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= mk;
      w = pack8(v);
    }
    st16(g + 8 * t, w);
  }
}

// The backward's partial sums in a fixed order, the results FP32 or BF16 (one
// rounding): the first wblocks blocks take those of the weight gradients (n
// float4 each, dW_in's n_in first), four threads per four elements, each a
// quarter of the parts; the others the rows of d_ln_w's and d_ln_b's, eight
// columns each.  A thread has its loads under way at once: what the launch
// takes is their latency.
constexpr int kSumRows = kTbPartRows / 32, kSumParts = 10;
struct SumParams {
  const float4* w;
  size_t n_in, n;
  int wparts;
  unsigned wblocks;
  const float *pg, *pb;
  int rows, C, bf16;
  void *d_w_in, *d_w_o, *d_ln_w, *d_ln_b;
};
__global__ void __launch_bounds__(256) transition_sum_kernel(const SumParams p) {
  if (blockIdx.x < p.wblocks) {
    __shared__ float4 quarter[3][64];
    const int q = threadIdx.x / 64, per = (p.wparts + 3) / 4;
    const size_t i = static_cast<size_t>(blockIdx.x) * 64 + threadIdx.x % 64;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4 v) {
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    };
    if (i < p.n) {
      const int end = min((q + 1) * per, p.wparts);
      for (int g = q * per; g < end; g += kSumParts) {
        float4 v[kSumParts];
#pragma unroll
        for (int k = 0; k < kSumParts; ++k)
          v[k] = g + k < end ? p.w[(g + k) * p.n + i] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kSumParts; ++k) add(v[k]);
      }
    }
    if (q > 0) quarter[q - 1][threadIdx.x % 64] = s;
    __syncthreads();
    if (q > 0 || i >= p.n) return;
#pragma unroll
    for (int k = 0; k < 3; ++k) add(quarter[k][threadIdx.x]);
    void* const dst = i < p.n_in ? p.d_w_in : p.d_w_o;
    const size_t at = i < p.n_in ? i : i - p.n_in;
    if (p.bf16) static_cast<uint2*>(dst)[at] = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
    else static_cast<float4*>(dst)[at] = s;
    return;
  }
  __shared__ float row[32][8];
  const int k8 = threadIdx.x & 7, rg = threadIdx.x >> 3;
  const int c0 = static_cast<int>(blockIdx.x - p.wblocks) * 8;  // of the 2 C columns
  const float* part = c0 < p.C ? p.pg : p.pb;
  void* dst = c0 < p.C ? p.d_ln_w : p.d_ln_b;
  const int c = (c0 < p.C ? c0 : c0 - p.C) + k8;
  float s = 0.f;
  for (int r0 = rg; r0 < p.rows; r0 += 32 * kSumRows) {
    float v[kSumRows];
#pragma unroll
    for (int k = 0; k < kSumRows; ++k)
      v[k] = r0 + 32 * k < p.rows ? part[static_cast<size_t>(r0 + 32 * k) * p.C + c] : 0.f;
#pragma unroll
    for (int k = 0; k < kSumRows; ++k) s += v[k];
  }
  row[rg][k8] = s;
  __syncthreads();
  if (rg > 0) return;
#pragma unroll
  for (int k = 1; k < 32; ++k) s += row[k][k8];
  if (p.bf16) static_cast<uint16_t*>(dst)[c] = static_cast<uint16_t>(pack_bf16x2(s, 0.f) & 0xFFFFu);
  else static_cast<float*>(dst)[c] = s;
}

// ---------------------------------------------------------------- host side
size_t rup(size_t x) { return (x + 255) / 256 * 256; }
bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }

struct TrDims {
  size_t M;
  int C, H, act;
  bool bf16;
};
TrDims tr_dims(const triattn_transition_shape* s) {
  return {static_cast<size_t>(s->M), s->C, s->H, s->activation, (s->flags & TRIATTN_FLAG_GRADS_BF16) != 0};
}

struct TrWs {
  size_t gemm, x, mean, rstd, P, h, g, dh, dx, wg, pg, pb, total;
};
TrWs tr_ws(const TrDims& d) {
  TrWs w;
  size_t o = 0;
  w.gemm = w.wg = o;
  if (transition_bwd_fused(d.C)) {
    w.x = o;  o += rup(d.M * d.C * 2);
    w.g = o;  o += rup(d.M * d.C * 2);
    w.wg = o; o += rup(transition_wgrad_bytes(static_cast<long long>(d.M), d.C, d.H));
    w.pg = o; o += rup(static_cast<size_t>(kTbPartRows) * d.C * 4);
    w.pb = o; o += rup(static_cast<size_t>(kTbPartRows) * d.C * 4);
    w.mean = w.rstd = w.P = w.h = w.dh = w.dx = w.total = o;
    return w;
  }
  o += rup(kGemmWorkspace);
  w.x = o;    o += rup(d.M * d.C * 2);
  w.mean = o; o += rup(d.M * 4);
  w.rstd = o; o += rup(d.M * 4);
  w.P = o;    o += rup(d.M * d.H * 4);
  w.h = o;    o += rup(d.M * d.H * 2);
  w.g = o;    o += rup(d.M * d.C * 2);
  w.dh = o;   o += rup(d.M * d.H * 2);
  w.dx = o;   o += rup(d.M * d.C * 4);  // FP32: BF16 would save 25 us of 950 and add a seventh to the error of dz
  w.pg = o;   o += rup(static_cast<size_t>(kLnBlocks) * d.C * 4);
  w.pb = o;   o += rup(static_cast<size_t>(kLnBlocks) * d.C * 4);
  w.total = o;
  return w;
}

triattn_status check_transition(const triattn_transition_shape* s) {
  if (s == nullptr || s->M < 0 || s->C < 1 || s->H < 1 || (s->flags & ~TRIATTN_FLAG_GRADS_BF16) != 0 ||
      s->activation < TRIATTN_ACT_SILU || s->activation > TRIATTN_ACT_GELU)
    return TRIATTN_ERR_INVALID_ARG;
  if (s->M > 0x7fffffffll || !ln_width_ok(s->C) || s->H % 32 != 0 || s->H > kMaxH) return TRIATTN_ERR_UNSUPPORTED;
  return TRIATTN_OK;
}

// f(std::integral_constant<int, C>) for the row widths that the fused backward
// does not take.
template <typename F>
cudaError_t by_c(int C, F&& f) {
  switch (C) {
    case 160: return f(std::integral_constant<int, 160>{});
    case 192: return f(std::integral_constant<int, 192>{});
    case 224: return f(std::integral_constant<int, 224>{});
    case 256: return f(std::integral_constant<int, 256>{});
  }
  return cudaErrorInvalidValue;
}

unsigned grid_for(size_t n) { return static_cast<unsigned>(n / 256 + 1 < 152 * 16 ? n / 256 + 1 : 152 * 16); }

cudaError_t ln_fwd_rows(const TrDims& d, const void* z, const void* mask, const float* ln_w, const float* ln_b,
                        uint8_t* ws, const TrWs& w, cudaStream_t s) {
  const uint16_t* zp = static_cast<const uint16_t*>(z);
  const uint16_t* mk = static_cast<const uint16_t*>(mask);
  uint16_t* x = reinterpret_cast<uint16_t*>(ws + w.x);
  float* mean = reinterpret_cast<float*>(ws + w.mean);
  float* rstd = reinterpret_cast<float*>(ws + w.rstd);
  return by_c(d.C, [&](auto ic) {
    constexpr int C = decltype(ic)::value;
    if (mk != nullptr) ln_fwd_kernel<C, true><<<kLnFwdBlocks, 256, 0, s>>>(zp, ln_w, ln_b, x, mean, rstd, d.M, mk);
    else ln_fwd_kernel<C><<<kLnFwdBlocks, 256, 0, s>>>(zp, ln_w, ln_b, x, mean, rstd, d.M);
    return cudaGetLastError();
  });
}

}  // namespace
}  // namespace triattn

using namespace triattn;

extern "C" {

size_t triattn_transition_workspace_bytes(const triattn_transition_shape* shape) {
  if (check_transition(shape) != TRIATTN_OK) return 0;
  return tr_ws(tr_dims(shape)).total;
}

triattn_status triattn_transition_fwd(const triattn_transition_shape* shape, const void* z, const void* mask,
                                      const float* ln_w, const float* ln_b, const void* w_in, const void* w_o,
                                      void* out, void* stream) {
  const triattn_status st = check_transition(shape);
  if (st != TRIATTN_OK) return st;
  if (shape->M == 0) return TRIATTN_OK;
  const void* req[] = {z, ln_w, ln_b, w_in, w_o, out};
  for (const void* q : req)
    if (q == nullptr || !al16(q)) return TRIATTN_ERR_INVALID_ARG;
  if (mask != nullptr && !al2(mask)) return TRIATTN_ERR_INVALID_ARG;
  const TrDims d = tr_dims(shape);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (shape->M <= kTrRowsMax) {
    const cudaError_t e = trace_call(kKTrRows, s, [&] {
      return launch_transition_rows(static_cast<int>(shape->M), d.C, d.H, d.act, z, mask, ln_w, ln_b, w_in, w_o, out,
                                    s);
    });
    return e == cudaSuccess ? TRIATTN_OK : TRIATTN_ERR_CUDA;
  }
  const cudaError_t e = trace_call(kKTrFwd, s, [&] {
    return launch_transition_fwd(shape->M, d.C, d.H, d.act, z, mask, ln_w, ln_b, w_in, w_o, out, current_wait_ctl(),
                                 s);
  });
  return e == cudaSuccess ? TRIATTN_OK : TRIATTN_ERR_CUDA;
}

triattn_status triattn_transition_bwd(const triattn_transition_shape* shape, const void* z, const void* mask,
                                      const float* ln_w, const float* ln_b, const void* w_in, const void* w_o,
                                      const void* d_out, void* dz, void* d_ln_w, void* d_ln_b, void* d_w_in,
                                      void* d_w_o, void* workspace, size_t workspace_bytes, void* stream) {
  const triattn_status st = check_transition(shape);
  if (st != TRIATTN_OK) return st;
  const TrDims d = tr_dims(shape);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const void* par[] = {d_ln_w, d_ln_b, d_w_in, d_w_o};
  for (const void* q : par)
    if (q == nullptr || !al16(q)) return TRIATTN_ERR_INVALID_ARG;
  if (d.M == 0) {  // no rows: the gradients are sums of nothing
    const size_t es = d.bf16 ? 2 : 4;
    const bool ok = cudaMemsetAsync(d_ln_w, 0, es * d.C, s) == cudaSuccess &&
                    cudaMemsetAsync(d_ln_b, 0, es * d.C, s) == cudaSuccess &&
                    cudaMemsetAsync(d_w_in, 0, es * d.C * 2 * d.H, s) == cudaSuccess &&
                    cudaMemsetAsync(d_w_o, 0, es * d.C * d.H, s) == cudaSuccess;
    return ok ? TRIATTN_OK : TRIATTN_ERR_CUDA;
  }
  const void* req[] = {z, ln_w, ln_b, w_in, w_o, d_out, dz};
  for (const void* q : req)
    if (q == nullptr || !al16(q)) return TRIATTN_ERR_INVALID_ARG;
  if (mask != nullptr && !al2(mask)) return TRIATTN_ERR_INVALID_ARG;
  const TrWs w = tr_ws(d);
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < w.total)
    return TRIATTN_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  void* const gws = ws + w.gemm;
  const int M = static_cast<int>(d.M), C = d.C, H = d.H;
  const uint16_t* mk = static_cast<const uint16_t*>(mask);
  uint16_t* P = reinterpret_cast<uint16_t*>(ws + w.P);
  uint16_t* h = reinterpret_cast<uint16_t*>(ws + w.h);
  uint16_t* dh = reinterpret_cast<uint16_t*>(ws + w.dh);
  const void* g = d_out;
  auto gemm = [&](bool ta, bool tb, int m, int n, int k, const void* A, int lda, const void* B, int ldb, void* Cp,
                  int ldc, bool f32) {
    return gemm_traced(kKTrGemm, gws, s, ta, tb, m, n, k, A, lda, B, ldb, Cp, ldc, f32) == TRIATTN_OK;
  };
  SumParams sum = {nullptr, 0, 0, 0, 0u, reinterpret_cast<float*>(ws + w.pg), reinterpret_cast<float*>(ws + w.pb),
                   kLnBlocks, C, d.bf16 ? 1 : 0, d_w_in, d_w_o, d_ln_w, d_ln_b};
  float* pg = reinterpret_cast<float*>(ws + w.pg);
  float* pb = reinterpret_cast<float*>(ws + w.pb);
  auto sums = [&] {
    return trace_call(kKTrColSum, s, [&] {
             transition_sum_kernel<<<sum.wblocks + static_cast<unsigned>(2 * C / 8), 256, 0, s>>>(sum);
             return cudaGetLastError();
           }) == cudaSuccess;
  };
  // Up to 128 features one kernel does everything before the weight gradients.
  // Wider rows of x, g and z do not fit the shared memory beside the weights:
  // there the steps are kernels of their own, with the gating in the epilogue
  // of the recomputed projections.  147456 masked rows, C / H 256 / 1024: 0.95 ms,
  // 4.0 times what the formula's products take at the tensor cores' rate;
  // 192 / 768 0.76 ms, 5.7 times; 160 / 320 0.49 ms, 10 times (the fused path: 3.5
  // times at 128 / 512, 5.6 at 64 / 256).  dh is rounded to BF16 on its way through
  // memory, as an operand of the gating's kernel.
  if (transition_bwd_fused(C)) {
    if (mk != nullptr) g = ws + w.g;
    float* const part = reinterpret_cast<float*>(ws + w.wg);
    if (trace_call(kKTrBwd, s, [&] {
          return launch_transition_bwd(shape->M, C, H, d.act, z, mask, ln_w, ln_b, w_in, w_o, d_out, dz, ws + w.x,
                                       ws + w.g, pg, pb, &sum.rows, current_wait_ctl(), s);
        }) != cudaSuccess ||
        trace_call(kKTrWgrad, s, [&] {
          return launch_transition_wgrad(shape->M, C, H, d.act, ws + w.x, g, w_in, w_o, part, &sum.wparts,
                                         current_wait_ctl(), s);
        }) != cudaSuccess)
      return TRIATTN_ERR_CUDA;
    sum.w = reinterpret_cast<const float4*>(part);
    sum.n_in = static_cast<size_t>(2) * C * H / 4;
    sum.n = static_cast<size_t>(3) * C * H / 4;
    sum.wblocks = static_cast<unsigned>((sum.n + 63) / 64);
    return sums() ? TRIATTN_OK : TRIATTN_ERR_CUDA;
  }
  if (trace_call(kKTrLn, s, [&] { return ln_fwd_rows(d, z, mask, ln_w, ln_b, ws, w, s); }) != cudaSuccess)
    return TRIATTN_ERR_CUDA;
  if (mk != nullptr) {
    g = ws + w.g;
    if (trace_call(kKTrGate, s, [&] {
          mask_rows_kernel<<<grid_for(d.M * C / 8), 256, 0, s>>>(static_cast<const uint16_t*>(d_out), mk,
                                                                 reinterpret_cast<uint16_t*>(ws + w.g), C, d.M);
          return cudaGetLastError();
        }) != cudaSuccess)
      return TRIATTN_ERR_CUDA;
  }
  if (!gemm(false, true, M, H, C, g, C, w_o, C, dh, H, false) ||
      trace_call(kKTrGate, s, [&] {
        return launch_transition_gate(shape->M, C, H, d.act, ws + w.x, w_in, dh, h, P, current_wait_ctl(), s);
      }) != cudaSuccess)
    return TRIATTN_ERR_CUDA;
  if (!gemm(true, false, H, C, M, h, H, g, C, d_w_o, C, !d.bf16) ||
      !gemm(true, false, C, 2 * H, M, ws + w.x, C, P, 2 * H, d_w_in, 2 * H, !d.bf16) ||
      !gemm(false, true, M, C, 2 * H, P, 2 * H, w_in, 2 * H, ws + w.dx, C, true))
    return TRIATTN_ERR_CUDA;
  if (trace_call(kKTrLnBwd, s, [&] {
        return by_c(C, [&](auto ic) {
          constexpr int kC = decltype(ic)::value;
          const uint16_t* zp = static_cast<const uint16_t*>(z);
          const float* dx = reinterpret_cast<const float*>(ws + w.dx);  // not rounded, as in the fused kernel
          const float* mean = reinterpret_cast<const float*>(ws + w.mean);
          const float* rstd = reinterpret_cast<const float*>(ws + w.rstd);
          uint16_t* dzp = static_cast<uint16_t*>(dz);
          if (mk != nullptr)
            ln_bwd_kernel<kC, true, float><<<kLnBlocks, 256, 0, s>>>(zp, dx, ln_w, mean, rstd, dzp, pg, pb, d.M, mk);
          else
            ln_bwd_kernel<kC, false, float><<<kLnBlocks, 256, 0, s>>>(zp, dx, ln_w, mean, rstd, dzp, pg, pb, d.M);
          return cudaGetLastError();
        });
      }) != cudaSuccess)
    return TRIATTN_ERR_CUDA;
  return sums() ? TRIATTN_OK : TRIATTN_ERR_CUDA;
}

}  // extern "C"
