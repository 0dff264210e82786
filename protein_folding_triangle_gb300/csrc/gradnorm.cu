// Global norm of a list of gradient tensors and clipping by it:
//
//   norm = sqrt(sum over tensors, elements of g^2)     or  max |g|
//   coef = min(1, max_norm / (norm + 1e-6)),  g <- coef g   (in place or into other tensors)
//
// for BF16 and FP32 tensors mixed, of any size and any element alignment.
//
// Every tensor is cut into chunks of 32 KB on 16-byte boundaries of the
// address space (the first and last chunk of a tensor may be partly outside
// it); a fixed grid walks the chunks of all tensors, so a list of many small
// tensors and a few large ones balance the same way.  The tensor table
// travels in the kernel's parameters: no copy to the device, nothing kept
// between calls, and a captured graph holds its own table.
//
// Pass 1 reads every gradient once: a thread adds squares in FP32 (at most a
// few thousand, eight chains), everything above it (warp, block, the sum of
// the blocks' partials) is added in FP64 in fixed order, so the result is
// bitwise reproducible and uses no atomics.  Pass 2 (clipping only): every
// block adds the same partials in the same order, so no block waits for
// another, and scales its chunks, last chunk first: what pass 1 read last is
// still in L2.  In place nothing is written when the coefficient is 1.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

#include "kernels.cuh"
#include "triattn.h"

namespace triattn {
namespace {

constexpr int kGnThreads = 256;
constexpr int kGnUnits = 8;                                   // 16-byte units per thread and chunk
constexpr long long kGnChunk = 16ll * kGnThreads * kGnUnits;  // 32 KB
constexpr int kGnGrid = 152 * 4;  // largest grid; the partials (and so the order of the sum) depend on it
// Table entries of one launch.  The large table nearly fills the 32,764 bytes
// of kernel parameters; the small one keeps the launch of a short list cheap.
constexpr int kGnSmall = 96, kGnLarge = 1152;

template <int K>
struct GnTable {
  uint64_t ptr[K];    // gradient
  uint64_t out[K];    // destination of the scaled gradient
  uint64_t numel[K];  // elements; bit 63: FP32
  uint32_t end[K];    // chunks of tensors 0 .. k
  int n;
};
static_assert(sizeof(GnTable<kGnLarge>) + 64 <= 32764, "kernel parameter limit");

struct GnChunk {
  const uint8_t* p;   // 16-byte aligned start of the chunk
  long long shift;    // destination address minus source address
  long long lo, hi;   // bytes of the chunk that belong to the tensor
  bool f32;
};

template <int K>
__device__ __forceinline__ GnChunk gn_chunk(const GnTable<K>& t, uint32_t c) {
  int lo = 0, hi = t.n - 1;  // first tensor whose end is above c
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (t.end[mid] > c) hi = mid;
    else lo = mid + 1;
  }
  const uint32_t first = lo > 0 ? t.end[lo - 1] : 0u;
  const uint64_t ne = t.numel[lo];
  GnChunk r;
  r.f32 = (ne >> 63) != 0;
  const long long bytes = static_cast<long long>(ne & ~(1ull << 63)) * (r.f32 ? 4 : 2);
  const uint64_t base = t.ptr[lo] & ~uint64_t(15);
  const long long head = static_cast<long long>(t.ptr[lo] - base);
  const long long off = static_cast<long long>(c - first) * kGnChunk;
  r.p = reinterpret_cast<const uint8_t*>(base + off);
  r.lo = max(head - off, 0ll);
  r.hi = min(head + bytes - off, kGnChunk);
  r.shift = static_cast<long long>(t.out[lo] - t.ptr[lo]);
  return r;
}

// Values of a 16-byte unit: 4 FP32 or 8 BF16.
__device__ __forceinline__ void gn_add(uint4 w, bool f32, bool inf, float (&acc)[8]) {
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (inf) {
      // |g| as integers: the order of the values, with NaN above infinity
      const uint32_t a = f32 ? (ws[e] & 0x7FFFFFFFu) : ((ws[e] << 16) & 0x7FFFFFFFu);
      const uint32_t b = f32 ? 0u : (ws[e] & 0x7FFF0000u);
      acc[e] = __uint_as_float(max(__float_as_uint(acc[e]), max(a, b)));
    } else if (f32) {
      const float v = __uint_as_float(ws[e]);
      acc[e] = fmaf(v, v, acc[e]);
    } else {
      const float a = bf16lo_to_f32(ws[e]), b = bf16hi_to_f32(ws[e]);
      acc[e] = fmaf(a, a, acc[e]);
      acc[4 + e] = fmaf(b, b, acc[4 + e]);
    }
  }
}

// The 16-byte unit at p of which only bytes [lo, hi) belong to the tensor;
// the others read as 0, and are not touched.
__device__ __forceinline__ uint4 gn_edge(const uint8_t* p, long long lo, long long hi, bool f32) {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int at = 2 * e;
    if (f32) {
      if ((e & 1) == 0 && at >= lo && at < hi) w[e >> 1] = *reinterpret_cast<const uint32_t*>(p + at);
    } else if (at >= lo && at < hi) {
      w[e >> 1] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p + at)) << (16 * (e & 1));
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The combined value of all lanes / warps / blocks: a sum of squares, or a
// maximum of |g| (NaN above everything).
__device__ __forceinline__ double gn_join(double a, double b, bool inf) {
  if (!inf) return a + b;
  return (isnan(a) || isnan(b)) ? nan("") : fmax(a, b);
}
__device__ double gn_block(double v, bool inf, double* red) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = gn_join(v, __shfl_xor_sync(0xffffffffu, v, off), inf);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = red[0];
#pragma unroll
  for (int w = 1; w < kGnThreads / 32; ++w) s = gn_join(s, red[w], inf);
  return s;
}

template <int K>
__global__ void __launch_bounds__(kGnThreads) grad_sum_kernel(const __grid_constant__ GnTable<K> t, int inf,
                                                              double* __restrict__ part) {
  __shared__ double red[kGnThreads / 32];
  const uint32_t chunks = t.n > 0 ? t.end[t.n - 1] : 0u;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const GnChunk k = gn_chunk(t, c);
    if (k.lo == 0 && k.hi == kGnChunk) {
      uint4 w[kGnUnits];
#pragma unroll
      for (int u = 0; u < kGnUnits; ++u)
        w[u] = __ldg(reinterpret_cast<const uint4*>(k.p) + threadIdx.x + u * kGnThreads);
#pragma unroll
      for (int u = 0; u < kGnUnits; ++u) gn_add(w[u], k.f32, inf != 0, acc);
    } else {
#pragma unroll
      for (int u = 0; u < kGnUnits; ++u) {
        const long long at = 16ll * (threadIdx.x + u * kGnThreads);
        if (at + 16 <= k.lo || at >= k.hi) continue;
        const uint4 w = at >= k.lo && at + 16 <= k.hi ? __ldg(reinterpret_cast<const uint4*>(k.p + at))
                                                      : gn_edge(k.p + at, k.lo - at, k.hi - at, k.f32);
        gn_add(w, k.f32, inf != 0, acc);
      }
    }
  }
  double v = acc[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) v = gn_join(v, acc[e], inf != 0);
  v = gn_block(v, inf != 0, red);
  if (threadIdx.x == 0) part[blockIdx.x] = v;
}

// The norm from the partials of every launch, the same in every block.
__device__ float gn_norm(const double* __restrict__ part, int n, bool inf, double* red) {
  double v = 0.0;
  for (int i = threadIdx.x; i < n; i += kGnThreads) v = gn_join(v, part[i], inf);
  v = gn_block(v, inf, red);
  return static_cast<float>(inf ? v : sqrt(v));
}

__global__ void __launch_bounds__(kGnThreads) grad_norm_kernel(const double* __restrict__ part, int n, int inf,
                                                               float* __restrict__ norm) {
  __shared__ double red[kGnThreads / 32];
  const float v = gn_norm(part, n, inf != 0, red);
  if (threadIdx.x == 0) *norm = v;
}

__device__ __forceinline__ uint4 gn_scale(uint4 w, float c, bool f32) {
  uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    ws[e] = f32 ? __float_as_uint(__uint_as_float(ws[e]) * c)
                : pack_bf16x2(bf16lo_to_f32(ws[e]) * c, bf16hi_to_f32(ws[e]) * c);
  return make_uint4(ws[0], ws[1], ws[2], ws[3]);
}

// The elements of a unit that lie in [lo, hi), stored one by one.
__device__ __forceinline__ void gn_store_edge(uint8_t* p, uint4 w, long long lo, long long hi, bool f32) {
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int at = 2 * e;
    if (at < lo || at >= hi) continue;
    if (f32) {
      if ((e & 1) == 0) *reinterpret_cast<uint32_t*>(p + at) = ws[e >> 1];
    } else {
      *reinterpret_cast<uint16_t*>(p + at) = static_cast<uint16_t>(ws[e >> 1] >> (16 * (e & 1)));
    }
  }
}

template <int K>
__global__ void __launch_bounds__(kGnThreads) grad_scale_kernel(const __grid_constant__ GnTable<K> t,
                                                                const double* __restrict__ part, int nparts, int inf,
                                                                float max_norm, int in_place,
                                                                float* __restrict__ norm) {
  __shared__ double red[kGnThreads / 32];
  const float nv = gn_norm(part, nparts, inf != 0, red);
  if (blockIdx.x == 0 && threadIdx.x == 0 && norm != nullptr) *norm = nv;
  const float q = max_norm / (nv + 1e-6f);
  const float coef = q > 1.f ? 1.f : q;  // NaN stays NaN
  if (in_place && coef == 1.f) return;
  const uint32_t chunks = t.n > 0 ? t.end[t.n - 1] : 0u;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const GnChunk k = gn_chunk(t, chunks - 1 - c);
    const bool vec = (k.shift & 15) == 0;  // source and destination units coincide
    uint8_t* dst = const_cast<uint8_t*>(k.p) + k.shift;
    if (vec && k.lo == 0 && k.hi == kGnChunk) {
      uint4 w[kGnUnits];
#pragma unroll
      for (int u = 0; u < kGnUnits; ++u)
        w[u] = reinterpret_cast<const uint4*>(k.p)[threadIdx.x + u * kGnThreads];
#pragma unroll
      for (int u = 0; u < kGnUnits; ++u)
        reinterpret_cast<uint4*>(dst)[threadIdx.x + u * kGnThreads] = gn_scale(w[u], coef, k.f32);
    } else {
#pragma unroll
      for (int u = 0; u < kGnUnits; ++u) {
        const long long at = 16ll * (threadIdx.x + u * kGnThreads);
        if (at + 16 <= k.lo || at >= k.hi) continue;
        const bool whole = at >= k.lo && at + 16 <= k.hi;
        const uint4 w = gn_scale(whole ? *reinterpret_cast<const uint4*>(k.p + at)
                                       : gn_edge(k.p + at, k.lo - at, k.hi - at, k.f32),
                                 coef, k.f32);
        if (whole && vec) *reinterpret_cast<uint4*>(dst + at) = w;
        else gn_store_edge(dst + at, w, k.lo - at, k.hi - at, k.f32);
      }
    }
  }
}

// ---------------------------------------------------------------- host side
int gn_launches(long long n) { return static_cast<int>((n + kGnLarge - 1) / kGnLarge); }

long long gn_bytes(const triattn_tensor& t) { return t.numel * (t.dtype == TRIATTN_DTYPE_FP32 ? 4 : 2); }

triattn_status gn_check(const triattn_tensor* ts, long long n) {
  if (n < 0 || n > (1ll << 24) || (n > 0 && ts == nullptr)) return TRIATTN_ERR_INVALID_ARG;
  for (long long i = 0; i < n; ++i) {
    const triattn_tensor& t = ts[i];
    if (t.dtype != TRIATTN_DTYPE_BF16 && t.dtype != TRIATTN_DTYPE_FP32) return TRIATTN_ERR_UNSUPPORTED;
    if (t.numel < 0) return TRIATTN_ERR_INVALID_ARG;
    if (t.numel == 0) continue;
    const uintptr_t es = t.dtype == TRIATTN_DTYPE_FP32 ? 4 : 2;
    if (t.data == nullptr || (reinterpret_cast<uintptr_t>(t.data) & (es - 1)) != 0) return TRIATTN_ERR_INVALID_ARG;
    // chunks are counted in 32 bits over one launch's tensors
    if (t.numel >= (1ll << 40)) return TRIATTN_ERR_UNSUPPORTED;
  }
  return TRIATTN_OK;
}

struct Span {
  uintptr_t lo, hi;
};
// The bytes of every tensor, by address (views of one buffer mostly come in order).
std::vector<Span> gn_spans(const triattn_tensor* ts, long long n) {
  std::vector<Span> v;
  v.reserve(static_cast<size_t>(n));
  for (long long i = 0; i < n; ++i)
    if (ts[i].numel > 0) {
      const uintptr_t lo = reinterpret_cast<uintptr_t>(ts[i].data);
      v.push_back({lo, lo + static_cast<uintptr_t>(gn_bytes(ts[i]))});
    }
  const auto less = [](const Span& a, const Span& b) { return a.lo < b.lo; };
  if (!std::is_sorted(v.begin(), v.end(), less)) std::sort(v.begin(), v.end(), less);
  return v;
}

// Table of tensors [i0, i1); false if their chunks exceed 32 bits.
template <int K>
bool gn_fill(GnTable<K>* t, const triattn_tensor* ts, const triattn_tensor* out, long long i0, long long i1) {
  t->n = 0;
  uint64_t end = 0;
  for (long long i = i0; i < i1; ++i) {
    if (ts[i].numel == 0) continue;
    const uint64_t p = reinterpret_cast<uint64_t>(ts[i].data);
    const int k = t->n++;
    t->ptr[k] = p;
    t->out[k] = out != nullptr ? reinterpret_cast<uint64_t>(out[i].data) : p;
    t->numel[k] = static_cast<uint64_t>(ts[i].numel) | (ts[i].dtype == TRIATTN_DTYPE_FP32 ? 1ull << 63 : 0ull);
    end += ((p & 15) + gn_bytes(ts[i]) + kGnChunk - 1) / kGnChunk;
    if (end > 0x7fffffffull) return false;
    t->end[k] = static_cast<uint32_t>(end);
  }
  return true;
}

// Blocks of a launch: one per chunk up to the full grid.  Several launches
// leave kGnGrid partials each, a single one as many as it has blocks.
template <int K>
unsigned gn_blocks(const GnTable<K>& t) {
  const uint32_t chunks = t.n > 0 ? t.end[t.n - 1] : 1u;
  return std::min<uint32_t>(chunks, kGnGrid);
}

template <int K, bool SCALE>
triattn_status gn_launch(const triattn_tensor* ts, const triattn_tensor* out, long long i0, long long i1, int inf,
                         double* part, int launches, float max_norm, float* norm, cudaStream_t s) {
  GnTable<K> t;
  if (!gn_fill(&t, ts, out, i0, i1)) return TRIATTN_ERR_UNSUPPORTED;
  const unsigned grid = gn_blocks(t);
  const cudaError_t e = trace_call(SCALE ? kKGradScale : kKGradSum, s, [&] {
    if constexpr (SCALE)
      grad_scale_kernel<K><<<grid, kGnThreads, 0, s>>>(t, part, launches > 1 ? launches * kGnGrid : grid, inf, max_norm,
                                                       out == nullptr ? 1 : 0, norm);
    else
      grad_sum_kernel<K><<<launches > 1 ? kGnGrid : grid, kGnThreads, 0, s>>>(t, inf, part);
    return cudaGetLastError();
  });
  return e == cudaSuccess ? TRIATTN_OK : TRIATTN_ERR_CUDA;
}

template <bool SCALE>
triattn_status gn_pass(const triattn_tensor* ts, const triattn_tensor* out, long long n, int inf, double* part,
                       float max_norm, float* norm, cudaStream_t s) {
  const int L = gn_launches(n);
  for (int j = 0; j < L; ++j) {
    const int l = SCALE ? L - 1 - j : j;  // the last tensors read first: they are in L2
    const long long i0 = static_cast<long long>(l) * kGnLarge, i1 = std::min<long long>(n, i0 + kGnLarge);
    double* p = SCALE ? part : part + static_cast<size_t>(l) * kGnGrid;
    float* nm = j == 0 ? norm : nullptr;
    const triattn_status st = i1 - i0 <= kGnSmall
                                  ? gn_launch<kGnSmall, SCALE>(ts, out, i0, i1, inf, p, L, max_norm, nm, s)
                                  : gn_launch<kGnLarge, SCALE>(ts, out, i0, i1, inf, p, L, max_norm, nm, s);
    if (st != TRIATTN_OK) return st;
  }
  return TRIATTN_OK;
}

// Partials that a single launch over these tensors leaves.
int gn_single_parts(const triattn_tensor* ts, long long n) {
  uint64_t chunks = 0;
  for (long long i = 0; i < n; ++i)
    if (ts[i].numel > 0)
      chunks += ((reinterpret_cast<uint64_t>(ts[i].data) & 15) + gn_bytes(ts[i]) + kGnChunk - 1) / kGnChunk;
  return static_cast<int>(std::min<uint64_t>(std::max<uint64_t>(chunks, 1), kGnGrid));
}

triattn_status gn_check_call(const triattn_tensor* ts, long long n, int norm_type, const float* norm,
                             const void* workspace, size_t workspace_bytes) {
  const triattn_status st = gn_check(ts, n);
  if (st != TRIATTN_OK) return st;
  if (norm_type != TRIATTN_NORM_L2 && norm_type != TRIATTN_NORM_MAX) return TRIATTN_ERR_INVALID_ARG;
  if (norm == nullptr || (reinterpret_cast<uintptr_t>(norm) & 3u) != 0) return TRIATTN_ERR_INVALID_ARG;
  if (n > 0 && (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
                workspace_bytes < triattn_grad_norm_workspace_bytes(n)))
    return TRIATTN_ERR_WORKSPACE;
  // every launch's chunk count fits before the first launch
  for (long long i0 = 0; i0 < n; i0 += kGnLarge) {
    uint64_t chunks = 0;
    for (long long i = i0; i < std::min<long long>(n, i0 + kGnLarge); ++i)
      chunks += (static_cast<uint64_t>(gn_bytes(ts[i])) + 15) / kGnChunk + 1;
    if (chunks > 0x7fffffffull) return TRIATTN_ERR_UNSUPPORTED;
  }
  return TRIATTN_OK;
}

}  // namespace
}  // namespace triattn

using namespace triattn;

extern "C" {

size_t triattn_grad_norm_workspace_bytes(long long n) {
  if (n < 0 || n > (1ll << 24)) return 0;
  return static_cast<size_t>(gn_launches(n)) * kGnGrid * sizeof(double);
}

triattn_status triattn_grad_norm(const triattn_tensor* tensors, long long n, int norm_type, float* norm,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  triattn_status st = gn_check_call(tensors, n, norm_type, norm, workspace, workspace_bytes);
  if (st != TRIATTN_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(workspace);
  const int inf = norm_type == TRIATTN_NORM_MAX;
  if ((st = gn_pass<false>(tensors, nullptr, n, inf, part, 0.f, nullptr, s)) != TRIATTN_OK) return st;
  const int nparts = gn_launches(n) == 1 ? gn_single_parts(tensors, n) : gn_launches(n) * kGnGrid;
  const cudaError_t e = trace_call(kKGradNorm, s, [&] {
    grad_norm_kernel<<<1, kGnThreads, 0, s>>>(part, nparts, inf, norm);
    return cudaGetLastError();
  });
  return e == cudaSuccess ? TRIATTN_OK : TRIATTN_ERR_CUDA;
}

triattn_status triattn_clip_grad_norm(const triattn_tensor* tensors, const triattn_tensor* out, long long n,
                                      int norm_type, float max_norm, float* norm, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  triattn_status st = gn_check_call(tensors, n, norm_type, norm, workspace, workspace_bytes);
  if (st != TRIATTN_OK) return st;
  if (!(max_norm >= 0.f)) return TRIATTN_ERR_INVALID_ARG;
  if (out != nullptr) {
    if ((st = gn_check(out, n)) != TRIATTN_OK) return st;
    for (long long i = 0; i < n; ++i)
      if (out[i].numel != tensors[i].numel || out[i].dtype != tensors[i].dtype) return TRIATTN_ERR_INVALID_ARG;
  }
  // Tensors that are written may share no byte with another one: each element
  // is scaled by one thread, without an order between them.  Sources may
  // overlap one another where they are only read.
  try {
    std::vector<Span> dst = gn_spans(out != nullptr ? out : tensors, n);
    for (size_t i = 1; i < dst.size(); ++i)
      if (dst[i].lo < dst[i - 1].hi) return TRIATTN_ERR_INVALID_ARG;
    if (out != nullptr) {
      const std::vector<Span> src = gn_spans(tensors, n);
      size_t k = 0;  // the first destination that ends above the source's start (they are disjoint)
      for (const Span& a : src) {
        while (k < dst.size() && dst[k].hi <= a.lo) ++k;
        if (k < dst.size() && dst[k].lo < a.hi) return TRIATTN_ERR_INVALID_ARG;
      }
    }
  } catch (const std::bad_alloc&) {
    return TRIATTN_ERR_WORKSPACE;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(workspace);
  const int inf = norm_type == TRIATTN_NORM_MAX;
  if (n == 0) {
    const cudaError_t e = trace_call(kKGradNorm, s, [&] {
      grad_norm_kernel<<<1, kGnThreads, 0, s>>>(part, 0, inf, norm);
      return cudaGetLastError();
    });
    return e == cudaSuccess ? TRIATTN_OK : TRIATTN_ERR_CUDA;
  }
  if ((st = gn_pass<false>(tensors, nullptr, n, inf, part, 0.f, nullptr, s)) != TRIATTN_OK) return st;
  return gn_pass<true>(tensors, out, n, inf, part, max_norm, norm, s);
}

}  // extern "C"
