// Global norm of a list of gradient tensors and clipping by it:
//
//   norm = sqrt(sum over tensors, elements of g^2)     or  max |g|
//   coef = min(1, max_norm / (norm + 1e-6)),  g <- coef g   (in place or into other tensors)
//
// for BF16 and FP32 tensors mixed, of any size and any element alignment.
//
// Every tensor is cut into chunks of 32 KB on 16-byte boundaries of the
// address space (the first and last chunk of a tensor may be partly outside
// it); each block of a fixed grid takes a run of consecutive chunks, so a list
// of many small tensors and a few large ones balance the same way, and looks a
// tensor up once, then steps.  The table of a short list travels in the
// kernels' parameters (3 KB), that of a long one is put into the workspace by a
// one-block kernel that has it in its parameters (32 KB, which make a launch
// some 10 us longer, so it is done once and not for both passes); either way
// nothing is copied from the host, nothing is kept between calls, and a
// captured graph holds its own table.
//
// Pass 1 reads every gradient once: a thread adds squares in FP32, in eight
// chains of BF16 or four of FP32 elements; after 64 chunks, 512 squares per
// chain, it joins the chains pairwise and adds them to a total, so that no sum is
// long however large the list (as one chain, 34 GB lose up to 2e-4 of it).  A
// block's threads are added pairwise in FP32 and the blocks' partials in FP64, all
// in fixed order, so the result is bitwise reproducible and uses no atomics.  It is bound by HBM: 480 MB of FP32
// in 72 us (6.7 TB/s).  Pass 2 (clipping only): every
// block adds the same partials in the same order, so no block waits for
// another, and scales its chunks, last chunk first: what pass 1 read last is
// still in L2 (480 MB read and written in 149 us).  In place nothing is
// written when the coefficient is 1.
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
static_assert(152 * 4 % 32 == 0, "the partials by one warp");
constexpr int kGnGrid = 152 * 4;  // largest grid; the partials (and so the order of the sum) depend on it
// Chunks after which a thread puts its chains' sums aside: 512 squares per chain.
constexpr uint64_t kGnFold = 64;
// Longest list whose table is a parameter, and entries that one upload carries.
constexpr int kGnSmall = 96, kGnUpload = 1000;

template <int K>
struct GnTable {
  uint64_t ptr[K];    // gradient
  uint64_t out[K];    // destination of the scaled gradient
  uint64_t numel[K];  // elements; bit 63: FP32
  uint64_t end[K];    // chunks of tensors 0 .. k
  int n;
};
static_assert(sizeof(GnTable<kGnUpload>) + 64 <= 32764, "kernel parameter limit");

// The same arrays in the workspace.
struct GnView {
  uint64_t *ptr, *out, *numel, *end;
  int n;
};

struct GnChunk {
  const uint8_t* p;   // 16-byte aligned start of the chunk
  long long shift;    // destination address minus source address
  long long lo, hi;   // bytes of the chunk that belong to the tensor
  bool f32;
};

__global__ void __launch_bounds__(256) grad_table_kernel(const __grid_constant__ GnTable<kGnUpload> t, GnView v,
                                                         int at) {
  for (int i = threadIdx.x; i < t.n; i += 256) {
    v.ptr[at + i] = t.ptr[i];
    v.out[at + i] = t.out[i];
    v.numel[at + i] = t.numel[i];
    v.end[at + i] = t.end[i];
  }
}

// First tensor whose end is above chunk c, by all lanes of a warp together.
__device__ __forceinline__ int gn_find(const GnView& t, uint64_t c) {
  int lo = 0, n = t.n;  // it is one of [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = static_cast<int>(threadIdx.x & 31) * step;  // the last entry of lane's part, or the last of all
    const int at = lo + min(i + step, n) - 1;
    const uint32_t above = __ballot_sync(0xffffffffu, i >= n || t.end[at] > c);
    const int part = __ffs(above) - 1;
    lo += part * step;
    n = min(step, n - part * step);
  }
  return lo;
}

// The run of chunks [c0, c1) of this block.
__device__ __forceinline__ void gn_run(uint64_t chunks, uint64_t& c0, uint64_t& c1) {
  const uint64_t per = chunks / gridDim.x, more = chunks % gridDim.x, b = blockIdx.x;
  c0 = b * per + (b < more ? b : more);
  c1 = c0 + per + (b < more ? 1 : 0);
}

// Chunk c of tensor k (k the one it belongs to).
__device__ __forceinline__ GnChunk gn_chunk(const GnView& t, int k, uint64_t c) {
  const uint64_t first = k > 0 ? t.end[k - 1] : 0u;
  const uint64_t ne = t.numel[k], ptr = t.ptr[k];
  GnChunk r;
  r.f32 = (ne >> 63) != 0;
  const long long bytes = static_cast<long long>(ne & ~(1ull << 63)) * (r.f32 ? 4 : 2);
  const uint64_t base = ptr & ~uint64_t(15);
  const long long head = static_cast<long long>(ptr - base);
  const long long off = static_cast<long long>(c - first) * kGnChunk;
  r.p = reinterpret_cast<const uint8_t*>(base + off);
  r.lo = max(head - off, 0ll);
  r.hi = min(head + bytes - off, kGnChunk);
  r.shift = static_cast<long long>(t.out[k] - ptr);
  return r;
}
template <bool SMALL>
__device__ __forceinline__ GnView gn_view(const GnTable<kGnSmall>& s, const GnView& v) {
  if constexpr (SMALL)
    return GnView{const_cast<uint64_t*>(s.ptr), const_cast<uint64_t*>(s.out), const_cast<uint64_t*>(s.numel),
                  const_cast<uint64_t*>(s.end), s.n};
  else
    return v;
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

// Two partial values joined: a sum of squares, or a maximum of |g| (NaN above
// everything).
template <typename V>
__device__ __forceinline__ V gn_join(V a, V b, bool inf) {
  if (!inf) return a + b;
  return (a != a || b != b) ? a + b : (a > b ? a : b);
}
template <typename V>
__device__ __forceinline__ V gn_warp(V v, bool inf) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = gn_join(v, __shfl_xor_sync(0xffffffffu, v, off), inf);
  return v;
}

template <bool SMALL>
__global__ void __launch_bounds__(kGnThreads) grad_sum_kernel(const __grid_constant__ GnTable<kGnSmall> small,
                                                              const __grid_constant__ GnView big, uint64_t chunks,
                                                              int inf, float* __restrict__ part) {
  __shared__ float red[kGnThreads / 32];
  const GnView t = gn_view<SMALL>(small, big);
  float acc[8], total = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  auto fold = [&] {  // the thread's chains pairwise, onto its total
#pragma unroll
    for (int n = 4; n > 0; n >>= 1)
#pragma unroll
      for (int e = 0; e < n; ++e) acc[e] = gn_join(acc[e], acc[e + n], inf != 0);
    total = gn_join(total, acc[0], inf != 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  };
  uint64_t c0, c1;
  gn_run(chunks, c0, c1);
  int i = c0 < c1 ? gn_find(t, c0) : 0;
  GnChunk k;
  if (c0 < c1) k = gn_chunk(t, i, c0);
  for (uint64_t c = c0; c < c1; ++c) {
    // the next chunk is looked up while this one's loads are under way
    GnChunk next = k;
    if (k.lo == 0 && k.hi == kGnChunk) {
      uint4 w[kGnUnits];
#pragma unroll
      for (int u = 0; u < kGnUnits; ++u)
        w[u] = __ldg(reinterpret_cast<const uint4*>(k.p) + threadIdx.x + u * kGnThreads);
      if (c + 1 < c1) {
        while (t.end[i] <= c + 1) ++i;
        next = gn_chunk(t, i, c + 1);
      }
#pragma unroll
      for (int u = 0; u < kGnUnits; ++u) gn_add(w[u], k.f32, inf != 0, acc);
    } else {
      if (c + 1 < c1) {
        while (t.end[i] <= c + 1) ++i;
        next = gn_chunk(t, i, c + 1);
      }
#pragma unroll
      for (int u = 0; u < kGnUnits; ++u) {
        const long long at = 16ll * (threadIdx.x + u * kGnThreads);
        if (at + 16 <= k.lo || at >= k.hi) continue;
        const uint4 w = at >= k.lo && at + 16 <= k.hi ? __ldg(reinterpret_cast<const uint4*>(k.p + at))
                                                      : gn_edge(k.p + at, k.lo - at, k.hi - at, k.f32);
        gn_add(w, k.f32, inf != 0, acc);
      }
    }
    k = next;
    if ((c - c0) % kGnFold == kGnFold - 1) fold();
  }
  // the block's 256 threads pairwise in FP32 (at most 11 roundings more)
  fold();
  const float v = gn_warp(total, inf != 0);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    const float s = gn_warp(threadIdx.x < kGnThreads / 32 ? red[threadIdx.x] : 0.f, inf != 0);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
  }
}

// The norm from the blocks' partials, the same in every block: by one warp,
// in FP64 (two adds per clock and SM: with every thread of every block taking
// part, this alone took 20 us).
__device__ float gn_norm(const float* __restrict__ part, int n, bool inf, float* red) {
  if (threadIdx.x < 32) {
    float p[kGnGrid / 32];  // every load under way before the first sum
#pragma unroll
    for (int k = 0; k < kGnGrid / 32; ++k) {
      const int i = threadIdx.x + 32 * k;
      p[k] = i < n ? part[i] : 0.f;
    }
    double v = 0.0;
#pragma unroll
    for (int k = 0; k < kGnGrid / 32; ++k) v = gn_join(v, static_cast<double>(p[k]), inf);
    v = gn_warp(v, inf);
    if (threadIdx.x == 0) *red = static_cast<float>(inf ? v : sqrt(v));
  }
  __syncthreads();
  return *red;
}

__global__ void __launch_bounds__(32) grad_norm_kernel(const float* __restrict__ part, int n, int inf,
                                                       float* __restrict__ norm) {
  __shared__ float red;
  const float v = gn_norm(part, n, inf != 0, &red);
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

template <bool SMALL>
__global__ void __launch_bounds__(kGnThreads) grad_scale_kernel(const __grid_constant__ GnTable<kGnSmall> small,
                                                                const __grid_constant__ GnView big, uint64_t chunks,
                                                                const float* __restrict__ part, int inf,
                                                                float max_norm, int in_place,
                                                                float* __restrict__ norm) {
  __shared__ float red;
  const float nv = gn_norm(part, gridDim.x, inf != 0, &red);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = nv;
  const float q = max_norm / (nv + 1e-6f);
  const float coef = q > 1.f ? 1.f : q;  // NaN stays NaN
  if (in_place && coef == 1.f) return;
  const GnView t = gn_view<SMALL>(small, big);
  uint64_t c0, c1;
  gn_run(chunks, c0, c1);
  int i = c0 < c1 ? gn_find(t, c1 - 1) : 0;
  for (uint64_t c = c1; c-- > c0;) {  // the block's last chunk first: it was read last
    while (i > 0 && t.end[i - 1] > c) --i;
    const GnChunk k = gn_chunk(t, i, c);
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

// Where a call's parts lie in the workspace: the blocks' partials, then the
// table's four columns (long lists).
struct GnWs {
  size_t part, table, total;
};
GnWs gn_ws(long long n) {
  GnWs w;
  w.part = 0;
  w.table = (kGnGrid * sizeof(float) + 255) / 256 * 256;
  w.total = w.table + (n > kGnSmall ? static_cast<size_t>(n) * 4 * sizeof(uint64_t) : 0);
  return w;
}

template <int K>
void gn_entry(GnTable<K>* t, const triattn_tensor& g, const triattn_tensor* out, uint64_t* end) {
  const uint64_t p = reinterpret_cast<uint64_t>(g.data);
  const int k = t->n++;
  t->ptr[k] = p;
  t->out[k] = out != nullptr ? reinterpret_cast<uint64_t>(out->data) : p;
  t->numel[k] = static_cast<uint64_t>(g.numel) | (g.dtype == TRIATTN_DTYPE_FP32 ? 1ull << 63 : 0ull);
  *end += ((p & 15) + gn_bytes(g) + kGnChunk - 1) / kGnChunk;
  t->end[k] = *end;
}

// One call's tables: the list without its empty tensors, in `small` or uploaded.
struct GnCall {
  GnTable<kGnSmall> small;
  GnView big;
  uint64_t chunks;
  bool is_small;
  unsigned grid;  // one block per chunk up to the full grid
  float* part;
};
triattn_status gn_prepare(GnCall* c, const triattn_tensor* ts, const triattn_tensor* out, long long n, void* workspace,
                          cudaStream_t s) {
  const GnWs w = gn_ws(n);
  c->part = static_cast<float*>(workspace);
  c->is_small = n <= kGnSmall;
  c->chunks = 0;
  c->small.n = 0;
  c->big.n = 0;
  if (c->is_small) {
    for (long long i = 0; i < n; ++i)
      if (ts[i].numel > 0) gn_entry(&c->small, ts[i], out != nullptr ? &out[i] : nullptr, &c->chunks);
  } else {
    uint64_t* col = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(workspace) + w.table);
    c->big.ptr = col;
    c->big.out = col + n;
    c->big.numel = col + 2 * n;
    c->big.end = col + 3 * n;
    GnTable<kGnUpload> t;
    for (long long i = 0; i < n;) {
      t.n = 0;
      for (; i < n && t.n < kGnUpload; ++i)
        if (ts[i].numel > 0) gn_entry(&t, ts[i], out != nullptr ? &out[i] : nullptr, &c->chunks);
      if (t.n == 0) break;
      const int at = c->big.n;
      const cudaError_t e = trace_call(kKGradTable, s, [&] {
        grad_table_kernel<<<1, 256, 0, s>>>(t, c->big, at);
        return cudaGetLastError();
      });
      if (e != cudaSuccess) return TRIATTN_ERR_CUDA;
      c->big.n += t.n;
    }
  }
  c->grid = static_cast<unsigned>(std::min<uint64_t>(std::max<uint64_t>(c->chunks, 1), kGnGrid));
  return TRIATTN_OK;
}

triattn_status gn_sum(const GnCall& c, int inf, cudaStream_t s) {
  const cudaError_t e = trace_call(kKGradSum, s, [&] {
    if (c.is_small) grad_sum_kernel<true><<<c.grid, kGnThreads, 0, s>>>(c.small, c.big, c.chunks, inf, c.part);
    else grad_sum_kernel<false><<<c.grid, kGnThreads, 0, s>>>(c.small, c.big, c.chunks, inf, c.part);
    return cudaGetLastError();
  });
  return e == cudaSuccess ? TRIATTN_OK : TRIATTN_ERR_CUDA;
}

triattn_status gn_check_call(const triattn_tensor* ts, long long n, int norm_type, const float* norm,
                             const void* workspace, size_t workspace_bytes) {
  const triattn_status st = gn_check(ts, n);
  if (st != TRIATTN_OK) return st;
  if (norm_type != TRIATTN_NORM_L2 && norm_type != TRIATTN_NORM_MAX) return TRIATTN_ERR_INVALID_ARG;
  if (norm == nullptr || (reinterpret_cast<uintptr_t>(norm) & 3u) != 0) return TRIATTN_ERR_INVALID_ARG;
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < gn_ws(n).total)
    return TRIATTN_ERR_WORKSPACE;
  return TRIATTN_OK;
}

}  // namespace
}  // namespace triattn

using namespace triattn;

extern "C" {

size_t triattn_grad_norm_workspace_bytes(long long n) {
  if (n < 0 || n > (1ll << 24)) return 0;
  return gn_ws(n).total;
}

triattn_status triattn_grad_norm(const triattn_tensor* tensors, long long n, int norm_type, float* norm,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  triattn_status st = gn_check_call(tensors, n, norm_type, norm, workspace, workspace_bytes);
  if (st != TRIATTN_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int inf = norm_type == TRIATTN_NORM_MAX;
  GnCall c;
  if ((st = gn_prepare(&c, tensors, nullptr, n, workspace, s)) != TRIATTN_OK) return st;
  if ((st = gn_sum(c, inf, s)) != TRIATTN_OK) return st;
  const cudaError_t e = trace_call(kKGradNorm, s, [&] {
    grad_norm_kernel<<<1, 32, 0, s>>>(c.part, static_cast<int>(c.grid), inf, norm);
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
  const int inf = norm_type == TRIATTN_NORM_MAX;
  GnCall c;
  if ((st = gn_prepare(&c, tensors, out, n, workspace, s)) != TRIATTN_OK) return st;
  if ((st = gn_sum(c, inf, s)) != TRIATTN_OK) return st;
  const cudaError_t e = trace_call(kKGradScale, s, [&] {
    const int in_place = out == nullptr ? 1 : 0;
    if (c.is_small)
      grad_scale_kernel<true><<<c.grid, kGnThreads, 0, s>>>(c.small, c.big, c.chunks, c.part, inf, max_norm, in_place,
                                                            norm);
    else
      grad_scale_kernel<false><<<c.grid, kGnThreads, 0, s>>>(c.small, c.big, c.chunks, c.part, inf, max_norm, in_place,
                                                             norm);
    return cudaGetLastError();
  });
  return e == cudaSuccess ? TRIATTN_OK : TRIATTN_ERR_CUDA;
}

}  // extern "C"
