// Learned relative position bias by buckets, and its gradient:
//
//   out[pair] = base[pair] + table[bucket(i, j)],  d_table[k] = sum of d_out over the pairs of bucket k
//
// for the planes of the attention core's bias [B, F, N, N] ("heads") and for the
// pair features [B, N, N, F] ("pairs").  The bucket of a pair is a function of
// the difference of two positions, cut off at +-R, or one row for all pairs of
// different chains.  The function travels with the launch as a list of 2 R + 1
// bytes made on the host, so clipped and logarithmic buckets are one code path
// and the borders of the logarithmic ones are exact.
//
// The forward is bound by HBM (2 bytes in, 2 out, an element); so is the
// gradient (2 or 4 bytes in).  What costs is finding the buckets: the planes'
// forward shares them between four heads, the planes' gradient recognises
// runs of eight elements of one bucket from the smallest and largest position
// among them, and the pair features' gradient is a product with a one-hot
// matrix on the tensor cores (relpos_pairs.cu).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "kernels.cuh"
#include "relpos.cuh"
#include "triattn.h"

namespace triattn {
namespace {

constexpr int kThreads = 256;
constexpr int kHeadGroup = 4;

// Places in shared memory, one word more every 32: lanes that read every
// eighth place meet in no bank.
__host__ __device__ constexpr int spread(int x) { return x + (x >> 5); }

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16lo_to_f32(w[i]);
    f[2 * i + 1] = bf16hi_to_f32(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// The planes' rows need not start on 16 bytes: chunk t of a row is the t-th
// aligned group of eight elements that holds elements of the row, [8 t - off,
// 8 t - off + 8) of it, off the place of the row's start in its group.
__host__ __device__ constexpr int chunks_of(int N) { return N % 8 == 0 ? N / 8 : (N + 14) / 8; }

// ------------------------------------------------------- planes, forward
// Block: a run of rows i of one example and G heads; thread: a chunk of eight
// columns.  The values of every bucket lie in shared memory by distance.
template <int G>
__global__ void __launch_bounds__(kThreads) relpos_heads_fwd_kernel(const __grid_constant__ RelposArgs a, int rows) {
  extern __shared__ float sh[];
  const int W = spread(2 * a.R + 1) + 1, NP = spread(a.N - 1) + 1;
  float* val = sh;                                   // [G][W]: distance + R, then the other chains' value
  int* pos = reinterpret_cast<int*>(val + G * W);    // [NP]
  int* chain = pos + NP;                             // [NP], with chains
  const int groups = (a.F + G - 1) / G, b = blockIdx.y / groups, h0 = (blockIdx.y % groups) * G;
  for (int d = threadIdx.x; d <= 2 * a.R + 1; d += kThreads) {
    const int k = d <= 2 * a.R ? a.lut[d] : a.buckets - 1;
#pragma unroll
    for (int g = 0; g < G; ++g)
      if (h0 + g < a.F) val[g * W + spread(d)] = a.table[static_cast<size_t>(k) * a.F + h0 + g];
  }
  for (int n = threadIdx.x; n < a.N; n += kThreads) {
    pos[spread(n)] = a.position(b, n);
    if (a.chain != nullptr) chain[spread(n)] = __ldg(a.chain + static_cast<size_t>(b) * a.N + n);
  }
  __syncthreads();
  const int nt = chunks_of(a.N);
  const int i0 = blockIdx.x * rows, items = (min(i0 + rows, a.N) - i0) * nt;
  const size_t plane = static_cast<size_t>(a.N) * a.N;
  for (int it = threadIdx.x; it < items; it += kThreads) {
    const int r = it / nt, i = i0 + r, t = it - r * nt;
    const size_t row = ((static_cast<size_t>(b) * a.F + h0) * a.N + i) * a.N;
    const int off = G == 1 ? static_cast<int>(row & 7) : 0;  // G > 1: rows start on 16 bytes
    const int j0 = 8 * t - off;
    const int pi = pos[spread(i)], ci = a.chain != nullptr ? chain[spread(i)] : 0;
    const bool whole = j0 >= 0 && j0 + 8 <= a.N;
    uint4 in[G];
    if (a.base != nullptr && whole) {
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (h0 + g < a.F) in[g] = *reinterpret_cast<const uint4*>(a.base + row + g * plane + j0);
    }
    int at[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int j = min(max(j0 + k, 0), a.N - 1);
      at[k] = distance(pi, pos[spread(j)], a.R);
      if (a.chain != nullptr && chain[spread(j)] != ci) at[k] = 2 * a.R + 1;
      at[k] = spread(at[k]);
    }
    if (whole) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (h0 + g >= a.F) break;
        float v[8];
        if (a.base != nullptr) unpack8(in[g], v);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = (a.base != nullptr ? v[k] : 0.f) + val[g * W + at[k]];
        *reinterpret_cast<uint4*>(a.out + row + g * plane + j0) = pack8(v);
      }
    } else {  // the ends of a row (G == 1), element by element
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = j0 + k;
        if (j < 0 || j >= a.N) continue;
        const float v = (a.base != nullptr ? bf16lo_to_f32(a.base[row + j]) : 0.f) + val[at[k]];
        a.out[row + j] = static_cast<uint16_t>(pack_bf16x2(v, 0.f) & 0xFFFFu);
      }
    }
  }
}

// ------------------------------------------------ pair features, forward
// Block: a run of segments of a row (b, i), as many as any other block's or one
// more; thread: eight features of four pairs of a segment, all four in flight.
// The table comes from L1.
constexpr int kPairsU = 4;
int pairs_threads(int F) { return kThreads / (F / 8) * (F / 8); }
int pairs_segment(int F) { return kPairsU * (kThreads / (F / 8)); }
__global__ void __launch_bounds__(kThreads) relpos_pairs_fwd_kernel(const __grid_constant__ RelposArgs a) {
  constexpr int U = kPairsU;
  __shared__ uint8_t lut[2 * kRelposMaxDistance + 1];
  for (int d = threadIdx.x; d <= 2 * a.R; d += blockDim.x) lut[d] = a.lut[d];
  __syncthreads();
  const int per = a.F / 8, f = (threadIdx.x % per) * 8, jt = threadIdx.x / per, step = blockDim.x / per;
  const int len = U * step, segs = (a.N + len - 1) / len;
  const long long all = static_cast<long long>(a.B) * a.N * segs;
  const long long s0 = all * blockIdx.x / gridDim.x, s1 = all * (blockIdx.x + 1) / gridDim.x;
  long long r = s0 / segs;
  int seg = static_cast<int>(s0 - r * segs);
  for (long long s = s0; s < s1; ++s) {
    const int b = static_cast<int>(r / a.N), i = static_cast<int>(r - static_cast<long long>(b) * a.N);
    const int pi = a.position(b, i);
    const int* chain = a.chain != nullptr ? a.chain + static_cast<size_t>(b) * a.N : nullptr;
    const int ci = chain != nullptr ? __ldg(chain + i) : 0;
    const size_t row = static_cast<size_t>(r) * a.N;
    uint4 in[U];
    int k[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = seg * len + u * step + jt;
      if (j >= a.N) break;
      if (a.base != nullptr) in[u] = *reinterpret_cast<const uint4*>(a.base + (row + j) * a.F + f);
      k[u] = chain != nullptr && __ldg(chain + j) != ci ? a.buckets - 1 : lut[distance(pi, a.position(b, j), a.R)];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = seg * len + u * step + jt;
      if (j >= a.N) break;
      const float4* e = reinterpret_cast<const float4*>(a.table + static_cast<size_t>(k[u]) * a.F + f);
      const float4 e0 = __ldg(e), e1 = __ldg(e + 1);
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (a.base != nullptr) unpack8(in[u], v);
      v[0] += e0.x;
      v[1] += e0.y;
      v[2] += e0.z;
      v[3] += e0.w;
      v[4] += e1.x;
      v[5] += e1.y;
      v[6] += e1.z;
      v[7] += e1.w;
      *reinterpret_cast<uint4*>(a.out + (row + j) * a.F + f) = pack8(v);
    }
    if (++seg == segs) {
      seg = 0;
      ++r;
    }
  }
}

// ------------------------------------------------------ planes, gradient
__device__ __forceinline__ void load8(const uint16_t* p, uint4 (&v)[1]) { v[0] = __ldg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ void load8(const float* p, uint4 (&v)[2]) {
  v[0] = __ldg(reinterpret_cast<const uint4*>(p));
  v[1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
}
__device__ __forceinline__ void values(const uint4 (&v)[1], float (&f)[8]) { unpack8(v[0], f); }
__device__ __forceinline__ void values(const uint4 (&v)[2], float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[4 * i] = __uint_as_float(v[i].x);
    f[4 * i + 1] = __uint_as_float(v[i].y);
    f[4 * i + 2] = __uint_as_float(v[i].z);
    f[4 * i + 3] = __uint_as_float(v[i].w);
  }
}
__device__ __forceinline__ float value(uint16_t v) { return bf16lo_to_f32(v); }
__device__ __forceinline__ float value(float v) { return v; }

// Block: a run of rows of one plane, a row per warp; lane: every 32nd chunk of
// eight columns, four in flight.  A chunk's positions are known by their smallest
// and largest (kept per chunk in shared memory): where both give one bucket (all
// but the pairs near the diagonal), the eight elements are added at once, the
// buckets of the far ends and of other chains in registers.  Everything else
// goes to a place of the lane's own (bucket by lane of its warp) in shared memory:
// no two threads share a sum, so the order is fixed.  The diagonal crosses a
// different chunk in every row, and every warp meets it as often as the others.
struct Window {
  int lo, hi, chain;  // positions of the chunk's columns; its chain
  int one;            // all of one chain
};
template <typename T>
__global__ void __launch_bounds__(kThreads) relpos_heads_bwd_kernel(const __grid_constant__ RelposArgs a, const T* d_out,
                                                                    int rows) {
  constexpr int U = 4;                  // chunks in flight
  constexpr int V = sizeof(T) / 2;      // 16-byte pieces of a chunk
  extern __shared__ float sh[];         // windows [chunks], sums [warps][buckets][32]
  __shared__ uint8_t lut[2 * kRelposMaxDistance + 1];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, nw = blockDim.x / 32;
  const int nt = chunks_of(a.N), b = blockIdx.y / a.F;
  Window* win = reinterpret_cast<Window*>(sh);
  float* hist = sh + 4 * nt;
  const int* chain = a.chain != nullptr ? a.chain + static_cast<size_t>(b) * a.N : nullptr;
  for (int d = threadIdx.x; d <= 2 * a.R; d += blockDim.x) lut[d] = a.lut[d];
  for (int e = threadIdx.x; e < nw * a.buckets * 32; e += blockDim.x) hist[e] = 0.f;
  for (int t = threadIdx.x; t < nt; t += blockDim.x) {
    // all columns that the chunk can hold, whatever its rows' alignment
    const int ja = max(0, a.N % 8 == 0 ? 8 * t : 8 * t - 7), jb = min(a.N, 8 * t + 8);
    Window w{0x7fffffff, -0x7fffffff - 1, chain != nullptr ? __ldg(chain + ja) : 0, 1};
    for (int j = ja; j < jb; ++j) {
      const int p = a.position(b, j);
      w.lo = min(w.lo, p);
      w.hi = max(w.hi, p);
      if (chain != nullptr && __ldg(chain + j) != w.chain) w.one = 0;
    }
    win[t] = w;
  }
  __syncthreads();
  float* mine = hist + warp * a.buckets * 32 + lane;
  const size_t plane = static_cast<size_t>(a.N) * a.N, p0 = blockIdx.y * plane;
  const size_t total = static_cast<size_t>(a.B) * a.F * plane;
  const int kl = lut[0], kh = lut[2 * a.R], ko = a.buckets - 1;  // far on either side, other chains
  float sl = 0.f, sh_ = 0.f, so = 0.f;
  const int i1 = min((static_cast<int>(blockIdx.x) + 1) * rows, a.N);
  for (int i = blockIdx.x * rows + warp; i < i1; i += nw) {
    const size_t s = p0 + static_cast<size_t>(i) * a.N;
    const int off = static_cast<int>(s & 7);
    const int pi = a.position(b, i), ci = chain != nullptr ? __ldg(chain + i) : 0;
    for (int t = lane; t < nt; t += U * 32) {
      uint4 raw[U][V];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const size_t e = s - off + 8 * static_cast<size_t>(t + 32 * u);
        if (t + 32 * u < nt && e + 8 <= total) load8(d_out + e, raw[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int tu = t + 32 * u, j0 = 8 * tu - off;
        if (tu >= nt || j0 >= a.N) break;
        float v[8];
        if (j0 >= 0 && j0 + 8 <= a.N) {
          values(raw[u], v);
        } else {  // the ends of a row: what lies outside it counts as zero
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = j0 + k >= 0 && j0 + k < a.N ? value(d_out[s + j0 + k]) : 0.f;
        }
        const Window w = win[tu];
        int ka = ko, kb = ko;
        if (w.chain == ci || !w.one) {
          ka = lut[distance(pi, w.hi, a.R)];
          kb = lut[distance(pi, w.lo, a.R)];
        }
        if (w.one && ka == kb) {
          const float x = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
          if (ka == kl) sl += x;
          else if (ka == kh) sh_ += x;
          else if (ka == ko) so += x;
          else mine[ka * 32] += x;
        } else {
          int kk[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int j = min(max(j0 + k, 0), a.N - 1);
            kk[k] = chain != nullptr && __ldg(chain + j) != ci ? ko : lut[distance(pi, a.position(b, j), a.R)];
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) mine[kk[k] * 32] += v[k];
        }
      }
    }
  }
  mine[kl * 32] += sl;
  mine[kh * 32] += sh_;
  mine[ko * 32] += so;
  __syncthreads();
  float* out = a.part + (static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x) * a.buckets;
  for (int k = warp; k < a.buckets; k += nw) {
    float v = 0.f;
    for (int w = 0; w < nw; ++w) v += hist[(w * a.buckets + k) * 32 + lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) out[k] = v;
  }
}

// out[y * oy + x * ox] = sum over (b, s) of part[b * pb + s * ps + y * py + x], 32 x by 32 slices
// of the sum per block, joined in a fixed order.
__global__ void __launch_bounds__(1024) relpos_sum_kernel(const float* __restrict__ part, float* __restrict__ out,
                                                          int nx, int ox, int oy, int nb, int ns, size_t pb, size_t ps,
                                                          size_t py) {
  __shared__ double sh[32][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5, x = blockIdx.x * 32 + lane;
  double v = 0.0;
  if (x < nx)
    for (int e = slice; e < nb * ns; e += 32) {
      const int b = e / ns, s = e - b * ns;
      v += part[b * pb + s * ps + blockIdx.y * py + x];
    }
  sh[slice][lane] = v;
  __syncthreads();
  if (slice == 0 && x < nx) {
    v = 0.0;
    for (int s = 0; s < 32; ++s) v += sh[s][lane];
    out[static_cast<size_t>(blockIdx.y) * oy + static_cast<size_t>(x) * ox] = static_cast<float>(v);
  }
}

// ------------------------------------------------------------------ host
// The table's row of every distance in [-R, R].
void fill_lut(const triattn_relpos_shape* s, bool chains, uint8_t* lut) {
  const int R = s->max_distance;
  if (s->kind == TRIATTN_BUCKETS_CLIP) {
    for (int d = -R; d <= R; ++d) lut[d + R] = static_cast<uint8_t>(d + R);
    return;
  }
  const int half = (s->buckets - (chains ? 1 : 0)) / 2, exact = half / 2;
  for (int m = 0; m <= R; ++m) {
    int k = m;
    if (m >= exact) {
      // the logarithm of a border is a whole number up to its rounding
      const double f = std::log(static_cast<double>(m) / exact) / std::log(static_cast<double>(R) / exact);
      k = std::min(half - 1, exact + static_cast<int>(std::floor(f * (half - exact) + 1e-9)));
    }
    lut[R + m] = static_cast<uint8_t>(k);
    if (m > 0) lut[R - m] = static_cast<uint8_t>(half + k);
  }
}

triattn_status check_shape(const triattn_relpos_shape* s) {
  if (s == nullptr || s->B < 1 || s->N < 1 || s->F < 1 || s->buckets < 1 || s->max_distance < 1)
    return TRIATTN_ERR_INVALID_ARG;
  if (s->layout != TRIATTN_RELPOS_HEADS && s->layout != TRIATTN_RELPOS_PAIRS) return TRIATTN_ERR_INVALID_ARG;
  if (s->kind != TRIATTN_BUCKETS_CLIP && s->kind != TRIATTN_BUCKETS_LOG) return TRIATTN_ERR_INVALID_ARG;
  if ((s->flags & ~TRIATTN_FLAG_DOUT_FP32) != 0) return TRIATTN_ERR_INVALID_ARG;
  if ((s->flags & TRIATTN_FLAG_DOUT_FP32) != 0 && s->layout == TRIATTN_RELPOS_PAIRS) return TRIATTN_ERR_UNSUPPORTED;
  if (s->buckets > kRelposMaxBuckets || s->max_distance > kRelposMaxDistance || s->N > kRelposMaxN)
    return TRIATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(s->B) * s->N * s->N >= (1ll << 31)) return TRIATTN_ERR_UNSUPPORTED;
  if (s->layout == TRIATTN_RELPOS_HEADS && static_cast<long long>(s->B) * s->F > 65535) return TRIATTN_ERR_UNSUPPORTED;
  if (s->layout == TRIATTN_RELPOS_PAIRS && (s->F % 8 != 0 || s->F > kRelposMaxF)) return TRIATTN_ERR_UNSUPPORTED;
  return TRIATTN_OK;
}
// The table's rows against the rule, with or without the row of other chains.
bool rule_ok(const triattn_relpos_shape* s, bool chains) {
  const int n = s->buckets - (chains ? 1 : 0);
  if (s->kind == TRIATTN_BUCKETS_CLIP) return n == 2 * s->max_distance + 1;
  return n >= 4 && n % 2 == 0 && s->max_distance > n / 4;
}

bool al(const void* p, uintptr_t a) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

RelposArgs args_of(const triattn_relpos_shape* s, const int* positions, const int* chains) {
  RelposArgs a;
  std::memset(&a, 0, sizeof(a));
  a.pos = positions;
  a.chain = chains;
  a.B = s->B;
  a.N = s->N;
  a.F = s->F;
  a.R = s->max_distance;
  a.buckets = s->buckets;
  fill_lut(s, chains != nullptr, a.lut);
  return a;
}

// Rows per block of `planes` planes of N rows, so that about `want` blocks run.
int rows_per_block(int N, long long planes, int want) {
  const long long blocks = std::max(1ll, std::min<long long>(N, want / planes));
  return static_cast<int>((N + blocks - 1) / blocks);
}

// Planes' gradient: as many warps as three, two or one blocks an SM have room
// for, at least four if they can be had.
struct BwdPlan {
  int warps, rows, splits;
  size_t smem;
};
BwdPlan bwd_plan(int B, int N, int F, int buckets) {
  BwdPlan p;
  const size_t win = static_cast<size_t>(chunks_of(N)) * sizeof(Window);
  p.warps = kThreads / 32;
  while (p.warps > 1 && win + static_cast<size_t>(p.warps) * buckets * 128 > (p.warps > 4 ? 72000u : 216000u)) p.warps /= 2;
  p.smem = win + static_cast<size_t>(p.warps) * buckets * 128;
  const int per_sm = std::max(1, std::min<int>(2048 / (32 * p.warps), static_cast<int>(220000 / (p.smem + 3200))));
  p.rows = rows_per_block(N, static_cast<long long>(B) * F, 152 * per_sm * 2);
  p.splits = (N + p.rows - 1) / p.rows;
  return p;
}

size_t part_bytes(const triattn_relpos_shape* s) {
  if (s->layout == TRIATTN_RELPOS_PAIRS)
    return static_cast<size_t>(relpos_pairs_parts(s->B, s->N)) * s->buckets * s->F * 4;
  return static_cast<size_t>(s->B) * s->F * bwd_plan(s->B, s->N, s->F, s->buckets).splits * s->buckets * 4;
}

// One limit per kernel whatever the call asks for: calls of other threads in
// between set the same.
constexpr int kMaxDynamic = 224 * 1024;
template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamic);
}

template <int G>
cudaError_t launch_heads_fwd(const RelposArgs& a, cudaStream_t s) {
  const int groups = (a.F + G - 1) / G;
  const size_t smem = 4ull * (G * (spread(2 * a.R + 1) + 1) + (a.chain != nullptr ? 2 : 1) * (spread(a.N - 1) + 1));
  cudaError_t e = allow_smem(relpos_heads_fwd_kernel<G>, smem);
  if (e != cudaSuccess) return e;
  const int rows = rows_per_block(a.N, static_cast<long long>(a.B) * groups, 152 * 6);
  relpos_heads_fwd_kernel<G><<<dim3((a.N + rows - 1) / rows, a.B * groups), kThreads, smem, s>>>(a, rows);
  return cudaGetLastError();
}

cudaError_t launch_pairs_fwd(const RelposArgs& a, cudaStream_t s) {
  const int len = pairs_segment(a.F);
  const long long all = static_cast<long long>(a.B) * a.N * ((a.N + len - 1) / len);
  relpos_pairs_fwd_kernel<<<static_cast<unsigned>(std::min(all, 152ll * 4)), pairs_threads(a.F), 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_heads_bwd(const RelposArgs& a, const void* d_out, const BwdPlan& p, cudaStream_t s) {
  cudaError_t e = allow_smem(relpos_heads_bwd_kernel<T>, p.smem);
  if (e != cudaSuccess) return e;
  relpos_heads_bwd_kernel<T><<<dim3(p.splits, a.B * a.F), p.warps * 32, p.smem, s>>>(
      a, static_cast<const T*>(d_out), p.rows);
  return cudaGetLastError();
}

}  // namespace
}  // namespace triattn

using namespace triattn;

extern "C" {

size_t triattn_relpos_workspace_bytes(const triattn_relpos_shape* shape) {
  if (check_shape(shape) != TRIATTN_OK) return 0;
  return (part_bytes(shape) + 255) / 256 * 256;
}

triattn_status triattn_relpos_fwd(const triattn_relpos_shape* shape, const float* table, const void* base,
                                  const int* positions, const int* chains, void* out, void* stream) {
  triattn_status st = check_shape(shape);
  if (st != TRIATTN_OK) return st;
  if (!rule_ok(shape, chains != nullptr)) return TRIATTN_ERR_INVALID_ARG;
  if (!al(table, 16) || !al(out, 16) || (base != nullptr && !al(base, 16)) || (positions != nullptr && !al(positions, 4)) ||
      (chains != nullptr && !al(chains, 4)))
    return TRIATTN_ERR_INVALID_ARG;
  RelposArgs a = args_of(shape, positions, chains);
  a.table = table;
  a.base = static_cast<const uint16_t*>(base);
  a.out = static_cast<uint16_t*>(out);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = trace_call(kKRelFwd, s, [&] {
    if (shape->layout == TRIATTN_RELPOS_PAIRS) return launch_pairs_fwd(a, s);
    // rows off 16 bytes start elsewhere in every plane: one head at a time
    return shape->N % 8 == 0 ? launch_heads_fwd<kHeadGroup>(a, s) : launch_heads_fwd<1>(a, s);
  });
  return e == cudaSuccess ? TRIATTN_OK : TRIATTN_ERR_CUDA;
}

triattn_status triattn_relpos_bwd(const triattn_relpos_shape* shape, const void* d_out, const int* positions,
                                  const int* chains, float* d_table, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  triattn_status st = check_shape(shape);
  if (st != TRIATTN_OK) return st;
  if (!rule_ok(shape, chains != nullptr)) return TRIATTN_ERR_INVALID_ARG;
  if (!al(d_out, 16) || !al(d_table, 4) || (positions != nullptr && !al(positions, 4)) ||
      (chains != nullptr && !al(chains, 4)))
    return TRIATTN_ERR_INVALID_ARG;
  if (!al(workspace, 256) || workspace_bytes < triattn_relpos_workspace_bytes(shape)) return TRIATTN_ERR_WORKSPACE;
  RelposArgs a = args_of(shape, positions, chains);
  a.part = static_cast<float*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (shape->layout == TRIATTN_RELPOS_PAIRS) {
    const int parts = relpos_pairs_parts(a.B, a.N);
    e = trace_call(kKRelBwd, s, [&] { return launch_relpos_pairs_bwd(a, d_out, parts, current_wait_ctl(), s); });
    if (e == cudaSuccess)
      e = trace_call(kKRelSum, s, [&] {  // partials [parts][buckets][F]
        relpos_sum_kernel<<<dim3((a.F + 31) / 32, a.buckets), 1024, 0, s>>>(
            a.part, d_table, a.F, 1, a.F, 1, parts, 0, static_cast<size_t>(a.buckets) * a.F, a.F);
        return cudaGetLastError();
      });
  } else {
    const BwdPlan p = bwd_plan(a.B, a.N, a.F, a.buckets);
    e = trace_call(kKRelBwd, s, [&] {
      return (shape->flags & TRIATTN_FLAG_DOUT_FP32) ? launch_heads_bwd<float>(a, d_out, p, s)
                                                     : launch_heads_bwd<uint16_t>(a, d_out, p, s);
    });
    if (e == cudaSuccess)
      e = trace_call(kKRelSum, s, [&] {  // partials [B][F][splits][buckets]
        const size_t per = static_cast<size_t>(p.splits) * a.buckets;
        relpos_sum_kernel<<<dim3((a.buckets + 31) / 32, a.F), 1024, 0, s>>>(a.part, d_table, a.buckets, a.F, 1, a.B,
                                                                           p.splits, a.F * per, a.buckets, per);
        return cudaGetLastError();
      });
  }
  return e == cudaSuccess ? TRIATTN_OK : TRIATTN_ERR_CUDA;
}

}  // extern "C"
