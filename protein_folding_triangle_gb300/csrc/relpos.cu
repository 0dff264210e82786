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
// forward shares them between four heads; both planes' kernels ask once for a
// chunk of columns, of its smallest and largest position and chain, whether all of
// it lies in one bucket or on a diagonal; and the pair features' gradient is a
// product with a one-hot matrix on the tensor cores (relpos_pairs.cu).
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

// An element (zero where `in` does not hold) of memory that the kernel may write,
// loaded on the spot: under a condition of the compiler's the loads would wait for one
// another.
__device__ __forceinline__ uint32_t load1_written(const uint16_t* p, bool in) {
  uint32_t v;
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n mov.u32 %0, 0;\n @p ld.global.u16 %0, [%1];\n}\n"
               : "=r"(v)
               : "l"(p), "r"(static_cast<uint32_t>(in))
               : "memory");
  return v;
}

// The planes' rows need not start on 16 bytes: chunk t of a row is the t-th
// aligned group of W elements that holds elements of the row, [W t - off,
// W t - off + W) of it, off the place of the row's start in its group.
__host__ __device__ constexpr int chunks_of(int N, int W) { return N % W == 0 ? N / W : (N + 2 * W - 2) / W; }

// What the columns that chunk t can hold (whatever its rows' off) have in common.
struct Window {
  int lo, hi;            // smallest and largest position
  int chain, chain_max;  // smallest and largest chain
  int run;               // the positions are lo, lo + 1, ..., in order
};
// First column of chunk t's window: of its aligned W columns, and where rows start
// anywhere of the W before them too.
template <int W>
__device__ __forceinline__ int first_column(int N, int t) { return N % W == 0 ? W * t : max(0, W * (t - 1)); }
// All windows, by all threads of the block (a multiple of W, W lanes to a group of
// columns); the caller waits for them.
template <int W>
__device__ __forceinline__ void make_windows(const RelposArgs& a, int b, int nt, Window* win) {
  constexpr int U = 4;  // groups of columns whose loads are under way together
  const int l = threadIdx.x % W, step = blockDim.x / W;
  const bool two = a.N % W != 0;
  const int* pos = a.pos != nullptr ? a.pos + static_cast<size_t>(b) * a.N : nullptr;
  const int* chain = a.chain != nullptr ? a.chain + static_cast<size_t>(b) * a.N : nullptr;
  for (int t0 = threadIdx.x / W; t0 - threadIdx.x / W < nt; t0 += U * step) {
    int p[U][2], c[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int g = 0; g < 2; ++g) {  // its own columns, and the W before
        const int j = min(max(W * (t0 + u * step - g) + l, 0), a.N - 1);
        p[u][g] = j;
        c[u][g] = 0;
        if (pos != nullptr && (g == 0 || two)) p[u][g] = __ldg(pos + j);
        if (chain != nullptr && (g == 0 || two)) c[u][g] = __ldg(chain + j);
      }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * step;
      Window w{0x7fffffff, -0x7fffffff - 1, 0x7fffffff, -0x7fffffff - 1, 1};
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int j = W * (t - g) + l;
        if ((g == 1 && !two) || j < 0 || j >= a.N) continue;
        w.lo = min(w.lo, p[u][g]);
        w.hi = max(w.hi, p[u][g]);
        w.chain = min(w.chain, c[u][g]);
        w.chain_max = max(w.chain_max, c[u][g]);
      }
#pragma unroll
      for (int o = W / 2; o > 0; o /= 2) {
        w.lo = min(w.lo, __shfl_xor_sync(0xffffffffu, w.lo, o));
        w.hi = max(w.hi, __shfl_xor_sync(0xffffffffu, w.hi, o));
        w.chain = min(w.chain, __shfl_xor_sync(0xffffffffu, w.chain, o));
        w.chain_max = max(w.chain_max, __shfl_xor_sync(0xffffffffu, w.chain_max, o));
      }
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int j = W * (t - g) + l;
        if ((g == 1 && !two) || j < 0 || j >= a.N) continue;
        if (static_cast<long long>(p[u][g]) - w.lo != j - first_column<W>(a.N, t)) w.run = 0;
      }
#pragma unroll
      for (int o = W / 2; o > 0; o /= 2) w.run &= __shfl_xor_sync(0xffffffffu, w.run, o);
      if (l == 0 && t < nt) win[t] = w;
    }
  }
}

// ------------------------------------------------------- planes, forward
// Four heads at a time: the buckets are found once for all.  A warp takes 32
// consecutive chunks of the example's rows, a lane to a chunk, and the warps of a block
// take turns at the same columns, as the ends of rows, gaps and meeting chains cost
// more.  The values of every bucket lie in shared memory by distance.  Chunks inside
// the row and of one chain are taken as a whole; the others of a warp (the ends of rows
// that do not start on a chunk, and where chains meet) go element by element, four
// chunks of every head at a time, a lane to an element.  ALIGNED: all rows start on 16
// bytes.  2048 tokens, 16 heads, four chains (268 MB): 51 us, 5.3 TB/s; 2049 tokens 68
// (without the turns 55 and 90; the four heads' different offsets in one pass over the
// chunks: 145).  Between a warp's loads and its stores lie the buckets.  Five, six or
// eight blocks an SM: a few us more; loads of 32 bytes: the same.
constexpr int kFwdBlocks = 4;  // an SM
template <bool ALIGNED>
__global__ void __launch_bounds__(kThreads, kFwdBlocks) relpos_heads_fwd_kernel(const __grid_constant__ RelposArgs a) {
  constexpr int G = kHeadGroup, W = 8;
  extern __shared__ float sh[];
  const int nt = chunks_of(a.N, W), VW = spread(2 * a.R + 1) + 1;
  Window* win = reinterpret_cast<Window*>(sh);                        // [chunks]
  float* val = sh + 5 * nt;                                           // [G][VW]: distance + R, then other chains
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int groups = (a.F + G - 1) / G, b = blockIdx.y / groups, h0 = (blockIdx.y % groups) * G, ng = min(G, a.F - h0);
  const int* chain = a.chain != nullptr ? a.chain + static_cast<size_t>(b) * a.N : nullptr;
  for (int d = threadIdx.x; d <= 2 * a.R + 1; d += kThreads) {
    const int k = d <= 2 * a.R ? a.lut[d] : a.buckets - 1;
#pragma unroll
    for (int g = 0; g < G; ++g)
      if (g < ng) val[g * VW + spread(d)] = a.table[static_cast<size_t>(k) * a.F + h0 + g];
  }
  make_windows<W>(a, b, nt, win);
  __syncthreads();
  const int other = spread(2 * a.R + 1);
  const size_t plane = static_cast<size_t>(a.N) * a.N;
  const int items = a.N * nt, pieces = (items + 31) / 32;
  const int u0 = static_cast<int>(static_cast<long long>(pieces) * blockIdx.x / gridDim.x);
  const int u1 = static_cast<int>(static_cast<long long>(pieces) * (blockIdx.x + 1) / gridDim.x);
  const size_t first = (static_cast<size_t>(b) * a.F + h0) * plane;
  auto place = [&](int pi, int ci, int j) {  // of column j, any chain
    return chain != nullptr && __ldg(chain + j) != ci ? other : spread(distance(pi, a.position(b, j), a.R));
  };
  constexpr int kWarps = kThreads / 32;
  for (int v0 = u0, turn = warp; v0 < u1; v0 += kWarps, ++turn) {
    const int u = v0 + turn % kWarps;  // what lies in the same columns comes to all warps in turn
    if (u >= u1) continue;
    const int e = min(32 * u + lane, items - 1), i = e / nt, t = e - i * nt;
    const bool mine = 32 * u + lane < items;
    const int pi = a.position(b, i), ci = chain != nullptr ? __ldg(chain + i) : 0;
    const size_t row = first + static_cast<size_t>(i) * a.N;
    int off[G];
#pragma unroll
    for (int g = 0; g < G; ++g) off[g] = ALIGNED ? 0 : static_cast<int>((row + g * plane) & (W - 1));
    const Window w = win[t];
    const bool apart = ci < w.chain || ci > w.chain_max;  // no column of the row's chain
    const bool one_chain = (apart || w.chain == w.chain_max) && mine;
    uint4 in[G];
    bool whole[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int j0 = W * t - off[g];
      whole[g] = g < ng && one_chain && (ALIGNED || (j0 >= 0 && j0 + W <= a.N));
      in[g] = make_uint4(0u, 0u, 0u, 0u);
      if (a.base != nullptr && whole[g]) in[g] = *reinterpret_cast<const uint4*>(a.base + row + g * plane + j0);
    }
    const int far = distance(pi, w.hi, a.R), near = distance(pi, w.lo, a.R);
    const bool single = one_chain && (apart || far == near);
    const int one = apart ? other : spread(far);
    if (single) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (!whole[g]) continue;
        const float2 x = make_float2(val[g * VW + one], val[g * VW + one]);
        const uint32_t p[4] = {in[g].x, in[g].y, in[g].z, in[g].w};
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 v = fadd2(make_float2(bf16lo_to_f32(p[k]), bf16hi_to_f32(p[k])), x);
          o[k] = pack_bf16x2(v.x, v.y);
        }
        *reinterpret_cast<uint4*>(a.out + row + g * plane + W * t - off[g]) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    } else if (one_chain) {
      int at[W];
      const bool run = w.run != 0;
      const int p0 = w.lo - first_column<W>(a.N, t);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int j0 = W * t - off[g];
        if (!whole[g]) continue;
        if (g == 0 || !ALIGNED) {
#pragma unroll
          for (int k = 0; k < W; ++k) at[k] = run ? spread(distance(pi, p0 + j0 + k, a.R)) : place(pi, ci, j0 + k);
        }
        float v[8];
        unpack8(in[g], v);
#pragma unroll
        for (int k = 0; k < W; ++k) v[k] += val[g * VW + at[k]];
        *reinterpret_cast<uint4*>(a.out + row + g * plane + j0) = pack8(v);
      }
    }
    uint32_t left[G], any = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      left[g] = __ballot_sync(0xffffffffu, g < ng && mine && !whole[g] && W * t - off[g] < a.N);
      any |= left[g];
    }
    while (any != 0) {  // all heads' loads before the stores
      size_t at[G];
      uint32_t x[G], in_ = 0;
      float v[G];
      any = 0;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        int q = 0;
        bool has = false;
#pragma unroll
        for (int k = 0; k < 32 / W; ++k) {
          if (left[g] != 0 && lane / W == k) {
            q = __ffs(left[g]) - 1;
            has = true;
          }
          left[g] &= left[g] - 1;
        }
        any |= left[g];
        const int iq = __shfl_sync(0xffffffffu, i, q), tq = __shfl_sync(0xffffffffu, t, q);
        const int pq = __shfl_sync(0xffffffffu, pi, q), cq = __shfl_sync(0xffffffffu, ci, q);
        const size_t start = first + g * plane + static_cast<size_t>(iq) * a.N;
        const int j = W * tq - (ALIGNED ? 0 : static_cast<int>(start & (W - 1))) + lane % W;
        has = has && j >= 0 && j < a.N;
        in_ |= has ? 1u << g : 0u;
        at[g] = start + j;
        x[g] = load1_written(a.base + at[g], has && a.base != nullptr);
        v[g] = val[min(g, ng - 1) * VW + place(pq, cq, min(max(j, 0), a.N - 1))];
      }
#pragma unroll
      for (int g = 0; g < G; ++g)
        if ((in_ >> g) & 1u)
          a.out[at[g]] = static_cast<uint16_t>(pack_bf16x2(bf16lo_to_f32(x[g]) + v[g], 0.f) & 0xFFFFu);
    }
  }
}

// ------------------------------------------------ pair features, forward
// Block: a run of segments of a row (b, i), as many as any other block's or one
// more; thread: eight features of four pairs of a segment, all four in flight.
// The table comes from L1.  768^2 pairs of 128 features (302 MB) take 52 us, 1920^2
// 299 us (6.4 TB/s).  Five blocks per SM were the fastest of three to six (at 1920^2 of
// 128 features: 331 us with three and six pairs, 321, 299, 338); loads of the next
// segment ahead of a segment's stores cost a tenth.
constexpr int kPairsU = 4, kPairsBlocks = 5;
int pairs_threads(int F) { return kThreads / (F / 8) * (F / 8); }
int pairs_segment(int F) { return kPairsU * (kThreads / (F / 8)); }
__global__ void __launch_bounds__(kThreads, kPairsBlocks)
    relpos_pairs_fwd_kernel(const __grid_constant__ RelposArgs a) {
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
// An element (zero where `in` does not hold) as it is loaded, a register to itself;
// volatile, so that the loads stay together in front of what uses them.
__device__ __forceinline__ uint32_t load1(const uint16_t* p, bool in) {
  uint32_t v;
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n mov.u32 %0, 0;\n @p ld.global.nc.u16 %0, [%1];\n}\n"
               : "=r"(v)
               : "l"(p), "r"(static_cast<uint32_t>(in)));
  return v;
}
__device__ __forceinline__ uint32_t load1(const float* p, bool in) {
  uint32_t v;
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n mov.u32 %0, 0;\n @p ld.global.nc.u32 %0, [%1];\n}\n"
               : "=r"(v)
               : "l"(p), "r"(static_cast<uint32_t>(in)));
  return v;
}
template <typename T>
__device__ __forceinline__ float value1(uint32_t v) { return sizeof(T) == 2 ? bf16lo_to_f32(v) : __uint_as_float(v); }
// 16 consecutive elements: their 16-byte pieces, and the values of the pieces.
template <int V>
__device__ __forceinline__ void load16(const void* p, uint4 (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = __ldg(static_cast<const uint4*>(p) + i);
}
__device__ __forceinline__ void values(const uint4 (&v)[2], float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[8 * i + 2 * k] = bf16lo_to_f32(w[k]);
      f[8 * i + 2 * k + 1] = bf16hi_to_f32(w[k]);
    }
  }
}
__device__ __forceinline__ void values(const uint4 (&v)[4], float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[4 * i] = __uint_as_float(v[i].x);
    f[4 * i + 1] = __uint_as_float(v[i].y);
    f[4 * i + 2] = __uint_as_float(v[i].z);
    f[4 * i + 3] = __uint_as_float(v[i].w);
  }
}

// A warp's work is a block of eight rows and 32 chunks of 16 columns of a plane, a
// chunk to a lane, and what its elements are is asked once for the block:
//   of other chains, or all of one bucket: all elements are added, in registers for
//     the buckets of the far ends and of other chains;
//   on the diagonal: where the positions count up along rows and columns, column j is
//     at distance i - j from row i in every row, and a lane adds the elements of six
//     distances of its own, in registers (where the table's distances fit them);
//   mixed (chains that meet, gaps, other buckets, the ends of rows that do not start
//     on a chunk): element by element, two rows at a time, a lane to an element, to
//     a place of the lane's own (bucket by lane of its warp) in shared memory.
// No two threads share a sum, so the order is fixed.  2048 tokens, 16 heads, four
// chains (134 MB): 33 us, 4.0 TB/s, the issue slots half full, about eight instructions
// an element of the diagonals' chunks and two of the others'; 2049 tokens 60 us.
// Tables of more distances (kNearMax: a max_distance above 47) go element by element on the
// diagonals' chunks, as all chunks with other buckets on them do.  The gradient and its sum
// in a graph, us in BF16 and FP32, four chains, 2048 tokens: max_distance 32 clipped 32 and
// 52, 47 42 and 69, 50 46 and 76, 100 68 and 117; logarithmic of 32 rows to 47 32 and 52, to
// 128 43 and 69; 2049 tokens: 59 and 93, 74 and 116, 88 and 154, 187 and 327, 59 and 93, 73
// and 119.  With 32 element by element along the diagonals it took 70 us, with equal buckets joined in a
// row 94, with three distances of each row in a lane 110; three blocks an SM with half
// as many loads in flight 45.
// Distances that the lanes hold, [-kNear, kNear), and those of a table that fit: a
// chunk with one of them in one of the rows has no other's distance above
// kNearMax + 2 (W - 1) + kRowsMax - 1.
constexpr int kBwdW = 16, kRowsMax = 8, kNear = 96, kNearMax = 47;
static_assert(kNearMax + 2 * (kBwdW - 1) + kRowsMax - 1 < kNear, "distances of a chunk on the diagonal");
template <typename T, int kRows>
__global__ void __launch_bounds__(kThreads, 2)
    relpos_heads_bwd_kernel(const __grid_constant__ RelposArgs a, const T* d_out) {
  constexpr int W = kBwdW;
  constexpr int V = sizeof(T);  // 16-byte pieces of a chunk
  constexpr int U = 16 / V < kRows ? 16 / V : kRows;  // rows in flight
  extern __shared__ float sh[];
  __shared__ uint8_t lut[2 * kRelposMaxDistance + 1];
  let_next_start();
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, nw = blockDim.x / 32;
  const int nt = chunks_of(a.N, W), b = blockIdx.y / a.F;
  Window* win = reinterpret_cast<Window*>(sh);  // [chunks]
  float* hist = sh + (5 * nt + 3) / 4 * 4;      // [warps][buckets][32]
  const int* chain = a.chain != nullptr ? a.chain + static_cast<size_t>(b) * a.N : nullptr;
  for (int d = threadIdx.x; d <= 2 * a.R; d += blockDim.x) lut[d] = a.lut[d];
  for (int e = threadIdx.x; e < nw * a.buckets * 8; e += blockDim.x)
    reinterpret_cast<float4*>(hist)[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  make_windows<W>(a, b, nt, win);
  __syncthreads();
  float* mine = hist + warp * a.buckets * 32 + lane;
  const size_t p0 = static_cast<size_t>(blockIdx.y) * a.N * a.N;
  const int kl = lut[0], kh = lut[2 * a.R], ko = a.buckets - 1;  // far on either side, other chains
  float sl = 0.f, sh_ = 0.f, so = 0.f, near[kNear / 16];
#pragma unroll
  for (int m = 0; m < kNear / 16; ++m) near[m] = 0.f;
  const int cols = (nt + 31) / 32, units = (a.N + kRows - 1) / kRows * cols;
  const int u0 = static_cast<int>(static_cast<long long>(units) * blockIdx.x / gridDim.x);
  const int u1 = static_cast<int>(static_cast<long long>(units) * (blockIdx.x + 1) / gridDim.x);
  for (int u = u0 + warp; u < u1; u += nw) {
    // the rows' diagonals come to all warps in turn
    const int rb = u / cols, cb = (u - rb * cols + rb * cols / nw) % cols;
    const int i0 = rb * kRows, nr = min(kRows, a.N - i0), t = 32 * cb + lane;
    const size_t s0 = p0 + static_cast<size_t>(i0) * a.N;
    auto off_of = [&](int r) { return static_cast<int>((s0 + static_cast<size_t>(r) * a.N) & (W - 1)); };
    // the rows' positions and chains
    const int pi = a.position(b, i0 + min(lane, nr - 1));
    const int ci = chain != nullptr ? __ldg(chain + i0 + min(lane, nr - 1)) : 0;
    const int rlo = __reduce_min_sync(0xffffffffu, pi), rhi = __reduce_max_sync(0xffffffffu, pi);
    const int rc = __reduce_min_sync(0xffffffffu, ci), rc1 = __reduce_max_sync(0xffffffffu, ci);
    const bool rrun = __all_sync(0xffffffffu, static_cast<long long>(pi) - rlo == min(lane, nr - 1));
    // what the lane's chunk is in all of them
    enum { kNone, kAll, kDiagonal, kMixed };
    int kind = kNone, k = ko;
    if (t < nt) {
      const Window w = win[t];
      if (a.N % W != 0 && (t == 0 || W * t + W > a.N)) {
        kind = kMixed;  // the ends of rows
      } else if (rc1 < w.chain || rc > w.chain_max) {
        kind = kAll;
      } else if (rc != rc1 || w.chain != w.chain_max) {
        kind = kMixed;
      } else {
        k = lut[distance(rhi, w.lo, a.R)];
        const bool diagonal = rrun && w.run && a.R <= kNearMax &&
                              static_cast<long long>(rlo) - w.lo == i0 - first_column<W>(a.N, t);
        kind = k == lut[distance(rlo, w.hi, a.R)] ? kAll : diagonal ? kDiagonal : kMixed;
      }
    }
    if (kind == kAll) {
      float2 x2 = {0.f, 0.f}, y2 = {0.f, 0.f};
      for (int r0 = 0; r0 < nr; r0 += U) {
        uint4 raw[U][V];
#pragma unroll
        for (int q = 0; q < U; ++q)
          if (r0 + q < nr) load16(d_out + (s0 + static_cast<size_t>(r0 + q) * a.N - off_of(r0 + q) + W * t), raw[q]);
#pragma unroll
        for (int q = 0; q < U; ++q) {
          if (r0 + q >= nr) break;
          float v[W];
          values(raw[q], v);
#pragma unroll
          for (int e = 0; e < W; e += 4) {
            x2 = fadd2(x2, make_float2(v[e], v[e + 1]));
            y2 = fadd2(y2, make_float2(v[e + 2], v[e + 3]));
          }
        }
      }
      const float x = (x2.x + x2.y) + (y2.x + y2.y);
      if (k == kl) sl += x;
      else if (k == kh) sh_ += x;
      else if (k == ko) so += x;
      else mine[k * 32] += x;
    }
    __syncwarp();
    const uint32_t diagonals = __ballot_sync(0xffffffffu, kind == kDiagonal);
    if (diagonals != 0) {
      for (int r0 = 0; r0 < nr; r0 += 4) {
        uint32_t x[4][kNear / 16];  // all loads before the first sum
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = r0 + q, j0 = i0 + r + kNear - lane;
          const int c0 = j0 + off_of(r) - 32 * W * cb;  // from the chunks' first column
          const T* row = d_out + s0 + static_cast<size_t>(r) * a.N;
#pragma unroll
          for (int m = 0; m < kNear / 16; ++m) {
            const int j = j0 - 32 * m, c = c0 - 32 * m;
            const bool in = (r < nr) & (j >= 0) & (j < a.N) & (c >= 0) & (c < 32 * W) &
                            ((diagonals >> ((c / W) & 31)) & 1u);
            x[q][m] = load1(row + j, in);
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int m = 0; m < kNear / 16; ++m) near[m] += value1<T>(x[q][m]);
      }
    }
    uint32_t left = __ballot_sync(0xffffffffu, kind == kMixed);
    auto gather = [&](int tq, bool some, int (&kk)[kRows / 2], uint32_t (&x)[kRows / 2]) {
#pragma unroll
      for (int q = 0; q < kRows / 2; ++q) {
        const int r = 2 * q + lane / W, i = i0 + min(r, nr - 1), j = W * tq - off_of(r) + lane % W;
        const bool in = some && r < nr && j >= 0 && j < a.N;
        const int jc = min(max(j, 0), a.N - 1);
        const bool apart = chain != nullptr && __ldg(chain + jc) != __ldg(chain + i);
        const int d = distance(a.position(b, i), a.position(b, jc), a.R);
        kk[q] = in ? (apart ? ko : lut[d]) : -1;
        x[q] = load1(d_out + s0 + static_cast<size_t>(r) * a.N + j, in);
      }
    };
    auto add = [&](const int (&kk)[kRows / 2], const uint32_t (&x)[kRows / 2]) {
#pragma unroll
      for (int q = 0; q < kRows / 2; ++q)
        if (kk[q] >= 0) mine[kk[q] * 32] += value1<T>(x[q]);
    };
    if constexpr (kRows == kRowsMax) {
      for (; left != 0; left &= left - 1) {
        int kk[kRows / 2];
        uint32_t x[kRows / 2];
        gather(32 * cb + __ffs(left) - 1, true, kk, x);
        add(kk, x);
      }
    } else {  // a few units a warp: the loads of four chunks together
      while (left != 0) {
        int kk[4][kRows / 2];
        uint32_t x[4][kRows / 2];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          gather(32 * cb + __ffs(left) - 1, left != 0, kk[m], x[m]);
          left &= left - 1;
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) add(kk[m], x[m]);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < kNear / 16; ++m) {
    const int d = 32 * m + lane - kNear;
    mine[lut[min(max(d, -a.R), a.R) + a.R] * 32] += near[m];
  }
  mine[kl * 32] += sl;
  mine[kh * 32] += sh_;
  mine[ko * 32] += so;
  __syncthreads();
  float* out = a.part + (static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x) * a.buckets;
  for (int k0 = 4 * warp; k0 < a.buckets; k0 += 4 * nw) {  // four buckets, eight lanes to a bucket's 32 places
    const int k = min(k0 + lane / 8, a.buckets - 1);
    float v = 0.f;
    for (int w = 0; w < nw; ++w) {
      const float4 x = reinterpret_cast<const float4*>(hist)[(w * a.buckets + k) * 8 + lane % 8];
      v += (x.x + x.y) + (x.z + x.w);
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane % 8 == 0 && k0 + lane / 8 < a.buckets) out[k] = v;
  }
}

// Planes: out[k * F + f] = sum over (b, s) of part[b][f][s][k], k along the lanes, 32 slices
// of the sum per block, joined in a fixed order.
__global__ void __launch_bounds__(1024) relpos_sum_kernel(const float* part, float* out, int buckets, int nb, int ns) {
  __shared__ float2 sh[32][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5, k = blockIdx.x * 32 + lane, F = gridDim.y;
  const size_t ps = buckets, py = ps * ns, pb = py * F;
  Sum2 v;
  after_previous();
  if (k < buckets) {
#pragma unroll 4
    for (int e = slice; e < nb * ns; e += 32) {
      const int b = e / ns, s = e - b * ns;
      v.add(part[b * pb + blockIdx.y * py + s * ps + k]);
    }
  }
  sh[slice][lane] = v.pair();
  __syncthreads();
  if (slice == 0 && k < buckets) {
    for (int s = 1; s < 32; ++s) v.add(sh[s][lane]);
    out[static_cast<size_t>(k) * F + blockIdx.y] = v.value();
  }
}

// Pair features: out[x] = sum over s of part[s][x], x in fours along the lanes, S slices of
// the sum per block, joined by a warp for each of the four.  32 slices, or eight where there
// are few partials.  Both measured, the gradient as a whole: 309^2 pairs of 256 features and
// 201 buckets (152 partials, 31 MB) 27 us with 32 and 31 with eight, 640^2 pairs of 128 and
// 65 28 and 34; 2 x 30^2 pairs of 256 and 201 (29 partials) 18.5 and 17.
template <int S>
__global__ void __launch_bounds__(32 * S) relpos_flat_sum_kernel(const float* part, float* out, int n4, int parts) {
  constexpr int U = S == 8 ? 8 : 5;  // loads under way together
  __shared__ float2 sh[S][4][32];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5, x = blockIdx.x * 32 + lane;
  Sum2 v[4];
  after_previous();
  if (x < n4) {
    const float4* p = reinterpret_cast<const float4*>(part) + x;
    for (int s0 = slice; s0 < parts; s0 += U * S) {
      float4 f[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        f[u] = s0 + u * S < parts ? p[static_cast<size_t>(s0 + u * S) * n4] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v[0].add(f[u].x);
        v[1].add(f[u].y);
        v[2].add(f[u].z);
        v[3].add(f[u].w);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) sh[slice][i][lane] = v[i].pair();
  __syncthreads();
  if (slice < 4 && x < n4) {
    Sum2 w;
#pragma unroll
    for (int s = 0; s < S; ++s) w.add(sh[s][slice][lane]);
    out[4 * static_cast<size_t>(x) + slice] = w.value();
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

// Planes' gradient: two blocks of eight warps an SM where their sums fit, otherwise
// fewer warps in a block, and fewer blocks.  Units of four rows where those of eight
// would leave warps without one (3 x 301 tokens, eight heads, FP32: 16.5 and 12 us; 2048
// tokens, sixteen heads: 33 us with eight, 37 with four).
struct BwdPlan {
  int warps, splits, rows;
  size_t smem;
};
BwdPlan bwd_plan(int B, int N, int F, int buckets) {
  BwdPlan p;
  const size_t win = (static_cast<size_t>(chunks_of(N, kBwdW)) * sizeof(Window) + 15) / 16 * 16;
  p.warps = kThreads / 32;
  while (p.warps > 1 && win + static_cast<size_t>(p.warps) * buckets * 128 > (p.warps > 4 ? 72000u : 216000u))
    p.warps /= 2;
  p.smem = win + static_cast<size_t>(p.warps) * buckets * 128;
  const int per_sm = std::max(1, std::min<int>(16 / p.warps, static_cast<int>(232448 / (p.smem + 3200))));
  const int cols = (chunks_of(N, kBwdW) + 31) / 32;
  const long long planes = static_cast<long long>(B) * F;
  p.rows = (N + 7) / 8 * cols * planes <= 152ll * per_sm * p.warps ? 4 : 8;
  const int units = (N + p.rows - 1) / p.rows * cols;
  p.splits = std::max(1, std::min((units + p.warps - 1) / p.warps, static_cast<int>(152ll * per_sm / planes)));
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

template <bool ALIGNED>
cudaError_t launch_heads_fwd(const RelposArgs& a, cudaStream_t s) {
  const int groups = (a.F + kHeadGroup - 1) / kHeadGroup;
  const int nt = chunks_of(a.N, 8);
  const size_t smem = sizeof(Window) * nt + 4ull * kHeadGroup * (spread(2 * a.R + 1) + 1);
  cudaError_t e = allow_smem(relpos_heads_fwd_kernel<ALIGNED>, smem);
  if (e != cudaSuccess) return e;
  const int units = (a.N * nt + 31) / 32, blocks = 152 * kFwdBlocks / (a.B * groups);
  relpos_heads_fwd_kernel<ALIGNED><<<dim3(std::max(1, std::min((units + 7) / 8, blocks)), a.B * groups), kThreads, smem,
                                     s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_pairs_fwd(const RelposArgs& a, cudaStream_t s) {
  const int len = pairs_segment(a.F);
  const long long all = static_cast<long long>(a.B) * a.N * ((a.N + len - 1) / len);
  relpos_pairs_fwd_kernel<<<static_cast<unsigned>(std::min(all, 152ll * kPairsBlocks)), pairs_threads(a.F), 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int ROWS>
cudaError_t launch_heads_bwd_rows(const RelposArgs& a, const void* d_out, const BwdPlan& p, cudaStream_t s) {
  cudaError_t e = allow_smem(relpos_heads_bwd_kernel<T, ROWS>, p.smem);
  if (e != cudaSuccess) return e;
  relpos_heads_bwd_kernel<T, ROWS><<<dim3(p.splits, a.B * a.F), p.warps * 32, p.smem, s>>>(
      a, static_cast<const T*>(d_out));
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_heads_bwd(const RelposArgs& a, const void* d_out, const BwdPlan& p, cudaStream_t s) {
  return p.rows == 4 ? launch_heads_bwd_rows<T, 4>(a, d_out, p, s) : launch_heads_bwd_rows<T, 8>(a, d_out, p, s);
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
  if (!al(table, 16) || !al(out, 16) || (base != nullptr && !al(base, 16)) ||
      (positions != nullptr && !al(positions, 4)) || (chains != nullptr && !al(chains, 4)))
    return TRIATTN_ERR_INVALID_ARG;
  RelposArgs a = args_of(shape, positions, chains);
  a.table = table;
  a.base = static_cast<const uint16_t*>(base);
  a.out = static_cast<uint16_t*>(out);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = trace_call(kKRelFwd, s, [&] {
    if (shape->layout == TRIATTN_RELPOS_PAIRS) return launch_pairs_fwd(a, s);
    return shape->N % 8 == 0 ? launch_heads_fwd<true>(a, s) : launch_heads_fwd<false>(a, s);
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
        const int n4 = a.buckets * a.F / 4;
        const bool few = parts <= 64;
        return launch_after(false, few ? relpos_flat_sum_kernel<8> : relpos_flat_sum_kernel<32>, dim3((n4 + 31) / 32),
                            few ? 256 : 1024, 0, s, a.part, d_table, n4, parts);
      });
  } else {
    const BwdPlan p = bwd_plan(a.B, a.N, a.F, a.buckets);
    e = trace_call(kKRelBwd, s, [&] {
      return (shape->flags & TRIATTN_FLAG_DOUT_FP32) ? launch_heads_bwd<float>(a, d_out, p, s)
                                                     : launch_heads_bwd<uint16_t>(a, d_out, p, s);
    });
    if (e == cudaSuccess)
      e = trace_call(kKRelSum, s, [&] {  // partials [B][F][splits][buckets]
        return launch_after(false, relpos_sum_kernel, dim3((a.buckets + 31) / 32, a.F), 1024, 0, s, a.part, d_table,
                            a.buckets, a.B, p.splits);
      });
  }
  return e == cudaSuccess ? TRIATTN_OK : TRIATTN_ERR_CUDA;
}

}  // extern "C"
