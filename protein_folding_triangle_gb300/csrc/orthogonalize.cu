// Orthogonalising a list of updates by Newton-Schulz products: for every matrix
// G, with X = G / (|G|_F + eps) of m <= n (the transposed of a tall matrix),
// `steps` times
//
//   A = X X^T,  B = b A + c A^2,  X <- a X + B X,
//
// which takes every singular value s to s (a + b s^2 + c s^4) and leaves the
// singular vectors.
//
// The products run on the tensor cores as products of FP16 pairs: a value x is
// held as hi + lo, hi = fp16(2^8 x), lo = fp16(2^8 x - hi), 22 bits, and a product
// is hi hi + hi lo + lo hi in one FP32 accumulator.  Single BF16 operands, as
// such updates are often computed, are off by 3 % of the result after five steps
// and by 80 % where a matrix has few directions (what rounding adds beside them
// is multiplied by a, 3.4, in every step); pairs of BF16 by up to 8e-4.  Pairs of
// FP16 stay within two to four times the error of FP32 products: with exact sums 2.4e-6
// against 6e-7 of the result (128 x 388 and 256 x 1037, noise beside a few directions),
// 4e-5 against 1.6e-5 (90 x 40 of two directions), 8e-5 against 3e-5 (256 x 300 of one);
// the one rounding to BF16 is 1.6e-3.  X carries the scale, which keeps its small values
// out of FP16's subnormals (its floor is 2^-33; the largest value is 255).  A, A' and B'
// do not: their floor is 2^-25, as small beside their diagonals, which are near one or
// beside b and a, as what FP32 products of norm one round off.
//
// With A' = c A + b I and B' = A' A + a I, a step is three plain products:
//   1  A = X X^T (and A' from the accumulator),  2  B' = A' A,  3  X <- B' X.
// Operands are kept in the workspace as the shared-memory image of their tiles,
// 128 rows x 64 columns with the 128-byte swizzle, hi then lo (32 KB), zero past
// the matrix: one untiled bulk copy loads a tile, for a K-major operand as for an
// MN-major one, and no tensor maps are needed for a list of any matrices.
//
// Kernels: sums of squares, X's tiles, then all steps of the matrices of at most 128
// rows (orth_solo.cu) and all steps of the others (orth_gemm_kernel); the start of
// each of the first three lies behind the one before.  The ten matrices of a block of
// 128 features take 62 us on the device, those of 48 blocks 273 (75 GFLOP by the
// formula, three times as many run), twelve of 256 x 1037 149, of which the steps' 135
// are 15 dependent phases of two to seven us of loads and products and some five of
// latency.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <type_traits>
#include <vector>

#include "kernels.cuh"
#include "orthogonalize.cuh"
#include "triattn.h"

namespace triattn {
namespace {

constexpr int kUpload = 256;
struct OrthTable {
  OrthMat mat[kUpload];
  int n;
};
static_assert(sizeof(OrthTable) + 32 <= 32764, "kernel parameter limit");

// A row of the table to memory, six lanes to a row.  Parameters that lanes read at
// places of their own come one after the other, so few of them lie on one SM (a block of
// 256 rows took 12 us).
__device__ __forceinline__ void put_row(const OrthTable& t, int k, int piece, OrthMat* to) {
  static_assert(sizeof(OrthMat) == 96, "six pieces");
  reinterpret_cast<uint4*>(to + k)[piece] = reinterpret_cast<const uint4*>(t.mat + k)[piece];
}
constexpr int kTableRows = 4;  // a block
__global__ void __launch_bounds__(32) orth_table_kernel(const __grid_constant__ OrthTable t, OrthMat* to) {
  let_next_start();
  after_previous();  // what last used the workspace
  const int k = kTableRows * blockIdx.x + threadIdx.x / 6;
  if (threadIdx.x < 6 * kTableRows && k < t.n) put_row(t, k, threadIdx.x % 6, to);
}

// The matrix that item `at` belongs to (the last whose first item is not above it), by a whole warp.
template <int OrthMat::* FIRST>
__device__ __forceinline__ int find(const OrthMat* mat, int count, int at) {
  int lo = 0, n = count;  // it is one of [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32, i = static_cast<int>(threadIdx.x & 31) * step;
    const uint32_t below = __ballot_sync(0xffffffffu, i < n && mat[lo + i].*FIRST <= at);
    const int part = 31 - __clz(below);
    lo += part * step;
    n = min(step, n - part * step);
  }
  return lo;
}

__device__ __forceinline__ float element(const OrthMat& q, long long at) {
  return (q.flags & kOrthFp32) ? __ldg(static_cast<const float*>(q.src) + at)
                           : bf16lo_to_f32(__ldg(static_cast<const uint16_t*>(q.src) + at));
}
// Eight consecutive elements from `at`, a multiple of eight from an address on 16 bytes.
__device__ __forceinline__ void elements8(const OrthMat& q, long long at, float (&y)[8]) {
  if (q.flags & kOrthFp32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(q.src) + at);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    y[0] = a.x;
    y[1] = a.y;
    y[2] = a.z;
    y[3] = a.w;
    y[4] = b.x;
    y[5] = b.y;
    y[6] = b.z;
    y[7] = b.w;
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(q.src) + at));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = bf16lo_to_f32(w[i]);
      y[2 * i + 1] = bf16hi_to_f32(w[i]);
    }
  }
}
__device__ __forceinline__ bool on16(const OrthMat& q) { return (reinterpret_cast<uintptr_t>(q.src) & 15) == 0; }

// Sums of squares, one partial per kNormPart elements of the source in the order of
// its rows: in FP32, and again in FP64 where FP32 does not hold the squares.  A short
// list's table is a parameter, whose rows the first blocks put where the later kernels
// look for them.
constexpr int kNormPart = 4096;
template <bool PARAM>
__global__ void __launch_bounds__(256) orth_norm_kernel(const __grid_constant__ OrthTable t, OrthView v, OrthMat* to) {
  __shared__ float sh[8];
  let_next_start();
  after_previous();  // the table, or what last used the workspace
  for (int i = blockIdx.x * 256 + threadIdx.x; i < v.n; i += gridDim.x * 256) v.done[i] = 0;
  if (PARAM && static_cast<int>(blockIdx.x) < t.n && threadIdx.x < 6) put_row(t, blockIdx.x, threadIdx.x, to);
  const OrthMat* mat = PARAM ? t.mat : v.mat;
  const OrthMat q = mat[find<&OrthMat::part0>(mat, PARAM ? t.n : v.n, blockIdx.x)];
  const int rows = (q.flags & kOrthTall) ? q.n : q.m, cols = (q.flags & kOrthTall) ? q.m : q.n;
  const long long n = static_cast<long long>(rows) * cols, e0 = static_cast<long long>(blockIdx.x - q.part0) * kNormPart;
  auto each = [&](int first, int step, auto&& f) {  // of the part's elements
    const int m = static_cast<int>(min(static_cast<long long>(kNormPart), n - e0));
    const long long r0 = e0 / cols;
    const int c0 = static_cast<int>(e0 - r0 * cols);
#pragma unroll 8
    for (int i = first; i < m; i += step) {
      const int r = (c0 + i) / cols;
      f(element(q, (r0 + r) * q.ld_src + (c0 + i - r * cols)));
    }
  };
  float s = 0.f;
  if (q.ld_src == cols && on16(q) && e0 + kNormPart <= n) {
#pragma unroll
    for (int u = 0; u < kNormPart / 2048; ++u) {
      float y[8];
      elements8(q, e0 + 2048 * u + 8 * threadIdx.x, y);
#pragma unroll
      for (int k = 0; k < 8; ++k) s += y[k] * y[k];
    }
  } else {
    each(threadIdx.x, 256, [&](float x) { s += x * x; });
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  s = 0.f;
  for (int w = 0; w < 8; ++w) s += sh[w];
  double d = s;
  if (!(s >= 0x1p-80f && s <= 0x1p126f)) {  // by one warp: FP32's range ends near it
    d = 0.0;
    each(threadIdx.x, 32, [&](float x) { d += static_cast<double>(x) * x; });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  }
  if (threadIdx.x == 0) v.part[blockIdx.x] = d;
}

// Eight elements of X from (row, col) on, zero outside it: loaded from the nearest
// places inside, so that no load waits for a condition.
template <typename S>
__device__ __forceinline__ void gather8(const OrthMat& q, int row, int col, float (&y)[8]) {
  const bool tall = (q.flags & kOrthTall) != 0;
  const S* p = static_cast<const S*>(q.src) + (tall ? min(row, q.m - 1) : min(row, q.m - 1) * q.ld_src);
  S x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int c = min(col + j, q.n - 1);
    x[j] = __ldg(p + (tall ? c * q.ld_src : c));
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool in = row < q.m && col + j < q.n;
    if constexpr (sizeof(S) == 4) y[j] = in ? x[j] : 0.f;
    else y[j] = in ? bf16lo_to_f32(x[j]) : 0.f;
  }
}

// One tile of X per block: normed, scaled, split, in the image's order.
__global__ void __launch_bounds__(256) orth_load_kernel(OrthView v, float eps) {
  __shared__ double sh[8];
  __shared__ float scaled[2];
  let_next_start();
  after_previous();
  const OrthMat q = v.mat[find<&OrthMat::tiles0>(v.mat, v.n, blockIdx.x)];
  const int t = blockIdx.x - q.tiles0, i = t / (2 * q.nt), c = t - i * 2 * q.nt;
  const bool tall = (q.flags & kOrthTall) != 0;
  const bool wide = !tall && on16(q) && q.ld_src % 8 == 0;
  float y[4][8];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int e = threadIdx.x + 256 * u;
    // lanes along what is contiguous in memory: columns, or rows of a transposed matrix
    const int r = tall ? e & 127 : e >> 3, p = tall ? e >> 7 : e & 7;
    const int row = i * 128 + r, col = c * 64 + p * 8;
    if (wide && row < q.m && col + 8 <= q.n) elements8(q, row * q.ld_src + col, y[u]);
    else if (q.flags & kOrthFp32) gather8<float>(q, row, col, y[u]);
    else gather8<uint16_t>(q, row, col, y[u]);
  }
  // by one warp where it can be: FP64 has two operations a clock and SM
  const bool many = q.parts > 256;
  if (many || threadIdx.x < 32) {
    double s = 0.0;
    for (int k = threadIdx.x; k < q.parts; k += many ? 256 : 32) s += v.part[q.part0 + k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
  }
  if (many) __syncthreads();
  if (threadIdx.x == 0) {
    double s = sh[0];
    for (int w = 1; many && w < 8; ++w) s += sh[w];
    if (s >= 0x1p-100 && s <= 0x1p126) {
      scaled[0] = 1.f;
      scaled[1] = kOrthScale / (sqrtf(static_cast<float>(s)) + eps);
    } else {  // in two factors, so that neither leaves FP32's range
      const double norm = sqrt(s) + eps, first = norm > 0x1p60 ? 0x1p-64 : norm < 0x1p-60 ? 0x1p64 : 1.0;
      scaled[0] = static_cast<float>(first);
      scaled[1] = static_cast<float>(kOrthScale / (norm * first));
    }
  }
  __syncthreads();
  const float first = scaled[0], scale = scaled[1];
  uint8_t* out = tile_at(v, q.x[0] + t);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int e = threadIdx.x + 256 * u, r = tall ? e & 127 : e >> 3, p = tall ? e >> 7 : e & 7;
#pragma unroll
    for (int j = 0; j < 8; ++j) y[u][j] = y[u][j] * first * scale;
    uint4 hi, lo;
    split8(y[u], hi, lo);
    *reinterpret_cast<uint4*>(out + sw128(r, p)) = hi;
    *reinterpret_cast<uint4*>(out + kOrthPlane + sw128(r, p)) = lo;
  }
}

// ------------------------------------------------------------- products
constexpr int kEpiWarps = 8;
constexpr int kThreads = (2 + kEpiWarps) * 32;
template <int W>  // columns of a product's tile, 64 or 128
struct Gemm {
  static constexpr int kStages = W == 64 ? 4 : 3;
  static constexpr int kStage = kOrthTile + W * 256;  // 64 of K: 128 rows of A, W columns of B, hi and lo
  static constexpr int kStg = 32 * W * 2;             // staging of 32 rows of a tile of the result, BF16
  static constexpr int kSmem = kStages * kStage + 4 * kStg + 1024;
  struct Bars {
    uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2];
    uint64_t pair[4];  // the two warps of a quarter of the rows
    uint32_t tmem_slot;
    int abort;
  };
};

struct OrthRun {
  float a, b, c;
  int steps, sq, mn;  // items of the phases of A and A', and of X
  WaitCtl wc;
};

template <int P>
using Phase = std::integral_constant<int, P>;

// A matrix's row of the table, which no kernel that takes it so writes.
__device__ __forceinline__ OrthMat constant(const OrthMat* p) {
  static_assert(sizeof(OrthMat) == 96, "six pieces");
  union {
    uint4 raw[6];
    OrthMat mat;
  } u;
#pragma unroll
  for (int i = 0; i < 6; ++i) u.raw[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  return u.mat;
}

// Bounded wait of a whole warp until what `n` others have stored before they added
// themselves to *p can be loaded by bulk copies.
__device__ __forceinline__ bool count_wait(const uint32_t* p, uint32_t n, const WaitCtl& wc, volatile int* abort) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) {
    const uint64_t t0 = global_timer_ns();
    while (ld_acquire_gpu(p) < n) {
      if (*abort != 0) ok = false;
      if (ok && global_timer_ns() - t0 > wc.limit_ns) {
        atomicOr(wc.status, kDevTimeout);
        *abort = 1;
        ok = false;
      }
      if (!ok) break;
    }
    fence_proxy_async_all();
  }
  return __shfl_sync(0xffffffffu, ok, 0);
}

// All steps of the matrices of more than 128 rows.  A phase is its product's tiles of
// 128 x W, shared out over one CTA per SM; warp 0 loads (64 of K per stage, 48 or
// 64 KB), warp 1 issues twelve MMAs per stage (four of K by three products), warps
// 2-9 take the accumulator (one of two) out, split it and store it.  The loads of a
// matrix's tiles wait until all of its tiles of the phase before have been counted (a
// cooperative launch: all CTAs run; each has its tiles phase by phase).  Where a
// CTA's tiles lie is looked up for 32 of them at once, a lane to a tile, before the
// wait.  A and B' are held without the scale.
template <int W>
__global__ void __launch_bounds__(kThreads, 1) orth_gemm_kernel(OrthView v, OrthRun st) {
  using G = Gemm<W>;
  constexpr int kStages = G::kStages, kStage = G::kStage, T = 128 / W;  // W-column tiles of 128 columns
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ typename G::Bars bars;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int* abort = &bars.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.acc_full[i], 1);
      mbar_init(&bars.acc_empty[i], kEpiWarps);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&bars.pair[i], 2);
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&bars.tmem_slot, 2 * W);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_slot;

  bool go = true;
  // body(matrix, tile row, tile column, stages of K) for this CTA's tiles of a phase
  auto tiles = [&](auto which, auto&& body) {
    constexpr int PHASE = decltype(which)::value;
    const int items = PHASE == 3 ? st.mn : st.sq, grid = gridDim.x;
    for (long long first = blockIdx.x; first < items && go; first += 32ll * grid) {
      const long long at = first + static_cast<long long>(lane) * grid;
      int k = 0, i = 0, j = 0, ks = 0;
      if (at < items) {
        int n = v.n;
        while (n > 1) {  // the last matrix whose first tile is not above it
          const int h = n / 2;
          const OrthMat* mid = v.mat + k + h;
          if (__ldg(PHASE == 3 ? &mid->mn0 : &mid->sq0) <= at) {
            k += h;
            n -= h;
          } else {
            n = h;
          }
        }
        const OrthMat* q = v.mat + k;
        const int r = static_cast<int>(at) - __ldg(PHASE == 3 ? &q->mn0 : &q->sq0);
        const int w = T * __ldg(PHASE == 3 ? &q->nt : &q->mt);
        i = r / w;
        j = r - i * w;
        ks = (__ldg(PHASE == 1 ? &q->n : &q->m) + 63) / 64;
      }
      const int count = static_cast<int>(min(32ll, (items - first + grid - 1) / grid));
      for (int l = 0; l < count && go; ++l)
        body(__shfl_sync(0xffffffffu, k, l), __shfl_sync(0xffffffffu, i, l), __shfl_sync(0xffffffffu, j, l),
             __shfl_sync(0xffffffffu, ks, l));
    }
  };

  if (warp == 0) {
    int stage = 0, phase = 0;
    auto load = [&](auto which, int step) {
      constexpr int PHASE = decltype(which)::value;
      const int in = step & 1;
      int ready = -1;  // the matrix whose operands are
      tiles(which, [&](int k, int i, int j, int ks) {
        const OrthMat q = constant(v.mat + k);
        const bool same = PHASE == 1 && i == j / T;  // B's columns are among A's rows
        const int x = in != 0 ? q.x[1] : q.x[0];
        const uint8_t *pa, *pb;  // of the first stage; both go on by a tile, B of phase 3 by half a tile's rows
        if constexpr (PHASE == 1) {
          pa = tile_at(v, x + i * 2 * q.nt);
          pb = tile_at(v, x + (j / T) * 2 * q.nt) + (j % T) * 8192;
        } else if constexpr (PHASE == 2) {
          pa = tile_at(v, q.a2 + i * 2 * q.mt);
          pb = tile_at(v, q.a + (j / T) * 2 * q.mt) + (j % T) * 8192;
        } else {
          pa = tile_at(v, q.b + i * 2 * q.mt);
          pb = tile_at(v, x + j * (W / 64));
        }
        if (k != ready) {
          const uint32_t sq = T * q.mt * q.mt, before = step * (2 * sq + T * q.mt * q.nt) + (PHASE - 1) * sq;
          go = before == 0 || count_wait(v.done + k, kEpiWarps * before, st.wc, abort);
          if (!go) return;
          ready = k;
        }
        for (int kk = 0; kk < ks; ++kk) {
          if (!__all_sync(0xffffffffu, mbar_wait(&bars.empty[stage], phase ^ 1, st.wc, abort))) {
            go = false;
            return;
          }
          if (lane == 0) {
            uint8_t* sa = sm + stage * kStage;
            uint8_t* sb = sa + kOrthTile;
            uint64_t* full = &bars.full[stage];
            mbar_expect_tx(full, same ? kOrthTile : kStage);
            bulk_load(sa, pa + static_cast<size_t>(kk) * kOrthTile, kOrthTile, full);
            if constexpr (PHASE == 3) {  // blocks of 64 columns, hi of all before lo
              const uint8_t* p = pb + static_cast<size_t>(kk >> 1) * 2 * q.nt * kOrthTile + (kk & 1) * 8192;
#pragma unroll
              for (int c = 0; c < W / 64; ++c) {
                bulk_load(sb + c * 8192, p + c * kOrthTile, 8192, full);
                bulk_load(sb + W * 128 + c * 8192, p + c * kOrthTile + kOrthPlane, 8192, full);
              }
            } else if (!same) {
              const uint8_t* p = pb + static_cast<size_t>(kk) * kOrthTile;
              if constexpr (W == 128) {
                bulk_load(sb, p, kOrthTile, full);
              } else {
                bulk_load(sb, p, 8192, full);
                bulk_load(sb + 8192, p + kOrthPlane, 8192, full);
              }
            }
          }
          __syncwarp();
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
      });
    };
    for (int k = 0; k < st.steps && go; ++k) {
      load(Phase<1>{}, k);
      load(Phase<2>{}, k);
      load(Phase<3>{}, k);
    }
  } else if (warp == 1) {
    constexpr uint32_t kPlaneW = kOrthPlane / 16, kStageW = kStage / 16;
    int stage = 0, phase = 0, local = 0;
    auto multiply = [&](auto which) {
      constexpr int PHASE = decltype(which)::value;
      const uint32_t idesc = idesc_f16_f32(128, W, 0, PHASE == 3 ? 1 : 0);
      const uint32_t s0 = smem_u32(sm) >> 4, a0 = s0 | (1u << 16), b0 = s0 | ((PHASE == 3 ? 512u : 1u) << 16);
      tiles(which, [&](int, int i, int j, int ks) {
        const int ab = local & 1;
        const bool same = PHASE == 1 && i == j / T;
        // B's low plane behind its high one, a tile's plane away where it is part of A
        const uint32_t b_at = same ? (j % T) * 512u : kOrthTile / 16, b_lo = same ? kPlaneW : W * 8u;
        if (!__all_sync(0xffffffffu, mbar_wait(&bars.acc_empty[ab], ((local >> 1) & 1) ^ 1, st.wc, abort))) {
          go = false;
          return;
        }
        tc_fence_after();
        for (int kk = 0; kk < ks; ++kk) {
          if (!__all_sync(0xffffffffu, mbar_wait(&bars.full[stage], phase, st.wc, abort))) {
            go = false;
            return;
          }
          tc_fence_after();
          const uint32_t xa = a0 + stage * kStageW, xb = b0 + stage * kStageW + b_at, d = tmem + ab * W;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t ka = xa + 2 * k, kb = xb + (PHASE == 3 ? 128 * k : 2 * k);
              mma_ss_w(d, ka, kb, idesc, (kk > 0 || k > 0) ? 1u : 0u);
              mma_ss_w(d, ka, kb + b_lo, idesc, 1u);
              mma_ss_w(d, ka + kPlaneW, kb, idesc, 1u);
            }
            mma_commit(&bars.empty[stage]);
            if (kk == ks - 1) mma_commit(&bars.acc_full[ab]);
          }
          __syncwarp();
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
        ++local;
      });
    };
    for (int k = 0; k < st.steps && go; ++k) {
      multiply(Phase<1>{});
      multiply(Phase<2>{});
      multiply(Phase<3>{});
    }
  } else {
    constexpr int H = W / 2;  // columns of a warp
    const int quarter = warp & 3, half = (warp - 2) >> 2, r = quarter * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    uint8_t* stg = sm + kStages * kStage + quarter * G::kStg;  // this quarter's rows of the result
    uint32_t pphase = 0;
    auto pair_sync = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.pair[quarter]);
      go = go && __all_sync(0xffffffffu, mbar_wait(&bars.pair[quarter], pphase, st.wc, abort));
      pphase ^= 1;
      return go;
    };
    // 32 rows and columns, from c0 on, of a product's tile, f(column, accumulator), to
    // the images from `tile` on: two pieces of eight columns lie side by side, in the
    // order of the swizzle
    auto store = [&](uint8_t* tile, int c0, const uint32_t (&acc)[32], auto&& f) {
      tile += (c0 / 64) * kOrthTile + r * 128;
#pragma unroll
      for (int c = 0; c < 4; c += 2) {
        uint4 h[2], l[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = f(c0 + 8 * (c + p) + e, __uint_as_float(acc[8 * (c + p) + e]));
          split8(y, h[p], l[p]);
        }
        const bool odd = (lane & 1) != 0;
        uint8_t* to = tile + (((c0 % 64 / 8 + c) ^ (lane & 6)) << 4);
        st_global_32(to, odd ? h[1] : h[0], odd ? h[0] : h[1]);
        st_global_32(to + kOrthPlane, odd ? l[1] : l[0], odd ? l[0] : l[1]);
      }
    };
    constexpr float kBack = 1.f / kOrthScale;
    int local = 0;
    auto take = [&](auto which, int step) {
      constexpr int PHASE = decltype(which)::value;
      const int in = step & 1;
      const bool last = PHASE == 3 && step == st.steps - 1;  // X goes to the destinations
      tiles(which, [&](int k, int i, int j, int) {
        const OrthMat q = constant(v.mat + k);
        const int ab = local & 1;
        go = __all_sync(0xffffffffu, mbar_wait(&bars.acc_full[ab], (local >> 1) & 1, st.wc, abort));
        if (!go) return;
        ++local;
        tc_fence_after();
        const int row0 = i * 128 + quarter * 32, col0 = j * W;
        if (PHASE == 3 && last && !(q.flags & kOrthTall) && !pair_sync()) return;  // the staging has been read
        const int diag = i * 128 + r - col0;  // the column of this row's diagonal element
#pragma unroll
        for (int g = 0; g < H; g += 32) {
          const int c0 = H * half + g;
          uint32_t u[32];
          tmem_ld32_wait(tmem + lane_addr + ab * W + c0, u);
          if (g + 32 == H) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.acc_empty[ab]);
          }
          if constexpr (PHASE == 1) {
            const int t = i * 2 * q.mt + j * (W / 64);
            store(tile_at(v, q.a + t), c0, u, [&](int, float x) { return x * (kBack * kBack); });
            store(tile_at(v, q.a2 + t), c0, u, [&](int col, float x) {
              return st.c * (x * (kBack * kBack)) + (col == diag ? st.b : 0.f);
            });
          } else if constexpr (PHASE == 2) {
            store(tile_at(v, q.b + i * 2 * q.mt + j * (W / 64)), c0, u,
                  [&](int col, float x) { return x + (col == diag ? st.a : 0.f); });
          } else if (!last) {
            store(tile_at(v, (in != 0 ? q.x[0] : q.x[1]) + i * 2 * q.nt + j * (W / 64)), c0, u,
                  [&](int, float x) { return x; });
          } else if (q.flags & kOrthTall) {
            // a transposed matrix's rows are contiguous across lanes
            uint16_t* dst = static_cast<uint16_t*>(q.dst);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int col = col0 + c0 + e;
              if (row0 + lane < q.m && col < q.n)
                dst[col * q.ld_dst + row0 + lane] =
                    static_cast<uint16_t>(pack_bf16x2(__uint_as_float(u[e]) * kBack, 0.f) & 0xFFFFu);
            }
          } else {
            // the others go through the staging, blocks of 64 columns of BF16, swizzled
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack_bf16x2(__uint_as_float(u[8 * c + 2 * e]) * kBack,
                                   __uint_as_float(u[8 * c + 2 * e + 1]) * kBack);
              *reinterpret_cast<uint4*>(stg + (c0 / 64) * 4096 + sw128(lane, c0 % 64 / 8 + c)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        if (!last) {
          __syncwarp();
          if (lane == 0) red_release_gpu(v.done + k, 1u);
        } else if (!(q.flags & kOrthTall)) {
          if (!pair_sync()) return;
          uint16_t* dst = static_cast<uint16_t*>(q.dst);
#pragma unroll 1
          for (int blk = 0; blk < W / 64; ++blk) {
            const int r0 = 16 * half, rows = min(16, q.m - row0 - r0), cols = min(64, q.n - col0 - 64 * blk);
            const uint8_t* from = stg + blk * 4096;
            uint16_t* to = dst + (row0 + r0) * q.ld_dst + col0 + 64 * blk;
            if (cols == 64 && (reinterpret_cast<uintptr_t>(to) & 15) == 0 && q.ld_dst % 8 == 0) {
              for (int e = lane; e < rows * 8; e += 32)
                *reinterpret_cast<uint4*>(to + (e >> 3) * q.ld_dst + (e & 7) * 8) =
                    *reinterpret_cast<const uint4*>(from + sw128(r0 + (e >> 3), e & 7));
            } else {
              for (int rr = 0; rr < rows; ++rr)
                for (int e = lane; e < cols; e += 32)
                  to[rr * q.ld_dst + e] = reinterpret_cast<const uint16_t*>(from + sw128(r0 + rr, e >> 3))[e & 7];
            }
          }
        }
      });
    };
    for (int k = 0; k < st.steps && go; ++k) {
      take(Phase<1>{}, k);
      take(Phase<2>{}, k);
      take(Phase<3>{}, k);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) settle_if_aborted(abort);
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * W);
  }
}

// ------------------------------------------------------------------ host
// The list as the kernels take it: the matrices of one row of tiles (m <= 128)
// first, the widest in front, then the others, and where their parts lie in the
// workspace.
struct Plan {
  std::vector<OrthMat> mats;
  int solo = 0, team = 1, width = 64;  // width: of the products' tiles of the larger matrices
  long long parts = 0, load_tiles = 0, sq = 0, mn = 0, tiles = 0;
  size_t done_off = 0, part_off = 0, tiles_off = 0, total = 0;
};

bool dims_ok(const triattn_matrix& g) { return g.rows > 0 && g.cols > 0; }

// CTAs per matrix of one row of tiles.  A CTA takes about 1.7 k cycles per chunk
// of 64 columns and step, and 4 k (alone) or 7 k (in a team, which adds its parts
// of A) between two passes; the list takes as long as its widest matrix or as its
// sum spread over the SMs (clusters of eight leave some of a GPC's idle).  A single wide
// matrix has eight SMs at most: 128 x 4096 takes 99 us, x 16384 251, x 65536 870, and
// eight of these 1035 together.
int team_of(const OrthMat* q, int n) {
  int best = 1;
  double least = 0.0;
  for (int t = 1; t <= 8; t *= 2) {
    double widest = 0.0, sum = 0.0;
    for (int k = 0; k < n; ++k) {
      const int chunks = (q[k].n + 63) / 64;
      const double c = 1.7 * ((chunks + t - 1) / t) + (t > 1 ? 7.0 : 4.0);
      widest = std::max(widest, c);
      sum += c * t;
    }
    const double time = std::max(widest, sum / (t == 8 ? 128 : 152));
    if (t == 1 || time < least) {
      best = t;
      least = time;
    }
  }
  return best;
}

// Columns of the larger matrices' tiles.  A stage of 64 columns takes about 0.7 of a
// unit, one of 128 about 0.9 (the MMAs read A from shared memory for half as many
// columns), a tile about one stage more; narrow tiles give a short list's products to
// twice the SMs.  Both measured, five steps, us with 64 and with 128: one 300 x 300 93
// and 112, 8 of them 101 and 117, 64 of them 418 and 299; 4 of 256 x 1037 117 and 139,
// 12 143 and 158, 40 334 and 272; 512 x 1100 135 and 164, 12 of them 338 and 274, 40
// 1007 and 752 (378 TFLOP/s); 4 of 1024 x 4096 1223 and 790 (489 TFLOP/s).
int width_of(const OrthMat* q, int n) {
  double least = 0.0;
  int best = 64;
  for (int w = 64; w <= 128; w *= 2) {
    const double stage = w == 64 ? 0.7 : 0.9;
    double tiles[3] = {}, stages[3] = {}, widest[3] = {}, time = 0.0;
    for (int k = 0; k < n; ++k) {
      const double sq = 128.0 / w * q[k].mt * q[k].mt, mn = 128.0 / w * q[k].mt * q[k].nt;
      const double ks[3] = {(q[k].n + 63) / 64 + 1.0, (q[k].m + 63) / 64 + 1.0, (q[k].m + 63) / 64 + 1.0};
      for (int p = 0; p < 3; ++p) {
        const double t = p < 2 ? sq : mn;
        tiles[p] += t;
        stages[p] += t * ks[p];
        widest[p] = std::max(widest[p], ks[p]);
      }
    }
    for (int p = 0; p < 3 && n > 0; ++p)
      time += stage * std::max(widest[p], stages[p] / tiles[p] * std::ceil(tiles[p] / 152));
    if (w == 64 || time < least) {
      best = w;
      least = time;
    }
  }
  return best;
}

// false: more than the kernels' 32-bit counts hold
bool plan_of(const triattn_matrix* in, const triattn_matrix* out, long long n, Plan* p) {
  p->mats.reserve(static_cast<size_t>(n));
  for (long long k = 0; k < n; ++k) {
    if (!dims_ok(in[k])) continue;
    OrthMat q{};
    const int rows = static_cast<int>(in[k].rows), cols = static_cast<int>(in[k].cols);
    q.src = in[k].data;
    q.ld_src = in[k].stride;
    if (out != nullptr) {
      q.dst = out[k].data;
      q.ld_dst = out[k].stride;
    }
    q.flags = (in[k].dtype == TRIATTN_DTYPE_FP32 ? kOrthFp32 : 0) | (rows > cols ? kOrthTall : 0);
    q.m = std::min(rows, cols);
    q.n = std::max(rows, cols);
    q.mt = (q.m + 127) / 128;
    q.nt = (q.n + 127) / 128;
    const long long parts = (in[k].rows * in[k].cols + kNormPart - 1) / kNormPart;
    q.parts = static_cast<int>(parts);
    p->mats.push_back(q);
  }
  const auto others = std::stable_partition(p->mats.begin(), p->mats.end(), [](const OrthMat& q) { return q.mt == 1; });
  p->solo = static_cast<int>(others - p->mats.begin());
  std::stable_sort(p->mats.begin(), others, [](const OrthMat& x, const OrthMat& y) { return x.n > y.n; });
  p->team = team_of(p->mats.data(), p->solo);
  p->width = width_of(p->mats.data() + p->solo, static_cast<int>(p->mats.size()) - p->solo);
  for (OrthMat& q : p->mats) {
    const long long xt = 2ll * q.mt * q.nt, at = 2ll * q.mt * q.mt;
    q.part0 = static_cast<int>(p->parts);
    q.tiles0 = static_cast<int>(p->load_tiles);
    p->parts += q.parts;
    p->load_tiles += xt;
    q.x[0] = static_cast<int>(p->tiles);
    p->tiles += xt;
    if (q.mt > 1) {
      q.sq0 = static_cast<int>(p->sq);
      q.mn0 = static_cast<int>(p->mn);
      p->sq += at * 64 / p->width;
      p->mn += xt * 64 / p->width;
      q.x[1] = static_cast<int>(p->tiles);
      q.a = static_cast<int>(p->tiles + xt);
      q.a2 = static_cast<int>(p->tiles + xt + at);
      q.b = static_cast<int>(p->tiles + xt + 2 * at);
      p->tiles += xt + 3 * at;
    } else if (p->team > 1) {
      q.a = static_cast<int>(p->tiles);
      p->tiles += 2 * (p->team + 1);
    }
    if (p->tiles >= (1ll << 31) || p->parts >= (1ll << 31)) return false;
  }
  auto up = [](size_t x) { return (x + 1023) / 1024 * 1024; };
  p->done_off = up(p->mats.size() * sizeof(OrthMat));
  p->part_off = up(p->done_off + p->mats.size() * 4);
  p->tiles_off = up(p->part_off + static_cast<size_t>(p->parts) * sizeof(double));
  p->total = p->tiles_off + static_cast<size_t>(p->tiles) * kOrthTile;
  return true;
}

// Whether no two outputs share an element, as far as it can be told from where they
// start: ranges of memory that meet are those of blocks of columns of the same rows,
// apart by their columns (the parts of a fused projection), or they are taken to.
bool outputs_apart(const triattn_matrix* out, long long n) {
  struct Span {
    uintptr_t lo, hi;  // bytes
    uintptr_t row, step;
  };
  std::vector<Span> dst, open;  // open: those that may reach beyond the next one's start
  dst.reserve(static_cast<size_t>(n));
  for (long long i = 0; i < n; ++i) {
    if (!dims_ok(out[i])) continue;
    const uintptr_t a = reinterpret_cast<uintptr_t>(out[i].data), row = 2 * static_cast<uintptr_t>(out[i].cols);
    const uintptr_t step = out[i].rows > 1 ? 2 * static_cast<uintptr_t>(out[i].stride) : row;
    dst.push_back({a, a + static_cast<uintptr_t>(out[i].rows - 1) * step + row, row, out[i].rows > 1 ? step : 0});
  }
  std::sort(dst.begin(), dst.end(), [](const Span& x, const Span& y) { return x.lo < y.lo; });
  for (const Span& y : dst) {
    size_t kept = 0;
    for (const Span& x : open) {
      if (x.hi <= y.lo) continue;
      const uintptr_t step = std::max(x.step, y.step);
      if (step == 0 || (x.step != 0 && y.step != 0 && x.step != y.step)) return false;
      const uintptr_t col = (y.lo - x.lo) % step;  // y's first column, counted from x's, in x's rows
      if (col < x.row || col + y.row > step) return false;
      open[kept++] = x;
    }
    open.resize(kept);
    open.push_back(y);
  }
  return true;
}

constexpr long long kMaxSide = 65536;

triattn_status check_list(const triattn_matrix* ms, long long n, bool output) {
  if (n < 0 || (n > 0 && ms == nullptr)) return TRIATTN_ERR_INVALID_ARG;
  if (n > (1 << 20)) return TRIATTN_ERR_UNSUPPORTED;
  for (long long i = 0; i < n; ++i) {
    const triattn_matrix& g = ms[i];
    if (g.rows < 0 || g.cols < 0) return TRIATTN_ERR_INVALID_ARG;
    if (g.dtype != TRIATTN_DTYPE_BF16 && (output || g.dtype != TRIATTN_DTYPE_FP32)) return TRIATTN_ERR_UNSUPPORTED;
    if (!dims_ok(g)) continue;
    if (g.rows > kMaxSide || g.cols > kMaxSide) return TRIATTN_ERR_UNSUPPORTED;
    if (g.stride < g.cols || g.stride >= (1ll << 36)) return TRIATTN_ERR_INVALID_ARG;
    if (g.data == nullptr || (reinterpret_cast<uintptr_t>(g.data) & (g.dtype == TRIATTN_DTYPE_FP32 ? 3u : 1u)) != 0)
      return TRIATTN_ERR_INVALID_ARG;
  }
  return TRIATTN_OK;
}

template <int W>
cudaError_t launch_gemm(const OrthView& v, const OrthRun& st, cudaStream_t s) {
  constexpr int kSmem = Gemm<W>::kSmem;
  const cudaError_t e = cudaFuncSetAttribute(orth_gemm_kernel<W>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  int device = 0, sms = 0;
  if (cudaGetDevice(&device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
    return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(std::min(st.mn, sms));  // m <= n: no phase has more tiles
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeCooperative;
  at.val.cooperative = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, orth_gemm_kernel<W>, v, st);
}

cudaError_t run(const Plan& p, int steps, const float* co, float eps, uint8_t* ws, const WaitCtl& wc, cudaStream_t s) {
  OrthMat* mats = reinterpret_cast<OrthMat*>(ws);
  OrthView v{mats, reinterpret_cast<double*>(ws + p.part_off), ws + p.tiles_off,
             reinterpret_cast<uint32_t*>(ws + p.done_off),
             static_cast<int>(p.mats.size())};
  OrthTable t;
  const bool small = p.mats.size() <= static_cast<size_t>(kUpload);
  cudaError_t e = cudaSuccess;
  for (size_t k = 0; k < p.mats.size() && e == cudaSuccess; k += kUpload) {
    t.n = static_cast<int>(std::min<size_t>(kUpload, p.mats.size() - k));
    std::copy_n(p.mats.data() + k, t.n, t.mat);
    if (!small)
      e = trace_call(kKOrthLoad, s, [&] {
        return launch_after(k == 0, orth_table_kernel, (t.n + kTableRows - 1) / kTableRows, 32, 0, s, t, mats + k);
      });
  }
  if (e == cudaSuccess)
    e = trace_call(kKOrthLoad, s, [&] {
      return launch_after(small, small ? orth_norm_kernel<true> : orth_norm_kernel<false>,
                          static_cast<unsigned>(p.parts), 256, 0, s, t, v, mats);
    });
  if (e == cudaSuccess)
    e = trace_call(kKOrthLoad, s, [&] {
      return launch_after(false, orth_load_kernel, static_cast<unsigned>(p.load_tiles), 256, 0, s, v, eps);
    });
  if (p.solo > 0 && e == cudaSuccess)
    e = trace_call(kKOrthSolo, s, [&] {
      return launch_orth_solo(mats, p.solo, v.tiles, steps, OrthCoef{co[0], co[1], co[2]}, p.team, wc, s);
    });
  v.mat += p.solo;
  v.done += p.solo;
  v.n -= p.solo;
  const OrthRun st{co[0], co[1], co[2], steps, static_cast<int>(p.sq), static_cast<int>(p.mn), wc};
  if (v.n > 0 && e == cudaSuccess)
    e = trace_call(kKOrthGemm, s, [&] {
      return p.width == 64 ? launch_gemm<64>(v, st, s) : launch_gemm<128>(v, st, s);
    });
  return e;
}

}  // namespace
}  // namespace triattn

using namespace triattn;

extern "C" {

size_t triattn_orthogonalize_workspace_bytes(const triattn_matrix* matrices, long long n) {
  if (check_list(matrices, n, false) != TRIATTN_OK) return 0;
  try {
    Plan p;
    return plan_of(matrices, nullptr, n, &p) ? std::max<size_t>(p.total, 256) : 0;
  } catch (const std::bad_alloc&) {
    return 0;
  }
}

triattn_status triattn_orthogonalize(const triattn_matrix* matrices, const triattn_matrix* out, long long n, int steps,
                                     const float* coefficients, float eps, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  triattn_status st = check_list(matrices, n, false);
  if (st == TRIATTN_OK) st = check_list(out, n, true);
  if (st != TRIATTN_OK) return st;
  if (coefficients == nullptr || steps < 1 || !(eps > 0.f) || !std::isfinite(eps)) return TRIATTN_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (!std::isfinite(coefficients[i])) return TRIATTN_ERR_INVALID_ARG;
  if (steps > 64) return TRIATTN_ERR_UNSUPPORTED;
  for (long long i = 0; i < n; ++i)
    if (out[i].rows != matrices[i].rows || out[i].cols != matrices[i].cols) return TRIATTN_ERR_INVALID_ARG;
  try {
    // outputs are written without an order between them; every input is read
    // before the first of them
    if (!outputs_apart(out, n)) return TRIATTN_ERR_INVALID_ARG;
    Plan p;
    if (!plan_of(matrices, out, n, &p)) return TRIATTN_ERR_UNSUPPORTED;
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
        workspace_bytes < std::max<size_t>(p.total, 256))
      return TRIATTN_ERR_WORKSPACE;
    if (p.mats.empty()) return TRIATTN_OK;
    const WaitCtl wc = current_wait_ctl();
    if (wc.status == nullptr) return TRIATTN_ERR_CUDA;
    const cudaError_t e = run(p, steps, coefficients, eps, static_cast<uint8_t*>(workspace), wc,
                              static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TRIATTN_OK : TRIATTN_ERR_CUDA;
  } catch (const std::bad_alloc&) {
    return TRIATTN_ERR_WORKSPACE;
  }
}

}  // extern "C"
