// What the kernels of the orthogonalisation share (orthogonalize.cu, orth_solo.cu).
#pragma once
#include <cuda_fp16.h>

#include <cstddef>
#include <cstdint>

#include "kernels.cuh"

namespace triattn {

constexpr int kOrthTile = 32768;     // bytes of a tile, hi and lo
constexpr int kOrthPlane = 16384;
constexpr float kOrthScale = 256.f;  // what is stored of a value

// One matrix of the list, as the kernels see it.
struct OrthMat {
  const void* src;
  void* dst;
  long long ld_src, ld_dst;  // elements between rows
  int m, n;                  // X
  int flags;                 // kOrthFp32: the source is FP32; kOrthTall: X is the transposed matrix
  int mt, nt;                // 128-row and 128-column tiles of X
  int x[2], a, a2, b;        // tiles of X (two copies), A, A', B'; a team's: X, and 2 (team + 1) at a
  int parts, part0;          // partial sums of squares
  int tiles0, sq0, mn0;      // 128 x 64 tiles of X (all matrices), of A and of X (several rows of tiles) before it
};
constexpr int kOrthFp32 = 1, kOrthTall = 2;

struct OrthView {
  const OrthMat* mat;
  double* part;
  uint8_t* tiles;
  uint32_t* done;  // tiles (by warps) that have been stored, of every larger matrix
  int n;
};
__device__ __forceinline__ uint8_t* tile_at(const OrthView& v, int t) {
  return v.tiles + static_cast<size_t>(t) * kOrthTile;
}

// Eight values as FP16 pairs, one 16-byte piece of each plane: hi is the value's
// leading 11 bits (cut off, so that no conversion back is needed), lo the rest
// rounded.  Below 2^-14 FP16 has fewer bits and rounds hi as well, to 2^-25 at most,
// which lo does not see: the floor of a pair is 2^-25 for hi and as much for lo.
__device__ __forceinline__ void split8(const float* y, uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float a = __uint_as_float(__float_as_uint(y[2 * e]) & 0xFFFFE000u);
    const float b = __uint_as_float(__float_as_uint(y[2 * e + 1]) & 0xFFFFE000u);
    h[e] = pack_f16x2(a, b);
    l[e] = pack_f16x2(y[2 * e] - a, y[2 * e + 1] - b);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// The values again.
__device__ __forceinline__ void join8(const uint4& hi, const uint4& lo, float* y) {
  const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h[e]));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&l[e]));
    y[2 * e] = a.x + b.x;
    y[2 * e + 1] = a.y + b.y;
  }
}

// A step's coefficients.
struct OrthCoef {
  float a, b, c;
};

// All steps of n matrices of at most 128 rows (X), clusters of `team` CTAs per
// matrix (1, 2, 4 or 8).
cudaError_t launch_orth_solo(const OrthMat* mats, int n, uint8_t* tiles, int steps, const OrthCoef& co, int team,
                             const WaitCtl& wc, cudaStream_t s);

}  // namespace triattn
