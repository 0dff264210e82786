// What the kernels of the relative position bias share (relpos.cu, relpos_pairs.cu).
#pragma once
#include <cstddef>
#include <cstdint>

#include "kernels.cuh"

namespace triattn {

constexpr int kRelposMaxDistance = 1024;  // the list of buckets travels with the launch
constexpr int kRelposMaxBuckets = 256;    // a bucket is a byte of it
constexpr int kRelposMaxN = 16384;        // positions and chains of an example in shared memory
constexpr int kRelposMaxF = 256;          // pair features

struct RelposArgs {
  const float* table;    // [buckets, F]
  const uint16_t* base;  // or null
  uint16_t* out;
  const int* pos;        // [B, N] or null: the token's index
  const int* chain;      // [B, N] or null: one chain
  float* part;           // gradient: partial sums
  int B, N, F, R, buckets;
  uint8_t lut[2 * kRelposMaxDistance + 1];  // the bucket of distance d at [d + R]
  __device__ __forceinline__ int position(int b, int n) const {
    return pos != nullptr ? __ldg(pos + static_cast<size_t>(b) * N + n) : n;
  }
};

// The difference of two positions cut off at +-R, plus R (the difference itself
// is cut off at the ends of 32 bits).
__device__ __forceinline__ int distance(int pi, int pj, int R) {
  int d;
  asm("sub.sat.s32 %0, %1, %2;" : "=r"(d) : "r"(pi), "r"(pj));
  return min(max(d, -R), R) + R;
}

// Pair features' gradient (relpos_pairs.cu): partial sums [parts][buckets][F] of
// d_out [B, N, N, F] (BF16) into a.part.
int relpos_pairs_parts(int B, int N);
cudaError_t launch_relpos_pairs_bwd(const RelposArgs& a, const void* d_out, int parts, const WaitCtl& wc,
                                    cudaStream_t s);

}  // namespace triattn
