// The relative position bias's gradient for pair features: with P pairs of F
// features and one-hot rows e(pair) of their buckets,
//
//   d_table^T [F, buckets] = d_out^T [F, P] . e [P, buckets]
//
// on the tensor cores: a product by 0 or 1 is exact, so this is a sum of d_out's
// BF16 values in FP32 accumulators, whatever the order of the buckets, with no
// atomics and no private copies of the table (34 KB each at 66 x 128).  The
// products are 2 P F buckets operations, 10 us of the tensor cores at 768^2
// pairs, 128 features and 66 buckets, against 22 us for the bytes of d_out,
// which bound it.
//
// 640^2 pairs, 128 features, 66 buckets (105 MB): 28 us with the sum of the runs' tables
// (5 MB); 1920^2 pairs 5.6 TB/s.  Short lists pay the start: barriers, TMEM, the first
// stages, the last accumulators take 5 us.
//
// One CTA per run of pairs, ten warps:
//   warp 0     TMA: per 64 pairs the rows of d_out as 64-feature boxes (128-byte
//              swizzle), which are A, features contiguous (MN-major).
//   warp 1     MMA issuer: per 64 pairs and 128 features four M = 128,
//              N = buckets (to 16), K = 16 MMAs.  Up to four accumulators take
//              turns, and a run is at most kRun blocks of 64 pairs, so that no
//              accumulator adds more than 4 kRun products of 16: the tensor
//              cores cut off what an FP32 accumulator cannot hold.
//   warps 2-9  one pair per thread, two warps per stage, in turn: its bucket (of
//              the next stage while they wait for this one), then the two bytes of
//              its one in B [buckets, 64 pairs] (K-major, swizzled), after the one
//              that the stage held before is put out.
// At the end eight warps add the accumulators and write the run's partial table.  A value
// that is not finite makes all buckets of its feature NaN in the product (0 x inf); the
// run's sums of such a feature are then added up one by one (640^2 pairs, 128 features:
// 2.4 ms with one infinity, 3.1 ms with no finite value at all).
#include <cudaTypedefs.h>

#include <algorithm>

#include "kernels.cuh"
#include "relpos.cuh"

namespace triattn {
namespace {

constexpr int kBlk = 64;     // pairs per stage
constexpr int kRun = 128;    // stages per CTA at most
constexpr int kStagesMax = 8;
constexpr uint16_t kNone = 0xFFFF;  // no one in the column
constexpr int kSmemMax = 220 * 1024;

struct Bars {
  uint64_t full[kStagesMax], empty[kStagesMax], done;
  uint32_t tmem_slot;
  int abort;
};

struct PairsBwd {
  long long P;                  // pairs
  int nb, mt, sets, stages;     // buckets to 16, 128-feature tiles, accumulators per tile, ring stages
  int groups;                   // that place the ones, a divisor of the stages: a stage's ones are always one group's
  int stage_bytes, a_bytes;
  const uint16_t* d_out;
  WaitCtl wc;
};

constexpr int kGroups = 4;  // of two warps that place the ones
constexpr int kPairThreads = 64 + 64 * kGroups;

// Sums of feature f over the pairs [q0, q1) of the 16 buckets from k0 on, into `out`, by
// one thread; `cell` is its place in shared memory, sums 128 apart.
__device__ __noinline__ void add_one_by_one(const RelposArgs& a, const uint16_t* d_out, const uint8_t* lut, long long q0,
                                            long long q1, int f, int k0, float2* cell, float* out) {
  for (int e = 0; e < 16; ++e) cell[128 * e] = make_float2(0.f, 0.f);
  const long long NN = static_cast<long long>(a.N) * a.N;
  int b = static_cast<int>(q0 / NN), i = static_cast<int>((q0 - b * NN) / a.N);
  int j = static_cast<int>(q0 - b * NN - static_cast<long long>(i) * a.N);
  for (long long q = q0; q < q1; ++q) {
    const size_t at = static_cast<size_t>(b) * a.N;
    const bool other = a.chain != nullptr && __ldg(a.chain + at + i) != __ldg(a.chain + at + j);
    const int k = (other ? a.buckets - 1 : lut[distance(a.position(b, i), a.position(b, j), a.R)]) - k0;
    if (k >= 0 && k < 16) {
      Sum2 v{cell[128 * k].x, cell[128 * k].y};
      v.add(bf16lo_to_f32(__ldg(d_out + q * a.F + f)));
      cell[128 * k] = v.pair();
    }
    if (++j == a.N) {
      j = 0;
      if (++i == a.N) {
        i = 0;
        ++b;
      }
    }
  }
  for (int e = 0; e < 16 && k0 + e < a.buckets; ++e)
    out[static_cast<size_t>(k0 + e) * a.F + f] = Sum2{cell[128 * e].x, cell[128 * e].y}.value();
}

__global__ void __launch_bounds__(kPairThreads, 1) relpos_pairs_bwd_kernel(const __grid_constant__ CUtensorMap tm,
                                                                  const __grid_constant__ RelposArgs a, PairsBwd p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Bars bars;
  __shared__ uint8_t lut[2 * kRelposMaxDistance + 1];
  __shared__ uint16_t held[kStagesMax][kBlk];  // where the stage's ones lie (element of B)
  let_next_start();
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int* abort = &bars.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int d = threadIdx.x; d <= 2 * a.R; d += kPairThreads) lut[d] = a.lut[d];
  const long long blocks = (p.P + kBlk - 1) / kBlk;
  const long long b0 = blocks * blockIdx.x / gridDim.x, b1 = blocks * (blockIdx.x + 1) / gridDim.x;
  const int n = static_cast<int>(b1 - b0);
  // the stages' B, of zeros at first
  const int pieces = p.nb * 8, used_stages = min(n, p.stages);
  for (int e = threadIdx.x; e < used_stages * pieces; e += kPairThreads) {
    const int stage = e / pieces;
    *reinterpret_cast<uint4*>(sm + stage * p.stage_bytes + p.a_bytes + (e - stage * pieces) * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&bars.full[s], 1 + 2);
      mbar_init(&bars.empty[s], 1);
    }
    mbar_init(&bars.done, 1);
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&bars.tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_slot;
  const int boxes = (a.F + 63) / 64;

  if (warp == 0) {
    if (lane == 0) {
      prefetch_tmap(&tm);
      int stage = 0, phase = 0;
      for (int k = 0; k < n; ++k) {
        if (!mbar_wait(&bars.empty[stage], phase ^ 1, p.wc, abort)) break;
        if (p.wc.starve == 0 || blockIdx.x != 0 || k != 0) {
          mbar_expect_tx(&bars.full[stage], boxes * kBlk * 128);
          for (int x = 0; x < boxes; ++x)
            tma_load_3d(sm + stage * p.stage_bytes + x * kBlk * 128, &tm, &bars.full[stage], 64 * x,
                        static_cast<int>((b0 + k) * kBlk), 0);
        }
        if (++stage == p.stages) { stage = 0; phase ^= 1; }
      }
    }
  } else if (warp == 1) {
    const uint32_t idesc = idesc_bf16_f32(128, p.nb, 1, 0);
    // operands by the low words of their descriptors: what the one issuing thread
    // computes per stage has to stay below the 700 cycles that a stage's bytes take
    const uint32_t s0 = smem_u32(sm) >> 4, stage_w = p.stage_bytes / 16;
    const uint32_t a0 = s0 | (kBlk * 128 / 16) << 16, e0 = (s0 + p.a_bytes / 16) | (1u << 16);
    const uint32_t set_cols = p.mt * p.nb;
    int stage = 0, phase = 0, set = 0;
    for (int k = 0; k < n; ++k) {
      if (!__all_sync(0xffffffffu, mbar_wait(&bars.full[stage], phase, p.wc, abort))) break;
      tc_fence_after();
      const uint32_t xa = a0 + stage * stage_w, xe = e0 + stage * stage_w, d = tmem + set * set_cols;
      const uint32_t more = k >= p.sets ? 1u : 0u;
      if (elect_one()) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          if (m == p.mt) break;
#pragma unroll
          for (int k16 = 0; k16 < kBlk / 16; ++k16)
            mma_ss_w(d + m * p.nb, xa + m * (2 * kBlk * 128 / 16) + k16 * 128, xe + k16 * 2, idesc, k16 > 0 ? 1u : more);
        }
        mma_commit(&bars.empty[stage]);
        if (k == n - 1) mma_commit(&bars.done);
      }
      __syncwarp();
      if (++set == p.sets) set = 0;
      if (++stage == p.stages) { stage = 0; phase ^= 1; }
    }
  } else {
    const int c = threadIdx.x & 63, group = (warp - 2) >> 1;  // the pair of the block
    long long q = (b0 + group) * kBlk + c;
    const long long NN = static_cast<long long>(a.N) * a.N;
    int b = static_cast<int>(q / NN), i = static_cast<int>((q - b * NN) / a.N);
    int j = static_cast<int>(q - b * NN - static_cast<long long>(i) * a.N);
    auto bucket = [&]() {  // of pair (b, i, j); none past the last
      if (q >= p.P) return -1;
      const size_t at = static_cast<size_t>(b) * a.N;
      const bool other = a.chain != nullptr && __ldg(a.chain + at + i) != __ldg(a.chain + at + j);
      return other ? a.buckets - 1 : static_cast<int>(lut[distance(a.position(b, i), a.position(b, j), a.R)]);
    };
    auto next = [&]() {  // to the group's next block
      q += p.groups * kBlk;
      j += p.groups * kBlk;
      if (j >= a.N) {
        const int w = j / a.N;
        j -= w * a.N;
        i += w;
        if (i >= a.N) {
          const int v = i / a.N;
          i -= v * a.N;
          b += v;
        }
      }
    };
    int row = bucket();
    for (int k = group; k < n && group < p.groups; k += p.groups) {
      const int stage = k % p.stages, phase = (k / p.stages) & 1;
      next();
      const int row_next = k + p.groups < n ? bucket() : -1;
      if (!__all_sync(0xffffffffu, mbar_wait(&bars.empty[stage], phase ^ 1, p.wc, abort))) break;
      uint16_t* e = reinterpret_cast<uint16_t*>(sm + stage * p.stage_bytes + p.a_bytes);
      if (k >= p.stages && held[stage][c] != kNone) e[held[stage][c]] = 0;
      const uint16_t at = row >= 0 ? static_cast<uint16_t>(sw128(row, c >> 3) / 2 + (c & 7)) : kNone;
      if (at != kNone) e[at] = 0x3F80;  // 1
      held[stage][c] = at;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.full[stage]);
      row = row_next;
    }
  }
  __syncwarp();
  const bool ok = __all_sync(0xffffffffu, mbar_wait(&bars.done, 0, p.wc, abort));
  tc_fence_after();
  if (ok && warp < 8) {  // two warps to a quarter of the features, buckets in turn
    float* out = a.part + static_cast<size_t>(blockIdx.x) * a.buckets * a.F;
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int used = min(n, p.sets);
    for (int m = 0; m < p.mt; ++m) {
      const int f = m * 128 + (warp & 3) * 32 + lane;
      float worst = 0.f;  // not finite where a sum is not
      for (int k0 = warp < 4 ? 0 : 16; k0 < p.nb; k0 += 32) {
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0.f;
        for (int s = 0; s < used; ++s) {
          uint32_t r[16];
          tmem_ld16_wait(tmem + lane_addr + (s * p.mt + m) * p.nb + k0, r);
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] += __uint_as_float(r[e]);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          worst += 0.f * v[e];
          if (f < a.F && k0 + e < a.buckets) out[static_cast<size_t>(k0 + e) * a.F + f] = v[e];
        }
      }
      if (f < a.F && worst != 0.f) {  // the ring's memory: all products are done
        float2* cell = reinterpret_cast<float2*>(sm) + (warp < 4 ? 0 : 16 * 128) + (warp & 3) * 32 + lane;
        for (int k0 = warp < 4 ? 0 : 16; k0 < a.buckets; k0 += 32)
          add_one_by_one(a, p.d_out, lut, b0 * kBlk, min(b1 * kBlk, p.P), f, k0, cell, out);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) settle_if_aborted(abort);
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

int relpos_pairs_parts(int B, int N) {
  const long long blocks = (static_cast<long long>(B) * N * N + kBlk - 1) / kBlk;
  // a wave of CTAs, or as many whole waves as keep the runs short
  const long long waves = (blocks + 152ll * kRun - 1) / (152ll * kRun);
  return static_cast<int>(std::min(blocks, 152 * waves));
}

cudaError_t launch_relpos_pairs_bwd(const RelposArgs& a, const void* d_out, int parts, const WaitCtl& wc,
                                    cudaStream_t s) {
  auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (encode == nullptr || wc.status == nullptr) return cudaErrorNotSupported;
  PairsBwd p;
  p.P = static_cast<long long>(a.B) * a.N * a.N;
  p.nb = (a.buckets + 15) / 16 * 16;
  p.mt = (a.F + 127) / 128;
  p.sets = std::min(4, 512 / (p.nb * p.mt));
  p.a_bytes = p.mt * 2 * kBlk * 128;
  p.stage_bytes = p.a_bytes + p.nb * 128;
  p.stage_bytes = (p.stage_bytes + 1023) / 1024 * 1024;
  p.stages = std::min(kStagesMax, (kSmemMax - 1024) / p.stage_bytes);
  p.groups = p.stages >= kGroups ? kGroups : 2;
  p.stages -= p.stages % p.groups;
  p.d_out = static_cast<const uint16_t*>(d_out);
  p.wc = wc;
  CUtensorMap tm;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.F), static_cast<cuuint64_t>(p.P), 1};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(a.F) * 2, static_cast<cuuint64_t>(a.F) * 2 * p.P};
  const cuuint32_t box[3] = {64u, kBlk, 1u}, es[3] = {1u, 1u, 1u};
  if (encode(&tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(d_out), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const cudaError_t e =
      cudaFuncSetAttribute(relpos_pairs_bwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
  if (e != cudaSuccess) return e;
  // all of an SM's shared memory, so that one CTA runs on it: it takes all of TMEM
  relpos_pairs_bwd_kernel<<<parts, kPairThreads, kSmemMax, s>>>(tm, a, p);
  return cudaGetLastError();
}

}  // namespace triattn
