// The orthogonalisation's steps for matrices whose X has at most 128 rows (every
// projection of a pair stack of 128 features): one kernel for all steps, a CTA
// or a cluster ("team") of 2, 4 or 8 per matrix, X cut along its columns.
//
// B' [128, 128] stays in shared memory and A in TMEM, and a step is one pass over
// the CTA's columns, 64 at a time: D = B' X_c, the epilogue turns D into the new
// X_c in the place of the old one, and A += X_c X_c^T for the next step follows at
// once, so a chunk is touched once per step and not once per product.  Up to five
// chunks per CTA stay in shared memory for all steps; more go through L2 (the
// working set of all CTAs, 64 KB a chunk, fits it).  Between two passes the team
// adds its parts of A through distributed shared memory, every CTA one band of
// rows, in the order of the ranks, and every CTA then makes all of B' = b A + c A^2
// + a I.
//
//   warp 0     loads of X's chunks (ring of five)
//   warp 1     MMAs: 24 of N = 64 for D and 12 of N = m for A per chunk, each three
//              products of FP16 pairs; 24 of N = m for A^2 per step
//   warps 2-9  D to X, A and A^2 to B': thread = row, 32 or 64 columns
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "kernels.cuh"
#include "orthogonalize.cuh"

namespace triattn {
namespace {

constexpr int kRing = 5;
constexpr int kB = 2 * kOrthTile;  // A, then B', as two tiles of 64 columns
constexpr int kSmem = kB + kRing * kOrthTile + 1024;
constexpr int kWarps = 8;  // epilogue
constexpr int kThreads = (2 + kWarps) * 32;
constexpr uint32_t kColA = 0, kColA2 = 128, kColD = 256;

struct SoloBars {
  uint64_t full[kRing];    // a chunk has been loaded
  uint64_t ready[kRing];   // the new chunk stands in the slot
  uint64_t used[kRing];    // the last product that reads the slot is done
  uint64_t stored[kRing];  // the slot has been copied out
  uint64_t dfull[2], dfree[2];
  uint64_t afull, aready, a2full, bready;
  uint64_t saved;          // a pass's chunks are in memory
  uint64_t team;
  uint64_t pair[4];        // the two warps of a quarter of the rows
  uint32_t tmem_slot;
  int abort;
};

__global__ void __launch_bounds__(kThreads, 1) orth_solo_kernel(const OrthMat* mats, uint8_t* tiles, int steps,
                                                                OrthCoef co, int T, WaitCtl wc) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ SoloBars bars;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = sm + kB;
  volatile int* abort = &bars.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = T > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const OrthMat q = mats[blockIdx.x / T];
  const int chunks = (q.n + 63) / 64;
  const int c0 = chunks * rank / T, nloc = chunks * (rank + 1) / T - c0;
  const bool resident = nloc <= kRing;
  uint8_t* const xt = tiles + static_cast<size_t>(q.x[0] + c0) * kOrthTile;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.ready[i], kWarps);
      mbar_init(&bars.used[i], 1);
      mbar_init(&bars.stored[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.dfull[i], 1);
      mbar_init(&bars.dfree[i], kWarps);
    }
    mbar_init(&bars.afull, 1);
    mbar_init(&bars.aready, kWarps);
    mbar_init(&bars.a2full, 1);
    mbar_init(&bars.bready, kWarps);
    mbar_init(&bars.saved, 4);
    mbar_init(&bars.team, T * kWarps);
    for (int i = 0; i < 4; ++i) mbar_init(&bars.pair[i], 2);
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&bars.tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  if (T > 1) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      // use g of the ring: chunk g % nloc of pass g / nloc; a slot is free when its
      // product is done and, from pass 1 on, its copy out too
      const int total = resident ? nloc : nloc * (steps + 1);
      uint32_t used = 0, stored = 0;  // phases, a bit per slot
      for (int g = 0; g < total; ++g) {
        const int slot = g % kRing, pass = g / nloc, c = g - pass * nloc;
        if (g >= kRing) {
          if (!mbar_wait(&bars.used[slot], (used >> slot) & 1, wc, abort)) break;
          used ^= 1u << slot;
          if (g - kRing >= nloc) {
            if (!mbar_wait(&bars.stored[slot], (stored >> slot) & 1, wc, abort)) break;
            stored ^= 1u << slot;
          }
        }
        if (c == 0 && pass >= 2) {
          if (!mbar_wait(&bars.saved, (pass - 2) & 1, wc, abort)) break;
          fence_proxy_async_all();
        }
        mbar_expect_tx(&bars.full[slot], kOrthTile);
        bulk_load(ring + slot * kOrthTile, xt + static_cast<size_t>(c) * kOrthTile, kOrthTile, &bars.full[slot]);
      }
    }
  } else if (warp == 1) {
    const int k16 = (q.m + 15) / 16;  // K = m and N = m, to 16
    const uint32_t ia = idesc_f16_f32(128, 16 * k16, 0, 0), id = idesc_f16_f32(128, 64, 0, 1);
    const uint32_t sB = smem_u32(sm), sR = smem_u32(ring);
    uint32_t full = 0, ready = 0;
    int dn = 0;  // accumulators D used
    bool go = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      go = go && __all_sync(0xffffffffu, mbar_wait(bar, parity, wc, abort));
      tc_fence_after();
      return go;
    };
    // the three products of 16 of K; descriptors by plane
    auto products = [&](uint32_t d, uint32_t a, uint32_t b, bool b_mn, uint32_t idesc, bool first) {
      const uint64_t a0 = smem_desc(a, 16, 1024, 2), a1 = smem_desc(a + kOrthPlane, 16, 1024, 2);
      const uint64_t b0 = b_mn ? smem_desc(b, 8192, 1024, 2) : smem_desc(b, 16, 1024, 2);
      const uint64_t b1 = b_mn ? smem_desc(b + kOrthPlane, 8192, 1024, 2) : smem_desc(b + kOrthPlane, 16, 1024, 2);
      mma_ss(d, a0, b0, idesc, first ? 0u : 1u);
      mma_ss(d, a0, b1, idesc, 1u);
      mma_ss(d, a1, b0, idesc, 1u);
    };
    auto add_chunk = [&](int slot, bool first, bool last) {  // A += X_c X_c^T
      if (elect_one()) {
        const uint32_t x = sR + slot * kOrthTile;
#pragma unroll
        for (int k = 0; k < 4; ++k) products(tmem + kColA, x + k * 32, x + k * 32, false, ia, first && k == 0);
        mma_commit(&bars.used[slot]);
        if (last) mma_commit(&bars.afull);
      }
      __syncwarp();
    };
    int g = 0;
    for (int c = 0; c < nloc && go; ++c, ++g) {
      const int slot = g % kRing;
      if (!wait(&bars.full[slot], (full >> slot) & 1)) break;
      full ^= 1u << slot;
      add_chunk(slot, c == 0, c == nloc - 1);
    }
    if (nloc == 0 && elect_one()) mma_commit(&bars.afull);
    __syncwarp();
    for (int p = 1; p <= steps && go; ++p) {
      if (!wait(&bars.aready, (p - 1) & 1)) break;
      if (elect_one()) {  // A^2: A is its own transposed
        for (int k = 0; k < k16; ++k) {
          const uint32_t at = sB + (k >> 2) * kOrthTile + (k & 3) * 32;
          products(tmem + kColA2, at, at, false, ia, k == 0);
        }
        mma_commit(&bars.a2full);
      }
      __syncwarp();
      if (!wait(&bars.bready, (p - 1) & 1)) break;
      const bool last = p == steps;
      const int g0 = g;
      auto slot_of = [&](int c) { return resident ? c : (g0 + c) % kRing; };
      auto add_ready = [&](int c) {
        const int slot = slot_of(c);
        if (!wait(&bars.ready[slot], (ready >> slot) & 1)) return;
        ready ^= 1u << slot;
        add_chunk(slot, c == 0, c == nloc - 1);
      };
      for (int c = 0; c < nloc && go; ++c, ++g) {
        const int slot = slot_of(c), db = dn & 1;
        if (!resident) {
          if (!wait(&bars.full[slot], (full >> slot) & 1)) break;
          full ^= 1u << slot;
        }
        if (!wait(&bars.dfree[db], ((dn >> 1) & 1) ^ 1)) break;
        if (elect_one()) {  // D = B' X_c, X_c [rows of K, 64 columns] as it lies
          const uint32_t x = sR + slot * kOrthTile;
          for (int k = 0; k < k16; ++k)
            products(tmem + kColD + 64 * db, sB + (k >> 2) * kOrthTile + (k & 3) * 32, x + k * 2048, true, id, k == 0);
          mma_commit(&bars.dfull[db]);
          if (last) mma_commit(&bars.used[slot]);
        }
        __syncwarp();
        ++dn;
        if (!last && c > 0) add_ready(c - 1);
      }
      if (!last && go) {
        if (nloc > 0) add_ready(nloc - 1);
        else if (elect_one()) mma_commit(&bars.afull);
        __syncwarp();
      }
    }
  } else {
    const int quarter = warp & 3, half = (warp - 2) >> 2, r = quarter * 32 + lane;
    const int te = threadIdx.x - 64;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    constexpr float kBack = 1.f / kOrthScale;  // products carry the scale twice
    uint32_t tphase = 0, pphase = 0;
    int dn = 0, g = resident ? 0 : nloc, last_slot = -1;
    bool go = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      go = go && __all_sync(0xffffffffu, mbar_wait(bar, parity, wc, abort));
      tc_fence_after();
      return go;
    };
    auto arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    auto team_sync = [&]() {
      __syncwarp();
      if (lane < T) mbar_arrive_cluster(&bars.team, lane);
      go = go && __all_sync(0xffffffffu, mbar_wait<true>(&bars.team, tphase, wc, abort));
      tphase ^= 1;
      return go;
    };
    auto pair_sync = [&]() {
      arrive(&bars.pair[quarter]);
      go = go && __all_sync(0xffffffffu, mbar_wait(&bars.pair[quarter], pphase, wc, abort));
      pphase ^= 1;
      return go;
    };
    uint8_t* const mine = sm + half * kOrthTile;  // this thread's 64 columns of A and B'
    for (int p = 1; p <= steps; ++p) {
      const bool last = p == steps;
      // ---- A to shared memory: the CTA's own, or the team's sum
      if (!wait(&bars.afull, (p - 1) & 1)) break;
      if (T == 1) {
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t v[32];
          tmem_ld32_wait(lane_addr + kColA + 64 * half + 32 * h, v);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(v[8 * c + e]) * kBack;
            uint4 hi, lo;
            split8(y, hi, lo);
            *reinterpret_cast<uint4*>(mine + sw128(r, 4 * h + c)) = hi;
            *reinterpret_cast<uint4*>(mine + kOrthPlane + sw128(r, 4 * h + c)) = lo;
          }
        }
      } else {
        const int RL = 128 / T, band = kB / T;
        if (!team_sync()) break;  // nobody reads its B' any more
        const uint32_t to = cluster_addr(sm + rank * band, r / RL);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t v[32];
          if (nloc > 0) {
            tmem_ld32_wait(lane_addr + kColA + 64 * half + 32 * h, v);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = 0u;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k)
            st_cluster_v4(to + ((half * 16 + h * 8 + k) * RL + r % RL) * 16,
                          make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]));
        }
        if (!team_sync()) break;  // the band's parts are here
        const int units = RL * 16;  // of eight columns
        float y[4][8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int u = te + 256 * k;
          if (u >= units) break;
#pragma unroll
          for (int e = 0; e < 8; ++e) y[k][e] = 0.f;
          for (int t = 0; t < T; ++t) {
            const float4* f = reinterpret_cast<const float4*>(sm + t * band) + 2 * (u / RL) * RL + u % RL;
            const float4 f0 = f[0], f1 = f[RL];
            y[k][0] += f0.x;
            y[k][1] += f0.y;
            y[k][2] += f0.z;
            y[k][3] += f0.w;
            y[k][4] += f1.x;
            y[k][5] += f1.y;
            y[k][6] += f1.z;
            y[k][7] += f1.w;
          }
        }
        if (!team_sync()) break;  // and have been read: A takes their place
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int u = te + 256 * k;
          if (u >= units) break;
          const int row = rank * RL + u % RL, ch = u / RL;
#pragma unroll
          for (int e = 0; e < 8; ++e) y[k][e] *= kBack;
          uint4 hi, lo;
          split8(y[k], hi, lo);
          uint8_t* at = sm + (ch >> 3) * kOrthTile + sw128(row, ch & 7);
          for (int t = 0; t < T; ++t) {
            st_cluster_v4(cluster_addr(at, t), hi);
            st_cluster_v4(cluster_addr(at + kOrthPlane, t), lo);
          }
        }
        fence_proxy_async_all();
        if (!team_sync()) break;
      }
      fence_proxy_async_smem();
      tc_fence_before();
      arrive(&bars.aready);
      // ---- B' = b A + c A^2 + a I over A
      if (!wait(&bars.a2full, (p - 1) & 1)) break;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        uint32_t v[32];
        tmem_ld32_wait(lane_addr + kColA2 + 64 * half + 32 * h, v);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint4* ph = reinterpret_cast<uint4*>(mine + sw128(r, 4 * h + c));
          uint4* pl = reinterpret_cast<uint4*>(mine + kOrthPlane + sw128(r, 4 * h + c));
          float y[8];
          join8(*ph, *pl, y);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y[e] = co.b * y[e] + co.c * (__uint_as_float(v[8 * c + e]) * kBack);
            if (64 * half + 32 * h + 8 * c + e == r) y[e] += co.a * kOrthScale;
          }
          uint4 hi, lo;
          split8(y, hi, lo);
          *ph = hi;
          *pl = lo;
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      arrive(&bars.bready);
      // ---- the chunks
      for (int c = 0; c < nloc; ++c, ++dn) {
        const int db = dn & 1, slot = resident ? c : (g + c) % kRing;
        if (!wait(&bars.dfull[db], (dn >> 1) & 1)) break;
        uint32_t v[32];
        tmem_ld32_wait(lane_addr + kColD + 64 * db + 32 * half, v);
        tc_fence_before();
        arrive(&bars.dfree[db]);
        uint8_t* x = ring + slot * kOrthTile;
        if (!last) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(v[8 * k + e]) * kBack;
            uint4 hi, lo;
            split8(y, hi, lo);
            *reinterpret_cast<uint4*>(x + sw128(r, 4 * half + k)) = hi;
            *reinterpret_cast<uint4*>(x + kOrthPlane + sw128(r, 4 * half + k)) = lo;
          }
          fence_proxy_async_smem();
          arrive(&bars.ready[slot]);
          if (!resident) {
            if (!pair_sync()) break;  // both halves of the quarter's rows
            if (half == 0 && lane == 0) {
              if (last_slot >= 0) {
                bulk_wait_read();
                mbar_arrive(&bars.stored[last_slot]);
              }
              uint8_t* to = xt + static_cast<size_t>(c) * kOrthTile + quarter * 4096;
              bulk_store_nc(to, x + quarter * 4096, 4096);
              bulk_store_nc(to + kOrthPlane, x + kOrthPlane + quarter * 4096, 4096);
              bulk_commit();
              last_slot = slot;
            }
          }
          continue;
        }
        // the result: a transposed matrix's rows are contiguous across lanes, an
        // ordinary one's go through the slot (64 columns of BF16, swizzled)
        uint16_t* dst = static_cast<uint16_t*>(q.dst);
        const int col0 = (c0 + c) * 64;
        if (q.flags & kOrthTall) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int col = col0 + 32 * half + e;
            if (r < q.m && col < q.n)
              dst[col * q.ld_dst + r] =
                  static_cast<uint16_t>(pack_bf16x2(__uint_as_float(v[e]) * (kBack * kBack), 0.f) & 0xFFFFu);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_bf16x2(__uint_as_float(v[8 * k + 2 * e]) * (kBack * kBack),
                                 __uint_as_float(v[8 * k + 2 * e + 1]) * (kBack * kBack));
            *reinterpret_cast<uint4*>(x + sw128(r, 4 * half + k)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          if (!pair_sync()) break;
          const int row0 = quarter * 32 + half * 16, rows = min(16, q.m - row0), cols = min(64, q.n - col0);
          uint16_t* to = dst + row0 * q.ld_dst + col0;
          if (cols == 64 && (reinterpret_cast<uintptr_t>(to) & 15) == 0 && q.ld_dst % 8 == 0) {
            for (int e = lane; e < rows * 8; e += 32)
              *reinterpret_cast<uint4*>(to + (e >> 3) * q.ld_dst + (e & 7) * 8) =
                  *reinterpret_cast<const uint4*>(x + sw128(row0 + (e >> 3), e & 7));
          } else {
            for (int rr = 0; rr < rows; ++rr)
              for (int e = lane; e < cols; e += 32)
                to[rr * q.ld_dst + e] = reinterpret_cast<const uint16_t*>(x + sw128(row0 + rr, e >> 3))[e & 7];
          }
        }
        if (!resident) {
          fence_proxy_async_smem();  // read before the next load writes it
          if (!pair_sync()) break;
          if (half == 0 && lane == 0) mbar_arrive(&bars.stored[slot]);
        }
      }
      if (!go) break;
      if (!resident) {
        g += nloc;
        if (!last && half == 0 && lane == 0) {
          bulk_wait_all();
          fence_proxy_async_all();
          mbar_arrive(&bars.stored[last_slot]);
          mbar_arrive(&bars.saved);
          last_slot = -1;
        }
        __syncwarp();
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) settle_if_aborted(abort);
  __syncthreads();
  if (T > 1) cluster_sync();  // nobody writes into a CTA that has ended
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_orth_solo(const OrthMat* mats, int n, uint8_t* tiles, int steps, const OrthCoef& co, int team,
                             const WaitCtl& wc, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(orth_solo_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(n) * team);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = team;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, orth_solo_kernel, mats, tiles, steps, co, team, wc);
}

}  // namespace triattn
