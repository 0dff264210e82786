// The orthogonalisation's steps for matrices whose X has at most 128 rows (every
// projection of a pair stack of 128 features): one kernel for all steps, a CTA
// or a cluster ("team") of 2, 4 or 8 per matrix, X cut along its columns.
//
// A step is one pass over the CTA's columns, 64 at a time: D = B' X_c, the
// epilogue turns D into the new X_c in the place of the old one, and
// A += X_c X_c^T for the next step follows at once, so a chunk is touched once per
// step and not once per product.  Up to five chunks per CTA stay in shared memory
// for all steps; more go through L2 (the working set of all CTAs, 64 KB a chunk,
// fits it).  The left operands B' and the new X_c are in TMEM: from shared memory
// both operands of an MMA of 64 columns take 68 cycles to read, 34 to multiply.
//
// Between two passes the team adds its parts of A, every CTA one band of rows in
// the order of the ranks, and every CTA then makes all of B' = b A + c A^2 + a I.
// The parts go through L2 (distributed shared memory took 20 us a step for a team
// of eight), and every CTA loads the bands of the sum from there, once all have said that
// theirs are written (one copy of a band to all CTAs of the team: 64 us for the ten
// matrices of a block, so 65).
//
// 480 matrices of 48 blocks of 128 features: 221 us, tensor pipe active 44 %; the ten
// of one block, teams of eight: 58 us, 11 us a step, most of it the team's sum.
//
//   warp 0      loads of X's chunks (ring of five)
//   warp 1      MMAs: 24 of N = 64 for D and 12 of N = m for A per chunk, each three
//               products of FP16 pairs; 24 of N = m for A^2 per step.  D runs two
//               chunks ahead of A, so that the epilogue's time is hidden
//   warps 2-17  D to X, A and A^2 to B': thread = row, 16 or 32 columns
//
// A and B' are held without the scale (their norms are near 1 and what matters is
// the error beside that), so the products' results need no factor.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "kernels.cuh"
#include "orthogonalize.cuh"

namespace triattn {
namespace {

constexpr int kRing = 5;
constexpr int kB = 2 * kOrthTile;  // A as two tiles of 64 columns
constexpr int kSmem = kB + kRing * kOrthTile + 1024;
constexpr int kWarps = 16;  // epilogue
constexpr int kAhead = 2;    // chunks that D is ahead of A
constexpr int kThreads = (2 + kWarps) * 32;
// TMEM: A, A^2 or two D, B' (hi, lo), two X_c (hi, lo)
constexpr uint32_t kColA = 0, kColA2 = 128, kColD = 128, kColB = 256, kColX = 384;

struct SoloBars {
  uint64_t full[kRing];    // a chunk has been loaded
  uint64_t ready[kRing];   // the new chunk stands in the slot
  uint64_t used[kRing];    // the last product that reads the slot is done
  uint64_t stored[kRing];  // the slot has been copied out
  uint64_t dfull[2], dfree[2];
  uint64_t xfree[2];       // the product that reads X_c in TMEM is done
  uint64_t afull, aready, a2full, bready;
  uint64_t aimage;         // the team's A has been loaded
  uint64_t saved;          // a pass's chunks are in memory
  uint64_t team, bands;    // the team's CTAs: the parts of A, the bands of their sum are in memory
  uint64_t quad[4];        // the four warps of a quarter of the rows
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
  let_next_start();
  after_previous();
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
      mbar_init(&bars.xfree[i], 1);
      mbar_init(&bars.dfull[i], 1);
      mbar_init(&bars.dfree[i], kWarps);
    }
    mbar_init(&bars.afull, 1);
    mbar_init(&bars.aready, kWarps);
    mbar_init(&bars.a2full, 1);
    mbar_init(&bars.bready, kWarps);
    mbar_init(&bars.saved, 4);
    mbar_init(&bars.team, T * kWarps);
    mbar_init(&bars.bands, T * kWarps);
    for (int i = 0; i < 4; ++i) mbar_init(&bars.quad[i], 4);
    mbar_init(&bars.aimage, 1);
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
        if (wc.starve != 0 && blockIdx.x == 0 && g == 0) continue;
        mbar_expect_tx(&bars.full[slot], kOrthTile);
        bulk_load(ring + slot * kOrthTile, xt + static_cast<size_t>(c) * kOrthTile, kOrthTile, &bars.full[slot]);
      }
    }
  } else if (warp == 1) {
    const int k16 = (q.m + 15) / 16;  // K = m and N = m, to 16
    const uint32_t ia = idesc_f16_f32(128, 16 * k16, 0, 0), id = idesc_f16_f32(128, 64, 0, 1);
    // operands by the low words of their descriptors (address and leading offset in
    // 16 bytes; the high word is the same for all): one thread issues 36 MMAs a
    // chunk, and what it computes for each counts
    constexpr uint32_t kPlaneW = kOrthPlane / 16, kTileW = kOrthTile / 16;
    const uint32_t sB = (smem_u32(sm) >> 4) | (1u << 16), sR = (smem_u32(ring) >> 4) | (1u << 16),
                   sN = (smem_u32(ring) >> 4) | (512u << 16);  // MN-major: 8192 bytes between blocks of 64 columns
    uint32_t full = 0, ready = 0;
    int dn = 0, xn = 0;  // accumulators D and operands X_c used
    bool go = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      go = go && __all_sync(0xffffffffu, mbar_wait(bar, parity, wc, abort));
      tc_fence_after();
      return go;
    };
    auto products = [&](uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool first) {  // of 16 of K
      mma_ss_w(d, a, b, idesc, first ? 0u : 1u);
      mma_ss_w(d, a, b + kPlaneW, idesc, 1u);
      mma_ss_w(d, a + kPlaneW, b, idesc, 1u);
    };
    auto products_t = [&](uint32_t d, uint32_t a, uint32_t lo, uint32_t b, uint32_t idesc, bool first) {  // a in TMEM
      mma_ts_w(d, a, b, idesc, first ? 0u : 1u);
      mma_ts_w(d, a, b + kPlaneW, idesc, 1u);
      mma_ts_w(d, a + lo, b, idesc, 1u);
    };
    int g = 0;
    for (int c = 0; c < nloc && go; ++c, ++g) {
      const int slot = g % kRing;
      if (!wait(&bars.full[slot], (full >> slot) & 1)) break;
      full ^= 1u << slot;
      const uint32_t x = sR + slot * kTileW;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k) products(tmem + kColA, x + 2 * k, x + 2 * k, ia, c == 0 && k == 0);
        mma_commit(&bars.used[slot]);
        if (c == nloc - 1) mma_commit(&bars.afull);
      }
      __syncwarp();
    }
    if (nloc == 0 && elect_one()) mma_commit(&bars.afull);
    __syncwarp();
    for (int p = 1; p <= steps && go; ++p) {
      if (!wait(T > 1 ? &bars.aimage : &bars.aready, (p - 1) & 1)) break;
      if (elect_one()) {  // A^2: A is its own transposed
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < k16) {
            const uint32_t at = sB + (k >> 2) * kTileW + (k & 3) * 2;
            products(tmem + kColA2, at, at, ia, k == 0);
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
        const uint32_t x = sR + slot * kTileW, at = tmem + kColX + 64 * (xn & 1);
        if (elect_one()) {  // A += X_c X_c^T
#pragma unroll
          for (int k = 0; k < 4; ++k) products_t(tmem + kColA, at + 8 * k, 32, x + 2 * k, ia, c == 0 && k == 0);
          mma_commit(&bars.used[slot]);
          mma_commit(&bars.xfree[xn & 1]);
          if (c == nloc - 1) mma_commit(&bars.afull);
        }
        __syncwarp();
        ++xn;
      };
      for (int c = 0; c < nloc + (last ? 0 : kAhead) && go; ++c) {
        if (c < nloc) {
          const int slot = slot_of(c), db = dn & 1;
          if (!resident) {
            if (!wait(&bars.full[slot], (full >> slot) & 1)) break;
            full ^= 1u << slot;
          }
          if (!wait(&bars.dfree[db], ((dn >> 1) & 1) ^ 1)) break;
          const uint32_t x = sN + slot * kTileW, d = tmem + kColD + 64 * db;
          if (elect_one()) {  // D = B' X_c, X_c [rows of K, 64 columns] as it lies
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (k < k16) products_t(d, tmem + kColB + 8 * k, 64, x + k * 128, id, k == 0);
            mma_commit(&bars.dfull[db]);
            if (last) mma_commit(&bars.used[slot]);
          }
          __syncwarp();
          ++dn;
          ++g;
        }
        if (!last && c >= kAhead) add_ready(c - kAhead);
      }
      if (!last && go && nloc == 0 && elect_one()) mma_commit(&bars.afull);
      __syncwarp();
    }
  } else {
    const int quarter = warp & 3, part = (warp - 2) >> 2, r = quarter * 32 + lane;
    const int te = threadIdx.x - 64;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    constexpr float kBack = 1.f / kOrthScale, kBackA = kBack * kBack;  // A carries the scale twice
    uint32_t tphase = 0, pphase = 0;
    int dn = 0, xn = 0, g = resident ? 0 : nloc, last_slot = -1;
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
    auto team_arrive = [&](uint64_t* bar) {  // in every CTA of the team
      __syncwarp();
      if (lane < T) mbar_arrive_cluster(bar, lane);
    };
    auto team_sync = [&]() {
      team_arrive(&bars.team);
      go = go && __all_sync(0xffffffffu, mbar_wait<true>(&bars.team, tphase, wc, abort));
      tphase ^= 1;
      return go;
    };
    auto quad_sync = [&]() {
      arrive(&bars.quad[quarter]);
      go = go && __all_sync(0xffffffffu, mbar_wait(&bars.quad[quarter], pphase, wc, abort));
      pphase ^= 1;
      return go;
    };
    // this thread's 32 columns of A and B': half a tile
    uint8_t* const mine = sm + (part >> 1) * kOrthTile;
    const int ch0 = 4 * (part & 1);
    // the team's exchange: [T] parts [32][128] of four columns, then A's image
    uint8_t* const ex = tiles + static_cast<size_t>(q.a) * kOrthTile;
    uint8_t* const image = ex + static_cast<size_t>(T) * kB;
    for (int p = 1; p <= steps; ++p) {
      const bool last = p == steps;
      // ---- A to shared memory: the CTA's own, or the team's sum
      if (!wait(&bars.afull, (p - 1) & 1)) break;
      uint32_t v[32];
      if (nloc > 0) {
        tmem_ld32_wait(lane_addr + kColA + 32 * part, v);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = 0u;
      }
      if (T == 1) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(v[8 * c + e]) * kBackA;
          uint4 hi, lo;
          split8(y, hi, lo);
          *reinterpret_cast<uint4*>(mine + sw128(r, ch0 + c)) = hi;
          *reinterpret_cast<uint4*>(mine + kOrthPlane + sw128(r, ch0 + c)) = lo;
        }
        fence_proxy_async_smem();
        tc_fence_before();
        arrive(&bars.aready);
      } else {
        uint4* out = reinterpret_cast<uint4*>(ex + static_cast<size_t>(rank) * kB);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          __stcg(out + (part * 8 + k) * 128 + r, make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]));
        tc_fence_before();
        if (!team_sync()) break;  // the parts are there
        const int RL = 128 / T;   // rows of the band
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int u = te + 32 * kWarps * k, row = rank * RL + u % RL, ch = u / RL;  // eight columns of a row
          if (u >= RL * 16) break;
          const float4* f = reinterpret_cast<const float4*>(ex) + 2 * ch * 128 + row;
          float y[8];
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // four columns, the parts' loads together
            float4 part_of[8], sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int t = 0; t < 8; ++t)
              if (t < T) part_of[t] = __ldcg(f + t * (kB / 16) + h * 128);
#pragma unroll
            for (int t = 0; t < 8; ++t)
              if (t < T) {
                sum.x += part_of[t].x;
                sum.y += part_of[t].y;
                sum.z += part_of[t].z;
                sum.w += part_of[t].w;
              }
            y[4 * h] = sum.x * kBackA;
            y[4 * h + 1] = sum.y * kBackA;
            y[4 * h + 2] = sum.z * kBackA;
            y[4 * h + 3] = sum.w * kBackA;
          }
          uint4 hi, lo;
          split8(y, hi, lo);
          uint8_t* at = image + (ch >> 3) * kOrthTile + sw128(row, ch & 7);
          *reinterpret_cast<uint4*>(at) = hi;
          *reinterpret_cast<uint4*>(at + kOrthPlane) = lo;
        }
        fence_proxy_async_all();  // the bands are read by bulk copies
        team_arrive(&bars.bands);
        if (te == 0 && mbar_wait<true>(&bars.bands, (p - 1) & 1, wc, abort)) {
          fence_proxy_async_all();
          mbar_expect_tx(&bars.aimage, kB);
#pragma unroll
          for (int k = 0; k < 4; ++k)  // hi and lo of both tiles
            bulk_load(sm + k * kOrthPlane, image + k * kOrthPlane, kOrthPlane, &bars.aimage);
        }
        __syncwarp();
        if (!wait(&bars.aimage, (p - 1) & 1)) break;
      }
      // ---- B' = b A + c A^2 + a I
      if (!wait(&bars.a2full, (p - 1) & 1)) break;
#pragma unroll
      for (int c2 = 0; c2 < 2; ++c2) {  // 16 columns
        // A: this CTA's own is still in TMEM, the team's sum only in its image
        uint32_t a2[16], a1[16], hi[8], lo[8];
        tmem_ld16x2_wait(lane_addr + kColA2 + 32 * part + 16 * c2, a2, lane_addr + kColA + 32 * part + 16 * c2, a1);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float y[8];
          if (T == 1) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(a1[8 * c + e]) * kBackA;
          } else {
            const uint8_t* at = mine + sw128(r, ch0 + 2 * c2 + c);
            join8(*reinterpret_cast<const uint4*>(at), *reinterpret_cast<const uint4*>(at + kOrthPlane), y);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y[e] = co.b * y[e] + co.c * __uint_as_float(a2[8 * c + e]);
            if (32 * part + 16 * c2 + 8 * c + e == r) y[e] += co.a;
          }
          uint4 h, l;
          split8(y, h, l);
          hi[4 * c] = h.x;
          hi[4 * c + 1] = h.y;
          hi[4 * c + 2] = h.z;
          hi[4 * c + 3] = h.w;
          lo[4 * c] = l.x;
          lo[4 * c + 1] = l.y;
          lo[4 * c + 2] = l.z;
          lo[4 * c + 3] = l.w;
        }
        tmem_st8(lane_addr + kColB + 16 * part + 8 * c2, hi);
        tmem_st8(lane_addr + kColB + 64 + 16 * part + 8 * c2, lo);
      }
      tc_wait_st();
      tc_fence_before();
      arrive(&bars.bready);
      // ---- the chunks
      for (int c = 0; c < nloc; ++c, ++dn) {
        const int db = dn & 1, slot = resident ? c : (g + c) % kRing;
        if (!wait(&bars.dfull[db], (dn >> 1) & 1)) break;
        uint32_t d[16];
        tmem_ld16_wait(lane_addr + kColD + 64 * db + 16 * part, d);
        tc_fence_before();
        arrive(&bars.dfree[db]);
        uint8_t* x = ring + slot * kOrthTile;
        if (!last) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(d[8 * k + e]);
            uint4 h, l;
            split8(y, h, l);
            *reinterpret_cast<uint4*>(x + sw128(r, 2 * part + k)) = h;
            *reinterpret_cast<uint4*>(x + kOrthPlane + sw128(r, 2 * part + k)) = l;
            hi[4 * k] = h.x;
            hi[4 * k + 1] = h.y;
            hi[4 * k + 2] = h.z;
            hi[4 * k + 3] = h.w;
            lo[4 * k] = l.x;
            lo[4 * k + 1] = l.y;
            lo[4 * k + 2] = l.z;
            lo[4 * k + 3] = l.w;
          }
          if (!wait(&bars.xfree[xn & 1], ((xn >> 1) & 1) ^ 1)) break;
          const uint32_t at = lane_addr + kColX + 64 * (xn & 1) + 8 * part;
          tmem_st8(at, hi);
          tmem_st8(at + 32, lo);
          ++xn;
          tc_wait_st();
          fence_proxy_async_smem();
          tc_fence_before();
          arrive(&bars.ready[slot]);
          if (!resident) {
            if (!quad_sync()) break;  // all columns of the quarter's rows
            if (part == 0 && lane == 0) {
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
          for (int e = 0; e < 16; ++e) {
            const int col = col0 + 16 * part + e;
            if (r < q.m && col < q.n)
              dst[col * q.ld_dst + r] =
                  static_cast<uint16_t>(pack_bf16x2(__uint_as_float(d[e]) * kBack, 0.f) & 0xFFFFu);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_bf16x2(__uint_as_float(d[8 * k + 2 * e]) * kBack,
                                 __uint_as_float(d[8 * k + 2 * e + 1]) * kBack);
            *reinterpret_cast<uint4*>(x + sw128(r, 2 * part + k)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          if (!quad_sync()) break;
          const int row0 = quarter * 32 + part * 8, rows = min(8, q.m - row0), cols = min(64, q.n - col0);
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
          if (!quad_sync()) break;
          if (part == 0 && lane == 0) mbar_arrive(&bars.stored[slot]);
        }
      }
      if (!go) break;
      if (!resident) {
        g += nloc;
        if (!last && part == 0 && lane == 0) {
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
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = team;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, orth_solo_kernel, mats, tiles, steps, co, team, wc);
}

}  // namespace triattn
