// The transition's backward up to the weight gradients, in one kernel: per
// row tile it computes x, a and b again, dh = g W_o^T, the activation's
// backward, dx = [da | db] W_in^T and the LayerNorm's backward, and leaves
// x and g in memory for the weight gradients (transition_wgrad.cu).
//
// A pair of CTAs (tcgen05 cta_group::2) takes tiles of 256 rows, 128 per CTA;
// each CTA holds one half of the N columns of every B operand.  The weights
// come through two rings per 64-wide hidden chunk, W_in and W_o as the
// operands of [a | b] (CTA 0: W_a, CTA 1: W_b) and dh, and W_in again, split
// along C instead of the hidden axis, as that of dx: 40 KB per chunk and CTA
// at C = 128 from L2, 15 bytes per clock at the pace below, and what is left of
// shared memory holds the row tiles.
//
// Per tile and chunk:
//   [a | b] = x [W_a | W_b]    M = 256, N = 128, K = C, A = x in TMEM
//   dh      = g W_o^T          M = 256, N = 64,  K = C, A = g in TMEM
//   da = dh b act'(a), db = dh act(a)                 (registers)
//   dx     += [da | db] W_in^T M = 256, N = C, K = 128, A in TMEM
// x, g (C / 2 columns each), dx (C), [a | b | dh] (192) and [da | db] (64) fill
// the 512 TMEM columns at C = 128.
//
// What bounds it is the chain of a chunk: the next [a | b] and dh are computed
// while the activation runs, but into the columns that it reads (TMEM has no
// second set), so products and activation overlap by half: 0.40 ms at 768 x 768
// rows, C = 128, H = 512, against 0.198 ms of products, the tensor pipe active for
// 40 %; the special-function unit is busy for 17 %, but the gate's exponential and
// reciprocal lengthen the chain (0.355 ms with the hardware tanh, which the next
// figures had too).  Loading a chunk's 96
// columns at once, to free them sooner, spills (0.41 ms).  Storing h, da and db
// here for library-shaped weight-gradient products cost 0.125 ms of writes (1.8 GB),
// and their products, bound by reading them, took 0.342 ms: computing them again
// (transition_wgrad.cu) took 0.404 ms, 0.06 ms less in all and no workspace of
// 6 H bytes per row.  Row tiles leave by TMA: x stored from registers, 32 bytes per
// row and instruction, took 0.08 ms more.
//
// Roundings: x, g = m d_out, da and db are BF16 because they are operands of the
// tensor cores; a, b, dh, dx and every sum stay FP32 up to dz's one rounding.
// Relative error of dz and of the parameters' gradients 3.0e-3 to 3.8e-3 with one
// rounding of their own.
//
// Warps: 0 loads weights, 2 tells CTA 0 that this CTA's are in; 1 and 3 (of
// CTA 0) issue the MMAs, one [a | b] and dh, one dx; 4-7 write x = LayerNorm(z)
// and g (thread = row), 8-11 take dx through the LayerNorm's backward; 12-19 the
// activation.
#include <algorithm>
#include <cstring>

#include "kernels.cuh"
#include "transition.cuh"

namespace triattn {
namespace {

constexpr int kTbThreads = 20 * 32;
// Registers per thread of the warpgroups (setmaxnreg): five shares of what the
// block was launched with (96 each).
constexpr int kRegsIssue = 40, kRegsRow = 88, kRegsLn = 144, kRegsAct = 104;
constexpr int kRegsSum = kRegsIssue + kRegsRow + kRegsLn + 2 * kRegsAct;
constexpr int kTbMaxSlots = 4;
constexpr int kTbBarBytes = 1024 + 1024;  // barriers, ln_w and ln_b
constexpr int kTbSmemMax = 232448;

struct TbBars {
  uint64_t a_load[kTbMaxSlots], a_ready[kTbMaxSlots], a_empty[kTbMaxSlots];  // ring of W_in, W_o: in this CTA (TMA
                                                                           // bytes) / in both (CTA 0) / read (both)
  uint64_t b_load[kTbMaxSlots], b_ready[kTbMaxSlots], b_empty[kTbMaxSlots];  // the same for dx's W_in
  uint64_t z_full[2], g_full;   // z and d_out tiles in shared memory (TMA bytes)
  uint64_t xg_full, xg_free;    // x and g written (CTA 0) / read (both)
  uint64_t abd_full, abd_free;  // [a | b | dh] complete (both) / read (CTA 0)
  uint64_t dab_full, dab_free;  // [da | db] written (CTA 0) / read (both)
  uint64_t dx_full, dx_free;    // dx complete (both) / read (CTA 0)
  uint32_t tmem_slot;
  int abort;
};
static_assert(sizeof(TbBars) <= 1024, "barrier block");

struct TbParams {
  long long M;
  int H, chunks, slots, tiles;
  const uint16_t* mask;
  const float *ln_w, *ln_b;
  uint16_t* g;
  float *part_g, *part_b;
  WaitCtl wc;
};

template <int C>
struct TbSmem {
  static constexpr int kKb = (C + 63) / 64;   // 64-wide blocks of a row
  static constexpr int kWin = C * 128;        // ring A: C rows (K) of 64 columns
  static constexpr int kWo = kKb * 32 * 128;  // ring A: 32 hidden rows (N) of C columns (K)
  static constexpr int kA = kWin + kWo;
  static constexpr int kWx = (C / 2) * 128;   // ring B: C / 2 rows (N) of 64 hidden columns (K), for a and for b
  static constexpr int kB = 2 * kWx;
  static constexpr int kRows = kKb * 16384;   // a tile of 128 rows
  static constexpr int bytes(int slots) { return slots * (kA + kB) + 3 * kRows + kTbBarBytes + 1024; }
};

// v[j] summed over the 8 threads t mod 4 + 4 q for every j, the thread of
// index q ending with the sum of v[q] (halving exchange, fixed order).
__device__ __forceinline__ float rows_scatter_sum(float (&v)[8], int lane) {
#pragma unroll
  for (int n = 4; n > 0; n >>= 1) {
    const bool up = (lane & (4 * n)) != 0;
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const float keep = up ? v[j + n] : v[j], send = up ? v[j] : v[j + n];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, send, 4 * n);
    }
  }
  return v[0];
}

template <int C, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTbThreads, 1)
    transition_bwd_kernel(const __grid_constant__ CUtensorMap tm_z, const __grid_constant__ CUtensorMap tm_do,
                          const __grid_constant__ CUtensorMap tm_dz, const __grid_constant__ CUtensorMap tm_x,
                          const __grid_constant__ CUtensorMap tm_win, const __grid_constant__ CUtensorMap tm_wo,
                          const __grid_constant__ CUtensorMap tm_wx, const TbParams p) {
  using L = TbSmem<C>;
  constexpr uint32_t kX = 0, kG = C / 2, kDx = C, kABD = 256, kDAB = 448;  // TMEM columns
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* const s_a = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const s_b = s_a + p.slots * L::kA;
  uint8_t* const s_z = s_b + p.slots * L::kB;  // two z tiles
  uint8_t* const s_g = s_z + 2 * L::kRows;
  TbBars* const bars = reinterpret_cast<TbBars*>(s_g + L::kRows);
  float* const s_gam = reinterpret_cast<float*>(s_g + L::kRows + 1024);
  float* const s_bet = s_gam + C;
  volatile int* abort = &bars->abort;
  const WaitCtl& wc = p.wc;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int mine = p.tiles > pair ? (p.tiles - 1 - pair) / pairs + 1 : 0;  // tiles of this pair
  const long long total = static_cast<long long>(mine) * p.chunks;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.slots; ++i) {
      mbar_init(&bars->a_load[i], 1);
      mbar_init(&bars->a_ready[i], 2);
      mbar_init(&bars->a_empty[i], 1);
      mbar_init(&bars->b_load[i], 1);
      mbar_init(&bars->b_ready[i], 2);
      mbar_init(&bars->b_empty[i], 1);
    }
    mbar_init(&bars->z_full[0], 1);
    mbar_init(&bars->z_full[1], 1);
    mbar_init(&bars->g_full, 1);
    mbar_init(&bars->xg_full, 8);
    mbar_init(&bars->xg_free, 1);
    mbar_init(&bars->abd_full, 1);
    mbar_init(&bars->abd_free, 16);
    mbar_init(&bars->dab_full, 16);
    mbar_init(&bars->dab_free, 1);
    mbar_init(&bars->dx_full, 1);
    mbar_init(&bars->dx_free, 8);
    bars->abort = 0;
    fence_mbar_init();
  }
  for (int c = threadIdx.x; c < C; c += kTbThreads) {
    s_gam[c] = p.ln_w[c];
    s_bet[c] = p.ln_b[c];
  }
  if (warp == 1) tmem_alloc_pair(&bars->tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before the first remote arrival
  tc_fence_after();
  const uint32_t tmem = bars->tmem_slot;
  // this thread's row of local tile u, and its tile's first row (thread-per-row warps)
  const int quarter = warp & 3, r = quarter * 32 + lane;
  const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
  auto tile_row = [&](int u) {
    return (static_cast<long long>(pair) + static_cast<long long>(u) * pairs) * 256 + rank * 128;
  };
  // a row tile into shared memory
  auto load_rows = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int u) {
    mbar_expect_tx(bar, L::kRows);
#pragma unroll
    for (int b = 0; b < L::kKb; ++b) tma_load_3d(dst + b * 16384, map, bar, 64 * b, static_cast<int>(tile_row(u)), 0);
  };

  if (warp < 4) regs_dec<kRegsIssue>();
  if (warp == 0) {
    // ------------------------------------------------------------ weights
    if (lane == 0) {
      int slot = 0, phase = 0, i = 0;
      for (long long g = 0; g < total; ++g) {
        if (!mbar_wait(&bars->a_empty[slot], phase ^ 1, wc, abort)) break;
        uint8_t* const a = s_a + slot * L::kA;
        mbar_expect_tx(&bars->a_load[slot], L::kA);
        tma_load_3d(a, &tm_win, &bars->a_load[slot], 64 * i, static_cast<int>(rank), 0);
#pragma unroll
        for (int b = 0; b < L::kKb; ++b)
          tma_load_3d(a + L::kWin + b * 4096, &tm_wo, &bars->a_load[slot], 64 * b,
                      64 * i + 32 * static_cast<int>(rank), 0);
        if (!mbar_wait(&bars->b_empty[slot], phase ^ 1, wc, abort)) break;
        uint8_t* const b = s_b + slot * L::kB;
        mbar_expect_tx(&bars->b_load[slot], L::kB);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          tma_load_3d(b + k * L::kWx, &tm_wx, &bars->b_load[slot], 64 * i, k, static_cast<int>(rank) * (C / 2));
        if (++i == p.chunks) i = 0;
        if (++slot == p.slots) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ weights' arrival, to CTA 0
    if (lane == 0) {
      int slot = 0, phase = 0;
      for (long long g = 0; g < total; ++g) {
        if (!mbar_wait(&bars->a_load[slot], phase, wc, abort)) break;
        mbar_arrive_cta(&bars->a_ready[slot], 0);
        if (!mbar_wait(&bars->b_load[slot], phase, wc, abort)) break;
        mbar_arrive_cta(&bars->b_ready[slot], 0);
        if (++slot == p.slots) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer: [a | b], dh
    if (rank == 0) {
      constexpr uint32_t id_ab = idesc_bf16_f32(256, 128, 0, 1);  // B: N contiguous
      constexpr uint32_t id_dh = idesc_bf16_f32(256, 64, 0, 0);   // B: K contiguous
      // operand descriptors; an offset of n bytes adds n / 16
      const uint64_t d_win = smem_desc(smem_u32(s_a), 64 * 128, 1024, 2);
      const uint64_t d_wo = smem_desc(smem_u32(s_a + L::kWin), 16, 1024, 2);
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity, wc, abort));
      };
      int t = 0, i = 0, slot = 0, phase = 0;
      for (long long g = 0; g < total; ++g) {
        wait(&bars->a_ready[slot], phase);
        if (i == 0) wait(&bars->xg_full, t & 1);
        if (g > 0) wait(&bars->abd_free, static_cast<uint32_t>(g - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t wa = d_win + slot * (L::kA / 16), wo = d_wo + slot * (L::kA / 16);
#pragma unroll
          for (int k = 0; k < C / 16; ++k)
            mma_ts_pair(tmem + kABD, tmem + kX + 8 * k, wa + k * (2048 / 16), id_ab, k > 0 ? 1u : 0u);
#pragma unroll
          for (int k = 0; k < C / 16; ++k)
            mma_ts_pair(tmem + kABD + 128, tmem + kG + 8 * k, wo + ((k >> 2) * 4096 + (k & 3) * 32) / 16, id_dh,
                        k > 0 ? 1u : 0u);
          mma_commit_pair(&bars->abd_full);
          mma_commit_pair(&bars->a_empty[slot]);
          if (i == p.chunks - 1) mma_commit_pair(&bars->xg_free);
        }
        __syncwarp();
        if (++slot == p.slots) {
          slot = 0;
          phase ^= 1;
        }
        if (++i == p.chunks) {
          i = 0;
          ++t;
        }
      }
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ MMA issuer: dx
    if (rank == 0) {
      constexpr uint32_t id_dx = idesc_bf16_f32(256, C, 0, 0);
      const uint64_t d_wx = smem_desc(smem_u32(s_b), 16, 1024, 2);
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity, wc, abort));
      };
      int t = 0, i = 0, slot = 0, phase = 0;
      for (long long g = 0; g < total; ++g) {
        wait(&bars->b_ready[slot], phase);
        if (i == 0 && t > 0) wait(&bars->dx_free, (t - 1) & 1);
        wait(&bars->dab_full, static_cast<uint32_t>(g) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t wx = d_wx + slot * (L::kB / 16);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ts_pair(tmem + kDx, tmem + kDAB + 8 * k, wx + ((k >> 2) * L::kWx + (k & 3) * 32) / 16, id_dx,
                        (i > 0 || k > 0) ? 1u : 0u);
          mma_commit_pair(&bars->dab_free);
          mma_commit_pair(&bars->b_empty[slot]);
          if (i == p.chunks - 1) mma_commit_pair(&bars->dx_full);
        }
        __syncwarp();
        if (++slot == p.slots) {
          slot = 0;
          phase ^= 1;
        }
        if (++i == p.chunks) {
          i = 0;
          ++t;
        }
      }
    }
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------ x = LayerNorm(z), g = m d_out
    regs_dec<kRegsRow>();
    const bool first = warp == 4 && lane == 0;
    auto write = [&](int u) -> bool {
      const long long row = tile_row(u) + r;
      const bool in = row < p.M;
      const float mk = !in ? 0.f : (p.mask != nullptr ? bf16lo_to_f32(p.mask[row]) : 1.f);
      const bool live = mk != 0.f;  // a row left out, or past the end: x = g = 0
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->z_full[u & 1], (u >> 1) & 1, wc, abort))) return false;
      const uint8_t* const zt = s_z + (u & 1) * L::kRows;
      auto z16 = [&](int c) { return reinterpret_cast<const uint4*>(zt + (c >> 3) * 16384 + sw128(r, c & 7)); };
      const float2 st = row_stats<C>(z16);
      const float2 nm = make_float2(-st.x, -st.x), rs = make_float2(st.y, st.y);
      // x in registers before the previous tile's has been read
      uint32_t x[C / 2];
#pragma unroll
      for (int c = 0; c < C / 8; ++c) {
        const uint4 w = *z16(c);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
        const float4* gm = reinterpret_cast<const float4*>(s_gam + 8 * c);
        const float4* bt = reinterpret_cast<const float4*>(s_bet + 8 * c);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 ga = gm[e], be = bt[e];
          const float2 x0 = ffma2(fmul2(fadd2(bf16x2_to_f32x2(ws[2 * e]), nm), rs), make_float2(ga.x, ga.y),
                                  make_float2(be.x, be.y));
          const float2 x1 = ffma2(fmul2(fadd2(bf16x2_to_f32x2(ws[2 * e + 1]), nm), rs), make_float2(ga.z, ga.w),
                                  make_float2(be.z, be.w));
          x[4 * c + 2 * e] = live ? pack_bf16x2(x0.x, x0.y) : 0u;
          x[4 * c + 2 * e + 1] = live ? pack_bf16x2(x1.x, x1.y) : 0u;
        }
        if (c % 2 == 1) asm volatile("" ::: "memory");  // no more rows unpacked at a time than fit
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->g_full, u & 1, wc, abort))) return false;
      if (u > 0 && !__all_sync(0xffffffffu, mbar_wait(&bars->xg_free, (u - 1) & 1, wc, abort))) return false;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < C / 16; ++c) {
        uint32_t v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = x[8 * c + e];
        tmem_st8(tmem + lane_addr + kX + 8 * c, v);
      }
#pragma unroll 1
      for (int c = 0; c < C / 8; c += 4) {  // g: 32 features = 16 columns at a time
        uint32_t v[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 w = *reinterpret_cast<const uint4*>(s_g + ((c + j) >> 3) * 16384 + sw128(r, (c + j) & 7));
          v[4 * j] = w.x;
          v[4 * j + 1] = w.y;
          v[4 * j + 2] = w.z;
          v[4 * j + 3] = w.w;
        }
        if (p.mask != nullptr) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            v[e] = live ? pack_bf16x2(bf16lo_to_f32(v[e]) * mk, bf16hi_to_f32(v[e]) * mk) : 0u;
        }
        tmem_st16(tmem + lane_addr + kG + 4 * c, v);
        if (p.mask != nullptr && in) {
          uint32_t lo[8], hi[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            lo[e] = v[e];
            hi[e] = v[8 + e];
          }
          st_global_v8(p.g + row * C + 8 * c, lo);
          st_global_v8(p.g + row * C + 8 * c + 16, hi);
        }
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&bars->xg_full, 0);
      // x for the weight gradients takes d_out's place in shared memory (the row
      // is this thread's) and goes out by TMA: stored from here, 32 bytes per
      // row and instruction, it cost 80 us at 768 x 768 rows
#pragma unroll
      for (int c = 0; c < C / 8; ++c)
        *reinterpret_cast<uint4*>(s_g + (c >> 3) * 16384 + sw128(r, c & 7)) =
            make_uint4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
      return true;
    };
    if (first && mine > 0) {
      load_rows(s_z, &tm_z, &bars->z_full[0], 0);
      load_rows(s_g, &tm_do, &bars->g_full, 0);
      if (mine > 1) load_rows(s_z + L::kRows, &tm_z, &bars->z_full[1], 1);
    }
    bool ok = true;
    for (int u = 0; u < mine; ++u) {  // no warp leaves the loop early: they meet at its barrier
      ok = ok && write(u);
      fence_proxy_async_smem();
      __syncwarp();
      named_bar_sync(1, 128);  // every row of the d_out tile is read, and x in its place
      if (first && ok) {
        if (tile_row(u) < p.M) {
#pragma unroll
          for (int b = 0; b < L::kKb; ++b)
            tma_store_3d(&tm_x, s_g + b * 16384, 64 * b, static_cast<int>(tile_row(u)), 0);
        }
        if (u + 1 < mine) {
          bulk_wait_read();
          load_rows(s_g, &tm_do, &bars->g_full, u + 1);
        }
      }
    }
    if (first) bulk_wait_all();
    __syncwarp();
  } else if (warp >= 8 && warp < 12) {
    // ------------------------------------------------------------ LayerNorm backward
    // dz = rstd (t - mean(t) - xhat mean(t xhat)), t = dx ln_w, over the rows of
    // dx, taken out of TMEM as matrix fragments of 16 rows: a thread holds 2 of
    // every 8 features of 2 of them, so a row's sums take two exchanges and a
    // feature's sum over the rows (for d_ln_w and d_ln_b) three; with a whole
    // row per thread that sum alone took 1500 instructions per tile.  Two
    // fragments at once would free TMEM earlier, but not fit the registers.
    regs_inc<kRegsLn>();
    const bool first = warp == 8 && lane == 0;
    const int q = lane >> 2, cl = 2 * (lane & 3);
    float accg[C / 32], accb[C / 32];
#pragma unroll
    for (int b = 0; b < C / 32; ++b) accg[b] = accb[b] = 0.f;
    auto ln_bwd = [&](int u) -> bool {
      uint8_t* const zt = s_z + (u & 1) * L::kRows;
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->z_full[u & 1], (u >> 1) & 1, wc, abort))) return false;
      // the statistics of row r, and whether it takes part, by its own thread
      const float2 st = row_stats<C>(
          [&](int c) { return reinterpret_cast<const uint4*>(zt + (c >> 3) * 16384 + sw128(r, c & 7)); });
      const long long row = tile_row(u) + r;
      const uint32_t lives =
          __ballot_sync(0xffffffffu, row < p.M && (p.mask == nullptr || (p.mask[row] & 0x7FFFu) != 0));
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->dx_full, u & 1, wc, abort))) return false;
      tc_fence_after();
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {  // rows 16 h + q and 16 h + q + 8 of the warp's 32
        uint32_t d[C / 2];
        const uint32_t at = tmem + lane_addr + (static_cast<uint32_t>(16 * h) << 16) + kDx;
#pragma unroll
        for (int c = 0; c + 64 <= C; c += 64) tmem_ld_frag_wait<32>(at + c, &d[c / 2]);
        if constexpr (C % 64 != 0) tmem_ld_frag_wait<16>(at + C - 32, &d[(C - 32) / 2]);
        if (h == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(&bars->dx_free, 0);
        }
        float2 nm[2], rs[2];
        bool live[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int src = 16 * h + 8 * k + q;
          const float mean = __shfl_sync(0xffffffffu, st.x, src), rstd = __shfl_sync(0xffffffffu, st.y, src);
          nm[k] = make_float2(-mean, -mean);
          rs[k] = make_float2(rstd, rstd);
          live[k] = ((lives >> src) & 1u) != 0;
        }
        // z of row k's features 8 j + cl, + 1: one word of shared memory
        uint8_t* const zr = zt + (quarter * 32 + 16 * h + q) * 128 + 2 * cl;
        auto zw = [&](int k, int j) {
          return reinterpret_cast<uint32_t*>(zr + (j >> 3) * 16384 + k * 1024 + (((j & 7) ^ (q & 7)) << 4));
        };
        auto xhat = [&](int k, int j) {
          const float2 v = fmul2(fadd2(bf16x2_to_f32x2(*zw(k, j)), nm[k]), rs[k]);
          // a row left out has dx = 0; xhat = 0 whatever z holds there
          return live[k] ? v : make_float2(0.f, 0.f);
        };
        auto dx = [&](int k, int j) {  // as zw
          return make_float2(__uint_as_float(d[4 * j + 2 * k]), __uint_as_float(d[4 * j + 2 * k + 1]));
        };
        float2 s1[2], s2[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) s1[k] = s2[k] = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < C / 8; ++j) {
          const float2 gm = *reinterpret_cast<const float2*>(s_gam + 8 * j + cl);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 t = fmul2(dx(k, j), gm);
            s1[k] = fadd2(s1[k], t);
            s2[k] = ffma2(t, xhat(k, j), s2[k]);
          }
          // z and ln_w are read again below: kept from here they would not fit
          if (j % 4 == 3) asm volatile("" ::: "memory");
        }
        float2 m1[2], m2[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float a = s1[k].x + s1[k].y, b = s2[k].x + s2[k].y;
#pragma unroll
          for (int off = 1; off < 4; off <<= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, off);
            b += __shfl_xor_sync(0xffffffffu, b, off);
          }
          a *= -rs[k].x * (1.f / C);
          b *= -rs[k].x * (1.f / C);
          m1[k] = make_float2(a, a);
          m2[k] = make_float2(b, b);
        }
#pragma unroll
        for (int b = 0; b < C / 32; ++b) {
          float vg[8], vb[8];
#pragma unroll
          for (int jj = 0; jj < 4; ++jj) {
            const int j = 4 * b + jj;
            const float2 gm = *reinterpret_cast<const float2*>(s_gam + 8 * j + cl);
            float2 cg = make_float2(0.f, 0.f), cb = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float2 xh = xhat(k, j), dv = dx(k, j);
              const float2 o = ffma2(xh, m2[k], ffma2(fmul2(dv, gm), rs[k], m1[k]));
              *zw(k, j) = live[k] ? pack_bf16x2(o.x, o.y) : 0u;  // dz in z's place: the word is this thread's
              cg = ffma2(dv, xh, cg);
              cb = fadd2(cb, dv);
            }
            vg[2 * jj] = cg.x;
            vg[2 * jj + 1] = cg.y;
            vb[2 * jj] = cb.x;
            vb[2 * jj + 1] = cb.y;
          }
          accg[b] += rows_scatter_sum(vg, lane);
          accb[b] += rows_scatter_sum(vb, lane);
        }
      }
      return true;
    };
    bool ok = true;
    for (int u = 0; u < mine; ++u) {  // no warp leaves the loop early: they meet at its barrier
      ok = ok && ln_bwd(u);
      fence_proxy_async_smem();
      __syncwarp();
      named_bar_sync(2, 128);
      if (first && ok) {
        uint8_t* const zt = s_z + (u & 1) * L::kRows;
        if (tile_row(u) < p.M) {
#pragma unroll
          for (int b = 0; b < L::kKb; ++b)
            tma_store_3d(&tm_dz, zt + b * 16384, 64 * b, static_cast<int>(tile_row(u)), 0);
        }
        if (u + 2 < mine) {
          bulk_wait_read();
          load_rows(zt, &tm_z, &bars->z_full[u & 1], u + 2);
        }
      }
    }
    if (first) bulk_wait_all();
    __syncwarp();
    const size_t part = static_cast<size_t>(blockIdx.x) * 4 + quarter;
#pragma unroll
    for (int b = 0; b < C / 32; ++b) {
      const int c = 32 * b + 8 * (q >> 1) + cl + (q & 1);
      p.part_g[part * C + c] = accg[b];
      p.part_b[part * C + c] = accb[b];
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------------ activation
    // Warp = 32 rows x 32 of the chunk's 64 hidden features, 16 at a time
    regs_inc<kRegsAct>();
    const int hf = (warp - 12) >> 2;
    const uint32_t abd = tmem + lane_addr + kABD + 32 * hf, dab = tmem + lane_addr + kDAB + 16 * hf;
    for (long long g = 0; g < total; ++g) {
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->abd_full, static_cast<uint32_t>(g) & 1, wc, abort))) break;
      tc_fence_after();
      bool ok = true;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t a[16], b[16], d[16];
        tmem_ld16x3_wait(abd + 16 * j, a, abd + 64 + 16 * j, b, abd + 128 + 16 * j, d);
        if (j == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(&bars->abd_free, 0);
        }
        uint32_t da[8], db[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float2 hv, av, bv;
          gate_bwd2<ACT>(make_float2(__uint_as_float(a[2 * e]), __uint_as_float(a[2 * e + 1])),
                         make_float2(__uint_as_float(b[2 * e]), __uint_as_float(b[2 * e + 1])),
                         make_float2(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1])), hv, av, bv);
          da[e] = pack_bf16x2(av.x, av.y);
          db[e] = pack_bf16x2(bv.x, bv.y);
        }
        if (j == 0 && g > 0) {  // the previous chunk's dx has read [da | db]
          ok = __all_sync(0xffffffffu, mbar_wait(&bars->dab_free, static_cast<uint32_t>(g - 1) & 1, wc, abort));
          tc_fence_after();
        }
        tmem_st8(dab + 8 * j, da);
        tmem_st8(dab + 32 + 8 * j, db);
      }
      tc_wait_st();
      if (!ok) break;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&bars->dab_full, 0);
    }
  }

  settle_if_aborted(abort);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no arrival is under way to a CTA that has left
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <int C>
int tb_slots() {
  for (int s = kTbMaxSlots; s > 2; --s)
    if (TbSmem<C>::bytes(s) <= kTbSmemMax) return s;
  static_assert(TbSmem<C>::bytes(2) <= kTbSmemMax, "shared memory");
  return 2;
}

struct TbMaps {
  CUtensorMap z, dout, dz, x, win, wo, wx;
};

template <int C, int ACT>
cudaError_t tb_launch(const TbMaps& m, TbParams p, int grid, cudaStream_t s) {
  p.slots = tb_slots<C>();
  const int bytes = TbSmem<C>::bytes(p.slots);
  const cudaError_t e = tf_allow(transition_bwd_kernel<C, ACT>, bytes, kTbThreads / 128, kRegsSum);
  if (e != cudaSuccess) return e;
  transition_bwd_kernel<C, ACT><<<grid, kTbThreads, bytes, s>>>(m.z, m.dout, m.dz, m.x, m.win, m.wo, m.wx, p);
  return cudaGetLastError();
}

}  // namespace

bool transition_bwd_fused(int C) { return C <= 128; }

cudaError_t launch_transition_bwd(long long M, int C, int H, int act, const void* z, const void* mask,
                                  const float* ln_w, const float* ln_b, const void* w_in, const void* w_o,
                                  const void* d_out, void* dz, void* x, void* g, float* part_g, float* part_b,
                                  int* parts, const WaitCtl& wc, cudaStream_t s) {
  TbMaps m;
  const cuuint64_t c = static_cast<cuuint64_t>(C), hh = static_cast<cuuint64_t>(H), mm = static_cast<cuuint64_t>(M);
  const cuuint64_t zd[3] = {c, mm, 1}, zs[2] = {2 * c, 2 * c * mm};
  const cuuint64_t wd[3] = {hh, 2, c}, ws[2] = {2 * hh, 4 * hh};  // the a and b columns apart: past H reads 0
  const cuuint64_t od[3] = {c, hh, 1}, os[2] = {2 * c, 2 * c * hh};
  if (!tf_map(&m.z, z, zd, zs, 128, 1) || !tf_map(&m.dout, d_out, zd, zs, 128, 1) ||
      !tf_map(&m.dz, dz, zd, zs, 128, 1) || !tf_map(&m.x, x, zd, zs, 128, 1) ||
      !tf_map(&m.win, w_in, wd, ws, 1, static_cast<cuuint32_t>(C)) || !tf_map(&m.wo, w_o, od, os, 32, 1) ||
      !tf_map(&m.wx, w_in, wd, ws, 1, static_cast<cuuint32_t>(C / 2)))
    return cudaErrorInvalidValue;
  TbParams p;
  std::memset(&p, 0, sizeof(p));
  p.M = M;
  p.H = H;
  p.chunks = (H + 63) / 64;
  p.tiles = static_cast<int>((M + 255) / 256);
  p.mask = static_cast<const uint16_t*>(mask);
  p.ln_w = ln_w;
  p.ln_b = ln_b;
  p.g = static_cast<uint16_t*>(g);
  p.part_g = part_g;
  p.part_b = part_b;
  p.wc = wc;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int grid = 2 * std::min(p.tiles, std::min(std::max(sms / 2, 1), kTbPartRows / 8));
  *parts = 4 * grid;
  return by_act(act, [&](auto ic) {
    constexpr int A = decltype(ic)::value;
    switch (C) {
      case 32: return tb_launch<32, A>(m, p, grid, s);
      case 64: return tb_launch<64, A>(m, p, grid, s);
      case 96: return tb_launch<96, A>(m, p, grid, s);
      case 128: return tb_launch<128, A>(m, p, grid, s);
    }
    return cudaErrorInvalidValue;
  });
}

}  // namespace triattn
