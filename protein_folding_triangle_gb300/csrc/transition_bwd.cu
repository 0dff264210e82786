// The transition's backward up to the weight gradients, in one kernel: per
// row tile it computes x, a and b again, dh = g W_o^T, the activation's
// backward, dx = [da | db] W_in^T and the LayerNorm's backward, and leaves
// x, g, h and [da | db] in memory for the weight-gradient GEMMs.
//
// A pair of CTAs (tcgen05 cta_group::2) takes tiles of 256 rows, 128 per CTA;
// each CTA holds one half of the N columns of every B operand.  W_in as the
// operand of [a | b] (CTA 0: W_a, CTA 1: W_b) stays in shared memory.  W_o as
// the operand of dh and W_in again as that of dx, split along C instead of
// the hidden axis, come through a ring per 64-wide hidden chunk: all three
// together do not fit (320 KB at C = 128, H = 512), and these two are 24 KB
// per chunk and CTA, about 18 bytes per clock.
//
// Per tile and chunk:
//   [a | b] = x [W_a | W_b]    M = 256, N = 128, K = C, A = x in TMEM
//   dh      = g W_o^T          M = 256, N = 64,  K = C, A = g in TMEM
//   h = act(a) b, da = dh b act'(a), db = dh act(a)   (registers; BF16 out)
//   dx     += [da | db] W_in^T M = 256, N = C, K = 128, A in TMEM
// x, g (C / 2 columns each), dx (C), [a | b | dh] (192) and [da | db] (64) fill
// the 512 TMEM columns at C = 128.  The issuer queues a chunk's [a | b] and dh
// before the previous chunk's dx, so the activation's arithmetic overlaps
// both.
//
// Warps: 0 loads weights, 1 (of CTA 0) issues the MMAs, 2 tells CTA 0 that
// this CTA's weights are in; 4-7 normalise rows into x, 8-11 write g, 12-15
// take dx through the LayerNorm's backward (thread = row for all three);
// 16-23 the activation.
#include <algorithm>
#include <cstring>

#include "kernels.cuh"
#include "transition.cuh"

namespace triattn {
namespace {

constexpr int kTbThreads = 24 * 32;
// Registers per thread of the warpgroups (setmaxnreg): six shares of what the
// block was launched with (80 each; g's warps keep theirs).
constexpr int kRegsIssue = 48, kRegsX = 88, kRegsG = 80, kRegsLn = 88, kRegsAct = 88;
constexpr int kRegsSum = kRegsIssue + kRegsX + kRegsG + kRegsLn + 2 * kRegsAct;
constexpr int kTbMaxChunks = 32;
constexpr int kTbMaxSlots = 4;
constexpr int kTbBarBytes = 1024 + 1024;  // barriers, ln_w and ln_b
constexpr int kTbSmemMax = 232448;

struct TbBars {
  uint64_t w_load[kTbMaxChunks];                           // a chunk of W_in is in this CTA (TMA bytes)
  uint64_t w_ready[kTbMaxChunks];                          // ... in both (CTA 0)
  uint64_t s_load[kTbMaxSlots], s_ready[kTbMaxSlots];      // the same for a ring slot
  uint64_t s_empty[kTbMaxSlots];                           // its last MMA is done (both)
  uint64_t xg_full, xg_free;                               // x and g written (CTA 0) / read (both)
  uint64_t abd_full, abd_free;                             // [a | b | dh] complete (both) / read (CTA 0)
  uint64_t dab_full, dab_free;                             // [da | db] written (CTA 0) / read (both)
  uint64_t dx_full, dx_free;                               // dx complete (both) / read (CTA 0)
  uint32_t tmem_slot;
  int abort;
};
static_assert(sizeof(TbBars) <= 1024, "barrier block");

struct TbParams {
  long long M;
  int H, chunks, slots, tiles;
  const uint16_t *z, *mask, *d_out;
  const float *ln_w, *ln_b;
  uint16_t *dz, *x, *g, *h, *dab;
  float *part_g, *part_b;
  WaitCtl wc;
};

template <int C>
struct TbSmem {
  static constexpr int kKb = (C + 63) / 64;       // 64-wide K blocks of W_o rows
  static constexpr int kWin = C * 128;            // resident chunk: C rows (K) of 64 columns
  static constexpr int kWo = kKb * 32 * 128;      // ring: 32 hidden rows (N) of C columns (K)
  static constexpr int kWx = (C / 2) * 128;       // ring: C / 2 rows (N) of 64 hidden columns (K), for a and for b
  static constexpr int kSlot = kWo + 2 * kWx;
  static constexpr int bytes(int chunks, int slots) { return chunks * kWin + slots * kSlot + kTbBarBytes + 1024; }
};

// v[j] summed over the 32 lanes for every j, lane l ending with the sum of
// v[l] (halving exchange, fixed order).
__device__ __forceinline__ float lane_scatter_sum(float (&v)[32], int lane) {
#pragma unroll
  for (int n = 16; n > 0; n >>= 1) {
    const bool up = (lane & n) != 0;
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const float keep = up ? v[j + n] : v[j], send = up ? v[j] : v[j + n];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, send, n);
    }
  }
  return v[0];
}

template <int C, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTbThreads, 1)
    transition_bwd_kernel(const __grid_constant__ CUtensorMap tm_win, const __grid_constant__ CUtensorMap tm_wo,
                          const __grid_constant__ CUtensorMap tm_wx, const TbParams p) {
  using L = TbSmem<C>;
  constexpr uint32_t kX = 0, kG = C / 2, kDx = C, kABD = 256, kDAB = 448;  // TMEM columns
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* const s_win = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const s_ring = s_win + p.chunks * L::kWin;
  uint8_t* const s_end = s_ring + p.slots * L::kSlot;
  TbBars* const bars = reinterpret_cast<TbBars*>(s_end);
  float* const s_gam = reinterpret_cast<float*>(s_end + 1024);
  float* const s_bet = s_gam + C;
  volatile int* abort = &bars->abort;
  const WaitCtl& wc = p.wc;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int mine = p.tiles > pair ? (p.tiles - 1 - pair) / pairs + 1 : 0;
  const long long total = static_cast<long long>(mine) * p.chunks;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.chunks; ++i) {
      mbar_init(&bars->w_load[i], 1);
      mbar_init(&bars->w_ready[i], 2);
    }
    for (int i = 0; i < p.slots; ++i) {
      mbar_init(&bars->s_load[i], 1);
      mbar_init(&bars->s_ready[i], 2);
      mbar_init(&bars->s_empty[i], 1);
    }
    mbar_init(&bars->xg_full, 16);
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
  // this thread's row of local tile u (thread-per-row warps)
  const int quarter = warp & 3, r = quarter * 32 + lane;
  const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
  auto row_of = [&](int u) {
    return (static_cast<long long>(pair) + static_cast<long long>(u) * pairs) * 256 + rank * 128 + r;
  };

  // each warpgroup sets its register budget at its start (warps 0-3 share one)
  if (warp < 4) regs_dec<kRegsIssue>();
  if (warp == 0) {
    // ------------------------------------------------------------ weights
    if (lane == 0) {
      int slot = 0, phase = 0;
      for (long long g = 0; g < total; ++g) {
        const int i = static_cast<int>(g % p.chunks);
        if (g < p.chunks) {
          mbar_expect_tx(&bars->w_load[i], L::kWin);
          tma_load_3d(s_win + i * L::kWin, &tm_win, &bars->w_load[i], 64 * i, static_cast<int>(rank), 0);
        }
        if (!mbar_wait(&bars->s_empty[slot], phase ^ 1, wc, abort)) break;
        uint8_t* const dst = s_ring + slot * L::kSlot;
        mbar_expect_tx(&bars->s_load[slot], L::kSlot);
#pragma unroll
        for (int b = 0; b < L::kKb; ++b)
          tma_load_3d(dst + b * 4096, &tm_wo, &bars->s_load[slot], 64 * b, 64 * i + 32 * static_cast<int>(rank), 0);
#pragma unroll
        for (int b = 0; b < 2; ++b)
          tma_load_3d(dst + L::kWo + b * L::kWx, &tm_wx, &bars->s_load[slot], 64 * i, b,
                      static_cast<int>(rank) * (C / 2));
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
        if (g < p.chunks) {
          if (!mbar_wait(&bars->w_load[g], 0, wc, abort)) break;
          mbar_arrive_cta(&bars->w_ready[g], 0);
        }
        if (!mbar_wait(&bars->s_load[slot], phase, wc, abort)) break;
        mbar_arrive_cta(&bars->s_ready[slot], 0);
        if (++slot == p.slots) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0) {
      constexpr uint32_t id_ab = idesc_bf16_f32(256, 128, 0, 1);  // B: N contiguous
      constexpr uint32_t id_dh = idesc_bf16_f32(256, 64, 0, 0);   // B: K contiguous
      constexpr uint32_t id_dx = idesc_bf16_f32(256, C, 0, 0);
      // operand descriptors; an offset of n bytes adds n / 16
      const uint64_t d_win = smem_desc(smem_u32(s_win), 64 * 128, 1024, 2);
      const uint64_t d_ring = smem_desc(smem_u32(s_ring), 16, 1024, 2);
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity, wc, abort));
      };
      int t = 0, i = 0, slot = 0, phase = 0;  // of the next [a | b]
      int xt = 0, xi = 0, xslot = 0;          // of the next dx
      uint32_t xg = 0;
      auto issue_dx = [&]() {
        wait(&bars->dab_full, xg & 1);
        if (xi == 0 && xt > 0) wait(&bars->dx_free, (xt - 1) & 1);
        if (!ok) return;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t wx = d_ring + (xslot * L::kSlot + L::kWo) / 16;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ts_pair(tmem + kDx, tmem + kDAB + 8 * k, wx + ((k >> 2) * L::kWx + (k & 3) * 32) / 16, id_dx,
                        (xi > 0 || k > 0) ? 1u : 0u);
          mma_commit_pair(&bars->dab_free);
          mma_commit_pair(&bars->s_empty[xslot]);
          if (xi == p.chunks - 1) mma_commit_pair(&bars->dx_full);
        }
        __syncwarp();
        ++xg;
        if (++xslot == p.slots) xslot = 0;
        if (++xi == p.chunks) {
          xi = 0;
          ++xt;
        }
      };
      for (long long g = 0; g < total && ok; ++g) {
        if (i == 0) wait(&bars->xg_full, t & 1);
        if (t == 0) wait(&bars->w_ready[i], 0);
        if (g > 0) wait(&bars->abd_free, static_cast<uint32_t>(g - 1) & 1);
        wait(&bars->s_ready[slot], phase);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t wa = d_win + i * L::kWin / 16, wo = d_ring + slot * L::kSlot / 16;
#pragma unroll
          for (int k = 0; k < C / 16; ++k)
            mma_ts_pair(tmem + kABD, tmem + kX + 8 * k, wa + k * 2048 / 16, id_ab, k > 0 ? 1u : 0u);
#pragma unroll
          for (int k = 0; k < C / 16; ++k)
            mma_ts_pair(tmem + kABD + 128, tmem + kG + 8 * k, wo + ((k >> 2) * 4096 + (k & 3) * 32) / 16, id_dh,
                        k > 0 ? 1u : 0u);
          mma_commit_pair(&bars->abd_full);
          if (i == p.chunks - 1) mma_commit_pair(&bars->xg_free);
        }
        __syncwarp();
        if (g > 0) issue_dx();
        if (++slot == p.slots) {
          slot = 0;
          phase ^= 1;
        }
        if (++i == p.chunks) {
          i = 0;
          ++t;
        }
      }
      if (ok && total > 0) issue_dx();
    }
  } else if (warp >= 4 && warp < 8) {
    regs_inc<kRegsX>();
    // ------------------------------------------------------------ x = LayerNorm(z)
    for (int u = 0; u < mine; ++u) {
      const long long row = row_of(u);
      const bool in = row < p.M;
      const bool live = in && (p.mask == nullptr || (p.mask[row] & 0x7FFFu) != 0);
      // three passes over the row (the later ones hit L1 or L2): the row in
      // FP32, or packed beside its result, would not fit the registers
      auto z16 = [&](int c, uint32_t (&v)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0u;
        if (live) ld_global_2v4(p.z + row * C + 16 * c, v);
      };
      float s = 0.f;
#pragma unroll 2
      for (int c = 0; c < C / 16; ++c) {
        uint32_t v[8];
        z16(c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += bf16lo_to_f32(v[e]) + bf16hi_to_f32(v[e]);
      }
      const float mean = s * (1.f / C);
      float q = 0.f;
#pragma unroll 2
      for (int c = 0; c < C / 16; ++c) {
        uint32_t v[8];
        z16(c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a = bf16lo_to_f32(v[e]) - mean, b = bf16hi_to_f32(v[e]) - mean;
          q = fmaf(a, a, fmaf(b, b, q));
        }
      }
      const float rstd = rsqrtf(q * (1.f / C) + 1e-5f);
      uint32_t w[C / 2];
#pragma unroll
      for (int c = 0; c < C / 16; ++c) {
        uint32_t v[8];
        z16(c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 gm = *reinterpret_cast<const float2*>(s_gam + 16 * c + 2 * e);
          const float2 bt = *reinterpret_cast<const float2*>(s_bet + 16 * c + 2 * e);
          const uint32_t x = pack_bf16x2(fmaf((bf16lo_to_f32(v[e]) - mean) * rstd, gm.x, bt.x),
                                         fmaf((bf16hi_to_f32(v[e]) - mean) * rstd, gm.y, bt.y));
          w[8 * c + e] = live ? x : 0u;  // a row left out, or past the end: x = 0
        }
      }
      if (u > 0 && !__all_sync(0xffffffffu, mbar_wait(&bars->xg_free, (u - 1) & 1, wc, abort))) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < C / 16; ++c) {
        uint32_t v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = w[8 * c + e];
        tmem_st8(tmem + lane_addr + kX + 8 * c, v);
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&bars->xg_full, 0);
      if (in) {
#pragma unroll
        for (int c = 0; c < C / 16; ++c) {
          uint32_t v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = w[8 * c + e];
          st_global_v8(p.x + row * C + 16 * c, v);
        }
      }
    }
  } else if (warp >= 8 && warp < 12) {
    // ------------------------------------------------------------ g = m d_out
    for (int u = 0; u < mine; ++u) {
      const long long row = row_of(u);
      const bool in = row < p.M;
      const float mk = !in ? 0.f : (p.mask != nullptr ? bf16lo_to_f32(p.mask[row]) : 1.f);
      uint32_t w[C / 2];
#pragma unroll
      for (int c = 0; c < C / 16; ++c) {
        uint32_t v[8] = {};
        if (mk != 0.f) ld_global_2v4(p.d_out + row * C + 16 * c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[8 * c + e] = v[e];
      }
      if (p.mask != nullptr) {
#pragma unroll
        for (int e = 0; e < C / 2; ++e)
          w[e] = mk != 0.f ? pack_bf16x2(bf16lo_to_f32(w[e]) * mk, bf16hi_to_f32(w[e]) * mk) : 0u;
      }
      if (u > 0 && !__all_sync(0xffffffffu, mbar_wait(&bars->xg_free, (u - 1) & 1, wc, abort))) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < C / 16; ++c) {
        uint32_t v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = w[8 * c + e];
        tmem_st8(tmem + lane_addr + kG + 8 * c, v);
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&bars->xg_full, 0);
      if (in && p.mask != nullptr) {
#pragma unroll
        for (int c = 0; c < C / 16; ++c) {
          uint32_t v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = w[8 * c + e];
          st_global_v8(p.g + row * C + 16 * c, v);
        }
      }
    }
  } else if (warp >= 12 && warp < 16) {
    regs_inc<kRegsLn>();
    // ------------------------------------------------------------ LayerNorm backward
    // dz = rstd (t - mean(t) - xhat mean(t xhat)), t = dx ln_w.  The row's
    // statistics and xhat are computed from z again (in L2); dx is read from
    // TMEM twice, first for the two means and the parameter gradients' sums
    // over the rows, which end one column per lane, then for dz.
    float accg[C / 32], accb[C / 32];
#pragma unroll
    for (int b = 0; b < C / 32; ++b) accg[b] = accb[b] = 0.f;
    for (int u = 0; u < mine; ++u) {
      const long long row = row_of(u);
      const bool in = row < p.M;
      const bool live = in && (p.mask == nullptr || (p.mask[row] & 0x7FFFu) != 0);
      const uint16_t* const zr = p.z + row * C;
      auto z32 = [&](int b, uint32_t (&zw)[16]) {  // features 32 b .. 32 b + 31
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t v[8] = {};
          if (live) ld_global_2v4(zr + 32 * b + 16 * c, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) zw[8 * c + e] = v[e];
        }
      };
      float s = 0.f, q = 0.f;
#pragma unroll 1
      for (int b = 0; b < C / 32; ++b) {
        uint32_t zw[16];
        z32(b, zw);
#pragma unroll
        for (int e = 0; e < 16; ++e) s += bf16lo_to_f32(zw[e]) + bf16hi_to_f32(zw[e]);
      }
      const float mean = s * (1.f / C);
#pragma unroll 1
      for (int b = 0; b < C / 32; ++b) {
        uint32_t zw[16];
        z32(b, zw);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float a0 = bf16lo_to_f32(zw[e]) - mean, a1 = bf16hi_to_f32(zw[e]) - mean;
          q = fmaf(a0, a0, fmaf(a1, a1, q));
        }
      }
      const float rstd = rsqrtf(q * (1.f / C) + 1e-5f);
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->dx_full, u & 1, wc, abort))) break;
      tc_fence_after();
      float sg = 0.f, sgx = 0.f;
#pragma unroll
      for (int b = 0; b < C / 32; ++b) {
        float v[32];
        {
          uint32_t d[32];
          tmem_ld32_wait(tmem + lane_addr + kDx + 32 * b, d);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t zw[8] = {};
            if (live) ld_global_2v4(zr + 32 * b + 16 * c, zw);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float zf = (e & 1) ? bf16hi_to_f32(zw[e >> 1]) : bf16lo_to_f32(zw[e >> 1]);
              const float dxe = __uint_as_float(d[16 * c + e]), xh = (zf - mean) * rstd;
              const float t = dxe * s_gam[32 * b + 16 * c + e];
              sg += t;
              sgx = fmaf(t, xh, sgx);
              v[16 * c + e] = dxe * xh;
            }
          }
        }
        accg[b] += lane_scatter_sum(v, lane);
        uint32_t d[32];  // once more, so that it need not be kept
        tmem_ld32_wait(tmem + lane_addr + kDx + 32 * b, d);
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(d[e]);
        accb[b] += lane_scatter_sum(v, lane);
      }
      const float m1 = sg * (1.f / C), m2 = sgx * (1.f / C);
#pragma unroll 1
      for (int b = 0; b < C / 32; ++b) {
        uint32_t zw[16], d[32];
        z32(b, zw);
        tmem_ld32_wait(tmem + lane_addr + kDx + 32 * b, d);
        if (b == C / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(&bars->dx_free, 0);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int k = 8 * c + e;
            const float x0 = (bf16lo_to_f32(zw[k]) - mean) * rstd, x1 = (bf16hi_to_f32(zw[k]) - mean) * rstd;
            const float2 gm = *reinterpret_cast<const float2*>(s_gam + 32 * b + 2 * k);
            o[e] = pack_bf16x2(rstd * (__uint_as_float(d[2 * k]) * gm.x - m1 - x0 * m2),
                               rstd * (__uint_as_float(d[2 * k + 1]) * gm.y - m1 - x1 * m2));
            if (!live) o[e] = 0u;
          }
          if (in) st_global_2v4(p.dz + row * C + 32 * b + 16 * c, o);
        }
      }
    }
    const int part = static_cast<int>(blockIdx.x) * 4 + quarter;
#pragma unroll
    for (int b = 0; b < C / 32; ++b) {
      p.part_g[static_cast<size_t>(part) * C + 32 * b + lane] = accg[b];
      p.part_b[static_cast<size_t>(part) * C + 32 * b + lane] = accb[b];
    }
  } else if (warp >= 16) {
    regs_inc<kRegsAct>();
    // ------------------------------------------------------------ activation
    // Warp = 32 rows x 32 of the chunk's 64 hidden features, 16 at a time.
    const int hf = (warp - 16) >> 2;
    const uint32_t base = tmem + lane_addr;
    int u = 0, i = 0;
    for (long long g = 0; g < total; ++g) {
      const long long row = row_of(u);
      const int hid = 64 * i + 32 * hf;
      const bool store = row < p.M && hid < p.H;
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->abd_full, static_cast<uint32_t>(g) & 1, wc, abort))) break;
      tc_fence_after();
      bool ok = true;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t a[16], b[16], d[16], ho[8], ao[8], bo[8];
        const uint32_t col = base + kABD + 32 * hf + 16 * j;
        tmem_ld16x3_wait(col, a, col + 64, b, col + 128, d);
        if (j == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(&bars->abd_free, 0);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float hv[2], av[2], bv[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float bb = __uint_as_float(b[2 * e + k]), dd = __uint_as_float(d[2 * e + k]);
            float f, df;
            act_both<ACT>(__uint_as_float(a[2 * e + k]), f, df);
            hv[k] = f * bb;
            av[k] = dd * bb * df;
            bv[k] = dd * f;
          }
          ho[e] = pack_bf16x2(hv[0], hv[1]);
          ao[e] = pack_bf16x2(av[0], av[1]);
          bo[e] = pack_bf16x2(bv[0], bv[1]);
        }
        if (j == 0 && g > 0) {  // the previous chunk's dx has read [da | db]
          ok = __all_sync(0xffffffffu, mbar_wait(&bars->dab_free, static_cast<uint32_t>(g - 1) & 1, wc, abort));
          if (!ok) break;
          tc_fence_after();
        }
        tmem_st8(base + kDAB + 16 * hf + 8 * j, ao);
        tmem_st8(base + kDAB + 32 + 16 * hf + 8 * j, bo);
        if (j == 1) {
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(&bars->dab_full, 0);
        }
        if (store) {
          st_global_v8(p.h + row * p.H + hid + 16 * j, ho);
          st_global_v8(p.dab + row * 2 * p.H + hid + 16 * j, ao);
          st_global_v8(p.dab + row * 2 * p.H + p.H + hid + 16 * j, bo);
        }
      }
      if (!ok) break;
      if (++i == p.chunks) {
        i = 0;
        ++u;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no arrival is under way to a CTA that has left
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <int C>
int tb_slots(int chunks) {
  for (int s = kTbMaxSlots; s >= 3; --s)
    if (TbSmem<C>::bytes(chunks, s) <= kTbSmemMax) return s;
  return 0;
}
int tb_slots_for(int C, int H) {
  const int chunks = (H + 63) / 64;
  if (chunks > kTbMaxChunks) return 0;
  switch (C) {
    case 32: return tb_slots<32>(chunks);
    case 64: return tb_slots<64>(chunks);
    case 96: return tb_slots<96>(chunks);
    case 128: return tb_slots<128>(chunks);
  }
  return 0;
}

template <int C, int ACT>
cudaError_t tb_launch(const CUtensorMap& ti, const CUtensorMap& to, const CUtensorMap& tx, const TbParams& p, int grid,
                      cudaStream_t s) {
  const int bytes = TbSmem<C>::bytes(p.chunks, p.slots);
  cudaError_t e = cudaFuncSetAttribute(transition_bwd_kernel<C, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       bytes);
  cudaFuncAttributes at;
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, transition_bwd_kernel<C, ACT>);
  if (e != cudaSuccess) return e;
  // a split above the launch's registers would wait for ever
  if (at.numRegs * (kTbThreads / 128) < kRegsSum) return cudaErrorInvalidConfiguration;
  transition_bwd_kernel<C, ACT><<<grid, kTbThreads, bytes, s>>>(ti, to, tx, p);
  return cudaGetLastError();
}

}  // namespace

bool transition_bwd_fused(int C, int H) { return tb_slots_for(C, H) > 0; }

cudaError_t launch_transition_bwd(long long M, int C, int H, int act, const void* z, const void* mask,
                                  const float* ln_w, const float* ln_b, const void* w_in, const void* w_o,
                                  const void* d_out, void* dz, void* x, void* g, void* h, void* dab, float* part_g,
                                  float* part_b, int* parts, const WaitCtl& wc, cudaStream_t s) {
  CUtensorMap ti, to, tx;
  const cuuint64_t c = static_cast<cuuint64_t>(C), hh = static_cast<cuuint64_t>(H);
  const cuuint64_t wd[3] = {hh, 2, c}, ws[2] = {2 * hh, 4 * hh};  // the a and b columns apart: past H reads 0
  const cuuint64_t od[3] = {c, hh, 1}, os[2] = {2 * c, 2 * c * hh};
  if (!tf_map(&ti, w_in, wd, ws, 1, static_cast<cuuint32_t>(C)) || !tf_map(&to, w_o, od, os, 32, 1) ||
      !tf_map(&tx, w_in, wd, ws, 1, static_cast<cuuint32_t>(C / 2)))
    return cudaErrorInvalidValue;
  TbParams p;
  std::memset(&p, 0, sizeof(p));
  p.M = M;
  p.H = H;
  p.chunks = (H + 63) / 64;
  p.slots = tb_slots_for(C, H);
  p.tiles = static_cast<int>((M + 255) / 256);
  p.z = static_cast<const uint16_t*>(z);
  p.mask = static_cast<const uint16_t*>(mask);
  p.d_out = static_cast<const uint16_t*>(d_out);
  p.ln_w = ln_w;
  p.ln_b = ln_b;
  p.dz = static_cast<uint16_t*>(dz);
  p.x = static_cast<uint16_t*>(x);
  p.g = static_cast<uint16_t*>(g);
  p.h = static_cast<uint16_t*>(h);
  p.dab = static_cast<uint16_t*>(dab);
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
      case 32: return tb_launch<32, A>(ti, to, tx, p, grid, s);
      case 64: return tb_launch<64, A>(ti, to, tx, p, grid, s);
      case 96: return tb_launch<96, A>(ti, to, tx, p, grid, s);
      case 128: return tb_launch<128, A>(ti, to, tx, p, grid, s);
    }
    return cudaErrorInvalidValue;
  });
}

}  // namespace triattn
