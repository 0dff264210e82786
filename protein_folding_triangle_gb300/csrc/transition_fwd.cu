// The transition's forward in one kernel: LayerNorm, both input projections,
// activation and product, output projection and row mask; z is read once and
// out written once, x, a, b and h stay on the chip.
//
// A pair of CTAs (cluster of two, tcgen05 cta_group::2) takes tiles of 256
// rows, 128 per CTA.  With cta_group::2 each CTA holds one half of the N
// columns of every B operand: CTA 0 W_a and columns [0, C/2) of W_o, CTA 1 W_b
// and columns [C/2, C).  Where it fits W_in is loaded once per pair and stays
// (128 KB per CTA at C = 128, H = 512; streaming it for every 128 rows would
// take 36 bytes per clock and SM from L2), else it comes through a ring of
// chunks, as W_o does, a third of the bytes.
//
// Per tile and 64-wide hidden chunk i (K = C, then K = 64):
//   [a | b] = x [W_a | W_b] chunk      M = 256, N = 128, A = x in TMEM
//   h = act(a) b                       registers, BF16 back into TMEM
//   out += h W_o chunk                 M = 256, N = C, A = h in TMEM
// At C <= 128 x, out, two stages of h and two of [a | b] fill the 512 TMEM
// columns; a stage of [a | b] is free for the next chunk but one as soon as
// the activation has read it, whatever becomes of its h.  Wider rows leave
// room for one stage and none for x, which is the A operand from shared
// memory instead (a third longer per MMA); a chunk's [a | b] then takes 16
// MMAs against the activation's reading it, so one stage is enough.
//
// Warps: 0 loads the weights, 3 tells CTA 0 that this CTA's are in; 1 and 2 (of
// CTA 0) issue the MMAs of both CTAs, one the input projections, one the output
// projection: a wait costs an issuer some 200 clocks even when the phase is
// complete, and the tensor cores' queue is shorter than that (one issuer for
// both kept them busy for 60% of the time); 4-7 normalise the next tile's rows,
// 8-11 drain out (thread = row for both; one group for both took 10,000 clocks
// a tile, more than its MMAs); 12-27 the activation, eight warps per stage, so
// that a chunk's arithmetic may take the time of two chunks' MMAs.
//
// What bounds it is the MMAs' pace and the waits between them: 0.160 ms at
// 768 x 768 rows, C = 128, H = 512, against 0.118 ms of products and 0.045 ms of
// memory; the tensor pipe is active for 61 % of it (103 clocks per MMA, all told,
// where the pipe needs 64).  384 x 384 rows, C = 256, H = 1024, GELU: 0.254 ms
// against 0.118, the pipe active for 38 %: with one stage of [a | b] the products of
// a chunk wait until the activation has read the chunk before.  640 x 640 rows,
// C = 64, H = 256: 0.056 ms against 0.021, 30 %: at K = 64 the LayerNorm and the
// activation take longer than the products.
//
// Roundings: x and h are BF16 because they are operands of the tensor cores (TF32
// runs at half the rate, and twice the bytes do not fit TMEM and shared memory
// beside the weights); a, b, the statistics and every sum are FP32.  The relative
// error of out is 3.4e-3, of which one rounding of the result is 1.7e-3.
#include <algorithm>
#include <cstring>

#include "kernels.cuh"
#include "transition.cuh"

namespace triattn {
namespace {

constexpr int kTfThreads = 28 * 32;
// Registers per thread of the warpgroups (setmaxnreg): seven shares of what
// the block was launched with (72 each).
constexpr int kTfRegsIssue = 40, kTfRegsLn = 56, kTfRegsOut = 88, kTfRegsAct = 80;
constexpr int kTfRegsSum = kTfRegsIssue + kTfRegsLn + kTfRegsOut + 4 * kTfRegsAct;
constexpr int kTfMaxSlots = 32;  // W_in chunks in shared memory
constexpr int kTfSlots = 3;  // W_o ring
constexpr int kTfSmemMax = 232448;

struct TfBars {
  uint64_t w_load[kTfMaxSlots];    // a chunk of W_in is in this CTA (TMA bytes)
  uint64_t w_ready[kTfMaxSlots];   // ... in both CTAs (CTA 0)
  uint64_t w_empty[kTfMaxSlots];   // ... read (both; where W_in does not stay)
  uint64_t o_load[kTfSlots], o_ready[kTfSlots], o_empty[kTfSlots];  // the same for W_o's ring; read (both)
  uint64_t z_full[2];              // z tile in shared memory (TMA bytes)
  uint64_t x_full, x_free;         // x tile written (CTA 0) / read by its last MMA (both)
  uint64_t ab_full[2], ab_free[2]; // [a | b] of a stage complete (both) / read (CTA 0)
  uint64_t h_full[2], h_free[2];   // h of a stage written (CTA 0) / read (both)
  uint64_t out_full, out_free;     // out complete (both) / drained (CTA 0)
  uint32_t tmem_slot;
  int abort;
};
static_assert(sizeof(TfBars) <= 1024, "barrier block");

struct TfParams {
  long long M;
  int chunks, tiles, slots;  // slots of W_in; as many as chunks where it stays
  const uint16_t* mask;
  const float *ln_w, *ln_b;
  WaitCtl wc;
};

template <int C>
struct TfSmem {
  static constexpr bool kXs = C > 128;         // x is an operand from shared memory
  static constexpr int kZBoxes = (C + 63) / 64;
  static constexpr int kZ = kZBoxes * 16384;
  static constexpr int kOBoxes = (C / 2 + 63) / 64;
  static constexpr int kWin = C * 128;            // one chunk: C rows (K) of 64 columns
  static constexpr int kWo = kOBoxes * 64 * 128;  // one chunk: 64 rows (K) of C / 2 columns, in blocks of 64
  static constexpr int kStg = 4 * 2048;           // out's staging: 32 rows of 32 features per warp
  static constexpr int kBar = 1024 + (8 * C + 1023) / 1024 * 1024;  // barriers; ln_w and ln_b
  static constexpr int rest(int zt) { return kTfSlots * kWo + zt * kZ + kStg + kBar + 1024; }  // + alignment
  static constexpr int fit(int zt) { return (kTfSmemMax - rest(zt)) / kWin; }
  // a second z tile where it leaves W_in at least two slots
  static constexpr int kZt = fit(2) >= 2 ? 2 : 1;
  static constexpr int kFit = fit(kZt) < kTfMaxSlots ? fit(kZt) : kTfMaxSlots;
  static_assert(kFit >= 2, "shared memory");
  static constexpr int bytes(int slots) { return rest(kZt) + slots * kWin; }
};

template <int C, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTfThreads, 1)
    transition_fwd_kernel(const __grid_constant__ CUtensorMap tm_z, const __grid_constant__ CUtensorMap tm_out,
                          const __grid_constant__ CUtensorMap tm_win, const __grid_constant__ CUtensorMap tm_wo,
                          const TfParams p) {
  using L = TfSmem<C>;
  constexpr bool kXs = L::kXs;
  // TMEM columns: x, out, two stages of h (32), two of [a | b] (128); or out, [a | b], h
  constexpr uint32_t kX = 0, kOut = kXs ? 0 : 64, kH = kXs ? 384 : 192, kAB = 256, kABStage = kXs ? 0 : 128;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* const s_win = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const s_wo = s_win + p.slots * L::kWin;
  uint8_t* const s_z = s_wo + kTfSlots * L::kWo;
  uint8_t* const s_stg = s_z + L::kZt * L::kZ;
  TfBars* const bars = reinterpret_cast<TfBars*>(s_stg + L::kStg);
  float* const s_gam = reinterpret_cast<float*>(s_stg + L::kStg + 1024);
  float* const s_bet = s_gam + C;
  volatile int* abort = &bars->abort;
  const WaitCtl& wc = p.wc;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int mine = p.tiles > pair ? (p.tiles - 1 - pair) / pairs + 1 : 0;  // tiles of this pair
  const long long total = static_cast<long long>(mine) * p.chunks;
  const bool stays = p.slots == p.chunks;  // W_in is loaded once

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.slots; ++i) {
      mbar_init(&bars->w_load[i], 1);
      mbar_init(&bars->w_ready[i], 2);
      mbar_init(&bars->w_empty[i], 1);
    }
    for (int i = 0; i < kTfSlots; ++i) {
      mbar_init(&bars->o_load[i], 1);
      mbar_init(&bars->o_ready[i], 2);
      mbar_init(&bars->o_empty[i], 1);
    }
    mbar_init(&bars->x_full, 8);
    mbar_init(&bars->x_free, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->z_full[i], 1);
      mbar_init(&bars->ab_full[i], 1);
      mbar_init(&bars->ab_free[i], 16);
      mbar_init(&bars->h_full[i], 16);
      mbar_init(&bars->h_free[i], 1);
    }
    mbar_init(&bars->out_full, 1);
    mbar_init(&bars->out_free, 8);
    bars->abort = 0;
    fence_mbar_init();
  }
  for (int c = threadIdx.x; c < C; c += kTfThreads) {
    s_gam[c] = p.ln_w[c];
    s_bet[c] = p.ln_b[c];
  }
  if (warp == 1) tmem_alloc_pair(&bars->tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before the first remote arrival
  tc_fence_after();
  const uint32_t tmem = bars->tmem_slot;

  if (warp < 4) regs_dec<kTfRegsIssue>();
  if (warp == 0) {
    // ------------------------------------------------------------ weights
    if (lane == 0) {
      auto load_win = [&](int i, int slot) {
        mbar_expect_tx(&bars->w_load[slot], L::kWin);
        tma_load_3d(s_win + slot * L::kWin, &tm_win, &bars->w_load[slot], 64 * i, static_cast<int>(rank), 0);
      };
      int slot = 0, phase = 0, ws = 0, wphase = 0, i = 0;
      for (long long g = 0; g < total; ++g) {
        if (!stays) {
          if (!mbar_wait(&bars->w_empty[ws], wphase ^ 1, wc, abort)) break;
          load_win(i, ws);
          if (++ws == p.slots) {
            ws = 0;
            wphase ^= 1;
          }
        } else if (g == 0) {
          load_win(0, 0);
        } else if (g == 1) {  // behind the first chunk's weights, the rest of W_in
          for (int k = 1; k < p.chunks; ++k) load_win(k, k);
        }
        if (!mbar_wait(&bars->o_empty[slot], phase ^ 1, wc, abort)) break;
        mbar_expect_tx(&bars->o_load[slot], L::kWo);
#pragma unroll
        for (int b = 0; b < L::kOBoxes; ++b)
          tma_load_3d(s_wo + slot * L::kWo + b * 8192, &tm_wo, &bars->o_load[slot],
                      static_cast<int>(rank) * (C / 2) + 64 * b, 64 * i, 0);
        if (++i == p.chunks) i = 0;
        if (++slot == kTfSlots) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ weights' arrival, to CTA 0
    if (lane == 0) {
      int slot = 0, phase = 0, ws = 0, wphase = 0;
      for (long long g = 0; g < total; ++g) {
        if (!stays || g < p.chunks) {
          if (!mbar_wait(&bars->w_load[ws], wphase, wc, abort)) break;
          mbar_arrive_cta(&bars->w_ready[ws], 0);
          if (++ws == p.slots) {
            ws = 0;
            wphase ^= 1;
          }
        }
        if (!mbar_wait(&bars->o_load[slot], phase, wc, abort)) break;
        mbar_arrive_cta(&bars->o_ready[slot], 0);
        if (++slot == kTfSlots) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer: [a | b]
    if (rank == 0) {
      constexpr uint32_t id_ab = idesc_bf16_f32(256, 128, 0, 1);
      const uint64_t d_win = smem_desc(smem_u32(s_win), 64 * 128, 1024, 2);  // an offset of n bytes adds n / 16
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity, wc, abort));
      };
      const uint64_t d_x = smem_desc(smem_u32(s_z), 16, 1024, 2);
      int t = 0, i = 0, ws = 0, wphase = 0;
      for (long long g = 0; g < total; ++g) {
        const uint32_t st = static_cast<uint32_t>(g & 1);
        // the chunk that had this stage's columns before has been read
        if constexpr (kXs) {
          if (g >= 1) wait(&bars->ab_free[st ^ 1], static_cast<uint32_t>((g - 1) >> 1) & 1);
        } else {
          if (g >= 2) wait(&bars->ab_free[st], static_cast<uint32_t>((g >> 1) - 1) & 1);
        }
        if (i == 0) ok = ok && __all_sync(0xffffffffu, mbar_wait<kXs>(&bars->x_full, t & 1, wc, abort));
        if (!stays || t == 0) wait(&bars->w_ready[ws], wphase);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t w = d_win + ws * (L::kWin / 16);
          const uint64_t x = d_x + (L::kZt == 2 ? (t & 1) : 0) * (L::kZ / 16);
#pragma unroll
          for (int k = 0; k < C / 16; ++k) {
            if constexpr (kXs)
              mma_ss_pair(tmem + kAB, x + ((k >> 2) * 16384 + (k & 3) * 32) / 16, w + k * (2048 / 16), id_ab,
                          k > 0 ? 1u : 0u);
            else
              mma_ts_pair(tmem + kAB + kABStage * st, tmem + kX + 8 * k, w + k * (2048 / 16), id_ab, k > 0 ? 1u : 0u);
          }
          mma_commit_pair(&bars->ab_full[st]);
          if (!stays) mma_commit_pair(&bars->w_empty[ws]);
          if (i == p.chunks - 1) mma_commit_pair(&bars->x_free);
        }
        __syncwarp();
        if (++ws == p.slots) {
          ws = 0;
          wphase ^= 1;
        }
        if (++i == p.chunks) {
          i = 0;
          ++t;
        }
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ MMA issuer: out
    if (rank == 0) {
      constexpr uint32_t id_out = idesc_bf16_f32(256, C, 0, 1);
      const uint64_t d_wo = smem_desc(smem_u32(s_wo), 64 * 128, 1024, 2);
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity, wc, abort));
      };
      int t = 0, i = 0, slot = 0, phase = 0;
      for (long long g = 0; g < total; ++g) {
        const uint32_t st = static_cast<uint32_t>(g & 1);
        wait(&bars->o_ready[slot], phase);
        if (i == 0 && t > 0) wait(&bars->out_free, (t - 1) & 1);
        wait(&bars->h_full[st], (g >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t w = d_wo + slot * (L::kWo / 16);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ts_pair(tmem + kOut, tmem + kH + 32 * st + 8 * k, w + k * (2048 / 16), id_out,
                        (i > 0 || k > 0) ? 1u : 0u);
          mma_commit_pair(&bars->h_free[st]);
          mma_commit_pair(&bars->o_empty[slot]);
          if (i == p.chunks - 1) mma_commit_pair(&bars->out_full);
        }
        __syncwarp();
        if (++slot == kTfSlots) {
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
    // ------------------------------------------------------------ x = LayerNorm(z)
    regs_dec<kTfRegsLn>();
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const bool first = warp == 4 && lane == 0;
    auto load_z = [&](int u) {
      const int row = (pair + u * pairs) * 256 + static_cast<int>(rank) * 128;
      const int zb = L::kZt == 2 ? (u & 1) : 0;
      uint64_t* const bar = &bars->z_full[u & 1];
      mbar_expect_tx(bar, L::kZ);
#pragma unroll
      for (int b = 0; b < L::kZBoxes; ++b)
        tma_load_3d(s_z + zb * L::kZ + b * 16384, &tm_z, bar, 64 * b, row, 0);
    };
    auto normalise = [&](int u) -> bool {
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->z_full[u & 1], (u >> 1) & 1, wc, abort))) return false;
      uint8_t* const zt = s_z + (L::kZt == 2 ? (u & 1) : 0) * L::kZ;
      auto z16 = [&](int c) { return reinterpret_cast<uint4*>(zt + (c >> 3) * 16384 + sw128(r, c & 7)); };
      const float2 st = row_stats<C>(z16);
      const float mean = st.x, rstd = st.y;
      const float2 nm = make_float2(-mean, -mean), rs = make_float2(rstd, rstd);
      // x over z in shared memory first, so that little is left to do once the
      // previous tile's x has been read
#pragma unroll 4
      for (int c = 0; c < C / 8; ++c) {
        const uint4 w = *z16(c);
        uint32_t ws[4] = {w.x, w.y, w.z, w.w};
        const float4* gm = reinterpret_cast<const float4*>(s_gam + 8 * c);
        const float4* bt = reinterpret_cast<const float4*>(s_bet + 8 * c);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 g = gm[e], b = bt[e];
          const float2 x0 = ffma2(fmul2(fadd2(bf16x2_to_f32x2(ws[2 * e]), nm), rs), make_float2(g.x, g.y),
                                  make_float2(b.x, b.y));
          const float2 x1 = ffma2(fmul2(fadd2(bf16x2_to_f32x2(ws[2 * e + 1]), nm), rs), make_float2(g.z, g.w),
                                  make_float2(b.z, b.w));
          ws[2 * e] = pack_bf16x2(x0.x, x0.y);
          ws[2 * e + 1] = pack_bf16x2(x1.x, x1.y);
        }
        *z16(c) = make_uint4(ws[0], ws[1], ws[2], ws[3]);
      }
      if constexpr (kXs) {
        // Before the arrival: as long as this tile's products cannot start, x_free
        // cannot pass the phase waited for; nor can x_full pass the one that the
        // issuer waits for, since it takes each x_full before it issues the
        // products that x_free stands for.
        if (u > 0 && !__all_sync(0xffffffffu, mbar_wait(&bars->x_free, (u - 1) & 1, wc, abort))) return false;
        fence_proxy_async_smem();
      } else {
        if (u > 0 && !__all_sync(0xffffffffu, mbar_wait(&bars->x_free, (u - 1) & 1, wc, abort))) return false;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < C / 8; c += 4) {  // 32 features = 16 columns at a time
          uint32_t x[16];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 w = *z16(c + j);
            x[4 * j] = w.x;
            x[4 * j + 1] = w.y;
            x[4 * j + 2] = w.z;
            x[4 * j + 3] = w.w;
          }
          tmem_st16(tmem + lane_addr + kX + 4 * c, x);
        }
        tc_wait_st();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) {
        // x in shared memory was stored by this CTA and is read for the MMAs that CTA
        // 0's issuer starts: release and acquire have to reach across the pair
        if constexpr (kXs) mbar_arrive_cluster(&bars->x_full, 0);
        else mbar_arrive_cta(&bars->x_full, 0);
      }
      return true;
    };
    bool ok = true;
    if (first && mine > 0) load_z(0);
    if constexpr (kXs) {
      for (int u = 0; u < mine && ok; ++u) {
        ok = normalise(u);
        // the next tile's z takes the place of an x that the MMAs have read: the
        // previous tile's, waited for above, or, with one z tile, this one's (whose
        // next phase needs the very z that is loaded here)
        if (first && ok && u + 1 < mine && (L::kZt == 2 || mbar_wait(&bars->x_free, u & 1, wc, abort))) load_z(u + 1);
        __syncwarp();
      }
    } else {
      if (first && mine > 1) load_z(1);
      for (int u = 0; u < mine; ++u) {  // no warp leaves the loop early: they meet at its barrier
        ok = ok && normalise(u);
        fence_proxy_async_smem();
        __syncwarp();
        named_bar_sync(1, 128);  // every row of the tile is in TMEM
        if (first && ok && u + 2 < mine) load_z(u + 2);
      }
    }
  } else if (warp >= 8 && warp < 12) {
    // ------------------------------------------------------------ out
    regs_inc<kTfRegsOut>();
    const int quarter = warp & 3;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    uint8_t* const stg = s_stg + quarter * 2048;
    for (int u = 0; u < mine; ++u) {
      const long long row = (static_cast<long long>(pair) + static_cast<long long>(u) * pairs) * 256 + rank * 128 +
                            quarter * 32 + lane;
      const bool in = row < p.M;
      const float mk = p.mask != nullptr && in ? bf16lo_to_f32(p.mask[row]) : 1.f;
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->out_full, u & 1, wc, abort))) break;
      tc_fence_after();
      // up to 128 features of the row out of TMEM before any of them is stored:
      // the next tile's first out MMA waits for the last
      constexpr int kPart = C < 128 ? C : 128;
#pragma unroll
      for (int c0 = 0; c0 < C; c0 += kPart) {
        uint32_t w[kPart / 2];
#pragma unroll
        for (int c = 0; c < kPart; c += 32) {
          if (c0 + c < C) {
            uint32_t v[32];
            tmem_ld32_wait(tmem + lane_addr + kOut + c0 + c, v);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 o = fmul2(make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])),
                                     make_float2(mk, mk));
              w[c / 2 + e] = pack_bf16x2(o.x, o.y);
            }
          }
        }
        if (c0 + kPart >= C) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(&bars->out_free, 0);
        }
        // 32 features at a time through the warp's staging buffer (64-byte
        // swizzled rows) and out by TMA, which leaves out rows past the end
#pragma unroll
        for (int c = 0; c < kPart / 32; ++c) {
          if (c0 + 32 * c < C) {
            if (lane == 0) bulk_wait_read();  // the store before has read the buffer
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t o[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) o[e] = mk == 0.f ? 0u : w[16 * c + 4 * j + e];  // left out: 0, even if NaN
              *reinterpret_cast<uint4*>(stg + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
                  make_uint4(o[0], o[1], o[2], o[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && in) tma_store_3d(&tm_out, stg, c0 + 32 * c, static_cast<int>(row), 0);  // the first row
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  } else if (warp >= 12) {
    // ------------------------------------------------------------ activation
    regs_inc<kTfRegsAct>();
    const int idx = warp - 12, st = idx >> 3, hf = (idx >> 2) & 1, quarter = warp & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t ab = lanes + kAB + kABStage * st + 32 * hf, hcol = lanes + kH + 32 * st + 16 * hf;
    for (long long g = st; g < total; g += 2) {
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->ab_full[st], (g >> 1) & 1, wc, abort))) break;
      tc_fence_after();
      // in two halves: all 64 values at once leave the registers no room for
      // the arithmetic of one to overlap that of the next (175 against 165 us)
      uint32_t h[16];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t a[16], b[16];
        tmem_ld16x2_wait(ab + 16 * j, a, ab + 64 + 16 * j, b);
        if (j == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(&bars->ab_free[st], 0);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 v = gate_fwd2<ACT>(make_float2(__uint_as_float(a[2 * e]), __uint_as_float(a[2 * e + 1])),
                                          make_float2(__uint_as_float(b[2 * e]), __uint_as_float(b[2 * e + 1])));
          h[8 * j + e] = pack_bf16x2(v.x, v.y);
        }
      }
      // the out MMAs of the chunk before last have read this stage's h
      if (g >= 2 &&
          !__all_sync(0xffffffffu, mbar_wait(&bars->h_free[st], static_cast<uint32_t>((g >> 1) - 1) & 1, wc, abort)))
        break;
      tc_fence_after();
      tmem_st16(hcol, h);
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&bars->h_full[st], 0);
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

template <int C, int ACT>
cudaError_t tf_launch(const CUtensorMap& tz, const CUtensorMap& to, const CUtensorMap& twi, const CUtensorMap& two,
                      TfParams p, int grid, cudaStream_t s) {
  p.slots = std::min(p.chunks, TfSmem<C>::kFit);
  const int bytes = TfSmem<C>::bytes(p.slots);
  const cudaError_t e =
      tf_allow(transition_fwd_kernel<C, ACT>, TfSmem<C>::bytes(TfSmem<C>::kFit), kTfThreads / 128, kTfRegsSum);
  if (e != cudaSuccess) return e;
  transition_fwd_kernel<C, ACT><<<grid, kTfThreads, bytes, s>>>(tz, to, twi, two, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_transition_fwd(long long M, int C, int H, int act, const void* z, const void* mask,
                                  const float* ln_w, const float* ln_b, const void* w_in, const void* w_o, void* out,
                                  const WaitCtl& wc, cudaStream_t s) {
  CUtensorMap tz, to, twi, two;
  const cuuint64_t m = static_cast<cuuint64_t>(M), c = static_cast<cuuint64_t>(C), h = static_cast<cuuint64_t>(H);
  const cuuint64_t zd[3] = {c, m, 1}, zs[2] = {2 * c, 2 * c * m};
  const cuuint64_t wd[3] = {h, 2, c}, ws[2] = {2 * h, 4 * h};  // the a and b columns apart: past H reads 0
  const cuuint64_t od[3] = {c, h, 1}, os[2] = {2 * c, 2 * c * h};
  if (!tf_map(&tz, z, zd, zs, 128, 1) || !tf_map32(&to, out, zd, zs) ||
      !tf_map(&twi, w_in, wd, ws, 1, static_cast<cuuint32_t>(C)) || !tf_map(&two, w_o, od, os, 64, 1))
    return cudaErrorInvalidValue;
  TfParams p;
  std::memset(&p, 0, sizeof(p));
  p.M = M;
  p.chunks = (H + 63) / 64;
  p.tiles = static_cast<int>((M + 255) / 256);
  p.mask = static_cast<const uint16_t*>(mask);
  p.ln_w = ln_w;
  p.ln_b = ln_b;
  p.wc = wc;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int grid = 2 * std::min(p.tiles, std::max(sms / 2, 1));
  return by_act(act, [&](auto ic) {
    constexpr int A = decltype(ic)::value;
    switch (C) {
      case 32: return tf_launch<32, A>(tz, to, twi, two, p, grid, s);
      case 64: return tf_launch<64, A>(tz, to, twi, two, p, grid, s);
      case 96: return tf_launch<96, A>(tz, to, twi, two, p, grid, s);
      case 128: return tf_launch<128, A>(tz, to, twi, two, p, grid, s);
      case 160: return tf_launch<160, A>(tz, to, twi, two, p, grid, s);
      case 192: return tf_launch<192, A>(tz, to, twi, two, p, grid, s);
      case 224: return tf_launch<224, A>(tz, to, twi, two, p, grid, s);
      case 256: return tf_launch<256, A>(tz, to, twi, two, p, grid, s);
    }
    return cudaErrorInvalidValue;
  });
}

}  // namespace triattn
