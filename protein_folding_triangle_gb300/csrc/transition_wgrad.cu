// The transition's weight gradients, dW_in = x^T [da | db] and dW_o = h^T g, over
// all rows, with h, da and db computed again from x and g instead of read from
// memory: 6 H bytes per row less to write, read and keep (1.8 GB at 768 x 768
// rows, H = 512) for as many products again as the gradients themselves take.
//
// A CTA owns one 64-wide slice of the hidden features, keeps that slice's
// weights in shared memory and its part of both gradients in TMEM, and walks
// its share of the row tiles (128 rows of x and g by TMA, two stages):
//
//   [a | b] = x [W_a | W_b] slice     M = 128 rows,     N = 128, K = C
//   dh      = g W_o^T slice           M = 128 rows,     N = 64,  K = C
//   h, da, db                         registers, then BF16 tiles in shared memory
//   dW_in^T += x^T [da | db]          M = 128 features, N = 128, K = 128 rows
//   dW_o^T  += g^T h                  M = 128 features, N = 64,  K = 128 rows
//
// The same shared-memory tiles of x and g are the row-major A operand of the
// first two and the feature-major one of the last two.  The groups of CTAs
// that share the rows out leave one FP32 partial of the gradients each, added
// in a fixed order by transition_sum_kernel (transition.cu).  TMEM: [a | b | dh]
// 192 columns, the gradients 192.
//
// What bounds it is shared memory: per row tile and slice the MMAs read 208 KB of
// operands, the loads write 64 KB and the activation 48 KB.  0.422 ms at 768 x 768
// rows, C = 128, H = 512, 95 bytes per clock, the tensor pipe active for 46 % of
// it (0.24 ms of products).  With the hardware tanh in the gates it was 0.403 ms,
// without the activation 0.397 ms, without that and the loads 0.326 ms.  Row tiles
// brought to L2 ahead change nothing.
// With C <= 64 x and g share the A operand of the gradients and four stages
// fit: 0.098 ms at 640 x 640 rows, C = 64, H = 256 (0.143 ms without both).
// Eight activation warps instead of sixteen: 0.43 ms (0.403 then).
//
// Warps: 0 loads, 1 issues the first two products, 2 the last two, 4-19 the
// activation (warp = 32 rows x 16 features) and, at the end, the partials.
#include <algorithm>
#include <cstring>

#include "kernels.cuh"
#include "transition.cuh"

namespace triattn {
namespace {

constexpr int kTwThreads = 20 * 32;
constexpr int kTwSmemMax = 232448;
constexpr int kTwMaxStages = 4;

struct TwBars {
  uint64_t w_full;                 // the slice's weights (TMA bytes)
  uint64_t xg_full[kTwMaxStages], xg_free[kTwMaxStages];  // a row tile (TMA bytes) / read by its last MMA
  uint64_t abd_full, abd_free;     // [a | b | dh] complete / read
  uint64_t hd_full, hd_free;       // h, da, db tiles written / read
  uint32_t tmem_slot;
  int abort;
};

struct TwParams {
  int H, slices, groups, tiles;
  float* part;  // [groups] of dW_in [C, 2H], dW_o [H, C]
  WaitCtl wc;
};

template <int C>
struct TwSmem {
  static constexpr int kKb = (C + 63) / 64;   // 64-wide blocks of a row
  static constexpr bool kBoth = kKb == 1;     // x and g in one A operand of the gradients
  static constexpr int kWin = C * 128;        // W_a or W_b: C rows (K) of 64 columns
  static constexpr int kWo = kKb * 64 * 128;  // W_o: 64 hidden rows (N) of C columns (K)
  static constexpr int kRows = kKb * 16384;   // a tile of 128 rows of x or g
  static constexpr int kHid = 16384;          // 128 rows of 64 hidden features
  static constexpr int kStages = C <= 64 ? 4 : 2;
  static constexpr int kTiles = 2 * kWin + kWo;
  static constexpr int kDa = kTiles + 2 * kStages * kRows;
  static constexpr int kBar = kDa + 3 * kHid;
  static constexpr int kBytes = kBar + 1024 + 1024;  // + alignment
  static_assert(kBytes <= kTwSmemMax, "shared memory");
};

template <int C, int ACT>
__global__ void __launch_bounds__(kTwThreads, 1)
    transition_wgrad_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_g,
                            const __grid_constant__ CUtensorMap tm_win, const __grid_constant__ CUtensorMap tm_wo,
                            const TwParams p) {
  using L = TwSmem<C>;
  constexpr uint32_t kABD = 0, kDin = 192, kDo = 320;  // TMEM columns
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* const sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const s_wo = sm + 2 * L::kWin;
  uint8_t* const s_x = sm + L::kTiles;  // stage st: x at 2 st kRows, g behind it
  uint8_t* const s_da = sm + L::kDa;    // da, db, h
  TwBars* const bars = reinterpret_cast<TwBars*>(sm + L::kBar);
  volatile int* abort = &bars->abort;
  const WaitCtl& wc = p.wc;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slice = blockIdx.x % p.slices, group = blockIdx.x / p.slices;
  const int mine = (p.tiles - 1 - group) / p.groups + 1;  // row tiles group, group + groups, ...

  if (threadIdx.x == 0) {
    mbar_init(&bars->w_full, 1);
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(&bars->xg_full[i], 1);
      mbar_init(&bars->xg_free[i], 1);
    }
    mbar_init(&bars->abd_full, 1);
    mbar_init(&bars->abd_free, 16);
    mbar_init(&bars->hd_full, 16);
    mbar_init(&bars->hd_free, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&bars->tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      mbar_expect_tx(&bars->w_full, 2 * L::kWin + L::kWo);
      tma_load_3d(sm, &tm_win, &bars->w_full, 64 * slice, 0, 0);
      tma_load_3d(sm + L::kWin, &tm_win, &bars->w_full, 64 * slice, 1, 0);
#pragma unroll
      for (int b = 0; b < L::kKb; ++b) tma_load_3d(s_wo + b * 8192, &tm_wo, &bars->w_full, 64 * b, 64 * slice, 0);
      for (int k = 0; k < mine; ++k) {
        const int st = k % L::kStages;
        if (!mbar_wait(&bars->xg_free[st], (k / L::kStages & 1) ^ 1, wc, abort)) break;
        const int row = (group + k * p.groups) * 128;
        uint8_t* const x = s_x + 2 * st * L::kRows;
        mbar_expect_tx(&bars->xg_full[st], 2 * L::kRows);
#pragma unroll
        for (int b = 0; b < L::kKb; ++b) {
          tma_load_3d(x + b * 16384, &tm_x, &bars->xg_full[st], 64 * b, row, 0);
          tma_load_3d(x + L::kRows + b * 16384, &tm_g, &bars->xg_full[st], 64 * b, row, 0);
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer: [a | b], dh
    constexpr uint32_t id_ab = idesc_bf16_f32(128, 128, 0, 1);  // A: K contiguous; B: N contiguous
    constexpr uint32_t id_dh = idesc_bf16_f32(128, 64, 0, 0);
    const uint64_t d_win = smem_desc(smem_u32(sm), L::kWin, 1024, 2);  // an offset of n bytes adds n / 16
    const uint64_t d_wo = smem_desc(smem_u32(s_wo), 16, 1024, 2);
    bool ok = __all_sync(0xffffffffu, mbar_wait(&bars->w_full, 0, wc, abort));
    for (int k = 0; k < mine && ok; ++k) {
      const int st = k % L::kStages;
      ok = __all_sync(0xffffffffu, mbar_wait(&bars->xg_full[st], k / L::kStages & 1, wc, abort));
      if (k > 0) ok = ok && __all_sync(0xffffffffu, mbar_wait(&bars->abd_free, (k - 1) & 1, wc, abort));
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t x = smem_desc(smem_u32(s_x + 2 * st * L::kRows), 16, 1024, 2);
#pragma unroll
        for (int i = 0; i < C / 16; ++i)
          mma_ss(tmem + kABD, x + ((i >> 2) * 16384 + (i & 3) * 32) / 16, d_win + i * (2048 / 16), id_ab, i > 0 ? 1u : 0u);
#pragma unroll
        for (int i = 0; i < C / 16; ++i)
          mma_ss(tmem + kABD + 128, x + (L::kRows + (i >> 2) * 16384 + (i & 3) * 32) / 16,
                 d_wo + ((i >> 2) * 8192 + (i & 3) * 32) / 16, id_dh, i > 0 ? 1u : 0u);
        mma_commit(&bars->abd_full);
      }
      __syncwarp();
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ MMA issuer: the gradients
    // A: features contiguous, two blocks of 64: those of x, then those of g;
    // with one block each (C <= 64), x and g side by side over [da | db | h],
    // whose h against x and da, db against g are not used
    constexpr uint32_t id_in = idesc_bf16_f32(128, L::kBoth ? 192 : 128, 1, 1), id_o = idesc_bf16_f32(128, 64, 1, 1);
    const uint64_t d_dab = smem_desc(smem_u32(s_da), L::kHid, 1024, 2);
    const uint64_t d_h = smem_desc(smem_u32(s_da + 2 * L::kHid), L::kHid, 1024, 2);
    bool ok = true;
    for (int k = 0; k < mine; ++k) {
      const int st = k % L::kStages;
      ok = __all_sync(0xffffffffu, mbar_wait(&bars->hd_full, k & 1, wc, abort));
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t x = smem_desc(smem_u32(s_x + 2 * st * L::kRows), 16384, 1024, 2);
#pragma unroll
        for (int i = 0; i < 8; ++i)  // 16 rows each
          mma_ss(tmem + kDin, x + i * (2048 / 16), d_dab + i * (2048 / 16), id_in, (k > 0 || i > 0) ? 1u : 0u);
        if constexpr (!L::kBoth) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            mma_ss(tmem + kDo, x + (L::kRows + i * 2048) / 16, d_h + i * (2048 / 16), id_o, (k > 0 || i > 0) ? 1u : 0u);
        }
        mma_commit(&bars->hd_free);
        mma_commit(&bars->xg_free[st]);
      }
      __syncwarp();
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ activation
    const int quarter = warp & 3, hq = (warp - 4) >> 2, r = quarter * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    bool ok = true;
    for (int k = 0; k < mine; ++k) {
      ok = __all_sync(0xffffffffu, mbar_wait(&bars->abd_full, k & 1, wc, abort));
      if (!ok) break;
      tc_fence_after();
      uint32_t a[16], b[16], d[16], h[8], da[8], db[8];
      tmem_ld16x3_wait(lanes + kABD + 16 * hq, a, lanes + kABD + 64 + 16 * hq, b, lanes + kABD + 128 + 16 * hq, d);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->abd_free);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float2 hv, av, bv;
        gate_bwd2<ACT>(make_float2(__uint_as_float(a[2 * e]), __uint_as_float(a[2 * e + 1])),
                       make_float2(__uint_as_float(b[2 * e]), __uint_as_float(b[2 * e + 1])),
                       make_float2(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1])), hv, av, bv);
        h[e] = pack_bf16x2(hv.x, hv.y);
        da[e] = pack_bf16x2(av.x, av.y);
        db[e] = pack_bf16x2(bv.x, bv.y);
      }
      // the previous tile's MMAs have read the buffers
      if (k > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bars->hd_free, (k - 1) & 1, wc, abort));
      if (!ok) break;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint8_t* const at = s_da + sw128(r, 2 * hq + c);
        *reinterpret_cast<uint4*>(at) = make_uint4(da[4 * c], da[4 * c + 1], da[4 * c + 2], da[4 * c + 3]);
        *reinterpret_cast<uint4*>(at + L::kHid) = make_uint4(db[4 * c], db[4 * c + 1], db[4 * c + 2], db[4 * c + 3]);
        *reinterpret_cast<uint4*>(at + 2 * L::kHid) = make_uint4(h[4 * c], h[4 * c + 1], h[4 * c + 2], h[4 * c + 3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->hd_full);
    }
    // the gradients are complete with the last tile's MMAs; TMEM lane = feature
    ok = ok && __all_sync(0xffffffffu, mbar_wait(&bars->hd_free, (mine - 1) & 1, wc, abort));
    if (ok) {
      tc_fence_after();
      const size_t H = static_cast<size_t>(p.H);
      float* const part = p.part + static_cast<size_t>(group) * 3 * C * H;
      uint32_t v[32];
      tmem_ld32_wait(lanes + kDin + 32 * hq, v);  // da (hq 0, 1) or db
      int hid = 64 * slice + 32 * (hq & 1);
      if (r < C && hid < p.H) {
        float4* dst = reinterpret_cast<float4*>(part + (r * 2 + (hq >> 1)) * H + hid);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          dst[c] = make_float4(__uint_as_float(v[4 * c]), __uint_as_float(v[4 * c + 1]), __uint_as_float(v[4 * c + 2]),
                               __uint_as_float(v[4 * c + 3]));
      }
      uint32_t w[16];
      tmem_ld16_wait(lanes + kDo + 16 * hq, w);
      hid = 64 * slice + 16 * hq;
      const int f = L::kBoth ? r - 64 : r;
      if (f >= 0 && f < C && hid < p.H) {
        float* dst = part + 2 * C * H + static_cast<size_t>(hid) * C + f;
#pragma unroll
        for (int c = 0; c < 16; ++c) dst[c * C] = __uint_as_float(w[c]);
      }
    }
  }

  settle_if_aborted(abort);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int C, int ACT>
cudaError_t tw_launch(const CUtensorMap& tx, const CUtensorMap& tg, const CUtensorMap& ti, const CUtensorMap& to,
                      const TwParams& p, cudaStream_t s) {
  const cudaError_t e = tf_allow(transition_wgrad_kernel<C, ACT>, TwSmem<C>::kBytes);
  if (e != cudaSuccess) return e;
  transition_wgrad_kernel<C, ACT><<<p.slices * p.groups, kTwThreads, TwSmem<C>::kBytes, s>>>(tx, tg, ti, to, p);
  return cudaGetLastError();
}

// Row groups: as many as give every SM one CTA (152 SMs: the order of the sums
// is the same on any device), never more than row tiles.
int tw_groups(long long M, int H) {
  const int slices = (H + 63) / 64;
  const long long tiles = (M + 127) / 128;
  return static_cast<int>(std::min<long long>(std::max(152 / slices, 1), tiles));
}

}  // namespace

size_t transition_wgrad_bytes(long long M, int C, int H) {
  return static_cast<size_t>(tw_groups(M, H)) * 3 * C * H * sizeof(float);
}

cudaError_t launch_transition_wgrad(long long M, int C, int H, int act, const void* x, const void* g, const void* w_in,
                                    const void* w_o, float* part, int* parts, const WaitCtl& wc, cudaStream_t s) {
  CUtensorMap tx, tg, ti, to;
  const cuuint64_t c = static_cast<cuuint64_t>(C), hh = static_cast<cuuint64_t>(H), m = static_cast<cuuint64_t>(M);
  const cuuint64_t zd[3] = {c, m, 1}, zs[2] = {2 * c, 2 * c * m};
  const cuuint64_t wd[3] = {hh, 2, c}, ws[2] = {2 * hh, 4 * hh};  // the a and b columns apart: past H reads 0
  const cuuint64_t od[3] = {c, hh, 1}, os[2] = {2 * c, 2 * c * hh};
  if (!tf_map(&tx, x, zd, zs, 128, 1) || !tf_map(&tg, g, zd, zs, 128, 1) ||
      !tf_map(&ti, w_in, wd, ws, 1, static_cast<cuuint32_t>(C)) || !tf_map(&to, w_o, od, os, 64, 1))
    return cudaErrorInvalidValue;
  TwParams p;
  std::memset(&p, 0, sizeof(p));
  p.H = H;
  p.slices = (H + 63) / 64;
  p.groups = tw_groups(M, H);
  p.tiles = static_cast<int>((M + 127) / 128);
  p.part = part;
  *parts = p.groups;
  p.wc = wc;
  return by_act(act, [&](auto ic) {
    constexpr int A = decltype(ic)::value;
    switch (C) {
      case 32: return tw_launch<32, A>(tx, tg, ti, to, p, s);
      case 64: return tw_launch<64, A>(tx, tg, ti, to, p, s);
      case 96: return tw_launch<96, A>(tx, tg, ti, to, p, s);
      case 128: return tw_launch<128, A>(tx, tg, ti, to, p, s);
    }
    return cudaErrorInvalidValue;
  });
}

}  // namespace triattn
