// The transition's forward in one kernel: LayerNorm, both input projections,
// activation and product, output projection and row mask; z is read once and
// out written once, x, a, b and h stay on the chip.
//
// A pair of CTAs (cluster of two, tcgen05 cta_group::2) takes tiles of 256
// rows, 128 per CTA.  With cta_group::2 each CTA holds one half of the N
// columns of every B operand, so the pair's shared memory holds all weights
// and they are loaded once per pair, not once per tile: CTA 0 keeps W_a and
// columns [0, C/2) of W_o, CTA 1 W_b and columns [C/2, C) (192 KB each at
// C = 128, H = 512; one CTA alone could not hold them, and streaming them for
// every 128 rows would take 54 bytes per clock and SM from L2).
//
// Per tile and 64-wide hidden chunk i (K = C, then K = 64):
//   [a | b] = x [W_a | W_b] chunk      M = 256, N = 128, A = x in TMEM
//   h = act(a) b                       registers, BF16 back into TMEM
//   out += h W_o chunk                 M = 256, N = C, A = h in TMEM
// x, out, two stages of h and two of [a | b] fill the 512 TMEM columns at
// C = 128.  A stage of [a | b] is free for the next chunk but one as soon as
// the activation has read it, whatever becomes of its h.
//
// Warps: 0 loads the weights; 1 and 22 (of CTA 0) issue the MMAs of both CTAs,
// one the input projections, one the output projection: a wait costs an
// issuer some 200 clocks even when the phase is complete, and the tensor
// cores' queue is shorter than that (one issuer for both kept them busy for
// 60% of the time); 2-5 normalise the next tile's rows (thread = row) and
// drain out; 6-21 the activation, eight warps per stage, so that a chunk's
// arithmetic may take the time of two chunks' MMAs.
#include <algorithm>
#include <cstring>

#include "kernels.cuh"
#include "transition.cuh"

namespace triattn {
namespace {

constexpr int kTfWarps = 23;
constexpr int kTfThreads = kTfWarps * 32;
constexpr int kTfMaxChunks = 32;
constexpr int kTfBarBytes = 2048;  // barriers (under 1 KB), ln_w and ln_b (1 KB)
constexpr int kTfSmemMax = 232448;

struct TfBars {
  uint64_t w_load[kTfMaxChunks];   // a chunk's weights are in this CTA (TMA bytes)
  uint64_t w_ready[kTfMaxChunks];  // ... in both CTAs (CTA 0)
  uint64_t z_full;                 // z tile in shared memory (TMA bytes)
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
  int H, chunks, tiles;
  const uint16_t* mask;
  const float *ln_w, *ln_b;
  WaitCtl wc;
};

template <int C>
struct TfSmem {
  static constexpr int kZBoxes = (C + 63) / 64;
  static constexpr int kZ = kZBoxes * 16384;
  static constexpr int kWin = C * 128;   // one chunk: C rows (K) of 64 columns
  static constexpr int kWo = 64 * 128;   // one chunk: 64 rows (K) of 64 columns, C / 2 of them used
  static constexpr int bytes(int chunks) { return chunks * (kWin + kWo) + kZ + kTfBarBytes + 1024; }  // + alignment
};

template <int C, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTfThreads, 1)
    transition_fwd_kernel(const __grid_constant__ CUtensorMap tm_z, const __grid_constant__ CUtensorMap tm_out,
                          const __grid_constant__ CUtensorMap tm_win, const __grid_constant__ CUtensorMap tm_wo,
                          const TfParams p) {
  using L = TfSmem<C>;
  constexpr uint32_t kX = 0, kOut = 64, kH = 192, kAB = 256;  // TMEM columns; two stages of h (32) and [a | b] (128)
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* const s_win = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const s_wo = s_win + p.chunks * L::kWin;
  uint8_t* const s_z = s_wo + p.chunks * L::kWo;
  TfBars* const bars = reinterpret_cast<TfBars*>(s_z + L::kZ);
  float* const s_gam = reinterpret_cast<float*>(s_z + L::kZ + 1024);
  float* const s_bet = s_gam + C;
  volatile int* abort = &bars->abort;
  const WaitCtl& wc = p.wc;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int mine = p.tiles > pair ? (p.tiles - 1 - pair) / pairs + 1 : 0;  // tiles of this pair
  const long long total = static_cast<long long>(mine) * p.chunks;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.chunks; ++i) {
      mbar_init(&bars->w_load[i], 1);
      mbar_init(&bars->w_ready[i], 2);
    }
    mbar_init(&bars->z_full, 1);
    mbar_init(&bars->x_full, 8);
    mbar_init(&bars->x_free, 1);
    for (int i = 0; i < 2; ++i) {
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

  if (warp == 0) {
    // ------------------------------------------------------------ weights
    if (lane == 0) {
      for (int i = 0; i < p.chunks; ++i) {
        mbar_expect_tx(&bars->w_load[i], L::kWin + L::kWo);
        tma_load_3d(s_win + i * L::kWin, &tm_win, &bars->w_load[i], 64 * i, static_cast<int>(rank), 0);
        tma_load_3d(s_wo + i * L::kWo, &tm_wo, &bars->w_load[i], static_cast<int>(rank) * (C / 2), 64 * i, 0);
      }
      for (int i = 0; i < p.chunks; ++i) {
        if (!mbar_wait(&bars->w_load[i], 0, wc, abort)) break;
        mbar_arrive_cta(&bars->w_ready[i], 0);
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
      int t = 0, i = 0;
      for (long long g = 0; g < total; ++g) {
        const uint32_t st = static_cast<uint32_t>(g & 1);
        if (g >= 2) wait(&bars->ab_free[st], static_cast<uint32_t>((g >> 1) - 1) & 1);
        if (i == 0) wait(&bars->x_full, t & 1);
        if (t == 0) wait(&bars->w_ready[i], 0);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t w = d_win + i * (L::kWin / 16);
#pragma unroll
          for (int k = 0; k < C / 16; ++k)
            mma_ts_pair(tmem + kAB + 128 * st, tmem + kX + 8 * k, w + k * (2048 / 16), id_ab, k > 0 ? 1u : 0u);
          mma_commit_pair(&bars->ab_full[st]);
          if (i == p.chunks - 1) mma_commit_pair(&bars->x_free);
        }
        __syncwarp();
        if (++i == p.chunks) {
          i = 0;
          ++t;
        }
      }
    }
  } else if (warp == kTfWarps - 1) {
    // ------------------------------------------------------------ MMA issuer: out
    if (rank == 0) {
      constexpr uint32_t id_out = idesc_bf16_f32(256, C, 0, 1);
      const uint64_t d_wo = smem_desc(smem_u32(s_wo), 64 * 128, 1024, 2);
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity, wc, abort));
      };
      int t = 0, i = 0;
      for (long long g = 0; g < total; ++g) {
        const uint32_t st = static_cast<uint32_t>(g & 1);
        if (t == 0) wait(&bars->w_ready[i], 0);
        if (i == 0 && t > 0) wait(&bars->out_free, (t - 1) & 1);
        wait(&bars->h_full[st], (g >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t w = d_wo + i * (L::kWo / 16);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ts_pair(tmem + kOut, tmem + kH + 32 * st + 8 * k, w + k * (2048 / 16), id_out,
                        (i > 0 || k > 0) ? 1u : 0u);
          mma_commit_pair(&bars->h_free[st]);
          if (i == p.chunks - 1) mma_commit_pair(&bars->out_full);
        }
        __syncwarp();
        if (++i == p.chunks) {
          i = 0;
          ++t;
        }
      }
    }
  } else if (warp < 6) {
    // ------------------------------------------------------------ rows
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const bool first = warp == 2 && lane == 0;
    auto load_z = [&](int tile) {
      mbar_expect_tx(&bars->z_full, L::kZ);
#pragma unroll
      for (int b = 0; b < L::kZBoxes; ++b)
        tma_load_3d(s_z + b * 16384, &tm_z, &bars->z_full, 64 * b, tile * 256 + static_cast<int>(rank) * 128, 0);
    };
    auto z16 = [&](int c) { return reinterpret_cast<uint4*>(s_z + (c >> 3) * 16384 + sw128(r, c & 7)); };
    // x of local tile u into TMEM once the previous tile's is read: the row's statistics in two passes
    auto normalise = [&](int u) -> bool {
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->z_full, u & 1, wc, abort))) return false;
      float s = 0.f;
#pragma unroll 4
      for (int c = 0; c < C / 8; ++c) {
        const uint4 w = *z16(c);
        s += ((bf16lo_to_f32(w.x) + bf16hi_to_f32(w.x)) + (bf16lo_to_f32(w.y) + bf16hi_to_f32(w.y))) +
             ((bf16lo_to_f32(w.z) + bf16hi_to_f32(w.z)) + (bf16lo_to_f32(w.w) + bf16hi_to_f32(w.w)));
      }
      const float mean = s * (1.f / C);
      float q = 0.f;
#pragma unroll 4
      for (int c = 0; c < C / 8; ++c) {
        const uint4 w = *z16(c);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = bf16lo_to_f32(ws[e]) - mean, b = bf16hi_to_f32(ws[e]) - mean;
          q = fmaf(a, a, fmaf(b, b, q));
        }
      }
      const float rstd = rsqrtf(q * (1.f / C) + 1e-5f);
      if (u > 0 && !__all_sync(0xffffffffu, mbar_wait(&bars->x_free, (u - 1) & 1, wc, abort))) return false;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < C / 8; c += 2) {  // 16 features = 8 columns at a time
        uint32_t x[8];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 w = *z16(c + j);
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
          const float4* gm = reinterpret_cast<const float4*>(s_gam + 8 * (c + j));
          const float4* bt = reinterpret_cast<const float4*>(s_bet + 8 * (c + j));
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float4 g = gm[e], b = bt[e];
            x[4 * j + 2 * e] = pack_bf16x2(fmaf((bf16lo_to_f32(ws[2 * e]) - mean) * rstd, g.x, b.x),
                                           fmaf((bf16hi_to_f32(ws[2 * e]) - mean) * rstd, g.y, b.y));
            x[4 * j + 2 * e + 1] = pack_bf16x2(fmaf((bf16lo_to_f32(ws[2 * e + 1]) - mean) * rstd, g.z, b.z),
                                               fmaf((bf16hi_to_f32(ws[2 * e + 1]) - mean) * rstd, g.w, b.w));
          }
        }
        tmem_st8(tmem + lane_addr + kX + 4 * c, x);
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&bars->x_full, 0);
      return true;
    };
    bool ok = mine > 0;
    if (ok) {
      if (first) load_z(pair);
      ok = normalise(0);
      __syncwarp();
      named_bar_sync(1, 128);  // every row of the z tile is read
      if (first && mine > 1) load_z(pair + pairs);
    }
    for (int u = 0; u < mine; ++u) {
      // next tile's rows before this tile's out: the issuer is never short of x
      if (ok && u + 1 < mine) ok = normalise(u + 1);
      ok = ok && __all_sync(0xffffffffu, mbar_wait(&bars->out_full, u & 1, wc, abort));
      if (ok) {
        tc_fence_after();
        const int tile = pair + u * pairs;
        const long long row = static_cast<long long>(tile) * 256 + rank * 128 + r;
        const float mk = p.mask != nullptr && row < p.M ? bf16lo_to_f32(p.mask[row]) : 1.f;
        // the row's part of the z tile is read: out takes its place
#pragma unroll 1
        for (int c = 0; c < C; c += 32) {
          uint32_t v[32];
          tmem_ld32_wait(tmem + lane_addr + kOut + c, v);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float lo = __uint_as_float(v[8 * j + 2 * e]) * mk, hi = __uint_as_float(v[8 * j + 2 * e + 1]) * mk;
              w[e] = mk == 0.f ? 0u : pack_bf16x2(lo, hi);  // a row left out is 0 even if it held NaN
            }
            *z16(c / 8 + j) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cta(&bars->out_free, 0);
        fence_proxy_async_smem();
      }
      __syncwarp();
      named_bar_sync(1, 128);
      if (first && ok) {
        const int tile = pair + u * pairs;
#pragma unroll
        for (int b = 0; b < L::kZBoxes; ++b)
          tma_store_3d(&tm_out, s_z + b * 16384, 64 * b, tile * 256 + static_cast<int>(rank) * 128, 0);
        bulk_wait_read();
        if (u + 2 < mine) load_z(pair + (u + 2) * pairs);
      }
    }
    if (first) bulk_wait_all();
  } else {
    // ------------------------------------------------------------ activation
    const int idx = warp - 6, st = idx >> 3, hf = (idx >> 2) & 1, quarter = warp & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t ab = lanes + kAB + 128 * st + 32 * hf, hcol = lanes + kH + 32 * st + 16 * hf;
    for (long long g = st; g < total; g += 2) {
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->ab_full[st], (g >> 1) & 1, wc, abort))) break;
      tc_fence_after();
      bool ok = true;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t a[16], b[16], h[8];
        tmem_ld16x2_wait(ab + 16 * j, a, ab + 64 + 16 * j, b);
        if (j == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(&bars->ab_free[st], 0);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          h[e] = pack_bf16x2(act_fwd<ACT>(__uint_as_float(a[2 * e])) * __uint_as_float(b[2 * e]),
                             act_fwd<ACT>(__uint_as_float(a[2 * e + 1])) * __uint_as_float(b[2 * e + 1]));
        if (j == 0 && g >= 2) {  // the out MMAs of the chunk before last have read this stage's h
          ok = __all_sync(0xffffffffu, mbar_wait(&bars->h_free[st], static_cast<uint32_t>((g >> 1) - 1) & 1, wc, abort));
          if (!ok) break;
          tc_fence_after();
        }
        tmem_st8(hcol + 8 * j, h);
      }
      if (!ok) break;
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&bars->h_full[st], 0);
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

template <int C, int ACT>
cudaError_t tf_launch(const CUtensorMap& tz, const CUtensorMap& to, const CUtensorMap& twi, const CUtensorMap& two,
                      const TfParams& p, int grid, cudaStream_t s) {
  const int bytes = TfSmem<C>::bytes(p.chunks);
  const cudaError_t e = cudaFuncSetAttribute(transition_fwd_kernel<C, ACT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  transition_fwd_kernel<C, ACT><<<grid, kTfThreads, bytes, s>>>(tz, to, twi, two, p);
  return cudaGetLastError();
}

int tf_bytes(int C, int chunks) {
  switch (C) {
    case 32: return TfSmem<32>::bytes(chunks);
    case 64: return TfSmem<64>::bytes(chunks);
    case 96: return TfSmem<96>::bytes(chunks);
    case 128: return TfSmem<128>::bytes(chunks);
  }
  return kTfSmemMax + 1;
}

}  // namespace

bool transition_fwd_fused(int C, int H) {
  const int chunks = (H + 63) / 64;
  return chunks <= kTfMaxChunks && tf_bytes(C, chunks) <= kTfSmemMax;
}

cudaError_t launch_transition_fwd(long long M, int C, int H, int act, const void* z, const void* mask,
                                  const float* ln_w, const float* ln_b, const void* w_in, const void* w_o, void* out,
                                  const WaitCtl& wc, cudaStream_t s) {
  CUtensorMap tz, to, twi, two;
  const cuuint64_t m = static_cast<cuuint64_t>(M), c = static_cast<cuuint64_t>(C), h = static_cast<cuuint64_t>(H);
  const cuuint64_t zd[3] = {c, m, 1}, zs[2] = {2 * c, 2 * c * m};
  const cuuint64_t wd[3] = {h, 2, c}, ws[2] = {2 * h, 4 * h};  // the a and b columns apart: past H reads 0
  const cuuint64_t od[3] = {c, h, 1}, os[2] = {2 * c, 2 * c * h};
  if (!tf_map(&tz, z, zd, zs, 128, 1) || !tf_map(&to, out, zd, zs, 128, 1) ||
      !tf_map(&twi, w_in, wd, ws, 1, static_cast<cuuint32_t>(C)) || !tf_map(&two, w_o, od, os, 64, 1))
    return cudaErrorInvalidValue;
  TfParams p;
  std::memset(&p, 0, sizeof(p));
  p.M = M;
  p.H = H;
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
    }
    return cudaErrorInvalidValue;
  });
}

}  // namespace triattn
