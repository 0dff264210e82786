// Norms of queries and keys for each head with the position rotation, in front
// of the attention core: for every row x (D features) of q and of k,
//
//   r = 1 / sqrt(mean_d x^2 + eps),  n = r x,  u = n * w[h],
//   y = R(t) u:  the pair (a, b) of frequency i turned by t_i = pos theta^(-2 i / D)
//
// and backwards  g = R(-t) dy,  dw[h] = sum of g * n,  dx = r (a - n mean_d(a n)),
// a = g * w.  Nothing is kept from the forward: r is computed again from x.
//
// Both passes only move bytes (about 20 operations an element against 4 to 6
// bytes): a thread holds eight pairs of a row, both of its 16-byte pieces, so
// that the rotation needs no exchange and a row of 32 features one shuffle.
// The row's token and head stay with the thread while it walks over the outer
// slices: cos, sin and the weights are computed once and stay in registers, and
// the weight gradients are sums in registers until the end.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "kernels.cuh"
#include "triattn.h"

namespace triattn {
namespace {

constexpr int kThreads = 256;
constexpr int kPairs = 8;  // pairs of features per thread

struct QkArgs {
  const uint16_t* x[2];   // q, k
  const uint16_t* dy[2];  // gradients of the outputs (backward)
  uint16_t* y[2];         // outputs, or dq, dk
  const float* w[2];
  const int* pos;         // [B, N] or null: the token's index
  float* part;            // backward: [2][chunks][tiles][slots][D]
  RowLayout lx, ldy, ly;
  long long HN;           // rows of a slice
  int N_o, N, H, w_heads;
  int per, cpb;           // slices per block, blocks per example along the outer axis
  int slots;
  float eps;
  unsigned long long freq[16];  // theta^(-2 i / D) / (2 pi) in units of 2^-64 turns
};

// Row j of a slice, in the order of the memory of x: heads side by side in a
// token's row (hn) or tokens side by side in a head.
__device__ __forceinline__ void row_of(const QkArgs& a, int j, int& h, int& n) {
  if (a.lx.hn) {
    n = j / a.H;
    h = j - n * a.H;
  } else {
    h = j / a.N;
    n = j - h * a.N;
  }
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16lo_to_f32(w[i]);
    f[2 * i + 1] = bf16hi_to_f32(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// The thread's two 16-byte pieces as pairs (a, b): the same place of both
// halves of the row (HALF), or neighbours.
template <bool SPLIT>
__device__ __forceinline__ void to_pairs(const uint4& lo, const uint4& hi, float (&a)[kPairs], float (&b)[kPairs]) {
  float f0[8], f1[8];
  unpack8(lo, f0);
  unpack8(hi, f1);
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    a[i] = SPLIT ? f0[i] : (i < 4 ? f0[(2 * i) & 7] : f1[(2 * i) & 7]);
    b[i] = SPLIT ? f1[i] : (i < 4 ? f0[(2 * i + 1) & 7] : f1[(2 * i + 1) & 7]);
  }
}
template <bool SPLIT>
__device__ __forceinline__ void from_pairs(const float (&a)[kPairs], const float (&b)[kPairs], uint4& lo, uint4& hi) {
  float f0[8], f1[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f0[i] = SPLIT ? a[i] : ((i & 1) ? b[i / 2] : a[i / 2]);
    f1[i] = SPLIT ? b[i] : ((i & 1) ? b[4 + i / 2] : a[4 + i / 2]);
  }
  lo = pack8(f0);
  hi = pack8(f1);
}

// cos and sin of position times frequency.  The angle is a whole number of
// 2^-64 turns, so the product wraps to the turn's fraction exactly and a far
// position costs no accuracy; its upper 32 bits are half turns times 2^-31.
__device__ __forceinline__ void angle(int pos, unsigned long long freq, float& c, float& s) {
  const long long t = static_cast<long long>(static_cast<unsigned long long>(static_cast<long long>(pos)) * freq);
  sincospif(static_cast<float>(static_cast<int>(t >> 32)) * 0x1p-31f, &s, &c);
}

template <int D>
__device__ __forceinline__ float row_sum(float v) {
  return D == 32 ? v + __shfl_xor_sync(0xffffffffu, v, 1) : v;
}

template <int D, int ROT>
struct Place {
  static constexpr bool kSplit = ROT == TRIATTN_ROTARY_HALF;
  static constexpr int kPer = D / 16;             // threads per row
  static constexpr int kRows = kThreads / kPer;   // rows per block
  int h, n, b, lo, hi;                            // head, token, example, elements of the two pieces
  bool live;
  __device__ __forceinline__ Place(const QkArgs& a) {
    const int j = blockIdx.x * kRows + threadIdx.x / kPer, part = threadIdx.x % kPer;
    live = j < a.HN;
    row_of(a, live ? j : 0, h, n);
    b = blockIdx.y / a.cpb;
    lo = kSplit ? 8 * part : 16 * part;
    hi = kSplit ? D / 2 + 8 * part : lo + 8;
  }
  __device__ __forceinline__ int pair(int i) const { return (kSplit ? lo : lo / 2) + i; }
  __device__ __forceinline__ void weights(const QkArgs& a, const float* w, float (&wa)[kPairs],
                                          float (&wb)[kPairs]) const {
    const float* p = w + (a.w_heads > 1 ? static_cast<size_t>(h) * D : 0);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      wa[i] = __ldg(p + (kSplit ? lo + i : lo + 2 * i));
      wb[i] = __ldg(p + (kSplit ? hi + i : lo + 2 * i + 1));
    }
  }
  __device__ __forceinline__ void turns(const QkArgs& a, float (&c)[kPairs], float (&s)[kPairs]) const {
    const int p = a.pos != nullptr ? __ldg(a.pos + static_cast<size_t>(b) * a.N + n) : n;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) angle(p, a.freq[pair(i)], c[i], s[i]);
  }
};

template <int D, int ROT>
__global__ void __launch_bounds__(kThreads, 2) qk_norm_fwd_kernel(const QkArgs a) {
  constexpr int U = 4;  // slices in flight
  using P = Place<D, ROT>;
  const P at(a);
  const int m = blockIdx.z;
  const uint16_t* x = m ? a.x[1] : a.x[0];
  uint16_t* y = m ? a.y[1] : a.y[0];
  // y_a = r (x_a ac - x_b bs),  y_b = r (x_a as + x_b bc): weights and rotation in one
  float ac[kPairs], bs[kPairs], as[kPairs], bc[kPairs];
  at.weights(a, m ? a.w[1] : a.w[0], ac, bc);
  if constexpr (ROT != TRIATTN_ROTARY_NONE) {
    float c[kPairs], s[kPairs];
    at.turns(a, c, s);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      as[i] = ac[i] * s[i];
      bs[i] = bc[i] * s[i];
      ac[i] *= c[i];
      bc[i] *= c[i];
    }
  }
  const int o0 = (blockIdx.y % a.cpb) * a.per, o1 = min(o0 + a.per, a.N_o);
  const long long xs = at.h * a.lx.head + at.n * a.lx.row, ys = at.h * a.ly.head + at.n * a.ly.row;
  for (int o = o0; o < o1; o += U) {
    uint4 lo[U], hi[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const uint16_t* p = x + (static_cast<long long>(at.b) * a.N_o + min(o + k, o1 - 1)) * a.lx.slice + xs;
      lo[k] = __ldg(reinterpret_cast<const uint4*>(p + at.lo));
      hi[k] = __ldg(reinterpret_cast<const uint4*>(p + at.hi));
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      float xa[kPairs], xb[kPairs], ss = 0.f;
      to_pairs<P::kSplit>(lo[k], hi[k], xa, xb);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) ss += xa[i] * xa[i] + xb[i] * xb[i];
      const float r = rsqrtf(row_sum<D>(ss) * (1.f / D) + a.eps);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float ra = r * xa[i], rb = r * xb[i];
        xa[i] = ROT != TRIATTN_ROTARY_NONE ? ra * ac[i] - rb * bs[i] : ra * ac[i];
        xb[i] = ROT != TRIATTN_ROTARY_NONE ? ra * as[i] + rb * bc[i] : rb * bc[i];
      }
      if (at.live && o + k < o1) {
        uint16_t* p = y + (static_cast<long long>(at.b) * a.N_o + o + k) * a.ly.slice + ys;
        uint4 l, g;
        from_pairs<P::kSplit>(xa, xb, l, g);
        *reinterpret_cast<uint4*>(p + at.lo) = l;
        *reinterpret_cast<uint4*>(p + at.hi) = g;
      }
    }
  }
}

template <int D, int ROT>
__global__ void __launch_bounds__(kThreads, 2) qk_norm_bwd_kernel(const QkArgs a) {
  constexpr int U = 2;  // slices in flight
  using P = Place<D, ROT>;
  __shared__ float sums[P::kRows][D + 1];
  __shared__ float parts[kThreads];
  const P at(a);
  const int m = blockIdx.z;
  const uint16_t* x = m ? a.x[1] : a.x[0];
  const uint16_t* dy = m ? a.dy[1] : a.dy[0];  // may be dx: read by plain loads, a piece before it is written
  uint16_t* dx = m ? a.y[1] : a.y[0];
  float wa[kPairs], wb[kPairs], c[kPairs], s[kPairs], da[kPairs], db[kPairs];
  at.weights(a, m ? a.w[1] : a.w[0], wa, wb);
  if constexpr (ROT != TRIATTN_ROTARY_NONE) at.turns(a, c, s);
#pragma unroll
  for (int i = 0; i < kPairs; ++i) da[i] = db[i] = 0.f;
  const int o0 = (blockIdx.y % a.cpb) * a.per, o1 = min(o0 + a.per, a.N_o);
  const long long xs = at.h * a.lx.head + at.n * a.lx.row, gs = at.h * a.ldy.head + at.n * a.ldy.row,
                  ys = at.h * a.ly.head + at.n * a.ly.row;
  for (int o = o0; o < o1; o += U) {
    uint4 lo[U], hi[U], gl[U], gh[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const long long bo = static_cast<long long>(at.b) * a.N_o + min(o + k, o1 - 1);
      const uint16_t* p = x + bo * a.lx.slice + xs;
      const uint16_t* q = dy + bo * a.ldy.slice + gs;
      lo[k] = __ldg(reinterpret_cast<const uint4*>(p + at.lo));
      hi[k] = __ldg(reinterpret_cast<const uint4*>(p + at.hi));
      gl[k] = *reinterpret_cast<const uint4*>(q + at.lo);
      gh[k] = *reinterpret_cast<const uint4*>(q + at.hi);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      float xa[kPairs], xb[kPairs], ga[kPairs], gb[kPairs], ss = 0.f, dot = 0.f;
      to_pairs<P::kSplit>(lo[k], hi[k], xa, xb);
      to_pairs<P::kSplit>(gl[k], gh[k], ga, gb);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) ss += xa[i] * xa[i] + xb[i] * xb[i];
      const float r = rsqrtf(row_sum<D>(ss) * (1.f / D) + a.eps);
      const bool live = at.live && o + k < o1;
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        if constexpr (ROT != TRIATTN_ROTARY_NONE) {  // back by the angle
          const float t = ga[i];
          ga[i] = t * c[i] + gb[i] * s[i];
          gb[i] = gb[i] * c[i] - t * s[i];
        }
        xa[i] *= r;  // n
        xb[i] *= r;
        if (live) {
          da[i] += ga[i] * xa[i];
          db[i] += gb[i] * xb[i];
        }
        ga[i] *= wa[i];
        gb[i] *= wb[i];
        dot += ga[i] * xa[i] + gb[i] * xb[i];
      }
      dot = row_sum<D>(dot) * (1.f / D);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        xa[i] = r * (ga[i] - xa[i] * dot);
        xb[i] = r * (gb[i] - xb[i] * dot);
      }
      if (live) {
        uint16_t* p = dx + (static_cast<long long>(at.b) * a.N_o + o + k) * a.ly.slice + ys;
        uint4 l, g;
        from_pairs<P::kSplit>(xa, xb, l, g);
        *reinterpret_cast<uint4*>(p + at.lo) = l;
        *reinterpret_cast<uint4*>(p + at.hi) = g;
      }
    }
  }
  // the block's sums by head, rows added in a fixed order
  const int row = threadIdx.x / P::kPer;
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    sums[row][P::kSplit ? at.lo + i : at.lo + 2 * i] = da[i];
    sums[row][P::kSplit ? at.hi + i : at.lo + 2 * i + 1] = db[i];
  }
  const int j0 = blockIdx.x * P::kRows, last = static_cast<int>(min(static_cast<long long>(P::kRows), a.HN - j0));
  const int d = threadIdx.x % D, part = threadIdx.x / D;
  constexpr int kParts = kThreads / D;
  float* out = a.part + ((static_cast<size_t>(m) * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x) * a.slots * D;
  for (int sl = 0; sl < a.slots; ++sl) {
    // rows of the slot: every H-th (heads in a row), or those of one head in sequence
    int first, end, step;
    if (a.lx.hn) {
      first = sl;
      end = last;
      step = a.H;
    } else {
      const int head = j0 / a.N + sl;
      first = static_cast<int>(max(0ll, static_cast<long long>(head) * a.N - j0));
      end = static_cast<int>(min(static_cast<long long>(last), (head + 1ll) * a.N - j0));
      step = 1;
    }
    __syncthreads();
    float v = 0.f;
    for (int rr = first + part * step; rr < end; rr += kParts * step) v += sums[rr][d];
    parts[threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x < D) {
      v = 0.f;
#pragma unroll
      for (int p = 0; p < kParts; ++p) v += parts[p * D + threadIdx.x];
      out[sl * D + threadIdx.x] = v;
    }
  }
}

// dw[h][d] (or dw[d], all heads) from the blocks' partial sums, in a fixed order.
__global__ void __launch_bounds__(1024) qk_norm_dw_kernel(const float* __restrict__ part, float* __restrict__ dwq,
                                                          float* __restrict__ dwk, int D, int rows, int tiles,
                                                          int chunks, int slots, int H, int N, int w_heads, int hn) {
  __shared__ double sh[1024];
  const int d = threadIdx.x % D, lane = threadIdx.x / D, lanes = 1024 / D;
  const float* p = part + static_cast<size_t>(blockIdx.y) * chunks * tiles * slots * D;
  const int h0 = w_heads > 1 ? blockIdx.x : 0, h1 = w_heads > 1 ? h0 + 1 : H;
  double v = 0.0;
  for (int h = h0; h < h1; ++h) {
    const int t0 = hn ? 0 : static_cast<int>(static_cast<long long>(h) * N / rows);
    const int t1 = hn ? tiles : static_cast<int>(((h + 1ll) * N - 1) / rows) + 1;
    const int nt = t1 - t0;
    for (int e = lane; e < nt * chunks; e += lanes) {
      const int t = t0 + e % nt, ch = e / nt;
      const long long j0 = static_cast<long long>(t) * rows;
      const int sl = hn ? static_cast<int>((h + H - j0 % H) % H) : h - static_cast<int>(j0 / N);
      if (sl < slots) v += p[((static_cast<size_t>(ch) * tiles + t) * slots + sl) * D + d];
    }
  }
  sh[threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.x < D) {
    v = 0.0;
    for (int l = 0; l < lanes; ++l) v += sh[l * D + threadIdx.x];
    (blockIdx.y ? dwk : dwq)[static_cast<size_t>(blockIdx.x) * D + threadIdx.x] = static_cast<float>(v);
  }
}

struct Plan {
  int rows, tiles, cpb, per, chunks, slots;
  size_t part_bytes;
};

// Blocks: a tile of rows of a slice times a run of slices, about `waves` times
// what the GPU holds at once (two blocks an SM).
Plan plan_of(const triattn_qk_norm_shape* s, bool hn, int waves) {
  Plan p;
  p.rows = kThreads / (s->D / 16);
  const long long HN = static_cast<long long>(s->H) * s->N;
  p.tiles = static_cast<int>((HN + p.rows - 1) / p.rows);
  const long long base = 2ll * p.tiles * s->B, want = 152ll * 2 * waves;
  long long cpb = std::max(1ll, std::min<long long>(want / base, s->N_o));
  cpb = std::min(cpb, 65535ll / s->B);
  p.per = static_cast<int>((s->N_o + cpb - 1) / cpb);
  p.cpb = (s->N_o + p.per - 1) / p.per;
  p.chunks = p.cpb * s->B;
  p.slots = hn ? std::min(s->H, p.rows) : static_cast<int>(std::min<long long>(s->H, (p.rows - 1) / s->N + 2));
  p.part_bytes = 2ull * p.chunks * p.tiles * p.slots * s->D * 4;
  return p;
}
constexpr int kFwdWaves = 4, kBwdWaves = 2;

triattn_status check(const triattn_qk_norm_shape* s, triattn_shape* core) {
  if (s == nullptr || s->B < 1 || s->N_o < 1 || s->N < 1 || s->H < 1 || s->D < 1 || s->flags != 0)
    return TRIATTN_ERR_INVALID_ARG;
  if (s->w_heads != 1 && s->w_heads != s->H) return TRIATTN_ERR_INVALID_ARG;
  if (s->rotary < TRIATTN_ROTARY_NONE || s->rotary > TRIATTN_ROTARY_INTERLEAVED) return TRIATTN_ERR_INVALID_ARG;
  if (!(s->eps > 0.f) || !std::isfinite(s->eps) || !(s->theta > 0.0) || !std::isfinite(s->theta))
    return TRIATTN_ERR_INVALID_ARG;
  if (s->D != 16 && s->D != 32) return TRIATTN_ERR_UNSUPPORTED;
  if (s->B > 65535 || static_cast<long long>(s->B) * s->N_o >= (1ll << 31) ||
      static_cast<long long>(s->H) * s->N >= (1ll << 30))
    return TRIATTN_ERR_UNSUPPORTED;
  *core = triattn_shape{s->B, s->N_o, s->N, s->H, s->D, 0u};
  return TRIATTN_OK;
}

bool al(const void* p, uintptr_t a) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

QkArgs args_of(const triattn_qk_norm_shape* s, const Plan& p, const RowLayout& lx, const RowLayout& ly,
               const float* w_q, const float* w_k, const int* positions) {
  QkArgs a{};
  a.w[0] = w_q;
  a.w[1] = w_k;
  a.pos = positions;
  a.lx = lx;
  a.ly = ly;
  a.HN = static_cast<long long>(s->H) * s->N;
  a.N_o = s->N_o;
  a.N = s->N;
  a.H = s->H;
  a.w_heads = s->w_heads;
  a.per = p.per;
  a.cpb = p.cpb;
  a.slots = p.slots;
  a.eps = s->eps;
  if (s->rotary != TRIATTN_ROTARY_NONE)
    for (int i = 0; i < s->D / 2; ++i) {
      // turns per position; whole turns change nothing (theta below 1)
      double t = std::pow(s->theta, -2.0 * i / s->D) / 6.283185307179586476925;
      t -= std::floor(t);
      a.freq[i] = static_cast<unsigned long long>(std::ldexp(t, 63)) << 1;
    }
  return a;
}

template <int D, int ROT>
cudaError_t launch(const QkArgs& a, dim3 grid, bool bwd, cudaStream_t s) {
  if (bwd) qk_norm_bwd_kernel<D, ROT><<<grid, kThreads, 0, s>>>(a);
  else qk_norm_fwd_kernel<D, ROT><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}
cudaError_t dispatch(const triattn_qk_norm_shape* sh, const QkArgs& a, dim3 grid, bool bwd, cudaStream_t s) {
  const bool d32 = sh->D == 32;
  switch (sh->rotary) {
    case TRIATTN_ROTARY_HALF:
      return d32 ? launch<32, TRIATTN_ROTARY_HALF>(a, grid, bwd, s) : launch<16, TRIATTN_ROTARY_HALF>(a, grid, bwd, s);
    case TRIATTN_ROTARY_INTERLEAVED:
      return d32 ? launch<32, TRIATTN_ROTARY_INTERLEAVED>(a, grid, bwd, s)
                 : launch<16, TRIATTN_ROTARY_INTERLEAVED>(a, grid, bwd, s);
    default:
      return d32 ? launch<32, TRIATTN_ROTARY_NONE>(a, grid, bwd, s) : launch<16, TRIATTN_ROTARY_NONE>(a, grid, bwd, s);
  }
}

}  // namespace
}  // namespace triattn

using namespace triattn;

extern "C" {

size_t triattn_qk_norm_workspace_bytes(const triattn_qk_norm_shape* shape) {
  triattn_shape core;
  if (check(shape, &core) != TRIATTN_OK) return 0;
  // the larger of the two orders of rows
  return (std::max(plan_of(shape, true, kBwdWaves).part_bytes, plan_of(shape, false, kBwdWaves).part_bytes) + 255) /
         256 * 256;
}

triattn_status triattn_qk_norm_fwd(const triattn_qk_norm_shape* shape, const void* q, const void* k,
                                   const triattn_layout* in_layout, const float* w_q, const float* w_k,
                                   const int* positions, void* q_out, void* k_out, const triattn_layout* out_layout,
                                   void* stream) {
  triattn_shape core;
  triattn_status st = check(shape, &core);
  if (st != TRIATTN_OK) return st;
  RowLayout lx, ly;
  if (!row_layout_from(in_layout, &core, &lx) || !row_layout_from(out_layout, &core, &ly))
    return TRIATTN_ERR_INVALID_ARG;
  for (const void* p : {q, k, static_cast<const void*>(q_out), static_cast<const void*>(k_out)})
    if (!al(p, 16)) return TRIATTN_ERR_INVALID_ARG;
  if (!al(w_q, 4) || !al(w_k, 4) || (positions != nullptr && !al(positions, 4))) return TRIATTN_ERR_INVALID_ARG;
  const Plan p = plan_of(shape, lx.hn != 0, kFwdWaves);
  QkArgs a = args_of(shape, p, lx, ly, w_q, w_k, positions);
  a.x[0] = static_cast<const uint16_t*>(q);
  a.x[1] = static_cast<const uint16_t*>(k);
  a.y[0] = static_cast<uint16_t*>(q_out);
  a.y[1] = static_cast<uint16_t*>(k_out);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(p.tiles, p.chunks, 2);
  return trace_call(kKQkFwd, s, [&] { return dispatch(shape, a, grid, false, s); }) == cudaSuccess ? TRIATTN_OK
                                                                                                    : TRIATTN_ERR_CUDA;
}

triattn_status triattn_qk_norm_bwd(const triattn_qk_norm_shape* shape, const void* q, const void* k,
                                   const triattn_layout* in_layout, const float* w_q, const float* w_k,
                                   const int* positions, const void* d_q_out, const void* d_k_out,
                                   const triattn_layout* d_out_layout, void* dq, void* dk,
                                   const triattn_layout* grad_layout, float* d_w_q, float* d_w_k, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  triattn_shape core;
  triattn_status st = check(shape, &core);
  if (st != TRIATTN_OK) return st;
  RowLayout lx, ldy, ly;
  if (!row_layout_from(in_layout, &core, &lx) || !row_layout_from(d_out_layout, &core, &ldy) ||
      !row_layout_from(grad_layout, &core, &ly))
    return TRIATTN_ERR_INVALID_ARG;
  for (const void* p : {q, k, d_q_out, d_k_out, static_cast<const void*>(dq), static_cast<const void*>(dk)})
    if (!al(p, 16)) return TRIATTN_ERR_INVALID_ARG;
  for (const void* p : {w_q, w_k, static_cast<const float*>(d_w_q), static_cast<const float*>(d_w_k)})
    if (!al(p, 4)) return TRIATTN_ERR_INVALID_ARG;
  if (positions != nullptr && !al(positions, 4)) return TRIATTN_ERR_INVALID_ARG;
  if (!al(workspace, 256) || workspace_bytes < triattn_qk_norm_workspace_bytes(shape)) return TRIATTN_ERR_WORKSPACE;
  const Plan p = plan_of(shape, lx.hn != 0, kBwdWaves);
  QkArgs a = args_of(shape, p, lx, ly, w_q, w_k, positions);
  a.ldy = ldy;
  a.x[0] = static_cast<const uint16_t*>(q);
  a.x[1] = static_cast<const uint16_t*>(k);
  a.dy[0] = static_cast<const uint16_t*>(d_q_out);
  a.dy[1] = static_cast<const uint16_t*>(d_k_out);
  a.y[0] = static_cast<uint16_t*>(dq);
  a.y[1] = static_cast<uint16_t*>(dk);
  a.part = static_cast<float*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(p.tiles, p.chunks, 2);
  cudaError_t e = trace_call(kKQkBwd, s, [&] { return dispatch(shape, a, grid, true, s); });
  if (e == cudaSuccess)
    e = trace_call(kKQkDw, s, [&] {
      qk_norm_dw_kernel<<<dim3(shape->w_heads, 2), 1024, 0, s>>>(a.part, d_w_q, d_w_k, shape->D, p.rows, p.tiles,
                                                                p.chunks, p.slots, shape->H, shape->N, shape->w_heads,
                                                                lx.hn);
      return cudaGetLastError();
    });
  return e == cudaSuccess ? TRIATTN_OK : TRIATTN_ERR_CUDA;
}

}  // extern "C"
