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
//
// 768^2 tokens and slices, four heads of 32 features, q and k (0.15 GB each): forward
// 91 us for 0.60 GB, 6.6 TB/s; backward 160 us for 0.91 GB, 5.7 TB/s.  From a
// projection's pair rows of 392 features, whose 512 bytes of q and k touch a fifth more
// sectors: 101 and 179 us.  The backward by copies into shared memory six slices
// ahead (174 and 213 us) and by four pairs a thread (170 and 186) were no faster.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "kernels.cuh"
#include "triattn.h"

namespace triattn {
namespace {

constexpr int kThreads = 256;

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

// The thread's two 16-byte pieces as four pairs of (a, b) values, two pairs to a
// packed operation: a[i] holds the first features of pairs 2 i and 2 i + 1, b[i]
// the second ones.  SPLIT: the pieces are the same place of both halves of the
// row; otherwise they are neighbours and a pair's features too.
template <bool SPLIT>
__device__ __forceinline__ void to_pairs(const uint4& lo, const uint4& hi, float2 (&a)[4], float2 (&b)[4]) {
  const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, h[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (SPLIT) {
      a[i] = make_float2(bf16lo_to_f32(l[i]), bf16hi_to_f32(l[i]));
      b[i] = make_float2(bf16lo_to_f32(h[i]), bf16hi_to_f32(h[i]));
    } else {
      const uint32_t u = i < 2 ? l[(2 * i) & 3] : h[(2 * i) & 3], v = i < 2 ? l[(2 * i + 1) & 3] : h[(2 * i + 1) & 3];
      a[i] = make_float2(bf16lo_to_f32(u), bf16lo_to_f32(v));
      b[i] = make_float2(bf16hi_to_f32(u), bf16hi_to_f32(v));
    }
  }
}
template <bool SPLIT>
__device__ __forceinline__ void from_pairs(const float2 (&a)[4], const float2 (&b)[4], uint4& lo, uint4& hi) {
  uint32_t l[4], h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (SPLIT) {
      l[i] = pack_bf16x2(a[i].x, a[i].y);
      h[i] = pack_bf16x2(b[i].x, b[i].y);
    } else {
      (i < 2 ? l : h)[(2 * i) & 3] = pack_bf16x2(a[i].x, b[i].x);
      (i < 2 ? l : h)[(2 * i + 1) & 3] = pack_bf16x2(a[i].y, b[i].y);
    }
  }
  lo = make_uint4(l[0], l[1], l[2], l[3]);
  hi = make_uint4(h[0], h[1], h[2], h[3]);
}
__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 neg(float2 x) { return make_float2(-x.x, -x.y); }

// cos and sin of position times frequency.  The angle is a whole number of
// 2^-64 turns, so the product wraps to the turn's fraction exactly and a far
// position costs no accuracy (but what the host's FP64 power is off by, times the
// position: 3e-7 for theta of at least 1); its upper 32 bits are half turns times 2^-31.
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
    const int j = (blockIdx.x >> 1) * kRows + threadIdx.x / kPer, part = threadIdx.x % kPer;
    live = j < a.HN;
    row_of(a, live ? j : 0, h, n);
    b = blockIdx.y / a.cpb;
    lo = kSplit ? 8 * part : 16 * part;
    hi = kSplit ? D / 2 + 8 * part : lo + 8;
  }
  __device__ __forceinline__ int pair(int i) const { return (kSplit ? lo : lo / 2) + i; }
  // features of pair i of the thread's eight
  __device__ __forceinline__ int first(int i) const { return kSplit ? lo + i : lo + 2 * i; }
  __device__ __forceinline__ int second(int i) const { return kSplit ? hi + i : lo + 2 * i + 1; }
  __device__ __forceinline__ void weights(const QkArgs& a, const float* w, float2 (&wa)[4], float2 (&wb)[4]) const {
    const float* p = w + (a.w_heads > 1 ? static_cast<size_t>(h) * D : 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      wa[i] = make_float2(__ldg(p + first(2 * i)), __ldg(p + first(2 * i + 1)));
      wb[i] = make_float2(__ldg(p + second(2 * i)), __ldg(p + second(2 * i + 1)));
    }
  }
  __device__ __forceinline__ void turns(const QkArgs& a, float2 (&c)[4], float2 (&s)[4]) const {
    const int p = a.pos != nullptr ? __ldg(a.pos + static_cast<size_t>(b) * a.N + n) : n;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      angle(p, a.freq[pair(2 * i)], c[i].x, s[i].x);
      angle(p, a.freq[pair(2 * i + 1)], c[i].y, s[i].y);
    }
  }
};

// Blocks of q and k alternate, so that both parts of a pair row are read at
// about the same time.
template <int D, int ROT>
__global__ void __launch_bounds__(kThreads, 2) qk_norm_fwd_kernel(const QkArgs a) {
  constexpr int U = 4;  // slices in flight
  using P = Place<D, ROT>;
  const P at(a);
  const int m = blockIdx.x & 1;
  const uint16_t* x = m ? a.x[1] : a.x[0];
  uint16_t* y = m ? a.y[1] : a.y[0];
  // y_a = r (x_a ac - x_b bs),  y_b = r (x_a as + x_b bc): weights and rotation in one
  float2 ac[4], bs[4], as[4], bc[4];
  at.weights(a, m ? a.w[1] : a.w[0], ac, bc);
  if constexpr (ROT != TRIATTN_ROTARY_NONE) {
    float2 c[4], s[4];
    at.turns(a, c, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      as[i] = fmul2(ac[i], s[i]);
      bs[i] = neg(fmul2(bc[i], s[i]));
      ac[i] = fmul2(ac[i], c[i]);
      bc[i] = fmul2(bc[i], c[i]);
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
      float2 xa[4], xb[4], ss = splat(0.f);
      to_pairs<P::kSplit>(lo[k], hi[k], xa, xb);
#pragma unroll
      for (int i = 0; i < 4; ++i) ss = ffma2(xa[i], xa[i], ffma2(xb[i], xb[i], ss));
      const float2 r = splat(rsqrtf(row_sum<D>(ss.x + ss.y) * (1.f / D) + a.eps));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 ra = fmul2(r, xa[i]), rb = fmul2(r, xb[i]);
        xa[i] = ROT != TRIATTN_ROTARY_NONE ? ffma2(ra, ac[i], fmul2(rb, bs[i])) : fmul2(ra, ac[i]);
        xb[i] = ROT != TRIATTN_ROTARY_NONE ? ffma2(ra, as[i], fmul2(rb, bc[i])) : fmul2(rb, bc[i]);
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
  let_next_start();
  const P at(a);
  const int m = blockIdx.x & 1, tile = blockIdx.x >> 1;
  const uint16_t* x = m ? a.x[1] : a.x[0];
  const uint16_t* dy = m ? a.dy[1] : a.dy[0];  // may be dx: read by plain loads, a piece before it is written
  uint16_t* dx = m ? a.y[1] : a.y[0];
  float2 wa[4], wb[4], c[4], s[4], da[4], db[4];
  at.weights(a, m ? a.w[1] : a.w[0], wa, wb);
  if constexpr (ROT != TRIATTN_ROTARY_NONE) at.turns(a, c, s);
#pragma unroll
  for (int i = 0; i < 4; ++i) da[i] = db[i] = splat(0.f);
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
      float2 xa[4], xb[4], ga[4], gb[4], ss = splat(0.f), dot = splat(0.f);
      to_pairs<P::kSplit>(lo[k], hi[k], xa, xb);
      to_pairs<P::kSplit>(gl[k], gh[k], ga, gb);
#pragma unroll
      for (int i = 0; i < 4; ++i) ss = ffma2(xa[i], xa[i], ffma2(xb[i], xb[i], ss));
      const float r = rsqrtf(row_sum<D>(ss.x + ss.y) * (1.f / D) + a.eps);
      const bool live = at.live && o + k < o1;
      const float2 rl = splat(live ? r : 0.f);  // a row that is not there adds nothing to dw
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (ROT != TRIATTN_ROTARY_NONE) {  // back by the angle
          const float2 t = ga[i];
          ga[i] = ffma2(gb[i], s[i], fmul2(t, c[i]));
          gb[i] = ffma2(neg(t), s[i], fmul2(gb[i], c[i]));
        }
        const float2 ua = fmul2(ga[i], xa[i]), ub = fmul2(gb[i], xb[i]);
        da[i] = ffma2(ua, rl, da[i]);
        db[i] = ffma2(ub, rl, db[i]);
        dot = ffma2(ua, wa[i], ffma2(ub, wb[i], dot));
        ga[i] = fmul2(ga[i], wa[i]);
        gb[i] = fmul2(gb[i], wb[i]);
      }
      // dx = r (a - n mean(a n)) = r a - x r^3 mean(a x)
      const float2 f = splat(-(r * r) * (r * (1.f / D) * row_sum<D>(dot.x + dot.y))), rr = splat(r);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        xa[i] = ffma2(xa[i], f, fmul2(ga[i], rr));
        xb[i] = ffma2(xb[i], f, fmul2(gb[i], rr));
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
  // the block's sums by head, rows added in a fixed order: thread (part, slot, feature)
  const int row = threadIdx.x / P::kPer;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sums[row][at.first(2 * i)] = da[i].x;
    sums[row][at.first(2 * i + 1)] = da[i].y;
    sums[row][at.second(2 * i)] = db[i].x;
    sums[row][at.second(2 * i + 1)] = db[i].y;
  }
  __syncthreads();
  const long long j0 = static_cast<long long>(tile) * P::kRows;
  const int last = static_cast<int>(min(static_cast<long long>(P::kRows), a.HN - j0));
  const int cells = a.slots * D, np = max(1, kThreads / cells);
  float* out = a.part + ((static_cast<size_t>(m) * gridDim.y + blockIdx.y) * (gridDim.x >> 1) + tile) * cells;
  for (int e = threadIdx.x; e < np * cells; e += np > 1 ? np * cells : kThreads) {
    const int part = e / cells, cell = e - part * cells, sl = cell / D, d = cell - sl * D;
    // rows of the slot: every H-th (heads in a row), or those of one head in sequence
    int first, end, step;
    if (a.w_heads == 1) {  // all of them
      first = 0;
      end = last;
      step = 1;
    } else if (a.lx.hn) {
      first = a.slots == a.H ? static_cast<int>((sl + a.H - j0 % a.H) % a.H) : sl;
      end = last;
      step = a.H;
    } else {
      const long long h0 = (j0 / a.N + sl) * a.N - j0;
      first = static_cast<int>(max(0ll, h0));
      end = static_cast<int>(min(static_cast<long long>(last), h0 + a.N));
      step = 1;
    }
    float v = 0.f;
    for (int rr = first + part * step; rr < end; rr += np * step) v += sums[rr][d];
    if (np > 1) parts[e] = v;
    else out[cell] = v;
  }
  if (np > 1) {
    __syncthreads();
    if (threadIdx.x < cells) {
      float v = 0.f;
      for (int p = 0; p < np; ++p) v += parts[p * cells + threadIdx.x];
      out[threadIdx.x] = v;
    }
  }
}

// dw[h][d] (or dw[d], all heads) from the blocks' partial sums, in a fixed order.
// Partials [chunks][tiles][slots][D]: a slot is all of a tile where the heads share a
// weight (2 x 131 tokens of six heads: 11 -> 2 us); with the heads in a row it is a head
// (the j0 + slot-th where a tile does not hold all of them), otherwise the
// slot-th head of the tile.
__global__ void __launch_bounds__(1024) qk_norm_dw_kernel(const float* part, float* dwq, float* dwk, int D, int rows,
                                                          int tiles, int chunks, int slots, int H, int N, int w_heads,
                                                          int hn) {
  __shared__ float2 sh[1024];
  after_previous();
  const int d = threadIdx.x % D, lane = threadIdx.x / D, lanes = 1024 / D;
  const float* p = part + static_cast<size_t>(blockIdx.y) * chunks * tiles * slots * D + d;
  const int h = blockIdx.x;
  Sum2 v;
  if (w_heads == 1) {  // everything
    const int n = chunks * tiles * slots;
#pragma unroll 4
    for (int e = lane; e < n; e += lanes) v.add(p[static_cast<size_t>(e) * D]);
  } else {
    const int t0 = hn ? 0 : static_cast<int>(static_cast<long long>(h) * N / rows);
    const int nt = (hn ? tiles : static_cast<int>(((h + 1ll) * N - 1) / rows) + 1) - t0;
#pragma unroll 4
    for (int e = lane; e < nt * chunks; e += lanes) {
      const int ch = e / nt, t = t0 + e - ch * nt;
      int sl = h;
      if (!hn) sl = h - static_cast<int>(static_cast<long long>(t) * rows / N);
      else if (slots < H) sl = static_cast<int>((h + H - static_cast<long long>(t) * rows % H) % H);
      if (sl < slots) v.add(p[((static_cast<size_t>(ch) * tiles + t) * slots + sl) * D]);
    }
  }
  sh[threadIdx.x] = v.pair();
  for (int o = lanes / 2; o > 0; o /= 2) {
    __syncthreads();
    if (lane < o) {
      v.add(sh[threadIdx.x + o * D]);
      sh[threadIdx.x] = v.pair();
    }
  }
  if (lane == 0) (blockIdx.y ? dwk : dwq)[static_cast<size_t>(h) * D + d] = v.value();
}

struct Plan {
  int rows, tiles, cpb, per, chunks, slots;
  size_t part_bytes;
};

// Blocks: a tile of rows of a slice times a run of slices.  Of one to six waves of
// what the GPU holds at once (two blocks an SM) the one with the shortest run of
// a SM's blocks, where what a block does before and after its slices takes as
// long as `extra` of them.
Plan plan_of(const triattn_qk_norm_shape* s, bool hn, int extra) {
  Plan p;
  p.rows = kThreads / (s->D / 16);
  const long long HN = static_cast<long long>(s->H) * s->N;
  p.tiles = static_cast<int>((HN + p.rows - 1) / p.rows);
  const long long base = 2ll * p.tiles * s->B, slots = 152 * 2;
  long long best = 1, least = -1;
  for (int w = 1; w <= 6; ++w) {
    const long long cpb = std::max(1ll, std::min<long long>({slots * w / base, s->N_o, 65535ll / s->B}));
    const long long per = (s->N_o + cpb - 1) / cpb, blocks = base * ((s->N_o + per - 1) / per);
    const long long time = (blocks + slots - 1) / slots * (per + extra);
    if (least < 0 || time < least) {
      best = cpb;
      least = time;
    }
  }
  p.per = static_cast<int>((s->N_o + best - 1) / best);
  p.cpb = (s->N_o + p.per - 1) / p.per;
  p.chunks = p.cpb * s->B;
  p.slots = s->w_heads == 1 ? 1
            : hn ? std::min(s->H, p.rows)
                 : static_cast<int>(std::min<long long>(s->H, (p.rows - 1) / s->N + 2));
  p.part_bytes = 2ull * p.chunks * p.tiles * p.slots * s->D * 4;
  return p;
}
Plan fwd_plan(const triattn_qk_norm_shape* s, bool hn) { return plan_of(s, hn, 3); }
Plan bwd_plan(const triattn_qk_norm_shape* s, bool hn) { return plan_of(s, hn, 8); }

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
  return (std::max(bwd_plan(shape, true).part_bytes, bwd_plan(shape, false).part_bytes) + 255) /
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
  if (q_out == k_out || q_out == q || q_out == k || k_out == q || k_out == k) return TRIATTN_ERR_INVALID_ARG;
  const Plan p = fwd_plan(shape, lx.hn != 0);
  QkArgs a = args_of(shape, p, lx, ly, w_q, w_k, positions);
  a.x[0] = static_cast<const uint16_t*>(q);
  a.x[1] = static_cast<const uint16_t*>(k);
  a.y[0] = static_cast<uint16_t*>(q_out);
  a.y[1] = static_cast<uint16_t*>(k_out);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(2 * p.tiles, p.chunks);
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
  auto same = [](const RowLayout& a, const RowLayout& b) {
    return a.slice == b.slice && a.head == b.head && a.row == b.row;
  };
  if (dq == dk || d_w_q == d_w_k || dq == q || dq == k || dk == q || dk == k || dq == d_k_out || dk == d_q_out ||
      ((dq == d_q_out || dk == d_k_out) && !same(ldy, ly)))
    return TRIATTN_ERR_INVALID_ARG;
  const Plan p = bwd_plan(shape, lx.hn != 0);
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
  const dim3 grid(2 * p.tiles, p.chunks);
  cudaError_t e = trace_call(kKQkBwd, s, [&] { return dispatch(shape, a, grid, true, s); });
  if (e == cudaSuccess)
    e = trace_call(kKQkDw, s, [&] {
      return launch_after(false, qk_norm_dw_kernel, dim3(shape->w_heads, 2), 1024, 0, s, a.part, d_w_q, d_w_k, shape->D,
                          p.rows, p.tiles, p.chunks, p.slots, shape->H, shape->N, shape->w_heads, lx.hn);
    });
  return e == cudaSuccess ? TRIATTN_OK : TRIATTN_ERR_CUDA;
}

}  // extern "C"
