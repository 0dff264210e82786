// The transition's forward for a few rows, where latency counts: products of
// one to four rows with the weights, on the FP32 units.
//
// A cluster of eight CTAs takes up to R rows.  Each CTA computes x for itself,
// its eighth of the hidden features and what they add to the rows' outputs; the
// eight parts are added through distributed shared memory, in ascending order.
// Within a CTA a thread takes four neighbouring columns of a weight matrix (8
// bytes) and every G-th of its rows, with 16 loads under way before the first
// product, W_in's even before the LayerNorm.  x, h and the parts stay FP32:
// only out is rounded.
//
// What bounds it is latency: a launch, the loads of z and of the weights, and
// the exchange.  5.2 us per call for one row at C = 128, H = 512, 6.1 to 6.5 for 2 to
// 48 (a CTA per SM) in a captured graph, where the tile kernel takes 13.  One to four
// rows at a time: the weights' loads are shared, and four sums per column stay in
// registers.
#include "kernels.cuh"
#include "transition.cuh"

namespace triattn {
namespace {

constexpr int kRwThreads = 256, kRwCtas = 8, kRwLoads = 16;
constexpr int kRwMaxSlice = 4096 / kRwCtas;  // hidden features of a CTA

struct RwParams {
  int M, C, H, act;
  const uint16_t *z, *mask;
  const float *ln_w, *ln_b;
  const uint16_t *w_in, *w_o;
  uint16_t* out;
};

__device__ __forceinline__ float rw_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ float rw_act(float a, int act) {
  // GELU as a sigmoid too: 1 + tanh(u) would leave nothing of a closed gate
  const float v = act == TRIATTN_ACT_GELU ? a * fmaf(a * a, 0.0713548163f, 1.5957691216f) : a;
  const float s = 1.f / (1.f + __expf(-v));
  return act == TRIATTN_ACT_SIGMOID ? s : a * s;
}

template <int R>
__global__ void __cluster_dims__(kRwCtas, 1, 1) __launch_bounds__(kRwThreads)
    transition_rows_kernel(const RwParams p) {
  __shared__ float s_x[R][256];
  __shared__ float4 s_part[R][kRwThreads];
  __shared__ float s_h[R][kRwMaxSlice];
  __shared__ float s_out[R][256];
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int row0 = static_cast<int>(blockIdx.x) / kRwCtas * R;
  const int hs = p.H / kRwCtas, j0 = rank * hs;  // hs: a multiple of 4

  // four columns of W (row stride ld, from `at`), rows g, g + G, ... below n;
  // two calls per product: loads(0) early, then the rest
  uint2 w[kRwLoads];
  auto loads = [&](const uint16_t* at, size_t ld, int g, int G, int n) {
#pragma unroll
    for (int k = 0; k < kRwLoads; ++k)
      w[k] = g + k * G < n ? __ldg(reinterpret_cast<const uint2*>(at + (g + k * G) * ld)) : make_uint2(0u, 0u);
  };
  // s_part[r][t] = sum over the thread's rows of v[r][row] * (its four columns)
  auto product = [&](const uint16_t* at, size_t ld, int g, int G, int n, const float* v, int vld) {
    float4 acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = g; i < n; i += kRwLoads * G) {
      if (i != g) loads(at, ld, i, G, n);
#pragma unroll
      for (int k = 0; k < kRwLoads; ++k) {
        const int c = i + k * G;
        if (c >= n) break;
        const float2 lo = bf16x2_to_f32x2(w[k].x), hi = bf16x2_to_f32x2(w[k].y);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float f = v[r * vld + c];
          acc[r].x = fmaf(f, lo.x, acc[r].x);
          acc[r].y = fmaf(f, lo.y, acc[r].y);
          acc[r].z = fmaf(f, hi.x, acc[r].z);
          acc[r].w = fmaf(f, hi.y, acc[r].w);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) s_part[r][t] = acc[r];
  };
  // column c of the product's row r: the sum over the G threads that share it
  auto column = [&](int r, int c, int items, int G) {
    const float* at = reinterpret_cast<const float*>(&s_part[r][0]) + c;
    float s = 0.f;
    for (int g = 0; g < G; ++g) s += at[g * items * 4];
    return s;
  };

  // [a | b]: columns j0 .. j0 + hs of each half
  const int in_items = hs / 2, in_g = min(kRwThreads / in_items, 32), gi = t / in_items, ii = t % in_items;
  const uint16_t* const in_at = p.w_in + (ii < hs / 4 ? 0 : p.H - hs) + j0 + 4 * ii;
  if (gi < in_g) loads(in_at, 2 * static_cast<size_t>(p.H), gi, in_g, p.C);

  if (warp < R) {  // x of row row0 + warp
    const int row = row0 + warp;
    const bool live = row < p.M && (p.mask == nullptr || (p.mask[row] & 0x7FFFu) != 0);
    float v[8], s = 0.f, q = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = lane + 32 * k;
      v[k] = live && c < p.C ? bf16lo_to_f32(p.z[static_cast<size_t>(row) * p.C + c]) : 0.f;
      s += v[k];
    }
    const float mean = rw_sum(s) / p.C;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = lane + 32 * k < p.C ? v[k] - mean : 0.f;
      q = fmaf(d, d, q);
    }
    const float rstd = rsqrtf(rw_sum(q) / p.C + 1e-5f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = lane + 32 * k;
      if (c < p.C) s_x[warp][c] = live ? fmaf((v[k] - mean) * rstd, p.ln_w[c], p.ln_b[c]) : 0.f;
    }
  }
  __syncthreads();
  if (gi < in_g) product(in_at, 2 * static_cast<size_t>(p.H), gi, in_g, p.C, &s_x[0][0], 256);
  const int o_items = p.C / 4, o_g = kRwThreads / o_items, go = t / o_items, io = t % o_items;
  const uint16_t* const o_at = p.w_o + static_cast<size_t>(j0) * p.C + 4 * io;
  if (go < o_g) loads(o_at, p.C, go, o_g, hs);
  __syncthreads();
  for (int e = t; e < R * hs; e += kRwThreads) {
    const int r = e / hs, j = e - r * hs;
    s_h[r][j] = rw_act(column(r, j, in_items, in_g), p.act) * column(r, hs + j, in_items, in_g);
  }
  __syncthreads();
  if (go < o_g) product(o_at, p.C, go, o_g, hs, &s_h[0][0], kRwMaxSlice);
  __syncthreads();
  for (int e = t; e < R * p.C; e += kRwThreads) {
    const int r = e / p.C, c = e - r * p.C;
    s_out[r][c] = column(r, c, o_items, o_g);
  }
  cluster_sync();
  // this CTA's eighth of the outputs, two neighbours per thread
  for (int e = 2 * (rank * kRwThreads + t); e < R * p.C; e += 2 * kRwCtas * kRwThreads) {
    const int r = e / p.C, c = e - r * p.C, row = row0 + r;
    if (row >= p.M) break;
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kRwCtas; ++k) s = fadd2(s, ld_cluster_f32x2(&s_out[r][c], k));
    const float mk = p.mask == nullptr ? 1.f : bf16lo_to_f32(p.mask[row]);
    *reinterpret_cast<uint32_t*>(p.out + static_cast<size_t>(row) * p.C + c) =
        mk != 0.f ? pack_bf16x2(s.x * mk, s.y * mk) : 0u;
  }
  cluster_sync();  // no CTA leaves while its part is read
}

}  // namespace

cudaError_t launch_transition_rows(int M, int C, int H, int act, const void* z, const void* mask, const float* ln_w,
                                   const float* ln_b, const void* w_in, const void* w_o, void* out, cudaStream_t s) {
  const RwParams p = {M, C, H, act, static_cast<const uint16_t*>(z), static_cast<const uint16_t*>(mask), ln_w, ln_b,
                      static_cast<const uint16_t*>(w_in), static_cast<const uint16_t*>(w_o),
                      static_cast<uint16_t*>(out)};
  if (M == 1) transition_rows_kernel<1><<<kRwCtas, kRwThreads, 0, s>>>(p);
  else transition_rows_kernel<4><<<(M + 3) / 4 * kRwCtas, kRwThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace triattn
