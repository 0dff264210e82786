// Orthogonalising a list of updates by Newton-Schulz products: for every matrix
// G, with X = G / (|G|_F + eps) of m <= n (the transposed of a tall matrix),
// `steps` times
//
//   A = X X^T,  B = b A + c A^2,  X <- a X + B X,
//
// which takes every singular value s to s (a + b s^2 + c s^4) and leaves the
// singular vectors.
//
// The products run on the tensor cores as products of FP16 pairs: a value x is
// held as hi + lo, hi = fp16(2^8 x), lo = fp16(2^8 x - hi), 22 bits, and a product
// is hi hi + hi lo + lo hi in one FP32 accumulator.  Single BF16 operands, as
// such updates are often computed, are off by 3 % of the result after five steps
// and by 80 % where a matrix has few directions (what rounding adds beside them
// is multiplied by a, 3.4, in every step); pairs of BF16 by up to 8e-4, pairs of
// FP16 by no more than FP32 products (3e-5).  The scale keeps both halves of the
// small values out of FP16's subnormals; the largest value is 255.
//
// With A' = c A + b I and B' = A' A + a I, a step is three plain products:
//   1  A = X X^T (and A' from the accumulator),  2  B' = A' A,  3  X <- B' X.
// Operands are kept in the workspace as the shared-memory image of their tiles,
// 128 rows x 64 columns with the 128-byte swizzle, hi then lo (32 KB), zero past
// the matrix: one untiled bulk copy loads a tile, for a K-major operand as for an
// MN-major one, and no tensor maps are needed for a list of any matrices.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

#include "kernels.cuh"
#include "orthogonalize.cuh"
#include "triattn.h"

namespace triattn {
namespace {

constexpr int kUpload = 256;
struct OrthTable {
  OrthMat mat[kUpload];
  int n;
};
static_assert(sizeof(OrthTable) + 32 <= 32764, "kernel parameter limit");

__global__ void __launch_bounds__(256) orth_table_kernel(const __grid_constant__ OrthTable t, OrthMat* to) {
  if (threadIdx.x < t.n) to[threadIdx.x] = t.mat[threadIdx.x];
}

// The matrix that item `at` belongs to (the last whose first item is not above it), by a whole warp.
template <int OrthMat::* FIRST>
__device__ __forceinline__ int find(const OrthView& v, int at) {
  int lo = 0, n = v.n;  // it is one of [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32, i = static_cast<int>(threadIdx.x & 31) * step;
    const uint32_t below = __ballot_sync(0xffffffffu, i < n && v.mat[lo + i].*FIRST <= at);
    const int part = 31 - __clz(below);
    lo += part * step;
    n = min(step, n - part * step);
  }
  return lo;
}

__device__ __forceinline__ float element(const OrthMat& q, long long at) {
  return (q.flags & kOrthFp32) ? __ldg(static_cast<const float*>(q.src) + at)
                           : bf16lo_to_f32(__ldg(static_cast<const uint16_t*>(q.src) + at));
}

// Sums of squares, one partial per run of rows of the source.
__global__ void __launch_bounds__(256) orth_norm_kernel(OrthView v) {
  __shared__ float sh[8];
  const int k = find<&OrthMat::part0>(v, blockIdx.x);
  const OrthMat q = v.mat[k];
  const int rows = (q.flags & kOrthTall) ? q.n : q.m, cols = (q.flags & kOrthTall) ? q.m : q.n;
  const int r0 = (blockIdx.x - q.part0) * q.part_rows, r1 = min(r0 + q.part_rows, rows);
  float s = 0.f;
  const int e = (r1 - r0) * cols;  // part_rows keeps this small unless a row is long
  for (int i = threadIdx.x; i < e; i += 256) {
    const int r = i / cols;
    const float x = element(q, (r0 + r) * q.ld_src + (i - r * cols));
    s += x * x;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.f;
    for (int w = 0; w < 8; ++w) s += sh[w];
    v.part[blockIdx.x] = s;
  }
}

// One tile of X per block: normed, scaled, split, in the image's order.
__global__ void __launch_bounds__(256) orth_load_kernel(OrthView v, float eps) {
  __shared__ double sh[256];
  const int k = find<&OrthMat::tiles0>(v, blockIdx.x);
  const OrthMat q = v.mat[k];
  double s = 0.0;
  for (int i = threadIdx.x; i < q.parts; i += 256) s += v.part[q.part0 + i];
  sh[threadIdx.x] = s;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (threadIdx.x < o) sh[threadIdx.x] += sh[threadIdx.x + o];
    __syncthreads();
  }
  const float scale = static_cast<float>(static_cast<double>(kOrthScale) / (sqrt(sh[0]) + eps));
  const int t = blockIdx.x - q.tiles0, i = t / (2 * q.nt), c = t - i * 2 * q.nt;
  uint8_t* out = tile_at(v, q.x[0] + t);
  const bool tall = (q.flags & kOrthTall) != 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int e = threadIdx.x + 256 * u;
    // lanes along what is contiguous in memory: columns, or rows of a transposed matrix
    const int r = tall ? e & 127 : e >> 3, p = tall ? e >> 7 : e & 7;
    const int row = i * 128 + r, col = c * 64 + p * 8;
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool in = row < q.m && col + j < q.n;
      const long long at = tall ? (col + j) * q.ld_src + row : row * q.ld_src + col + j;
      y[j] = in ? element(q, at) * scale : 0.f;
    }
    uint4 hi, lo;
    split8(y, hi, lo);
    *reinterpret_cast<uint4*>(out + sw128(r, p)) = hi;
    *reinterpret_cast<uint4*>(out + kOrthPlane + sw128(r, p)) = lo;
  }
}

// ------------------------------------------------------------- products
constexpr int kStages = 3;
constexpr int kStage = 2 * kOrthTile;  // the A and the B operand of 64 of K
constexpr int kEpiWarps = 4;
constexpr int kStg = 8192;         // staging of an epilogue warp: 32 rows of a tile, hi and lo
constexpr int kThreads = (2 + kEpiWarps) * 32;
constexpr int kSmem = kStages * kStage + kEpiWarps * kStg + 1024;

struct GemmBars {
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2];
  uint32_t tmem_slot;
  int abort;
};

struct OrthStep {
  float a, b, c;
  int in;    // which copy of X is read
  int last;  // the last step: X goes to the destinations
  int items;
  WaitCtl wc;
};

// Operand pairs of one 128 x 128 tile of phase PHASE's product.  One CTA per SM,
// tiles in turn: warp 0 loads (64 of K per stage, 64 KB), warp 1 issues twelve
// MMAs per stage (four of K by three products), warps 2-5 take the accumulator
// (one of two) out, scale it, split it and store it through shared memory as bulk
// copies of 4 KB.
template <int PHASE>
__global__ void __launch_bounds__(kThreads, 1) orth_gemm_kernel(OrthView v, OrthStep st) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ GemmBars bars;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int* abort = &bars.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.acc_full[i], 1);
      mbar_init(&bars.acc_empty[i], kEpiWarps * 32);
    }
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&bars.tmem_slot, 256);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_slot;

  struct Item {
    OrthMat q;
    int i, j, ks;  // tile (i, j) of the product, stages of K
  };
  auto item = [&](int at) {
    Item t;
    const int k = PHASE == 3 ? find<&OrthMat::mn0>(v, at) : find<&OrthMat::sq0>(v, at);
    t.q = v.mat[k];
    const int r = at - (PHASE == 3 ? t.q.mn0 : t.q.sq0), w = PHASE == 3 ? t.q.nt : t.q.mt;
    t.i = r / w;
    t.j = r - t.i * w;
    t.ks = ((PHASE == 1 ? t.q.n : t.q.m) + 63) / 64;
    return t;
  };

  if (warp == 0) {
    int stage = 0, phase = 0;
    bool go = true;
    for (int at = blockIdx.x; at < st.items && go; at += gridDim.x) {
      const Item t = item(at);
      const OrthMat& q = t.q;
      for (int kk = 0; kk < t.ks; ++kk) {
        if (!__all_sync(0xffffffffu, mbar_wait(&bars.empty[stage], phase ^ 1, st.wc, abort))) { go = false; break; }
        if (lane == 0) {
          uint8_t* sa = sm + stage * kStage;
          uint8_t* sb = sa + kOrthTile;
          uint64_t* full = &bars.full[stage];
          const bool same = PHASE == 1 && t.i == t.j;
          mbar_expect_tx(full, same ? kOrthTile : kStage);
          const int x = q.x[st.in];
          if constexpr (PHASE == 1) {
            bulk_load(sa, tile_at(v, x + t.i * 2 * q.nt + kk), kOrthTile, full);
            if (!same) bulk_load(sb, tile_at(v, x + t.j * 2 * q.nt + kk), kOrthTile, full);
          } else if constexpr (PHASE == 2) {
            bulk_load(sa, tile_at(v, q.a2 + t.i * 2 * q.mt + kk), kOrthTile, full);
            bulk_load(sb, tile_at(v, q.a + t.j * 2 * q.mt + kk), kOrthTile, full);
          } else {
            bulk_load(sa, tile_at(v, q.b + t.i * 2 * q.mt + kk), kOrthTile, full);
            // 64 rows of two tiles side by side: blocks of 64 columns, hi then lo
            const uint8_t* p = tile_at(v, x + (kk >> 1) * 2 * q.nt + 2 * t.j) + (kk & 1) * 8192;
            bulk_load(sb, p, 8192, full);
            bulk_load(sb + 8192, p + kOrthTile, 8192, full);
            bulk_load(sb + 16384, p + kOrthPlane, 8192, full);
            bulk_load(sb + 24576, p + kOrthTile + kOrthPlane, 8192, full);
          }
        }
        __syncwarp();
        if (++stage == kStages) { stage = 0; phase ^= 1; }
      }
    }
  } else if (warp == 1) {
    const uint32_t idesc = idesc_f16_f32(128, 128, 0, PHASE == 3 ? 1 : 0);
    int stage = 0, phase = 0, local = 0;
    bool go = true;
    for (int at = blockIdx.x; at < st.items && go; at += gridDim.x, ++local) {
      const Item t = item(at);
      const int ab = local & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(&bars.acc_empty[ab], ((local >> 1) & 1) ^ 1, st.wc, abort))) break;
      tc_fence_after();
      for (int kk = 0; kk < t.ks; ++kk) {
        if (!__all_sync(0xffffffffu, mbar_wait(&bars.full[stage], phase, st.wc, abort))) { go = false; break; }
        tc_fence_after();
        const uint32_t sa = smem_u32(sm + stage * kStage), sb = PHASE == 1 && t.i == t.j ? sa : sa + kOrthTile;
        if (elect_one()) {
#pragma unroll
          for (int k16 = 0; k16 < 4; ++k16) {
            uint64_t da[2], db[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              da[p] = smem_desc(sa + p * kOrthPlane + k16 * 32, 16, 1024, 2);
              db[p] = PHASE == 3 ? smem_desc(sb + p * kOrthPlane + k16 * 2048, 8192, 1024, 2)
                                 : smem_desc(sb + p * kOrthPlane + k16 * 32, 16, 1024, 2);
            }
            mma_ss(tmem + ab * 128, da[0], db[0], idesc, (kk > 0 || k16 > 0) ? 1u : 0u);
            mma_ss(tmem + ab * 128, da[0], db[1], idesc, 1u);
            mma_ss(tmem + ab * 128, da[1], db[0], idesc, 1u);
          }
          mma_commit(&bars.empty[stage]);
          if (kk == t.ks - 1) mma_commit(&bars.acc_full[ab]);
        }
        __syncwarp();
        if (++stage == kStages) { stage = 0; phase ^= 1; }
      }
    }
  } else {
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    uint8_t* stg = sm + kStages * kStage + (warp - 2) * kStg;
    // 64 columns of this warp's rows, f(column, accumulator) times the scale, into a tile
    auto store = [&](uint8_t* tile, const uint32_t (&lo)[32], const uint32_t (&hi)[32], auto&& f) {
      if (lane == 0) bulk_wait_read();  // the staging has been read
      __syncwarp();
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          y[e] = f(8 * c + e, __uint_as_float(c < 4 ? lo[(8 * c + e) & 31] : hi[(8 * c + e) & 31]));
        uint4 h, l;
        split8(y, h, l);
        const uint32_t o = lane * 128 + ((c ^ (lane & 7)) << 4);
        *reinterpret_cast<uint4*>(stg + o) = h;
        *reinterpret_cast<uint4*>(stg + 4096 + o) = l;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        bulk_store_nc(tile + quarter * 4096, stg, 4096);
        bulk_store_nc(tile + kOrthPlane + quarter * 4096, stg + 4096, 4096);
        bulk_commit();
      }
    };
    int local = 0;
    for (int at = blockIdx.x; at < st.items; at += gridDim.x, ++local) {
      const Item t = item(at);
      const OrthMat& q = t.q;
      const int ab = local & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(&bars.acc_full[ab], (local >> 1) & 1, st.wc, abort))) break;
      tc_fence_after();
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        uint32_t u[32], w[32];
        const uint32_t ta = tmem + lane_addr + ab * 128 + 64 * h;
        tmem_ld32x2_wait(ta, u, ta + 32, w);
        if (h == 1) {
          tc_fence_before();
          mbar_arrive(&bars.acc_empty[ab]);
        }
        const int diag = t.i * 128 + r - (t.j * 128 + 64 * h);  // the column of this row's diagonal element
        constexpr float kBack = 1.f / kOrthScale;                   // products carry the scale twice
        if constexpr (PHASE == 1) {
          const int tt = t.i * 2 * q.mt + 2 * t.j + h;
          store(tile_at(v, q.a + tt), u, w, [&](int, float x) { return x * kBack; });
          store(tile_at(v, q.a2 + tt), u, w, [&](int col, float x) {
            return st.c * (x * kBack) + (col == diag ? st.b * kOrthScale : 0.f);
          });
        } else if constexpr (PHASE == 2) {
          store(tile_at(v, q.b + t.i * 2 * q.mt + 2 * t.j + h), u, w,
                [&](int col, float x) { return x * kBack + (col == diag ? st.a * kOrthScale : 0.f); });
        } else if (!st.last) {
          store(tile_at(v, q.x[st.in ^ 1] + t.i * 2 * q.nt + 2 * t.j + h), u, w,
                [&](int, float x) { return x * kBack; });
        } else {
          const int row = t.i * 128 + r, col0 = t.j * 128 + 64 * h;
          uint16_t* dst = static_cast<uint16_t*>(q.dst);
          if (row < q.m) {
#pragma unroll
            for (int e = 0; e < 64; ++e) {
              if (col0 + e >= q.n) break;
              const float x = __uint_as_float(e < 32 ? u[e & 31] : w[e & 31]) * (kBack * kBack);
              const long long o = (q.flags & kOrthTall) ? (col0 + e) * q.ld_dst + row : row * q.ld_dst + col0 + e;
              dst[o] = static_cast<uint16_t>(pack_bf16x2(x, 0.f) & 0xFFFFu);
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) settle_if_aborted(abort);
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// ------------------------------------------------------------------ host
// The list as the kernels take it: the matrices of one row of tiles (m <= 128)
// first, the widest in front, then the others, and where their parts lie in the
// workspace.
struct Plan {
  std::vector<OrthMat> mats;
  int solo = 0, team = 1;
  long long parts = 0, load_tiles = 0, sq = 0, mn = 0, tiles = 0;
  size_t part_off = 0, tiles_off = 0, total = 0;
};

bool dims_ok(const triattn_matrix& g) { return g.rows > 0 && g.cols > 0; }

// CTAs per matrix of one row of tiles.  A CTA takes about 1.7 k cycles per chunk
// of 64 columns and step, and 4 k (alone) or 7 k (in a team, which adds its parts
// of A) between two passes; the list takes as long as its widest matrix or as its
// sum spread over the SMs (clusters of eight leave some of a GPC's idle).
int team_of(const OrthMat* q, int n) {
  int best = 1;
  double least = 0.0;
  for (int t = 1; t <= 8; t *= 2) {
    double widest = 0.0, sum = 0.0;
    for (int k = 0; k < n; ++k) {
      const int chunks = (q[k].n + 63) / 64;
      const double c = 1.7 * ((chunks + t - 1) / t) + (t > 1 ? 7.0 : 4.0);
      widest = std::max(widest, c);
      sum += c * t;
    }
    const double time = std::max(widest, sum / (t == 8 ? 128 : 152));
    if (t == 1 || time < least) {
      best = t;
      least = time;
    }
  }
  return best;
}

// false: more than the kernels' 32-bit counts hold
bool plan_of(const triattn_matrix* in, const triattn_matrix* out, long long n, Plan* p) {
  p->mats.reserve(static_cast<size_t>(n));
  for (long long k = 0; k < n; ++k) {
    if (!dims_ok(in[k])) continue;
    OrthMat q{};
    const int rows = static_cast<int>(in[k].rows), cols = static_cast<int>(in[k].cols);
    q.src = in[k].data;
    q.ld_src = in[k].stride;
    if (out != nullptr) {
      q.dst = out[k].data;
      q.ld_dst = out[k].stride;
    }
    q.flags = (in[k].dtype == TRIATTN_DTYPE_FP32 ? kOrthFp32 : 0) | (rows > cols ? kOrthTall : 0);
    q.m = std::min(rows, cols);
    q.n = std::max(rows, cols);
    q.mt = (q.m + 127) / 128;
    q.nt = (q.n + 127) / 128;
    q.part_rows = std::max(1, 16384 / cols);
    q.parts = (rows + q.part_rows - 1) / q.part_rows;
    p->mats.push_back(q);
  }
  const auto others = std::stable_partition(p->mats.begin(), p->mats.end(), [](const OrthMat& q) { return q.mt == 1; });
  p->solo = static_cast<int>(others - p->mats.begin());
  std::stable_sort(p->mats.begin(), others, [](const OrthMat& x, const OrthMat& y) { return x.n > y.n; });
  p->team = team_of(p->mats.data(), p->solo);
  for (OrthMat& q : p->mats) {
    const long long xt = 2ll * q.mt * q.nt, at = 2ll * q.mt * q.mt;
    q.part0 = static_cast<int>(p->parts);
    q.tiles0 = static_cast<int>(p->load_tiles);
    p->parts += q.parts;
    p->load_tiles += xt;
    q.x[0] = static_cast<int>(p->tiles);
    p->tiles += xt;
    if (q.mt > 1) {
      q.sq0 = static_cast<int>(p->sq);
      q.mn0 = static_cast<int>(p->mn);
      p->sq += at / 2;
      p->mn += xt / 2;
      q.x[1] = static_cast<int>(p->tiles);
      q.a = static_cast<int>(p->tiles + xt);
      q.a2 = static_cast<int>(p->tiles + xt + at);
      q.b = static_cast<int>(p->tiles + xt + 2 * at);
      p->tiles += xt + 3 * at;
    } else if (p->team > 1) {
      q.a = static_cast<int>(p->tiles);
      p->tiles += 2 * (p->team + 1);
    }
    if (p->tiles >= (1ll << 31) || p->parts >= (1ll << 31)) return false;
  }
  auto up = [](size_t x) { return (x + 1023) / 1024 * 1024; };
  p->part_off = up(p->mats.size() * sizeof(OrthMat));
  p->tiles_off = up(p->part_off + static_cast<size_t>(p->parts) * 4);
  p->total = p->tiles_off + static_cast<size_t>(p->tiles) * kOrthTile;
  return true;
}

constexpr long long kMaxSide = 65536;

triattn_status check_list(const triattn_matrix* ms, long long n, bool output) {
  if (n < 0 || (n > 0 && ms == nullptr)) return TRIATTN_ERR_INVALID_ARG;
  if (n > (1 << 20)) return TRIATTN_ERR_UNSUPPORTED;
  for (long long i = 0; i < n; ++i) {
    const triattn_matrix& g = ms[i];
    if (g.rows < 0 || g.cols < 0) return TRIATTN_ERR_INVALID_ARG;
    if (g.dtype != TRIATTN_DTYPE_BF16 && (output || g.dtype != TRIATTN_DTYPE_FP32)) return TRIATTN_ERR_UNSUPPORTED;
    if (!dims_ok(g)) continue;
    if (g.rows > kMaxSide || g.cols > kMaxSide) return TRIATTN_ERR_UNSUPPORTED;
    if (g.stride < g.cols || g.stride >= (1ll << 36)) return TRIATTN_ERR_INVALID_ARG;
    if (g.data == nullptr || (reinterpret_cast<uintptr_t>(g.data) & (g.dtype == TRIATTN_DTYPE_FP32 ? 3u : 1u)) != 0)
      return TRIATTN_ERR_INVALID_ARG;
  }
  return TRIATTN_OK;
}

template <int PHASE>
cudaError_t launch_phase(const OrthView& v, const OrthStep& st, int sms, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(orth_gemm_kernel<PHASE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  return trace_call(kKOrthGemm, s, [&] {
    orth_gemm_kernel<PHASE><<<std::min(st.items, sms), kThreads, kSmem, s>>>(v, st);
    return cudaGetLastError();
  });
}

cudaError_t run(const Plan& p, int steps, const float* co, float eps, uint8_t* ws, const WaitCtl& wc, cudaStream_t s) {
  OrthMat* mats = reinterpret_cast<OrthMat*>(ws);
  OrthView v{mats, reinterpret_cast<float*>(ws + p.part_off), ws + p.tiles_off, static_cast<int>(p.mats.size())};
  OrthTable t;
  cudaError_t e = cudaSuccess;
  for (size_t k = 0; k < p.mats.size() && e == cudaSuccess; k += kUpload) {
    t.n = static_cast<int>(std::min<size_t>(kUpload, p.mats.size() - k));
    std::copy_n(p.mats.data() + k, t.n, t.mat);
    e = trace_call(kKOrthLoad, s, [&] {
      orth_table_kernel<<<1, 256, 0, s>>>(t, mats + k);
      return cudaGetLastError();
    });
  }
  if (e == cudaSuccess)
    e = trace_call(kKOrthLoad, s, [&] {
      orth_norm_kernel<<<static_cast<unsigned>(p.parts), 256, 0, s>>>(v);
      return cudaGetLastError();
    });
  if (e == cudaSuccess)
    e = trace_call(kKOrthLoad, s, [&] {
      orth_load_kernel<<<static_cast<unsigned>(p.load_tiles), 256, 0, s>>>(v, eps);
      return cudaGetLastError();
    });
  if (p.solo > 0 && e == cudaSuccess)
    e = trace_call(kKOrthSolo, s, [&] {
      return launch_orth_solo(mats, p.solo, v.tiles, steps, OrthCoef{co[0], co[1], co[2]},
                              p.team, wc, s);
    });
  v.mat += p.solo;
  v.n -= p.solo;
  OrthStep st{co[0], co[1], co[2], 0, 0, 0, wc};
  for (int k = 0; k < steps && v.n > 0 && e == cudaSuccess; ++k) {
    st.in = k & 1;
    st.last = k == steps - 1;
    st.items = static_cast<int>(p.sq);
    e = launch_phase<1>(v, st, 152, s);
    if (e == cudaSuccess) e = launch_phase<2>(v, st, 152, s);
    st.items = static_cast<int>(p.mn);
    if (e == cudaSuccess) e = launch_phase<3>(v, st, 152, s);
  }
  return e;
}

}  // namespace
}  // namespace triattn

using namespace triattn;

extern "C" {

size_t triattn_orthogonalize_workspace_bytes(const triattn_matrix* matrices, long long n) {
  if (check_list(matrices, n, false) != TRIATTN_OK) return 0;
  try {
    Plan p;
    return plan_of(matrices, nullptr, n, &p) ? std::max<size_t>(p.total, 256) : 0;
  } catch (const std::bad_alloc&) {
    return 0;
  }
}

triattn_status triattn_orthogonalize(const triattn_matrix* matrices, const triattn_matrix* out, long long n, int steps,
                                     const float* coefficients, float eps, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  triattn_status st = check_list(matrices, n, false);
  if (st == TRIATTN_OK) st = check_list(out, n, true);
  if (st != TRIATTN_OK) return st;
  if (coefficients == nullptr || steps < 1 || !(eps > 0.f) || !std::isfinite(eps)) return TRIATTN_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (!std::isfinite(coefficients[i])) return TRIATTN_ERR_INVALID_ARG;
  if (steps > 64) return TRIATTN_ERR_UNSUPPORTED;
  for (long long i = 0; i < n; ++i)
    if (out[i].rows != matrices[i].rows || out[i].cols != matrices[i].cols) return TRIATTN_ERR_INVALID_ARG;
  try {
    // outputs are written without an order between them; every input is read
    // before the first of them
    struct Span {
      uintptr_t lo, hi;
    };
    std::vector<Span> dst;
    dst.reserve(static_cast<size_t>(n));
    for (long long i = 0; i < n; ++i)
      if (dims_ok(out[i])) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(out[i].data);
        dst.push_back({a, a + 2 * static_cast<uintptr_t>((out[i].rows - 1) * out[i].stride + out[i].cols)});
      }
    std::sort(dst.begin(), dst.end(), [](const Span& x, const Span& y) { return x.lo < y.lo; });
    for (size_t i = 1; i < dst.size(); ++i)
      if (dst[i].lo < dst[i - 1].hi) return TRIATTN_ERR_INVALID_ARG;
    Plan p;
    if (!plan_of(matrices, out, n, &p)) return TRIATTN_ERR_UNSUPPORTED;
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
        workspace_bytes < std::max<size_t>(p.total, 256))
      return TRIATTN_ERR_WORKSPACE;
    if (p.mats.empty()) return TRIATTN_OK;
    const WaitCtl wc = current_wait_ctl();
    if (wc.status == nullptr) return TRIATTN_ERR_CUDA;
    const cudaError_t e = run(p, steps, coefficients, eps, static_cast<uint8_t*>(workspace), wc,
                              static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TRIATTN_OK : TRIATTN_ERR_CUDA;
  } catch (const std::bad_alloc&) {
    return TRIATTN_ERR_WORKSPACE;
  }
}

}  // extern "C"
