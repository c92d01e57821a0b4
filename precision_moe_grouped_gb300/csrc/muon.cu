// muon.cu -- one step over weight matrices whose update is made (nearly)
// orthogonal by Newton-Schulz steps.
//
//   m <- mu m + (1 - mu) g,  u = mu m + (1 - mu) g (nesterov) or m
//   X0 = u / (|u|_F + eps);  X <- a X + (b G + c G^2) X with G = X X^T, `steps` times
//   p <- p (1 - lr wd) - lr s X
//
// X is taken with its short side m as rows.  All the steps' polynomials of G
// commute, so they are carried out on m x m matrices: with P = a I + b G + c G^2
// a step is X <- P X, G <- P G P, and three of them are X <- Q X with Q <- P Q.
// (P is formed as c G (G + (b / c) I) + a I: the sum in brackets differs from G
// on the diagonal alone, so G's diagonal blocks are kept a second time.)
// The long side is then met twice in three steps (G = X X^T, Q X) instead of
// twice in each, and every m x m product is symmetric and computed by half.
// After three steps X is formed and G taken from it anew: a small singular value
// s of X enters G as s^2 beside 1 and the steps multiply its errors by up to a^2
// each; three of them lose as little as the plain form in 32 bits does (five
// in one go lose up to 50 times as much for a decaying spectrum).
//
// Numbers between the products are two fp16 terms, hi + lo, of the value times
// a power of two (22 bits; the powers follow from the coefficients, which
// bound every matrix), and a product is lo hi + hi lo + hi hi (terms.cuh).
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>
#include <utility>

#include "dense.cuh"
#include "entry.h"
#include "muon.cuh"
#include "terms.cuh"

namespace moe {
namespace {

using dense::Elem;
using dense::EpiWarp;
using terms::Maps;
using dense::Tile;

constexpr uint64_t kTimeoutNs = 1000000000ull;
constexpr int kPartSteps = kMuonPartSteps;
constexpr int kChainSide = 384;   // of the m x m products that one launch carries out
constexpr int kThreads = 256;

// ------------------------------------------------------------ elementwise
constexpr int kChunk = 16384, kChunkSmall = 2048;   // elements of a block's share
constexpr int64_t kL2Bytes = 100 << 20;   // of the 129 MB, what two readings in turn may count on

// The new momentum, and each chunk's sum of u^2 (matrix z, chunk c at
// sums[z chunks + c]).
__global__ void __launch_bounds__(kThreads)
    muon_momentum_kernel(const Momentum a, int64_t size, int chunk, int vec, float* sums) {
  __shared__ float warp_sums[kThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const float gs = a.grad_scale ? __ldg(a.grad_scale) : 1.0f;
  const int64_t base = static_cast<int64_t>(blockIdx.y) * size;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * chunk;
  const int64_t i1 = i0 + chunk < size ? i0 + chunk : size;
  float s = 0.f;
  if (vec) {
#pragma unroll 4
    for (int64_t i = i0 + 4 * threadIdx.x; i < i1; i += 4 * kThreads) {
      float4 m = *reinterpret_cast<const float4*>(a.m + base + i);
      float g[4];
      if (a.bf16) {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.grad) + base + i);
        const float2 lo = dense::unpack_bf16(v.x), hi = dense::unpack_bf16(v.y);
        g[0] = lo.x, g[1] = lo.y, g[2] = hi.x, g[3] = hi.y;
      } else {
        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.grad) + base + i);
        g[0] = v.x, g[1] = v.y, g[2] = v.z, g[3] = v.w;
      }
      float* e = &m.x;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float gk = gs * g[k];
        e[k] = fmaf(a.mu, e[k], a.rest * gk);
        const float u = update_of(a, e[k], gk);
        s = fmaf(u, u, s);
      }
      *reinterpret_cast<float4*>(a.m + base + i) = m;
    }
  } else {
    // eight loads of each in flight; beyond the end the last element, unused
    for (int64_t i = i0 + threadIdx.x; i < i1; i += 8 * kThreads) {
      float g[8], m[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t at = base + (i + k * kThreads < i1 ? i + k * kThreads : i1 - 1);
        m[k] = a.m[at];
        g[k] = grad_at(a, at, gs);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (i + k * kThreads < i1) {
          m[k] = fmaf(a.mu, m[k], a.rest * g[k]);
          a.m[base + i + k * kThreads] = m[k];
          const float u = update_of(a, m[k], g[k]);
          s = fmaf(u, u, s);
        }
      }
    }
  }
  s = block_sum<kThreads>(s, warp_sums);
  if (threadIdx.x == 0) sums[static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x] = s;
}

// Four neighbours as hi and lo terms.
__device__ __forceinline__ void put_terms(const float (&v)[4], __half* to, int64_t lo_off) {
  uint2 hi, lo;
  hi.x = dense::pack_f16(v[0], v[1]);
  hi.y = dense::pack_f16(v[2], v[3]);
  const float2 p = dense::unpack_f16(hi.x), q = dense::unpack_f16(hi.y);
  lo.x = dense::pack_f16(v[0] - p.x, v[1] - p.y);
  lo.y = dense::pack_f16(v[2] - q.x, v[3] - q.y);
  *reinterpret_cast<uint2*>(to) = hi;
  *reinterpret_cast<uint2*>(to + lo_off) = lo;
}

// X0's planes: hi and lo fp16 terms of scale * u / (|u| + eps), [mp][np] per
// matrix with zeros beyond m x n; a tall matrix [n, m] is turned on the way.  A
// block takes a square of 64, a thread four neighbours in each of four rows.
constexpr int kSide = 64;
__global__ void __launch_bounds__(kThreads)
    muon_planes_kernel(const Momentum a, int rows, int cols, int vec, const float* sums, int chunks, float eps,
                       float scale, __half* planes, int64_t lo_off, int mp, int np) {
  __shared__ float warp_sums[kThreads / 32];
  __shared__ float tile[kSide][kSide + 1];
  griddep_wait();
  griddep_launch_dependents();
  const float gs = a.grad_scale ? __ldg(a.grad_scale) : 1.0f;
  const int z = blockIdx.z;
  const bool tall = rows > cols;
  const int64_t base = static_cast<int64_t>(z) * rows * cols;
  // the source's square: rows r0.., columns c0..
  const int r0 = (tall ? blockIdx.x : blockIdx.y) * kSide, c0 = (tall ? blockIdx.y : blockIdx.x) * kSide;
  const int tx = (threadIdx.x & 15) * 4, ty = threadIdx.x >> 4;
  float mv[4][4], gv[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + ty + 16 * i, c = c0 + tx;
    const int64_t at = base + static_cast<int64_t>(r) * cols + c;
    if (vec && r < rows && c + 4 <= cols) {
      const float4 m = *reinterpret_cast<const float4*>(a.m + at);
      mv[i][0] = m.x, mv[i][1] = m.y, mv[i][2] = m.z, mv[i][3] = m.w;
      if (a.bf16) {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.grad) + at);
        const float2 lo = dense::unpack_bf16(v.x), hi = dense::unpack_bf16(v.y);
        gv[i][0] = lo.x, gv[i][1] = lo.y, gv[i][2] = hi.x, gv[i][3] = hi.y;
      } else {
        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.grad) + at);
        gv[i][0] = v.x, gv[i][1] = v.y, gv[i][2] = v.z, gv[i][3] = v.w;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) gv[i][k] *= gs;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool in = r < rows && c + k < cols;
        mv[i][k] = in ? a.m[at + k] : 0.f;
        gv[i][k] = in ? grad_at(a, at + k, gs) : 0.f;
      }
    }
  }
  float s = 0.f;
  for (int i = threadIdx.x; i < chunks; i += kThreads) s += sums[static_cast<int64_t>(z) * chunks + i];
  s = block_sum<kThreads>(s, warp_sums);
  const float mul = scale / (sqrtf(s) + eps);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool in = r0 + ty + 16 * i < rows && c0 + tx + k < cols;
      mv[i][k] = in ? update_of(a, mv[i][k], gv[i][k]) * mul : 0.f;   // (0 stays 0 beside a NaN norm)
    }
  if (tall) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) tile[tx + k][ty + 16 * i] = mv[i][k];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) mv[i][k] = tile[ty + 16 * i][tx + k];
  }
  const int64_t out = (static_cast<int64_t>(z) * mp + blockIdx.y * kSide + ty) * np + blockIdx.x * kSide + tx;
#pragma unroll
  for (int i = 0; i < 4; ++i) put_terms(mv[i], planes + out + static_cast<int64_t>(16 * i) * np, lo_off);
}

// -------------------------------------------------------------- epilogues
// A matrix as planes, hi and lo terms of v = c D + a I.  A symmetric one is
// computed and stored by its 256 x 256 blocks on and above the diagonal; with
// map_diag the diagonal blocks go there a second time, as v + h I.
struct EpiPlanes {
  struct Args {
    float c, a, h;
    int32_t map, map_diag;   // stores of 32 x 32; 0: none
    int32_t lo_rows;         // rows from the hi to the lo plane
    int32_t m, rows, cols;   // rows of I; stored rows (a multiple of 64) and columns
  };
  static __device__ __forceinline__ void ahead(const Args&, const Tile&, const EpiWarp&, int, int) {}
  template <class M>
  static __device__ __forceinline__ void run(const Args& a, const Tile& o, const EpiWarp& w, int col0, int n,
                                             const M& maps, float (&d)[128]) {
    if (w.row >= a.rows) return;
    const int row = o.z * a.rows + w.row;
#pragma unroll
    for (int c = 0; c < 128; c += 32) {
      const int col = col0 + c;
      if (c >= n || col >= a.cols) continue;
#pragma unroll
      for (int i = 0; i < 32; ++i) d[c + i] *= a.c;
      const int on = w.row + w.lane - col;   // this row's place on the diagonal
      const bool diag = col == w.row;        // (both are multiples of 32)
      if (diag && w.row + w.lane < a.m) {
#pragma unroll
        for (int i = 0; i < 32; ++i) d[c + i] += on == i ? a.a : 0.f;
      }
      store(d, c, w, maps.m[a.map], col, row, a.lo_rows);
      if (a.map_diag && (col >> 8) == o.i) {
        if (diag && w.row + w.lane < a.m) {
#pragma unroll
          for (int i = 0; i < 32; ++i) d[c + i] += on == i ? a.h : 0.f;
        }
        store(d, c, w, maps.m[a.map_diag], col & 255, row, a.lo_rows);
      }
    }
  }
  // 32 columns through the warp's box: two halves of 32 rows of 64 bytes, in the
  // 64-byte swizzle
  static __device__ __forceinline__ void store(const float (&d)[128], int c, const EpiWarp& w,
                                               const CUtensorMap& m, int col, int row, int lo_rows) {
    constexpr int kHalf = dense::kStageBox / 2;
    if (w.lane == 0) dense::box_wait_read();
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x = d[c + 8 * i + 2 * k], y = d[c + 8 * i + 2 * k + 1];
        hi[k] = dense::pack_f16(x, y);
        const float2 f = dense::unpack_f16(hi[k]);
        lo[k] = dense::pack_f16(x - f.x, y - f.y);
      }
      uint8_t* at = w.box + w.lane * 64 + ((i ^ ((w.lane >> 1) & 3)) << 4);
      *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(at + kHalf) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (w.lane == 0) {
      dense::box_store(&m, w.box, col, row);
      dense::box_store(&m, w.box + kHalf, col, row + lo_rows);
    }
  }
};

// A share of a long sum, in float: row r of share s of matrix z at row
// (s batch + z) rows + r.
struct EpiShare {
  struct Args {
    int32_t map, rows, batch;   // rows: a multiple of 64
  };
  static __device__ __forceinline__ void ahead(const Args&, const Tile&, const EpiWarp&, int, int) {}
  static __device__ __forceinline__ void run(const Args& a, const Tile& o, const EpiWarp& w, int col0, int n,
                                             const Maps& maps, float (&d)[128]) {
    if (w.row >= a.rows) return;
#pragma unroll
    for (int c = 0; c < 128; c += 32) {
      if (c >= n || col0 + c >= a.rows) continue;
      if (w.lane == 0) dense::box_wait_read();
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *dense::box_piece(w.box, w.lane, i) =
            make_uint4(__float_as_uint(d[c + 4 * i]), __float_as_uint(d[c + 4 * i + 1]),
                       __float_as_uint(d[c + 4 * i + 2]), __float_as_uint(d[c + 4 * i + 3]));
      fence_proxy_async_smem();
      __syncwarp();
      if (w.lane == 0)
        dense::box_store(&maps.m[a.map], w.box, col0 + c, (o.s * a.batch + o.z) * a.rows + w.row);
    }
  }
};

constexpr int kJoinThreads = 64;
// The shares joined in order: G's planes (and its diagonal blocks + h I), as
// EpiPlanes stores them.  Four columns a thread.
__global__ void __launch_bounds__(kJoinThreads)
    muon_join_kernel(const float* shares, int splits, int64_t batch, int mp, int m, float c, float h, __half* g,
                     __half* diag) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kJoinThreads + threadIdx.x;
  const int64_t row = i / (mp / 4);   // of all matrices
  if (row >= batch * mp) return;
  const int col = static_cast<int>(i - row * (mp / 4)) * 4, r = static_cast<int>(row % mp);
  const int side = (col >> 8) - (r >> 8);
  if (side < 0) return;
  const float* at = shares + row * mp + col;
  const int64_t step = batch * mp * mp;
  float4 v = make_float4(0, 0, 0, 0);
  for (int s0 = 0; s0 < splits; s0 += 8) {   // eight shares' loads in flight
    float4 x[8];
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (s0 + s < splits) x[s] = *reinterpret_cast<const float4*>(at + (s0 + s) * step);
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (s0 + s < splits) v = make_float4(v.x + x[s].x, v.y + x[s].y, v.z + x[s].z, v.w + x[s].w);
  }
  float d[4] = {v.x * c, v.y * c, v.z * c, v.w * c};
  put_terms(d, g + row * mp + col, batch * mp * mp);
  if (side == 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (col + k == r && r < m) d[k] += h;
    put_terms(d, diag + row * dense::kTile + (col & 255), batch * mp * dense::kTile);
  }
}

// p <- decay p - step D, and the copy.  D's rows run along p's contiguous side
// (element (r, c) of D at p[c rows + r]), so that a warp's 32 rows are 128 bytes.
struct EpiUpdate {
  struct Args {
    float* p;
    __nv_bfloat16* copy;   // or null
    float decay, step;
    int32_t rows, cols;
  };
  // p's lines into L2 while the products run
  static __device__ __forceinline__ void ahead(const Args& a, const Tile& o, const EpiWarp& w, int col, int n) {
    if (w.row >= a.rows) return;
    const int64_t base = static_cast<int64_t>(o.z) * a.rows * a.cols + w.row;
    for (int c = col + w.lane; c < col + n && c < a.cols; c += 32)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a.p + base + static_cast<int64_t>(c) * a.rows));
  }
  static __device__ __forceinline__ void run(const Args& a, const Tile& o, const EpiWarp& w, int col0, int n,
                                             const Maps&, float (&d)[128]) {
    const int r = w.row + w.lane;
    if (r >= a.rows) return;
    const int64_t base = (static_cast<int64_t>(o.z) * a.cols + col0) * a.rows + r;
    float* p = a.p + base;
    __nv_bfloat16* copy = a.copy + base;
    const int end = a.cols - col0 < n ? a.cols - col0 : n;
#pragma unroll
    for (int c = 0; c < 128; c += 16) {
      if (c + 16 <= end) {   // the loads of 16 columns are in flight together
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = p[static_cast<int64_t>(c + i) * a.rows];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int64_t at = static_cast<int64_t>(c + i) * a.rows;
          const float x = fmaf(-a.step, d[c + i], a.decay * v[i]);
          p[at] = x;
          if (a.copy) copy[at] = __float2bfloat16_rn(x);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (c + i < end) {
            const int64_t at = static_cast<int64_t>(c + i) * a.rows;
            const float x = fmaf(-a.step, d[c + i], a.decay * p[at]);
            p[at] = x;
            if (a.copy) copy[at] = __float2bfloat16_rn(x);
          }
        }
      }
    }
  }
};

// ------------------------------------------------------------------- plans
// Bounds of every matrix of a schedule, from the polynomials on a grid over the
// singular values (all at most 1 at first, as |X0|_F is), and the powers of two
// that bring each to at most 2^14: fp16 then holds it with room for the grid's
// and the arithmetic's errors.
constexpr int kMaxSteps = 12;
struct StepScales {
  float g, p, q, s;   // of G and P of the step, of Q after it, of S = P G
};
struct Scales {
  StepScales step[kMaxSteps];
  float x[kMaxSteps + 1];   // of X before each part, [parts]: after the last (unused)
};

bool power_for(double bound, float* out) {
  if (!(bound < 1e6)) return false;   // NaN too
  int e;
  std::frexp(std::max(bound, 1e-6), &e);   // bound < 2^e
  *out = std::ldexp(1.0f, 14 - e);
  return true;
}

bool make_scales(const moe_muon_options* o, Scales* out) {
  constexpr int kGrid = 512;
  const double a = o->coefficients[0], b = o->coefficients[1], c = o->coefficients[2];
  double top = 1.0;
  int part = 0;
  for (int done = 0; done < o->ns_steps; done += kPartSteps, ++part) {
    const int n = std::min(kPartSteps, o->ns_steps - done);
    double mg[kPartSteps] = {}, mp[kPartSteps] = {}, mq[kPartSteps] = {}, ms[kPartSteps] = {}, mx = 0;
    for (int i = 0; i <= kGrid; ++i) {
      const double s = top * i / kGrid;
      double g = s * s, q = 1;
      for (int k = 0; k < n; ++k) {
        const double p = a + b * g + c * g * g;
        q *= p;
        mg[k] = std::max(mg[k], std::fabs(g));
        mp[k] = std::max(mp[k], std::fabs(p));
        mq[k] = std::max(mq[k], std::fabs(q));
        ms[k] = std::max(ms[k], std::fabs(p * g));
        g = p * p * g;
      }
      mx = std::max(mx, std::fabs(q * s));
    }
    if (!power_for(top, &out->x[part])) return false;
    for (int k = 0; k < n; ++k) {
      StepScales& t = out->step[done + k];
      if (!power_for(mg[k] + std::fabs(b / c), &t.g) || !power_for(mp[k], &t.p) || !power_for(mq[k], &t.q) ||
          !power_for(ms[k], &t.s))
        return false;
    }
    if (!(mx < 1e3)) return false;
    top = std::max(mx, 1e-3);
  }
  return true;
}

// One group: the tensors whose matrices are m x n (or n x m), `all` of them in the
// tensors' order; it runs in equal slices of up to `each`, of which this one has
// `batch` matrices from number `first` on.
struct Shape {
  int32_t m, n, mp, np;
  int64_t all, each, first, batch;
};
Shape shape_of(const moe_muon_tensor& t) {
  Shape s;
  s.m = std::min(t.rows, t.cols);
  s.n = std::max(t.rows, t.cols);
  s.mp = (s.m + 63) / 64 * 64;
  s.np = (s.n + 63) / 64 * 64;
  s.all = s.each = s.first = s.batch = 0;
  return s;
}
bool same(const moe_muon_tensor& t, const Shape& s) {
  return !muon_empty(t) && std::min(t.rows, t.cols) == s.m && std::max(t.rows, t.cols) == s.n;
}
// Blocks' shares: long ones, unless they would leave SMs idle.
int chunk_of(const Shape& s) {
  return static_cast<int64_t>(s.m) * s.n * s.each >= int64_t(600) * kChunk ? kChunk : kChunkSmall;
}
int chunks_of(const Shape& s) {
  return static_cast<int>(dense::cdiv(static_cast<int64_t>(s.m) * s.n, chunk_of(s)));
}

// Tiles on and above the diagonal.
int64_t upper_tiles(int64_t mp) {
  const int64_t n = dense::cdiv(mp, dense::kTile);
  return n * (n + 1) / 2;
}
// Shares of the sum over the long side, of at least four K blocks, where the
// halves of X X^T's tiles leave half of the pairs without one.
int gram_splits(const Shape& s) {
  const int64_t units = 2 * upper_tiles(s.mp) * s.each, kb = s.np / dense::kBK;
  return static_cast<int>(std::max<int64_t>(1, std::min(dense::kPlanPairs / units, kb / 4)));
}

struct GroupWs {
  size_t sums, x, x1, g, h, s, p, qa, qb, shares, total;
};
GroupWs group_ws(const Shape& s) {
  GroupWs w = {};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += ws_up(bytes);
    return o;
  };
  const size_t big = 4ull * s.batch * s.mp * s.np, small = 4ull * s.batch * s.mp * s.mp;
  w.sums = take(4ull * s.batch * chunks_of(s));
  w.x = take(big);
  w.x1 = take(big);
  w.g = take(small);
  w.h = take(4ull * s.batch * s.mp * dense::kTile);
  w.s = take(small);
  w.p = take(small);
  w.qa = take(small);
  w.qb = take(small);
  const int splits = gram_splits(s);
  w.shares = take(splits > 1 ? static_cast<size_t>(splits) * small : 0);
  w.total = at;
  return w;
}

// What the launches of a call share.
struct Call {
  const moe_muon_tensor* t;
  int32_t count;
  const moe_muon_options* o;
  Scales sc;
  int32_t* status;
  cudaStream_t st;
  int pairs_planes, pairs_update, pairs_share;
};
// A matrix [rows of the batch][ld] as planes, times `scale`.
struct Planes {
  __half* at;
  float scale;
  int32_t ld;
  bool sym;
  __half* diag;   // G's diagonal blocks + (b / c) I, or null
};

struct Group {
  Shape s;
  GroupWs w;
  uint8_t* ws;
  Planes x, g, p, q;
  __half* planes(size_t off) const { return reinterpret_cast<__half*>(ws + off); }
  Planes square(size_t off, float scale) const { return {planes(off), scale, s.mp, true, nullptr}; }
};
constexpr int kMostGroups = terms::kChainGroups;   // that share their launches: two products each in terms::Launch
int64_t rows_of(const Shape& s) { return s.batch * s.mp; }

// A launch in the making, of one phase or (terms::Chain) of several.
template <class Epi, class L = terms::Launch<typename Epi::Args>, class M = Maps>
struct Build {
  static constexpr bool kChain = !std::is_same<M, Maps>::value;
  M m;
  L l;
  std::pair<const __half*, int> made[kChain ? terms::kChainMaps : 1];   // a chain's maps, which its phases share

  explicit Build(const Call& c) : l{} {
    l.status = c.status;
    l.timeout_ns = kTimeoutNs;
    l.maps = 1;   // map 0 stands for none
    m.m[0] = CUtensorMap{};
  }
  int32_t map(const Shape& s, const __half* at, int64_t cols, int box_cols, int box_rows, dense::Swizzle sw,
              int32_t* index) {
    if (kChain) {
      for (int32_t i = 1; i < l.maps; ++i) {
        if (made[i] == std::make_pair(at, box_cols)) {
          *index = i;
          return MOE_OK;
        }
      }
      made[l.maps] = {at, box_cols};
    }
    *index = l.maps++;
    return dense::make_map(&m.m[*index], at, Elem::kF16, 2 * rows_of(s), cols, cols, box_cols, box_rows, sw);
  }
  // The operand as rows of a tile or, with mn, its transpose; from matrix z on.
  int32_t operand(const Shape& s, const Planes& p, bool mn, int64_t z, terms::Operand* o) {
    *o = {};
    o->hi = static_cast<int32_t>(z * s.mp);
    o->lo = static_cast<int32_t>(rows_of(s) + z * s.mp);
    o->batch = s.mp;
    o->mn = mn;
    o->sym = p.sym;
    MOE_TRY(map(s, p.at, p.ld, dense::kBK, dense::kBK, dense::Swizzle::k128, &o->map));
    if (p.diag) MOE_TRY(map(s, p.diag, dense::kTile, dense::kBK, dense::kBK, dense::Swizzle::k128, &o->diag));
    return MOE_OK;
  }
  terms::Problem& problem(int64_t tile_rows, int64_t tile_cols, int64_t batch, int64_t kb) {
    terms::Problem& p = l.p[l.problems++];
    p.tiles_m = static_cast<int32_t>(dense::cdiv(tile_rows, dense::kTile));
    p.tiles_n = static_cast<int32_t>(dense::cdiv(tile_cols, dense::kTile));
    p.per_matrix = p.tiles_m * p.tiles_n;
    p.batch = static_cast<int32_t>(batch);
    p.splits = 1;
    p.kb = p.kb_split = static_cast<int32_t>(kb);
    return p;
  }
};

using BuildPlanes = Build<EpiPlanes>;
using BuildChain = Build<EpiPlanes, terms::Chain<EpiPlanes::Args>, terms::ChainMaps>;

// out = c A B^T + a I, symmetric [mp, mp]; A and B [mp, k], B's second copy of the
// diagonal blocks used when use_diag.
template <class B>
int32_t add_symmetric(B& b, const Shape& s, const Planes& x, Planes y, bool use_diag, const Planes& out, float c,
                      float a, float ratio) {
  if (!use_diag) y.diag = nullptr;
  Planes left = x;
  left.diag = nullptr;
  terms::Problem& p = b.problem(s.mp, s.mp, s.batch, x.ld / dense::kBK);
  p.upper = 1;
  p.per_matrix = static_cast<int32_t>(upper_tiles(s.mp));
  MOE_TRY(b.operand(s, left, false, 0, &p.a));
  MOE_TRY(b.operand(s, y, false, 0, &p.b));
  EpiPlanes::Args& e = b.l.e[b.l.problems - 1];
  e = {};
  e.c = c * out.scale / (x.scale * y.scale);
  e.a = a * out.scale;
  MOE_TRY(b.map(s, out.at, s.mp, 32, 32, dense::Swizzle::k64, &e.map));
  if (out.diag) {
    MOE_TRY(b.map(s, out.diag, dense::kTile, 32, 32, dense::Swizzle::k64, &e.map_diag));
    e.h = ratio * out.scale;
  }
  e.lo_rows = static_cast<int32_t>(rows_of(s));
  e.m = s.m;
  e.rows = e.cols = s.mp;
  return MOE_OK;
}

int32_t run(const Call& c, BuildPlanes& b) {
  if (b.l.problems) MOE_CUDA(terms::launch<EpiPlanes>(b.m, b.l, c.pairs_planes, c.st));
  return MOE_OK;
}

// G = X X^T with its second diagonal blocks (+ ratio I), by shares of the long
// side where there are few tiles.
int32_t gram(const Call& c, Group* gs, int n, float ratio) {
  BuildPlanes whole(c);
  Build<EpiShare> b(c);
  for (Group* g = gs; g < gs + n; ++g) {
    const Shape& s = g->s;
    const int splits = gram_splits(s);
    if (splits == 1) {
      MOE_TRY(add_symmetric(whole, s, g->x, g->x, false, g->g, 1.0f, 0.f, ratio));
      continue;
    }
    terms::Problem& p = b.problem(s.mp, s.mp, s.batch, s.np / dense::kBK);
    EpiShare::Args& e = b.l.e[b.l.problems - 1];
    p.upper = 1;
    p.per_matrix = static_cast<int32_t>(upper_tiles(s.mp));
    p.kb_split = static_cast<int32_t>(dense::cdiv(p.kb, splits));
    p.splits = static_cast<int32_t>(dense::cdiv(p.kb, p.kb_split));
    MOE_TRY(b.operand(s, g->x, false, 0, &p.a));
    p.b = p.a;
    e.map = b.l.maps++;
    e.rows = s.mp;
    e.batch = static_cast<int32_t>(s.batch);
    MOE_TRY(dense::make_map(&b.m.m[e.map], g->ws + g->w.shares, Elem::kF32, p.splits * rows_of(s), s.mp, s.mp, 32,
                            32));
  }
  MOE_TRY(run(c, whole));
  if (b.l.problems) MOE_CUDA(terms::launch<EpiShare>(b.m, b.l, c.pairs_share, c.st));
  int i = 0;
  for (Group* g = gs; g < gs + n; ++g) {
    const Shape& s = g->s;
    if (gram_splits(s) == 1) continue;
    const int64_t blocks = dense::cdiv(rows_of(s) * (s.mp / 4), kJoinThreads);
    MOE_CUDA(launch_pdl(muon_join_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kJoinThreads), 0, c.st,
                        reinterpret_cast<const float*>(g->ws + g->w.shares), static_cast<int>(b.l.p[i++].splits),
                        s.batch, s.mp, s.m, g->g.scale / (g->x.scale * g->x.scale), ratio * g->g.scale, g->g.at,
                        g->g.diag));
  }
  return MOE_OK;
}

// X <- Q X as planes, in the other one of two places.
int32_t apply(const Call& c, Group* gs, int n, float scale) {
  BuildPlanes b(c);
  for (Group* g = gs; g < gs + n; ++g) {
    const Shape& s = g->s;
    Planes out = g->x;
    out.at = g->planes(g->x.at == g->planes(g->w.x) ? g->w.x1 : g->w.x);
    out.scale = scale;
    terms::Problem& p = b.problem(s.mp, s.np, s.batch, s.mp / dense::kBK);
    EpiPlanes::Args& e = b.l.e[b.l.problems - 1];
    MOE_TRY(b.operand(s, g->q, false, 0, &p.a));
    MOE_TRY(b.operand(s, g->x, true, 0, &p.b));
    e = {};
    e.c = out.scale / (g->q.scale * g->x.scale);
    MOE_TRY(b.map(s, out.at, s.np, 32, 32, dense::Swizzle::k64, &e.map));
    e.lo_rows = static_cast<int32_t>(rows_of(s));
    e.rows = s.mp;
    e.cols = s.np;
    g->x = out;
  }
  return run(c, b);
}

// What a slice has of a tensor: `count` matrices from number `at` on.
struct Part {
  int32_t tensor;
  int64_t at, count, before;   // before: the group's matrices in the tensors ahead
};
// The slice's next part, beginning with {}; false: none.
bool next_part(const Call& c, const Shape& s, Part* part) {
  for (int32_t& i = part->tensor; i < c.count; ++i) {
    if (!same(c.t[i], s)) continue;
    const int64_t n = c.t[i].count, from = std::max(s.first, part->before), to = std::min(s.first + s.batch, part->before + n);
    if (part->count == 0 && from < to) {
      part->at = from - part->before;
      part->count = to - from;
      return true;
    }
    part->count = 0;
    part->before += n;
  }
  return false;
}

// p <- decay p - lr s Q X for the groups' tensors, as many in a launch as it
// holds.
int32_t update(const Call& c, Group* gs, int n) {
  Build<EpiUpdate> b(c);
  auto send = [&]() -> int32_t {
    if (b.l.problems) MOE_CUDA(terms::launch<EpiUpdate>(b.m, b.l, c.pairs_update, c.st));
    b = Build<EpiUpdate>(c);
    return MOE_OK;
  };
  for (Group* g = gs; g < gs + n; ++g) {
    const Shape& s = g->s;
    const int64_t size = static_cast<int64_t>(s.m) * s.n;
    int64_t z = 0;
    for (Part part = {}; next_part(c, s, &part);) {
      const moe_muon_tensor& t = c.t[part.tensor];
      const bool tall = t.rows > t.cols;
      EpiUpdate::Args& e = b.l.e[b.l.problems];
      terms::Problem& p = b.problem(tall ? s.m : s.n, tall ? s.n : s.m, part.count, s.mp / dense::kBK);
      MOE_TRY(b.operand(s, tall ? g->q : g->x, !tall, z, &p.a));
      MOE_TRY(b.operand(s, tall ? g->x : g->q, tall, z, &p.b));
      e.p = t.param + part.at * size;
      e.copy = t.param_bf16 ? static_cast<__nv_bfloat16*>(t.param_bf16) + part.at * size : nullptr;
      e.decay = muon_decay(c.o);
      e.step = static_cast<float>(muon_step(c.o, t) / (static_cast<double>(g->q.scale) * g->x.scale));
      e.rows = tall ? s.m : s.n;
      e.cols = tall ? s.n : s.m;
      z += part.count;
      if (b.l.problems == terms::kMaxProblems) MOE_TRY(send());
    }
  }
  return send();
}

// The momenta and X0's planes of one group.
int32_t first_planes(const Call& c, const Group& g) {
  const Shape& s = g.s;
  float* sums = reinterpret_cast<float*>(g.ws + g.w.sums);
  const int chunks = chunks_of(s);
  const int64_t size = static_cast<int64_t>(s.m) * s.n;
  const bool bf16 = c.o->grad_dtype == MOE_DTYPE_BF16;
  // Matrices whose momentum and gradient stay in L2 go one after another, so
  // that the second reading finds them there; as many small ones at once as do.
  const int64_t at_once = std::min<int64_t>(65535, std::max<int64_t>(1, kL2Bytes / (size * (bf16 ? 6 : 8))));
  int64_t z = 0;
  for (Part p = {}; next_part(c, s, &p);) {
    const moe_muon_tensor& t = c.t[p.tensor];
    Momentum a = {t.grad, t.momentum, c.o->grad_scale, static_cast<float>(c.o->momentum),
                  static_cast<float>(1.0 - c.o->momentum), bf16, c.o->nesterov};
    const int vec = size % 4 == 0 && ptr_aligned(t.momentum, 16) && ptr_aligned(t.grad, bf16 ? 8 : 16);
    const int vec_rows = vec && t.cols % 4 == 0;
    for (int64_t at = 0; at < p.count; at += at_once) {
      const unsigned n = static_cast<unsigned>(std::min<int64_t>(p.count - at, at_once));
      a.m = t.momentum + (p.at + at) * size;
      a.grad = static_cast<const uint8_t*>(t.grad) + (p.at + at) * size * (bf16 ? 2 : 4);
      float* part = sums + (z + at) * chunks;
      MOE_CUDA(launch_pdl(muon_momentum_kernel, dim3(chunks, n), dim3(kThreads), 0, c.st, a, size, chunk_of(s), vec,
                          part));
      MOE_CUDA(launch_pdl(muon_planes_kernel, dim3(s.np / kSide, s.mp / kSide, n), dim3(kThreads), 0, c.st, a,
                          t.rows, t.cols, vec_rows, static_cast<const float*>(part), chunks,
                          static_cast<float>(c.o->eps), c.sc.x[0], g.planes(g.w.x) + (z + at) * s.mp * s.np,
                          rows_of(s) * s.np, s.mp, s.np));
    }
    z += p.count;
  }
  return MOE_OK;
}

// CTAs of a cluster that carries out the steps' m x m products in one launch, or 0:
// each in a launch of its own.  One launch is faster while a phase has a unit of 64
// columns or two a pair and all matrices are resident (256 x 7168: 140 against 167 us,
// 384 x 4096 163 / 190, 3 of 333 x 1001 and 2 of 777 x 129 179 / 213, 12 of 200 x 1000
// 169 / 204); beyond, the whole GPU is (448 x 1000: 223 / 186, 512 x 512 233 / 189).  A
// cluster of 16 takes 2 us off for short sides of up to 256, too, but holds half as many.
int chain_size(const Group* gs, int n, int* error) {
  *error = MOE_OK;
  int mp = 0;
  int64_t matrices = 0;
  for (const Group* g = gs; g < gs + n; ++g) {
    mp = std::max(mp, g->s.mp);
    matrices += g->s.batch;
  }
  if (mp > kChainSide) return 0;
  const int size = mp <= dense::kTile ? 8 : 16;
  int clusters;
  const cudaError_t e = terms::resident_chains<EpiPlanes>(size, &clusters);
  if (e != cudaSuccess) *error = entry_launched(e);
  return e == cudaSuccess && matrices <= clusters ? size : 0;
}

// `steps` steps on G: Q from G, the products of a phase added to b and ended by
// flush().
template <class B, class F>
int32_t add_steps(const Call& c, Group* gs, int n, const StepScales* sc, int steps, B& b, F flush) {
  const float fa = static_cast<float>(c.o->coefficients[0]), fc = static_cast<float>(c.o->coefficients[2]);
  const float ratio = static_cast<float>(c.o->coefficients[1] / c.o->coefficients[2]);
  Group* const end = gs + n;
  for (int k = 0; k < steps; ++k) {
    const bool last = k == steps - 1;
    for (Group* g = gs; g < end; ++g) {   // P = c G (G + (b / c) I) + a I
      g->p = g->square(k == 0 ? g->w.qa : g->w.p, sc[k].p);
      MOE_TRY(add_symmetric(b, g->s, g->g, g->g, true, g->p, fc, fa, 0.f));
    }
    MOE_TRY(flush());
    for (Group* g = gs; g < end; ++g) {   // S = P G, Q <- P Q
      if (!last)
        MOE_TRY(add_symmetric(b, g->s, g->p, g->g, false, g->square(g->w.s, sc[k].s), 1.0f, 0.f, 0.f));
      if (k == 0) {
        g->q = g->p;
      } else {
        const Planes next = g->square(k & 1 ? g->w.qb : g->w.qa, sc[k].q);
        MOE_TRY(add_symmetric(b, g->s, g->p, g->q, false, next, 1.0f, 0.f, 0.f));
        // P Q and not P Q^T: what is left of Q's asymmetry belongs to the X that the
        // next Gram matrix is taken of
        b.l.p[b.l.problems - 1].b.turned = 1;
        g->q = next;
      }
    }
    MOE_TRY(flush());
    if (last) return MOE_OK;
    for (Group* g = gs; g < end; ++g) {   // G <- S P
      g->g.scale = sc[k + 1].g;
      MOE_TRY(add_symmetric(b, g->s, g->square(g->w.s, sc[k].s), g->p, false, g->g, 1.0f, 0.f, ratio));
    }
    MOE_TRY(flush());
  }
  return MOE_OK;
}

// All steps of up to kMostGroups groups, whose products share their launches.
int32_t run_groups(const Call& c, Group* gs, int n) {
  const float ratio = static_cast<float>(c.o->coefficients[1] / c.o->coefficients[2]);
  Group* const end = gs + n;
  int error;
  const int chain = chain_size(gs, n, &error);
  if (error != MOE_OK) return error;
  for (Group* g = gs; g < end; ++g) {
    MOE_TRY(first_planes(c, *g));
    g->x = {g->planes(g->w.x), c.sc.x[0], g->s.np, false, nullptr};
  }
  int part = 0;
  for (int done = 0; done < c.o->ns_steps; done += kPartSteps, ++part) {
    const int steps = std::min(kPartSteps, c.o->ns_steps - done);
    const StepScales* sc = c.sc.step + done;
    for (Group* g = gs; g < end; ++g) {
      g->g = g->square(g->w.g, sc[0].g);
      g->g.diag = g->planes(g->w.h);
    }
    MOE_TRY(gram(c, gs, n, ratio));
    if (chain) {
      BuildChain b(c);
      MOE_TRY(add_steps(c, gs, n, sc, steps, b, [&]() -> int32_t {
        if (b.l.problems > (b.l.phases ? b.l.end[b.l.phases - 1] : 0)) b.l.end[b.l.phases++] = b.l.problems;
        return MOE_OK;
      }));
      int matrices = 0;
      for (Group* g = gs; g < end; ++g) {
        b.l.mp[b.l.groups] = g->s.mp;
        b.l.first[b.l.groups++] = matrices;
        matrices += static_cast<int>(g->s.batch);
      }
      MOE_CUDA(terms::launch_chain<EpiPlanes>(b.m, b.l, chain, matrices, c.st));
    } else {
      BuildPlanes b(c);
      MOE_TRY(add_steps(c, gs, n, sc, steps, b, [&]() -> int32_t {
        MOE_TRY(run(c, b));
        b = BuildPlanes(c);
        return MOE_OK;
      }));
    }
    if (done + steps < c.o->ns_steps) MOE_TRY(apply(c, gs, n, c.sc.x[part + 1]));
  }
  return update(c, gs, n);
}

int32_t check_tensor(const moe_muon_tensor& t, int i, bool bf16) {
  if (t.count < 0 || t.rows < 0 || t.cols < 0)
    return entry_fail(MOE_ERR_INVALID_ARG, "tensor %d: a negative size", i);
  if (t.reserved) return entry_fail(MOE_ERR_INVALID_ARG, "tensor %d: reserved must be zero", i);
  if (muon_empty(t)) return MOE_OK;
  if (!t.param || !t.grad || !t.momentum)
    return entry_fail(MOE_ERR_INVALID_ARG, "tensor %d: param, grad or momentum is NULL", i);
  if (t.rows > MOE_MUON_MAX_SIDE || t.cols > MOE_MUON_MAX_SIDE || std::min(t.rows, t.cols) > MOE_MUON_MAX_SHORT)
    return entry_fail(MOE_ERR_UNSUPPORTED, "tensor %d: sides of at most %d, the shorter at most %d", i,
                      MOE_MUON_MAX_SIDE, MOE_MUON_MAX_SHORT);
  if (!ptr_aligned(t.param, 4) || !ptr_aligned(t.grad, bf16 ? 2 : 4) || !ptr_aligned(t.momentum, 4) ||
      !ptr_aligned(t.param_bf16, 2))
    return entry_fail(MOE_ERR_MISALIGNED, "tensor %d: a pointer is not aligned to its type", i);
  return MOE_OK;
}

int32_t check_call(const moe_muon_tensor* t, int32_t count, const moe_muon_options* o, Scales* sc) {
  if (!o) return entry_fail(MOE_ERR_INVALID_ARG, "options is NULL");
  if (count < 0) return entry_fail(MOE_ERR_INVALID_ARG, "count < 0");
  if (count > 0 && !t) return entry_fail(MOE_ERR_INVALID_ARG, "tensors is NULL");
  if (o->grad_dtype != MOE_DTYPE_F32 && o->grad_dtype != MOE_DTYPE_BF16)
    return entry_fail(MOE_ERR_INVALID_ARG, "grad_dtype %d unknown", o->grad_dtype);
  if (o->update_scale != MOE_MUON_RMS && o->update_scale != MOE_MUON_SPECTRAL)
    return entry_fail(MOE_ERR_INVALID_ARG, "update_scale %d unknown", o->update_scale);
  if (!(o->momentum >= 0 && o->momentum < 1))
    return entry_fail(MOE_ERR_INVALID_ARG, "momentum must be in [0, 1)");
  // (with the sum of u^2 in float: a norm that underflows leaves X bounded)
  if (!(o->eps >= 1e-16) || !std::isfinite(o->eps) || !std::isfinite(o->lr) || !std::isfinite(o->weight_decay))
    return entry_fail(MOE_ERR_INVALID_ARG, "lr, eps and weight_decay must be finite, eps at least 1e-16");
  if (o->ns_steps < 1 || o->ns_steps > kMaxSteps)
    return entry_fail(MOE_ERR_INVALID_ARG, "ns_steps must be in [1, %d]", kMaxSteps);
  if (o->reserved[0] || o->reserved[1]) return entry_fail(MOE_ERR_INVALID_ARG, "reserved must be zero");
  if (!ptr_aligned(o->grad_scale, 4))
    return entry_fail(MOE_ERR_MISALIGNED, "grad_scale must be 4-byte aligned");
  if (!std::isfinite(o->coefficients[0]) || !std::isfinite(o->coefficients[2]) ||
      o->coefficients[2] == 0 ||
      !(std::fabs(o->coefficients[1]) <= 64 * std::fabs(o->coefficients[2])))
    return entry_fail(MOE_ERR_UNSUPPORTED, "coefficients (%g, %g, %g): c must be at least |b| / 64", o->coefficients[0],
                      o->coefficients[1], o->coefficients[2]);
  if (!make_scales(o, sc))
    return entry_fail(MOE_ERR_UNSUPPORTED, "the Newton-Schulz steps of these coefficients grow without bound");
  for (int i = 0; i < count; ++i) MOE_TRY(check_tensor(t[i], i, o->grad_dtype == MOE_DTYPE_BF16));
  return MOE_OK;
}

// (More matrices than any GPU holds: a slice's indices stay within 32 bits.)
int32_t check_group(const Shape& s) {
  if (2 * s.all * s.mp >= (int64_t(1) << 31) || s.all * chunks_of(s) >= (int64_t(1) << 31) ||
      s.all * dense::cdiv(s.mp, 128) * dense::cdiv(s.np, 128) >= (int64_t(1) << 31))
    return entry_fail(MOE_ERR_UNSUPPORTED, "too many matrices of %d x %d", s.m, s.n);
  return MOE_OK;
}

// A slice is as many matrices as this much workspace holds, and one at least.  All at once
// take as much as they are many (256 experts' 768 of 2048 x 1024: 27.8 GiB) and gain what a
// slice's last rounds of tiles leave idle: 768 of 2048 x 1024 62.6 ms at once, in slices of 4 GiB
// 63.5, of 2 65.4, of 1 68.9; 96 of 2048 x 7168 67.2 / 68.2 / 69.7 / 72.3; 1600 of 512 x 512
// 18.3 / 18.8 / 19.6 / 20.9.
constexpr size_t kSliceBytes = size_t(4) << 30;
// The slice that follows `s` (batch 0: the first); false: none.
bool next_slice(Shape* s) {
  if (s->batch == 0) {
    Shape one = *s;
    one.batch = 1;
    one.each = dense::kPlanPairs;   // (without the shares that few matrices' sums are split into, some MB)
    const int64_t most = std::max<int64_t>(1, kSliceBytes / group_ws(one).total);
    s->each = dense::cdiv(s->all, dense::cdiv(s->all, most));
    s->first = 0;
  } else {
    s->first += s->batch;
  }
  s->batch = std::min(s->each, s->all - s->first);
  return s->batch > 0;
}

// The next group at or after tensor *i, whose first tensor it is; false: none.
bool next_shape(const moe_muon_tensor* t, int32_t count, int32_t* i, Shape* s) {
  for (; *i < count; ++*i) {
    if (muon_empty(t[*i]) || muon_is_small(t[*i])) continue;
    *s = shape_of(t[*i]);
    bool seen = false;
    for (int j = 0; j < *i && !seen; ++j) seen = same(t[j], *s);
    if (seen) continue;
    for (int j = *i; j < count; ++j)
      if (same(t[j], *s)) s->all += t[j].count;
    ++*i;
    return true;
  }
  return false;
}

// Calls f with each set of slices that share their launches (and the bytes that
// they need), in the order of their groups' first tensors: as many as kMostGroups and
// the memory of the largest slice, or kSharedBytes, hold.  Stops at the first
// error.
constexpr size_t kSharedBytes = size_t(256) << 20;
template <class F>
int32_t each_set(const moe_muon_tensor* t, int32_t count, F f) {
  size_t most = kSharedBytes;
  Shape s;
  for (int32_t i = 0; next_shape(t, count, &i, &s);) {
    next_slice(&s);   // the others have no more matrices
    MOE_TRY(check_group(s));
    most = std::max(most, group_ws(s).total);
  }
  Group set[kMostGroups] = {};
  int n = 0;
  size_t bytes = 0;
  for (int32_t i = 0; next_shape(t, count, &i, &s);) {
    while (next_slice(&s)) {
      const GroupWs w = group_ws(s);
      if (n == kMostGroups || (n && bytes + w.total > most)) {
        MOE_TRY(f(set, n, bytes));
        n = 0;
        bytes = 0;
      }
      set[n].s = s;
      set[n++].w = w;
      bytes += w.total;
    }
  }
  return n ? f(set, n, bytes) : MOE_OK;
}

int32_t total_ws(const moe_muon_tensor* t, int32_t count, size_t* need) {
  *need = std::max(kWsAlign, muon_small_ws(t, count));
  return each_set(t, count, [&](Group*, int, size_t bytes) -> int32_t {
    *need = std::max(*need, bytes);
    return MOE_OK;
  });
}

}  // namespace

bool muon_empty(const moe_muon_tensor& t) { return t.count == 0 || t.rows == 0 || t.cols == 0; }
float muon_decay(const moe_muon_options* o) { return static_cast<float>(1.0 - o->lr * o->weight_decay); }
double muon_step(const moe_muon_options* o, const moe_muon_tensor& t) {
  const double rows = t.rows, cols = t.cols;
  return o->lr * (o->update_scale == MOE_MUON_RMS ? 0.2 * std::sqrt(std::max(rows, cols))
                                                  : std::sqrt(std::max(1.0, rows / cols)));
}

}  // namespace moe

extern "C" size_t moe_muon_workspace_size(const moe_muon_tensor* tensors, int32_t count,
                                          const moe_muon_options* options) {
  using namespace moe;
  Scales sc;
  size_t need;
  if (check_call(tensors, count, options, &sc) != MOE_OK || total_ws(tensors, count, &need) != MOE_OK) return 0;
  return need;
}

extern "C" int32_t moe_muon_step(const moe_muon_tensor* tensors, int32_t count, const moe_muon_options* o,
                                 void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
  using namespace moe;
  Call g = {};
  size_t need;
  MOE_TRY(check_call(tensors, count, o, &g.sc));
  MOE_TRY(total_ws(tensors, count, &need));
  bool any = false;
  for (int i = 0; i < count; ++i) any = any || !muon_empty(tensors[i]);
  if (!any) return MOE_OK;
  if (!status) return entry_fail(MOE_ERR_INVALID_ARG, "status is NULL");
  if (!ptr_aligned(status, 4)) return entry_fail(MOE_ERR_MISALIGNED, "status must be 4-byte aligned");
  if (!workspace) return entry_fail(MOE_ERR_INVALID_ARG, "workspace is NULL");
  if (!ptr_aligned(workspace, kWsAlign))
    return entry_fail(MOE_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  if (workspace_bytes < need)
    return entry_fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  int sms = 0;
  MOE_TRY(check_device(&sms));
  MOE_CUDA(terms::resident_pairs<EpiPlanes>(sms, &g.pairs_planes));
  MOE_CUDA(terms::resident_pairs<EpiUpdate>(sms, &g.pairs_update));
  MOE_CUDA(terms::resident_pairs<EpiShare>(sms, &g.pairs_share));
  g.t = tensors;
  g.count = count;
  g.o = o;
  g.status = status;
  g.st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  MOE_TRY(muon_small_step(tensors, count, o, ws, g.st));
  return each_set(tensors, count, [&](Group* set, int n, size_t) -> int32_t {
    size_t at = 0;
    for (int i = 0; i < n; ++i) {
      set[i].ws = ws + at;
      at += set[i].w.total;
    }
    return run_groups(g, set, n);
  });
}
