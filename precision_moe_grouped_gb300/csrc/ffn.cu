// ffn.cu -- a gated feed-forward block in bf16 and its gradients: the shared
// expert, or a dense layer, beside the routed experts.
//
//   g = x Wg^T, u = x Wu^T, h = silu(g) u, out = base + h Wd^T
//   dh = dout Wd, s = sigmoid(g): du = dh g s, dg = dh u s (1 + g (1 - s))
//   dx = dx_base + dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dWd = dout^T h
//
// Sums are float; h, dg and du enter the second products as bf16, each
// rounded once (half a step of 2^-8), as the outputs are: an output's error is
// then about sqrt(2) of its own rounding's.
#include <cuda_bf16.h>

#include <algorithm>

#include "dense.cuh"
#include "entry.h"

namespace moe {
namespace {

using dense::Elem;
using dense::EpiWarp;
using dense::Maps;
using dense::Problem;
using dense::Tile;

constexpr uint64_t kTimeoutNs = 1000000000ull;
constexpr int kDecodeTokens = 32;   // at most: the products that stream the weights once

// ------------------------------------------------------------- activation
// silu(g) = g / (1 + e^-g), its factor s = 1 / (1 + e^-g): fast exponential and
// division (relative error about 1e-6, far below the bf16 rounding that follows).
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }
__device__ __forceinline__ float swiglu(float g, float u) {
  return __fdividef(g, 1.0f + __expf(-g)) * u;
}
struct Grads {
  float h, dg, du;
};
__device__ __forceinline__ Grads swiglu_grads(float g, float u, float dh) {
  const float s = sigmoid(g), a = g * s;
  return {a * u, dh * u * (s * (1.0f + g * (1.0f - s))), dh * a};
}

// -------------------------------------------------------------- epilogues
// bf16 out = base + D.
struct EpiOut {
  struct Args {
    const __nv_bfloat16* base;   // or null
    int64_t ld_base;
    int32_t map, rows, cols;
  };
  static __device__ __forceinline__ void run(const Args& a, const Problem& p, const Tile& o,
                                             const EpiWarp& w, const Maps& maps) {
    if (w.row >= a.rows) return;
    const int c0 = w.half * (p.bn >> 1);
    const bool mine = w.row + w.lane < a.rows;
    for (int c = c0; c < c0 + (p.bn >> 1); c += 64) {
      const int col = o.j * p.bn + c;
      if (col >= a.cols) return;
      uint32_t lo[32], hi[32];
      dense::tmem_ld_x32(w.tmem + c, lo);
      dense::tmem_ld_x32(w.tmem + c + 32, hi);
      uint4 b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        b[i] = make_uint4(0, 0, 0, 0);
        if (a.base && mine && col + 8 * i < a.cols)
          b[i] = *reinterpret_cast<const uint4*>(a.base + (w.row + w.lane) * a.ld_base + col + 8 * i);
      }
      dense::tmem_wait(lo);
      dense::tmem_wait(hi);
      if (w.lane == 0) dense::box_wait_read();
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t* v = i < 4 ? lo + 8 * i : hi + 8 * (i - 4);
        uint32_t r[4];
        const uint32_t bb[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = dense::unpack_bf16(bb[k]);
          r[k] = dense::pack_bf16(__uint_as_float(v[2 * k]) + f.x, __uint_as_float(v[2 * k + 1]) + f.y);
        }
        *dense::box_piece(w.box, w.lane, i) = make_uint4(r[0], r[1], r[2], r[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (w.lane == 0) dense::box_store(&maps.m[a.map], w.box, col, w.row);
    }
  }
};

// Float sums as they are: shares of K, or what a later kernel's epilogue reads.
// Row r of share s goes to row s rows_pad + r, rows_pad a multiple of 32.
struct EpiSum {
  struct Args {
    int32_t map, rows_pad, cols;
  };
  static __device__ __forceinline__ void run(const Args& a, const Problem& p, const Tile& o,
                                             const EpiWarp& w, const Maps& maps) {
    if (w.row >= a.rows_pad) return;
    const int c0 = w.half * (p.bn >> 1);
    for (int c = c0; c < c0 + (p.bn >> 1); c += 32) {
      const int col = o.j * p.bn + c;
      if (col >= a.cols) return;
      uint32_t v[32];
      dense::tmem_ld_x32(w.tmem + c, v);
      dense::tmem_wait(v);
      if (w.lane == 0) dense::box_wait_read();
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *dense::box_piece(w.box, w.lane, i) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      fence_proxy_async_smem();
      __syncwarp();
      if (w.lane == 0) dense::box_store(&maps.m[a.map], w.box, col, o.s * a.rows_pad + w.row);
    }
  }
};

// A warp's 32 features [f, f + 32) as bf16 through its box, at the box's
// column 32 * part; the store follows when the box's last part is written
// (64 features), or at once (alone: one part of 32).
__device__ __forceinline__ void put_features(const uint32_t (&v)[16], const EpiWarp& w, int part) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *dense::box_piece(w.box, w.lane, 4 * part + i) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}
__device__ __forceinline__ void row_features(const uint32_t (&v)[16], __nv_bfloat16* row, int f, int I) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (f + 8 * i < I)
      *reinterpret_cast<uint4*>(row + f + 8 * i) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

// h = silu(g) u; D's columns: bn / 2 of the gate's, then the same features' up.
struct EpiGate {
  struct Args {
    __nv_bfloat16* h;   // [T, I]
    int32_t map, rows, inter;
  };
  static __device__ __forceinline__ void run(const Args& a, const Problem& p, const Tile& o,
                                             const EpiWarp& w, const Maps& maps) {
    if (w.row >= a.rows) return;
    const int n = p.bn >> 2;   // 64 or 32 features of this warp's half
    const int f0 = o.j * p.b_step + w.half * n;
    if (f0 >= a.inter) return;
    const bool mine = w.row + w.lane < a.rows;
    for (int part = 0; part < n / 32; ++part) {
      uint32_t g[32], u[32], r[16];
      dense::tmem_ld_x32(w.tmem + w.half * n + 32 * part, g);
      dense::tmem_ld_x32(w.tmem + (p.bn >> 1) + w.half * n + 32 * part, u);
      dense::tmem_wait(g);
      dense::tmem_wait(u);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        r[i] = dense::pack_bf16(swiglu(__uint_as_float(g[2 * i]), __uint_as_float(u[2 * i])),
                                swiglu(__uint_as_float(g[2 * i + 1]), __uint_as_float(u[2 * i + 1])));
      if (n == 64) {
        if (part == 0) {
          if (w.lane == 0) dense::box_wait_read();
          __syncwarp();
        }
        put_features(r, w, part);
      } else if (mine) {
        row_features(r, a.h + static_cast<int64_t>(w.row + w.lane) * a.inter, f0, a.inter);
      }
    }
    if (n == 64) {
      fence_proxy_async_smem();
      __syncwarp();
      if (w.lane == 0) dense::box_store(&maps.m[a.map], w.box, f0, w.row);
    }
  }
};

// h, dg and du from D (as EpiGate's) and dh.
struct EpiGateGrad {
  struct Args {
    __nv_bfloat16 *h, *dgu;   // [T, I], [T, 2 I]
    const float* dh;          // [rows rounded up to 32, ld_dh]
    int64_t ld_dh;
    int32_t rows, inter;
  };
  static __device__ __forceinline__ void run(const Args& a, const Problem& p, const Tile& o,
                                             const EpiWarp& w, const Maps& maps) {
    if (w.row >= a.rows) return;
    const int n = p.bn >> 2;
    const int f0 = o.j * p.b_step + w.half * n;
    const bool mine = w.row + w.lane < a.rows;
    const int64_t row = w.row + w.lane;
    for (int part = 0; part < n / 32; ++part) {
      const int f = f0 + 32 * part;
      if (f >= a.inter) return;
      uint32_t g[32], u[32], rh[16], rg[16], ru[16];
      dense::tmem_ld_x32(w.tmem + w.half * n + 32 * part, g);
      dense::tmem_ld_x32(w.tmem + (p.bn >> 1) + w.half * n + 32 * part, u);
      float4 d[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        d[i] = mine && f + 4 * i < a.inter ? *reinterpret_cast<const float4*>(a.dh + row * a.ld_dh + f + 4 * i)
                                           : make_float4(0, 0, 0, 0);
      dense::tmem_wait(g);
      dense::tmem_wait(u);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float d0 = i & 1 ? d[i >> 1].z : d[i >> 1].x, d1 = i & 1 ? d[i >> 1].w : d[i >> 1].y;
        const Grads x = swiglu_grads(__uint_as_float(g[2 * i]), __uint_as_float(u[2 * i]), d0);
        const Grads y = swiglu_grads(__uint_as_float(g[2 * i + 1]), __uint_as_float(u[2 * i + 1]), d1);
        rh[i] = dense::pack_bf16(x.h, y.h);
        rg[i] = dense::pack_bf16(x.dg, y.dg);
        ru[i] = dense::pack_bf16(x.du, y.du);
      }
      if (mine) {
        row_features(rh, a.h + row * a.inter, f, a.inter);
        row_features(rg, a.dgu + row * 2 * a.inter, f, a.inter);
        row_features(ru, a.dgu + row * 2 * a.inter + a.inter, f, a.inter);
      }
    }
  }
};

// ------------------------------------------------------- joining K's shares
// Batches of few hundred tokens: the weights are the 256 rows of a tile, the
// tokens its columns, and K is shared out until the pairs are busy.  Sums are
// [shares][rows][tp], the tokens side by side; a block joins 16 features of 64
// tokens, four tokens of a feature a thread, and turns them through shared
// memory, so that both sides are met in long runs.
constexpr int kJoinThreads = 256, kJoinFeatures = 16, kJoinTokens = 64;   // a feature's four tokens a thread

struct Sums {
  const float* at;
  int32_t shares, rows, tp;
};
// Four tokens from t on of row r, over the shares in order; the loads of up to
// eight shares are in flight together.
struct Joined {
  float4 v[8];

  __device__ __forceinline__ void load(const Sums& s, int r, int t, int first) {
    const float* p = s.at + static_cast<int64_t>(r) * s.tp + t;
    const int64_t step = static_cast<int64_t>(s.rows) * s.tp;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (first + i < s.shares) v[i] = *reinterpret_cast<const float4*>(p + (first + i) * step);
  }
  __device__ __forceinline__ float4 sum(const Sums& s, int r, int t) {
    float4 x = v[0];
    for (int first = 0;;) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (first + i < s.shares && first + i > 0)
          x = make_float4(x.x + v[i].x, x.y + v[i].y, x.z + v[i].z, x.w + v[i].w);
      }
      if ((first += 8) >= s.shares) return x;
      load(s, r, t, first);
    }
  }
};

struct Turned {
  __nv_bfloat16 v[kJoinTokens][kJoinFeatures + 8];   // rows 48 bytes apart

  __device__ __forceinline__ void put(int f, int t, float4 x) {
    v[t][f] = __float2bfloat16_rn(x.x);
    v[t + 1][f] = __float2bfloat16_rn(x.y);
    v[t + 2][f] = __float2bfloat16_rn(x.z);
    v[t + 3][f] = __float2bfloat16_rn(x.w);
  }
  // this thread's eight features of one token
  __device__ __forceinline__ void send(__nv_bfloat16* to, int64_t ld, int f0, int t0, int features, int tokens) const {
    const int t = threadIdx.x >> 1, f = (threadIdx.x & 1) * 8;
    if (t < kJoinTokens && t0 + t < tokens && f0 + f < features)
      *reinterpret_cast<uint4*>(to + static_cast<int64_t>(t0 + t) * ld + f0 + f) =
          *reinterpret_cast<const uint4*>(&v[t][f]);
  }
};

// h from x [Wg; Wu]^T.
__global__ void __launch_bounds__(kJoinThreads)
    join_gate_kernel(const Sums s, int tokens, int inter, __nv_bfloat16* h) {
  __shared__ __align__(16) Turned turned;
  griddep_wait();
  griddep_launch_dependents();
  const int f0 = blockIdx.x * kJoinFeatures, t0 = blockIdx.y * kJoinTokens;
  const int t = (threadIdx.x & 15) * 4;
  const int f = threadIdx.x >> 4;
  if (f0 + f < inter) {
    Joined jg, ju;
    jg.load(s, f0 + f, t0 + t, 0);
    ju.load(s, inter + f0 + f, t0 + t, 0);
    const float4 g = jg.sum(s, f0 + f, t0 + t), u = ju.sum(s, inter + f0 + f, t0 + t);
    turned.put(f, t, make_float4(swiglu(g.x, u.x), swiglu(g.y, u.y), swiglu(g.z, u.z), swiglu(g.w, u.w)));
  }
  __syncthreads();
  turned.send(h, inter, f0, t0, inter, tokens);
}

// out = base + the sums: added in float, rounded once.
__global__ void __launch_bounds__(kJoinThreads)
    join_out_kernel(const Sums s, int tokens, int cols, const __nv_bfloat16* base, int64_t ld_base,
                    __nv_bfloat16* out, int64_t ld_out) {
  __shared__ __align__(16) float turned[kJoinTokens][kJoinFeatures + 4];
  griddep_wait();
  griddep_launch_dependents();
  const int f0 = blockIdx.x * kJoinFeatures, t0 = blockIdx.y * kJoinTokens;
  const int t = (threadIdx.x & 15) * 4;
  const int feature = threadIdx.x >> 4;
  if (f0 + feature < cols) {
    Joined j;
    j.load(s, f0 + feature, t0 + t, 0);
    const float4 v = j.sum(s, f0 + feature, t0 + t);
    turned[t][feature] = v.x;
    turned[t + 1][feature] = v.y;
    turned[t + 2][feature] = v.z;
    turned[t + 3][feature] = v.w;
  }
  __syncthreads();
  const int tt = threadIdx.x >> 1, f = (threadIdx.x & 1) * 8;
  if (tt >= kJoinTokens || t0 + tt >= tokens || f0 + f >= cols) return;
  uint4 b = make_uint4(0, 0, 0, 0);
  if (base) b = *reinterpret_cast<const uint4*>(base + (t0 + tt) * ld_base + f0 + f);
  const uint32_t bb[4] = {b.x, b.y, b.z, b.w};
  uint32_t r[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = dense::unpack_bf16(bb[k]);
    r[k] = dense::pack_bf16(turned[tt][f + 2 * k] + x.x, turned[tt][f + 2 * k + 1] + x.y);
  }
  *reinterpret_cast<uint4*>(out + (t0 + tt) * ld_out + f0 + f) = make_uint4(r[0], r[1], r[2], r[3]);
}

// h, dg, du from x [Wg; Wu]^T and dout Wd.
__global__ void __launch_bounds__(kJoinThreads)
    join_grad_kernel(const Sums gu, const Sums dh, int tokens, int inter, __nv_bfloat16* h, __nv_bfloat16* dgu) {
  __shared__ __align__(16) Turned th, tg, tu;
  griddep_wait();
  griddep_launch_dependents();
  const int f0 = blockIdx.x * kJoinFeatures, t0 = blockIdx.y * kJoinTokens;
  const int t = (threadIdx.x & 15) * 4;
  const int f = threadIdx.x >> 4;
  if (f0 + f < inter) {
    Joined jg, ju, jd;
    jg.load(gu, f0 + f, t0 + t, 0);
    ju.load(gu, inter + f0 + f, t0 + t, 0);
    jd.load(dh, f0 + f, t0 + t, 0);
    const float4 g = jg.sum(gu, f0 + f, t0 + t), u = ju.sum(gu, inter + f0 + f, t0 + t);
    const float4 d = jd.sum(dh, f0 + f, t0 + t);
    const Grads a = swiglu_grads(g.x, u.x, d.x), b = swiglu_grads(g.y, u.y, d.y);
    const Grads c = swiglu_grads(g.z, u.z, d.z), e = swiglu_grads(g.w, u.w, d.w);
    th.put(f, t, make_float4(a.h, b.h, c.h, e.h));
    tg.put(f, t, make_float4(a.dg, b.dg, c.dg, e.dg));
    tu.put(f, t, make_float4(a.du, b.du, c.du, e.du));
  }
  __syncthreads();
  th.send(h, inter, f0, t0, inter, tokens);
  tg.send(dgu, 2 * static_cast<int64_t>(inter), f0, t0, inter, tokens);
  tu.send(dgu + inter, 2 * static_cast<int64_t>(inter), f0, t0, inter, tokens);
}

// ------------------------------------------------------ batches of few tokens
// Up to 32 tokens: a product is the weights streamed once from HBM.  A CTA
// takes an equal share of the output rows, its eight warps share K; a lane
// loads 16 bytes of a weight row (K order is free as long as both operands
// use the same: lane t of a quad holds elements 8 t .. 8 t + 7 of each 32), and
// mma.sync.m16n8k16 takes 16 weight rows against eight tokens, straight from
// the registers.  The next steps' loads are issued ahead of a step's products
// (64 KB an SM in flight); none hangs on a condition, as rows and tokens beyond
// the end read a valid one and are not stored.  The warps' sums are joined in
// shared memory in warp order.  The first product's CTAs ask L2 for the second
// one's weights when their own are loaded, so that HBM works through the change
// of kernels.
constexpr int kDecodeThreads = 256, kDecodeWarps = 8;
constexpr int64_t kAheadBytes = 32 << 20;   // of the next weights that L2 is asked for

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load_once(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

struct DecodeArgs {
  const __nv_bfloat16* w;      // [rows, K]
  const __nv_bfloat16* in;     // [T, K], rows ld_in apart
  const __nv_bfloat16* base;   // DOWN: added, or null
  __nv_bfloat16* out;
  int64_t ld_in, ld_base, ld_out;
  int32_t tokens, units, k;    // units: features (two weight rows each), or rows
  const uint8_t* next;         // the next product's weights, [next_rows] of next_row bytes
  int32_t next_rows, next_row;
  int64_t next_most;           // of them, bytes a CTA asks for at most
};

// MT: tiles of 16 weight rows at once; NT: of eight tokens; U: K steps of 32
// that are loaded together.
template <bool DOWN, int MT, int NT, int U>
struct DecodeStep {
  uint4 w[U][MT][2], x[U][NT];

  __device__ __forceinline__ static int column(int s, int i, int t, int K) {
    const int k = (s + i) * 32 + 8 * t;
    return k < K ? k : 0;
  }
  __device__ __forceinline__ void load_w(const __nv_bfloat16* const (&rows)[MT][2], int s, int t, int K) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int k = column(s, i, t, K);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j) w[i][m][j] = load_once(rows[m][j] + k);
    }
  }
  __device__ __forceinline__ void load_x(const __nv_bfloat16* const (&rows)[NT], int s, int t, int K) {
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n) x[i][n] = *reinterpret_cast<const uint4*>(rows[n] + column(s, i, t, K));
  }
  __device__ __forceinline__ void multiply(float (&acc)[MT][NT][4], int s, int s1, int t, int K) {
    if (s + U > s1 || (s + U) * 32 > K) {   // nothing beyond the warp's share or the end of K
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (s + i < s1 && (s + i) * 32 + 8 * t < K) continue;
#pragma unroll
        for (int m = 0; m < MT; ++m) w[i][m][0] = w[i][m][1] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int n = 0; n < NT; ++n) x[i][n] = make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 &p = w[i][m][0], &q = w[i][m][1], &v = x[i][n];
          mma_bf16(acc[m][n], p.x, q.x, p.y, q.y, v.x, v.y);
          mma_bf16(acc[m][n], p.z, q.z, p.w, q.w, v.z, v.w);
        }
  }
};

template <bool DOWN, int MT, int NT, int U>
__global__ void __launch_bounds__(kDecodeThreads)
    decode_kernel(const DecodeArgs a) {
  constexpr int MS = MT * NT > 12 ? MT / 2 : MT;   // tiles whose sums are joined together
  __shared__ float sums[kDecodeWarps][MS * NT * 4][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int K = a.k, steps = (K + 31) >> 5;
  const int s0 = static_cast<int>(static_cast<int64_t>(steps) * warp / kDecodeWarps);
  const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (warp + 1) / kDecodeWarps);
  const int u0 = static_cast<int>(static_cast<int64_t>(a.units) * blockIdx.x / gridDim.x);
  const int u1 = static_cast<int>(static_cast<int64_t>(a.units) * (blockIdx.x + 1) / gridDim.x);
  constexpr int kPer = DOWN ? 16 : 8;   // units of a tile
  const __nv_bfloat16* xr[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) xr[n] = a.in + (8 * n + g < a.tokens ? 8 * n + g : 0) * a.ld_in;
  if constexpr (!DOWN) {
    griddep_wait();
    griddep_launch_dependents();
  }
  bool waited = !DOWN;
  for (int u = u0; u < u1; u += MT * kPer) {
    float acc[MT][NT][4] = {};
    // the lane's two weight rows of each tile (g and g + 8 of the MMA's 16)
    const __nv_bfloat16* rows[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int lo = u + m * kPer + g, hi = DOWN ? lo + 8 : lo;
      rows[m][0] = a.w + static_cast<int64_t>(lo < u1 ? lo : u0) * K;
      rows[m][1] = a.w + static_cast<int64_t>((hi < u1 ? hi : u0) + (DOWN ? 0 : a.units)) * K;
    }
    DecodeStep<DOWN, MT, NT, U> even, odd;
    if (s0 < s1) even.load_w(rows, s0, t, K);
    if (!waited) {   // the weights are the call's inputs, h is the kernel before's
      griddep_wait();
      griddep_launch_dependents();
      waited = true;
    }
    if (s0 < s1) even.load_x(xr, s0, t, K);
    for (int s = s0; s < s1; s += 2 * U) {
      if (s + U < s1) {
        odd.load_w(rows, s + U, t, K);
        odd.load_x(xr, s + U, t, K);
      }
      even.multiply(acc, s, s1, t, K);
      if (s + 2 * U < s1) {
        even.load_w(rows, s + 2 * U, t, K);
        even.load_x(xr, s + 2 * U, t, K);
      }
      if (s + U < s1) odd.multiply(acc, s + U, s1, t, K);
    }
    if (!DOWN && u + MT * kPer >= u1) {
      // this CTA's rows of the next weights, 4 KB a request
      const int64_t n0 = static_cast<int64_t>(a.next_rows) * blockIdx.x / gridDim.x * a.next_row;
      const int64_t n1 = min(static_cast<int64_t>(a.next_rows) * (blockIdx.x + 1) / gridDim.x * a.next_row,
                             n0 + a.next_most);
      for (int64_t at = n0 + 4096 * threadIdx.x; at < n1; at += 4096 * kDecodeThreads)
        bulk_prefetch_l2(a.next + at, static_cast<uint32_t>(n1 - at < 4096 ? n1 - at : 4096));
    }
#pragma unroll
    for (int m0 = 0; m0 < MT; m0 += MS) {
#pragma unroll
      for (int m = 0; m < MS; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) sums[warp][(m * NT + n) * 4 + i][lane] = acc[m0 + m][n][i];
      __syncthreads();
      // value i of (tile m, token tile n): row g + 8 (i >> 1), token 2 t + (i & 1)
      for (int at = threadIdx.x; at < MS * NT * (DOWN ? 4 : 2) * 32; at += kDecodeThreads) {
        const int l = at & 31, v = at >> 5;
        const int i = DOWN ? v & 3 : v & 1, mn = DOWN ? v >> 2 : v >> 1;
        const int n = mn % NT, m = m0 + mn / NT;
        const int token = 8 * n + 2 * (l & 3) + (i & 1);
        const int unit = u + m * kPer + (l >> 2) + (DOWN ? 8 * (i >> 1) : 0);
        if (token >= a.tokens || unit >= u1) continue;
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int j = 0; j < kDecodeWarps; ++j) {
          x += sums[j][mn * 4 + i][l];
          if constexpr (!DOWN) y += sums[j][mn * 4 + i + 2][l];
        }
        if constexpr (DOWN) {
          if (a.base) x += __bfloat162float(a.base[token * a.ld_base + unit]);
          a.out[token * a.ld_out + unit] = __float2bfloat16_rn(x);
        } else {
          a.out[token * a.ld_out + unit] = __float2bfloat16_rn(swiglu(x, y));
        }
      }
      __syncthreads();
    }
  }
  if (DOWN && !waited) griddep_wait();
}

template <bool DOWN, int MT, int NT>
cudaError_t launch_decode(const DecodeArgs& a, int grid, cudaStream_t s) {
  // about as many bytes in flight whatever the rows, as far as the registers go
  constexpr int U = (NT == 1 ? 2 : 1) * (MT == 1 ? 4 : MT == 4 ? 1 : 2);
  return launch_pdl(decode_kernel<DOWN, MT, NT, U>, dim3(static_cast<unsigned>(grid)), dim3(kDecodeThreads), 0, s, a);
}
// The tiles of weight rows at once with which a CTA loads the least: each pass
// over its rows reads MT KB of them and NT / 2 KB of x a step of K, rows beyond
// its own included.
template <bool DOWN, int NT>
cudaError_t launch_decode(const DecodeArgs& a, int sms, cudaStream_t s) {
  const int grid = static_cast<int>(std::min<int64_t>(sms, (a.units + 7) / 8));
  const int tiles = static_cast<int>(dense::cdiv(dense::cdiv(a.units, grid), DOWN ? 16 : 8));
  int best = 0, least = 0;
  for (int mt = 1; mt <= 4; ++mt) {
    const int loads = static_cast<int>(dense::cdiv(tiles, mt)) * (2 * mt + NT);
    if (best && loads >= least) continue;
    best = mt;
    least = loads;
  }
  return best == 1   ? launch_decode<DOWN, 1, NT>(a, grid, s)
         : best == 2 ? launch_decode<DOWN, 2, NT>(a, grid, s)
         : best == 3 ? launch_decode<DOWN, 3, NT>(a, grid, s)
                     : launch_decode<DOWN, 4, NT>(a, grid, s);
}
template <bool DOWN>
cudaError_t launch_decode(const DecodeArgs& a, int sms, cudaStream_t s) {
  const int nt = (a.tokens + 7) / 8;
  return nt <= 1   ? launch_decode<DOWN, 1>(a, sms, s)
         : nt == 2 ? launch_decode<DOWN, 2>(a, sms, s)
         : nt == 3 ? launch_decode<DOWN, 3>(a, sms, s)
                   : launch_decode<DOWN, 4>(a, sms, s);
}

// ------------------------------------------------------------------- plans
constexpr int64_t up32(int64_t v) { return (v + 31) / 32 * 32; }

// A product whose tokens are the columns of a tile (of two or more equal ones above
// 256): weights [rows, K], K shared out over the pairs, at least four blocks a
// share.
struct TurnPlan : dense::Plan {
  int32_t tp;   // tokens of all tiles
};
TurnPlan turned_plan(int64_t tokens, int64_t rows, int64_t kb, int64_t pairs) {
  TurnPlan p;
  const int64_t tn = std::max<int64_t>(1, dense::cdiv(tokens, 256));
  p.bn = static_cast<int32_t>((dense::cdiv(tokens, tn) + 63) / 64 * 64);
  p.tp = static_cast<int32_t>(tn * p.bn);
  const int64_t tiles = dense::cdiv(rows, dense::kTile) * tn;
  const int64_t s = std::max<int64_t>(1, std::min(pairs / tiles, kb / 4));
  p.kb_split = static_cast<int32_t>(dense::cdiv(kb, s));
  p.splits = static_cast<int32_t>(dense::cdiv(kb, p.kb_split));
  return p;
}
int64_t sums_bytes(const TurnPlan& p, int64_t rows) { return 4 * p.splits * up32(rows) * p.tp; }

// Where that is the faster way (measured at 7168 x 2048, 4096 x 1800, 2048 x 1024,
// 7168 x 256 and 512 x 256).  Forward: both ways are two products, and shares of K cost two joins of
// some 3 us, more with the tokens; they pay where the products are long (64
// tokens: 7168 x 2048 27.9 against 38 us, 512 x 256 12.5 against 10.9; 131 tokens:
// 7168 x 256 22.6 against 32.2, 2048 x 1024 19.1 against 18.3; 256 tokens level or
// behind but for the narrow block).  Backward: one join for two products
// (300 tokens: 98.8 against 111.9, 30.8 against 42.1, 14.8 against 21.3; 700:
// 133 against 148, 39.9 against 46.6; 1024: 191 against 173, 48.6 against 49.9).
constexpr int kTurnForward = 256, kTurnBackward = 768;   // tokens, at most
bool turned(const moe_ffn_shape* s, bool backward) {
  const int64_t blocks = dense::cdiv(s->hidden, dense::kBK) + dense::cdiv(s->inter, dense::kBK);
  if (backward) return s->num_tokens <= kTurnBackward;
  return s->num_tokens <= kTurnForward && blocks >= 16 + s->num_tokens / 4;
}

struct FfnWs {
  dense::Plan gate, down;   // forward; gate also in the backward pass
  dense::Plan dh, dx;
  TurnPlan t_gate, t_down, t_dh;   // those of them whose tokens are columns
  bool turned;              // gate, down and dh as turned_plan's
  size_t h, dgu, sums, sums2, total;
};

FfnWs ffn_ws(const moe_ffn_shape* s, bool backward) {
  const int64_t T = s->num_tokens, H = s->hidden, I = s->inter;
  const int64_t tm = dense::cdiv(T, dense::kTile), rp = up32(T);
  FfnWs w = {};
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t o = at;
    at += ws_up(static_cast<size_t>(bytes));
    return o;
  };
  w.h = take(2 * T * I);
  if (!backward && T <= kDecodeTokens) {
    w.total = at;
    return w;
  }
  const int64_t kh = dense::cdiv(H, dense::kBK), ki = dense::cdiv(I, dense::kBK);
  w.turned = turned(s, backward);
  if (w.turned && !backward) {
    w.t_gate = turned_plan(T, 2 * I, kh, dense::kPlanPairs);
    w.t_down = turned_plan(T, H, ki, dense::kPlanPairs);
    w.sums = take(sums_bytes(w.t_gate, 2 * I));
    w.sums2 = take(sums_bytes(w.t_down, H));
  } else if (w.turned) {   // x [Wg; Wu]^T and dout Wd in one launch: two and one of three parts
    w.t_gate = turned_plan(T, 2 * I, kh, dense::kPlanPairs * 2 / 3);
    w.t_dh = turned_plan(T, I, kh, dense::kPlanPairs / 3);
    w.sums = take(sums_bytes(w.t_dh, I));
    w.sums2 = take(sums_bytes(w.t_gate, 2 * I));
  } else {
    w.gate = dense::make_plan(tm, 2 * I, kh);
    w.down = dense::make_plan(tm, H, ki);
    w.dh = dense::make_plan(tm, I, kh);
    w.sums = take(backward ? 4 * rp * I : 0);
  }
  if (backward) {
    w.dgu = take(4 * T * I);
    w.dx = dense::make_plan(tm, H, dense::cdiv(2 * I, dense::kBK));
  }
  w.total = at;
  return w;
}

int32_t check_shape(const moe_ffn_shape* s) {
  if (!s) return entry_fail(MOE_ERR_INVALID_ARG, "shape is NULL");
  if (s->num_tokens < 0 || s->hidden <= 0 || s->inter <= 0)
    return entry_fail(MOE_ERR_INVALID_ARG, "num_tokens, hidden and inter must be positive, got %d, %d, %d",
                      s->num_tokens, s->hidden, s->inter);
  if (s->hidden % 8 || s->inter % 8)
    return entry_fail(MOE_ERR_MISALIGNED, "hidden and inter must be multiples of 8, got %d and %d", s->hidden,
                      s->inter);
  if (s->num_tokens > MOE_FFN_MAX_TOKENS || s->hidden > MOE_FFN_MAX_FEATURES ||
      s->inter > MOE_FFN_MAX_FEATURES)
    return entry_fail(MOE_ERR_UNSUPPORTED, "at most %d tokens and %d features", MOE_FFN_MAX_TOKENS,
                      MOE_FFN_MAX_FEATURES);
  return MOE_OK;
}

int32_t check_matrix(const void* p, const char* name, int64_t ld, int64_t cols) {
  if (!p) return entry_fail(MOE_ERR_INVALID_ARG, "%s is NULL", name);
  if (ld < cols || ld >= (int64_t(1) << 31))
    return entry_fail(MOE_ERR_INVALID_ARG, "%s: rows of %lld elements, %lld apart", name,
                      static_cast<long long>(cols), static_cast<long long>(ld));
  if (!ptr_aligned(p, 16) || ld % 8)
    return entry_fail(MOE_ERR_MISALIGNED, "%s must be 16-byte aligned, its row stride a multiple of 8", name);
  return MOE_OK;
}

int32_t check_weights(const void* w_gate_up, const void* w_down, const void* ws, size_t have, size_t need,
                      const int32_t* status) {
  if (!w_gate_up || !w_down) return entry_fail(MOE_ERR_INVALID_ARG, "w_gate_up or w_down is NULL");
  if (!ptr_aligned(w_gate_up, 16) || !ptr_aligned(w_down, 16))
    return entry_fail(MOE_ERR_MISALIGNED, "w_gate_up and w_down must be 16-byte aligned");
  if (!status) return entry_fail(MOE_ERR_INVALID_ARG, "status is NULL");
  if (!ptr_aligned(status, 4)) return entry_fail(MOE_ERR_MISALIGNED, "status must be 4-byte aligned");
  if (!ws) return entry_fail(MOE_ERR_INVALID_ARG, "workspace is NULL");
  if (!ptr_aligned(ws, kWsAlign)) return entry_fail(MOE_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  if (have < need)
    return entry_fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, needs %zu", have, need);
  return MOE_OK;
}

// A tensor's bytes: rows of `width`, `step` apart; no rows: none.
struct Span {
  const char* name;
  int64_t at, rows, step, width;
};
Span span(const char* name, const void* p, int64_t rows, int64_t ld, int64_t cols) {
  return {name, static_cast<int64_t>(reinterpret_cast<uintptr_t>(p)), p ? rows : 0, 2 * ld, 2 * cols};
}
Span span(const char* name, const void* p, size_t bytes) {
  return {name, static_cast<int64_t>(reinterpret_cast<uintptr_t>(p)), p ? 1 : 0, 0, static_cast<int64_t>(bytes)};
}
// Rows and columns of one buffer may be shared out to several tensors, so that
// ranges from the first byte to the last may meet where the tensors do not.
bool meet(const Span& a, const Span& b) {
  if (!a.rows || !b.rows) return false;
  if (a.rows > b.rows) return meet(b, a);
  const int64_t d = b.at - a.at;
  if (d >= (a.rows - 1) * a.step + a.width || -d >= (b.rows - 1) * b.step + b.width) return false;
  // the first k from `from` on with -b.width < d + k step; whether it is below `to`, and d + k step below a.width
  auto hits = [&](int64_t d, int64_t step, int64_t from, int64_t to) {
    const int64_t need = -b.width - d;   // k step > need
    int64_t k = step == 0 ? from : need < 0 ? -((-need + step - 1) / step) + 1 : need / step + 1;
    k = std::max(k, from);
    return k < to && d + k * step > -b.width && d + k * step < a.width;
  };
  // with equal strides only the rows' difference counts
  if (a.step == b.step) return hits(d, a.step, 1 - a.rows, b.rows);
  for (int64_t i = 0; i < a.rows; ++i)
    if (hits(d - i * a.step, b.step, 0, b.rows)) return true;
  return false;
}
int32_t check_apart(const Span& a, const Span& b) {
  if (!meet(a, b)) return MOE_OK;
  return entry_fail(MOE_ERR_INVALID_ARG, "%s overlaps %s", a.name, b.name);
}
// ... unless they are the same rows.
int32_t check_apart_or_same(const Span& a, const Span& b) {
  const bool same = a.at == b.at && (a.rows <= 1 || a.step == b.step);
  return same ? MOE_OK : check_apart(a, b);
}

template <class Epi>
dense::Launch<typename Epi::Args> new_launch(int32_t* status) {
  dense::Launch<typename Epi::Args> l = {};
  l.status = status;
  l.timeout_ns = kTimeoutNs;
  return l;
}

dim3 join_grid(int64_t tokens, int64_t features) {
  return dim3(static_cast<unsigned>(dense::cdiv(features, kJoinFeatures)),
              static_cast<unsigned>(dense::cdiv(tokens, kJoinTokens)));
}

// Boxes of the operands: K-major rows of a tile (128 of A, bn / 2 of B), and
// MN-major squares of 64.
constexpr int kSquare = dense::kBK;

// Adds the sums of W x^T (turned_plan): weights w [rows, K], or [K, rows] with
// mn, against tokens x [T, K].
int32_t add_turned(Maps* m, dense::Launch<EpiSum::Args>* l, const TurnPlan& plan, const void* w, int64_t rows,
                   int64_t k, bool mn, const void* x, int64_t ld_x, int64_t tokens, float* sums, Sums* out) {
  const int i = l->problems++, at = l->maps;
  l->maps += 3;
  if (mn) MOE_TRY(dense::make_map(&m->m[at], w, Elem::kBf16, k, rows, rows, kSquare, kSquare));
  else MOE_TRY(dense::make_map(&m->m[at], w, Elem::kBf16, rows, k, k, dense::kBK, 128));
  MOE_TRY(dense::make_map(&m->m[at + 1], x, Elem::kBf16, tokens, k, ld_x, dense::kBK, plan.bn / 2));
  MOE_TRY(dense::make_map(&m->m[at + 2], sums, Elem::kF32, plan.splits * up32(rows), plan.tp, plan.tp, 32, 32));
  l->p[i] = dense::make_problem(plan, rows, plan.tp, dense::cdiv(k, dense::kBK), at, mn, at + 1, false);
  l->e[i] = {at + 2, static_cast<int32_t>(up32(rows)), plan.tp};
  *out = {sums, plan.splits, static_cast<int32_t>(up32(rows)), plan.tp};
  return MOE_OK;
}

// The launch of D = x [Wg; Wu]^T whose tiles hold both projections of a feature:
// gate rows in rank 0's half of B, up rows in rank 1's.
Problem gate_problem(const dense::Plan& plan, int64_t tokens, int64_t inter, int64_t kb) {
  Problem p = dense::make_problem(plan, tokens, 2 * inter, kb, 0, false, 1, false);
  p.b_step = plan.bn / 2;
  p.b_rank = static_cast<int32_t>(inter);
  p.tiles_n = static_cast<int32_t>(dense::cdiv(inter, plan.bn / 2));
  p.per_matrix = p.tiles_m * p.tiles_n;
  return p;
}

int32_t ffn_forward(const moe_ffn_shape* s, const void* x, int64_t ld_x, const void* wgu, const void* wd,
                    const void* base, int64_t ld_base, void* out, int64_t ld_out, uint8_t* ws,
                    int32_t* status, int sms, cudaStream_t st) {
  const int64_t T = s->num_tokens, H = s->hidden, I = s->inter;
  const FfnWs w = ffn_ws(s, false);
  __nv_bfloat16* h = reinterpret_cast<__nv_bfloat16*>(ws + w.h);
  const __nv_bfloat16* add = static_cast<const __nv_bfloat16*>(base);
  __nv_bfloat16* to = static_cast<__nv_bfloat16*>(out);
  if (T <= kDecodeTokens) {
    DecodeArgs a = {static_cast<const __nv_bfloat16*>(wgu), static_cast<const __nv_bfloat16*>(x), nullptr, h,
                    ld_x, 0, I, s->num_tokens, s->inter, s->hidden, static_cast<const uint8_t*>(wd), s->hidden,
                    2 * s->inter, kAheadBytes / sms / 16 * 16};
    MOE_CUDA(launch_decode<false>(a, sms, st));
    DecodeArgs b = {static_cast<const __nv_bfloat16*>(wd), h, add, to, I, ld_base, ld_out, s->num_tokens, s->hidden,
                    s->inter, nullptr, 0, 0, 0};
    MOE_CUDA(launch_decode<true>(b, sms, st));
    return MOE_OK;
  }
  int pairs;
  Maps m;
  if (w.turned) {
    MOE_CUDA(dense::resident_pairs<EpiSum>(sms, &pairs));
    Sums sums;
    auto l = new_launch<EpiSum>(status);
    MOE_TRY(add_turned(&m, &l, w.t_gate, wgu, 2 * I, H, false, x, ld_x, T, reinterpret_cast<float*>(ws + w.sums), &sums));
    MOE_CUDA(dense::launch<EpiSum>(m, l, pairs, st));
    MOE_CUDA(launch_pdl(join_gate_kernel, join_grid(T, I), dim3(kJoinThreads), 0, st, sums, s->num_tokens, s->inter,
                        h));
    l = new_launch<EpiSum>(status);
    l.early = dense::kEarlyA;
    MOE_TRY(add_turned(&m, &l, w.t_down, wd, H, I, false, h, I, T, reinterpret_cast<float*>(ws + w.sums2), &sums));
    MOE_CUDA(dense::launch<EpiSum>(m, l, pairs, st));
    MOE_CUDA(launch_pdl(join_out_kernel, join_grid(T, H), dim3(kJoinThreads), 0, st, sums, s->num_tokens, s->hidden,
                        add, ld_base, to, ld_out));
    return MOE_OK;
  }
  {
    auto l = new_launch<EpiGate>(status);
    MOE_TRY(dense::make_map(&m.m[0], x, Elem::kBf16, T, H, ld_x, dense::kBK, 128));
    MOE_TRY(dense::make_map(&m.m[1], wgu, Elem::kBf16, 2 * I, H, H, dense::kBK, w.gate.bn / 2));
    MOE_TRY(dense::make_map(&m.m[2], h, Elem::kBf16, T, I, I, 64, 32));
    l.problems = 1;
    l.maps = 3;
    l.p[0] = gate_problem(w.gate, T, I, dense::cdiv(H, dense::kBK));
    l.e[0] = {h, 2, s->num_tokens, s->inter};
    MOE_CUDA(dense::resident_pairs<EpiGate>(sms, &pairs));
    MOE_CUDA(dense::launch<EpiGate>(m, l, pairs, st));
  }
  auto l = new_launch<EpiOut>(status);
  MOE_TRY(dense::make_map(&m.m[0], h, Elem::kBf16, T, I, I, dense::kBK, 128));
  MOE_TRY(dense::make_map(&m.m[1], wd, Elem::kBf16, H, I, I, dense::kBK, w.down.bn / 2));
  MOE_TRY(dense::make_map(&m.m[2], out, Elem::kBf16, T, H, ld_out, 64, 32));
  l.problems = 1;
  l.maps = 3;
  l.early = dense::kEarlyB;
  l.p[0] = dense::make_problem(w.down, T, H, dense::cdiv(I, dense::kBK), 0, false, 1, false);
  l.e[0] = {add, ld_base, 2, s->num_tokens, s->hidden};
  MOE_CUDA(dense::resident_pairs<EpiOut>(sms, &pairs));
  MOE_CUDA(dense::launch<EpiOut>(m, l, pairs, st));
  return MOE_OK;
}

int32_t ffn_backward(const moe_ffn_shape* s, const void* dout, int64_t ld_dout, const void* x, int64_t ld_x,
                     const void* wgu, const void* wd, const void* dx_base, int64_t ld_base, void* dx,
                     int64_t ld_dx, void* dw_gate_up, void* dw_down, uint8_t* ws, int32_t* status, int sms,
                     cudaStream_t st) {
  const int64_t T = s->num_tokens, H = s->hidden, I = s->inter;
  const FfnWs w = ffn_ws(s, true);
  const int64_t rp = up32(T), kh = dense::cdiv(H, dense::kBK), ki2 = dense::cdiv(2 * I, dense::kBK);
  const int64_t kt = dense::cdiv(T, dense::kBK);
  __nv_bfloat16* h = reinterpret_cast<__nv_bfloat16*>(ws + w.h);
  __nv_bfloat16* dgu = reinterpret_cast<__nv_bfloat16*>(ws + w.dgu);
  float* dh = reinterpret_cast<float*>(ws + w.sums);
  int pairs;
  Maps m;
  MOE_CUDA(dense::resident_pairs<EpiSum>(sms, &pairs));
  if (w.turned) {
    Sums sums_gu, sums_dh;
    auto l = new_launch<EpiSum>(status);
    MOE_TRY(add_turned(&m, &l, w.t_gate, wgu, 2 * I, H, false, x, ld_x, T, reinterpret_cast<float*>(ws + w.sums2),
                       &sums_gu));
    MOE_TRY(add_turned(&m, &l, w.t_dh, wd, I, H, true, dout, ld_dout, T, dh, &sums_dh));
    MOE_CUDA(dense::launch<EpiSum>(m, l, pairs, st));
    MOE_CUDA(launch_pdl(join_grad_kernel, join_grid(T, I), dim3(kJoinThreads), 0, st, sums_gu, sums_dh,
                        s->num_tokens, s->inter, h, dgu));
  } else {
    {   // dh = dout Wd (Wd [H, I] is MN-major there), in float for the next epilogue
      auto l = new_launch<EpiSum>(status);
      MOE_TRY(dense::make_map(&m.m[0], dout, Elem::kBf16, T, H, ld_dout, dense::kBK, 128));
      MOE_TRY(dense::make_map(&m.m[1], wd, Elem::kBf16, H, I, I, kSquare, kSquare));
      MOE_TRY(dense::make_map(&m.m[2], dh, Elem::kF32, rp, I, I, 32, 32));
      l.maps = 3;
      l.p[0] = dense::make_problem(w.dh, T, I, kh, 0, false, 1, true);
      l.e[0] = {2, static_cast<int32_t>(rp), s->inter};
      l.problems = 1;
      MOE_CUDA(dense::launch<EpiSum>(m, l, pairs, st));
    }
    auto l = new_launch<EpiGateGrad>(status);
    MOE_TRY(dense::make_map(&m.m[0], x, Elem::kBf16, T, H, ld_x, dense::kBK, 128));
    MOE_TRY(dense::make_map(&m.m[1], wgu, Elem::kBf16, 2 * I, H, H, dense::kBK, w.gate.bn / 2));
    l.maps = 2;
    l.problems = 1;
    l.p[0] = gate_problem(w.gate, T, I, kh);
    l.e[0] = {h, dgu, dh, I, s->num_tokens, s->inter};
    MOE_CUDA(dense::resident_pairs<EpiGateGrad>(sms, &pairs));
    MOE_CUDA(dense::launch<EpiGateGrad>(m, l, pairs, st));
  }
  // dx = [dg du] [Wg; Wu] (the weights MN-major), and the weights' gradients,
  // sums over the tokens (both operands MN-major), in one launch
  auto l = new_launch<EpiOut>(status);
  if (dx) {
    const int i = l.problems++, k = l.maps;
    l.maps += 3;
    MOE_TRY(dense::make_map(&m.m[k], dgu, Elem::kBf16, T, 2 * I, 2 * I, dense::kBK, 128));
    MOE_TRY(dense::make_map(&m.m[k + 1], wgu, Elem::kBf16, 2 * I, H, H, kSquare, kSquare));
    MOE_TRY(dense::make_map(&m.m[k + 2], dx, Elem::kBf16, T, H, ld_dx, 64, 32));
    l.p[i] = dense::make_problem(w.dx, T, H, ki2, k, false, k + 1, true);
    l.e[i] = {static_cast<const __nv_bfloat16*>(dx_base), ld_base, k + 2, static_cast<int32_t>(T),
              static_cast<int32_t>(H)};
  }
  if (dw_gate_up) {
    const dense::Plan g = dense::make_plan(dense::cdiv(2 * I, dense::kTile), H, kt);
    const dense::Plan d = dense::make_plan(dense::cdiv(H, dense::kTile), I, kt);
    int i = l.problems++, k = l.maps;
    l.maps += 3;
    MOE_TRY(dense::make_map(&m.m[k], dgu, Elem::kBf16, T, 2 * I, 2 * I, kSquare, kSquare));
    MOE_TRY(dense::make_map(&m.m[k + 1], x, Elem::kBf16, T, H, ld_x, kSquare, kSquare));
    MOE_TRY(dense::make_map(&m.m[k + 2], dw_gate_up, Elem::kBf16, 2 * I, H, H, 64, 32));
    l.p[i] = dense::make_problem(g, 2 * I, H, kt, k, true, k + 1, true);
    l.e[i] = {nullptr, 0, k + 2, static_cast<int32_t>(2 * I), static_cast<int32_t>(H)};
    i = l.problems++, k = l.maps;
    l.maps += 3;
    MOE_TRY(dense::make_map(&m.m[k], dout, Elem::kBf16, T, H, ld_dout, kSquare, kSquare));
    MOE_TRY(dense::make_map(&m.m[k + 1], h, Elem::kBf16, T, I, I, kSquare, kSquare));
    MOE_TRY(dense::make_map(&m.m[k + 2], dw_down, Elem::kBf16, H, I, I, 64, 32));
    l.p[i] = dense::make_problem(d, H, I, kt, k, true, k + 1, true);
    l.e[i] = {nullptr, 0, k + 2, static_cast<int32_t>(H), static_cast<int32_t>(I)};
  }
  MOE_CUDA(dense::resident_pairs<EpiOut>(sms, &pairs));
  MOE_CUDA(dense::launch<EpiOut>(m, l, pairs, st));
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_ffn_workspace_size(const moe_ffn_shape* shape, int32_t backward) {
  using namespace moe;
  if (check_shape(shape) != MOE_OK) return 0;
  return std::max(ffn_ws(shape, backward != 0).total, kWsAlign);
}

extern "C" int32_t moe_ffn_forward(const moe_ffn_shape* s, const void* x, int64_t ld_x,
                                   const void* w_gate_up, const void* w_down, const void* base,
                                   int64_t ld_base, void* out, int64_t ld_out, void* workspace,
                                   size_t workspace_bytes, int32_t* status, void* stream) {
  using namespace moe;
  MOE_TRY(check_shape(s));
  if (s->num_tokens == 0) return MOE_OK;
  MOE_TRY(check_matrix(x, "x", ld_x, s->hidden));
  if (base) MOE_TRY(check_matrix(base, "base", ld_base, s->hidden));
  MOE_TRY(check_matrix(out, "out", ld_out, s->hidden));
  const size_t need = ffn_ws(s, false).total;
  MOE_TRY(check_weights(w_gate_up, w_down, workspace, workspace_bytes, need, status));
  {
    const int64_t T = s->num_tokens, H = s->hidden, I = s->inter;
    const Span to = span("out", out, T, ld_out, H), ws = span("workspace", workspace, need);
    const Span from[] = {span("x", x, T, ld_x, H), span("base", base, T, ld_base, H),
                         span("w_gate_up", w_gate_up, 1, 0, 2 * I * H), span("w_down", w_down, 1, 0, H * I),
                         span("status", status, 4)};
    for (int i = 0; i < 5; ++i) {
      MOE_TRY(i < 2 ? check_apart_or_same(to, from[i]) : check_apart(to, from[i]));
      MOE_TRY(check_apart(ws, from[i]));
    }
    MOE_TRY(check_apart(ws, to));
  }
  int sms = 0;
  MOE_TRY(check_device(&sms));
  return ffn_forward(s, x, ld_x, w_gate_up, w_down, base, ld_base, out, ld_out,
                     static_cast<uint8_t*>(workspace), status, sms, static_cast<cudaStream_t>(stream));
}

extern "C" int32_t moe_ffn_backward(const moe_ffn_shape* s, const void* dout, int64_t ld_dout,
                                    const void* x, int64_t ld_x, const void* w_gate_up,
                                    const void* w_down, const void* dx_base, int64_t ld_dx_base, void* dx,
                                    int64_t ld_dx, void* dw_gate_up, void* dw_down, void* workspace,
                                    size_t workspace_bytes, int32_t* status, void* stream) {
  using namespace moe;
  MOE_TRY(check_shape(s));
  if (!dw_gate_up != !dw_down)
    return entry_fail(MOE_ERR_INVALID_ARG, "dw_gate_up and dw_down go together");
  if (dw_gate_up && s->num_tokens > MOE_FFN_MAX_SUMMED)
    return entry_fail(MOE_ERR_UNSUPPORTED, "weights' gradients of at most %d tokens a call", MOE_FFN_MAX_SUMMED);
  if (!ptr_aligned(dw_gate_up, 16) || !ptr_aligned(dw_down, 16))
    return entry_fail(MOE_ERR_MISALIGNED, "dw_gate_up and dw_down must be 16-byte aligned");
  if (dw_gate_up) {   // tiles of one are stored while others are still to be read
    for (const void* g : {dw_gate_up, dw_down})
      if (g == w_gate_up || g == w_down || g == x || g == dout || g == dx)
        return entry_fail(MOE_ERR_INVALID_ARG, "dw_gate_up and dw_down must be memory of their own");
    if (dw_gate_up == dw_down)
      return entry_fail(MOE_ERR_INVALID_ARG, "dw_gate_up and dw_down must be memory of their own");
  }
  const int64_t T = s->num_tokens, H = s->hidden, I = s->inter;
  const Span dw[2] = {span("dw_gate_up", dw_gate_up, 1, 0, 2 * I * H), span("dw_down", dw_down, 1, 0, H * I)};
  const Span w[2] = {span("w_gate_up", w_gate_up, 1, 0, 2 * I * H), span("w_down", w_down, 1, 0, H * I)};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {   // sums over no tokens
    if (!dw_gate_up) return MOE_OK;
    MOE_TRY(check_apart(dw[0], dw[1]));
    for (int i = 0; i < 4; ++i) MOE_TRY(check_apart(dw[i & 1], w[i >> 1]));
    MOE_TRY(check_device(nullptr));
    const size_t n = static_cast<size_t>(s->hidden) * s->inter * 2;
    MOE_CUDA(cudaMemsetAsync(dw_gate_up, 0, 2 * n, st));
    MOE_CUDA(cudaMemsetAsync(dw_down, 0, n, st));
    return MOE_OK;
  }
  MOE_TRY(check_matrix(dout, "dout", ld_dout, s->hidden));
  MOE_TRY(check_matrix(x, "x", ld_x, s->hidden));
  if (dx_base) MOE_TRY(check_matrix(dx_base, "dx_base", ld_dx_base, s->hidden));
  if (dx) MOE_TRY(check_matrix(dx, "dx", ld_dx, s->hidden));
  const size_t need = ffn_ws(s, true).total;
  MOE_TRY(check_weights(w_gate_up, w_down, workspace, workspace_bytes, need, status));
  {
    const Span to = span("dx", dx, T, ld_dx, H), add = span("dx_base", dx ? dx_base : nullptr, T, ld_dx_base, H);
    const Span ws = span("workspace", workspace, need);
    const Span from[] = {span("x", x, T, ld_x, H), span("dout", dout, T, ld_dout, H), w[0], w[1],
                         span("status", status, 4)};
    for (const Span& t : from) {
      for (const Span& written : {to, dw[0], dw[1], ws}) MOE_TRY(check_apart(written, t));
    }
    MOE_TRY(check_apart_or_same(to, add));
    for (const Span& t : {to, add, ws}) {
      for (const Span& g : dw) MOE_TRY(check_apart(g, t));
    }
    MOE_TRY(check_apart(dw[0], dw[1]));
    MOE_TRY(check_apart(ws, to));
    MOE_TRY(check_apart(ws, add));
  }
  if (!dx && !dw_gate_up) return MOE_OK;
  int sms = 0;
  MOE_TRY(check_device(&sms));
  return ffn_backward(s, dout, ld_dout, x, ld_x, w_gate_up, w_down, dx_base, ld_dx_base, dx, ld_dx,
                      dw_gate_up, dw_down, static_cast<uint8_t*>(workspace), status, sms, st);
}
