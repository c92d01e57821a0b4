// adapters.cu -- low-rank adapters of many requests beside a shared
// projection: out = base + scale_a B_a (A_a x), and its gradients.
//
// Tokens are grouped by adapter on the device (group_kernel: a stable
// counting sort and a list of tiles of up to 64 tokens that share an
// adapter), then:
//   forward:   v = A x                  (shrink_x_kernel, contracts over H)
//              out = base + B (s v)     (expand_kernel, contracts over r)
//   backward:  v = A x,  u = s B^T dout (shrink_x_kernel, shrink_d_kernel)
//              dx = dx_base + A^T u     (expand_kernel)
//              dA = sum u x^T, dB = s sum dout v^T   (grad_kernel, contracts
//                                       over the adapter's tokens)
// With ranks of 8 to 128 every one of these does r multiply-adds for each
// element it moves, far below the ~290 a byte at which tensor throughput
// would bind, so the layout serves the memory stream: operands go straight
// from global memory into the fragments of mma.sync (16x8x16, bf16, float
// accumulators) with 16-byte loads and no staging.  The contraction index and
// the column index of a fragment are free to be permuted as long as both
// operands (or the store) use the same order; each kernel picks the order in
// which a lane's share is contiguous in memory.  (tcgen05 would need the
// gathered rows staged in shared memory through another pass, for tiles
// whose N is r.)
//
// v and u are kept in float [T, r] and enter the following product as two
// bf16 terms, hi = bf16(v) and lo = bf16(v - hi): a relative error below
// 2^-17, so that float outputs (router logits, dA, dB) keep float accuracy.
// Float gradients dout are split the same way.
#include <cuda_bf16.h>

#include "cluster.cuh"
#include "entry.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kTile = 64;          // tokens of a tile
constexpr int kGroupThreads = 1024;
constexpr int kWarps = 8;          // warps of the product kernels
constexpr int kThreads = 32 * kWarps;

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Words (lo0, lo1) and (hi0, hi1) of two words of two bf16 each.
__device__ __forceinline__ uint32_t pack_lo(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
__device__ __forceinline__ uint32_t pack_hi(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }

// v = hi + lo + an error below 2^-17 |v|.  Beyond bf16's finite range the
// residual is dropped (inf - inf would make an infinity a NaN).
__device__ __forceinline__ void split(float v, __nv_bfloat16* hi, __nv_bfloat16* lo) {
  const __nv_bfloat16 h = __float2bfloat16_rn(v);
  const float f = __bfloat162float(h);
  *hi = h;
  *lo = __float2bfloat16_rn(fabsf(f) < INFINITY ? v - f : 0.f);
}
__device__ __forceinline__ uint32_t word(__nv_bfloat16 a, __nv_bfloat16 b) {
  return static_cast<uint32_t>(__bfloat16_as_ushort(a)) |
         static_cast<uint32_t>(__bfloat16_as_ushort(b)) << 16;
}
__device__ __forceinline__ void split2(float x, float y, uint32_t* hi, uint32_t* lo) {
  __nv_bfloat16 hx, lx, hy, ly;
  split(x, &hx, &lx);
  split(y, &hy, &ly);
  *hi = word(hx, hy);
  *lo = word(lx, ly);
}

__device__ __forceinline__ uint4 ldg16(const void* p) { return __ldg(static_cast<const uint4*>(p)); }

// ------------------------------------------------------------ grouping
struct Groups {
  int32_t* perm;      // [T] token of each sorted position
  int32_t* offsets;   // [NA + 2] first position of adapter a; [NA]: of the tokens without one
  int4* tiles;        // (adapter or -1, first position, tokens, 0)
  int32_t* num_tiles;
};

__host__ __device__ inline int64_t max_tiles(int64_t T, int64_t NA) {
  return T / kTile + (NA + 1 < T ? NA + 1 : T) + 1;
}

// Position of ids in the order (adapter 0 .. NA-1, none), stable in the token.
// One CTA: warp w owns the w-th contiguous 32nd of the tokens and a histogram
// of it; the histograms' running sums give each warp its bases, and a warp
// hands out positions to its tokens in order.
__global__ void __launch_bounds__(kGroupThreads) group_kernel(const int32_t* __restrict__ ids,
                                                              int T, int NA, Groups g) {
  extern __shared__ __align__(16) uint8_t sm[];
  const int C = NA + 1;                 // columns: the adapters and "none"
  int32_t* hist = reinterpret_cast<int32_t*>(sm);   // [32][C]
  int32_t* first = hist + 32 * C;         // [C + 1] first position
  int32_t* tfirst = first + C + 1;      // [C + 1] first tile
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  griddep_launch_dependents();
  for (int i = threadIdx.x; i < 32 * C; i += kGroupThreads) hist[i] = 0;
  __syncthreads();
  const int per = ((T + 31) / 32 + 31) / 32 * 32;   // tokens of a warp, whole rounds
  const int64_t t0 = static_cast<int64_t>(per) * warp;
  const int t1 = static_cast<int>(min(t0 + per, static_cast<int64_t>(T)));
  for (int64_t t = t0 + lane; t < t1; t += 32) {
    const int id = ids[t];
    atomicAdd(&hist[warp * C + (static_cast<unsigned>(id) < static_cast<unsigned>(NA) ? id : NA)], 1);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < C; c += kGroupThreads) {
    int sum = 0;
    for (int w = 0; w < 32; ++w) {
      const int n = hist[w * C + c];
      hist[w * C + c] = sum;            // tokens of this column in earlier warps
      sum += n;
    }
    first[c] = sum;
    tfirst[c] = (sum + kTile - 1) / kTile;
  }
  __syncthreads();
  if (warp == 0) {   // exclusive sums over the columns
    int run = 0, trun = 0;
    for (int c0 = 0; c0 < C; c0 += 32) {
      const int c = c0 + lane;
      const int n = c < C ? first[c] : 0, tn = c < C ? tfirst[c] : 0;
      int x = n, y = tn;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int px = __shfl_up_sync(0xFFFFFFFFu, x, o), py = __shfl_up_sync(0xFFFFFFFFu, y, o);
        if (lane >= o) x += px, y += py;
      }
      if (c < C) first[c] = run + x - n, tfirst[c] = trun + y - tn;
      run += __shfl_sync(0xFFFFFFFFu, x, 31);
      trun += __shfl_sync(0xFFFFFFFFu, y, 31);
    }
    if (lane == 0) first[C] = run, tfirst[C] = trun, *g.num_tiles = trun;
  }
  __syncthreads();
  for (int c = threadIdx.x; c <= C; c += kGroupThreads) g.offsets[c] = first[c];
  const int tiles = tfirst[C];
  for (int i = threadIdx.x; i < tiles; i += kGroupThreads) {
    int lo = 0, hi = C;                 // the last column whose first tile is at or before i
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tfirst[mid] <= i) lo = mid;
      else hi = mid;
    }
    const int p = first[lo] + (i - tfirst[lo]) * kTile;
    g.tiles[i] = make_int4(lo < NA ? lo : -1, p, min(kTile, first[lo + 1] - p), 0);
  }
  for (int64_t tt = t0; tt < t1; tt += 32) {
    const int64_t t = tt + lane;
    int c = -1;                         // past the end: matches no column
    if (t < t1) {
      const int id = ids[t];
      c = static_cast<unsigned>(id) < static_cast<unsigned>(NA) ? id : NA;
    }
    const unsigned same = __match_any_sync(0xFFFFFFFFu, c);
    const int rank = __popc(same & ((1u << lane) - 1));
    int base = 0;
    if (c >= 0) base = hist[warp * C + c];
    __syncwarp();
    if (c >= 0) {
      g.perm[first[c] + base + rank] = static_cast<int32_t>(t);
      if (rank == 0) hist[warp * C + c] = base + __popc(same);
    }
    __syncwarp();
  }
}

// ------------------------------------------------------- v = A x
struct ShrinkArgs {
  const void* src;     // x (bf16) or dout
  int64_t ld;
  const __nv_bfloat16* pool;
  const float* scale;  // null: 1
  float* dst;          // [T, r] by sorted position
  const int32_t* perm;
  const int4* tiles;
  const int32_t* num_tiles;
  int32_t r, K;        // K: contracted length
};

// Adds the warps' partial tiles [kTile][rp] in warp order into `red`, then
// the cluster's CTAs' in rank order, and writes the tile's rows of dst.
template <typename F>
__device__ __forceinline__ void reduce_tile(float* red, int rp, int r, int4 tile, int wk, int nwk,
                                            float scale, float* dst, F&& add) {
  for (int i = threadIdx.x; i < kTile * rp; i += kThreads) red[i] = 0.f;
  __syncthreads();
  for (int w = 0; w < nwk; ++w) {
    if (wk == w) add();
    __syncthreads();
  }
  cluster_sync();
  const int S = static_cast<int>(cluster_size());
  const int total = tile.z * r;
  for (int i = static_cast<int>(cluster_rank()) * kThreads + threadIdx.x; i < total;
       i += S * kThreads) {
    const int t = i / r, j = i - t * r;
    float v = 0.f;
    for (int c = 0; c < S; ++c) v += cluster_load(red + t * rp + j, c);
    dst[static_cast<int64_t>(tile.y + t) * r + j] = v * scale;
  }
  cluster_sync();   // no CTA leaves while another reads its shared memory
}

// Cluster of S CTAs per tile, S * WK warps sharing out the 32-element chunks
// of K.  Rank is MMA-M, tokens are MMA-N: lane (g, t) of a chunk loads the 8
// elements at 8 t of rank rows g and g + 8 and of token g, two MMAs deep.
template <int RT>
__global__ void __launch_bounds__(kThreads) shrink_x_kernel(const ShrinkArgs a) {
  constexpr int NT = RT <= 2 ? 8 : RT == 4 ? 4 : 2;   // 8-token columns of a warp
  constexpr int WT = kTile / (8 * NT);                // warps side by side on a tile
  constexpr int WK = kWarps / WT;
  constexpr int RP = 16 * RT;
  __shared__ float red[kTile * RP];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int wt = warp % WT, wk = warp / WT;
  griddep_wait();
  griddep_launch_dependents();
  const int S = static_cast<int>(cluster_size());
  const int ti = blockIdx.x / S;
  if (ti >= *a.num_tiles) return;        // the whole cluster
  const int4 tile = a.tiles[ti];
  if (tile.x < 0) return;
  float acc[RT][NT][4];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i][j][q] = 0.f;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.src);
  const __nv_bfloat16* row[NT];          // null: no such token
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int i = 8 * (wt * NT + j) + g;
    row[j] = i < tile.z ? src + static_cast<int64_t>(a.perm[tile.y + i]) * a.ld + 8 * t : nullptr;
  }
  const int live = min(NT, (tile.z - 8 * wt * NT + 7) / 8);   // columns with a token
  const __nv_bfloat16* pool = a.pool + static_cast<int64_t>(tile.x) * a.r * a.K + 8 * t;
  const int chunks = (a.K + 31) / 32, parts = S * WK;
  const int per = (chunks + parts - 1) / parts;
  const int c0 = (static_cast<int>(cluster_rank()) * WK + wk) * per, c1 = min(c0 + per, chunks);
  if (live > 0)
#pragma unroll 2
    for (int c = c0; c < c1; ++c) {
      const int k = 32 * c;
      const bool in = k + 8 * t < a.K;
      uint4 p[RT][2], x[NT];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int rank = 16 * i + 8 * h + g;
          p[i][h] = in && rank < a.r ? ldg16(pool + static_cast<int64_t>(rank) * a.K + k)
                                     : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
      for (int j = 0; j < NT; ++j)
        x[j] = in && row[j] ? ldg16(row[j] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        if (j < live)
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            mma(acc[i][j], p[i][0].x, p[i][1].x, p[i][0].y, p[i][1].y, x[j].x, x[j].y);
            mma(acc[i][j], p[i][0].z, p[i][1].z, p[i][0].w, p[i][1].w, x[j].z, x[j].w);
          }
    }
  reduce_tile(red, RP, a.r, tile, wk, WK, 1.0f, a.dst, [&] {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          red[(8 * (wt * NT + j) + 2 * t + (q & 1)) * RP + 16 * i + g + 8 * (q >> 1)] += acc[i][j][q];
  });
}

// ------------------------------------------------------- u = s B^T dout
// Eight values of dout at p as four words of two bf16 (and, from float, the
// words of their residuals).
template <bool F32>
__device__ __forceinline__ void load8(const void* p, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  if constexpr (F32) {
    const float4 a = __ldg(static_cast<const float4*>(p)), b = __ldg(static_cast<const float4*>(p) + 1);
    split2(a.x, a.y, &hi[0], &lo[0]);
    split2(a.z, a.w, &hi[1], &lo[1]);
    split2(b.x, b.y, &hi[2], &lo[2]);
    split2(b.z, b.w, &hi[3], &lo[3]);
  } else {
    const uint4 a = ldg16(p);
    hi[0] = a.x, hi[1] = a.y, hi[2] = a.z, hi[3] = a.w;
  }
}

// W words (2 W bf16) at p, 4 W-byte aligned (16 for W >= 4).
template <int W>
__device__ __forceinline__ void load_words(const __nv_bfloat16* p, uint32_t (&o)[W]) {
  if constexpr (W == 1) {
    o[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  } else if constexpr (W == 2) {
    const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
    o[0] = q.x, o[1] = q.y;
  } else {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const uint4 q = ldg16(p + 8 * i);
      o[4 * i] = q.x, o[4 * i + 1] = q.y, o[4 * i + 2] = q.z, o[4 * i + 3] = q.w;
    }
  }
}

// As shrink_x_kernel with the pool contracted over its rows (B [N, r]):
// tokens are MMA-M, ranks MMA-N.  Lane (g, t) takes the 8 pool rows at 8 t of
// a chunk, ranks 2 RT g .. + 2 RT - 1; column g of rank tile i is rank
// 2 RT g + i, so that a lane's words of two rows pair up into fragments.
template <int RT, bool F32>
__global__ void __launch_bounds__(kThreads) shrink_d_kernel(const ShrinkArgs a) {
  constexpr int MT = RT <= 2 ? 4 : RT == 4 ? 2 : 1;   // 16-token rows of a warp
  constexpr int WT = kTile / (16 * MT);
  constexpr int WK = kWarps / WT;
  constexpr int RP = 16 * RT;
  constexpr size_t ES = F32 ? 4 : 2;
  __shared__ float red[kTile * RP];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int wt = warp % WT, wk = warp / WT;
  griddep_wait();
  griddep_launch_dependents();
  const int S = static_cast<int>(cluster_size());
  const int ti = blockIdx.x / S;
  if (ti >= *a.num_tiles) return;
  const int4 tile = a.tiles[ti];
  if (tile.x < 0) return;
  float acc[MT][2 * RT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 2 * RT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i][j][q] = 0.f;
  const uint8_t* row[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = 16 * (wt * MT + m) + 8 * h + g;
      row[m][h] = i < tile.z ? static_cast<const uint8_t*>(a.src) +
                                   (static_cast<int64_t>(a.perm[tile.y + i]) * a.ld + 8 * t) * ES
                             : nullptr;
    }
  const int live = min(MT, (tile.z - 16 * wt * MT + 15) / 16);
  const __nv_bfloat16* pool = a.pool + static_cast<int64_t>(tile.x) * a.r * a.K;
  const int chunks = (a.K + 31) / 32, parts = S * WK;
  const int per = (chunks + parts - 1) / parts;
  const int c0 = (static_cast<int>(cluster_rank()) * WK + wk) * per, c1 = min(c0 + per, chunks);
  // the lane's ranks exist, by halves of 8 (ranks are a multiple of 8)
  const int rank0 = 2 * RT * g;
  if (live > 0)
    for (int c = c0; c < c1; ++c) {
      const int k = 32 * c;
      const bool in = k + 8 * t < a.K;
      uint32_t w[8][RT];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const __nv_bfloat16* p = pool + static_cast<int64_t>(k + 8 * t + q) * a.r + rank0;
#pragma unroll
        for (int i = 0; i < RT; ++i) w[q][i] = 0;
        if constexpr (RT == 8) {
          uint32_t h[4];
          if (in && rank0 < a.r) {
            load_words<4>(p, h);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[q][i] = h[i];
          }
          if (in && rank0 + 8 < a.r) {
            load_words<4>(p + 8, h);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[q][4 + i] = h[i];
          }
        } else {
          if (in && rank0 < a.r) load_words<RT>(p, w[q]);
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (m >= live) continue;
        uint32_t h0[4] = {0, 0, 0, 0}, h1[4] = {0, 0, 0, 0}, l0[4] = {0, 0, 0, 0}, l1[4] = {0, 0, 0, 0};
        if (in && row[m][0]) load8<F32>(row[m][0] + k * ES, h0, l0);
        if (in && row[m][1]) load8<F32>(row[m][1] + k * ES, h1, l1);
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int j = 0; j < 2 * RT; ++j) {
            const uint32_t r0 = w[4 * half][j / 2], r1 = w[4 * half + 1][j / 2];
            const uint32_t r2 = w[4 * half + 2][j / 2], r3 = w[4 * half + 3][j / 2];
            const uint32_t b0 = j & 1 ? pack_hi(r0, r1) : pack_lo(r0, r1);
            const uint32_t b1 = j & 1 ? pack_hi(r2, r3) : pack_lo(r2, r3);
            mma(acc[m][j], h0[2 * half], h1[2 * half], h0[2 * half + 1], h1[2 * half + 1], b0, b1);
            if constexpr (F32)
              mma(acc[m][j], l0[2 * half], l1[2 * half], l0[2 * half + 1], l1[2 * half + 1], b0, b1);
          }
      }
    }
  const float scale = a.scale ? __ldg(a.scale + tile.x) : 1.0f;
  reduce_tile(red, RP, a.r, tile, wk, WK, scale, a.dst, [&] {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 2 * RT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          red[(16 * (wt * MT + m) + g + 8 * (q >> 1)) * RP + 2 * RT * (2 * t + (q & 1)) + j] += acc[m][j][q];
  });
}

// ---------------------------------------- out = base + pool-product of v
struct ExpandArgs {
  const float* v;        // [T, r] by sorted position
  const __nv_bfloat16* pool;
  const float* scale;    // applied to v; null: 1
  const void* base;      // null: zero
  int64_t ld_base;
  void* out;
  int64_t ld_out;
  const int32_t* perm;
  const int4* tiles;
  const int32_t* num_tiles;
  int32_t r, N;          // N: output features
  int32_t per_cta;       // features of a CTA, a multiple of kWarps * the warp's
};

// Row stride (bytes) of v in shared memory: the 8-byte reads of 4 rows x 4
// lanes fall into distinct banks.
constexpr int v_stride(int RT) { return RT == 1 ? 32 : 32 * RT + 32; }

// Eight consecutive outputs: base (or zero) plus d, rounded once.
template <bool F32>
__device__ __forceinline__ void add8(const void* base, void* out, const float (&d)[8]) {
  if constexpr (F32) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    if (base) x = static_cast<const float4*>(base)[0], y = static_cast<const float4*>(base)[1];
    static_cast<float4*>(out)[0] = make_float4(x.x + d[0], x.y + d[1], x.z + d[2], x.w + d[3]);
    static_cast<float4*>(out)[1] = make_float4(y.x + d[4], y.y + d[5], y.z + d[6], y.w + d[7]);
  } else {
    uint4 q = make_uint4(0, 0, 0, 0);
    if (base) q = *static_cast<const uint4*>(base);
    uint32_t* w = &q.x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = word(__float2bfloat16_rn(__uint_as_float(w[i] << 16) + d[2 * i]),
                  __float2bfloat16_rn(__uint_as_float(w[i] & 0xFFFF0000u) + d[2 * i + 1]));
    *static_cast<uint4*>(out) = q;
  }
}

// Tokens without an adapter: out = base (nothing to do when they are the
// same memory).
template <bool F32>
__device__ __forceinline__ void copy_rows(const ExpandArgs& a, int4 tile, int n0, int n1) {
  constexpr size_t ES = F32 ? 4 : 2;
  if (a.base == a.out && a.ld_base == a.ld_out) return;
  const int cols = (n1 - n0) / 8;
  for (int i = threadIdx.x; i < tile.z * cols; i += kThreads) {
    const int row = i / cols, n = n0 + 8 * (i - row * cols);
    const int64_t t = a.perm[tile.y + row];
    const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    void* out = static_cast<uint8_t*>(a.out) + (t * a.ld_out + n) * ES;
    const void* base = a.base ? static_cast<const uint8_t*>(a.base) + (t * a.ld_base + n) * ES : nullptr;
    if (!base) {
      add8<F32>(nullptr, out, zero);
    } else {   // bit for bit
#pragma unroll
      for (int q = 0; q < static_cast<int>(ES) / 2; ++q)
        static_cast<uint4*>(out)[q] = static_cast<const uint4*>(base)[q];
    }
  }
}

// One CTA per (tile, range of features); a warp takes a group of features,
// holds the pool's fragments of it and runs the tile's tokens, 16 at a time.
// Tokens are MMA-M (v from shared memory, hi and lo), features MMA-N.
//   !ROWS: pool [N, r]: 32 features; column n of feature tile j is feature
//          8 (n / 2) + 2 j + n % 2
//   ROWS:  pool [r, N]: 8 FL features; lane (g, t) of a 16-rank step loads FL
//          features of rank rows 4 t .. + 3; column n of tile j is FL n + j
// so that a lane ends with 8 (or 16) consecutive features of its two tokens.
template <int RT, bool ROWS, bool F32>
__global__ void __launch_bounds__(kThreads) expand_kernel(const ExpandArgs a) {
  constexpr int FL = RT == 8 ? 4 : 8;
  constexpr int JT = ROWS ? FL : 4;           // 8-feature tiles of a warp
  constexpr int FW = 8 * JT;                  // features of a warp
  constexpr int VS = v_stride(RT);
  constexpr size_t ES = F32 ? 4 : 2;
  __shared__ __align__(16) uint8_t vh[kTile * VS], vl[kTile * VS];
  __shared__ int32_t tok[kTile];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  griddep_wait();
  griddep_launch_dependents();
  if (static_cast<int>(blockIdx.x) >= *a.num_tiles) return;
  const int4 tile = a.tiles[blockIdx.x];
  const int n0 = blockIdx.y * a.per_cta, n1 = min(n0 + a.per_cta, a.N);
  if (tile.x < 0) {
    copy_rows<F32>(a, tile, n0, n1);
    return;
  }
  const float scale = a.scale ? __ldg(a.scale + tile.x) : 1.0f;
  const int live = (tile.z + 15) / 16;
  for (int i = threadIdx.x; i < live * 16 * 8 * RT; i += kThreads) {   // two ranks each
    const int row = i / (8 * RT), j = 2 * (i - row * 8 * RT);
    float2 v = make_float2(0.f, 0.f);
    if (row < tile.z && j < a.r)
      v = *reinterpret_cast<const float2*>(a.v + static_cast<int64_t>(tile.y + row) * a.r + j);
    uint32_t h, l;
    split2(v.x * scale, v.y * scale, &h, &l);
    *reinterpret_cast<uint32_t*>(vh + row * VS + 2 * j) = h;
    *reinterpret_cast<uint32_t*>(vl + row * VS + 2 * j) = l;
  }
  if (threadIdx.x < kTile)
    tok[threadIdx.x] = static_cast<int>(threadIdx.x) < tile.z ? a.perm[tile.y + threadIdx.x] : -1;
  __syncthreads();
  const __nv_bfloat16* pool = a.pool + static_cast<int64_t>(tile.x) * a.r * a.N;
  for (int f = n0 + warp * FW; f < n1; f += kWarps * FW) {
    uint32_t b[RT][JT][2];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      if constexpr (ROWS) {
        uint32_t w[4][FL / 2];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int rank = 16 * i + 4 * t + q;
#pragma unroll
          for (int c = 0; c < FL / 2; ++c) w[q][c] = 0;
          if (rank < a.r && f + FL * g < a.N)
            load_words<FL / 2>(pool + static_cast<int64_t>(rank) * a.N + f + FL * g, w[q]);
        }
#pragma unroll
        for (int j = 0; j < JT; ++j) {
          b[i][j][0] = j & 1 ? pack_hi(w[0][j / 2], w[1][j / 2]) : pack_lo(w[0][j / 2], w[1][j / 2]);
          b[i][j][1] = j & 1 ? pack_hi(w[2][j / 2], w[3][j / 2]) : pack_lo(w[2][j / 2], w[3][j / 2]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < JT; ++j) {
          const int n = f + 8 * (g >> 1) + 2 * j + (g & 1), rank = 16 * i + 4 * t;
          uint32_t w[2] = {0, 0};
          if (n < a.N && rank < a.r) load_words<2>(pool + static_cast<int64_t>(n) * a.r + rank, w);
          b[i][j][0] = w[0];
          b[i][j][1] = w[1];
        }
      }
    }
#pragma unroll 2
    for (int m = 0; m < live; ++m) {
      float acc[JT][4];
#pragma unroll
      for (int j = 0; j < JT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[j][q] = 0.f;
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int o0 = (16 * m + g) * VS + 32 * i + 8 * t, o1 = o0 + 8 * VS;
        const uint2 h0 = *reinterpret_cast<const uint2*>(vh + o0);
        const uint2 h1 = *reinterpret_cast<const uint2*>(vh + o1);
        const uint2 l0 = *reinterpret_cast<const uint2*>(vl + o0);
        const uint2 l1 = *reinterpret_cast<const uint2*>(vl + o1);
#pragma unroll
        for (int j = 0; j < JT; ++j) {
          mma(acc[j], h0.x, h1.x, h0.y, h1.y, b[i][j][0], b[i][j][1]);
          mma(acc[j], l0.x, l1.x, l0.y, l1.y, b[i][j][0], b[i][j][1]);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t row = tok[16 * m + 8 * h + g];
        if (row < 0) continue;
        uint8_t* out = static_cast<uint8_t*>(a.out) + row * a.ld_out * ES;
        const uint8_t* base = a.base ? static_cast<const uint8_t*>(a.base) + row * a.ld_base * ES : nullptr;
        if constexpr (ROWS && FL == 8) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int n = f + 16 * t + 8 * c;
            float d[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = acc[j][2 * h + c];
            if (n < a.N) add8<F32>(base ? base + n * ES : nullptr, out + n * ES, d);
          }
        } else {
          const int n = f + 8 * t;
          float d[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (ROWS) {
              d[j] = acc[j][2 * h];
              d[4 + j] = acc[j][2 * h + 1];
            } else {
              d[2 * j] = acc[j][2 * h];
              d[2 * j + 1] = acc[j][2 * h + 1];
            }
          }
          if (n < a.N) add8<F32>(base ? base + n * ES : nullptr, out + n * ES, d);
        }
      }
    }
  }
}

// ------------------------------------------------- dA = sum u x^T, dB
struct GradArgs {
  const float* left;     // u or v, [T, r] by sorted position
  const float* scale;    // applied to left; null: 1
  const void* src;       // x or dout
  int64_t ld;
  const int32_t* perm;
  const int32_t* offsets;
  float* out;            // dA [NA, r, N], or (transposed) dB [NA, N, r]
  int32_t r, N;
  int32_t transposed;
};

constexpr int kGradTok = 16 * kWarps;              // tokens a CTA takes at a time
constexpr int kGradVS = 2 * kGradTok + 32;         // bytes of a rank row of left
template <int RT, bool F32>
constexpr int grad_fl() { return (F32 ? RT <= 2 : RT <= 4) ? 8 : 4; }
template <int RT, bool F32>
constexpr size_t grad_smem() {
  const size_t stage = 2 * 16 * RT * kGradVS, red = 16 * RT * (8 * grad_fl<RT, F32>() + 1) * 4;
  return stage > red ? stage : red;
}

// Cluster of C CTAs per (range of 8 FL features, adapter): the adapter's
// tokens in rounds of 128, CTA by CTA, 16 to a warp.  Ranks are MMA-M (left
// from shared memory, transposed), features MMA-N, tokens contracted: lane
// (g, t) loads FL features of the token rows 4 t .. + 3 of the warp's 16.
template <int RT, bool F32>
__global__ void __launch_bounds__(kThreads) grad_kernel(const GradArgs a) {
  constexpr int FL = grad_fl<RT, F32>();
  constexpr int FW = 8 * FL;
  constexpr int RP = 16 * RT, RS = FW + 1;
  constexpr size_t ES = F32 ? 4 : 2;
  extern __shared__ __align__(16) uint8_t sm[];
  uint8_t* uh = sm;
  uint8_t* ul = sm + RP * kGradVS;
  float* red = reinterpret_cast<float*>(sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  griddep_wait();
  griddep_launch_dependents();
  const int C = static_cast<int>(cluster_size()), rank_c = static_cast<int>(cluster_rank());
  const int f = (blockIdx.x / C) * FW, ad = blockIdx.y;
  const int p0 = a.offsets[ad], p1 = a.offsets[ad + 1];
  const float scale = a.scale ? __ldg(a.scale + ad) : 1.0f;
  float acc[RT][FL][4];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < FL; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i][j][q] = 0.f;
  const bool in = f + FL * g < a.N;
  for (int p = p0 + rank_c * kGradTok; p < p1; p += C * kGradTok) {
    const int n = min(kGradTok, p1 - p);
    // the warp's token rows, in flight while left is staged
    uint32_t w[4][FL / 2], wl[4][FL / 2];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
#pragma unroll
      for (int c = 0; c < FL / 2; ++c) w[q][c] = 0, wl[q][c] = 0;
      const int i = 16 * warp + 4 * t + q;
      if (in && i < n) {
        const uint8_t* s = static_cast<const uint8_t*>(a.src) +
                           (static_cast<int64_t>(a.perm[p + i]) * a.ld + f + FL * g) * ES;
        if constexpr (F32) {
#pragma unroll
          for (int c = 0; c < FL / 4; ++c) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(s) + c);
            split2(x.x, x.y, &w[q][2 * c], &wl[q][2 * c]);
            split2(x.z, x.w, &w[q][2 * c + 1], &wl[q][2 * c + 1]);
          }
        } else {
          load_words<FL / 2>(reinterpret_cast<const __nv_bfloat16*>(s), w[q]);
        }
      }
    }
    __syncthreads();   // the previous round's reads are done
    for (int i = threadIdx.x; i < kGradTok * RP; i += kThreads) {
      const int tk = i / RP, j = i - tk * RP;
      float v = 0.f;
      if (tk < n && j < a.r) v = a.left[static_cast<int64_t>(p + tk) * a.r + j] * scale;
      split(v, reinterpret_cast<__nv_bfloat16*>(uh + j * kGradVS) + tk,
            reinterpret_cast<__nv_bfloat16*>(ul + j * kGradVS) + tk);
    }
    __syncthreads();
    if (16 * warp < n)
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int o0 = (16 * i + g) * kGradVS + 32 * warp + 8 * t, o1 = o0 + 8 * kGradVS;
        const uint2 h0 = *reinterpret_cast<const uint2*>(uh + o0);
        const uint2 h1 = *reinterpret_cast<const uint2*>(uh + o1);
        const uint2 l0 = *reinterpret_cast<const uint2*>(ul + o0);
        const uint2 l1 = *reinterpret_cast<const uint2*>(ul + o1);
#pragma unroll
        for (int j = 0; j < FL; ++j) {
          const uint32_t b0 = j & 1 ? pack_hi(w[0][j / 2], w[1][j / 2]) : pack_lo(w[0][j / 2], w[1][j / 2]);
          const uint32_t b1 = j & 1 ? pack_hi(w[2][j / 2], w[3][j / 2]) : pack_lo(w[2][j / 2], w[3][j / 2]);
          mma(acc[i][j], h0.x, h1.x, h0.y, h1.y, b0, b1);
          mma(acc[i][j], l0.x, l1.x, l0.y, l1.y, b0, b1);
          if constexpr (F32) {
            const uint32_t c0 = j & 1 ? pack_hi(wl[0][j / 2], wl[1][j / 2]) : pack_lo(wl[0][j / 2], wl[1][j / 2]);
            const uint32_t c1 = j & 1 ? pack_hi(wl[2][j / 2], wl[3][j / 2]) : pack_lo(wl[2][j / 2], wl[3][j / 2]);
            mma(acc[i][j], h0.x, h1.x, h0.y, h1.y, c0, c1);
          }
        }
      }
  }
  // the warps' sums in warp order, then the cluster's in rank order
  __syncthreads();
  for (int i = threadIdx.x; i < RP * RS; i += kThreads) red[i] = 0.f;
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) {
    if (warp == w)
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < FL; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            red[(16 * i + g + 8 * (q >> 1)) * RS + FL * (2 * t + (q & 1)) + j] += acc[i][j][q];
    __syncthreads();
  }
  cluster_sync();
  const int cols = min(FW, a.N - f), total = a.r * cols;
  for (int i = rank_c * kThreads + threadIdx.x; i < total; i += C * kThreads) {
    int j, n;
    if (a.transposed) n = i / a.r, j = i - n * a.r;
    else j = i / cols, n = i - j * cols;
    float v = 0.f;
    for (int c = 0; c < C; ++c) v += cluster_load(red + j * RS + n, c);
    float* out = a.out + static_cast<int64_t>(ad) * a.r * a.N;
    if (a.transposed) out[static_cast<int64_t>(f + n) * a.r + j] = v;
    else out[static_cast<int64_t>(j) * a.N + f + n] = v;
  }
  cluster_sync();
}

// ------------------------------------------------------------- host side
struct AdapterWs {
  size_t perm, offsets, tiles, num_tiles, v, u, total;
};

AdapterWs adapter_ws(const moe_adapter_shape* s, bool backward) {
  const size_t T = static_cast<size_t>(s->num_tokens), NA = static_cast<size_t>(s->num_adapters);
  AdapterWs w;
  w.perm = 0;
  w.offsets = ws_up(T * 4);
  w.tiles = w.offsets + ws_up((NA + 2) * 4);
  w.num_tiles = w.tiles + ws_up(static_cast<size_t>(max_tiles(s->num_tokens, s->num_adapters)) * 16);
  w.v = w.num_tiles + kWsAlign;
  const size_t low = ws_up(T * static_cast<size_t>(s->rank) * 4);
  w.u = w.v + low;
  w.total = w.u + (backward ? low : 0);
  return w;
}

int32_t check_adapter(const moe_adapter_shape* s) {
  if (!s) return entry_fail(MOE_ERR_INVALID_ARG, "shape is NULL");
  if (s->num_tokens < 0) return entry_fail(MOE_ERR_INVALID_ARG, "num_tokens < 0");
  if (s->num_adapters < 1 || s->num_adapters > 1024)
    return entry_fail(MOE_ERR_INVALID_ARG, "num_adapters must be in [1, 1024]");
  if (s->rank < 1 || s->rank > 128)
    return entry_fail(MOE_ERR_INVALID_ARG, "rank must be in [8, 128]");
  if (s->in_features < 1 || s->out_features < 1)
    return entry_fail(MOE_ERR_INVALID_ARG, "in_features and out_features must be positive");
  if (s->in_features > (1 << 20) || s->out_features > (1 << 20))
    return entry_fail(MOE_ERR_UNSUPPORTED, "in_features and out_features must be at most 2^20");
  if (s->rank % 8 || s->in_features % 8 || s->out_features % 8)
    return entry_fail(MOE_ERR_MISALIGNED,
                      "rank (%d), in_features (%d) and out_features (%d) must be multiples of 8",
                      s->rank, s->in_features, s->out_features);
  if (s->out_dtype != MOE_DTYPE_BF16 && s->out_dtype != MOE_DTYPE_F32)
    return entry_fail(MOE_ERR_INVALID_ARG, "out_dtype %d unknown", s->out_dtype);
  return MOE_OK;
}

// Rows of `len` elements `ld` apart from p.
int32_t check_rows(const char* name, const void* p, int64_t ld, int64_t len) {
  if (!ptr_aligned(p, 16)) return entry_fail(MOE_ERR_MISALIGNED, "%s must be 16-byte aligned", name);
  if (ld < len) return entry_fail(MOE_ERR_INVALID_ARG, "row stride of %s below the row's length", name);
  if (ld % 8) return entry_fail(MOE_ERR_MISALIGNED, "row stride of %s must be a multiple of 8", name);
  if (ld > (int64_t(1) << 31)) return entry_fail(MOE_ERR_INVALID_ARG, "row stride of %s too large", name);
  return MOE_OK;
}

// Launches a kernel whose grid.x is a multiple of the cluster size, with PDL.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), dim3 grid, int cluster, size_t smem,
                           cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

cudaError_t launch_group(const int32_t* ids, int T, int NA, const Groups& g, cudaStream_t st) {
  static DeviceOnce once;
  const size_t smem = (32 * static_cast<size_t>(NA + 1) + 2 * (NA + 2)) * 4;
  const cudaError_t e = set_smem_limit_once(group_kernel, (32 * 1025 + 2 * 1026) * 4, once);
  if (e != cudaSuccess) return e;
  return launch_pdl(group_kernel, dim3(1), dim3(kGroupThreads), smem, st, ids, T, NA, g);
}

// CTAs that share a unit of work: the cluster sizes up to 8 while the units
// leave SMs idle (two CTAs an SM).
int cluster_for(int64_t units, int sms) {
  int c = 1;
  while (c < 8 && units * c < 2 * sms) c *= 2;
  return c;
}

int rt_of(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8; }

cudaError_t launch_shrink_x(const ShrinkArgs& a, int64_t tiles, int sms, cudaStream_t st) {
  const int c = cluster_for(tiles, sms);
  const dim3 grid(static_cast<unsigned>(tiles * c));
  switch (rt_of(a.r)) {
    case 1: return launch_cluster(shrink_x_kernel<1>, grid, c, 0, st, a);
    case 2: return launch_cluster(shrink_x_kernel<2>, grid, c, 0, st, a);
    case 4: return launch_cluster(shrink_x_kernel<4>, grid, c, 0, st, a);
    default: return launch_cluster(shrink_x_kernel<8>, grid, c, 0, st, a);
  }
}

template <bool F32>
cudaError_t launch_shrink_d(const ShrinkArgs& a, int64_t tiles, int sms, cudaStream_t st) {
  const int c = cluster_for(tiles, sms);
  const dim3 grid(static_cast<unsigned>(tiles * c));
  switch (rt_of(a.r)) {
    case 1: return launch_cluster(shrink_d_kernel<1, F32>, grid, c, 0, st, a);
    case 2: return launch_cluster(shrink_d_kernel<2, F32>, grid, c, 0, st, a);
    case 4: return launch_cluster(shrink_d_kernel<4, F32>, grid, c, 0, st, a);
    default: return launch_cluster(shrink_d_kernel<8, F32>, grid, c, 0, st, a);
  }
}

template <int RT, bool ROWS, bool F32>
cudaError_t launch_expand_as(ExpandArgs a, int64_t tiles, int sms, cudaStream_t st) {
  constexpr int unit = kWarps * (ROWS ? 8 * (RT == 8 ? 4 : 8) : 32);   // features of a CTA's round
  const int rounds = (a.N + unit - 1) / unit;
  // as many rounds a CTA as leave four CTAs an SM
  int64_t per = tiles * rounds / (4 * static_cast<int64_t>(sms));
  per = per < 1 ? 1 : per > rounds ? rounds : per;
  a.per_cta = static_cast<int>(per) * unit;
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>((rounds + per - 1) / per));
  return launch_pdl(expand_kernel<RT, ROWS, F32>, grid, dim3(kThreads), 0, st, a);
}

template <bool ROWS, bool F32>
cudaError_t launch_expand(const ExpandArgs& a, int64_t tiles, int sms, cudaStream_t st) {
  switch (rt_of(a.r)) {
    case 1: return launch_expand_as<1, ROWS, F32>(a, tiles, sms, st);
    case 2: return launch_expand_as<2, ROWS, F32>(a, tiles, sms, st);
    case 4: return launch_expand_as<4, ROWS, F32>(a, tiles, sms, st);
    default: return launch_expand_as<8, ROWS, F32>(a, tiles, sms, st);
  }
}

template <int RT, bool F32>
cudaError_t launch_grad_as(const GradArgs& a, int NA, int64_t T, int sms, cudaStream_t st) {
  static DeviceOnce once;
  constexpr size_t smem = grad_smem<RT, F32>();
  const cudaError_t e = set_smem_limit_once(grad_kernel<RT, F32>, smem, once);
  if (e != cudaSuccess) return e;
  const int fw = 8 * grad_fl<RT, F32>();
  const int64_t slabs = (a.N + fw - 1) / fw;
  int c = cluster_for(slabs * NA, sms);
  while (c > 1 && static_cast<int64_t>(c) * kGradTok > T) c /= 2;   // rounds to share
  return launch_cluster(grad_kernel<RT, F32>, dim3(static_cast<unsigned>(slabs * c), NA), c, smem,
                        st, a);
}

template <bool F32>
cudaError_t launch_grad(const GradArgs& a, int NA, int64_t T, int sms, cudaStream_t st) {
  switch (rt_of(a.r)) {
    case 1: return launch_grad_as<1, F32>(a, NA, T, sms, st);
    case 2: return launch_grad_as<2, F32>(a, NA, T, sms, st);
    case 4: return launch_grad_as<4, F32>(a, NA, T, sms, st);
    default: return launch_grad_as<8, F32>(a, NA, T, sms, st);
  }
}

struct AdapterCall {
  AdapterWs w;
  Groups g;
  float *v, *u;
  int64_t tiles;
  int sms;
  cudaStream_t st;
};

AdapterCall adapter_call(const moe_adapter_shape* s, bool backward, void* workspace, int sms,
                         void* stream) {
  AdapterCall c;
  uint8_t* base = static_cast<uint8_t*>(workspace);
  c.w = adapter_ws(s, backward);
  c.g.perm = reinterpret_cast<int32_t*>(base + c.w.perm);
  c.g.offsets = reinterpret_cast<int32_t*>(base + c.w.offsets);
  c.g.tiles = reinterpret_cast<int4*>(base + c.w.tiles);
  c.g.num_tiles = reinterpret_cast<int32_t*>(base + c.w.num_tiles);
  c.v = reinterpret_cast<float*>(base + c.w.v);
  c.u = reinterpret_cast<float*>(base + c.w.u);
  c.tiles = max_tiles(s->num_tokens, s->num_adapters);
  c.sms = sms;
  c.st = static_cast<cudaStream_t>(stream);
  return c;
}

ShrinkArgs shrink_args(const AdapterCall& c, const void* src, int64_t ld, const void* pool,
                       const float* scale, float* dst, int r, int K) {
  ShrinkArgs a;
  a.src = src;
  a.ld = ld;
  a.pool = static_cast<const __nv_bfloat16*>(pool);
  a.scale = scale;
  a.dst = dst;
  a.perm = c.g.perm;
  a.tiles = c.g.tiles;
  a.num_tiles = c.g.num_tiles;
  a.r = r;
  a.K = K;
  return a;
}

ExpandArgs expand_args(const AdapterCall& c, const float* v, const void* pool, const float* scale,
                       const void* base, int64_t ld_base, void* out, int64_t ld_out, int r, int N) {
  ExpandArgs a;
  a.v = v;
  a.pool = static_cast<const __nv_bfloat16*>(pool);
  a.scale = scale;
  a.base = base;
  a.ld_base = ld_base;
  a.out = out;
  a.ld_out = ld_out;
  a.perm = c.g.perm;
  a.tiles = c.g.tiles;
  a.num_tiles = c.g.num_tiles;
  a.r = r;
  a.N = N;
  a.per_cta = 0;
  return a;
}

GradArgs grad_args(const AdapterCall& c, const float* left, const float* scale, const void* src,
                   int64_t ld, float* out, int r, int N, bool transposed) {
  GradArgs a;
  a.left = left;
  a.scale = scale;
  a.src = src;
  a.ld = ld;
  a.perm = c.g.perm;
  a.offsets = c.g.offsets;
  a.out = out;
  a.r = r;
  a.N = N;
  a.transposed = transposed;
  return a;
}

int32_t check_common(const moe_adapter_shape* s, const void* x, int64_t ld_x, const int32_t* ids,
                     const void* a, const void* b, const float* scale, const void* workspace,
                     size_t workspace_bytes, bool backward) {
  if (!x || !ids || !a || !b || !workspace)
    return entry_fail(MOE_ERR_INVALID_ARG, "x, adapter_ids, a, b or workspace is NULL");
  int32_t rc = check_rows("x", x, ld_x, s->in_features);
  if (rc != MOE_OK) return rc;
  if (!ptr_aligned(a, 16) || !ptr_aligned(b, 16))
    return entry_fail(MOE_ERR_MISALIGNED, "a and b must be 16-byte aligned");
  if (!ptr_aligned(ids, 4) || !ptr_aligned(scale, 4))
    return entry_fail(MOE_ERR_MISALIGNED, "adapter_ids and scale must be 4-byte aligned");
  if (!ptr_aligned(workspace, kWsAlign))
    return entry_fail(MOE_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  const size_t need = adapter_ws(s, backward).total;
  if (workspace_bytes < need)
    return entry_fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, needs %zu",
                      workspace_bytes, need);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_adapter_workspace_size(const moe_adapter_shape* shape, int32_t backward) {
  if (moe::check_adapter(shape) != MOE_OK) return 0;
  return moe::adapter_ws(shape, backward != 0).total;
}

extern "C" int32_t moe_adapter_forward(const moe_adapter_shape* s, const void* x, int64_t ld_x,
                                       const int32_t* adapter_ids, const void* a, const void* b,
                                       const float* scale, const void* base, int64_t ld_base,
                                       void* out, int64_t ld_out, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  using namespace moe;
  int32_t rc = check_adapter(s);
  if (rc != MOE_OK) return rc;
  if (s->num_tokens == 0) return MOE_OK;
  rc = check_common(s, x, ld_x, adapter_ids, a, b, scale, workspace, workspace_bytes, false);
  if (rc != MOE_OK) return rc;
  if (!out) return entry_fail(MOE_ERR_INVALID_ARG, "out is NULL");
  if ((rc = check_rows("out", out, ld_out, s->out_features)) != MOE_OK) return rc;
  if (base && (rc = check_rows("base", base, ld_base, s->out_features)) != MOE_OK) return rc;
  int sms = 0;
  if ((rc = check_device(&sms)) != MOE_OK) return rc;
  const AdapterCall c = adapter_call(s, false, workspace, sms, stream);
  cudaError_t e = launch_group(adapter_ids, s->num_tokens, s->num_adapters, c.g, c.st);
  if (e == cudaSuccess)
    e = launch_shrink_x(shrink_args(c, x, ld_x, a, nullptr, c.v, s->rank, s->in_features), c.tiles,
                        sms, c.st);
  if (e == cudaSuccess) {
    const ExpandArgs ea = expand_args(c, c.v, b, scale, base, ld_base, out, ld_out, s->rank,
                                      s->out_features);
    e = s->out_dtype == MOE_DTYPE_F32 ? launch_expand<false, true>(ea, c.tiles, sms, c.st)
                                      : launch_expand<false, false>(ea, c.tiles, sms, c.st);
  }
  return entry_launched(e);
}

extern "C" int32_t moe_adapter_backward(const moe_adapter_shape* s, const void* dout,
                                        int64_t ld_dout, const void* x, int64_t ld_x,
                                        const int32_t* adapter_ids, const void* a, const void* b,
                                        const float* scale, const void* dx_base,
                                        int64_t ld_dx_base, void* dx, int64_t ld_dx, float* da,
                                        float* db, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  using namespace moe;
  int32_t rc = check_adapter(s);
  if (rc != MOE_OK) return rc;
  if (!da != !db) return entry_fail(MOE_ERR_INVALID_ARG, "da and db go together");
  if (!ptr_aligned(da, 16) || !ptr_aligned(db, 16))
    return entry_fail(MOE_ERR_MISALIGNED, "da and db must be 16-byte aligned");
  const bool tokens = s->num_tokens > 0;
  if (tokens) {
    rc = check_common(s, x, ld_x, adapter_ids, a, b, scale, workspace, workspace_bytes, true);
    if (rc != MOE_OK) return rc;
    if (!dout) return entry_fail(MOE_ERR_INVALID_ARG, "dout is NULL");
    if ((rc = check_rows("dout", dout, ld_dout, s->out_features)) != MOE_OK) return rc;
    if (dx && (rc = check_rows("dx", dx, ld_dx, s->in_features)) != MOE_OK) return rc;
    if (dx && (dx == x || dx == dout))
      return entry_fail(MOE_ERR_INVALID_ARG, "dx must not be x or dout");
    if (dx && dx_base && (rc = check_rows("dx_base", dx_base, ld_dx_base, s->in_features)) != MOE_OK)
      return rc;
  }
  if (!tokens && !da) return MOE_OK;
  if (!dx && !da) return MOE_OK;
  int sms = 0;
  if ((rc = check_device(&sms)) != MOE_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t na_r = static_cast<size_t>(s->num_adapters) * s->rank;
  if (!tokens) {   // gradients of nothing
    cudaError_t e = cudaMemsetAsync(da, 0, na_r * s->in_features * 4, st);
    if (e == cudaSuccess) e = cudaMemsetAsync(db, 0, na_r * s->out_features * 4, st);
    return entry_launched(e);
  }
  const bool f32 = s->out_dtype == MOE_DTYPE_F32;
  const int T = s->num_tokens, NA = s->num_adapters, r = s->rank;
  const AdapterCall c = adapter_call(s, true, workspace, sms, stream);
  cudaError_t e = launch_group(adapter_ids, T, NA, c.g, st);
  if (e == cudaSuccess) {
    const ShrinkArgs sa = shrink_args(c, dout, ld_dout, b, scale, c.u, r, s->out_features);
    e = f32 ? launch_shrink_d<true>(sa, c.tiles, sms, st) : launch_shrink_d<false>(sa, c.tiles, sms, st);
  }
  if (e == cudaSuccess && dx)
    e = launch_expand<true, false>(expand_args(c, c.u, a, nullptr, dx_base, ld_dx_base, dx, ld_dx, r,
                                               s->in_features), c.tiles, sms, st);
  if (e == cudaSuccess && da)
    e = launch_grad<false>(grad_args(c, c.u, nullptr, x, ld_x, da, r, s->in_features, false), NA, T,
                           sms, st);
  if (e == cudaSuccess && da)
    e = launch_shrink_x(shrink_args(c, x, ld_x, a, nullptr, c.v, r, s->in_features), c.tiles, sms, st);
  if (e == cudaSuccess && da) {
    const GradArgs ga = grad_args(c, c.v, scale, dout, ld_dout, db, r, s->out_features, true);
    e = f32 ? launch_grad<true>(ga, NA, T, sms, st) : launch_grad<false>(ga, NA, T, sms, st);
  }
  return entry_launched(e);
}
