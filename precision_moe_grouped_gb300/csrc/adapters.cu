// adapters.cu -- low-rank adapters of many requests beside a shared
// projection: out = base + scale_a B_a (A_a x), and its gradients.
//
// Tokens are grouped by adapter on the device into tiles of up to 64 tokens
// (group_kernel; batches of up to kSmallTokens group inside the product
// kernels, tiles of up to 16), then:
//   forward:   w = s A x                contracts over H      (shrink_x)
//              out = base + B w         contracts over r      (expand)
//   backward:  w = s A x, u = s B^T dout                      (shrink_x, shrink_d)
//              dx = dx_base + A^T u                           (expand)
//              dA = sum u x^T, dB = sum dout w^T              (grad: contracts over
//                                                              the adapter's tokens)
// With ranks of 8 to 128 every one of these does r multiply-adds for each
// element it moves, far below the ~290 operations a byte at which tensor
// throughput would bind, so the layout serves the memory stream: operands
// go straight from global memory into the fragments of mma.sync (16x8x16,
// bf16, float accumulators), with no staging and no barrier in the loops.
// The contraction index and the column index of a fragment are free to be
// permuted as long as both operands (or the store) use the same order; each
// kernel picks the order in which a lane's share is contiguous in memory.
// (tcgen05 would need the gathered rows staged in shared memory through
// another pass, for tiles whose N is r.)
//
// u and w are computed in float and leave as bf16 planes that add up to them:
// hi = bf16(v), then mid (and lo) the rounded rests.  Two planes (an error
// below 2^-17) feed the products that are rounded to bf16 or added to a
// float base, three (2^-25) the float sums dA and dB.  A float dout is split the
// same way.  Ranks are padded with zeros to RP = 16, 32, 64 or 128.
#include <cuda_bf16.h>

#include "cluster.cuh"
#include "entry.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kTile = 64;            // tokens of a tile
constexpr int kSmallTile = 16;       // and of a small batch's
constexpr int kSmallTokens = 256;
constexpr int kGroupThreads = 1024;
constexpr int kWarps = 8;            // warps of the product kernels
constexpr int kThreads = 32 * kWarps;

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The low (high) halves of two words: element 0 (1) of two rows.
template <int ODD>
__device__ __forceinline__ uint32_t pair(uint32_t a, uint32_t b) {
  return __byte_perm(a, b, ODD ? 0x7632 : 0x5410);
}

__device__ __forceinline__ uint32_t word(__nv_bfloat16 a, __nv_bfloat16 b) {
  return static_cast<uint32_t>(__bfloat16_as_ushort(a)) |
         static_cast<uint32_t>(__bfloat16_as_ushort(b)) << 16;
}

// One bf16 plane of (x, y), which keep the rests.  Beyond bf16's finite range
// there is no rest (inf - inf would make an infinity a NaN).
__device__ __forceinline__ uint32_t peel(float& x, float& y) {
  const __nv_bfloat16 a = __float2bfloat16_rn(x), b = __float2bfloat16_rn(y);
  const float fa = __bfloat162float(a), fb = __bfloat162float(b);
  x = fabsf(fa) < INFINITY ? x - fa : 0.f;
  y = fabsf(fb) < INFINITY ? y - fb : 0.f;
  return word(a, b);
}

// 16 bytes of a stream that no other warp of the SM wants.
__device__ __forceinline__ uint4 ldg16_stream(const void* p) {
  uint4 q;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
               : "l"(p));
  return q;
}
__device__ __forceinline__ uint4 ldg16(const void* p) { return __ldg(static_cast<const uint4*>(p)); }

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

// ------------------------------------------------------------ grouping
struct Groups {
  int32_t* perm;      // [tiles, kTile] token of each slot, -1 past a tile's end
  int32_t* counts;    // [NA + 1] tokens of adapter a; [NA]: without one
  int32_t* first;     // [NA + 2] first tile of adapter a
  int4* tiles;        // (adapter or -1, tokens, 0, 0)
  int32_t* num_tiles;
};

__host__ __device__ inline int64_t max_tiles(int64_t T, int64_t NA) {
  return T / kTile + (NA + 1 < T ? NA + 1 : T) + 1;
}

// Slots of the tokens in the order (adapter 0 .. NA-1, none), stable in the
// token.  One CTA: warp w owns the w-th contiguous 32nd of the tokens and a
// histogram of it; the histograms' running sums give each warp its bases, and
// a warp hands out slots to its tokens in order.
__global__ void __launch_bounds__(kGroupThreads) group_kernel(const int32_t* __restrict__ ids,
                                                              int T, int NA, Groups g) {
  extern __shared__ __align__(16) uint8_t sm[];
  const int C = NA + 1;                 // columns: the adapters and "none"
  int32_t* hist = reinterpret_cast<int32_t*>(sm);   // [32][C]
  int32_t* count = hist + 32 * C;       // [C + 1] tokens
  int32_t* tfirst = count + C + 1;      // [C + 1] first tile
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
    count[c] = sum;
    g.counts[c] = sum;
  }
  __syncthreads();
  if (warp == 0) {   // exclusive sum of the columns' tiles
    int run = 0;
    for (int c0 = 0; c0 < C; c0 += 32) {
      const int c = c0 + lane;
      const int n = c < C ? (count[c] + kTile - 1) / kTile : 0;
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int px = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += px;
      }
      if (c < C) tfirst[c] = run + x - n;
      run += __shfl_sync(0xFFFFFFFFu, x, 31);
    }
    if (lane == 0) tfirst[C] = run, *g.num_tiles = run;
  }
  __syncthreads();
  for (int c = threadIdx.x; c <= C; c += kGroupThreads) g.first[c] = tfirst[c];
  const int tiles = tfirst[C];
  for (int i = threadIdx.x; i < tiles; i += kGroupThreads) {
    int lo = 0, hi = C;                 // the last column whose first tile is at or before i
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tfirst[mid] <= i) lo = mid;
      else hi = mid;
    }
    g.tiles[i] = make_int4(lo < NA ? lo : -1, min(kTile, count[lo] - (i - tfirst[lo]) * kTile), 0, 0);
  }
  for (int i = threadIdx.x; i < C * kTile; i += kGroupThreads) {   // the ends of the last tiles
    const int c = i / kTile, slot = count[c] + i % kTile;
    if (slot < (tfirst[c + 1] - tfirst[c]) * kTile)
      g.perm[static_cast<int64_t>(tfirst[c]) * kTile + slot] = -1;
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
      g.perm[static_cast<int64_t>(tfirst[c]) * kTile + base + rank] = static_cast<int32_t>(t);
      if (rank == 0) hist[warp * C + c] = base + __popc(same);
    }
    __syncwarp();
  }
}

// A tile as the product kernels see it: adapter (-1: none), tokens, first slot
// of its rows in the planes and in perm.
struct Tile {
  int adapter, n;
  int64_t slot;
};

// Where the tiles come from: the group kernel's lists, or (SMALL) the ids.
struct TileSource {
  const int32_t* ids;
  int32_t T, NA;
  const int32_t* perm;
  const int4* tiles;
  const int32_t* num_tiles;
};

// SMALL: CTA t of the grid leads the tile that begins with token t, if t is
// the first, 17th, 33rd, ... token of its adapter: the token and the next 15
// that share it.  False: no tile.  tok [kSmallTile] receives the tokens.
template <bool SMALL>
__device__ __forceinline__ bool find_tile(const TileSource& src, int i, Tile* tile, int32_t* tok) {
  if constexpr (!SMALL) {
    if (i >= *src.num_tiles) return false;
    const int4 q = src.tiles[i];
    tile->adapter = q.x;
    tile->n = q.y;
    tile->slot = static_cast<int64_t>(i) * kTile;
    return true;
  } else {
    static_assert(kSmallTokens <= kThreads, "a thread per token");
    __shared__ unsigned same[kThreads / 32];
    const unsigned NA = static_cast<unsigned>(src.NA);
    const int want = src.ids[i], mine = static_cast<int>(threadIdx.x) < src.T ? src.ids[threadIdx.x] : 0;
    const bool none = static_cast<unsigned>(want) >= NA;
    const bool eq = static_cast<int>(threadIdx.x) < src.T &&
                    (none ? static_cast<unsigned>(mine) >= NA : mine == want);
    const unsigned b = __ballot_sync(0xFFFFFFFFu, eq);
    if ((threadIdx.x & 31) == 0) same[threadIdx.x >> 5] = b;
    if (threadIdx.x < kSmallTile) tok[threadIdx.x] = -1;
    __syncthreads();
    int before_i = 0, before_me = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const int n = __popc(same[w]);
      total += n;
      if (w < (i >> 5)) before_i += n;
      if (w < static_cast<int>(threadIdx.x >> 5)) before_me += n;
    }
    before_i += __popc(same[i >> 5] & ((1u << (i & 31)) - 1));
    before_me += __popc(b & ((1u << (threadIdx.x & 31)) - 1));
    if (before_i % kSmallTile != 0) return false;
    if (eq && before_me >= before_i && before_me < before_i + kSmallTile)
      tok[before_me - before_i] = static_cast<int32_t>(threadIdx.x);
    __syncthreads();
    tile->adapter = none ? -1 : want;
    tile->n = min(kSmallTile, total - before_i);
    tile->slot = static_cast<int64_t>(i) * kSmallTile;
    return true;
  }
}

// ------------------------------------------- w = s A x, u = s B^T dout
// Low-rank rows leave as planes: `row` two planes [slots, RP], `col` three
// planes [tiles, RP, kTile] (each may be null); slots past a tile's tokens are
// zero.
struct Planes {
  __nv_bfloat16* row;
  __nv_bfloat16* col;
  int64_t size;        // elements of a plane
};

struct ShrinkArgs {
  TileSource tiles;
  const void* src;     // x (bf16) or dout
  int64_t ld;
  const __nv_bfloat16* pool;
  const float* scale;  // null: 1
  Planes dst;
  int32_t r, K;        // K: contracted length
};

// Sums the CTA's WK partial tiles [WK][NTOK][RP + 1] in warp order, then the
// cluster's in rank order, and writes the planes.
template <int RP, int WK, int NTOK>
__device__ __forceinline__ void finish_tile(float* red, const Tile& tile, float scale,
                                            const Planes& dst) {
  constexpr int RS = RP + 1;
  __syncthreads();
  if constexpr (WK > 1) {
    for (int i = threadIdx.x; i < NTOK * RS; i += kThreads) {
      float v = red[i];
#pragma unroll
      for (int w = 1; w < WK; ++w) v += red[w * NTOK * RS + i];
      red[i] = v;
    }
  }
  const int S = static_cast<int>(cluster_size());
  if (S > 1) cluster_sync();
  else __syncthreads();
  const int step = S * kThreads, start = static_cast<int>(cluster_rank()) * kThreads + threadIdx.x;
  auto value = [&](int t, int j) {
    if (S == 1) return red[t * RS + j] * scale;
    float v = 0.f;
    for (int c = 0; c < S; ++c) v += cluster_load(red + t * RS + j, c);
    return v * scale;
  };
  if (dst.row)
    for (int i = start; i < NTOK * RP / 2; i += step) {   // two ranks of a token
      const int t = i / (RP / 2), j = 2 * (i % (RP / 2));
      float x = value(t, j), y = value(t, j + 1);
      __nv_bfloat16* o = dst.row + (tile.slot + t) * RP + j;
      *reinterpret_cast<uint32_t*>(o) = peel(x, y);
      *reinterpret_cast<uint32_t*>(o + dst.size) = peel(x, y);
    }
  if (dst.col)
    for (int i = start; i < NTOK * RP / 2; i += step) {   // two tokens of a rank
      const int j = i / (NTOK / 2), t = 2 * (i % (NTOK / 2));
      float x = value(t, j), y = value(t + 1, j);
      __nv_bfloat16* o = dst.col + tile.slot * RP + j * kTile + t;
      *reinterpret_cast<uint32_t*>(o) = peel(x, y);
      *reinterpret_cast<uint32_t*>(o + dst.size) = peel(x, y);
      *reinterpret_cast<uint32_t*>(o + 2 * dst.size) = peel(x, y);
    }
  if (S > 1) cluster_sync();   // no CTA leaves while another reads its shared memory
}

// The 32-element chunks of K a warp contracts: its share of the cluster's.
__device__ __forceinline__ int2 chunk_range(int K, int wk, int WK) {
  const int chunks = (K + 31) / 32, parts = static_cast<int>(cluster_size()) * WK;
  const int part = static_cast<int>(cluster_rank()) * WK + wk;
  return make_int2(static_cast<int>(static_cast<int64_t>(chunks) * part / parts),
                   static_cast<int>(static_cast<int64_t>(chunks) * (part + 1) / parts));
}

// Shapes of shrink_x: 8-token columns of a warp, warps side by side.
template <int RT, bool SMALL>
struct ShrinkX {
  static constexpr int NTOK = SMALL ? kSmallTile : kTile;
  static constexpr int NT = SMALL ? 2 : RT == 1 ? 8 : RT == 8 ? 2 : 4;
  static constexpr int WT = NTOK / (8 * NT), WK = kWarps / WT;
  static constexpr int RP = 16 * RT;
  static constexpr size_t smem = sizeof(float) * WK * NTOK * (RP + 1);
};

// Rank is MMA-M, tokens are MMA-N: lane (g, t) of a chunk loads the 8
// elements at 8 t of rank rows g and g + 8 and of token g, two MMAs deep.
template <int RT, bool SMALL>
__device__ __forceinline__ void shrink_x_tile(const ShrinkArgs& a, const Tile& tile,
                                              const int32_t* tok, float* red) {
  using C = ShrinkX<RT, SMALL>;
  constexpr int NT = C::NT, WT = C::WT, WK = C::WK, RS = C::RP + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int wt = warp % WT, wk = warp / WT;
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
    const int64_t id = SMALL ? tok[i] : a.tiles.perm[tile.slot + i];
    row[j] = id >= 0 ? src + id * a.ld + 8 * t : nullptr;
  }
  const int live = min(NT, (tile.n - 8 * wt * NT + 7) / 8);   // columns with a token
  const __nv_bfloat16* pool = a.pool + static_cast<int64_t>(tile.adapter) * a.r * a.K + 8 * t;
  const int2 c = chunk_range(a.K, wk, WK);
  if (live > 0)
#pragma unroll(SMALL ? 4 : 1)
    for (int k = 32 * c.x; k < 32 * c.y; k += 32) {
      const bool in = k + 8 * t < a.K;
      uint4 p[RT][2], x[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j)
        x[j] = in && row[j] ? ldg16_stream(row[j] + k) : make_uint4(0, 0, 0, 0);
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
        if (j < live)
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            mma(acc[i][j], p[i][0].x, p[i][1].x, p[i][0].y, p[i][1].y, x[j].x, x[j].y);
            mma(acc[i][j], p[i][0].z, p[i][1].z, p[i][0].w, p[i][1].w, x[j].z, x[j].w);
          }
    }
  float* mine = red + wk * C::NTOK * RS;
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        mine[(8 * (wt * NT + j) + 2 * t + (q & 1)) * RS + 16 * i + g + 8 * (q >> 1)] = acc[i][j][q];
  const float scale = a.scale ? __ldg(a.scale + tile.adapter) : 1.0f;
  finish_tile<C::RP, WK, C::NTOK>(red, tile, scale, a.dst);
}

// Cluster of S CTAs per tile, all their warps sharing out the chunks of K.
template <int RT, bool SMALL>
__global__ void __launch_bounds__(kThreads, RT == 8 ? 1 : 2) shrink_x_kernel(const ShrinkArgs a) {
  extern __shared__ __align__(16) uint8_t sm[];
  __shared__ int32_t tok[kSmallTile];
  griddep_wait();
  griddep_launch_dependents();
  Tile tile;
  if (!find_tile<SMALL>(a.tiles, blockIdx.x / cluster_size(), &tile, tok) || tile.adapter < 0) return;
  shrink_x_tile<RT, SMALL>(a, tile, tok, reinterpret_cast<float*>(sm));
}

// Eight values of dout at p as four words of two bf16 (and, from float, the
// words of the rests).
template <bool F32>
__device__ __forceinline__ void load8(const void* p, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  if constexpr (F32) {
    const uint4 q[2] = {ldg16_stream(p), ldg16_stream(static_cast<const uint4*>(p) + 1)};
    const uint32_t* w = &q[0].x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x = __uint_as_float(w[2 * i]), y = __uint_as_float(w[2 * i + 1]);
      hi[i] = peel(x, y);
      lo[i] = peel(x, y);
    }
  } else {
    const uint4 a = ldg16_stream(p);
    hi[0] = a.x, hi[1] = a.y, hi[2] = a.z, hi[3] = a.w;
  }
}

template <int RT>
struct ShrinkD {
  static constexpr int MT = RT == 1 ? 4 : RT == 2 ? 2 : 1;   // 16-token rows of a warp
  static constexpr int WT = kTile / (16 * MT), WK = kWarps / WT;
  static constexpr int RP = 16 * RT;
  static constexpr size_t smem = sizeof(float) * WK * kTile * (RP + 1);
};

// As shrink_x with the pool contracted over its rows (B [N, r]): tokens are
// MMA-M, ranks MMA-N.  Lane (g, t) takes the 8 pool rows at 8 t of a chunk,
// ranks 2 RT g .. + 2 RT - 1; column g of rank tile i is rank 2 RT g + i, so
// that a lane's words of two rows pair up into fragments.
template <int RT, bool F32>
__device__ __forceinline__ void shrink_d_tile(const ShrinkArgs& a, const Tile& tile, float* red) {
  using C = ShrinkD<RT>;
  constexpr int MT = C::MT, WT = C::WT, WK = C::WK, RS = C::RP + 1;
  constexpr size_t ES = F32 ? 4 : 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int wt = warp % WT, wk = warp / WT;
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
      const int64_t id = a.tiles.perm[tile.slot + 16 * (wt * MT + m) + 8 * h + g];
      row[m][h] = id >= 0 ? static_cast<const uint8_t*>(a.src) + (id * a.ld + 8 * t) * ES : nullptr;
    }
  const int live = min(MT, (tile.n - 16 * wt * MT + 15) / 16);
  const __nv_bfloat16* pool = a.pool + static_cast<int64_t>(tile.adapter) * a.r * a.K;
  const int2 c = chunk_range(a.K, wk, WK);
  const int rank0 = 2 * RT * g;   // the lane's ranks exist, by halves of 8 at RT = 8
  if (live > 0)
    for (int k = 32 * c.x; k < 32 * c.y; k += 32) {
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
          for (int j = 0; j < RT; ++j) {
            const uint32_t* const w0 = w[4 * half];
            const uint32_t r0 = w0[j], r1 = w[4 * half + 1][j], r2 = w[4 * half + 2][j],
                           r3 = w[4 * half + 3][j];
            const uint32_t b[2][2] = {{pair<0>(r0, r1), pair<0>(r2, r3)},
                                      {pair<1>(r0, r1), pair<1>(r2, r3)}};
#pragma unroll
            for (int o = 0; o < 2; ++o) {
              float(&d)[4] = acc[m][2 * j + o];
              mma(d, h0[2 * half], h1[2 * half], h0[2 * half + 1], h1[2 * half + 1], b[o][0], b[o][1]);
              if constexpr (F32)
                mma(d, l0[2 * half], l1[2 * half], l0[2 * half + 1], l1[2 * half + 1], b[o][0], b[o][1]);
            }
          }
      }
    }
  float* mine = red + wk * kTile * RS;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < 2 * RT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        mine[(16 * (wt * MT + m) + g + 8 * (q >> 1)) * RS + 2 * RT * (2 * t + (q & 1)) + j] = acc[m][j][q];
  const float scale = a.scale ? __ldg(a.scale + tile.adapter) : 1.0f;
  finish_tile<C::RP, WK, kTile>(red, tile, scale, a.dst);
}

// Both of the backward's, in one launch: the first `d_units` clusters take
// dout, the others x.
template <int RT, bool F32>
__global__ void __launch_bounds__(kThreads, RT == 8 ? 1 : 2)
    shrink_both_kernel(const ShrinkArgs d, const ShrinkArgs x, int d_units) {
  extern __shared__ __align__(16) uint8_t sm[];
  griddep_wait();
  griddep_launch_dependents();
  int unit = blockIdx.x / cluster_size();
  Tile tile;
  if (unit < d_units) {
    if (!find_tile<false>(d.tiles, unit, &tile, nullptr) || tile.adapter < 0) return;
    shrink_d_tile<RT, F32>(d, tile, reinterpret_cast<float*>(sm));
  } else {
    unit -= d_units;
    if (!find_tile<false>(x.tiles, unit, &tile, nullptr) || tile.adapter < 0) return;
    shrink_x_tile<RT, false>(x, tile, nullptr, reinterpret_cast<float*>(sm));
  }
}

// ---------------------------------------- out = base + pool-product of w
struct ExpandArgs {
  TileSource tiles;
  Planes v;              // row planes
  const __nv_bfloat16* pool;
  const void* base;      // null: zero
  int64_t ld_base;
  void* out;
  int64_t ld_out;
  int32_t r, N;          // N: output features
};

// Eight consecutive values of the base (zero without one).
template <bool F32>
struct Base8 {
  uint4 q[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p) {
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i)
      q[i] = p ? static_cast<const uint4*>(p)[i] : make_uint4(0, 0, 0, 0);
  }
  // out = base + d, rounded once
  __device__ __forceinline__ void store(void* out, const float (&d)[8]) const {
    uint4 o[F32 ? 2 : 1];
    const uint32_t* w = &q[0].x;
    uint32_t* p = &o[0].x;
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = __float_as_uint(__uint_as_float(w[i]) + d[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        p[i] = word(__float2bfloat16_rn(__uint_as_float(w[i] << 16) + d[2 * i]),
                    __float2bfloat16_rn(__uint_as_float(w[i] & 0xFFFF0000u) + d[2 * i + 1]));
    }
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) static_cast<uint4*>(out)[i] = o[i];
  }
};

// Features of a warp: as many as hold its fragments (RT / 4 registers each)
// beside the accumulators.
template <int RT>
constexpr int expand_width() { return RT >= 4 ? 32 : 64; }

// A warp takes a group of features, holds the pool's fragments of it and runs
// the tile's tokens, 16 at a time.  Tokens are MMA-M, features MMA-N.
//   !ROWS: pool [N, r]: column n of feature tile j is feature
//          32 (j / 4) + 8 (n / 2) + 2 (j % 4) + n % 2
//   ROWS:  pool [r, N]: lane (g, t) of a 16-rank step loads FL = 8 (4)
//          features of rank rows 4 t .. + 3; column n of tile j is FL n + j
// so that a lane ends with 8 consecutive features of its two tokens, twice.
// The pool's, the base's and the tile's loads do not depend on the kernel
// before (inputs, and lists that were complete before that one began): they
// are issued ahead of the grid wait.
template <int RT, bool ROWS, bool F32, bool SMALL>
__device__ __forceinline__ void expand_tile(const ExpandArgs& a, const Tile& tile, int f,
                                            const int32_t* tok) {
  constexpr int FW = expand_width<RT>();
  constexpr int JT = FW / 8;                  // 8-feature tiles of a warp
  constexpr int FL = FW / 8;                  // ROWS: features a lane loads
  constexpr int RP = 16 * RT;
  constexpr int NB = FW / 32;                 // runs of 8 features of a lane
  constexpr size_t ES = F32 ? 4 : 2;
  constexpr int MT = SMALL ? 1 : kTile / 16;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint32_t b[RT][JT][2];
  const __nv_bfloat16* pool = a.pool + static_cast<int64_t>(tile.adapter) * a.r * a.N;
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
      for (int j = 0; j < JT / 2; ++j) {
        b[i][2 * j][0] = pair<0>(w[0][j], w[1][j]);
        b[i][2 * j][1] = pair<0>(w[2][j], w[3][j]);
        b[i][2 * j + 1][0] = pair<1>(w[0][j], w[1][j]);
        b[i][2 * j + 1][1] = pair<1>(w[2][j], w[3][j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < JT; ++j) {
        const int n = f + 32 * (j / 4) + 8 * (g >> 1) + 2 * (j % 4) + (g & 1), rank = 16 * i + 4 * t;
        uint32_t w[2] = {0, 0};
        if (n < a.N && rank < a.r) load_words<2>(pool + static_cast<int64_t>(n) * a.r + rank, w);
        b[i][j][0] = w[0];
        b[i][j][1] = w[1];
      }
    }
  }
  // first feature of the lane's run c
  auto run = [&](int c) { return ROWS && FL == 8 ? f + 16 * t + 8 * c : f + 32 * c + 8 * t; };
  const int live = (tile.n + 15) / 16;
  griddep_wait();   // (again in backward_out_kernel: returns at once)
#pragma unroll(ROWS || F32 || RT > 2 ? 1 : 2)
  for (int m = 0; m < MT; ++m) {
    if (m >= live) break;
    int64_t row[2];
    Base8<F32> base[2][NB];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = 16 * m + 8 * h + g;
      row[h] = SMALL ? tok[i] : a.tiles.perm[tile.slot + i];
      const uint8_t* p = a.base && row[h] >= 0
                             ? static_cast<const uint8_t*>(a.base) + row[h] * a.ld_base * ES
                             : nullptr;
#pragma unroll
      for (int c = 0; c < NB; ++c) base[h][c].load(p && run(c) < a.N ? p + run(c) * ES : nullptr);
    }
    float acc[JT][4];
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[j][q] = 0.f;
    const __nv_bfloat16* v = a.v.row + (tile.slot + 16 * m + g) * RP + 4 * t;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int plane = 0; plane < 2; ++plane) {
        const uint2 v0 = *reinterpret_cast<const uint2*>(v + plane * a.v.size + 16 * i);
        const uint2 v1 = *reinterpret_cast<const uint2*>(v + plane * a.v.size + 8 * RP + 16 * i);
#pragma unroll
        for (int j = 0; j < JT; ++j) mma(acc[j], v0.x, v1.x, v0.y, v1.y, b[i][j][0], b[i][j][1]);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (row[h] < 0) continue;
      uint8_t* out = static_cast<uint8_t*>(a.out) + row[h] * a.ld_out * ES;
#pragma unroll
      for (int c = 0; c < NB; ++c) {
        float d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if constexpr (ROWS && FL == 8) d[j] = acc[j][2 * h + c];
          else if constexpr (ROWS) d[j] = acc[j % 4][2 * h + j / 4];
          else d[j] = acc[4 * c + j / 2][2 * h + j % 2];
        }
        if (run(c) < a.N) base[h][c].store(out + run(c) * ES, d);
      }
    }
  }
}

// Tokens without an adapter: out = base, bit for bit (nothing to do when they
// are the same memory); the warp's features.
template <bool F32, bool SMALL>
__device__ __forceinline__ void copy_rows(const ExpandArgs& a, const Tile& tile, int f, int width,
                                          const int32_t* tok) {
  constexpr size_t ES = F32 ? 4 : 2;
  if (a.base == a.out && a.ld_base == a.ld_out) return;
  const int per = width / 8, lane = threadIdx.x & 31;
  for (int i = lane; i < tile.n * per; i += 32) {
    const int row = i / per, n = f + 8 * (i % per);
    if (n >= a.N) continue;
    const int64_t id = SMALL ? tok[row] : a.tiles.perm[tile.slot + row];
    Base8<F32> q;
    q.load(a.base ? static_cast<const uint8_t*>(a.base) + (id * a.ld_base + n) * ES : nullptr);
    uint4* out = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + (id * a.ld_out + n) * ES);
#pragma unroll
    for (int c = 0; c < (F32 ? 2 : 1); ++c) out[c] = q.q[c];
  }
}

// One CTA per (tile, 8 groups of features).
template <int RT, bool ROWS, bool F32, bool SMALL>
__global__ void __launch_bounds__(kThreads) expand_kernel(const ExpandArgs a) {
  constexpr int FW = expand_width<RT>();
  __shared__ int32_t tok[kSmallTile];
  griddep_launch_dependents();
  Tile tile;
  const bool some = find_tile<SMALL>(a.tiles, blockIdx.x, &tile, tok);
  const int f = (blockIdx.y * kWarps + (threadIdx.x >> 5)) * FW;
  if (some && f < a.N && tile.adapter >= 0) {
    expand_tile<RT, ROWS, F32, SMALL>(a, tile, f, tok);
    return;
  }
  griddep_wait();   // every CTA: this kernel ends after the one before it
  if (some && f < a.N) copy_rows<F32, SMALL>(a, tile, f, FW, tok);
}

// ------------------------------------------------- dA = sum u x^T, dB
struct GradArgs {
  const __nv_bfloat16* left;   // col planes of u or w
  int64_t plane;
  const void* src;             // x or dout
  int64_t ld;
  const int32_t* perm;
  const int32_t* first;
  const int32_t* counts;
  float* out;                  // dA [NA, r, N], or (transposed) dB [NA, N, r]
  int32_t r, N;
  int32_t transposed;
};

// Features a lane loads: 8 while the accumulators (16 RT x 8 FL floats a warp)
// leave room for two CTAs an SM.
template <int RT, bool F32>
constexpr int grad_fl() { return RT == 1 || (RT == 2 && !F32) ? 8 : 4; }
template <int RT, bool F32>
constexpr size_t grad_smem() {
  return sizeof(float) * kWarps * 16 * RT * (8 * grad_fl<RT, F32>() + 1);
}

// Cluster of C CTAs per (range of 8 FL features, adapter): the adapter's
// tokens by 16, warp by warp over the cluster.  Ranks are MMA-M, features
// MMA-N, tokens contracted: lane (g, t) loads FL features of the token rows
// 4 t .. + 3, and ranks g and g + 8 of those tokens from the col planes.
template <int RT, bool F32>
__device__ __forceinline__ void grad_part(const GradArgs& a, int slab, int adapter, float* red) {
  constexpr int FL = grad_fl<RT, F32>();
  constexpr int FW = 8 * FL, RP = 16 * RT, RS = FW + 1;
  constexpr int XP = F32 ? 3 : 1;   // planes of the features
  constexpr size_t ES = F32 ? 4 : 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int C = static_cast<int>(cluster_size()), rank_c = static_cast<int>(cluster_rank());
  const int f = slab * FW;
  const int steps = (a.counts[adapter] + 15) / 16;
  const int64_t slot0 = static_cast<int64_t>(a.first[adapter]) * kTile;
  float acc[RT][FL][4];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < FL; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i][j][q] = 0.f;
  const bool in = f + FL * g < a.N;
  const uint8_t* src = static_cast<const uint8_t*>(a.src) + (f + FL * g) * ES;
  const int stride = C * kWarps;
  int s = rank_c * kWarps + warp;
  int4 id = make_int4(-1, -1, -1, -1);
  if (s < steps) id = *reinterpret_cast<const int4*>(a.perm + slot0 + 16 * s + 4 * t);
  for (; s < steps; s += stride) {
    uint32_t w[XP][4][FL / 2];
    const int ids[4] = {id.x, id.y, id.z, id.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
#pragma unroll
      for (int x = 0; x < XP; ++x)
#pragma unroll
        for (int c = 0; c < FL / 2; ++c) w[x][q][c] = 0;
      if (in && ids[q] >= 0) {
        const uint8_t* p = src + static_cast<int64_t>(ids[q]) * a.ld * ES;
        if constexpr (F32) {
#pragma unroll
          for (int c = 0; c < FL / 4; ++c) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(p) + c);
            float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int x = 0; x < 3; ++x) {
              w[x][q][2 * c] = peel(e[0], e[1]);
              w[x][q][2 * c + 1] = peel(e[2], e[3]);
            }
          }
        } else {
          load_words<FL / 2>(reinterpret_cast<const __nv_bfloat16*>(p), w[0][q]);
        }
      }
    }
    // [tile, RP, kTile]: 16 consecutive slots of a rank row
    const int64_t at = slot0 + 16 * s;
    const __nv_bfloat16* u = a.left + at / kTile * (RP * kTile) + at % kTile + g * kTile + 4 * t;
    if (s + stride < steps)
      id = *reinterpret_cast<const int4*>(a.perm + at + 16 * stride + 4 * t);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int plane = 0; plane < 3; ++plane) {
        const __nv_bfloat16* up = u + plane * a.plane + 16 * i * kTile;
        const uint2 u0 = *reinterpret_cast<const uint2*>(up);
        const uint2 u1 = *reinterpret_cast<const uint2*>(up + 8 * kTile);
#pragma unroll
        for (int x = 0; x < XP; ++x) {
          if (plane + x > 2) continue;   // below the float sums' own rounding
#pragma unroll
          for (int j = 0; j < FL / 2; ++j) {
            const uint32_t r0 = w[x][0][j], r1 = w[x][1][j], r2 = w[x][2][j], r3 = w[x][3][j];
            mma(acc[i][2 * j], u0.x, u1.x, u0.y, u1.y, pair<0>(r0, r1), pair<0>(r2, r3));
            mma(acc[i][2 * j + 1], u0.x, u1.x, u0.y, u1.y, pair<1>(r0, r1), pair<1>(r2, r3));
          }
        }
      }
  }
  // the warps' sums in warp order, then the cluster's in rank order
  float* mine = red + warp * RP * RS;
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < FL; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        mine[(16 * i + g + 8 * (q >> 1)) * RS + FL * (2 * t + (q & 1)) + j] = acc[i][j][q];
  __syncthreads();
  for (int i = threadIdx.x; i < RP * RS; i += kThreads) {
    float v = red[i];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) v += red[w * RP * RS + i];
    red[i] = v;
  }
  if (C > 1) cluster_sync();
  else __syncthreads();
  const int cols = min(FW, a.N - f), total = a.r * cols;
  float* out = a.out + static_cast<int64_t>(adapter) * a.r * a.N;
  for (int i = rank_c * kThreads + threadIdx.x; i < total; i += C * kThreads) {
    int j, n;
    if (a.transposed) n = i / a.r, j = i - n * a.r;
    else j = i / cols, n = i - j * cols;
    float v = 0.f;
    if (C == 1) v = red[j * RS + n];
    else
      for (int c = 0; c < C; ++c) v += cluster_load(red + j * RS + n, c);
    if (a.transposed) out[static_cast<int64_t>(f + n) * a.r + j] = v;
    else out[static_cast<int64_t>(j) * a.N + f + n] = v;
  }
  if (C > 1) cluster_sync();
}

// The backward's outputs in one launch: dA's units (slab, adapter), then
// dB's, a cluster each, then dx's (tile, 8 groups of features), a CTA each.
struct OutArgs {
  GradArgs da, db;
  ExpandArgs dx;
  int32_t da_slabs, db_slabs, NA;   // slabs 0: not wanted
  int32_t dx_cols;
};

template <int RT, bool F32>
__global__ void __launch_bounds__(kThreads, RT == 8 ? 1 : 2) backward_out_kernel(const OutArgs a) {
  extern __shared__ __align__(16) uint8_t sm[];
  float* red = reinterpret_cast<float*>(sm);
  griddep_wait();
  griddep_launch_dependents();
  const int C = static_cast<int>(cluster_size());
  int unit = blockIdx.x / C;
  const int na = a.da_slabs * a.NA, nb = a.db_slabs * a.NA;
  if (unit < na) {
    grad_part<RT, false>(a.da, unit % a.da_slabs, unit / a.da_slabs, red);
  } else if (unit < na + nb) {
    unit -= na;
    grad_part<RT, F32>(a.db, unit % a.db_slabs, unit / a.db_slabs, red);
  } else {
    constexpr int FW = expand_width<RT>();
    const int cta = blockIdx.x - (na + nb) * C;
    const int ti = cta / a.dx_cols;
    const int f = ((cta - ti * a.dx_cols) * kWarps + (threadIdx.x >> 5)) * FW;
    Tile tile;
    if (!find_tile<false>(a.dx.tiles, ti, &tile, nullptr) || f >= a.dx.N) return;
    if (tile.adapter < 0) copy_rows<false, false>(a.dx, tile, f, FW, nullptr);
    else expand_tile<RT, true, false, false>(a.dx, tile, f, nullptr);
  }
}

// ------------------------------------------------------------- host side
int rt_of(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8; }

struct AdapterWs {
  size_t perm, counts, first, tiles, num_tiles, planes, total;
  int64_t units;    // tiles at most
  int64_t plane;    // elements of a plane
  bool small;
};

AdapterWs adapter_ws(const moe_adapter_shape* s, bool backward) {
  const int64_t T = s->num_tokens, NA = s->num_adapters;
  AdapterWs w = {};
  w.small = !backward && T <= kSmallTokens;
  w.units = w.small ? T : max_tiles(T, NA);
  w.plane = w.units * (w.small ? kSmallTile : kTile) * 16 * rt_of(s->rank);
  size_t off = 0;
  auto take = [&](int64_t bytes) {
    const size_t o = off;
    off += ws_up(static_cast<size_t>(bytes));
    return o;
  };
  if (!w.small) {
    w.perm = take(w.units * kTile * 4);
    w.counts = take((NA + 1) * 4);
    w.first = take((NA + 2) * 4);
    w.tiles = take(w.units * 16);
    w.num_tiles = take(4);
  }
  // two row planes; backward: three col planes of u and of w as well
  w.planes = take(w.plane * 2 * (backward ? 8 : 2));
  w.total = off > 0 ? off : kWsAlign;
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

// CTAs that share a tile: powers of two up to 8, while all clusters are
// resident at once (two CTAs an SM) and every warp has a chunk of 32 to
// contract.
int shrink_cluster(int64_t units, int K, int warps_k, int sms) {
  int c = 1;
  while (c < 8 && units * c <= sms && K >= 32 * 2 * c * warps_k) c *= 2;
  return c;
}

template <int RT, bool SMALL>
cudaError_t launch_shrink_x(const ShrinkArgs& a, int64_t units, int sms, cudaStream_t st) {
  using S = ShrinkX<RT, SMALL>;
  static DeviceOnce once;
  const cudaError_t e = set_smem_limit_once(shrink_x_kernel<RT, SMALL>, S::smem, once);
  if (e != cudaSuccess) return e;
  const int c = shrink_cluster(units, a.K, S::WK, sms);
  return launch_cluster(shrink_x_kernel<RT, SMALL>, dim3(static_cast<unsigned>(units * c)), c, S::smem,
                        st, a);
}

template <int RT, bool F32, bool SMALL>
cudaError_t launch_expand(const ExpandArgs& a, int64_t units, cudaStream_t st) {
  constexpr int unit = kWarps * expand_width<RT>();
  const dim3 grid(static_cast<unsigned>(units), static_cast<unsigned>((a.N + unit - 1) / unit));
  return launch_pdl(expand_kernel<RT, false, F32, SMALL>, grid, dim3(kThreads), 0, st, a);
}

template <int RT, bool SMALL>
cudaError_t launch_forward(const ShrinkArgs& sa, const ExpandArgs& ea, bool f32, int64_t units,
                           int sms, cudaStream_t st) {
  const cudaError_t e = launch_shrink_x<RT, SMALL>(sa, units, sms, st);
  if (e != cudaSuccess) return e;
  return f32 ? launch_expand<RT, true, SMALL>(ea, units, st)
             : launch_expand<RT, false, SMALL>(ea, units, st);
}

template <bool SMALL>
cudaError_t forward_products(const ShrinkArgs& sa, const ExpandArgs& ea, bool f32, int64_t units,
                             int sms, cudaStream_t st) {
  switch (rt_of(sa.r)) {
    case 1: return launch_forward<1, SMALL>(sa, ea, f32, units, sms, st);
    case 2: return launch_forward<2, SMALL>(sa, ea, f32, units, sms, st);
    case 4: return launch_forward<4, SMALL>(sa, ea, f32, units, sms, st);
    default: return launch_forward<8, SMALL>(sa, ea, f32, units, sms, st);
  }
}

struct Backward {
  ShrinkArgs d, x;
  bool want_x;
  OutArgs out;      // without the slabs and columns
  bool want_dx;
  int64_t units;
  int T, NA, sms;
};

template <int RT, bool F32>
cudaError_t launch_backward(const Backward& b, cudaStream_t st) {
  static DeviceOnce once_s, once_o;
  constexpr size_t xs = ShrinkX<RT, false>::smem, ds = ShrinkD<RT>::smem;
  constexpr size_t smem_s = xs > ds ? xs : ds;
  cudaError_t e = set_smem_limit_once(shrink_both_kernel<RT, F32>, smem_s, once_s);
  if (e != cudaSuccess) return e;
  const int64_t both = b.units * (b.want_x ? 2 : 1);
  // (the same split whichever outputs are wanted: their sums do not depend on it)
  int c = shrink_cluster(2 * b.units, b.x.K > b.d.K ? b.x.K : b.d.K, ShrinkX<RT, false>::WK, b.sms);
  e = launch_cluster(shrink_both_kernel<RT, F32>, dim3(static_cast<unsigned>(both * c)), c, smem_s, st,
                     b.d, b.x, static_cast<int>(b.units));
  if (e != cudaSuccess) return e;
  constexpr size_t gx = grad_smem<RT, false>(), gd = grad_smem<RT, F32>();
  constexpr size_t smem_o = gx > gd ? gx : gd;
  e = set_smem_limit_once(backward_out_kernel<RT, F32>, smem_o, once_o);
  if (e != cudaSuccess) return e;
  OutArgs o = b.out;
  const int fx = 8 * grad_fl<RT, false>(), fd = 8 * grad_fl<RT, F32>(), fe = kWarps * expand_width<RT>();
  o.NA = b.NA;
  o.da_slabs = b.want_x ? (o.da.N + fx - 1) / fx : 0;
  o.db_slabs = b.want_x ? (o.db.N + fd - 1) / fd : 0;
  o.dx_cols = (o.dx.N + fe - 1) / fe;
  const int64_t grads = static_cast<int64_t>(o.da_slabs + o.db_slabs) * b.NA;
  // CTAs that share an adapter's tokens: while the gradients' units leave SMs
  // idle and each CTA has a round of 16 tokens a warp
  c = 1;
  while (c < 8 && grads * c < 2 * b.sms && b.T >= 2 * c * 16 * kWarps) c *= 2;
  int64_t ctas = b.want_dx ? b.units * o.dx_cols : 0;
  ctas = grads * c + (ctas + c - 1) / c * c;
  if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  return launch_cluster(backward_out_kernel<RT, F32>, dim3(static_cast<unsigned>(ctas)), c, smem_o, st, o);
}

template <bool F32>
cudaError_t backward_products(const Backward& b, cudaStream_t st) {
  switch (rt_of(b.d.r)) {
    case 1: return launch_backward<1, F32>(b, st);
    case 2: return launch_backward<2, F32>(b, st);
    case 4: return launch_backward<4, F32>(b, st);
    default: return launch_backward<8, F32>(b, st);
  }
}

struct AdapterCall {
  AdapterWs w;
  Groups g;
  TileSource tiles;
  __nv_bfloat16* planes;
};

AdapterCall adapter_call(const moe_adapter_shape* s, bool backward, const int32_t* ids,
                         void* workspace) {
  AdapterCall c;
  uint8_t* base = static_cast<uint8_t*>(workspace);
  c.w = adapter_ws(s, backward);
  c.g.perm = reinterpret_cast<int32_t*>(base + c.w.perm);
  c.g.counts = reinterpret_cast<int32_t*>(base + c.w.counts);
  c.g.first = reinterpret_cast<int32_t*>(base + c.w.first);
  c.g.tiles = reinterpret_cast<int4*>(base + c.w.tiles);
  c.g.num_tiles = reinterpret_cast<int32_t*>(base + c.w.num_tiles);
  c.tiles.ids = ids;
  c.tiles.T = s->num_tokens;
  c.tiles.NA = s->num_adapters;
  c.tiles.perm = c.g.perm;
  c.tiles.tiles = c.g.tiles;
  c.tiles.num_tiles = c.g.num_tiles;
  c.planes = reinterpret_cast<__nv_bfloat16*>(base + c.w.planes);
  return c;
}

// row / col: the plane each set of planes begins at, -1 for none.
ShrinkArgs shrink_args(const AdapterCall& c, const void* src, int64_t ld, const void* pool,
                       const float* scale, int row, int col, int r, int K) {
  ShrinkArgs a;
  a.tiles = c.tiles;
  a.src = src;
  a.ld = ld;
  a.pool = static_cast<const __nv_bfloat16*>(pool);
  a.scale = scale;
  a.dst.row = row < 0 ? nullptr : c.planes + row * c.w.plane;
  a.dst.col = col < 0 ? nullptr : c.planes + col * c.w.plane;
  a.dst.size = c.w.plane;
  a.r = r;
  a.K = K;
  return a;
}

ExpandArgs expand_args(const AdapterCall& c, const void* pool, const void* base, int64_t ld_base,
                       void* out, int64_t ld_out, int r, int N) {
  ExpandArgs a;
  a.tiles = c.tiles;
  a.v.row = c.planes;
  a.v.col = nullptr;
  a.v.size = c.w.plane;
  a.pool = static_cast<const __nv_bfloat16*>(pool);
  a.base = base;
  a.ld_base = ld_base;
  a.out = out;
  a.ld_out = ld_out;
  a.r = r;
  a.N = N;
  return a;
}

GradArgs grad_args(const AdapterCall& c, int col, const void* src, int64_t ld, float* out, int r,
                   int N, bool transposed) {
  GradArgs a;
  a.left = c.planes + col * c.w.plane;
  a.plane = c.w.plane;
  a.src = src;
  a.ld = ld;
  a.perm = c.g.perm;
  a.first = c.g.first;
  a.counts = c.g.counts;
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
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const AdapterCall c = adapter_call(s, false, adapter_ids, workspace);
  const ShrinkArgs sa = shrink_args(c, x, ld_x, a, scale, 0, -1, s->rank, s->in_features);
  const ExpandArgs ea = expand_args(c, b, base, ld_base, out, ld_out, s->rank, s->out_features);
  const bool f32 = s->out_dtype == MOE_DTYPE_F32;
  if (c.w.small) return entry_launched(forward_products<true>(sa, ea, f32, c.w.units, sms, st));
  cudaError_t e = launch_group(adapter_ids, s->num_tokens, s->num_adapters, c.g, st);
  if (e == cudaSuccess) e = forward_products<false>(sa, ea, f32, c.w.units, sms, st);
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
  const int r = s->rank, H = s->in_features, N = s->out_features;
  const AdapterCall c = adapter_call(s, true, adapter_ids, workspace);
  constexpr int kURow = 0, kUCol = 2, kWCol = 5;   // first planes
  Backward w;
  w.d = shrink_args(c, dout, ld_dout, b, scale, dx ? kURow : -1, da ? kUCol : -1, r, N);
  w.x = shrink_args(c, x, ld_x, a, scale, -1, kWCol, r, H);
  w.want_x = da != nullptr;
  w.out.da = grad_args(c, kUCol, x, ld_x, da, r, H, false);
  w.out.db = grad_args(c, kWCol, dout, ld_dout, db, r, N, true);
  w.out.dx = expand_args(c, a, dx_base, ld_dx_base, dx, ld_dx, r, H);
  w.want_dx = dx != nullptr;
  w.units = c.w.units;
  w.T = s->num_tokens;
  w.NA = s->num_adapters;
  w.sms = sms;
  cudaError_t e = launch_group(adapter_ids, w.T, w.NA, c.g, st);
  if (e == cudaSuccess)
    e = s->out_dtype == MOE_DTYPE_F32 ? backward_products<true>(w, st) : backward_products<false>(w, st);
  return entry_launched(e);
}
