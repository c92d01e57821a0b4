// adapters.cu -- low-rank adapters of many requests beside a shared
// projection: out = base + scale_a B_a (A_a x), and its gradients.
//
// Tokens are grouped by adapter on the device into tiles of up to 64 tokens
// (group_kernel), then:
//   forward:   w = s A x                contracts over H      (shrink_x)
//              out = base + B w         contracts over r      (expand)
//   backward:  w = s A x, u = s B^T dout                      (shrink_x, shrink_d)
//              dx = dx_base + A^T u                           (expand)
//              dA = sum u x^T, dB = sum dout w^T              (grad: contracts over
//                                                              the adapter's tokens)
// A small batch's forward is one kernel (small_kernel), which finds tiles of up
// to 16 tokens by itself.
// With ranks of 8 to 128 every one of these does r multiply-adds for each
// element it moves, mostly far below the ~290 operations a byte at which tensor
// throughput would bind, so the layout serves the memory stream: the long
// operand is staged by asynchronous copies (small batches: loaded straight
// into fragments) and multiplied by mma.sync (16x8x16, bf16, float
// accumulators).  Only the gradients' sums at rank 64 and more are held up by
// it (the tensor pipe 0.4 busy): there tcgen05, which reads its operands from
// shared memory whoever staged them, would lift the limit.  It is not built.
// (Registers: the contractions at rank 128, both of them at rank 32 with a float
// dout, and small batches at rank 64 are held to 128 for two CTAs an SM and spill up
// to 72 bytes a thread; the others 16 at most.)
//
// A call's kernels overlap by programmatic dependent launch; its last one lets
// no successor start early (it would only wait, on SMs that this call fills).
//
// u and w are computed in float and leave as bf16 planes that add up to them:
// hi = bf16(v), then mid (and lo) the rounded rests.  Two planes (an error
// below 2^-17) feed the products that are rounded to bf16, three (2^-25) a
// float out and the float sums dA and dB.  A float dout is split in three as
// well.  Ranks are padded with zeros to RP = 16, 32, 64 or 128.
#include <cuda_bf16.h>

#include "cluster.cuh"
#include "entry.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kTile = 64;            // tokens of a tile
constexpr int kSmallTile = 16;       // and of a small batch's
constexpr int kSmallTokens = 1024;   // of a small batch at most
constexpr int kGroupThreads = 512;
constexpr int kGroupCtas = 8;
constexpr int kWarps = 8;            // warps of the product kernels
constexpr int kThreads = 32 * kWarps;

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(   // no side effect: free to be scheduled
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Long sums run in short pieces: an MMA truncates its sum to the accumulator's
// last place, always downwards in magnitude, and a chain of hundreds of them
// would drift by that bias (measured: 1e-6 of the result after 256 steps); the
// pieces are added with rounding.
__device__ __forceinline__ void add(float (&d)[4], const float (&s)[4]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) d[q] += s[q];
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

__device__ __forceinline__ uint4 ldg16(const void* p) { return __ldg(static_cast<const uint4*>(p)); }

// 16 bytes into shared memory, asynchronously; zeros where !some.
__device__ __forceinline__ void cp16(void* dst, const void* src, bool some) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(some ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {   // all but the last N groups have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four 8x8 matrices of bf16: lane l gives the address of row l % 8 of matrix
// l / 8.  (Volatile keeps them behind the barriers; nothing else writes what
// they read in between.)
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// Byte offset of 16-byte piece `c` of row `row` in a staged tile of ROW-byte
// rows: pieces are permuted so that the 8 rows one matrix of an ldmatrix reads
// lie in distinct banks.
template <int ROW>
__device__ __forceinline__ uint32_t piece(int row, int c) {
  constexpr int P = ROW / 16;
  const int x = P >= 8 ? row & 7 : P == 4 ? (row >> 1) & 3 : (row >> 2) & 1;
  return static_cast<uint32_t>(row * ROW + 16 * (c ^ x));
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
// token.  One cluster: each of its warps owns a contiguous run of the tokens
// and a histogram of it; the histograms' running sums, over the CTA's warps and
// then over the CTAs, give each warp its bases, and it hands out slots to its
// tokens in order.  Bound by the latency of its stages, and from some 10^4
// tokens by the shared-memory atomics and matches of its SMs, hence eight
// (a whole call at 64 x 64 features and rank 8, tokens of 200 adapters at
// random: 12.4 us at 8192 tokens and 31 at 65,536, against 19 and 90 with one
// CTA of 1024 threads).
__global__ void __launch_bounds__(kGroupThreads) group_kernel(const int32_t* __restrict__ ids,
                                                              int T, int NA, Groups g) {
  extern __shared__ __align__(128) uint8_t sm[];
  constexpr int kGroupWarps = kGroupThreads / 32;
  const int C = NA + 1;                 // columns: the adapters and "none"
  int32_t* hist = reinterpret_cast<int32_t*>(sm);   // [warps][C]
  int32_t* mine = hist + kGroupWarps * C;   // [C] this CTA's tokens
  int32_t* count = mine + C;            // [C] all tokens
  int32_t* start = count + C;           // [C] slots of the column before this CTA's
  int32_t* tfirst = start + C;          // [C + 1] first tile
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = static_cast<int>(cluster_rank());
  constexpr int threads = kGroupCtas * kGroupThreads;
  const int first = cta * kGroupThreads + static_cast<int>(threadIdx.x);   // in the cluster
  griddep_wait();
  griddep_launch_dependents();
  for (int i = threadIdx.x; i < kGroupWarps * C; i += kGroupThreads) hist[i] = 0;
  __syncthreads();
  const int per = (T + threads - 1) / threads * 32;   // tokens of a warp, whole rounds
  const int64_t t0 = static_cast<int64_t>(per) * (first / 32);
  const int t1 = static_cast<int>(min(t0 + per, static_cast<int64_t>(T)));
  for (int64_t t = t0 + lane; t < t1; t += 32) {
    const int id = ids[t];
    atomicAdd(&hist[warp * C + (static_cast<unsigned>(id) < static_cast<unsigned>(NA) ? id : NA)], 1);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < C; c += kGroupThreads) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kGroupWarps; ++w) {
      const int n = hist[w * C + c];
      hist[w * C + c] = sum;            // tokens of this column in earlier warps
      sum += n;
    }
    mine[c] = sum;
  }
  cluster_sync();
  for (int c = threadIdx.x; c < C; c += kGroupThreads) {
    int n[kGroupCtas], sum = 0, before = 0;
#pragma unroll
    for (int q = 0; q < kGroupCtas; ++q) n[q] = cluster_load(mine + c, q);
#pragma unroll
    for (int q = 0; q < kGroupCtas; ++q) {
      if (q < cta) before += n[q];
      sum += n[q];
    }
    count[c] = sum;
    start[c] = before;
    if (cta == 0) g.counts[c] = sum;
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
    if (lane == 0) {
      tfirst[C] = run;
      if (cta == 0) *g.num_tiles = run;
    }
  }
  __syncthreads();
  for (int c = first; c <= C; c += threads) g.first[c] = tfirst[c];
  const int tiles = tfirst[C];
  for (int i = first; i < tiles; i += threads) {
    int lo = 0, hi = C;                 // the last column whose first tile is at or before i
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tfirst[mid] <= i) lo = mid;
      else hi = mid;
    }
    g.tiles[i] = make_int4(lo < NA ? lo : -1, min(kTile, count[lo] - (i - tfirst[lo]) * kTile), 0, 0);
  }
  for (int i = first; i < C * kTile; i += threads) {   // the ends of the last tiles
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
      g.perm[static_cast<int64_t>(tfirst[c]) * kTile + start[c] + base + rank] = static_cast<int32_t>(t);
      if (rank == 0) hist[warp * C + c] = base + __popc(same);
    }
    __syncwarp();
  }
  cluster_sync();   // no CTA leaves while another reads its shared memory
}

// A tile as the product kernels see it: adapter (-1: none), tokens, first slot
// of its rows in the planes and in perm.
struct Tile {
  int adapter, n;
  int64_t slot;
};

// Where the tiles come from: the group kernel's lists, or (small batches) the ids.
struct TileSource {
  const int32_t* ids;
  int32_t T, NA;
  const int32_t* perm;
  const int4* tiles;
  const int32_t* num_tiles;
};

__device__ __forceinline__ bool find_tile(const TileSource& src, int i, Tile* tile) {
  const int n = *src.num_tiles;
  const int4 q = src.tiles[i];   // (allocated for every CTA's i; both loads in flight)
  if (i >= n) return false;
  tile->adapter = q.x;
  tile->n = q.y;
  tile->slot = static_cast<int64_t>(i) * kTile;
  return true;
}

// Small batches: the tiles of up to 16 tokens that share an adapter, found by
// every CTA for itself.  A tile begins with the tokens of rank 0, 16, 32, ...
// among their adapter's; their bits are set in `leaders`.
struct SmallTiles {
  int32_t ids[kSmallTokens];                // adapter (NA: none, -1: no such token)
  int32_t count[MOE_ADAPTER_MAX + 1];       // tokens seen of each adapter
  uint16_t rank[kSmallTokens];
  unsigned leaders[kSmallTokens / 32];
  int32_t tok[kSmallTile];                  // the tile in hand: its tokens, -1 past the end
  int32_t head[2];                          // its adapter and first rank

  // All threads; returns the number of tiles.
  __device__ __forceinline__ int find(const TileSource& src) {
    const int end = (src.T + 31) / 32 * 32;
    for (int t = threadIdx.x; t < end; t += kThreads) {
      int id = -1;
      if (t < src.T) {
        const int v = src.ids[t];
        id = static_cast<unsigned>(v) < static_cast<unsigned>(src.NA) ? v : src.NA;
      }
      ids[t] = id;
    }
    for (int c = threadIdx.x; c <= src.NA; c += kThreads) count[c] = 0;
    __syncthreads();
    if (threadIdx.x < 32) {   // in token order, 32 at a time
      const int lane = threadIdx.x;
      int id = ids[lane];
      for (int t = 0; t < end; t += 32) {
        const int next = t + 32 < end ? ids[t + 32 + lane] : -1;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, id);
        const int before = __popc(same & ((1u << lane) - 1));
        const int seen = id >= 0 ? count[id] : 0;
        __syncwarp();
        if (id >= 0 && before == 0) count[id] = seen + __popc(same);
        __syncwarp();
        rank[t + lane] = static_cast<uint16_t>(seen + before);
        const unsigned b = __ballot_sync(0xFFFFFFFFu, id >= 0 && (seen + before) % kSmallTile == 0);
        if (lane == 0) leaders[t / 32] = b;
        id = next;
      }
    }
    __syncthreads();
    int tiles = 0;
    for (int w = 0; w < end / 32; ++w) tiles += __popc(leaders[w]);
    return tiles;
  }

  // All threads: tile q, its tokens in tok.
  __device__ __forceinline__ Tile take(int q, const TileSource& src) {
    if (threadIdx.x < kSmallTile) tok[threadIdx.x] = -1;
    if (threadIdx.x == 0) {
      int w = 0, left = q;
      while (left >= __popc(leaders[w])) left -= __popc(leaders[w++]);
      const int t = 32 * w + static_cast<int>(__fns(leaders[w], 0, left + 1));
      head[0] = ids[t], head[1] = rank[t];
    }
    __syncthreads();
    const int adapter = head[0], first = head[1];
    for (int t = threadIdx.x; t < src.T; t += kThreads)
      if (ids[t] == adapter && rank[t] >= first && rank[t] < first + kSmallTile)
        tok[rank[t] - first] = t;
    __syncthreads();
    Tile tile;
    const int lane = threadIdx.x & 31;
    tile.n = __popc(__ballot_sync(0xFFFFFFFFu, lane < kSmallTile && tok[lane % kSmallTile] >= 0));
    tile.adapter = adapter < src.NA ? adapter : -1;
    tile.slot = 0;
    return tile;
  }
};

// ------------------------------------------- w = s A x, u = s B^T dout
// Low-rank rows leave as planes: `row` two or three planes [slots, RP], `col`
// three planes [tiles, RP, kTile] (each may be null); slots past a tile's
// tokens are zero.
struct Planes {
  __nv_bfloat16* row;
  int32_t rows;        // row planes
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

// The four floats at `p` of each CTA of the cluster, added in rank order; the
// loads of all of them in flight at once.
__device__ __forceinline__ float4 cluster_sum4(const float* p, int S) {
  if (S == 1) return *reinterpret_cast<const float4*>(p);
  float4 v[8];
#pragma unroll
  for (int c = 0; c < 8; ++c)
    if (c < S) v[c] = cluster_load4(p, c);
#pragma unroll
  for (int c = 1; c < 8; ++c)
    if (c < S) v[0].x += v[c].x, v[0].y += v[c].y, v[0].z += v[c].z, v[0].w += v[c].w;
  return v[0];
}

// Row stride (floats) of a CTA's partial tile of RP ranks.
constexpr int red_stride(int RP) { return RP + 4; }

// Each CTA of the cluster takes a share of the tile's tokens: it sums their
// WK partial rows [WK][NTOK][RP + 4] over warps and CTAs, in that order, and
// writes the planes; zeros from rank r on, where an infinite row of the source
// has left NaN (0 * inf).
template <int RP, int WK, int NTOK>
__device__ __forceinline__ void finish_tile(float* red, const Tile& tile, float scale, int r,
                                            const Planes& dst) {
  constexpr int RS = red_stride(RP);
  const int S = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  if (S > 1) cluster_sync();
  else __syncthreads();
  const int per = NTOK / S, t0 = rank * per;
  for (int i = threadIdx.x; i < per * RP / 4; i += kThreads) {
    float* p = red + (t0 + i / (RP / 4)) * RS + i % (RP / 4) * 4;
    float4 v = cluster_sum4(p, S);
#pragma unroll
    for (int w = 1; w < WK; ++w) {
      const float4 u = cluster_sum4(p + w * NTOK * RS, S);
      v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
    }
    // these rows of this CTA are read by no other
    *reinterpret_cast<float4*>(p) = i % (RP / 4) * 4 < r
        ? make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();
  if (dst.row)
    for (int i = threadIdx.x; i < per * RP / 2; i += kThreads) {   // two ranks of a token
      const int t = t0 + i / (RP / 2), j = 2 * (i % (RP / 2));
      float x = red[t * RS + j], y = red[t * RS + j + 1];
      __nv_bfloat16* o = dst.row + (tile.slot + t) * RP + j;
      *reinterpret_cast<uint32_t*>(o) = peel(x, y);
      *reinterpret_cast<uint32_t*>(o + dst.size) = peel(x, y);
      if (dst.rows > 2) *reinterpret_cast<uint32_t*>(o + 2 * dst.size) = peel(x, y);
    }
  if (dst.col)
    for (int i = threadIdx.x; i < per * RP / 2; i += kThreads) {   // two tokens of a rank
      const int j = i / (per / 2), t = t0 + 2 * (i % (per / 2));
      float x = red[t * RS + j], y = red[(t + 1) * RS + j];
      __nv_bfloat16* o = dst.col + tile.slot * RP + j * kTile + t;
      *reinterpret_cast<uint32_t*>(o) = peel(x, y);
      *reinterpret_cast<uint32_t*>(o + dst.size) = peel(x, y);
      *reinterpret_cast<uint32_t*>(o + 2 * dst.size) = peel(x, y);
    }
  if (S > 1) cluster_sync();   // no CTA leaves while another reads its shared memory
}

// Chunks of `chunk` elements of K that part `part` of `parts` contracts.
__device__ __forceinline__ int2 chunk_range(int K, int chunk, int part, int parts) {
  const int64_t n = (K + chunk - 1) / chunk;
  return make_int2(static_cast<int>(n * part / parts), static_cast<int>(n * (part + 1) / parts));
}

// Tiles of 64 tokens: the CTA's chunks of 128 elements of K (float: 64) come into shared
// memory by asynchronous copies, STAGES deep (gathered rows of src, and the
// pool's rows), and feed ldmatrix.  Bound by the copies' latency with two
// CTAs' stages an SM (8192 tokens of 7168, rank 16: 22 us cold, 95 MB at 4.2
// TB/s).  Tokens are MMA-M, 16 to a warp; the two
// warps that share 16 tokens split the ranks, or at RT = 1 the chunk.
//   !ROWS (x):    pool [r, K], its rows are the fragments' columns
//   ROWS (dout):  pool [K, r], read through the transposing ldmatrix
// A float src is staged as it is and split when it is read.
template <int RT, bool ROWS, bool F32>
struct Shrink {
  static constexpr int RP = 16 * RT, KC = F32 ? 64 : 128;
  static constexpr int WN = RT >= 2 ? 2 : 1, WK = 2 / WN;   // warps along ranks, along K
  static constexpr int NT = 2 * RT / WN;                    // 8-rank columns of a warp
  static constexpr int SROW = F32 ? 4 * KC + 32 : 2 * KC;   // bytes of a staged row of src
  static constexpr int PROW = ROWS ? 2 * RP : 2 * KC;       // and of the pool
  static constexpr int SRC = kTile * SROW, POOL = (ROWS ? KC : RP) * PROW;
  static constexpr int STAGE = SRC + POOL;
  // as many as leave room for a second CTA on the SM
  static constexpr int FIT = 110 * 1024 / STAGE;
  static constexpr int STAGES = FIT > 4 ? 4 : FIT < 2 ? 2 : FIT;
  static constexpr size_t red = sizeof(float) * WK * kTile * red_stride(RP);
  static constexpr size_t smem = STAGES * STAGE > red ? STAGES * STAGE : red;
};

template <int RT, bool ROWS, bool F32>
__device__ __forceinline__ void shrink_tile(const ShrinkArgs& a, const Tile& tile, uint8_t* sm) {
  using C = Shrink<RT, ROWS, F32>;
  constexpr int NT = C::NT, RS = red_stride(C::RP), KC = C::KC;
  constexpr int XP = F32 ? 3 : 1;                      // planes of src
  constexpr int ES = F32 ? 4 : 2;
  constexpr int PIECES = KC * ES / 16;                 // 16-byte pieces of a row of src
  constexpr int MINE = kTile * PIECES / kThreads;      // and a thread's
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int wm = warp & 3, wo = warp >> 2;             // 16 tokens; ranks or part of the chunk
  const int wn = C::WN == 2 ? wo : 0, wk = C::WK == 2 ? wo : 0;
  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[j][q] = 0.f;
  const uint8_t* row[MINE];                            // null: no such token
#pragma unroll
  for (int i = 0; i < MINE; ++i) {
    const int64_t id = a.tiles.perm[tile.slot + (threadIdx.x + i * kThreads) / PIECES];
    row[i] = id >= 0 ? static_cast<const uint8_t*>(a.src) + id * a.ld * ES : nullptr;
  }
  const int sc = threadIdx.x % PIECES;                 // the thread's piece of its rows
  const __nv_bfloat16* pool = a.pool + static_cast<int64_t>(tile.adapter) * a.r * a.K;
  const int2 c = chunk_range(a.K, KC, static_cast<int>(cluster_rank()), static_cast<int>(cluster_size()));
  auto fetch = [&](int chunk) {
    if (chunk < c.y) {
      uint8_t* s = sm + (chunk - c.x) % C::STAGES * C::STAGE;
      const int k = chunk * KC;
#pragma unroll
      for (int i = 0; i < MINE; ++i) {
        const int r = (threadIdx.x + i * kThreads) / PIECES, at = k + sc * (16 / ES);
        const bool some = row[i] && at < a.K;
        cp16(s + (F32 ? static_cast<uint32_t>(r * C::SROW + 16 * sc) : piece<2 * KC>(r, sc)),
             some ? row[i] + static_cast<int64_t>(at) * ES : static_cast<const uint8_t*>(a.src), some);
      }
      uint8_t* p = s + C::SRC;
      constexpr int PP = C::PROW / 16, ALL = C::POOL / 16;
#pragma unroll
      for (int i = 0; i < (ALL + kThreads - 1) / kThreads; ++i) {
        const int x = threadIdx.x + i * kThreads;
        if (ALL % kThreads && x >= ALL) break;
        const int r = x / PP, q = x % PP;              // row and piece
        const int rank = ROWS ? 8 * q : r, kk = ROWS ? k + r : k + 8 * q;
        const bool some = rank < a.r && kk < a.K;
        cp16(p + piece<C::PROW>(r, q),
             some ? pool + (ROWS ? static_cast<int64_t>(kk) * a.r + rank
                                 : static_cast<int64_t>(rank) * a.K + kk)
                  : a.pool, some);
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < C::STAGES - 1; ++i) fetch(c.x + i);
  for (int chunk = c.x; chunk < c.y; ++chunk) {
    cp_wait<C::STAGES - 2>();
    __syncthreads();
    fetch(chunk + C::STAGES - 1);   // into the stage that every warp has left
    const uint8_t* s = sm + (chunk - c.x) % C::STAGES * C::STAGE;
    const uint32_t sp = smem_u32(s), pp = sp + C::SRC;
    float part[NT][4];   // of this chunk (see `add`)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) part[j][q] = 0.f;
#pragma unroll
    for (int kk = 0; kk < KC / 16 / C::WK; ++kk) {
      const int k16 = wk * (KC / 16 / C::WK) + kk;
      uint32_t x[XP][4];
      if constexpr (F32) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {   // rows g, g + 8; columns 2 t, 2 t + 8
          float2 v = *reinterpret_cast<const float2*>(
              s + (16 * wm + g + 8 * (q & 1)) * C::SROW + 4 * (16 * k16 + 8 * (q >> 1) + 2 * t));
#pragma unroll
          for (int p = 0; p < XP; ++p) x[p][q] = peel(v.x, v.y);
        }
      } else {
        ldm4(x[0], sp + piece<2 * KC>(16 * wm + (lane & 15), 2 * k16 + (lane >> 4)));
      }
#pragma unroll
      for (int j = 0; j < NT; j += 2) {   // two columns of 8 ranks
        const int n = wn * NT + j;
        uint32_t b[4];
        if constexpr (ROWS)
          ldm4t(b, pp + piece<C::PROW>(16 * k16 + (lane & 15), n + (lane >> 4)));
        else
          ldm4(b, pp + piece<C::PROW>(8 * n + (lane & 7) + 8 * (lane >> 4), 2 * k16 + ((lane >> 3) & 1)));
#pragma unroll
        for (int p = 0; p < XP; ++p) {
          mma(part[j], x[p][0], x[p][1], x[p][2], x[p][3], b[0], b[1]);
          mma(part[j + 1], x[p][0], x[p][1], x[p][2], x[p][3], b[2], b[3]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) add(acc[j], part[j]);
  }
  cp_wait<0>();
  __syncthreads();   // the stages become the partial tiles
  float* red = reinterpret_cast<float*>(sm);
  float* mine = red + wk * kTile * RS;
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      mine[(16 * wm + g + 8 * (q >> 1)) * RS + 8 * (wn * NT + j) + 2 * t + (q & 1)] = acc[j][q];
  const float scale = a.scale ? __ldg(a.scale + tile.adapter) : 1.0f;
  finish_tile<C::RP, C::WK, kTile>(red, tile, scale, a.r, a.dst);
}

// Cluster of S CTAs per tile, sharing out the chunks of K.
template <int RT>
__global__ void __launch_bounds__(kThreads, 2) shrink_x_kernel(const ShrinkArgs a) {
  extern __shared__ __align__(128) uint8_t sm[];
  griddep_wait();
  griddep_launch_dependents();
  Tile tile;
  if (!find_tile(a.tiles, blockIdx.x / cluster_size(), &tile) || tile.adapter < 0) return;
  shrink_tile<RT, false, false>(a, tile, sm);
}

// Both of the backward's, in one launch: the first `d_units` clusters take
// dout, the others x.
template <int RT, bool F32>
__global__ void __launch_bounds__(kThreads, 2) shrink_both_kernel(const ShrinkArgs d, const ShrinkArgs x,
                                                               int d_units) {
  extern __shared__ __align__(128) uint8_t sm[];
  griddep_wait();
  griddep_launch_dependents();
  int unit = blockIdx.x / cluster_size();
  Tile tile;
  if (unit < d_units) {
    if (!find_tile(d.tiles, unit, &tile) || tile.adapter < 0) return;
    shrink_tile<RT, true, F32>(d, tile, sm);
  } else {
    unit -= d_units;
    if (!find_tile(x.tiles, unit, &tile) || tile.adapter < 0) return;
    shrink_tile<RT, false, false>(x, tile, sm);
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
  int32_t units;         // tiles at most
  int32_t cols, parts;   // blocks of features, CTAs they are split among
};

// A CTA takes a tile and a range of features, FB at a time: the tile's rows of
// the base and the pool's rows come into shared memory by asynchronous copies,
// STAGES deep; tokens are MMA-M (16 a warp, w's planes in registers
// throughout), features MMA-N; the sums go back into the staged base, rounded
// once, and leave as whole rows.  Bound by HBM in both directions, with 0.68 of
// the issue slots taken (8192 tokens, rank 16, 7168 features: 47 us cold, the
// base and out at 5.0 TB/s).
//   !ROWS: pool [N, r], its rows are the fragments' columns
//   ROWS:  pool [r, N], read through the transposing ldmatrix
template <int RT, bool ROWS, bool F32, bool SMALL>
struct Expand {
  static constexpr int RP = 16 * RT;
  // features of a block: more where a block has few tokens, for fewer barriers
  static constexpr int FB = SMALL && RT <= 2 ? 256 : 128;
  // CTAs that share a tile's tokens: two where the base outweighs the pool's
  // rows, which each of them stages (8192 tokens, rank 16, 7168 features:
  // 73.3 us for the forward against 75.7)
  static constexpr int SUB = SMALL || ROWS || RT > 2 ? 1 : 2;
  static constexpr int NTOK = SMALL ? kSmallTile : kTile / SUB;
  static constexpr int WT = NTOK / 16, WF = kWarps / WT;      // warps along tokens, features
  static constexpr int NT = FB / 8 / WF;                      // 8-feature columns of a warp
  static constexpr int ES = F32 ? 4 : 2;
  static constexpr int BROW = FB * ES + (F32 ? 32 : 16);      // bytes of a staged row of the base
  static constexpr int PROW = ROWS ? 2 * FB : 2 * RP;         // and of the pool
  static constexpr int BASE = NTOK * BROW, POOL = (ROWS ? RP : FB) * PROW, V = NTOK * 2 * RP;
  static constexpr int VN = F32 ? 3 : 2;                      // planes of w
  static constexpr int STAGE = BASE + POOL;
  static constexpr int FIT = 40 * 1024 / STAGE;   // stages that leave room for other CTAs
  static constexpr int STAGES = SMALL && FIT > 2 ? (FIT < 4 ? FIT : 4) : 2;
  static constexpr size_t smem = STAGES * STAGE + VN * V;
};

// Share `sub` of a tile's tokens; false: it has none.
template <typename C>
__device__ __forceinline__ bool take_share(int sub, Tile* tile) {
  tile->slot += sub * C::NTOK;
  tile->n = min(tile->n - sub * C::NTOK, C::NTOK);
  return tile->n > 0;
}

// Tokens without an adapter: out = base, bit for bit (nothing to do when they
// are the same memory).  token(i): the tile's i-th.
template <bool F32, typename Token>
__device__ __forceinline__ void copy_rows(const ExpandArgs& a, const Tile& tile, int f, int width,
                                          Token&& token) {
  constexpr int ES = F32 ? 4 : 2;
  if (a.base == a.out && a.ld_base == a.ld_out) return;
  const int per = width * ES / 16;
  for (int i = threadIdx.x; i < tile.n * per; i += kThreads) {
    const int row = i / per, n = f + i % per * (16 / ES);
    if (n >= a.N) continue;
    const int64_t id = token(row);
    uint4 q = make_uint4(0, 0, 0, 0);
    if (a.base)
      q = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.base) + (id * a.ld_base + n) * ES);
    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + (id * a.ld_out + n) * ES) = q;
  }
}

// A thread's part in a CTA's blocks of FB features up to c1: its pieces of the
// tile's rows (whose tokens are `row`, -1: none) and of the pool.
template <int RT, bool ROWS, bool F32, bool SMALL>
struct Blocks {
  using C = Expand<RT, ROWS, F32, SMALL>;
  static constexpr int ES = C::ES, NT = C::NT, FB = C::FB;
  static constexpr int PIECES = FB * ES / 16, MINE = (C::NTOK * PIECES + kThreads - 1) / kThreads;
  const ExpandArgs& a;
  const __nv_bfloat16* pool;
  uint8_t* sm;
  int c1;
  int bc;          // first feature of the thread's piece
  int row[MINE];

  template <typename Token>
  __device__ __forceinline__ Blocks(const ExpandArgs& args, int adapter, int end, uint8_t* smem, Token&& token)
      : a(args), pool(args.pool + static_cast<int64_t>(adapter) * args.r * args.N), sm(smem), c1(end),
        bc(threadIdx.x % PIECES * (16 / ES)) {
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      const int r = (threadIdx.x + i * kThreads) / PIECES;
      row[i] = r < C::NTOK ? token(r) : -1;
    }
  }

  // The copies of block c, as one group.
  __device__ __forceinline__ void fetch(int c, int stage) const {
    if (c < c1) {
      uint8_t* s = sm + stage * C::STAGE;
      const int f = c * FB;
      if (a.base) {
        const bool in = f + bc < a.N;
#pragma unroll
        for (int i = 0; i < MINE; ++i)
          if (row[i] >= 0)
            cp16(s + (threadIdx.x + i * kThreads) / PIECES * C::BROW + bc * ES,
                 static_cast<const uint8_t*>(a.base) + (in ? row[i] * a.ld_base + f + bc : 0) * ES, in);
      }
      constexpr int PP = C::PROW / 16, ALL = C::POOL / 16;
#pragma unroll
      for (int i = 0; i < (ALL + kThreads - 1) / kThreads; ++i) {
        const int x = threadIdx.x + i * kThreads;
        if (ALL % kThreads && x >= ALL) break;
        const int r = x / PP, q = x % PP;
        const int rank = ROWS ? r : 8 * q, n = ROWS ? f + 8 * q : f + r;
        const bool some = rank < a.r && n < a.N;
        cp16(s + C::BASE + piece<C::PROW>(r, q),
             some ? pool + (ROWS ? static_cast<int64_t>(rank) * a.N + n : static_cast<int64_t>(n) * a.r + rank)
                  : a.pool, some);
      }
    }
    cp_commit();
  }

  // Blocks c0 .. c1 - 1 for a tile of n tokens; blocks c0 .. c0 + STAGES - 2 are
  // fetched already, and w's planes lie in v_s.
  __device__ __forceinline__ void run(int c0, int n, const uint8_t* v_s) const {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int wt = warp % C::WT, wf = warp / C::WT;
    const uint32_t vp = smem_u32(v_s);
    uint32_t v[RT][C::VN][4];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int p = 0; p < C::VN; ++p)
        ldm4(v[i][p], vp + p * C::V + piece<2 * C::RP>(16 * wt + (lane & 15), 2 * i + (lane >> 4)));
    int stage = 0;
    for (int c = c0; c < c1; ++c) {
      fetch(c + C::STAGES - 1, stage == 0 ? C::STAGES - 1 : stage - 1);
      cp_wait<C::STAGES - 1>();
      __syncthreads();
      uint8_t* s = sm + stage * C::STAGE;
      const uint32_t pp = smem_u32(s) + C::BASE;
      stage = stage + 1 == C::STAGES ? 0 : stage + 1;
      if (16 * wt < n) {
#pragma unroll(RT == 1 ? 4 : 1)
        for (int j = 0; j < NT; j += 2) {
          const int col = wf * NT + j;   // two columns of 8 features
          float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            uint32_t b[4];
            if constexpr (ROWS)
              ldm4t(b, pp + piece<C::PROW>(16 * i + (lane & 15), col + (lane >> 4)));
            else
              ldm4(b, pp + piece<C::PROW>(8 * col + (lane & 7) + 8 * (lane >> 4), 2 * i + ((lane >> 3) & 1)));
#pragma unroll
            for (int p = 0; p < C::VN; ++p) {
              mma(acc[0], v[i][p][0], v[i][p][1], v[i][p][2], v[i][p][3], b[0], b[1]);
              mma(acc[1], v[i][p][0], v[i][p][1], v[i][p][2], v[i][p][3], b[2], b[3]);
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint8_t* o = s + (16 * wt + 8 * h + g) * C::BROW + (8 * (col + e) + 2 * t) * ES;
              const float x = acc[e][2 * h], y = acc[e][2 * h + 1];
              if constexpr (F32) {
                const float2 q = a.base ? *reinterpret_cast<const float2*>(o) : make_float2(0.f, 0.f);
                *reinterpret_cast<float2*>(o) = make_float2(q.x + x, q.y + y);
              } else {
                const uint32_t q = a.base ? *reinterpret_cast<const uint32_t*>(o) : 0u;
                *reinterpret_cast<uint32_t*>(o) =
                    word(__float2bfloat16_rn(__uint_as_float(q << 16) + x),
                         __float2bfloat16_rn(__uint_as_float(q & 0xFFFF0000u) + y));
              }
            }
        }
      }
      __syncthreads();
      if (c * FB + bc < a.N) {
#pragma unroll
        for (int i = 0; i < MINE; ++i)
          if (row[i] >= 0)
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + (row[i] * a.ld_out + c * FB + bc) * ES) =
                *reinterpret_cast<const uint4*>(s + (threadIdx.x + i * kThreads) / PIECES * C::BROW + bc * ES);
      }
      __syncthreads();   // before the stage is filled again
    }
    cp_wait<0>();
  }
};

// Blocks [c0, c1) of a tile.  The inputs' first loads (base, pool, and the
// tile's lists, which were complete before the kernel before this one began)
// are issued ahead of the grid wait.
template <int RT, bool ROWS, bool F32>
__device__ __forceinline__ void expand_tile(const ExpandArgs& a, const Tile& tile, int c0, int c1,
                                            uint8_t* sm) {
  using C = Expand<RT, ROWS, F32, false>;
  constexpr int RP = C::RP;
  uint8_t* v_s = sm + C::STAGES * C::STAGE;
  const Blocks<RT, ROWS, F32, false> blocks(a, tile.adapter, c1, sm,
                                            [&](int i) { return a.tiles.perm[tile.slot + i]; });
#pragma unroll
  for (int i = 0; i < C::STAGES - 1; ++i) blocks.fetch(c0 + i, i);
  griddep_wait();   // (again in backward_out_kernel: returns at once)
  constexpr int VP = RP / 8, ALLV = C::VN * C::NTOK * VP;   // pieces of a row of a plane, of all planes
#pragma unroll
  for (int i = 0; i < (ALLV + kThreads - 1) / kThreads; ++i) {
    const int x = threadIdx.x + i * kThreads;
    if (ALLV % kThreads && x >= ALLV) break;
    const int p = x / (C::NTOK * VP), r = x / VP % C::NTOK, q = x % VP;
    cp16(v_s + p * C::V + piece<2 * RP>(r, q), a.v.row + p * a.v.size + (tile.slot + r) * RP + 8 * q, true);
  }
  cp_commit();
  cp_wait<0>();
  __syncthreads();
  blocks.run(c0, tile.n, v_s);
}

template <int RT, bool F32>
__global__ void __launch_bounds__(kThreads) expand_kernel(const ExpandArgs a) {
  using C = Expand<RT, false, F32, false>;
  extern __shared__ __align__(128) uint8_t sm[];
  Tile tile;
  const int part = blockIdx.x / (a.units * C::SUB), unit = blockIdx.x - part * a.units * C::SUB;
  const int c0 = a.cols * part / a.parts, c1 = a.cols * (part + 1) / a.parts;
  const bool some = find_tile(a.tiles, unit / C::SUB, &tile) && take_share<C>(unit % C::SUB, &tile);
  if (some && tile.adapter >= 0) {
    expand_tile<RT, false, F32>(a, tile, c0, c1, sm);
    return;
  }
  griddep_wait();   // every CTA: this kernel ends after the one before it
  if (some)
    copy_rows<F32>(a, tile, c0 * C::FB, (c1 - c0) * C::FB,
                   [&](int i) { return a.tiles.perm[tile.slot + i]; });
}

// ------------------------------------------------------- small batches
// The whole forward of a small batch in one kernel: a
// cluster takes a tile (16 tokens that share an adapter).  Its warps
// share out the 32-element chunks of H (ranks are MMA-M, tokens MMA-N; lane (g, t)
// of a chunk loads the 8 elements at 8 t of rank rows g and g + 8 and of token g
// straight from global memory, a few chunks a warp and all in flight at
// once), every CTA adds up the partial sums over distributed shared memory,
// and the CTAs share out the output's blocks, whose first base and pool rows
// have been on their way since the tile's start.  Bound by latency at one token
// (two dependent trips to HBM and the cluster's barriers), by the touched
// pools' bytes at many (7168 x 7168, rank 16: 7.2 us for one token; 64 tokens of
// 48 adapters of rank 32, 7168 x 4096: 11.8 us, 3.1 TB/s).
template <int RT, bool F32>
struct Small {
  using E = Expand<RT, false, F32, true>;
  static constexpr int NT = kSmallTile / 8, RP = 16 * RT, RS = red_stride(RP);
  static constexpr size_t red = sizeof(float) * kWarps * kSmallTile * RS;
  static constexpr size_t smem = E::smem + red;
};

template <int RT, bool F32>
__global__ void __launch_bounds__(kThreads, RT == 8 ? 1 : 2)
    small_kernel(const ShrinkArgs a, const ExpandArgs e) {
  using S = Small<RT, F32>;
  using C = typename S::E;
  constexpr int NT = S::NT, RS = S::RS, RP = S::RP;
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ SmallTiles tiles;
  uint8_t* v_s = sm + C::STAGES * C::STAGE;
  float* red = reinterpret_cast<float*>(sm + C::smem);
  griddep_wait();
  const int CS = static_cast<int>(cluster_size()), rank_c = static_cast<int>(cluster_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int c0 = e.cols * rank_c / CS, c1 = e.cols * (rank_c + 1) / CS;
  const int q = blockIdx.x / CS;
  if (q >= tiles.find(a.tiles)) return;   // the whole cluster
  const Tile tile = tiles.take(q, a.tiles);
  if (tile.adapter < 0) {
    copy_rows<F32>(e, tile, c0 * C::FB, (c1 - c0) * C::FB, [&](int i) { return tiles.tok[i]; });
    return;
  }
  const Blocks<RT, false, F32, true> blocks(e, tile.adapter, c1, sm, [&](int i) { return tiles.tok[i]; });
#pragma unroll
  for (int i = 0; i < C::STAGES - 1; ++i) blocks.fetch(c0 + i, i);
  float acc[RT][NT][4];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i][j][q] = 0.f;
  const __nv_bfloat16* row[NT];          // null: no such token
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t id = tiles.tok[8 * j + g];
    row[j] = id >= 0 ? static_cast<const __nv_bfloat16*>(a.src) + id * a.ld + 8 * t : nullptr;
  }
  const int live = (tile.n + 7) / 8;     // columns with a token
  const __nv_bfloat16* pool = a.pool + static_cast<int64_t>(tile.adapter) * a.r * a.K + 8 * t;
  const int2 c = chunk_range(a.K, 32, rank_c * kWarps + warp, CS * kWarps);
  constexpr int U = RT == 1 ? 4 : RT == 2 ? 3 : RT == 4 ? 2 : 1;   // chunks in flight
#pragma unroll 1
  for (int k0 = 32 * c.x; k0 < 32 * c.y; k0 += 32 * U) {
    uint4 p[U][RT][2], x[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + 32 * u;
      const bool in = k < 32 * c.y && k + 8 * t < a.K;
#pragma unroll
      for (int j = 0; j < NT; ++j)
        x[u][j] = in && row[j] ? *reinterpret_cast<const uint4*>(row[j] + k)   // (may be out's)
                               : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int rank = 16 * i + 8 * h + g;
          p[u][i][h] = in && rank < a.r ? ldg16(pool + static_cast<int64_t>(rank) * a.K + k)
                                        : make_uint4(0, 0, 0, 0);
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
      if (j < live)
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          float part[4] = {0.f, 0.f, 0.f, 0.f};   // of these chunks (see `add`)
#pragma unroll
          for (int u = 0; u < U; ++u) {
            mma(part, p[u][i][0].x, p[u][i][1].x, p[u][i][0].y, p[u][i][1].y, x[u][j].x, x[u][j].y);
            mma(part, p[u][i][0].z, p[u][i][1].z, p[u][i][0].w, p[u][i][1].w, x[u][j].z, x[u][j].w);
          }
          add(acc[i][j], part);
        }
  }
  float* mine = red + warp * kSmallTile * RS;
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        mine[(8 * j + 2 * t + (q & 1)) * RS + 16 * i + g + 8 * (q >> 1)] = acc[i][j][q];
  __syncthreads();
  // the CTA's own warps first: one round over the cluster
  for (int i = threadIdx.x; i < kSmallTile * RS / 4; i += kThreads) {
    float4 v[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v[w] = reinterpret_cast<const float4*>(red + w * kSmallTile * RS)[i];
#pragma unroll
    for (int w = 1; w < kWarps; ++w)
      v[0].x += v[w].x, v[0].y += v[w].y, v[0].z += v[w].z, v[0].w += v[w].w;
    reinterpret_cast<float4*>(red)[i] = v[0];
  }
  if (CS > 1) cluster_sync();
  else __syncthreads();
  const float scale = a.scale ? __ldg(a.scale + tile.adapter) : 1.0f;
  for (int i = threadIdx.x; i < kSmallTile * RP / 4; i += kThreads) {   // four ranks of a token
    const int r = i / (RP / 4), j = i % (RP / 4) * 4;
    float4 v = cluster_sum4(red + r * RS + j, CS);
    v.x *= scale, v.y *= scale, v.z *= scale, v.w *= scale;
    if (j >= a.r) v = make_float4(0.f, 0.f, 0.f, 0.f);   // (as in finish_tile)
    uint8_t* o = v_s + piece<2 * RP>(r, j / 8) + 2 * (j % 8);
#pragma unroll
    for (int p = 0; p < C::VN; ++p) {
      const uint32_t lo = peel(v.x, v.y), hi = peel(v.z, v.w);
      *reinterpret_cast<uint2*>(o + p * C::V) = make_uint2(lo, hi);
    }
  }
  __syncthreads();
  blocks.run(c0, tile.n, v_s);
  if (CS > 1) cluster_sync();   // no CTA leaves while another reads its shared memory
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

// A CTA's tile of the gradient: RP ranks x 128 features; warps 16 ranks x 128 / (8 / RT)
// features each.  The adapter's tokens come TK slots at a time: the
// col planes of u and the gathered rows of x, by asynchronous copies, STAGES
// deep.  Bound by the latency of mma.sync and ldmatrix at two to four CTAs an SM:
// 5003 tokens of 2048 x 2048, rank 64, 6 adapters take 45 us with dx, the tensor
// pipe 0.40 busy.  Three planes instead of two cost a tenth of that and keep dA
// and dB at the error of a float product (3e-7 of them against 2.5e-6).
template <int RT, bool F32>
struct Grad {
  static constexpr int RP = 16 * RT, FB = 128;
  static constexpr int TK = RT <= 4 && !F32 ? kTile : kTile / 2;  // slots of a stage
  static constexpr int WF = kWarps / RT;                 // warps along the features
  static constexpr int NT = FB / 8 / WF;                 // 8-feature columns of a warp
  static constexpr int XROW = F32 ? 4 * FB + 16 : 2 * FB;
  static constexpr int X = TK * XROW, U = RP * 2 * TK;   // U: one plane
  static constexpr int STAGE = X + 3 * U;
  static constexpr int STAGES = 3 * STAGE <= 40 * 1024 ? 3 : 2;
  static constexpr size_t red = sizeof(float) * RP * (FB + 4);
  static constexpr size_t smem = STAGES * STAGE > red ? STAGES * STAGE : red;
};

// Cluster of C CTAs per (128 features, adapter), sharing out the adapter's
// stages.  Ranks are MMA-M, features MMA-N, tokens contracted.
template <int RT, bool F32>
__device__ __forceinline__ void grad_part(const GradArgs& a, int slab, int adapter, uint8_t* sm) {
  using G = Grad<RT, F32>;
  constexpr int NT = G::NT, RP = G::RP, FB = G::FB, RS = FB + 4, TK = G::TK;
  constexpr int XP = F32 ? 3 : 1;                       // planes of the features
  constexpr int ES = F32 ? 4 : 2;
  constexpr int PIECES = FB * ES / 16, MINE = TK * PIECES / kThreads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int wf = warp % G::WF, wr = warp / G::WF;
  const int C = static_cast<int>(cluster_size()), rank_c = static_cast<int>(cluster_rank());
  const int f = slab * FB;
  const int steps = (a.counts[adapter] + TK - 1) / TK;   // stages of TK slots
  const int64_t slot0 = static_cast<int64_t>(a.first[adapter]) * kTile;
  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[j][q] = 0.f;
  const int xc = threadIdx.x % PIECES;                  // the thread's piece of its rows
  const bool in = f + xc * (16 / ES) < a.N;
  const uint8_t* src = static_cast<const uint8_t*>(a.src) + (f + xc * (16 / ES)) * static_cast<int64_t>(ES);
  int ids[MINE];                                        // rows of the stage to fetch next
  auto tokens = [&](int i) {
#pragma unroll
    for (int m = 0; m < MINE; ++m)
      ids[m] = i < steps ? a.perm[slot0 + i * TK + (threadIdx.x + m * kThreads) / PIECES] : -1;
  };
  auto fetch = [&](int i, int stage) {
    if (i < steps) {
      uint8_t* s = sm + stage * G::STAGE;
#pragma unroll
      for (int m = 0; m < MINE; ++m) {
        const int r = (threadIdx.x + m * kThreads) / PIECES;
        const bool some = in && ids[m] >= 0;
        cp16(s + (F32 ? static_cast<uint32_t>(r * G::XROW + 16 * xc) : piece<2 * FB>(r, xc)),
             some ? src + static_cast<int64_t>(ids[m]) * a.ld * ES : static_cast<const uint8_t*>(a.src), some);
      }
      const int64_t at = slot0 + i * TK;   // the planes are [tile, RP, kTile]
      const __nv_bfloat16* u = a.left + at / kTile * (RP * kTile) + at % kTile;
      constexpr int UP = TK / 8, ALL = 3 * RP * UP;
#pragma unroll
      for (int m = 0; m < (ALL + kThreads - 1) / kThreads; ++m) {
        const int x = threadIdx.x + m * kThreads;
        if (ALL % kThreads && x >= ALL) break;
        const int plane = x / (RP * UP), r = x / UP % RP, q = x % UP;
        cp16(s + G::X + plane * G::U + piece<2 * TK>(r, q), u + plane * a.plane + r * kTile + 8 * q, true);
      }
    }
    cp_commit();
  };
  int next = rank_c;                                    // the stage whose rows ids names
  tokens(next);
#pragma unroll
  for (int i = 0; i < G::STAGES - 1; ++i) {
    fetch(next, i);
    next += C;
    tokens(next);
  }
  int stage = 0;
  for (int i = rank_c; i < steps; i += C) {
    cp_wait<G::STAGES - 2>();
    __syncthreads();
    fetch(next, stage == 0 ? G::STAGES - 1 : stage - 1);   // the stage that every warp has left
    next += C;
    tokens(next);
    const uint8_t* s = sm + stage * G::STAGE;
    const uint32_t xp = smem_u32(s), up = xp + G::X;
    stage = stage + 1 == G::STAGES ? 0 : stage + 1;
    uint32_t u[TK / 16][3][4];
#pragma unroll
    for (int k = 0; k < TK / 16; ++k)
#pragma unroll
      for (int p = 0; p < 3; ++p)
        ldm4(u[k][p], up + p * G::U + piece<2 * TK>(16 * wr + (lane & 15), 2 * k + (lane >> 4)));
#pragma unroll
    for (int j = 0; j < NT; j += 2) {
      const int n = wf * NT + j;                        // two columns of 8 features
      float part[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};   // of this stage (see `add`)
#pragma unroll
      for (int k = 0; k < TK / 16; ++k) {
        uint32_t b[XP][4];
        if constexpr (F32) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {                 // token pairs 2 t, 2 t + 8; columns n, n + 1
            const uint8_t* e = s + (16 * k + 2 * t + 8 * (q & 1)) * G::XROW + 4 * (8 * (n + (q >> 1)) + g);
            float x = *reinterpret_cast<const float*>(e), y = *reinterpret_cast<const float*>(e + G::XROW);
#pragma unroll
            for (int p = 0; p < XP; ++p) b[p][q] = peel(x, y);
          }
        } else {
          ldm4t(b[0], xp + piece<2 * FB>(16 * k + (lane & 15), n + (lane >> 4)));
        }
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (int x = 0; x < XP; ++x) {
            if (p + x > 2) continue;                    // below the float sums' own rounding
            mma(part[0], u[k][p][0], u[k][p][1], u[k][p][2], u[k][p][3], b[x][0], b[x][1]);
            mma(part[1], u[k][p][0], u[k][p][1], u[k][p][2], u[k][p][3], b[x][2], b[x][3]);
          }
      }
      add(acc[j], part[0]);
      add(acc[j + 1], part[1]);
    }
  }
  cp_wait<0>();
  __syncthreads();   // the stages become the CTA's tile
  float* red = reinterpret_cast<float*>(sm);
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      red[(16 * wr + g + 8 * (q >> 1)) * RS + 8 * (wf * NT + j) + 2 * t + (q & 1)] = acc[j][q];
  if (C > 1) cluster_sync();
  else __syncthreads();
  // each CTA of the cluster sums and writes a share of the tile
  float* out = a.out + static_cast<int64_t>(adapter) * a.r * a.N;
  if (!a.transposed) {   // of the ranks: rows of dA
    const int per = RP / C, j0 = rank_c * per;
    for (int i = threadIdx.x; i < per * FB / 4; i += kThreads) {
      const int j = j0 + i / (FB / 4), n = i % (FB / 4) * 4;
      if (j < a.r && f + n < a.N)
        *reinterpret_cast<float4*>(out + static_cast<int64_t>(j) * a.N + f + n) =
            cluster_sum4(red + j * RS + n, C);
    }
  } else {               // of the features: rows of dB
    const int per = FB / C, n0 = rank_c * per;
    if (C > 1) {
      for (int i = threadIdx.x; i < RP * per / 4; i += kThreads) {
        float* p = red + i / (per / 4) * RS + n0 + i % (per / 4) * 4;
        *reinterpret_cast<float4*>(p) = cluster_sum4(p, C);   // read by no other CTA
      }
      __syncthreads();
    }
    const int quads = a.r / 4;
    for (int i = threadIdx.x; i < per * quads; i += kThreads) {
      const int n = n0 + i / quads, j = i % quads * 4;
      if (f + n < a.N)
        *reinterpret_cast<float4*>(out + static_cast<int64_t>(f + n) * a.r + j) =
            make_float4(red[j * RS + n], red[(j + 1) * RS + n], red[(j + 2) * RS + n], red[(j + 3) * RS + n]);
    }
  }
  if (C > 1) cluster_sync();
}

// The backward's outputs in one launch: dA's units (slab, adapter), then
// dB's, a cluster each, then dx's (tile, 8 groups of features), a CTA each.
struct OutArgs {
  GradArgs da, db;
  ExpandArgs dx;
  int32_t da_slabs, db_slabs, NA;   // slabs 0: not wanted
};

template <int RT, bool F32>
__global__ void __launch_bounds__(kThreads, RT == 1 ? 4 : 2) backward_out_kernel(const OutArgs a) {
  extern __shared__ __align__(128) uint8_t sm[];
  griddep_wait();
  const int C = static_cast<int>(cluster_size());
  int unit = blockIdx.x / C;
  const int na = a.da_slabs * a.NA, nb = a.db_slabs * a.NA;
  if (unit < na) {
    grad_part<RT, false>(a.da, unit % a.da_slabs, unit / a.da_slabs, sm);
  } else if (unit < na + nb) {
    unit -= na;
    grad_part<RT, F32>(a.db, unit % a.db_slabs, unit / a.db_slabs, sm);
  } else {
    using E = Expand<RT, true, false, false>;
    const int cta = blockIdx.x - (na + nb) * C;
    const int part = cta / (a.dx.units * E::SUB), ti = cta - part * a.dx.units * E::SUB;
    const int c0 = a.dx.cols * part / a.dx.parts, c1 = a.dx.cols * (part + 1) / a.dx.parts;
    Tile tile;
    if (part >= a.dx.parts || !find_tile(a.dx.tiles, ti / E::SUB, &tile) ||
        !take_share<E>(ti % E::SUB, &tile))
      return;
    if (tile.adapter < 0)
      copy_rows<false>(a.dx, tile, c0 * E::FB, (c1 - c0) * E::FB,
                       [&](int i) { return a.dx.tiles.perm[tile.slot + i]; });
    else
      expand_tile<RT, true, false>(a.dx, tile, c0, c1, sm);
  }
}

// ------------------------------------------------------------- host side
int rt_of(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8; }

struct AdapterWs {
  size_t perm, counts, first, tiles, num_tiles, planes, total;
  int64_t units;    // tiles at most
  int64_t plane;    // elements of a plane
  bool small;       // forward of a small batch: no workspace
};

AdapterWs adapter_ws(const moe_adapter_shape* s, bool backward) {
  const int64_t T = s->num_tokens, NA = s->num_adapters;
  AdapterWs w = {};
  // One kernel up to where three catch up (7168 x 7168, rank 16, 8 adapters:
  // 8.3 us against 12.9 at 128 tokens, 9.9 / 13.8 at 256, 17.8 / 20.3 at 1021; 64
  // adapters: 24.2 / 28.6).  At rank 64 the two meet near 1024 tokens: with 8 adapters
  // 32.8 / 31.3 at 1021, with 64 46.5 / 56.0.  At rank 128 its tiles of 16 tokens read
  // the pools too often (2048 x 2048: 10.1 / 14.2 at 64 tokens, 20.2 / 14.6 at 256).
  // What it costs is the pools' rows times the tiles, so that the rule, which sees
  // neither the features nor the adapters, is a little off near its edge.
  w.small = !backward && T <= (s->rank <= 64 ? kSmallTokens : 64);
  // an adapter with n tokens has at most n / 16 + 1 tiles
  const int64_t small_units = T / kSmallTile + NA + 1;
  w.units = w.small ? (small_units < T ? small_units : T) : max_tiles(T, NA);
  w.total = kWsAlign;
  if (w.small) return w;   // unused
  w.plane = w.units * kTile * 16 * rt_of(s->rank);
  size_t off = 0;
  auto take = [&](int64_t bytes) {
    const size_t o = off;
    off += ws_up(static_cast<size_t>(bytes));
    return o;
  };
  w.perm = take(w.units * kTile * 4);
  w.counts = take((NA + 1) * 4);
  w.first = take((NA + 2) * 4);
  w.tiles = take(w.units * 16);
  w.num_tiles = take(4);
  // three row planes, or (backward) two of u and three col planes of u and of w
  w.planes = take(w.plane * 2 * (backward ? 8 : 3));
  w.total = off;
  return w;
}

int32_t check_adapter(const moe_adapter_shape* s) {
  if (!s) return entry_fail(MOE_ERR_INVALID_ARG, "shape is NULL");
  if (s->num_tokens < 0) return entry_fail(MOE_ERR_INVALID_ARG, "num_tokens < 0");
  if (s->num_tokens > (1 << 30))   // the lists' counts stay inside 32 bits
    return entry_fail(MOE_ERR_UNSUPPORTED, "num_tokens must be at most 2^30");
  if (s->num_adapters < 1 || s->num_adapters > MOE_ADAPTER_MAX)
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
                           cudaStream_t st, int threads, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
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
  auto smem = [](int na) { return (kGroupThreads / 32 + 4) * (na + 2) * sizeof(int32_t); };
  const cudaError_t e = set_smem_limit_once(group_kernel, smem(MOE_ADAPTER_MAX), once);
  if (e != cudaSuccess) return e;
  return launch_cluster(group_kernel, dim3(kGroupCtas), kGroupCtas, smem(NA), st, kGroupThreads,
                        ids, T, NA, g);
}

// CTAs that share a tile of `units` expected: powers of two up to 8, while all
// of them are resident, two an SM (a tenth more for the first split, the most
// worth), and every CTA keeps 256 elements of K.
// (Two with four stages each and one wave: 4096 tokens, rank 16, 7168 x 7168 in
// 45 us, 50 with three of three stages and more than a wave; rank 64: 64 and 76.
// Only tiles of few tokens want more CTAs: 3000 tokens of 200 adapters 63 and 59.)
int shrink_cluster(int64_t units, int K, int sms) {
  int c = 1;
  while (c < 8 && units * c <= sms + (c == 1 ? sms / 10 : 0) && K >= 2 * c * 256) c *= 2;
  return c;
}
// About as many tiles as T tokens of NA adapters make.
int64_t likely_tiles(int64_t T, int NA) {
  const int64_t filled = T / kTile + (NA + 1) / 2, one_each = T < NA ? T : NA;
  return filled > one_each ? filled : one_each;
}

// Splits the features of expand's tiles into WAVES times the CTAs that an SM
// holds by shared memory: ragged tiles even out over a few waves, more lose to
// each CTA's start (4 waves forward, 2 beside the backward's sums).
template <typename C, int WAVES>
void split_features(ExpandArgs* a, int sms) {
  constexpr int resident = static_cast<int>(220 * 1024 / (C::smem + 1024));
  a->cols = (a->N + C::FB - 1) / C::FB;
  int64_t want = static_cast<int64_t>(resident < 6 ? resident : 6) * WAVES * sms /
                 (static_cast<int64_t>(a->units) * C::SUB);
  if (want < 1) want = 1;
  a->parts = static_cast<int32_t>(want < a->cols ? want : a->cols);
}

template <int RT, bool F32>
cudaError_t launch_small(const ShrinkArgs& sa, ExpandArgs e, int sms, cudaStream_t st) {
  using S = Small<RT, F32>;
  static DeviceOnce once;
  const cudaError_t err = set_smem_limit_once(small_kernel<RT, F32>, S::smem, once);
  if (err != cudaSuccess) return err;
  e.cols = (e.N + S::E::FB - 1) / S::E::FB;
  // a cluster per possible tile; the more CTAs in it, the shorter its chain of
  // loads, while (about) all of them are resident, two an SM (64 tokens, 64
  // adapters of rank 16: 11.6 us at four, 16.5 at eight, 13.4 at two)
  const int64_t u = e.units;
  const int c = 8 * u <= 2 * sms ? 8 : 4 * u <= 3 * sms ? 4 : 2 * u <= 4 * sms ? 2 : 1;
  return launch_cluster(small_kernel<RT, F32>, dim3(static_cast<unsigned>(u * c)), c, S::smem, st, kThreads, sa, e);
}

template <int RT, bool F32>
cudaError_t launch_forward(const ShrinkArgs& sa, ExpandArgs e, int sms, cudaStream_t st) {
  using S = Shrink<RT, false, false>;
  static DeviceOnce once_s, once_e;
  cudaError_t err = set_smem_limit_once(shrink_x_kernel<RT>, S::smem, once_s);
  if (err != cudaSuccess) return err;
  const int c = shrink_cluster(likely_tiles(sa.tiles.T, sa.tiles.NA), sa.K, sms);
  err = launch_cluster(shrink_x_kernel<RT>, dim3(static_cast<unsigned>(e.units) * c), c, S::smem, st, kThreads,
                       sa);
  if (err != cudaSuccess) return err;
  using C = Expand<RT, false, F32, false>;
  err = set_smem_limit_once(expand_kernel<RT, F32>, C::smem, once_e);
  if (err != cudaSuccess) return err;
  split_features<C, 4>(&e, sms);
  const int64_t ctas = static_cast<int64_t>(e.units) * C::SUB * e.parts;
  if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  return launch_pdl(expand_kernel<RT, F32>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), C::smem,
                    st, e);
}

template <bool F32>
cudaError_t forward_products(const ShrinkArgs& sa, const ExpandArgs& e, bool small, int sms,
                             cudaStream_t st) {
  switch (rt_of(sa.r)) {
    case 1: return small ? launch_small<1, F32>(sa, e, sms, st) : launch_forward<1, F32>(sa, e, sms, st);
    case 2: return small ? launch_small<2, F32>(sa, e, sms, st) : launch_forward<2, F32>(sa, e, sms, st);
    case 4: return small ? launch_small<4, F32>(sa, e, sms, st) : launch_forward<4, F32>(sa, e, sms, st);
    default: return small ? launch_small<8, F32>(sa, e, sms, st) : launch_forward<8, F32>(sa, e, sms, st);
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
  constexpr size_t xs = Shrink<RT, false, false>::smem, ds = Shrink<RT, true, F32>::smem;
  constexpr size_t smem_s = xs > ds ? xs : ds;
  cudaError_t e = set_smem_limit_once(shrink_both_kernel<RT, F32>, smem_s, once_s);
  if (e != cudaSuccess) return e;
  const int64_t both = b.units * (b.want_x ? 2 : 1);
  // (the same split whichever outputs are wanted: their sums do not depend on it)
  // The shorter product's CTAs count as their share of the work, but for an
  // eighth at least: what one costs beside its chunks.
  const int longer = b.x.K > b.d.K ? b.x.K : b.d.K, shorter = b.x.K + b.d.K - longer;
  const int64_t tiles = likely_tiles(b.T, b.NA);
  int c = shrink_cluster(tiles + tiles * (8 * shorter > longer ? shorter : longer / 8) / longer, longer, b.sms);
  e = launch_cluster(shrink_both_kernel<RT, F32>, dim3(static_cast<unsigned>(both * c)), c, smem_s, st,
                     kThreads, b.d, b.x, static_cast<int>(b.units));
  if (e != cudaSuccess) return e;
  constexpr size_t gx = Grad<RT, false>::smem, gd = Grad<RT, F32>::smem;
  using E = Expand<RT, true, false, false>;
  constexpr size_t gm = gx > gd ? gx : gd, smem_o = gm > E::smem ? gm : E::smem;
  e = set_smem_limit_once(backward_out_kernel<RT, F32>, smem_o, once_o);
  if (e != cudaSuccess) return e;
  OutArgs o = b.out;
  const int fb = Grad<RT, F32>::FB;
  o.NA = b.NA;
  o.da_slabs = b.want_x ? (o.da.N + fb - 1) / fb : 0;
  o.db_slabs = b.want_x ? (o.db.N + fb - 1) / fb : 0;
  split_features<E, 2>(&o.dx, b.sms);
  const int64_t grads = static_cast<int64_t>(o.da_slabs + o.db_slabs) * b.NA;
  // CTAs that share an adapter's tokens: while the gradients' units leave SMs
  // idle and each has a tile or two
  c = 1;
  while (c < 8 && grads * c < 2 * b.sms && b.T >= 2 * c * kTile) c *= 2;
  int64_t ctas = b.want_dx ? b.units * E::SUB * o.dx.parts : 0;
  ctas = grads * c + (ctas + c - 1) / c * c;
  if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  return launch_cluster(backward_out_kernel<RT, F32>, dim3(static_cast<unsigned>(ctas)), c,
                        grads ? smem_o : E::smem, st, kThreads, o);
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
                       const float* scale, int row, int rows, int col, int r, int K) {
  ShrinkArgs a;
  a.tiles = c.tiles;
  a.src = src;
  a.ld = ld;
  a.pool = static_cast<const __nv_bfloat16*>(pool);
  a.scale = scale;
  a.dst.row = row < 0 ? nullptr : c.planes + row * c.w.plane;
  a.dst.rows = rows;
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
  a.v.rows = 0;
  a.v.col = nullptr;
  a.v.size = c.w.plane;
  a.pool = static_cast<const __nv_bfloat16*>(pool);
  a.base = base;
  a.ld_base = ld_base;
  a.out = out;
  a.ld_out = ld_out;
  a.r = r;
  a.N = N;
  a.cols = a.parts = 0;
  a.units = static_cast<int32_t>(c.w.units);
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
  if (!x || !ids || !a || !b)
    return entry_fail(MOE_ERR_INVALID_ARG, "x, adapter_ids, a or b is NULL");
  int32_t rc = check_rows("x", x, ld_x, s->in_features);
  if (rc != MOE_OK) return rc;
  if (!ptr_aligned(a, 16) || !ptr_aligned(b, 16))
    return entry_fail(MOE_ERR_MISALIGNED, "a and b must be 16-byte aligned");
  if (!ptr_aligned(ids, 4) || !ptr_aligned(scale, 4))
    return entry_fail(MOE_ERR_MISALIGNED, "adapter_ids and scale must be 4-byte aligned");
  const AdapterWs w = adapter_ws(s, backward);
  if (w.small) return MOE_OK;
  if (!workspace) return entry_fail(MOE_ERR_INVALID_ARG, "workspace is NULL");
  if (!ptr_aligned(workspace, kWsAlign))
    return entry_fail(MOE_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  const size_t need = w.total;
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
  const ExpandArgs ea = expand_args(c, b, base, ld_base, out, ld_out, s->rank, s->out_features);
  const bool f32 = s->out_dtype == MOE_DTYPE_F32;
  const ShrinkArgs sa = shrink_args(c, x, ld_x, a, scale, 0, f32 ? 3 : 2, -1, s->rank, s->in_features);
  cudaError_t e = cudaSuccess;
  if (!c.w.small) e = launch_group(adapter_ids, s->num_tokens, s->num_adapters, c.g, st);
  if (e == cudaSuccess)
    e = f32 ? forward_products<true>(sa, ea, c.w.small, sms, st)
            : forward_products<false>(sa, ea, c.w.small, sms, st);
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
  w.d = shrink_args(c, dout, ld_dout, b, scale, dx ? kURow : -1, 2, da ? kUCol : -1, r, N);
  w.x = shrink_args(c, x, ld_x, a, scale, -1, 0, kWCol, r, H);
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
