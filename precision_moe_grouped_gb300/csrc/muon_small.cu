// muon_small.cu -- the orthogonalised step for matrices with a short side m of up
// to 64 (pools of adapters, small heads): muon.cu's steps on m x m matrices, in
// float on the CUDA cores, and the products with the long side on mma.sync.
//
// tcgen05 would compute tiles of 128 x 256 for matrices of 16 x 16.  Here a
// matrix is a stream: a block takes a run of its columns (its long side), tile
// by tile through shared memory, whose loads bound multiply-adds from there
// (48 of 16 x 7168 and 48 of 4096 x 16: 86 us, 80 on mma.sync; 300 of 16 x 4096 156 / 140;
// 96 of 32 x 4096 189 / 181; 40 of 64 x 4096, which the m x m steps and the legacy
// pipe's rate bound, 363 / 369, 64 of 2000 x 33 246 / 231).
//   gram:  m <- mu m + (1 - mu) g, u; or u again and Y = Q u; each block's
//          share of u u^T (whose trace is |u|^2) or Y Y^T
//   steps: one block a matrix joins the shares in order and carries out up to
//          three steps; Q <- P Q.  Q is kept transposed, as the products here are
//          A B^T: with P Q^T instead, what rounding leaves of Q's asymmetry would
//          not be that of the X whose Gram matrix follows (errors 6 to 20 times
//          larger where a singular value is small)
//   apply: p <- decay p - step Q u
// Memory is met in packs of four elements where rows and addresses allow it, which
// takes three instructions of four off the elementwise parts (48 of 16 x 7168 and 48 of
// 4096 x 16: 97 -> 86 us; 96 of 32 x 4096 212 -> 189).
// All tensors of a size class go in one launch of each kernel.  Matrices that fit
// into the shared memory of a cluster go through all of it in one kernel, which
// reads and writes every tensor once; the three kernels are for longer ones, and for
// few others beside them.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "cluster.cuh"
#include "entry.h"
#include "muon.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kCap = 40;           // tensors of a launch: its kernel parameter stays below 4 KB
constexpr int kTargetBlocks = 304; // two blocks an SM, all resident at once

struct Entry {
  Momentum mo;
  float* p;
  __nv_bfloat16* copy;
  float step;
  int32_t m, n, tall;
  int32_t blocks;       // of a matrix
  int32_t first_block;  // of the launch
  int32_t first_matrix;
};
struct Table {
  Entry e[kCap];
  int32_t count;
  float decay;
};

// MP: m rounded up to 16, 32 or 64.  A tile is MP x NC (4096 elements, 16 a
// thread); in products with a tile a thread computes 4 x 4 elements, which
// keeps shared memory's reads at two floats for four multiply-adds.
template <int MP>
struct Cfg {
  static constexpr int NC = 4096 / MP;
  static constexpr int TR = MP / 16;   // m x m products: TR x TR elements a thread
  static constexpr int LD = NC + 4;    // rows 16 bytes apart modulo the banks
  static constexpr int LDM = MP + 4;
  static constexpr int PER = 16;
  // Warps in products with a tile: one of the MP / 16 strips of 16 rows each, one
  // of kStrips runs of 32 columns of the tile.  In a Gram matrix a warp sums over
  // its run, and covers all of a strip, or (64 rows) half of it.
  static constexpr int kRows = MP / 16, kRuns = 8 / kRows;
  static constexpr int kSums = MP == 64 ? 1 : kRuns;        // Gram matrices of a tile
  static constexpr int kGramTiles = MP == 16 ? 2 : 4;       // of 16 x 8, a warp's
  static constexpr int kGramCols = NC / kSums;              // columns that a warp sums over
  static_assert(NC == 32 * kRuns, "a run has 32 columns");
  static_assert(kSums * MP * MP <= MP * LD || kSums == 1, "the sums are joined in the tile's memory");
};

template <int MP>
__device__ __forceinline__ void zero(float (&c)[Cfg<MP>::TR][Cfg<MP>::TR]) {
#pragma unroll
  for (int r = 0; r < Cfg<MP>::TR; ++r)
#pragma unroll
    for (int s = 0; s < Cfg<MP>::TR; ++s) c[r][s] = 0.f;
}
// This thread's rows i = (tid / 16) + 16 r and columns j = (tid % 16) + 16 s.
__device__ __forceinline__ int ti() { return threadIdx.x >> 4; }
__device__ __forceinline__ int tj() { return threadIdx.x & 15; }

// c[i][j] += sum over k of a[i][k] b[j][k], k < K, rows ld apart.
template <int MP, int K, int LD>
__device__ __forceinline__ void dot_rows(const float* a, const float* b, float (&c)[Cfg<MP>::TR][Cfg<MP>::TR]) {
  constexpr int TR = Cfg<MP>::TR;
#pragma unroll 4
  for (int k = 0; k < K; k += 4) {
    float4 x[TR], y[TR];
#pragma unroll
    for (int r = 0; r < TR; ++r) {
      x[r] = *reinterpret_cast<const float4*>(a + (ti() + 16 * r) * LD + k);
      y[r] = *reinterpret_cast<const float4*>(b + (tj() + 16 * r) * LD + k);
    }
#pragma unroll
    for (int r = 0; r < TR; ++r)
#pragma unroll
      for (int s = 0; s < TR; ++s)
        c[r][s] = fmaf(x[r].x, y[s].x, fmaf(x[r].y, y[s].y, fmaf(x[r].z, y[s].z, fmaf(x[r].w, y[s].w, c[r][s]))));
  }
}
template <int MP>
__device__ __forceinline__ void put(float* to, const float (&c)[Cfg<MP>::TR][Cfg<MP>::TR]) {
#pragma unroll
  for (int r = 0; r < Cfg<MP>::TR; ++r)
#pragma unroll
    for (int s = 0; s < Cfg<MP>::TR; ++s) to[(ti() + 16 * r) * Cfg<MP>::LDM + tj() + 16 * s] = c[r][s];
}

// What a block works on.
struct Work {
  int32_t e, z, part;
};
__device__ __forceinline__ Work find_block(const Table& t, int b) {
  Work w;
  w.e = 0;
  while (w.e + 1 < t.count && b >= t.e[w.e + 1].first_block) ++w.e;
  b -= t.e[w.e].first_block;
  w.z = b / t.e[w.e].blocks;
  w.part = b - w.z * t.e[w.e].blocks;
  return w;
}

// V neighbours in memory, met in one access.
template <class T, int V>
struct alignas(V * sizeof(T)) Pack {
  T v[V];
};
template <int V, class T>
__device__ __forceinline__ Pack<T, V> load_pack(const T* p) {
  return *reinterpret_cast<const Pack<T, V>*>(p);
}

// This thread's 16 elements of the tile at column n0, in packs of V along the
// memory's rows: pack k at row i + k di and column j + k dj of X, `at + k step` in
// the matrix.  Packs outside of the matrix read its first one: loads without
// branches stay in flight together.  (V = 4: the rows in memory are multiples of
// 4, so that a pack is inside or outside as a whole.)
template <int MP, int V>
struct Elements {
  static constexpr int kPacks = Cfg<MP>::PER / V;
  int i, j, di, dj, m, cols;
  int at, step;   // below 2^26: m <= 64, n <= 2^20
  bool tall;

  __device__ __forceinline__ Elements(const Entry& e, int n0, int n1) : m(e.m), cols(n1 - n0), tall(e.tall) {
    constexpr int NC = Cfg<MP>::NC;
    const int t = threadIdx.x;
    if (tall) {
      i = t % (MP / V) * V, j = t / (MP / V), di = 0, dj = kThreads / (MP / V);
      at = (n0 + j) * e.m + i;
      step = dj * e.m;
    } else {
      i = t / (NC / V), j = t % (NC / V) * V, di = kThreads / (NC / V), dj = 0;
      at = i * e.n + n0 + j;
      step = di * e.n;
    }
  }
  __device__ __forceinline__ bool in(int k) const { return i + k * di < m && j + k * dj < cols; }
  __device__ __forceinline__ int where(int k) const { return in(k) ? at + k * step : 0; }
  template <class T>
  __device__ __forceinline__ void store(T* p, int k, const Pack<T, V>& v) const {
    if (in(k)) *reinterpret_cast<Pack<T, V>*>(p + where(k)) = v;
  }
  // the pack's place in the tile: a run of a row, or of a column of a tall matrix
  __device__ __forceinline__ void to_tile(float* u, int k, const Pack<float, V>& v, int ld) const {
    float* to = u + (i + k * di) * ld + j + k * dj;
    if (V == 1 || !tall) {
      *reinterpret_cast<Pack<float, V>*>(to) = v;
    } else {
#pragma unroll
      for (int c = 0; c < V; ++c) to[c * ld] = v.v[c];
    }
  }
  __device__ __forceinline__ Pack<float, V> from_tile(const float* u, int k, int ld) const {
    const float* from = u + (i + k * di) * ld + j + k * dj;
    if (V == 1 || !tall) return *reinterpret_cast<const Pack<float, V>*>(from);
    Pack<float, V> v;
#pragma unroll
    for (int c = 0; c < V; ++c) v.v[c] = from[c * ld];
    return v;
  }
};

template <bool BF16>
using Grad = typename std::conditional<BF16, __nv_bfloat16, float>::type;

// A tile's momentum and gradient, from memory to registers ...
template <int MP, bool BF16, int V>
struct Fetched {
  using X = Elements<MP, V>;
  Pack<float, V> m[X::kPacks];
  Pack<Grad<BF16>, V> g[X::kPacks];

  __device__ __forceinline__ void fetch(const X& x, const float* mp, const Grad<BF16>* gp, bool need_g) {
#pragma unroll
    for (int k = 0; k < X::kPacks; ++k) m[k] = load_pack<V>(mp + x.where(k));
    if (need_g) {
#pragma unroll
      for (int k = 0; k < X::kPacks; ++k) g[k] = load_pack<V>(gp + x.where(k));
    }
  }
  // ... and u from there to shared memory, zero outside of the matrix; FIRST:
  // with the momentum's update.
  template <bool FIRST>
  __device__ __forceinline__ void put(const X& x, const Momentum& mo, float* mp, float gs, float* u,
                                      int ld = Cfg<MP>::LD) const {
#pragma unroll
    for (int k = 0; k < X::kPacks; ++k) {
      Pack<float, V> mv = m[k], uv;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float gv = FIRST || mo.nesterov ? static_cast<float>(g[k].v[c]) * gs : 0.f;
        if (FIRST) mv.v[c] = fmaf(mo.mu, mv.v[c], mo.rest * gv);
        uv.v[c] = x.in(k) ? update_of(mo, mv.v[c], gv) : 0.f;
      }
      if (FIRST) x.store(mp, k, mv);
      x.to_tile(u, k, uv, ld);
    }
  }
};

// p <- decay p - step Y and the copy, for the tile's Y = Q u.
template <int MP, int V>
__device__ __forceinline__ void put_params(const Elements<MP, V>& x, const Pack<float, V> (&pv)[Elements<MP, V>::kPacks],
                                           const Entry& e, float decay, const float* y, int ld, float* p,
                                           __nv_bfloat16* copy) {
#pragma unroll
  for (int k = 0; k < Elements<MP, V>::kPacks; ++k) {
    Pack<float, V> v = x.from_tile(y, k, ld);
    Pack<__nv_bfloat16, V> c;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v.v[i] = fmaf(-e.step, v.v[i], decay * pv[k].v[i]);
      c.v[i] = __float2bfloat16_rn(v.v[i]);
    }
    x.store(p, k, v);
    if (e.copy) x.store(copy, k, c);
  }
}

// Products with a tile run on mma.sync with each number as two tf32 terms of 11
// bits, hi + lo, and three products, lo hi + hi lo + hi hi: 22 bits, and sums in
// float.  Multiply-adds from shared memory would be bound by its 16-byte loads, which cost
// four cycles each whatever their lanes share.
struct Terms {
  uint32_t hi, lo;
  __device__ __forceinline__ Terms() {}
  __device__ __forceinline__ Terms(float x) {
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(x - __uint_as_float(hi)));
  }
};
__device__ __forceinline__ void mma_tf32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d += a b: a's rows g and g + 8 at columns t and t + 4, b's rows t and t + 4 at column g.
__device__ __forceinline__ void mma_terms(float (&d)[4], const Terms (&a)[4], const Terms& b0, const Terms& b1) {
  mma_tf32(d, a[0].lo, a[1].lo, a[2].lo, a[3].lo, b0.hi, b1.hi);
  mma_tf32(d, a[0].hi, a[1].hi, a[2].hi, a[3].hi, b0.lo, b1.lo);
  mma_tf32(d, a[0].hi, a[1].hi, a[2].hi, a[3].hi, b0.hi, b1.hi);
}

// c += sum over this warp's columns of u[i][k] u[j][k], i of its strip, j of its
// kGramTiles blocks of 8: c[n] is an MMA's result.  The MMA cuts its sums off, so
// a tile's are added in float.
template <int MP>
__device__ __forceinline__ void gram_tile(const float* u, int ld, float (&c)[4][4]) {
  using C = Cfg<MP>;
  const int warp = threadIdx.x >> 5, g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
  const int strip = warp % C::kRows, part = warp / C::kRows;
  const int j0 = MP == 64 ? part * 32 : 0, k0 = MP == 64 ? 0 : part * C::kGramCols;
  float d[C::kGramTiles][4] = {};
#pragma unroll 2
  for (int k = k0; k < k0 + C::kGramCols; k += 8) {
    const float* at = u + k + t;
    Terms a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = Terms(at[(strip * 16 + g + 8 * (i & 1)) * ld + 4 * (i >> 1)]);
#pragma unroll
    for (int n = 0; n < C::kGramTiles; ++n) {
      // (16 rows: what a holds already)
      const float* row = at + (j0 + 8 * n + g) * ld;
      const Terms b0 = MP == 16 ? a[n & 1] : Terms(row[0]), b1 = MP == 16 ? a[2 + (n & 1)] : Terms(row[4]);
      mma_terms(d[n], a, b0, b1);
    }
  }
#pragma unroll
  for (int n = 0; n < C::kGramTiles; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) c[n][i] += d[n][i];
}
// The parts' sums joined in order, through the tile's memory, to `to`.  What lies
// below the diagonal is taken from above, so that the matrix is symmetric.
template <int MP>
__device__ __forceinline__ void put_gram(float (&c)[4][4], float* u, float* to) {
  using C = Cfg<MP>;
  const int warp = threadIdx.x >> 5, g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
  const int strip = warp % C::kRows, part = warp / C::kRows;
  float* at = C::kSums == 1 ? to : u + part * MP * MP;
#pragma unroll
  for (int n = 0; n < C::kGramTiles; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = strip * 16 + g + 8 * (i >> 1), col = (MP == 64 ? part * 32 : 0) + 8 * n + 2 * t + (i & 1);
      if (row > col) continue;
      at[row * MP + col] = c[n][i];
      at[col * MP + row] = c[n][i];
    }
  if (C::kSums == 1) return;
  __syncthreads();
  for (int i = threadIdx.x; i < MP * MP; i += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < C::kSums; ++j) v += u[j * MP * MP + i];
    to[i] = v;
  }
}

// u <- Q u for the tile, a strip of rows and a run of columns a warp; q holds Q^T.
template <int MP>
__device__ __forceinline__ void mul_tile(const float* q, float* u, int ld) {
  using C = Cfg<MP>;
  const int warp = threadIdx.x >> 5, g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
  const int row = (warp % C::kRows) * 16 + g, col = warp / C::kRows * 32;
  float y[4][4] = {};
#pragma unroll 2
  for (int k = 0; k < MP; k += 8) {
    Terms a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = Terms(q[(k + t + 4 * (i >> 1)) * C::LDM + row + 8 * (i & 1)]);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const float* at = u + (k + t) * ld + col + 8 * n + g;
      mma_terms(y[n], a, Terms(at[0]), Terms(at[4 * ld]));
    }
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < 4; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<float2*>(u + (row + 8 * i) * ld + col + 8 * n + 2 * t) = make_float2(y[n][2 * i], y[n][2 * i + 1]);
  __syncthreads();
}
template <int MP>
__device__ __forceinline__ void load_q(const float* from, float* q) {
  for (int k = threadIdx.x; k < MP * MP; k += kThreads) q[(k / MP) * Cfg<MP>::LDM + k % MP] = from[k];
}

template <int MP>
__device__ __forceinline__ void columns_of(const Entry& e, int part, int* n0, int* n1) {
  const int tiles = (e.n + Cfg<MP>::NC - 1) / Cfg<MP>::NC;
  *n0 = static_cast<int>(static_cast<int64_t>(tiles) * part / e.blocks) * Cfg<MP>::NC;
  *n1 = min(e.n, static_cast<int>(static_cast<int64_t>(tiles) * (part + 1) / e.blocks) * Cfg<MP>::NC);
}

// Each block's share of u u^T (FIRST) or of Y Y^T, Y = Q u.
template <int MP, bool FIRST, bool BF16, int V>
__global__ void __launch_bounds__(kThreads, 2)
    muon_small_gram_kernel(const __grid_constant__ Table t, const float* qs, float* shares) {
  using C = Cfg<MP>;
  __shared__ __align__(16) float u[MP * C::LD];
  __shared__ __align__(16) float q[FIRST ? 4 : MP * C::LDM];
  griddep_wait();
  griddep_launch_dependents();
  const Work w = find_block(t, blockIdx.x);
  const Entry& e = t.e[w.e];
  const float gs = e.mo.grad_scale ? __ldg(e.mo.grad_scale) : 1.0f;
  const int64_t base = static_cast<int64_t>(w.z) * e.m * e.n;
  if (!FIRST) load_q<MP>(qs + static_cast<int64_t>(e.first_matrix + w.z) * MP * MP, q);
  float* mp = e.mo.m + base;
  const Grad<BF16>* gp = static_cast<const Grad<BF16>*>(e.mo.grad) + base;
  const bool need_g = FIRST || e.mo.nesterov;
  int n0, n1;
  columns_of<MP>(e, w.part, &n0, &n1);
  float c[4][4] = {};
  Fetched<MP, BF16, V> f;
  f.fetch(Elements<MP, V>(e, n0, n1), mp, gp, need_g);
  for (; n0 < n1; n0 += C::NC) {
    f.template put<FIRST>(Elements<MP, V>(e, n0, n1), e.mo, mp, gs, u);
    __syncthreads();
    if (n0 + C::NC < n1) f.fetch(Elements<MP, V>(e, n0 + C::NC, n1), mp, gp, need_g);   // under the products
    if (!FIRST) mul_tile<MP>(q, u, C::LD);
    gram_tile<MP>(u, C::LD, c);
    __syncthreads();
  }
  put_gram<MP>(c, u, shares + static_cast<int64_t>(blockIdx.x) * MP * MP);
}

// `n` steps on G, all three [MP][LDM] in shared memory: Q <- P Q, or, `fresh`, Q
// begins as `first` I.  q holds Q^T.
template <int MP>
__device__ __forceinline__ void newton_schulz(float* g, float* p, float* q, int n, bool fresh, float first, int m,
                                              float ca, float cb, float cc) {
  using C = Cfg<MP>;
  float c[C::TR][C::TR];
  for (int step = 0; step < n; ++step) {
    zero<MP>(c);
    dot_rows<MP, MP, C::LDM>(g, g, c);
#pragma unroll
    for (int r = 0; r < C::TR; ++r)
#pragma unroll
      for (int s = 0; s < C::TR; ++s) {
        const int i = ti() + 16 * r, j = tj() + 16 * s;
        c[r][s] = fmaf(cc, c[r][s], cb * g[i * C::LDM + j]) + (i == j && i < m ? ca : 0.f);
      }
    put<MP>(p, c);
    __syncthreads();
    if (fresh && step == 0) {
#pragma unroll
      for (int r = 0; r < C::TR; ++r)
#pragma unroll
        for (int s = 0; s < C::TR; ++s) c[r][s] *= first;
    } else {
      zero<MP>(c);
      dot_rows<MP, MP, C::LDM>(q, p, c);   // Q^T P^T
      __syncthreads();
    }
    put<MP>(q, c);
    if (step + 1 < n) {   // G <- (P G) P
      zero<MP>(c);
      dot_rows<MP, MP, C::LDM>(p, g, c);
      __syncthreads();
      put<MP>(g, c);
      __syncthreads();
      zero<MP>(c);
      dot_rows<MP, MP, C::LDM>(g, p, c);
      __syncthreads();
      put<MP>(g, c);
    }
    __syncthreads();
  }
}

// One matrix a block: `n` steps from G, the sum of its shares.
template <int MP, bool FIRST>
__global__ void __launch_bounds__(kThreads)
    muon_small_steps_kernel(const __grid_constant__ Table t, const float* shares, float* qs, int n, float ca,
                            float cb, float cc, float eps) {
  using C = Cfg<MP>;
  extern __shared__ __align__(16) float mem[];
  float *g = mem, *p = g + MP * C::LDM, *q = p + MP * C::LDM;
  griddep_wait();
  griddep_launch_dependents();
  int k = 0;
  while (k + 1 < t.count && static_cast<int>(blockIdx.x) >= t.e[k + 1].first_matrix) ++k;
  const Entry& e = t.e[k];
  const int z = static_cast<int>(blockIdx.x) - e.first_matrix;
  const float* from = shares + (static_cast<int64_t>(e.first_block) + static_cast<int64_t>(z) * e.blocks) * MP * MP;
  float* to = qs + static_cast<int64_t>(blockIdx.x) * MP * MP;
  if (!FIRST) load_q<MP>(to, q);
  float c[C::TR][C::TR];
  zero<MP>(c);
#pragma unroll 4
  for (int b = 0; b < e.blocks; ++b)
#pragma unroll
    for (int r = 0; r < C::TR; ++r)
#pragma unroll
      for (int s = 0; s < C::TR; ++s)
        c[r][s] += from[static_cast<int64_t>(b) * MP * MP + (ti() + 16 * r) * MP + tj() + 16 * s];
  put<MP>(g, c);
  __syncthreads();
  float inv = 1.0f;
  if (FIRST) {   // |u|^2 is the trace
    float s = 0.f;
    for (int i = 0; i < e.m; ++i) s += g[i * C::LDM + i];
    inv = 1.0f / (sqrtf(s) + eps);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < C::TR; ++r)
#pragma unroll
      for (int v = 0; v < C::TR; ++v) c[r][v] = (c[r][v] * inv) * inv;
    put<MP>(g, c);
    __syncthreads();
  }
  newton_schulz<MP>(g, p, q, n, FIRST, inv, e.m, ca, cb, cc);
  for (int i = threadIdx.x; i < MP * MP; i += kThreads) to[i] = q[(i / MP) * C::LDM + i % MP];
}

// p <- decay p - step Q u, and the copy.
template <int MP, bool BF16, int V>
__global__ void __launch_bounds__(kThreads, 2)
    muon_small_apply_kernel(const __grid_constant__ Table t, const float* qs) {
  using C = Cfg<MP>;
  __shared__ __align__(16) float u[MP * C::LD];
  __shared__ __align__(16) float q[MP * C::LDM];
  griddep_wait();
  griddep_launch_dependents();
  const Work w = find_block(t, blockIdx.x);
  const Entry& e = t.e[w.e];
  const float gs = e.mo.grad_scale ? __ldg(e.mo.grad_scale) : 1.0f;
  const int64_t base = static_cast<int64_t>(w.z) * e.m * e.n;
  load_q<MP>(qs + static_cast<int64_t>(e.first_matrix + w.z) * MP * MP, q);
  float *mp = e.mo.m + base, *p = e.p + base;
  const Grad<BF16>* gp = static_cast<const Grad<BF16>*>(e.mo.grad) + base;
  __nv_bfloat16* copy = e.copy + base;
  int n0, n1;
  columns_of<MP>(e, w.part, &n0, &n1);
  Fetched<MP, BF16, V> f;
  f.fetch(Elements<MP, V>(e, n0, n1), mp, gp, e.mo.nesterov);
  for (; n0 < n1; n0 += C::NC) {
    const Elements<MP, V> x(e, n0, n1);
    f.template put<false>(x, e.mo, mp, gs, u);
    Pack<float, V> pv[x.kPacks];
#pragma unroll
    for (int k = 0; k < x.kPacks; ++k) pv[k] = load_pack<V>(&p[x.where(k)]);
    __syncthreads();
    mul_tile<MP>(q, u, C::LD);
    if (n0 + C::NC < n1) f.fetch(Elements<MP, V>(e, n0 + C::NC, n1), mp, gp, e.mo.nesterov);
    put_params(x, pv, e, t.decay, u, C::LD, p, copy);
    __syncthreads();
  }
}

// The whole step of a matrix in one cluster: u stays in the shared memory of its
// CTAs, each with an equal run of columns, from the momentum's update to the
// parameter's, so that every tensor is met once.  Shares of a Gram matrix are
// read from all CTAs in rank order, and every CTA carries out the m x m steps for
// itself.
struct Schedule {
  int32_t steps;
  float a, b, c, eps;
};
template <int MP>
__host__ __device__ constexpr int cluster_scratch() {   // floats beside u: G, P, Q, this CTA's share, the groups' sums
  return 3 * MP * Cfg<MP>::LDM + MP * MP + (Cfg<MP>::kSums > 1 ? Cfg<MP>::kSums * MP * MP : 0);
}

template <int MP, bool BF16, int V>
__global__ void __launch_bounds__(kThreads, 2)
    muon_cluster_kernel(const __grid_constant__ Table t, const Schedule sc) {
  using C = Cfg<MP>;
  extern __shared__ __align__(16) float mem[];
  float *g = mem, *p = g + MP * C::LDM, *q = p + MP * C::LDM, *share = q + MP * C::LDM;
  float* groups = share + MP * MP;
  float* u = mem + cluster_scratch<MP>();
  griddep_wait();
  griddep_launch_dependents();
  const int ranks = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int matrix = static_cast<int>(blockIdx.x) / ranks;
  int at = 0;
  while (at + 1 < t.count && matrix >= t.e[at + 1].first_matrix) ++at;
  const Entry& e = t.e[at];
  const float gs = e.mo.grad_scale ? __ldg(e.mo.grad_scale) : 1.0f;
  const int64_t base = static_cast<int64_t>(matrix - e.first_matrix) * e.m * e.n;
  float *mp = e.mo.m + base, *pp = e.p + base;
  const Grad<BF16>* gp = static_cast<const Grad<BF16>*>(e.mo.grad) + base;
  __nv_bfloat16* copy = e.copy + base;
  const int tiles = (e.n + C::NC - 1) / C::NC;
  const int first = tiles * rank / ranks * C::NC, last = tiles * (rank + 1) / ranks * C::NC;
  const int end = min(e.n, last), ld = (tiles + ranks - 1) / ranks * C::NC + 4;
  {
    Fetched<MP, BF16, V> f, next;
    f.fetch(Elements<MP, V>(e, first, end), mp, gp, true);
    for (int n0 = first; n0 < last; n0 += C::NC) {
      if (n0 + C::NC < last) next.fetch(Elements<MP, V>(e, n0 + C::NC, end), mp, gp, true);
      f.template put<true>(Elements<MP, V>(e, n0, end), e.mo, mp, gs, u + (n0 - first), ld);
      f = next;
    }
  }
  __syncthreads();
  for (int done = 0; done < sc.steps; done += kMuonPartSteps) {
    float c[4][4] = {};
    for (int n0 = first; n0 < last; n0 += C::NC) gram_tile<MP>(u + (n0 - first), ld, c);
    if (done) cluster_sync();   // the others have read the last share
    put_gram<MP>(c, groups, share);
    cluster_sync();
    for (int i = threadIdx.x; i < MP * MP / 4; i += kThreads) {
      float4 x[8];   // all ranks' loads in flight together
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < ranks) x[r] = cluster_load4(share + 4 * i, r);
      float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < ranks) v = make_float4(v.x + x[r].x, v.y + x[r].y, v.z + x[r].z, v.w + x[r].w);
      *reinterpret_cast<float4*>(g + (4 * i / MP) * C::LDM + 4 * i % MP) = v;
    }
    __syncthreads();
    float inv = 1.0f;
    if (done == 0) {   // |u|^2 is the trace
      float s = 0.f;
      for (int i = 0; i < e.m; ++i) s += g[i * C::LDM + i];
      inv = 1.0f / (sqrtf(s) + sc.eps);
      __syncthreads();
      for (int i = threadIdx.x; i < MP * MP; i += kThreads) {
        float& v = g[(i / MP) * C::LDM + i % MP];
        v = (v * inv) * inv;
      }
      __syncthreads();
    }
    const int n = min(kMuonPartSteps, sc.steps - done);
    newton_schulz<MP>(g, p, q, n, true, inv, e.m, sc.a, sc.b, sc.c);
    if (done + n < sc.steps) {
      for (int n0 = first; n0 < last; n0 += C::NC) mul_tile<MP>(q, u + (n0 - first), ld);
    } else {
      if constexpr (MP < 64 && V == 4) {
        for (int n0 = first; n0 < last; n0 += C::NC) {
          const Elements<MP, V> x(e, n0, end);
          Pack<float, V> pv[x.kPacks];
#pragma unroll
          for (int k = 0; k < x.kPacks; ++k) pv[k] = load_pack<V>(&pp[x.where(k)]);
          mul_tile<MP>(q, u + (n0 - first), ld);
          put_params(x, pv, e, t.decay, u + (n0 - first), ld, pp, copy);
        }
      } else {   // the products, or the single loads, are long enough for the next tile's p to be worth its registers
        Pack<float, V> pv[Elements<MP, V>::kPacks], next[Elements<MP, V>::kPacks];
        for (int n0 = first - C::NC; n0 < last; n0 += C::NC) {
          const Elements<MP, V> x(e, n0, end), y(e, n0 + C::NC, end);
          if (n0 >= first) mul_tile<MP>(q, u + (n0 - first), ld);
          if (n0 + C::NC < last) {
#pragma unroll
            for (int k = 0; k < x.kPacks; ++k) next[k] = load_pack<V>(&pp[y.where(k)]);
          }
          if (n0 >= first) put_params(x, pv, e, t.decay, u + (n0 - first), ld, pp, copy);
#pragma unroll
          for (int k = 0; k < x.kPacks; ++k) pv[k] = next[k];
        }
      }
    }
  }
  cluster_sync();   // no CTA leaves while another may read its share
}

int size_class(const moe_muon_tensor& t) {
  const int m = std::min(t.rows, t.cols);
  return m <= 16 ? 16 : m <= 32 ? 32 : 64;
}

bool of_class(const moe_muon_tensor& t, int mp) {
  return !muon_empty(t) && muon_is_small(t) && size_class(t) == mp;
}

constexpr int64_t kMaxBlocks = int64_t(1) << 22;
int64_t tiles_of(const moe_muon_tensor& t) {
  const int nc = 4096 / size_class(t);
  return (std::max(t.rows, t.cols) + nc - 1) / nc;
}

// Shared memory of a cluster's CTA that holds `tiles` of a matrix; a CTA has at most kWholeSm.
constexpr int kHalfSm = 113 * 1024, kWholeSm = 227 * 1024;
constexpr int kMaxRanks = 8;
template <int MP>
constexpr int64_t cluster_smem(int64_t tiles) {
  return 4 * (cluster_scratch<MP>() + MP * (tiles * Cfg<MP>::NC + 4));
}
// Whether a cluster holds the tensor's matrices.
bool is_resident(const moe_muon_tensor& t) {
  const int64_t each = (tiles_of(t) + kMaxRanks - 1) / kMaxRanks;
  const int mp = size_class(t);
  return (mp == 16 ? cluster_smem<16>(each) : mp == 32 ? cluster_smem<32>(each) : cluster_smem<64>(each)) <= kWholeSm;
}

// A launch's tensors, of one class.
struct Batch {
  int32_t index[kCap];
  int32_t count;
  int64_t matrices, blocks;
  int64_t tiles;   // of a block, at most
  bool resident;   // clusters hold all of them
};
// Tensors that a cluster holds go with longer ones of their class through the three kernels,
// which saves the cluster kernel's launch, unless they are more matrices than this.  Beside 8 x 70000,
// together and apart: 48 of 16 x 4096 61 and 89 us, 300 265 / 196, 1000 744 / 467; 30 x 20000: 48 of 32 x 4096
// 158 / 184, 300 515 / 565, 1000 1767 / 1662; 64 x 20000: 48 of 64 x 4096 351 / 650, 1000 5096 / 8327, 1000 of
// 64 x 400 893 / 905.  (They also take no workspace apart: Q and the shares of many small matrices are
// larger than these.)
constexpr int64_t joined_matrices(int mp) { return mp == 16 ? 128 : mp == 32 ? 512 : INT64_MAX; }
enum class Pick { kAll, kResident, kLonger };
int64_t blocks_of(const moe_muon_tensor& t, const Batch& b) { return (tiles_of(t) + b.tiles - 1) / b.tiles; }

// The next batch of class mp at or after *at (a tensor's index); false: none.
// Its blocks take as few tiles each as leaves all of them resident at once; where
// that would be more than twice their fair share (many matrices beside a longer one),
// they take that, and the blocks that have no place at first follow the others.
bool next_batch(const moe_muon_tensor* t, int32_t count, int mp, Pick pick, int32_t* at, Batch* b) {
  b->count = 0;
  b->resident = true;
  b->matrices = 0;
  int64_t all = 0, most = 1;
  for (; *at < count && b->count < kCap; ++*at) {
    if (!of_class(t[*at], mp)) continue;
    const bool resident = is_resident(t[*at]);
    if (pick != Pick::kAll && (pick == Pick::kResident) != resident) continue;
    if (b->count && b->matrices + t[*at].count > kMaxBlocks) break;
    b->index[b->count++] = *at;
    b->resident = b->resident && resident;
    b->matrices += t[*at].count;
    all += t[*at].count * tiles_of(t[*at]);
    most = std::max(most, tiles_of(t[*at]));
  }
  const int64_t fair = std::min(most, std::max<int64_t>(1, (all + kTargetBlocks - 1) / kTargetBlocks));
  auto cut = [&](int64_t tiles) {
    b->tiles = tiles;
    b->blocks = 0;
    for (int i = 0; i < b->count; ++i) b->blocks += t[b->index[i]].count * blocks_of(t[b->index[i]], *b);
    return b->blocks <= kTargetBlocks;
  };
  int64_t tiles = fair;
  while (!cut(tiles) && tiles < std::min(most, 2 * fair)) ++tiles;
  if (b->blocks > kTargetBlocks) cut(fair);
  return b->count > 0;
}
// Calls f(class, batch) with all batches.  Stops at the first error.
template <class F>
int32_t each_batch(const moe_muon_tensor* t, int32_t count, F f) {
  Batch b;
  for (int mp : {16, 32, 64}) {
    int64_t held = 0;
    bool longer = false;
    for (int i = 0; i < count; ++i) {
      if (!of_class(t[i], mp)) continue;
      if (is_resident(t[i])) held += t[i].count;
      else longer = true;
    }
    const bool apart = longer && held > joined_matrices(mp);
    for (Pick pick : {apart ? Pick::kResident : Pick::kAll, Pick::kLonger}) {
      if (pick == Pick::kLonger && !apart) break;
      for (int32_t at = 0; next_batch(t, count, mp, pick, &at, &b);) MOE_TRY(f(mp, b));
    }
  }
  return MOE_OK;
}

// Whether the tensor can be met in packs of four.
bool in_fours(const moe_muon_tensor& x, bool bf16) {
  return x.cols % 4 == 0 && ptr_aligned(x.param, 16) && ptr_aligned(x.momentum, 16) &&
         ptr_aligned(x.grad, bf16 ? 8 : 16) && ptr_aligned(x.param_bf16, 8);
}
// A launch meets its tensors in packs if it can all of them.  Beside ones that cannot be, matrices
// of up to 16 rows in clusters have a launch of their own from this many tiles on (with 1 of 16 x 333,
// one launch and two: 48 of 16 x 4096, 768 tiles, 41 and 46 us; 96 60 / 64; 48 of 16 x 7168 and 48 of
// 4096 x 16, 2112 tiles, 97 / 91; 600 of 16 x 4096 325 / 267).  Those of up to 32 rows gain less: 48 of
// 32 x 4096 113 / 127, 96 202 / 200.  (Both ways in one kernel, by tensor, cost registers: 81 -> 83 us for
// the pools without an odd one, 40 of 64 x 4096 370 -> 425.)
constexpr int64_t kPackedTiles = 2000;

// How many clusters of 1 .. 8 CTAs are resident at once, with half of an SM's
// memory a CTA and with all of it; asked once per kernel and device.
template <int MP, bool BF16, int V>
cudaError_t resident_clusters(int ranks, bool whole, int* n) {
  static DeviceOnce table[16];
  cudaError_t e;
  std::atomic<int>* at = device_entry(table[2 * (ranks - 1) + whole], &e);
  if (!at) return e;
  *n = at->load(std::memory_order_acquire);
  if (*n) return cudaSuccess;
  auto kern = muon_cluster_kernel<MP, BF16, V>;
  static DeviceOnce once;
  if ((e = set_smem_limit_once(kern, kWholeSm, once)) != cudaSuccess) return e;
  cudaLaunchConfig_t q = {};
  q.gridDim = dim3(static_cast<unsigned>(ranks));
  q.blockDim = dim3(kThreads);
  q.dynamicSmemBytes = whole ? kWholeSm : kHalfSm;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  q.attrs = attr;
  q.numAttrs = 1;
  if ((e = cudaOccupancyMaxActiveClusters(n, kern, &q)) != cudaSuccess) return e;
  if (*n < 1) return cudaErrorInvalidConfiguration;
  at->store(*n, std::memory_order_release);
  return cudaSuccess;
}

// CTAs of a cluster, and their shared memory: the number that takes the least
// time, by the rounds of resident clusters, each as long as its longest matrix:
// 10, 14 or 40 us for the m x m steps and the exchanges, 5, 7 or 12 us a tile.  (These were
// measured element by element on the CUDA cores; the present kernels take 7.5, 17 or 47 and 3.3, 4.9
// or 8.  Of 28 batches of 1 to 1000 matrices, the sizes chosen so are within 3 % of the best of
// all eight.)  The steps of 64 rows fill an SM's pipes, so that two CTAs on one take half
// as long again: 100 of 64 x 1000 237 us in clusters of four, 325 in clusters of eight, two an SM; 18 of them
// in clusters of six 69, of eight 98.
struct ClusterPlan {
  int ranks, smem;
};
template <int MP, bool BF16, int V>
cudaError_t cluster_plan(const moe_muon_tensor* t, const Batch& b, int64_t most_tiles, ClusterPlan* best) {
  constexpr int64_t kOwn = MP == 16 ? 10 : MP == 32 ? 14 : 40, kTile = MP == 16 ? 5 : MP == 32 ? 7 : 12;
  *best = {0, 0};
  int64_t least = 0;
  for (int ranks = 1; ranks <= kMaxRanks; ++ranks) {
    auto tiles = [&](int64_t all) { return (all + ranks - 1) / ranks; };
    const int64_t smem = cluster_smem<MP>(tiles(most_tiles));
    if (smem > kWholeSm || (ranks > 1 && ranks > most_tiles)) continue;
    int n, apart;   // apart: with an SM to each CTA
    cudaError_t e = resident_clusters<MP, BF16, V>(ranks, smem > kHalfSm, &n);
    if (e == cudaSuccess) e = resident_clusters<MP, BF16, V>(ranks, true, &apart);
    if (e != cudaSuccess) return e;
    const bool crowded = MP == 64 && smem <= kHalfSm && b.matrices > apart;
    int64_t time = 0, left = 0;   // left: places of the round in the making, whose longest is `longest`
    int64_t longest = 0;
    for (int i = 0; i < b.count; ++i) {
      const int64_t each = kOwn + kTile * tiles(tiles_of(t[b.index[i]]));
      int64_t count = t[b.index[i]].count;
      const int64_t joined = std::min(count, left);
      if (joined) longest = std::max(longest, each);
      count -= joined;
      left -= joined;
      if (count) {
        const int64_t rounds = (count + n - 1) / n;
        time += longest + (rounds - 1) * each;
        longest = each;
        left = rounds * n - count;
      }
    }
    time += longest;
    if (crowded) time += time / 2;
    if (best->ranks && time >= least) continue;
    *best = {ranks, static_cast<int>(smem)};
    least = time;
  }
  return cudaSuccess;
}

struct SmallWs {
  size_t shares, q, total;
};
SmallWs small_ws(const Batch& b, int mp) {
  SmallWs w;
  w.shares = 0;
  w.q = ws_up(4ull * b.blocks * mp * mp);
  w.total = w.q + ws_up(4ull * b.matrices * mp * mp);
  return w;
}

template <int MP, bool BF16, int V>
int32_t run_batch(const moe_muon_tensor* t, const Batch& b, const moe_muon_options* o, uint8_t* ws,
                  cudaStream_t st) {
  Table tab = {};
  tab.count = b.count;
  tab.decay = muon_decay(o);
  int64_t blocks = 0, matrices = 0;
  for (int i = 0; i < b.count; ++i) {
    const moe_muon_tensor& x = t[b.index[i]];
    Entry& e = tab.e[i];
    e.mo = {x.grad, x.momentum, o->grad_scale, static_cast<float>(o->momentum),
            static_cast<float>(1.0 - o->momentum), o->grad_dtype == MOE_DTYPE_BF16, o->nesterov};
    e.p = x.param;
    e.copy = static_cast<__nv_bfloat16*>(x.param_bf16);
    e.step = static_cast<float>(muon_step(o, x));
    e.m = std::min(x.rows, x.cols);
    e.n = std::max(x.rows, x.cols);
    e.tall = x.rows > x.cols;
    e.blocks = static_cast<int32_t>(blocks_of(x, b));
    e.first_block = static_cast<int32_t>(blocks);
    e.first_matrix = static_cast<int32_t>(matrices);
    blocks += x.count * static_cast<int64_t>(e.blocks);
    matrices += x.count;
  }
  const float a = static_cast<float>(o->coefficients[0]), c1 = static_cast<float>(o->coefficients[1]),
              c2 = static_cast<float>(o->coefficients[2]), eps = static_cast<float>(o->eps);
  if (b.resident) {
    int64_t most_tiles = 1;
    for (int i = 0; i < b.count; ++i) most_tiles = std::max(most_tiles, tiles_of(t[b.index[i]]));
    ClusterPlan plan;
    MOE_CUDA((cluster_plan<MP, BF16, V>(t, b, most_tiles, &plan)));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(b.matrices * plan.ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = plan.smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(plan.ranks);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const Schedule sc = {o->ns_steps, a, c1, c2, eps};
    MOE_CUDA(cudaLaunchKernelEx(&cfg, muon_cluster_kernel<MP, BF16, V>, tab, sc));
    return MOE_OK;
  }
  const SmallWs w = small_ws(b, MP);
  float* shares = reinterpret_cast<float*>(ws + w.shares);
  float* qs = reinterpret_cast<float*>(ws + w.q);
  const dim3 grid(static_cast<unsigned>(blocks)), block(kThreads);
  constexpr int kSteps = 3 * MP * Cfg<MP>::LDM * 4;
  static DeviceOnce once_first, once_next;
  MOE_CUDA(set_smem_limit_once(muon_small_steps_kernel<MP, true>, kSteps, once_first));
  MOE_CUDA(set_smem_limit_once(muon_small_steps_kernel<MP, false>, kSteps, once_next));
  for (int done = 0; done < o->ns_steps; done += kMuonPartSteps) {
    const int n = std::min(kMuonPartSteps, o->ns_steps - done);
    const dim3 each(static_cast<unsigned>(matrices));
    if (done == 0) {
      MOE_CUDA(launch_pdl(muon_small_gram_kernel<MP, true, BF16, V>, grid, block, 0, st, tab,
                          static_cast<const float*>(qs), shares));
      MOE_CUDA(launch_pdl(muon_small_steps_kernel<MP, true>, each, block, kSteps, st, tab,
                          static_cast<const float*>(shares), qs, n, a, c1, c2, eps));
    } else {
      MOE_CUDA(launch_pdl(muon_small_gram_kernel<MP, false, BF16, V>, grid, block, 0, st, tab,
                          static_cast<const float*>(qs), shares));
      MOE_CUDA(launch_pdl(muon_small_steps_kernel<MP, false>, each, block, kSteps, st, tab,
                          static_cast<const float*>(shares), qs, n, a, c1, c2, eps));
    }
  }
  MOE_CUDA(launch_pdl(muon_small_apply_kernel<MP, BF16, V>, grid, block, 0, st, tab, static_cast<const float*>(qs)));
  return MOE_OK;
}

}  // namespace

bool muon_is_small(const moe_muon_tensor& t) { return std::min(t.rows, t.cols) <= kMuonSmall; }

size_t muon_small_ws(const moe_muon_tensor* t, int32_t count) {
  size_t need = 0;
  each_batch(t, count, [&](int mp, const Batch& b) -> int32_t {
    if (!b.resident) need = std::max(need, small_ws(b, mp).total);
    return MOE_OK;
  });
  return need;
}

int32_t muon_small_step(const moe_muon_tensor* t, int32_t count, const moe_muon_options* o, uint8_t* ws,
                        cudaStream_t st) {
  const bool bf16 = o->grad_dtype == MOE_DTYPE_BF16;
  return each_batch(t, count, [&](int mp, const Batch& b) -> int32_t {
    Batch part[2] = {b, b};   // element by element, in packs
    part[0].count = part[1].count = 0;
    part[0].matrices = part[1].matrices = 0;
    int64_t packed = 0;
    for (int i = 0; i < b.count; ++i) {
      const moe_muon_tensor& x = t[b.index[i]];
      const bool fours = in_fours(x, bf16);
      Batch& to = part[fours];
      to.index[to.count++] = b.index[i];
      to.matrices += x.count;
      if (fours) packed += x.count * tiles_of(x);
    }
    auto run = [&](auto size, const Batch& b, bool four) -> int32_t {
      constexpr int MP = decltype(size)::value;
      return bf16 ? (four ? run_batch<MP, true, 4>(t, b, o, ws, st) : run_batch<MP, true, 1>(t, b, o, ws, st))
                  : (four ? run_batch<MP, false, 4>(t, b, o, ws, st) : run_batch<MP, false, 1>(t, b, o, ws, st));
    };
    auto send = [&](const Batch& b, bool four) -> int32_t {
      return mp == 16   ? run(std::integral_constant<int, 16>(), b, four)
             : mp == 32 ? run(std::integral_constant<int, 32>(), b, four)
                        : run(std::integral_constant<int, 64>(), b, four);
    };
    if (!part[0].count || !part[1].count || !b.resident || mp > 16 || packed < kPackedTiles) return send(b, !part[0].count);
    MOE_TRY(send(part[1], true));
    return send(part[0], false);
  });
}

}  // namespace moe
