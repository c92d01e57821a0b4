// terms.cuh -- dense products of matrices held as two fp16 terms, on CTA pairs:
// D = (A_hi + A_lo)(B_hi + B_lo) without A_lo B_lo, in float.
//
// dense.cuh's tiles, tile list and operand majors; what differs:
// - A stage holds both terms of both operands for a K block of 64 (64 KB a CTA
//   at BN = 256, three stages) and feeds three products, so that each term
//   is loaded once.
// - An MMA aligns its 16 products and the accumulator to the largest of them
//   and cuts each off at 24 bits: a sum of n terms of one sign shrinks by about n 2^-27
//   of itself.  So sums run in pieces of two K blocks, which alternate between
//   the two accumulators; the epilogue warps add the pieces up in registers
//   (rounded to nearest) while the next one runs.
//   Noise of 333 x 1001 through five steps is 1.7e-5 off (4.2e-5 without
//   pieces), 16 x 7168 1.0e-6 (3.9e-5); plain 32-bit arithmetic 2.6e-6, 0.8e-6.
#pragma once

#include "dense.cuh"

namespace moe {
namespace terms {

using dense::EpiWarp;
using dense::kABytes;
using dense::kBBytes;
using dense::kBK;
using dense::kEpiWarp0;
using dense::kNumEpiWarps;
using dense::kStageBox;
using dense::kThreads;
using dense::kTile;
using dense::Tile;

constexpr int kMaxMaps = 32, kMaxProblems = 8;
using Maps = dense::MapList<kMaxMaps>;
constexpr int kStages = 3;
constexpr int kPiece = 2;     // K blocks of a piece
constexpr int kStageBytes = 2 * (kABytes + kBBytes);   // A hi, A lo, B hi, B lo
constexpr int kOffStage = kStages * kStageBytes;
constexpr int kOffBar = kOffStage + kNumEpiWarps * kStageBox;
constexpr int kOffMisc = kOffBar + 8 * (2 * kStages + 4 + 1);
constexpr int kSmemBytes = kOffMisc + 16 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget exceeded");

// An operand of a product.  A symmetric matrix is stored by its 256 x 256 blocks
// on and above the diagonal only: a K block right of its rows' block is read
// K-major, one left of it MN-major from the block across the diagonal.  With
// `diag` the diagonal blocks come from a matrix of their own ([rows][256], block
// by block).
// Boxes are 64 x 64 for either major.
struct Operand {
  int32_t map;
  int32_t hi, lo;         // rows of the first matrix's terms
  int32_t batch;          // rows between matrices
  int32_t mn, sym, diag;  // MN-major throughout; symmetric; map of the diagonal blocks, or 0 for none
  int32_t turned;         // symmetric, diagonal blocks read transposed (they are symmetric but for roundings)
};
struct Problem {
  Operand a, b;
  int32_t tiles_m, tiles_n;   // of 256 x 256
  int32_t upper;              // symmetric D: only tiles on and above the diagonal
  int32_t per_matrix, batch, splits;
  int32_t kb, kb_split;
  int32_t first_tile;
};
// The launch's tiles of 256 x 256 are taken whole up to `whole`; each of the rest
// is `cut` units of 256 / cut columns, where those all fit into the last round of
// the pairs.
template <typename Args>
struct Launch {
  static constexpr int kMost = kMaxProblems;
  Problem p[kMaxProblems];
  Args e[kMaxProblems];
  int32_t problems, tiles, whole, cut, maps;
  int32_t* status;
  uint64_t timeout_ns;
};

// A unit: tile o, columns [col, col + bn).
struct Unit {
  Tile o;
  int32_t bn, col;
};
template <typename L>
__device__ __forceinline__ int num_units(const L& l) {
  return l.whole + l.cut * (l.tiles - l.whole);
}
template <typename L>
__device__ __forceinline__ Unit find_unit(const L& l, int u) {
  const int rest = u - l.whole;
  Unit x;
  const int tile = rest < 0 ? u : l.whole + rest / l.cut;
  x.bn = rest < 0 ? 256 : 256 / l.cut;
  x.o = dense::find_tile(l, tile);
  x.col = x.o.j * 256 + (rest < 0 ? 0 : (rest - (tile - l.whole) * l.cut) * x.bn);
  return x;
}

// Whether operand o's K block kb is read MN-major by a tile at row block tr.
__device__ __forceinline__ bool mn_at(const Operand& o, int tr, int kb) {
  return o.mn || (o.sym && (kb >> 2) < tr + o.turned);
}

// What the roles of a CTA share.
struct Bars {
  uint64_t *full, *empty, *tfull, *tempty;
  uint32_t rank, base;   // in the pair; the pair's first CTA in the cluster
  uint64_t timeout_ns;
  int32_t* status;
  volatile int32_t* abort_flag;
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) const {
    return mbar_poll_warp(bar, parity, timeout_ns, status, kDevTimeout, abort_flag);
  }
};
// A role's place in the ring of slots.
struct Ring {
  uint32_t stage = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
};
// ... and among the two accumulators.
struct Turn {
  int acc = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void next() {
    round ^= static_cast<uint32_t>(acc);
    acc ^= 1;
  }
};

// The producer of one operand (see dense::produce): both terms of a unit's
// stages.  False: a wait ran out.
template <bool IS_A, class M>
__device__ __forceinline__ bool produce(const M& maps, const Problem& p, const Unit& x, uint8_t* smem, const Bars& b,
                                        uint32_t full0, Ring& r, bool& issued) {
  constexpr int kSlot = IS_A ? kABytes : kBBytes;   // of one term
  const int lane = threadIdx.x & 31;
  uint8_t* const slots = smem + (IS_A ? 0 : 2 * kABytes);
  const Operand& o = IS_A ? p.a : p.b;
  const int at = IS_A ? x.o.i * kTile + static_cast<int>(b.rank) * 128
                      : x.col + static_cast<int>(b.rank) * (x.bn >> 1);
  // (of a box's 64 rows, units of 64 columns use 32)
  const int tr = IS_A ? x.o.i : x.o.j, rows = IS_A || x.bn == 256 ? 128 : 64;
  const uint32_t bytes = 4u * static_cast<uint32_t>(rows) * 128u;   // both terms, both CTAs
  const int hi = o.hi + x.o.z * o.batch, lo = o.lo + x.o.z * o.batch;
  const int k0 = x.o.s * p.kb_split, k1 = min(p.kb, k0 + p.kb_split);
  for (int kb = k0; kb < k1; ++kb) {
    const bool mn = mn_at(o, tr, kb), diag = o.diag && (kb >> 2) == tr;
    const CUtensorMap* m = &maps.m[diag ? o.diag : o.map];
    const int k = (diag ? kb & 3 : kb) * kBK;
    const int cx = mn ? at : k, cy = mn ? k : at, dx = mn ? 64 : 0, dy = mn ? 0 : 64;
    if (!b.wait(b.empty + r.stage, r.phase ^ 1u)) return false;
    if (lane == 0) {
      uint8_t* dst = slots + r.stage * kStageBytes;
      const uint32_t bar = full0 + 8 * r.stage;
      if (b.rank == 0) mbar_arrive_expect_tx(b.full + r.stage, bytes);
      tma_load_2d_pair(dst, m, cx, cy + hi, bar);
      tma_load_2d_pair(dst + kSlot, m, cx, cy + lo, bar);
      if (rows == 128) {
        tma_load_2d_pair(dst + 8192, m, cx + dx, cy + dy + hi, bar);
        tma_load_2d_pair(dst + kSlot + 8192, m, cx + dx, cy + dy + lo, bar);
      }
    }
    issued = true;
    r.next();
  }
  return true;
}
// Rank 0's, at its end: every copy of both CTAs has landed before either may leave.
__device__ __forceinline__ void drain_copies(const Bars& b, const Ring& r) {
  int32_t none = 0;
  for (uint32_t s = 0; s < kStages; ++s)
    mbar_wait_warp(b.full + s, s < r.stage ? r.phase : r.phase ^ 1u, b.timeout_ns, b.status, kDevTimeout, &none);
}

// A unit's products, by pieces.  False: a wait ran out.
__device__ __forceinline__ bool multiply(const Problem& p, const Unit& x, const uint8_t* smem, const Bars& b,
                                         uint32_t tmem, Ring& r, Turn& turn) {
  const Tile& o = x.o;
  const uint16_t both = static_cast<uint16_t>(3u << b.base);
  const int k0 = o.s * p.kb_split, k1 = min(p.kb, k0 + p.kb_split);
  for (int kb = k0; kb < k1; kb += kPiece) {
    const int n = min(kPiece, k1 - kb);
    if (!b.wait(b.tempty + turn.acc, turn.round ^ 1u)) return false;
    tc_fence_after();
    const uint32_t d = tmem + static_cast<uint32_t>(turn.acc * 256);
    for (int k = 0; k < n; ++k) {
      if (!b.wait(b.full + r.stage, r.phase)) return false;
      tc_fence_after();
      const bool amn = mn_at(p.a, o.i, kb + k), bmn = mn_at(p.b, o.j, kb + k);
      const uint64_t a_step = amn ? 2048 >> 4 : 32 >> 4, b_step = bmn ? 2048 >> 4 : 32 >> 4;
      const uint32_t at = smem_u32(smem + r.stage * kStageBytes);
      const uint64_t ad = smem_desc(at, amn ? 8192 : 0, 1024, 2);
      const uint64_t bd = smem_desc(at + 2 * kABytes, bmn ? 8192 : 0, 1024, 2);
      const uint32_t idesc = dense::idesc_f16(false, amn, bmn, x.bn);
      // the small products first: they lose nothing to a sum that is still small
      dense::mma_quad_warp(d, ad + (kABytes >> 4), bd, a_step, b_step, idesc, k > 0 ? 1u : 0u);
      dense::mma_quad_warp(d, ad, bd + (kBBytes >> 4), a_step, b_step, idesc, 1u);
      dense::mma_quad_warp(d, ad, bd, a_step, b_step, idesc, 1u);
      tc2_commit_both_warp(b.empty + r.stage, both);
      r.next();
    }
    tc2_commit_both_warp(b.tfull + turn.acc, both);
    turn.next();
  }
  return true;
}
// At the issuer's end: no MMA may still run when TMEM is freed.
__device__ __forceinline__ void drain_products(uint64_t* drain, const Bars& b) {
  tc2_commit_local_warp(drain);
  int32_t none = 0;
  mbar_wait_warp(drain, 0, b.timeout_ns, b.status, kDevTimeout, &none);
}

// A unit's pieces added up, and its epilogue.  False: a wait ran out.
template <class Epi, class M>
__device__ __forceinline__ bool finish(const M& maps, const typename Epi::Args& e, const Problem& p, const Unit& x,
                                       const Bars& b, uint32_t release, uint32_t tmem, EpiWarp& w, Turn& turn) {
  const Tile& o = x.o;
  const int quarter = (threadIdx.x >> 5) & 3;
  const int half = x.bn >> 1, col = x.col + w.half * half;
  w.row = o.i * kTile + static_cast<int>(b.rank) * 128 + 32 * quarter;
  float sums[128];
#pragma unroll
  for (int i = 0; i < 128; ++i) sums[i] = 0.f;
  const int k0 = o.s * p.kb_split, k1 = min(p.kb, k0 + p.kb_split);
  Epi::ahead(e, o, w, col, half);
  for (int kb = k0; kb < k1; kb += kPiece) {
    if (!b.wait(b.tfull + turn.acc, turn.round)) return false;
    tc_fence_after();
    const uint32_t at = tmem + static_cast<uint32_t>(turn.acc * 256 + w.half * half) +
                        (static_cast<uint32_t>(32 * quarter) << 16);
#pragma unroll
    for (int c = 0; c < 128; c += 32) {
      if (c < half) {
        uint32_t v[32];
        dense::tmem_ld_x32(at + c, v);
        dense::tmem_wait(v);
#pragma unroll
        for (int i = 0; i < 32; ++i) sums[c + i] += __uint_as_float(v[i]);
      }
    }
    tc_fence_before();
    __syncwarp();
    if (w.lane == 0) mbar_arrive_cluster(release + static_cast<uint32_t>(8 * turn.acc));
    turn.next();
  }
  Epi::run(e, o, w, col, half, maps, sums);
  return true;
}

// Epi: struct Args; static run(args, tile, warp, col, n, maps, sums): the warp's
// row (lane), columns [col, col + n) in sums[0 .. n), n 128, 64 or 32; and static
// ahead(args, tile, warp, col, n), called before the unit's products.
// Shared memory, barriers and tensor memory of a CTA, and its place.
struct Setup {
  uint8_t* smem;
  Bars b;
  uint64_t* drain;
  uint32_t tmem;

  __device__ __forceinline__ Setup(uint8_t* smem_raw, uint64_t timeout_ns, int32_t* status, int maps,
                                   const CUtensorMap* map) {
    // the same offset in both CTAs, which the pair's descriptors rely on
    smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    b.full = reinterpret_cast<uint64_t*>(smem + kOffBar);
    b.empty = b.full + kStages;
    b.tfull = b.empty + kStages;
    b.tempty = b.tfull + 2;
    drain = b.tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
    b.abort_flag = reinterpret_cast<volatile int32_t*>(smem + kOffMisc + 4);
    const uint32_t in_cluster = cluster_rank();
    b.rank = in_cluster & 1u;
    b.base = in_cluster & ~1u;
    b.timeout_ns = timeout_ns;
    b.status = status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
      for (int s = 0; s < kStages; ++s) {
        mbar_init(b.full + s, 2);   // rank 0's producers, plus the bytes of both CTAs
        mbar_init(b.empty + s, 1);
      }
      for (int a = 0; a < 2; ++a) {
        mbar_init(b.tfull + a, 1);
        mbar_init(b.tempty + a, 2 * kNumEpiWarps);
      }
      mbar_init(drain, 1);
      *b.abort_flag = 0;
      fence_mbar_init();
    }
    if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
    if (warp == 3) {
      for (int i = 1 + lane; i < maps; i += 32) prefetch_tmap(map + i);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    tmem = *tmem_slot;
  }
  __device__ __forceinline__ EpiWarp epi_warp() const {
    const int e = static_cast<int>(threadIdx.x >> 5) - kEpiWarp0;
    EpiWarp w;
    w.box = smem + kOffStage + e * kStageBox;
    w.half = e >> 2;
    w.lane = threadIdx.x & 31;
    w.tmem = 0;
    return w;
  }
  __device__ __forceinline__ void leave() const {
    tc_fence_before();
    __syncthreads();
    // Neither CTA leaves while the other may still use its memory: rank 0 has
    // drained its MMAs and every copy of both CTAs.
    cluster_sync_all();
    if (threadIdx.x >> 5 == 1) {
      tc_fence_after();
      tmem_dealloc_pair(tmem, 512);
    }
  }
};

template <class Epi>
__global__ void __launch_bounds__(kThreads, 1)
    terms_kernel(const __grid_constant__ Maps maps,
                 const __grid_constant__ Launch<typename Epi::Args> l) {
  extern __shared__ uint8_t smem_raw[];
  const Setup c(smem_raw, l.timeout_ns, l.status, l.maps, maps.m);
  const Bars& b = c.b;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int units = num_units(l);
  const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
  griddep_wait();
  griddep_launch_dependents();

  if (warp == 0 || warp == 2) {
    asm volatile("fence.proxy.async.global;" ::: "memory");
    const uint32_t full0 = cluster_addr(b.full, 0);
    Ring r;
    bool ok = true, issued = false;
    for (int t = pair; ok && t < units; t += pairs) {
      const Unit x = find_unit(l, t);
      const Problem& p = l.p[x.o.p];
      ok = warp == 0 ? produce<true>(maps, p, x, c.smem, b, full0, r, issued)
                     : produce<false>(maps, p, x, c.smem, b, full0, r, issued);
    }
    if (b.rank == 0 && issued) drain_copies(b, r);
  } else if (warp == 1) {
    if (b.rank == 0) {
      Ring r;
      Turn turn;
      bool ok = true;
      for (int t = pair; ok && t < units; t += pairs) {
        const Unit x = find_unit(l, t);
        ok = multiply(l.p[x.o.p], x, c.smem, b, c.tmem, r, turn);
      }
      drain_products(c.drain, b);
    }
  } else if (warp >= kEpiWarp0) {
    const uint32_t release = cluster_addr(b.tempty, 0);
    EpiWarp w = c.epi_warp();
    Turn turn;
    bool ok = true;
    for (int t = pair; ok && t < units; t += pairs) {
      const Unit x = find_unit(l, t);
      ok = finish<Epi>(maps, l.e[x.o.p], l.p[x.o.p], x, b, release, c.tmem, w, turn);
    }
    if (lane == 0) dense::box_wait_read();
  }
  c.leave();
}

// Phases of symmetric products [mp, mp], mp <= 512, each of which reads what the
// one before stored: a cluster takes a matrix, its pairs units of 64 columns of
// the tiles on and above the diagonal, and the cluster's barrier stands between
// two phases.  A phase of one 256 x 256 product takes some 6 us (2 until the last of
// its 128 KB a CTA has come from L2, 1 of MMAs, 2 of epilogue and stores, the
// barrier), 7.6 as a launch of its own, whose exit and the next one's grid wait
// come on top.
constexpr int kMaxPhases = 8, kChainGroups = 4;   // three steps; a group's six matrices, read and stored
constexpr int kChainMaps = 12 * kChainGroups + 1, kChainProblems = 9 * kChainGroups;
using ChainMaps = dense::MapList<kChainMaps>;
template <typename Args>
struct Chain {
  Problem p[kChainProblems];   // by phase; of a phase, as many a group, by group
  Args e[kChainProblems];
  int32_t problems, maps;
  int32_t phases, end[kMaxPhases];                 // of a phase's problems
  int32_t groups, mp[kChainGroups], first[kChainGroups];   // a group's first matrix of the launch
  int32_t* status;
  uint64_t timeout_ns;
};

template <class Epi>
__global__ void __launch_bounds__(kThreads, 1)
    chain_kernel(const __grid_constant__ ChainMaps maps, const __grid_constant__ Chain<typename Epi::Args> l) {
  extern __shared__ uint8_t smem_raw[];
  const Setup c(smem_raw, l.timeout_ns, l.status, l.maps, maps.m);
  const Bars& b = c.b;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int size = static_cast<int>(cluster_size()), pairs = size >> 1;
  const int pair = static_cast<int>(b.base >> 1), matrix = static_cast<int>(blockIdx.x) / size;
  int g = 0;
  while (g + 1 < l.groups && matrix >= l.first[g + 1]) ++g;
  const int row0 = l.mp[g] / 64, each = row0 + max(0, row0 - 4);   // units of a problem: of its first row of tiles, all
  Unit x;
  x.bn = 64;
  x.o.z = matrix - l.first[g];
  x.o.s = 0;
  const uint32_t full0 = cluster_addr(b.full, b.base), release = cluster_addr(b.tempty, b.base);
  EpiWarp w = c.epi_warp();
  Ring r;
  Turn turn;
  bool ok = true, issued = false;
  griddep_wait();
  griddep_launch_dependents();

  for (int phase = 0; phase < l.phases; ++phase) {
    const int from = phase ? l.end[phase - 1] : 0, per = (l.end[phase] - from) / l.groups;
    if (warp == 0 || warp == 2) asm volatile("fence.proxy.async.global;" ::: "memory");
    for (int u = pair; ok && u < per * each; u += pairs) {
      const int q = u / each, v = u - q * each;
      x.o.p = from + g * per + q;
      x.o.i = v >= row0;
      x.col = 64 * (v < row0 ? v : v - row0 + 4);
      x.o.j = x.col >> 8;
      const Problem& p = l.p[x.o.p];
      if (warp == 0) ok = produce<true>(maps, p, x, c.smem, b, full0, r, issued);
      else if (warp == 2) ok = produce<false>(maps, p, x, c.smem, b, full0, r, issued);
      else if (warp == 1) ok = b.rank || multiply(p, x, c.smem, b, c.tmem, r, turn);
      else if (warp >= kEpiWarp0) ok = finish<Epi>(maps, l.e[x.o.p], p, x, b, release, c.tmem, w, turn);
    }
    if (warp >= kEpiWarp0) {   // the phase's matrices are written
      if (lane == 0) {
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        asm volatile("fence.proxy.async.global;" ::: "memory");
      }
    }
    __syncwarp();
    cluster_sync_all();
  }
  if (b.rank == 0) {
    if ((warp == 0 || warp == 2) && issued) drain_copies(b, r);
    if (warp == 1) drain_products(c.drain, b);
  }
  c.leave();
}

template <class Epi>
cudaError_t resident_pairs(int num_sms, int* pairs) {
  static DeviceOnce cache;
  return dense::resident_pairs(terms_kernel<Epi>, kSmemBytes, cache, num_sms, pairs);
}
// The last round is cut where all of its parts fit into one: a unit of 128 columns
// takes about 0.7 of the time of a whole tile, one of 64 about half.
template <class Epi>
cudaError_t launch(const Maps& maps, Launch<typename Epi::Args>& l, int pairs, cudaStream_t s) {
  int tiles = 0;
  for (int i = 0; i < l.problems; ++i) tiles += l.p[i].per_matrix * l.p[i].batch * l.p[i].splits;
  const int rest = tiles % pairs;
  l.cut = 4 * rest <= pairs ? 4 : 2;
  l.whole = 2 * rest <= pairs ? tiles - rest : tiles;
  return dense::launch(terms_kernel<Epi>, kSmemBytes, maps, l, pairs, s, l.whole + l.cut * (tiles - l.whole));
}

// Clusters of `size` CTAs of the chain that are resident at once.
template <class Epi>
cudaError_t resident_chains(int size, int* clusters) {
  static DeviceOnce table[2];
  cudaError_t e;
  std::atomic<int>* at = device_entry(table[size > 8], &e);
  if (!at) return e;
  if ((*clusters = at->load(std::memory_order_acquire) - 1) >= 0) return cudaSuccess;
  auto kern = chain_kernel<Epi>;
  if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes)) != cudaSuccess ||
      (e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
    return e;
  cudaLaunchConfig_t q = {};
  q.gridDim = dim3(static_cast<unsigned>(size));
  q.blockDim = dim3(kThreads);
  q.dynamicSmemBytes = kSmemBytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(size);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  q.attrs = attr;
  q.numAttrs = 1;
  if ((e = cudaOccupancyMaxActiveClusters(clusters, kern, &q)) != cudaSuccess) return e;
  at->store(*clusters + 1, std::memory_order_release);
  return cudaSuccess;
}
template <class Epi>
cudaError_t launch_chain(const ChainMaps& maps, const Chain<typename Epi::Args>& l, int size, int matrices,
                         cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(size * matrices));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(size);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, chain_kernel<Epi>, maps, l);
}

}  // namespace terms
}  // namespace moe
