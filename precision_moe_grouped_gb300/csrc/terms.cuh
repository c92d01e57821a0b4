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

// The producer of one operand (see dense::produce): both terms of a stage.
template <bool IS_A, class L>
__device__ __forceinline__ void produce(const Maps& maps, const L& l, uint8_t* smem, uint64_t* full, uint64_t* empty,
                                        uint32_t rank, int pair, int pairs, volatile int32_t* abort_flag) {
  constexpr int kSlot = IS_A ? kABytes : kBBytes;   // of one term
  const int lane = threadIdx.x & 31, units = num_units(l);
  const uint32_t full0 = cluster_addr(full, 0);
  uint8_t* const slots = smem + (IS_A ? 0 : 2 * kABytes);
  asm volatile("fence.proxy.async.global;" ::: "memory");
  uint32_t stage = 0, phase = 0;
  bool ok = true, issued = false;
  for (int t = pair; ok && t < units; t += pairs) {
    const Unit x = find_unit(l, t);
    const Problem& p = l.p[x.o.p];
    const Operand& o = IS_A ? p.a : p.b;
    const int at = IS_A ? x.o.i * kTile + static_cast<int>(rank) * 128
                        : x.col + static_cast<int>(rank) * (x.bn >> 1);
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
      if (!mbar_poll_warp(empty + stage, phase ^ 1u, l.timeout_ns, l.status, kDevTimeout, abort_flag)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        uint8_t* dst = slots + stage * kStageBytes;
        const uint32_t bar = full0 + 8 * stage;
        if (rank == 0) mbar_arrive_expect_tx(full + stage, bytes);
        tma_load_2d_pair(dst, m, cx, cy + hi, bar);
        tma_load_2d_pair(dst + kSlot, m, cx, cy + lo, bar);
        if (rows == 128) {
          tma_load_2d_pair(dst + 8192, m, cx + dx, cy + dy + hi, bar);
          tma_load_2d_pair(dst + kSlot + 8192, m, cx + dx, cy + dy + lo, bar);
        }
      }
      issued = true;
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
  // rank 0: every copy of both CTAs has landed before either may leave
  if (rank == 0 && issued) {
    int32_t none = 0;
    for (int s = 0; s < kStages; ++s) {
      const uint32_t par = s < static_cast<int>(stage) ? phase : phase ^ 1u;
      mbar_wait_warp(full + s, par, l.timeout_ns, l.status, kDevTimeout, &none);
    }
  }
}

// Epi: struct Args; static run(args, tile, warp, col, n, maps, sums): the warp's
// row (lane), columns [col, col + n) in sums[0 .. n), n 128, 64 or 32; and static
// ahead(args, tile, warp, col, n), called before the unit's products.
template <class Epi>
__global__ void __launch_bounds__(kThreads, 1)
    terms_kernel(const __grid_constant__ Maps maps,
                 const __grid_constant__ Launch<typename Epi::Args> l) {
  extern __shared__ uint8_t smem_raw[];
  // the same offset in both CTAs, which the pair's descriptors rely on
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(smem + kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int units = num_units(l);
  const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + s, 2);   // rank 0's producers, plus the bytes of both CTAs
      mbar_init(empty + s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull + a, 1);
      mbar_init(tempty + a, 2 * kNumEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
  if (warp == 3 && lane > 0 && lane < l.maps) prefetch_tmap(&maps.m[lane]);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  if (warp == 0) {
    produce<true>(maps, l, smem, full, empty, rank, pair, pairs, abort_flag);
  } else if (warp == 2) {
    produce<false>(maps, l, smem, full, empty, rank, pair, pairs, abort_flag);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0) {
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      int acc = 0;
      uint32_t round = 0;
      for (int t = pair; ok && t < units; t += pairs) {
        const Unit x = find_unit(l, t);
        const Tile& o = x.o;
        const Problem& p = l.p[o.p];
        const int k0 = o.s * p.kb_split, k1 = min(p.kb, k0 + p.kb_split);
        for (int kb = k0; ok && kb < k1; kb += kPiece) {
          const int n = min(kPiece, k1 - kb);
          if (!mbar_poll_warp(tempty + acc, round ^ 1u, l.timeout_ns, l.status, kDevTimeout, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + static_cast<uint32_t>(acc * 256);
          for (int k = 0; k < n; ++k) {
            if (!mbar_poll_warp(full + stage, phase, l.timeout_ns, l.status, kDevTimeout, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const bool amn = mn_at(p.a, o.i, kb + k), bmn = mn_at(p.b, o.j, kb + k);
            const uint64_t a_step = amn ? 2048 >> 4 : 32 >> 4, b_step = bmn ? 2048 >> 4 : 32 >> 4;
            const uint32_t at = smem_u32(smem + stage * kStageBytes);
            const uint64_t a = smem_desc(at, amn ? 8192 : 0, 1024, 2);
            const uint64_t b = smem_desc(at + 2 * kABytes, bmn ? 8192 : 0, 1024, 2);
            const uint32_t idesc = dense::idesc_f16(false, amn, bmn, x.bn);
            // the small products first: they lose nothing to a sum that is still small
            dense::mma_quad_warp(d, a + (kABytes >> 4), b, a_step, b_step, idesc, k > 0 ? 1u : 0u);
            dense::mma_quad_warp(d, a, b + (kBBytes >> 4), a_step, b_step, idesc, 1u);
            dense::mma_quad_warp(d, a, b, a_step, b_step, idesc, 1u);
            tc2_commit_both_warp(empty + stage);
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (ok) tc2_commit_both_warp(tfull + acc);
          round ^= static_cast<uint32_t>(acc);
          acc ^= 1;
        }
      }
      tc2_commit_local_warp(drain);
      int32_t none = 0;
      mbar_wait_warp(drain, 0, l.timeout_ns, l.status, kDevTimeout, &none);
    }
  } else if (warp >= kEpiWarp0) {
    // ------------------------------------------------------------ epilogue
    const int e = warp - kEpiWarp0, quarter = warp & 3;
    const uint32_t release = cluster_addr(tempty, 0);
    EpiWarp w;
    w.box = smem + kOffStage + e * kStageBox;
    w.half = e >> 2;
    w.lane = lane;
    w.tmem = 0;
    int acc = 0;
    uint32_t round = 0;
    bool ok = true;
    for (int t = pair; ok && t < units; t += pairs) {
      const Unit x = find_unit(l, t);
      const Tile& o = x.o;
      const Problem& p = l.p[o.p];
      const int half = x.bn >> 1, col = x.col + w.half * half;
      w.row = o.i * kTile + static_cast<int>(rank) * 128 + 32 * quarter;
      float sums[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) sums[i] = 0.f;
      const int k0 = o.s * p.kb_split, k1 = min(p.kb, k0 + p.kb_split);
      Epi::ahead(l.e[o.p], o, w, col, half);
      for (int kb = k0; kb < k1; kb += kPiece) {
        if (!mbar_poll_warp(tfull + acc, round, l.timeout_ns, l.status, kDevTimeout, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t at = tmem + static_cast<uint32_t>(acc * 256 + w.half * half) +
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
        if (lane == 0) mbar_arrive_cluster(release + static_cast<uint32_t>(8 * acc));
        round ^= static_cast<uint32_t>(acc);
        acc ^= 1;
      }
      if (!ok) break;
      Epi::run(l.e[o.p], o, w, col, half, maps, sums);
    }
    if (lane == 0) dense::box_wait_read();
  }

  tc_fence_before();
  __syncthreads();
  // Neither CTA leaves while the other may still use its memory: rank 0 has
  // drained its MMAs and every copy of both CTAs.
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
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

}  // namespace terms
}  // namespace moe
