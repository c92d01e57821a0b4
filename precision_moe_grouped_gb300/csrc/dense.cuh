// dense.cuh -- dense products of bf16 matrices on CTA pairs, the core of the
// gated feed-forward block (ffn.cu); terms.cuh, on which the orthogonalised update
// (muon.cu) runs, takes its tiles and its building blocks from here.
//
// One persistent launch runs a list of problems D = A B, each D cut into tiles
// of 256 x BN (BN = 64 to 256): a CTA pair takes a tile, rank r holds its rows
// 128 r .. 128 r + 127 in its tensor memory (tcgen05.mma.cta_group::2, M = 256,
// both operands from shared memory, float accumulators).
// Operands are K-major ([rows, K], K contiguous) or MN-major ([K, rows], rows
// contiguous); the TMA boxes and the descriptors differ, the loop does not, so
// no operand is ever transposed in memory.
//
// Per K block of 64 a CTA stages its 128 rows of A and its half of B (16 +
// 16 KB at BN = 256); six stages, or up to nine smaller ones, keep 192 KB in
// flight.  Two accumulators of 256 columns let the epilogue of a tile run under
// the next one's products.
//   warps 0, 2: TMA producers of A, B   warp 1: MMA issuer (rank 0), TMEM
//   warps 4-11: epilogue, two per lane quarter, each with half of the columns
// One warp an operand: a single producer's instructions for both stood between a
// freed slot and its refill (8192 tokens of 7168 x 2048: 521 us against 463).
// All waits are bounded (ptx.cuh); they sleep, as polling ones cost the issuer
// slots (489 against 481).
//
// Large products are bound by the tensor pipe and, for more than a few hundred
// us, the power cap: 8192 x 4096 x 7168 runs with the pipe 0.88 busy (250 us, 122
// registers a thread), 8192 x 7168 x 2048 0.75 (144 us); both in turn at
// 1.57-1.60 PFLOP/s, 0.92-0.94 of the library's sustained 1.71.  Small ones by the
// kernel's fixed time: some 7 us of launch, first loads, one tile's epilogue.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_internal.h"
#include "pair.cuh"
#include "ptx.cuh"

namespace moe {
namespace dense {

constexpr int kTile = 256;     // rows of a tile (128 per CTA)
constexpr int kBK = 64;        // K elements of a stage: one 128-byte swizzle row
constexpr int kMaxStages = 9;
constexpr int kMaxMaps = 9;
constexpr int kMaxProblems = 3;
template <int N>
struct MapList {
  CUtensorMap m[N];
};
constexpr int kThreads = 384;
constexpr int kEpiWarp0 = 4, kNumEpiWarps = 8;
constexpr int kABytes = 128 * 128, kBBytes = 128 * 128;   // of a stage, B's at most
constexpr int kOperandBytes = 6 * (kABytes + kBBytes);    // all stages
constexpr int kStageBox = 4096;                           // an epilogue warp's: 32 rows x 128 bytes
constexpr int kOffStage = kOperandBytes;
constexpr int kOffBar = kOffStage + kNumEpiWarps * kStageBox;
constexpr int kNumBars = 2 * kMaxStages + 4 + 1;
constexpr int kOffMisc = kOffBar + 8 * kNumBars;
constexpr int kSmemBytes = kOffMisc + 16 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget exceeded");

using Maps = MapList<kMaxMaps>;

// Tile t of a problem -> (matrix z, split s, tile row i, tile column j).
struct Problem {
  static constexpr int32_t batch = 1, upper = 0;   // (terms.cuh's have several, and symmetric ones)
  int32_t a_map, b_map;        // index into Maps
  int32_t a_mn, b_mn;          // 1: the operand is MN-major
  int32_t bn;                  // 64, 128, 192 or 256
  int32_t b_step;              // columns of D between tiles (bn, or bn / 2 for two halves)
  int32_t b_rank;              // where rank 1's half of B begins, from rank 0's
  int32_t tiles_m, tiles_n;
  int32_t per_matrix;          // tiles of a split
  int32_t splits;
  int32_t kb, kb_split;        // K blocks, of a split's share
  int32_t idesc;
  int32_t first_tile;          // of the launch's list
};

struct Tile {
  int32_t p, z, s, i, j;
};

// An operand that no kernel of the call writes is copied ahead of the grid wait,
// as far as the slots go: the kernel before has passed its own, behind which the
// call's inputs are complete.  Its producer comes to the grid wait before its first
// bounded one, whose limit so covers this kernel's progress alone, however long the
// kernel before still runs.
constexpr int kEarlyA = 1, kEarlyB = 2;

template <typename Args>
struct Launch {
  static constexpr int kMost = kMaxProblems;
  Problem p[kMaxProblems];
  Args e[kMaxProblems];        // the epilogue's arguments
  int32_t problems, tiles, maps;
  int32_t stages, slot;        // slots of the operands, bytes of one
  int32_t early;               // kEarlyA, kEarlyB: that operand is the call's input, and this not its first kernel
  int32_t* status;
  uint64_t timeout_ns;
};

// The tile list's order keeps the operands of the tiles that run together few:
// eight tile rows at a time, column by column.
constexpr int kRasterRows = 8;

template <typename L>
__device__ __forceinline__ Tile find_tile(const L& l, int t) {
  Tile o;
  o.p = 0;
#pragma unroll
  for (int q = 1; q < L::kMost; ++q)
    if (q < l.problems && t >= l.p[q].first_tile) o.p = q;
  const auto& p = l.p[o.p];
  t -= p.first_tile;
  const int zs = t / p.per_matrix;
  t -= zs * p.per_matrix;
  o.z = zs / p.splits;
  o.s = zs - o.z * p.splits;
  if (p.upper) {
    int i = 0;
    while (t >= p.tiles_n - i) {
      t -= p.tiles_n - i;
      ++i;
    }
    o.i = i;
    o.j = i + t;
  } else {
    const int g = t / (kRasterRows * p.tiles_n);
    t -= g * kRasterRows * p.tiles_n;
    const int rows = min(kRasterRows, p.tiles_m - g * kRasterRows);
    o.j = t / rows;
    o.i = g * kRasterRows + t - o.j * rows;
  }
  return o;
}

// fp16 x fp16 or bf16 x bf16 into float, M = 256: types, majors, N, M.
__host__ __device__ constexpr uint32_t idesc_f16(bool bf16, bool a_mn, bool b_mn, int n) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) | ((256u >> 4) << 24);
}

// The four MMAs (K = 16 each) of one stage and the commits that free its slot
// in both CTAs, from one elected lane.  The first MMA starts the accumulator
// when acc0 == 0.
__device__ __forceinline__ void mma_stage_warp(uint32_t d, uint64_t a, uint64_t b, uint64_t a_step,
                                               uint64_t b_step, uint32_t idesc, uint32_t acc0,
                                               uint64_t* empty) {
  asm volatile(
      "{\n\t.reg .pred e, p, q;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.b32 q, %4, %4;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %5, %6, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %7, %8, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %9, %10, %3, q;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%11], %12;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc0), "l"(a + a_step), "l"(b + b_step), "l"(a + 2 * a_step),
      "l"(b + 2 * b_step), "l"(a + 3 * a_step), "l"(b + 3 * b_step), "r"(smem_u32(empty)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// The same four without a commit: one product of a stage that holds several.
__device__ __forceinline__ void mma_quad_warp(uint32_t d, uint64_t a, uint64_t b, uint64_t a_step,
                                              uint64_t b_step, uint32_t idesc, uint32_t acc0) {
  asm volatile(
      "{\n\t.reg .pred e, p, q;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.b32 q, %4, %4;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %5, %6, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %7, %8, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %9, %10, %3, q;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc0), "l"(a + a_step), "l"(b + b_step), "l"(a + 2 * a_step),
      "l"(b + 2 * b_step), "l"(a + 3 * a_step), "l"(b + 3 * b_step)
      : "memory");
}

// 32 lanes x 32 columns: thread i receives lane (quarter * 32 + i).  The
// registers hold the values only after tmem_wait().
__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// Ties the registers to the wait, so that no use moves ahead of it.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_bf16(uint32_t v) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}

// An epilogue warp's staging box: 32 rows of 128 bytes in the 128-byte
// swizzle of the TMA store that empties it.
__device__ __forceinline__ uint4* box_piece(uint8_t* box, int row, int piece) {
  return reinterpret_cast<uint4*>(box + row * 128 + ((piece ^ (row & 7)) << 4));
}
__device__ __forceinline__ void box_store(const CUtensorMap* m, const uint8_t* box, int32_t col,
                                          int32_t row) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(col), "r"(row), "r"(smem_u32(box))
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Before a box is written again: the store that read it has done so.
__device__ __forceinline__ void box_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// What an epilogue warp works on: its 32 rows (first one `row`, this lane's
// `row + lane`) and the columns of its half.
struct EpiWarp {
  uint32_t tmem;     // lane quarter and accumulator included
  uint8_t* box;      // kStageBox bytes of its own
  int32_t row;       // of the tile's matrix
  int32_t half;      // 0 or 1
  int32_t lane;
};

// A slot ring's producer: one warp copies A's share of every stage, another one
// B's, so that neither's instructions stand between a freed slot and its
// refill.  The whole warp runs the loop, one lane issues; a tile's last slot is
// followed by the next tile's first without a pause.
template <bool IS_A, bool EARLY, class L>
__device__ __forceinline__ void produce(const Maps& maps, const L& l, uint8_t* smem, uint64_t* full, uint64_t* empty,
                                        uint32_t rank, int pair, int pairs, volatile int32_t* abort_flag) {
  const int lane = threadIdx.x & 31;
  const uint32_t full0 = cluster_addr(full, 0), stages = static_cast<uint32_t>(l.stages);
  uint8_t* const slots = smem + (IS_A ? 0 : kABytes);
  asm volatile("fence.proxy.async.global;" ::: "memory");   // the kernel before used plain stores
  uint32_t stage = 0, phase = 0;
  bool ok = true, issued = false, ahead = EARLY;   // ahead: of the grid wait, in slots that are free from the start
  for (int t = pair; ok && t < l.tiles; t += pairs) {
    const Tile o = find_tile(l, t);
    const Problem& p = l.p[o.p];
    const int k0 = o.s * p.kb_split, n = min(p.kb, k0 + p.kb_split) - k0;
    const bool mn = IS_A ? p.a_mn : p.b_mn;
    const int at = IS_A ? o.i * kTile + static_cast<int>(rank) * 128
                        : o.j * p.b_step + static_cast<int>(rank) * p.b_rank;
    const int dx = mn ? 0 : kBK, dy = mn ? kBK : 0;
    const bool two = mn && (IS_A || p.bn == 256);   // boxes of 64 columns
    const uint32_t bytes = IS_A ? 2u * kABytes : 128u * static_cast<uint32_t>(p.bn);   // both CTAs'
    const CUtensorMap* m = &maps.m[IS_A ? p.a_map : p.b_map];
    int x = mn ? at : k0 * kBK, y = mn ? k0 * kBK : at;
    for (int k = 0; k < n; ++k, x += dx, y += dy) {
      if (ahead && phase) {
        griddep_wait();
        ahead = false;
      }
      if (!ahead && !mbar_wait_warp(empty + stage, phase ^ 1u, l.timeout_ns, l.status, kDevTimeout, abort_flag)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        uint8_t* dst = slots + stage * static_cast<uint32_t>(l.slot);
        if (rank == 0) mbar_arrive_expect_tx(full + stage, bytes);
        tma_load_2d_pair(dst, m, x, y, full0 + 8 * stage);
        if (two) tma_load_2d_pair(dst + 8192, m, x + 64, y, full0 + 8 * stage);
      }
      issued = true;
      if (++stage == stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
  if (ahead) griddep_wait();
  // Rank 0: every copy of both CTAs has landed before either may leave
  // (bounded, whatever the abort flag says): the last fill of each slot.
  if (rank == 0 && issued) {
    int32_t none = 0;
    for (uint32_t s = 0; s < stages; ++s) {
      // slots below `stage` were last filled in this round of the ring, the others in the one before
      // (a slot never filled has its fresh barrier pass at once)
      const uint32_t par = s < stage ? phase : phase ^ 1u;
      mbar_wait_warp(full + s, par, l.timeout_ns, l.status, kDevTimeout, &none);
    }
  }
}

// Epi: struct Args; static run(args, problem, tile, warp, maps).
template <class Epi>
__global__ void __launch_bounds__(kThreads, 1)
    dense_kernel(const __grid_constant__ Maps maps,
                 const __grid_constant__ Launch<typename Epi::Args> l) {
  extern __shared__ uint8_t smem_raw[];
  // the same offset in both CTAs, which the pair's descriptors rely on
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* empty = full + kMaxStages;
  uint64_t* tfull = empty + kMaxStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(smem + kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
  const uint32_t stages = static_cast<uint32_t>(l.stages), slot = static_cast<uint32_t>(l.slot);

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < stages; ++s) {
      mbar_init(full + s, 2);    // rank 0's producers, plus the bytes of both CTAs
      mbar_init(empty + s, 1);   // the MMA commit
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
  if (warp == 3 && lane < l.maps) prefetch_tmap(&maps.m[lane]);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // (a producer of an early operand reads nothing that a kernel of the call writes)
  const bool early = (warp == 0 && l.early == kEarlyA) || (warp == 2 && l.early == kEarlyB);
  if (!early) {
    griddep_wait();
    griddep_launch_dependents();
  }

  if (warp == 0) {
    if (early) produce<true, true>(maps, l, smem, full, empty, rank, pair, pairs, abort_flag);
    else produce<true, false>(maps, l, smem, full, empty, rank, pair, pairs, abort_flag);
  } else if (warp == 2) {
    if (early) produce<false, true>(maps, l, smem, full, empty, rank, pair, pairs, abort_flag);
    else produce<false, false>(maps, l, smem, full, empty, rank, pair, pairs, abort_flag);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0) {
      const uint32_t a0 = smem_u32(smem), b0 = smem_u32(smem + kABytes);
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      int it = 0;
      for (int t = pair; ok && t < l.tiles; t += pairs, ++it) {
        const Tile o = find_tile(l, t);
        const Problem& p = l.p[o.p];
        const int k0 = o.s * p.kb_split, steps = min(p.kb, k0 + p.kb_split) - k0;
        // MN-major: 64 x 64 boxes of 8 KB side by side, 8 K rows 1024 bytes
        // apart; K-major: rows of 128 bytes, 8 rows 1024 bytes apart.
        const uint64_t ad0 = smem_desc(a0, p.a_mn ? 8192 : 0, 1024, 2);
        const uint64_t bd0 = smem_desc(b0, p.b_mn ? 8192 : 0, 1024, 2);
        const uint64_t a_step = p.a_mn ? 2048 >> 4 : 32 >> 4, b_step = p.b_mn ? 2048 >> 4 : 32 >> 4;
        const int acc = it & 1;
        if (!mbar_wait_warp(tempty + acc, static_cast<uint32_t>((it >> 1) & 1) ^ 1u, l.timeout_ns,
                            l.status, kDevTimeout, abort_flag))
          break;
        asm volatile("fence.acq_rel.cluster;" ::: "memory");
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(acc * 256);
        for (int k = 0; k < steps; ++k) {
          if (!mbar_wait_warp(full + stage, phase, l.timeout_ns, l.status, kDevTimeout, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          mma_stage_warp(d, ad0 + stage * (slot >> 4), bd0 + stage * (slot >> 4), a_step, b_step,
                         static_cast<uint32_t>(p.idesc), k > 0 ? 1u : 0u, empty + stage);
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) tc2_commit_both_warp(tfull + acc);
      }
      // no MMA may still run when TMEM is freed
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
    int it = 0;
    for (int t = pair; t < l.tiles; t += pairs, ++it) {
      const Tile o = find_tile(l, t);
      const int acc = it & 1;
      if (!mbar_wait_warp(tfull + acc, static_cast<uint32_t>((it >> 1) & 1), l.timeout_ns, l.status,
                          kDevTimeout, abort_flag))
        break;
      tc_fence_after();
      w.tmem = tmem + static_cast<uint32_t>(acc * 256) + (static_cast<uint32_t>(32 * quarter) << 16);
      w.row = o.i * kTile + static_cast<int>(rank) * 128 + 32 * quarter;
      Epi::run(l.e[o.p], l.p[o.p], o, w, maps);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(release + static_cast<uint32_t>(8 * acc));
    }
    if (lane == 0) box_wait_read();   // the kernel's end waits for the writes
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

// ---------------------------------------------------------------- host side

// Row-major [rows, cols] matrix of 2- or 4-byte elements, rows ld elements
// apart; the box is box_cols x box_rows in the 128-byte swizzle.
enum class Elem { kBf16, kF16, kF32 };
enum class Swizzle { k128, k64 };
int32_t make_map(CUtensorMap* m, const void* base, Elem type, int64_t rows, int64_t cols, int64_t ld,
                 int box_cols, int box_rows, Swizzle swizzle = Swizzle::k128);

// How a product is cut: columns of a tile, and shares of K where there are too
// few tiles for the pairs.
struct Plan {
  int32_t bn, splits, kb_split;
};

// A GB300's CTA pairs: what a plan, and so a workspace's size, is made for.
constexpr int kPlanPairs = 76;

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles of 128 columns, which take about 0.7 of the time of 256, where they fill
// the last wave better.
inline Plan make_plan(int64_t tiles_m, int64_t cols, int64_t kb) {
  const int64_t t256 = tiles_m * cdiv(cols, 256), t128 = tiles_m * cdiv(cols, 128);
  return {10 * cdiv(t256, kPlanPairs) <= 7 * cdiv(t128, kPlanPairs) ? 256 : 128, 1, static_cast<int32_t>(kb)};
}

// One operand pair, tiles over rows x cols (cols counts D's columns, or the
// columns of each half).
inline Problem make_problem(const Plan& plan, int64_t rows, int64_t cols, int64_t kb, int a_map,
                            bool a_mn, int b_map, bool b_mn) {
  Problem p = {};
  p.a_map = a_map;
  p.b_map = b_map;
  p.a_mn = a_mn;
  p.b_mn = b_mn;
  p.bn = p.b_step = plan.bn;
  p.b_rank = plan.bn / 2;
  p.tiles_m = static_cast<int32_t>(cdiv(rows, kTile));
  p.tiles_n = static_cast<int32_t>(cdiv(cols, plan.bn));
  p.per_matrix = p.tiles_m * p.tiles_n;
  p.splits = plan.splits;
  p.kb = static_cast<int32_t>(kb);
  p.kb_split = plan.kb_split;
  p.idesc = static_cast<int32_t>(idesc_f16(true, a_mn, b_mn, plan.bn));
  return p;
}

// Launch grid: as many CTA pairs as can be resident.  `cache` is the kernel's,
// by device.
template <class Kernel>
cudaError_t resident_pairs(Kernel kern, int smem, DeviceOnce& cache, int num_sms, int* pairs) {
  cudaError_t e;
  std::atomic<int>* at = device_entry(cache, &e);
  if (!at) return e;
  int n = at->load(std::memory_order_acquire);
  if (n == 0) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
      return e;
    cudaLaunchConfig_t q = {};
    q.gridDim = dim3(static_cast<unsigned>(num_sms & ~1));
    q.blockDim = dim3(kThreads);
    q.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    q.attrs = attr;
    q.numAttrs = 1;
    if ((e = cudaOccupancyMaxActiveClusters(&n, kern, &q)) != cudaSuccess) return e;
    if (n > num_sms / 2) n = num_sms / 2;
    if (n < 1) return cudaErrorInvalidConfiguration;
    at->store(n, std::memory_order_release);
  }
  *pairs = n;
  return cudaSuccess;
}

template <class Epi>
cudaError_t resident_pairs(int num_sms, int* pairs) {
  static DeviceOnce cache;
  return resident_pairs(dense_kernel<Epi>, kSmemBytes, cache, num_sms, pairs);
}

template <class Kernel, class M, class L>
cudaError_t launch(Kernel kern, int smem, const M& maps, L& l, int pairs, cudaStream_t s, int units = 0) {
  int tiles = 0;
  for (int i = 0; i < l.problems; ++i) {
    l.p[i].first_tile = tiles;
    tiles += l.p[i].per_matrix * l.p[i].batch * l.p[i].splits;
  }
  l.tiles = tiles;
  if (tiles == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  if (units < tiles) units = tiles;
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (units < pairs ? units : pairs)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, maps, l);
}
template <class Epi>
cudaError_t launch(const Maps& maps, Launch<typename Epi::Args>& l, int pairs, cudaStream_t s) {
  int bn = 64;
  for (int i = 0; i < l.problems; ++i) bn = l.p[i].bn > bn ? l.p[i].bn : bn;
  l.slot = kABytes + bn * 64;
  l.stages = kOperandBytes / l.slot < kMaxStages ? kOperandBytes / l.slot : kMaxStages;
  return launch(dense_kernel<Epi>, kSmemBytes, maps, l, pairs, s);
}

}  // namespace dense
}  // namespace moe
