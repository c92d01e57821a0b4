// balance.cu -- the router's load-balance loss, the per-expert counts and the
// gradient of the router logits, in one pass over the logits.
//
// Over the valid tokens of sequence s (n_s of them), with c_se the slots that
// went to expert e, p_t the softmax of the logits over all experts:
//   f_se = E c_se / (k n_s)
//   loss = coef / S' * sum_s 1/n_s sum_t sum_e f_se p_te      (S' sequences with n_s > 0)
//   dloss/dz_te = coef / (S' n_s) * p_te (f_se - sum_j f_sj p_tj)
// f is the usual non-differentiable factor.  The mean probability of an expert
// appears only inside the sum over experts, so a token contributes one number,
// d_t = sum_e f_se p_te, which its gradient needs anyway: no [E] sums of
// probabilities are kept, and the gradient does not wait for the loss.  What
// it does wait for are the counts, hence two kernels, or one cluster's barrier
// where a small batch is one kernel.
//
// Bound by HBM: logits are read once and the gradient is written once, 8 E
// bytes a token; the counts read 4 k bytes a token.  65,536 tokens of 256
// experts, top-8, with the gate's gradient: 31.5 us, 4.5 TB/s of those bytes
// (the copy's rate would be 21 us), with 0.65 of the issue slots taken by the
// softmax's arithmetic.  (A call's last kernel lets no successor start early:
// it would only wait, on SMs that this call fills.)
#include <cfloat>

#include "cluster.cuh"
#include "entry.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kCountCtas = 8;       // one cluster of CTAs counts a sequence
constexpr int kCountThreads = 1024;
constexpr int kMainThreads = 256;

// Sequence bounds, held inside [0, T] and in order whatever the offsets hold.
__device__ __forceinline__ int2 seq_range(const int32_t* seq, int s, int T) {
  if (!seq) return make_int2(0, T);
  const int a = min(max(seq[s], 0), T);
  return make_int2(a, max(a, min(max(seq[s + 1], 0), T)));
}

// Cluster s counts sequence s: the slots of its valid tokens by expert, and
// its valid tokens.  Integer sums, so their order does not matter.  Each CTA
// takes a contiguous eighth of the tokens and then writes an eighth of the
// experts: counts, and f without the factors that main applies.
template <bool PARTS>
__global__ void __cluster_dims__(kCountCtas, 1, 1) __launch_bounds__(kCountThreads)
    balance_count_kernel(const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask,
                         const int32_t* __restrict__ seq, int T, int E, int k,
                         int parts, int32_t* __restrict__ counts, int32_t* __restrict__ n_valid,
                         uint32_t* __restrict__ ticket) {
  extern __shared__ int32_t hist[];   // [E] slots by expert, [E]: valid tokens
  griddep_wait();
  griddep_launch_dependents();
  const int unit = blockIdx.x / kCountCtas, s = PARTS ? 0 : unit;
  const int rank = static_cast<int>(cluster_rank());
  for (int i = threadIdx.x; i <= E; i += kCountThreads) hist[i] = 0;
  __syncthreads();
  const int2 r = seq_range(seq, s, T);
  const int64_t n = r.y - r.x;
  const int nth = PARTS ? static_cast<int>(blockIdx.x) : rank, of = PARTS ? parts * kCountCtas : kCountCtas;
  const int a = r.x + static_cast<int>(n * nth / of);
  const int b = r.x + static_cast<int>(n * (nth + 1) / of);
  // a token a thread (64 bits: the step past the last one may pass 2^31); its
  // slots in groups of 8 loads that do not wait for one another or for the mask
  int valid = 0;
  for (int64_t t = static_cast<int64_t>(a) + threadIdx.x; t < b; t += kCountThreads) {
    const bool ok = !mask || mask[t];
    const int32_t* row = ids + t * k;
    for (int j0 = 0; j0 < k; j0 += 8) {
      int e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = j0 + j < k ? row[j0 + j] : -1;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (ok && static_cast<unsigned>(e[j]) < static_cast<unsigned>(E)) atomicAdd(&hist[e[j]], 1);
    }
    valid += ok;
  }
  valid = __reduce_add_sync(0xFFFFFFFFu, valid);
  if ((threadIdx.x & 31) == 0 && valid) atomicAdd(&hist[E], valid);
  cluster_sync();
  const int e0 = E * rank / kCountCtas, e1 = E * (rank + 1) / kCountCtas;
  for (int e = e0 + threadIdx.x; e < e1; e += kCountThreads) {
    int sum = 0;
    for (int c = 0; c < kCountCtas; ++c) sum += cluster_load(hist + e, c);
    counts[static_cast<int64_t>(unit) * E + e] = sum;
  }
  if (rank == 0 && threadIdx.x == 0) {
    int sum = 0;
    for (int c = 0; c < kCountCtas; ++c) sum += cluster_load(hist + E, c);
    n_valid[unit] = sum;
    if (unit == 0) *ticket = 0;
  }
  cluster_sync();   // no CTA leaves while another reads its shared memory
}

struct BalanceArgs {
  const float* logits;
  const int32_t* ids;
  const uint8_t* mask;
  const int32_t* seq;
  const float* weights;
  const float* dweights;
  const int32_t* counts;
  const int32_t* n_valid;
  float* partial;        // one per CTA
  uint32_t* ticket;
  float* loss;
  float* dlogits;
  int32_t T, E, k, S;
  float coef;
  int32_t vec;           // logits and dlogits allow 16-byte accesses
};

// One sequence's counts in parts.
struct Parts {
  int32_t n;
  const int32_t* counts;   // [n, E]
  int32_t* sums;           // [E]
};

template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o, G));
  return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o, G);
  return v;
}

struct Slot {
  int id;
  float w, dw;
};

// Rows as G lanes hold them: lane l the experts 4 (l + G i) .. + 3, i < V.
// The gate gradient is scattered through shared memory: lane j writes slot j's
// value at its expert, the lanes add what they find there.
template <int G, int V>
struct Rows {
  static constexpr int kGroups = kMainThreads / G;   // tokens a CTA has in hand
  const BalanceArgs& a;
  const int lane, group;
  float* const gate;
  const bool gates, slots;   // slots: one a lane, where the lanes are enough for them

  // gate_s [kGroups * G * 4 V] in shared memory, visible after a barrier.
  __device__ __forceinline__ Rows(const BalanceArgs& args, float* gate_s)
      : a(args), lane(threadIdx.x % G), group(threadIdx.x / G), gate(gate_s + group * (G * 4 * V)),
        gates(args.weights && args.dlogits), slots(gates && args.k <= G) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      *reinterpret_cast<float4*>(gate + 4 * (lane + G * i)) = make_float4(0.f, 0.f, 0.f, 0.f);
  }

  __device__ __forceinline__ int expert(int i) const { return 4 * (lane + G * i); }

  // Token t's logits; -inf where it is not `on` and past the experts.
  __device__ __forceinline__ void load(int64_t t, bool on, float (&z)[4 * V]) const {
    const float* row = a.logits + t * a.E;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = expert(i);
#pragma unroll
      for (int q = 0; q < 4; ++q) z[4 * i + q] = -INFINITY;
      if (!on) continue;
      if (a.vec) {
        if (e < a.E) {
          const float4 v = __ldcs(reinterpret_cast<const float4*>(row + e));
          z[4 * i] = v.x, z[4 * i + 1] = v.y, z[4 * i + 2] = v.z, z[4 * i + 3] = v.w;
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (e + q < a.E) z[4 * i + q] = row[e + q];
      }
    }
  }

  __device__ __forceinline__ Slot slot_of(int64_t t, bool in) const {
    Slot s = {-1, 0.f, 0.f};
    if (slots && in && lane < a.k) {
      const int64_t r = t * a.k + lane;
      s.id = a.ids[r], s.w = a.weights[r], s.dw = a.dweights[r];
    }
    return s;
  }

  // f of a sequence with n valid tokens from its counts.
  __device__ __forceinline__ void factors(const int32_t* counts, int n, float (&f)[4 * V]) const {
    const float unit = n > 0 ? static_cast<float>(a.E) / (static_cast<float>(a.k) * static_cast<float>(n)) : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int e = expert(i) + q;
        f[4 * i + q] = e < a.E ? unit * static_cast<float>(counts[e]) : 0.f;
      }
  }

  // Token t (in: it exists; valid: it counts) with its sequence's f and weight
  // c: writes its gradient, returns c d_t (on lane 0; 0 elsewhere).  All
  // threads of the warp.
  __device__ __forceinline__ float take(int64_t t, bool in, bool valid, float (&z)[4 * V], const Slot& slot,
                                        const float (&f)[4 * V], float c) const {
    float top = z[0];
#pragma unroll
    for (int i = 1; i < 4 * V; ++i) top = fmaxf(top, z[i]);
    top = group_max<G>(top);
    // a row without a finite or infinite logit has no probabilities: p = 0
    // (a NaN beside it still shows: exp(NaN))
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < 4 * V; ++i) {
      // within 2 + 1.2 |z - base| units in the last place: in proportion to how
      // rare the expert is (the issue slots, not the precision, bound this kernel)
      z[i] = __expf(z[i] - base);
      sum += z[i];
      dot = fmaf(z[i], f[i], dot);
    }
    sum = group_sum<G>(sum);
    dot = group_sum<G>(dot);
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    dot *= inv;
    const float mine = valid && lane == 0 ? c * dot : 0.f;
    if (!a.dlogits) return mine;
    const float scale = valid ? c * inv : 0.f;
#pragma unroll
    for (int i = 0; i < 4 * V; ++i) z[i] = valid ? scale * z[i] * (f[i] - dot) : 0.f;
    if (slots) {
      const bool some = static_cast<unsigned>(slot.id) < static_cast<unsigned>(a.E);
      const float inner = group_sum<G>(some ? slot.w * slot.dw : 0.f);
      const float g = slot.w * (slot.dw - inner);
      // an expert named twice (never by the router): its slots one after the other
      const unsigned same =
          __match_any_sync(0xFFFFFFFFu, some ? slot.id + group * 1024 : -1 - static_cast<int>(threadIdx.x));
      const unsigned earlier = same & ((1u << (threadIdx.x & 31)) - 1);
      if (some && !earlier) gate[slot.id] = g;
      __syncwarp();
      if (__any_sync(0xFFFFFFFFu, earlier != 0)) {
        for (int l = 0; l < 32; ++l) {
          if (some && earlier && l == static_cast<int>(threadIdx.x & 31)) gate[slot.id] += g;
          __syncwarp();
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(gate + expert(i));
        z[4 * i] += v.x, z[4 * i + 1] += v.y, z[4 * i + 2] += v.z, z[4 * i + 3] += v.w;
      }
      __syncwarp();
      if (some) gate[slot.id] = 0.f;
      __syncwarp();
    } else if (gates && in) {   // more slots than lanes: few experts
      const int64_t r0 = t * a.k;
      float inner = 0.f;
      for (int j = 0; j < a.k; ++j)
        if (static_cast<unsigned>(a.ids[r0 + j]) < static_cast<unsigned>(a.E))
          inner = fmaf(a.weights[r0 + j], a.dweights[r0 + j], inner);
      for (int j = 0; j < a.k; ++j) {
        const int e = a.ids[r0 + j];
        const float g = a.weights[r0 + j] * (a.dweights[r0 + j] - inner);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (expert(i) + q == e && e < a.E) z[4 * i + q] += g;
      }
    }
    if (!in) return mine;
    float* out = a.dlogits + t * a.E;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = expert(i);
      if (a.vec) {
        if (e < a.E)
          __stcs(reinterpret_cast<float4*>(out + e),
                 make_float4(z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]));
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (e + q < a.E) out[e + q] = z[4 * i + q];
      }
    }
    return mine;
  }
};

// The CTA's threads' values, added in a fixed order; on thread 0.
__device__ __forceinline__ float block_sum(float v, float* sums) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  if (threadIdx.x == 0)
    for (int w = 0; w < kMainThreads / 32; ++w) v += sums[w];
  return v;
}

// CTAs an SM, all resident (65,536 tokens of 256 experts: 31 us at four with
// the registers they leave, 39 at two, 47 at five, which spill).
constexpr int main_ctas(int V) { return V <= 4 ? 4 : 2; }

// A CTA takes a contiguous range of tokens, its groups of lanes in turn.
// PARTS: one sequence, whose counts come in parts.  An own instantiation, with
// a parameter of its own, leaves the others the registers they had (65,536
// tokens of 256 experts in 24 sequences: 31.5 us; 33.8 with a condition).
template <int G, int V, bool PARTS>
__global__ void __launch_bounds__(kMainThreads, main_ctas(V)) balance_main_kernel(const BalanceArgs a, const Parts p) {
  constexpr int kGroups = Rows<G, V>::kGroups;
  __shared__ float sums[kMainThreads / 32];
  __shared__ __align__(16) float gate_s[kMainThreads * 4 * V];
  __shared__ int live_s;
  __shared__ bool last;
  int* whole = nullptr;   // the parts' sums
  if constexpr (PARTS) {
    __shared__ int sums_of_parts[1024];
    whole = sums_of_parts;
  }
  const Rows<G, V> rows(a, gate_s);
  if (threadIdx.x == 0) live_s = 0;
  __syncthreads();
  const int64_t t0 = static_cast<int64_t>(a.T) * blockIdx.x / gridDim.x;
  const int64_t t1 = static_cast<int64_t>(a.T) * (blockIdx.x + 1) / gridDim.x;
  auto is_on = [&](int64_t t) { return t < t1 && (!a.mask || a.mask[t]); };
  float mine = 0.f;
  int s = -1, s_end = -1;   // the sequence of the token in hand, and where it ends
  float f[4 * V], c = 0.f;
#pragma unroll
  for (int i = 0; i < 4 * V; ++i) f[i] = 0.f;
  int64_t t = t0 + rows.group;
  bool on = is_on(t), on_next = is_on(t + kGroups);
  // so far only the call's inputs; now the counts
  griddep_wait();
  [[maybe_unused]] int n_whole = 0;
  if constexpr (PARTS) {
    for (int q = 0; q < p.n; ++q) n_whole += a.n_valid[q];
    for (int e = threadIdx.x; e < a.E; e += kMainThreads) {
      int sum = 0;
#pragma unroll 8
      for (int q = 0; q < p.n; ++q) sum += p.counts[q * a.E + e];
      whole[e] = sum;
      if (blockIdx.x == 0) p.sums[e] = sum;
    }
  } else {
    int live = 0;
    for (int i = threadIdx.x; i < a.S; i += kMainThreads) live += a.n_valid[i] > 0;
    if (live) atomicAdd(&live_s, live);
  }
  __syncthreads();
  const float share = a.coef / static_cast<float>(max(live_s, 1));
  // every lane of a warp runs the same number of rounds (the shuffles)
  for (int64_t tt = t0; tt < t1; tt += kGroups, t += kGroups) {
    const bool in = t < t1, masked_in = on;
    float z[4 * V];
    const Slot slot = rows.slot_of(t, in);
    rows.load(t, on, z);
    on = on_next;
    on_next = is_on(t + 2 * kGroups);
    if (in && t >= s_end) {
      // the last sequence that begins at or before t
      int lo = 0, hi = a.S;
      if (a.seq)
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (a.seq[mid] <= t) lo = mid;
          else hi = mid;
        }
      const int2 r = seq_range(a.seq, lo, a.T);
      const bool inside = t >= r.x && t < r.y;   // not: a token of no sequence
      s = inside ? lo : -1;
      s_end = inside ? r.y : static_cast<int>(t) + 1;
      const int n = !inside ? 0 : PARTS ? n_whole : a.n_valid[s];
      c = n > 0 ? share / static_cast<float>(n) : 0.f;
      if constexpr (PARTS) rows.factors(whole, n, f);
      else rows.factors(a.counts + static_cast<int64_t>(lo) * a.E, n, f);
    }
    mine += rows.take(t, in, masked_in && s >= 0, z, slot, f, c);
  }
  // The loss: the CTAs' sums, added in CTA order by the last CTA to finish,
  // so that it does not depend on which one that is.
  mine = block_sum(mine, sums);
  if (threadIdx.x == 0) {
    __stcg(a.partial + blockIdx.x, mine);
    __threadfence();
    last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (last) {
    __threadfence();
    float v = 0.f;
    for (unsigned b = threadIdx.x; b < gridDim.x; b += kMainThreads) v += __ldcg(a.partial + b);
    v = block_sum(v, sums);
    if (threadIdx.x == 0) *a.loss = v;
  }
}

// A small batch of one sequence, whole, by one cluster: its CTAs count an
// eighth of the tokens each, add the counts up over distributed shared
// memory, and take their tokens' rows.  One launch and no workspace, for
// batches whose time is that of a launch (201 tokens of 8 experts: 4.1 us
// against 6.1 in two kernels).
constexpr int kSmallRounds = 2;   // tokens a group of lanes may have to take
__host__ __device__ constexpr int small_tokens(int lanes) {
  return kCountCtas * kSmallRounds * (kMainThreads / lanes);
}

template <int G, int V>
__global__ void __cluster_dims__(kCountCtas, 1, 1) __launch_bounds__(kMainThreads)
    balance_small_kernel(const BalanceArgs a, int32_t* __restrict__ counts_out) {
  constexpr int kGroups = Rows<G, V>::kGroups;
  __shared__ float sums[kMainThreads / 32];
  __shared__ __align__(16) float gate_s[kMainThreads * 4 * V];
  __shared__ int32_t hist[1025], total[1025];   // [E] slots by expert, [E]: valid tokens
  __shared__ __align__(16) float part[4];
  const Rows<G, V> rows(a, gate_s);
  const int rank = static_cast<int>(cluster_rank());
  for (int i = threadIdx.x; i <= a.E; i += kMainThreads) hist[i] = 0;
  __syncthreads();
  griddep_wait();
  const int t0 = static_cast<int>(static_cast<int64_t>(a.T) * rank / kCountCtas);
  const int t1 = static_cast<int>(static_cast<int64_t>(a.T) * (rank + 1) / kCountCtas);
  const int2 range = seq_range(a.seq, 0, a.T);
  auto is_on = [&](int t) { return t >= range.x && t < range.y && (!a.mask || a.mask[t]); };
  bool on[kSmallRounds];
  float z[kSmallRounds][4 * V];
#pragma unroll
  for (int i = 0; i < kSmallRounds; ++i) {
    const int t = t0 + i * kGroups + rows.group;
    on[i] = t < t1 && is_on(t);
    rows.load(t, on[i], z[i]);
    if (rows.lane == 0 && on[i]) atomicAdd(&hist[a.E], 1);
  }
  for (int i = t0 * a.k + static_cast<int>(threadIdx.x); i < t1 * a.k; i += kMainThreads) {
    const int e = a.ids[i];
    if (static_cast<unsigned>(e) < static_cast<unsigned>(a.E) && is_on(i / a.k))
      atomicAdd(&hist[e], 1);
  }
  cluster_sync();
  for (int e = threadIdx.x; e <= a.E; e += kMainThreads) {
    int32_t n[kCountCtas];
#pragma unroll
    for (int c = 0; c < kCountCtas; ++c) n[c] = cluster_load(hist + e, c);
#pragma unroll
    for (int c = 1; c < kCountCtas; ++c) n[0] += n[c];
    total[e] = n[0];
    if (e < a.E && e % kCountCtas == rank) counts_out[e] = n[0];
  }
  __syncthreads();
  const int n = total[a.E];
  float f[4 * V], mine = 0.f;
  const float c = n > 0 ? a.coef / static_cast<float>(n) : 0.f;
  rows.factors(total, n, f);
#pragma unroll
  for (int i = 0; i < kSmallRounds; ++i) {
    const int t = t0 + i * kGroups + rows.group;
    mine += rows.take(t, t < t1, on[i], z[i], rows.slot_of(t, t < t1), f, c);
  }
  mine = block_sum(mine, sums);
  if (threadIdx.x == 0) part[0] = mine;
  cluster_sync();
  if (rank == 0 && threadIdx.x == 0) {
    float v = 0.f;
    for (int r = 0; r < kCountCtas; ++r) v += cluster_load4(part, r).x;
    *a.loss = v;
  }
  cluster_sync();   // no CTA leaves while another reads its shared memory
}

__global__ void balance_empty_kernel(float* loss, int32_t* counts, int64_t n) {
  griddep_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i == 0) *loss = 0.f;
  if (i < n) counts[i] = 0;
}

constexpr int kMaxCtas = 152 * 8;   // CTAs the partial sums have room for

// Clusters that count a batch of one sequence: one for each round of their
// threads (32,768 tokens of 64 experts, top-8: 13 us against 16 with one, at
// 131,072 of 256 54 against 73; more than eight gain nothing).  Several sequences
// have a cluster each: as good from eight on (131,072 tokens in eight: 54 us), not
// below (in two: 62.5).
int count_parts(const moe_balance_shape* s) {
  const int parts = s->num_sequences > 1 ? 1 : s->num_tokens / (kCountCtas * kCountThreads);
  return parts < 1 ? 1 : parts < 8 ? parts : 8;
}

struct BalanceWs {
  int32_t parts;
  size_t n_valid, part_counts, partial, ticket, total;
};

BalanceWs balance_ws(const moe_balance_shape* s) {
  BalanceWs w;
  w.parts = count_parts(s);
  w.n_valid = 0;
  w.part_counts = ws_up(static_cast<size_t>(s->num_sequences) * w.parts * 4);
  w.partial = w.part_counts + (w.parts > 1 ? ws_up(static_cast<size_t>(w.parts) * s->num_experts * 4) : 0);
  w.ticket = w.partial + ws_up(kMaxCtas * 4);
  w.total = w.ticket + kWsAlign;
  return w;
}

int32_t check_balance(const moe_balance_shape* s) {
  if (!s) return entry_fail(MOE_ERR_INVALID_ARG, "shape is NULL");
  if (s->num_tokens < 0 || s->num_experts < 1 || s->num_experts > 1024 || s->top_k < 1 ||
      s->top_k > 32 || s->top_k > s->num_experts)
    return entry_fail(MOE_ERR_INVALID_ARG, "need num_tokens >= 0, 1 <= num_experts <= 1024, "
                                           "1 <= top_k <= min(num_experts, 32)");
  if (static_cast<int64_t>(s->num_tokens) * s->top_k >= (int64_t(1) << 31))
    return entry_fail(MOE_ERR_INVALID_ARG, "num_tokens * top_k must be < 2^31");
  if (s->num_sequences < 1 || s->num_sequences > (1 << 20))
    return entry_fail(MOE_ERR_INVALID_ARG, "num_sequences must be in [1, 2^20]");
  if (!(s->coef - s->coef == 0.f)) return entry_fail(MOE_ERR_INVALID_ARG, "coef must be finite");
  return MOE_OK;
}

// Lanes per token: as many as hold its experts by fours up to 64 experts, then
// half a warp (two tokens share the reductions' instructions) while four groups
// of four a lane do; and those groups.
struct Split {
  int lanes, v;
};
Split split_of(int E) {
  if (E <= 8) return {2, 1};
  if (E <= 16) return {4, 1};
  if (E <= 32) return {8, 1};
  if (E <= 64) return {16, 1};
  if (E <= 128) return {16, 2};
  if (E <= 256) return {16, 4};
  return {32, E <= 384 ? 3 : E <= 512 ? 4 : 8};
}

bool is_small(const moe_balance_shape* s) {
  return s->num_sequences == 1 && s->num_tokens <= small_tokens(split_of(s->num_experts).lanes);
}

template <int G, int V>
cudaError_t launch_rows(const BalanceArgs& a, const Parts& p, bool small, int sms, cudaStream_t st) {
  if (small)
    return launch_pdl(balance_small_kernel<G, V>, dim3(kCountCtas), dim3(kMainThreads), 0, st, a, p.sums);
  const int per_round = kMainThreads / G;
  const int64_t rounds = (static_cast<int64_t>(a.T) + per_round - 1) / per_round;
  int ctas = sms * main_ctas(V);   // one wave
  if (ctas > kMaxCtas) ctas = kMaxCtas;
  return launch_pdl(p.n > 1 ? balance_main_kernel<G, V, true> : balance_main_kernel<G, V, false>,
                    dim3(static_cast<unsigned>(rounds < ctas ? rounds : ctas)), dim3(kMainThreads), 0, st, a, p);
}

cudaError_t launch_by_experts(const BalanceArgs& a, const Parts& parts, bool small, int sms, cudaStream_t st) {
  const Split p = split_of(a.E);
  switch (p.lanes) {
    case 2: return launch_rows<2, 1>(a, parts, small, sms, st);
    case 4: return launch_rows<4, 1>(a, parts, small, sms, st);
    case 8: return launch_rows<8, 1>(a, parts, small, sms, st);
    case 16:
      return p.v == 1   ? launch_rows<16, 1>(a, parts, small, sms, st)
             : p.v == 2 ? launch_rows<16, 2>(a, parts, small, sms, st)
                        : launch_rows<16, 4>(a, parts, small, sms, st);
    default:
      return p.v == 3   ? launch_rows<32, 3>(a, parts, small, sms, st)
             : p.v == 4 ? launch_rows<32, 4>(a, parts, small, sms, st)
                        : launch_rows<32, 8>(a, parts, small, sms, st);
  }
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_balance_workspace_size(const moe_balance_shape* shape) {
  if (moe::check_balance(shape) != MOE_OK) return 0;
  return moe::is_small(shape) ? moe::kWsAlign : moe::balance_ws(shape).total;
}

extern "C" int32_t moe_balance_loss(const moe_balance_shape* shape, const float* logits,
                                    const int32_t* ids, const uint8_t* token_mask,
                                    const int32_t* seq_offsets, const float* weights,
                                    const float* dweights, float* loss, int32_t* counts,
                                    float* dlogits, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  using namespace moe;
  int32_t rc = check_balance(shape);
  if (rc != MOE_OK) return rc;
  const int T = shape->num_tokens, E = shape->num_experts, S = shape->num_sequences;
  if (!loss || !counts) return entry_fail(MOE_ERR_INVALID_ARG, "loss or counts is NULL");
  const bool small = is_small(shape), use_ws = T > 0 && !small;
  if (T > 0 && (!logits || !ids)) return entry_fail(MOE_ERR_INVALID_ARG, "logits or ids is NULL");
  if (use_ws && !workspace) return entry_fail(MOE_ERR_INVALID_ARG, "workspace is NULL");
  if (S > 1 && !seq_offsets)
    return entry_fail(MOE_ERR_INVALID_ARG, "num_sequences > 1 needs seq_offsets");
  if (!weights != !dweights)
    return entry_fail(MOE_ERR_INVALID_ARG, "weights and dweights go together");
  const void* ptrs[8] = {logits, ids, seq_offsets, weights, dweights, loss, counts, dlogits};
  for (const void* p : ptrs)
    if (!ptr_aligned(p, 4)) return entry_fail(MOE_ERR_MISALIGNED, "a pointer is not 4-byte aligned");
  if (use_ws && !ptr_aligned(workspace, kWsAlign))
    return entry_fail(MOE_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  const BalanceWs w = balance_ws(shape);
  if (use_ws && workspace_bytes < w.total)
    return entry_fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, needs %zu",
                      workspace_bytes, w.total);
  int sms = 0;
  if ((rc = check_device(&sms)) != MOE_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    const int64_t n = static_cast<int64_t>(S) * E;
    return entry_launched(launch_pdl(balance_empty_kernel,
                                     dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0,
                                     st, loss, counts, n));
  }
  uint8_t* base = static_cast<uint8_t*>(workspace);
  int32_t* n_valid = small ? nullptr : reinterpret_cast<int32_t*>(base + w.n_valid);
  int32_t* part_counts = small ? nullptr : reinterpret_cast<int32_t*>(base + w.part_counts);
  uint32_t* ticket = small ? nullptr : reinterpret_cast<uint32_t*>(base + w.ticket);
  cudaError_t e = cudaSuccess;
  if (!small)
    e = launch_pdl(w.parts > 1 ? balance_count_kernel<true> : balance_count_kernel<false>,
                   dim3(static_cast<unsigned>(S) * w.parts * kCountCtas),
                   dim3(kCountThreads), (E + 1) * sizeof(int32_t), st, ids, token_mask, seq_offsets, T,
                   E, shape->top_k, w.parts, w.parts > 1 ? part_counts : counts, n_valid, ticket);
  if (e != cudaSuccess) return entry_launched(e);
  BalanceArgs a;
  a.logits = logits;
  a.ids = ids;
  a.mask = token_mask;
  a.seq = seq_offsets;
  a.weights = weights;
  a.dweights = dweights;
  a.counts = counts;
  a.n_valid = n_valid;
  a.partial = small ? nullptr : reinterpret_cast<float*>(base + w.partial);
  a.ticket = ticket;
  a.loss = loss;
  a.dlogits = dlogits;
  a.T = T, a.E = E, a.k = shape->top_k, a.S = S;
  a.coef = shape->coef;
  a.vec = E % 4 == 0 && ptr_aligned(logits, 16) && ptr_aligned(dlogits, 16);
  return entry_launched(launch_by_experts(a, {w.parts, part_counts, counts}, small, sms, st));
}
