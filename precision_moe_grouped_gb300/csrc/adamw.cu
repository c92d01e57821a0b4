// adamw.cu -- one AdamW step over many tensors in one launch, with the
// moments in 32 bits or as 8-bit codes.
//
// Per element, with b1, b2 the decay rates and t the step:
//   m <- b1 m + (1 - b1) g          v <- b2 v + (1 - b2) g^2
//   p <- p (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// Every operation is one IEEE float32 operation in the order written (no
// contraction), so that the 8-bit codes do not depend on how the compiler
// groups them.  The scalars come from the host, computed in double and
// rounded once.
//
// 8-bit moments: blocks of 256 consecutive elements of a tensor share one
// float scale.  The block's new values x (m, or r = sqrt(v)) become E4M3
// codes of x * (448 / amax) and the scale amax / 448, the rule of the forward's
// per-token FP8 activations.  The second moment is kept as its root: E4M3
// spans 2.3e5 between its largest and its least value, which is then the
// span of the gradients' sizes inside a block and not of their squares.  A
// root above zero never becomes code 0 (it is lifted to the least code), so
// a small second moment cannot leave a moment to be divided by eps alone.
// The scale is a float and not a power of two because it carries the decay: a
// block whose gradients stop has all its values shrink alike, codes unchanged,
// where rounding each value to 3 bits of mantissa would leave 0.999 v at v.
// A block with a NaN or an infinity becomes NaN altogether.
//
// Bound by HBM: 26 or 28 bytes an element (32-bit moments, float or bf16
// gradients, 2 more for a bf16 copy of the parameter), 14.06 or 16.06 with
// 8-bit moments.  200 M elements with bf16 gradients and copies: 787 us (7.1
// TB/s, a little above a plain copy) with 32-bit moments, 543 us (5.9 TB/s, 0.83
// of the issue slots) with 8-bit ones.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cmath>
#include <cstring>

#include "entry.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kBlock8 = MOE_ADAMW_BLOCK;   // elements that share a scale: one warp's
constexpr int kThreads = 256;
constexpr int kChunk = kThreads * 8;       // elements of one CTA
static_assert(kBlock8 == 256, "a warp takes 8 elements a lane");

struct Entry {
  float* p;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  __nv_bfloat16* copy;
  int64_t n;
  int32_t first_chunk;
  int32_t vec;   // every pointer allows 4-element accesses
};

// The tensors of one launch travel as a kernel parameter (at most 32,764
// bytes), so that a step copies nothing to the device.  Captured into a graph it
// repeats its table and its scalars, so one step number, at every replay.  The
// table comes in three sizes because its bytes are copied at each launch.
template <int CAP>
struct Table {
  int32_t count;
  Entry e[CAP];
};
constexpr int kCapSmall = 16, kCapMid = 112, kCapLarge = 400;
static_assert(sizeof(Table<kCapLarge>) < 32500, "kernel parameters");

struct Scalars {
  float b1, c1, b2, c2, decay, step, root, eps;
  const float* grad_scale;
};

struct Moments {
  float p, m, r;   // r = sqrt(v)
  float v;
};

__device__ __forceinline__ Moments update(float p, float g, float m, float v, const Scalars& s) {
  Moments o;
  o.m = __fadd_rn(__fmul_rn(m, s.b1), __fmul_rn(g, s.c1));
  o.v = __fadd_rn(__fmul_rn(v, s.b2), __fmul_rn(__fmul_rn(g, g), s.c2));
  o.r = __fsqrt_rn(o.v);
  const float den = __fadd_rn(__fmul_rn(o.r, s.root), s.eps);
  o.p = __fsub_rn(__fmul_rn(p, s.decay), __fdiv_rn(__fmul_rn(o.m, s.step), den));
  return o;
}

// Block scale and its inverse from the largest magnitude's bits (ordered as
// integers a NaN is above infinity, so that it survives the maximum).
__device__ __forceinline__ void block_scale(uint32_t amax_bits, float* inv, float* scale) {
  const float amax = __uint_as_float(amax_bits);
  const bool some = !(amax < 7.888609052210118e-31f);   // 2^-100; true for a NaN
  *inv = some ? __fdiv_rn(448.0f, amax) : 0.0f;
  *scale = some ? __fdiv_rn(amax, 448.0f) : 1.0f;
}

// Codes of four values times inv, first in the low byte; `least` (zero or the
// least positive value) below which a positive value does not go.
template <bool POSITIVE>
__device__ __forceinline__ uint32_t encode4(const float* x, float inv, float least) {
  float q[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    q[c] = __fmul_rn(x[c], inv);
    if (POSITIVE && x[c] > 0.f) q[c] = fmaxf(q[c], least);
  }
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[2], q[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// Four codes times their scale.
__device__ __forceinline__ void decode4(uint32_t codes, float scale, float* o) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(codes >> (16 * h)), __NV_E4M3);
    const float2 f = __half22float2(__half2(r));
    o[2 * h] = __fmul_rn(f.x, scale);
    o[2 * h + 1] = __fmul_rn(f.y, scale);
  }
}

template <bool BF16G>
__device__ __forceinline__ void load_grad4(const void* g, int i, float* o) {
  if constexpr (BF16G) {
    const uint2 q = __ldcs(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(g) + i));
    o[0] = __uint_as_float(q.x << 16);
    o[1] = __uint_as_float(q.x & 0xFFFF0000u);
    o[2] = __uint_as_float(q.y << 16);
    o[3] = __uint_as_float(q.y & 0xFFFF0000u);
  } else {
    const float4 q = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(g) + i));
    o[0] = q.x, o[1] = q.y, o[2] = q.z, o[3] = q.w;
  }
}

template <bool BF16G>
__device__ __forceinline__ float load_grad(const void* g, int i) {
  if constexpr (BF16G) return __bfloat162float(static_cast<const __nv_bfloat16*>(g)[i]);
  else return static_cast<const float*>(g)[i];
}

// 256 consecutive elements from w0 (an 8-bit block) by one warp, lane l the
// groups of four at 4 l and 128 + 4 l.  VEC: all of them exist, and every pointer
// allows 4-element accesses.
template <bool BITS8, bool BF16G, bool VEC>
__device__ __forceinline__ void take_block(const Entry& t, int64_t w0, const Scalars& s, float gs) {
  const int lane = threadIdx.x & 31;
  const int64_t i0 = w0 + 4 * lane;
  float* const tp = t.p + i0;
  const void* const tg = BF16G ? static_cast<const void*>(static_cast<const __nv_bfloat16*>(t.g) + i0)
                               : static_cast<const void*>(static_cast<const float*>(t.g) + i0);
  float* const tm = static_cast<float*>(t.m) + i0;
  float* const tv = static_cast<float*>(t.v) + i0;
  uint8_t* const cm = static_cast<uint8_t*>(t.m) + i0;
  uint8_t* const cv = static_cast<uint8_t*>(t.v) + i0;
  __nv_bfloat16* const tc = t.copy ? t.copy + i0 : nullptr;
  const int left = VEC ? 256 : static_cast<int>(min(t.n - i0, static_cast<int64_t>(256)));
  auto has = [&](int k) { return k < left; };   // element i0 + k exists
  float p[8], g[8], m[8], v[8];
  float ms = 1.f, vs = 1.f;
  if constexpr (BITS8) {
    ms = t.m_scale[w0 / kBlock8];
    vs = t.v_scale[w0 / kBlock8];
  }
  uint32_t mc[2] = {0, 0}, vc[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if constexpr (VEC) {
      load_grad4<BF16G>(tg, 128 * j, g + 4 * j);
      const float4 q = __ldcs(reinterpret_cast<const float4*>(tp + 128 * j));
      p[4 * j] = q.x, p[4 * j + 1] = q.y, p[4 * j + 2] = q.z, p[4 * j + 3] = q.w;
      if constexpr (BITS8) {
        mc[j] = __ldcs(reinterpret_cast<const uint32_t*>(cm + 128 * j));
        vc[j] = __ldcs(reinterpret_cast<const uint32_t*>(cv + 128 * j));
      } else {
        const float4 a = __ldcs(reinterpret_cast<const float4*>(tm + 128 * j));
        const float4 b = __ldcs(reinterpret_cast<const float4*>(tv + 128 * j));
        m[4 * j] = a.x, m[4 * j + 1] = a.y, m[4 * j + 2] = a.z, m[4 * j + 3] = a.w;
        v[4 * j] = b.x, v[4 * j + 1] = b.y, v[4 * j + 2] = b.z, v[4 * j + 3] = b.w;
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) {   // an element beyond the tensor's end is zero and stays zero
        const int k = 128 * j + c, e = 4 * j + c;
        p[e] = g[e] = m[e] = v[e] = 0.f;
        if (has(k)) {
          g[e] = load_grad<BF16G>(tg, k);
          p[e] = tp[k];
          if constexpr (BITS8) {
            mc[j] |= static_cast<uint32_t>(cm[k]) << (8 * c);
            vc[j] |= static_cast<uint32_t>(cv[k]) << (8 * c);
          } else {
            m[e] = tm[k];
            v[e] = tv[k];
          }
        }
      }
    }
  }
  uint32_t ma = 0, ra = 0;
  float r[8];
  if constexpr (BITS8) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      decode4(mc[j], ms, m + 4 * j);
      decode4(vc[j], vs, v + 4 * j);
    }
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float vo = BITS8 ? __fmul_rn(v[c], v[c]) : v[c];
    const Moments o = update(p[c], s.grad_scale ? __fmul_rn(g[c], gs) : g[c], m[c], vo, s);
    p[c] = o.p, m[c] = o.m, v[c] = o.v, r[c] = o.r;
    if constexpr (BITS8) {
      ma = max(ma, __float_as_uint(o.m) & 0x7FFFFFFFu);
      ra = max(ra, __float_as_uint(o.r) & 0x7FFFFFFFu);
    }
  }
  if constexpr (BITS8) {
    float minv, rinv;
    ma = __reduce_max_sync(0xFFFFFFFFu, ma);
    ra = __reduce_max_sync(0xFFFFFFFFu, ra);
    block_scale(ma, &minv, &ms);
    block_scale(ra, &rinv, &vs);
    if (lane == 0) {
      t.m_scale[w0 / kBlock8] = ms;
      t.v_scale[w0 / kBlock8] = vs;
    }
    const float least = rinv > 0.f ? 0.001953125f : 0.f;   // 2^-9, the least code's value
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      mc[j] = encode4<false>(m + 4 * j, minv, 0.f);
      vc[j] = encode4<true>(r + 4 * j, rinv, least);
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if constexpr (VEC) {
      __stcs(reinterpret_cast<float4*>(tp + 128 * j),
             make_float4(p[4 * j], p[4 * j + 1], p[4 * j + 2], p[4 * j + 3]));
      if (tc) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(p[4 * j], p[4 * j + 1]);
        const __nv_bfloat162 b = __floats2bfloat162_rn(p[4 * j + 2], p[4 * j + 3]);
        uint2 q;
        memcpy(&q.x, &a, 4);
        memcpy(&q.y, &b, 4);
        __stcs(reinterpret_cast<uint2*>(tc + 128 * j), q);
      }
      if constexpr (BITS8) {
        __stcs(reinterpret_cast<uint32_t*>(cm + 128 * j), mc[j]);
        __stcs(reinterpret_cast<uint32_t*>(cv + 128 * j), vc[j]);
      } else {
        __stcs(reinterpret_cast<float4*>(tm + 128 * j),
               make_float4(m[4 * j], m[4 * j + 1], m[4 * j + 2], m[4 * j + 3]));
        __stcs(reinterpret_cast<float4*>(tv + 128 * j),
               make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int k = 128 * j + c, e = 4 * j + c;
        if (!has(k)) continue;
        tp[k] = p[e];
        if (tc) tc[k] = __float2bfloat16_rn(p[e]);
        if constexpr (BITS8) {
          cm[k] = static_cast<uint8_t>(mc[j] >> (8 * c));
          cv[k] = static_cast<uint8_t>(vc[j] >> (8 * c));
        } else {
          tm[k] = m[e];
          tv[k] = v[e];
        }
      }
    }
  }
}

// One CTA per chunk of one tensor, a block of 256 a warp.  One block and no
// more: the next CTA's loads then run under this one's arithmetic, about 70
// instructions an element with 8-bit moments (200 M elements: 542 us at six
// CTAs an SM; 720 with two blocks a warp in turn).  Six CTAs leave the 8-bit form
// 40 registers, and it spills: 120 bytes of stores and 152 of loads a thread, some
// 8 of those instructions.
template <bool BITS8, bool BF16G, int CAP>
__global__ void __launch_bounds__(kThreads, BITS8 ? 6 : 4)
    adamw_kernel(const __grid_constant__ Table<CAP> tab, const Scalars s) {
  const int chunk = blockIdx.x;
  int lo = 0, hi = tab.count;   // the last entry that begins at or before this chunk
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tab.e[mid].first_chunk <= chunk) lo = mid;
    else hi = mid;
  }
  const Entry& t = tab.e[lo];
  griddep_wait();
  const float gs = s.grad_scale ? __ldg(s.grad_scale) : 1.0f;
  const int64_t w0 = static_cast<int64_t>(chunk - t.first_chunk) * kChunk + (threadIdx.x >> 5) * kBlock8;
  if (w0 >= t.n) return;
  if (t.vec && w0 + kBlock8 <= t.n) take_block<BITS8, BF16G, true>(t, w0, s, gs);
  else take_block<BITS8, BF16G, false>(t, w0, s, gs);
}

template <int CAP>
cudaError_t launch_table(const Table<CAP>& tab, int64_t chunks, const Scalars& s, bool bits8,
                         bool bf16g, cudaStream_t st) {
  auto kern = bits8 ? (bf16g ? adamw_kernel<true, true, CAP> : adamw_kernel<true, false, CAP>)
                    : (bf16g ? adamw_kernel<false, true, CAP> : adamw_kernel<false, false, CAP>);
  return launch_pdl(kern, dim3(static_cast<unsigned>(chunks)), dim3(kThreads), 0, st, tab, s);
}

int64_t chunks_of(int64_t n) { return (n + kChunk - 1) / kChunk; }

// The tensors [at, at + count) in one launch.  Empty ones take no chunk (and
// no entry); a launch holds at most 2^30 chunks.
template <int CAP>
cudaError_t launch_group(const moe_adamw_tensor* t, int count, const Scalars& s, bool bits8,
                         bool bf16g, cudaStream_t st) {
  Table<CAP> tab;
  tab.count = 0;
  int64_t chunks = 0;
  for (int i = 0; i < count; ++i) {
    if (t[i].n == 0) continue;
    Entry& e = tab.e[tab.count++];
    e.p = t[i].param;
    e.g = t[i].grad;
    e.m = t[i].m;
    e.v = t[i].v;
    e.m_scale = t[i].m_scale;
    e.v_scale = t[i].v_scale;
    e.copy = static_cast<__nv_bfloat16*>(t[i].param_bf16);
    e.n = t[i].n;
    e.first_chunk = static_cast<int32_t>(chunks);
    const size_t state = bits8 ? 4 : 16;
    e.vec = ptr_aligned(e.p, 16) && ptr_aligned(e.g, bf16g ? 8 : 16) && ptr_aligned(e.m, state) &&
            ptr_aligned(e.v, state) && ptr_aligned(e.copy, 8);
    chunks += chunks_of(t[i].n);
  }
  if (chunks == 0) return cudaSuccess;
  return launch_table(tab, chunks, s, bits8, bf16g, st);
}

int32_t check_tensor(const moe_adamw_tensor& t, int i, bool bits8, bool bf16g) {
  if (t.n < 0) return entry_fail(MOE_ERR_INVALID_ARG, "tensor %d: n < 0", i);
  if (t.n == 0) return MOE_OK;
  if (!t.param || !t.grad || !t.m || !t.v)
    return entry_fail(MOE_ERR_INVALID_ARG, "tensor %d: param, grad, m or v is NULL", i);
  if (bits8 && (!t.m_scale || !t.v_scale))
    return entry_fail(MOE_ERR_INVALID_ARG, "tensor %d: 8-bit moments need m_scale and v_scale", i);
  if (chunks_of(t.n) > (int64_t(1) << 30))
    return entry_fail(MOE_ERR_UNSUPPORTED, "tensor %d: more than 2^41 elements", i);
  const size_t state = bits8 ? 1 : 4;
  if (!ptr_aligned(t.param, 4) || !ptr_aligned(t.grad, bf16g ? 2 : 4) || !ptr_aligned(t.m, state) ||
      !ptr_aligned(t.v, state) || (bits8 && (!ptr_aligned(t.m_scale, 4) || !ptr_aligned(t.v_scale, 4))) ||
      !ptr_aligned(t.param_bf16, 2))
    return entry_fail(MOE_ERR_MISALIGNED, "tensor %d: a pointer is not aligned to its type", i);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" int32_t moe_adamw_step(const moe_adamw_tensor* tensors, int32_t count,
                                  const moe_adamw_options* o, void* stream) {
  using namespace moe;
  if (!o) return entry_fail(MOE_ERR_INVALID_ARG, "options is NULL");
  if (count < 0) return entry_fail(MOE_ERR_INVALID_ARG, "count < 0");
  if (o->state_bits != 8 && o->state_bits != 32)
    return entry_fail(MOE_ERR_INVALID_ARG, "state_bits must be 8 or 32");
  if (o->grad_dtype != MOE_DTYPE_F32 && o->grad_dtype != MOE_DTYPE_BF16)
    return entry_fail(MOE_ERR_INVALID_ARG, "grad_dtype %d unknown", o->grad_dtype);
  if (o->step < 1) return entry_fail(MOE_ERR_INVALID_ARG, "step must be at least 1");
  if (!(o->beta1 >= 0 && o->beta1 < 1) || !(o->beta2 >= 0 && o->beta2 < 1))
    return entry_fail(MOE_ERR_INVALID_ARG, "beta1 and beta2 must be in [0, 1)");
  if (!(o->eps >= 0) || !std::isfinite(o->eps) || !std::isfinite(o->lr) ||
      !std::isfinite(o->weight_decay))
    return entry_fail(MOE_ERR_INVALID_ARG, "lr, eps and weight_decay must be finite, eps >= 0");
  if (!ptr_aligned(o->grad_scale, 4))
    return entry_fail(MOE_ERR_MISALIGNED, "grad_scale must be 4-byte aligned");
  if (o->reserved[0] || o->reserved[1])
    return entry_fail(MOE_ERR_INVALID_ARG, "reserved must be zero");
  if (count == 0) return MOE_OK;
  if (!tensors) return entry_fail(MOE_ERR_INVALID_ARG, "tensors is NULL");
  const bool bits8 = o->state_bits == 8, bf16g = o->grad_dtype == MOE_DTYPE_BF16;
  bool any = false;
  for (int i = 0; i < count; ++i) {
    const int32_t rc = check_tensor(tensors[i], i, bits8, bf16g);
    if (rc != MOE_OK) return rc;
    any = any || tensors[i].n > 0;
  }
  if (!any) return MOE_OK;
  const int32_t rc = check_device(nullptr);
  if (rc != MOE_OK) return rc;
  Scalars s;
  s.b1 = static_cast<float>(o->beta1);
  s.c1 = static_cast<float>(1.0 - o->beta1);
  s.b2 = static_cast<float>(o->beta2);
  s.c2 = static_cast<float>(1.0 - o->beta2);
  s.decay = static_cast<float>(1.0 - o->lr * o->weight_decay);
  s.step = static_cast<float>(o->lr / (1.0 - std::pow(o->beta1, o->step)));
  s.root = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(o->beta2, o->step)));
  s.eps = static_cast<float>(o->eps);
  s.grad_scale = o->grad_scale;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  for (int at = 0; at < count;) {
    // as many tensors as a table and 2^30 chunks hold
    int64_t chunks = chunks_of(tensors[at].n);
    int n = 1;
    while (at + n < count && n < kCapLarge &&
           chunks + chunks_of(tensors[at + n].n) <= (int64_t(1) << 30))
      chunks += chunks_of(tensors[at + n++].n);
    const moe_adamw_tensor* t = tensors + at;
    const cudaError_t e = n <= kCapSmall ? launch_group<kCapSmall>(t, n, s, bits8, bf16g, st)
                          : n <= kCapMid ? launch_group<kCapMid>(t, n, s, bits8, bf16g, st)
                                         : launch_group<kCapLarge>(t, n, s, bits8, bf16g, st);
    if (e != cudaSuccess) return entry_launched(e);
    at += n;
  }
  return MOE_OK;
}
