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
// 8-bit moments.
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
// bytes), so that a step copies nothing to the device and can be captured
// into a graph.  The table comes in three sizes because its bytes are copied
// at each launch.
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

__device__ __forceinline__ uint32_t e4m3(float x, float inv) {
  return __nv_cvt_float_to_fp8(__fmul_rn(x, inv), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float from_e4m3(uint32_t code) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3);
  return __half2float(__half(h));
}

template <bool BF16G>
__device__ __forceinline__ void load_grad4(const void* g, int64_t i, float (&o)[4]) {
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
__device__ __forceinline__ float load_grad(const void* g, int64_t i) {
  if constexpr (BF16G) return __bfloat162float(static_cast<const __nv_bfloat16*>(g)[i]);
  else return static_cast<const float*>(g)[i];
}

// One CTA per chunk of 2048 elements of one tensor; a warp holds 256
// consecutive ones (an 8-bit block), lane l the groups of four at 4 l and
// 128 + 4 l.
template <bool BITS8, bool BF16G, int CAP>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Table<CAP> tab,
                                                         const Scalars s) {
  const int chunk = blockIdx.x;
  int lo = 0, hi = tab.count;   // the last entry that begins at or before this chunk
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tab.e[mid].first_chunk <= chunk) lo = mid;
    else hi = mid;
  }
  const Entry& t = tab.e[lo];
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t w0 = static_cast<int64_t>(chunk - t.first_chunk) * kChunk + (threadIdx.x >> 5) * 256;
  const int64_t n = t.n;
  if (w0 >= n) return;
  const bool vec = t.vec && w0 + 256 <= n;
  const float gs = s.grad_scale ? __ldg(s.grad_scale) : 1.0f;
  float p[8], g[8], m[8], v[8];
  float ms = 1.f, vs = 1.f;
  if constexpr (BITS8) {
    ms = t.m_scale[w0 / kBlock8];
    vs = t.v_scale[w0 / kBlock8];
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t i = w0 + 128 * j + 4 * lane;
    float gg[4] = {0.f, 0.f, 0.f, 0.f}, pp[4] = {0.f, 0.f, 0.f, 0.f};
    float mm[4] = {0.f, 0.f, 0.f, 0.f}, vv[4] = {0.f, 0.f, 0.f, 0.f};
    if (vec) {
      load_grad4<BF16G>(t.g, i, gg);
      const float4 q = __ldcs(reinterpret_cast<const float4*>(t.p + i));
      pp[0] = q.x, pp[1] = q.y, pp[2] = q.z, pp[3] = q.w;
      if constexpr (BITS8) {
        const uint32_t mc = __ldcs(reinterpret_cast<const uint32_t*>(static_cast<uint8_t*>(t.m) + i));
        const uint32_t vc = __ldcs(reinterpret_cast<const uint32_t*>(static_cast<uint8_t*>(t.v) + i));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mm[c] = from_e4m3((mc >> (8 * c)) & 0xFF);
          vv[c] = from_e4m3((vc >> (8 * c)) & 0xFF);
        }
      } else {
        const float4 a = __ldcs(reinterpret_cast<const float4*>(static_cast<float*>(t.m) + i));
        const float4 b = __ldcs(reinterpret_cast<const float4*>(static_cast<float*>(t.v) + i));
        mm[0] = a.x, mm[1] = a.y, mm[2] = a.z, mm[3] = a.w;
        vv[0] = b.x, vv[1] = b.y, vv[2] = b.z, vv[3] = b.w;
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (i + c < n) {
          gg[c] = load_grad<BF16G>(t.g, i + c);
          pp[c] = t.p[i + c];
          if constexpr (BITS8) {
            mm[c] = from_e4m3(static_cast<uint8_t*>(t.m)[i + c]);
            vv[c] = from_e4m3(static_cast<uint8_t*>(t.v)[i + c]);
          } else {
            mm[c] = static_cast<float*>(t.m)[i + c];
            vv[c] = static_cast<float*>(t.v)[i + c];
          }
        }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
      p[4 * j + c] = pp[c], g[4 * j + c] = gg[c], m[4 * j + c] = mm[c], v[4 * j + c] = vv[c];
  }
  uint32_t ma = 0, ra = 0;
  float r[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    float mo = m[c], vo = v[c];
    if constexpr (BITS8) {
      mo = __fmul_rn(mo, ms);
      vo = __fmul_rn(vo, vs);
      vo = __fmul_rn(vo, vo);
    }
    const float gc = s.grad_scale ? __fmul_rn(g[c], gs) : g[c];
    const Moments o = update(p[c], gc, mo, vo, s);
    p[c] = o.p, m[c] = o.m, v[c] = o.v, r[c] = o.r;
    if constexpr (BITS8) {
      // an element beyond the tensor's end is zero and stays zero
      ma = max(ma, __float_as_uint(o.m) & 0x7FFFFFFFu);
      ra = max(ra, __float_as_uint(o.r) & 0x7FFFFFFFu);
    }
  }
  float minv = 0.f, rinv = 0.f;
  if constexpr (BITS8) {
    ma = __reduce_max_sync(0xFFFFFFFFu, ma);
    ra = __reduce_max_sync(0xFFFFFFFFu, ra);
    block_scale(ma, &minv, &ms);
    block_scale(ra, &rinv, &vs);
    if (lane == 0) {
      t.m_scale[w0 / kBlock8] = ms;
      t.v_scale[w0 / kBlock8] = vs;
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t i = w0 + 128 * j + 4 * lane;
    uint32_t mc[4], vc[4];
    if constexpr (BITS8) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mc[c] = e4m3(m[4 * j + c], minv);
        vc[c] = e4m3(r[4 * j + c], rinv);
        if (vc[c] == 0 && r[4 * j + c] > 0.f && rinv > 0.f) vc[c] = 1;
      }
    }
    if (vec) {
      __stcs(reinterpret_cast<float4*>(t.p + i),
             make_float4(p[4 * j], p[4 * j + 1], p[4 * j + 2], p[4 * j + 3]));
      if (t.copy) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(p[4 * j], p[4 * j + 1]);
        const __nv_bfloat162 b = __floats2bfloat162_rn(p[4 * j + 2], p[4 * j + 3]);
        uint2 q;
        memcpy(&q.x, &a, 4);
        memcpy(&q.y, &b, 4);
        __stcs(reinterpret_cast<uint2*>(t.copy + i), q);
      }
      if constexpr (BITS8) {
        __stcs(reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.m) + i),
               mc[0] | mc[1] << 8 | mc[2] << 16 | mc[3] << 24);
        __stcs(reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.v) + i),
               vc[0] | vc[1] << 8 | vc[2] << 16 | vc[3] << 24);
      } else {
        __stcs(reinterpret_cast<float4*>(static_cast<float*>(t.m) + i),
               make_float4(m[4 * j], m[4 * j + 1], m[4 * j + 2], m[4 * j + 3]));
        __stcs(reinterpret_cast<float4*>(static_cast<float*>(t.v) + i),
               make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (i + c < n) {
          t.p[i + c] = p[4 * j + c];
          if (t.copy) t.copy[i + c] = __float2bfloat16_rn(p[4 * j + c]);
          if constexpr (BITS8) {
            static_cast<uint8_t*>(t.m)[i + c] = static_cast<uint8_t>(mc[c]);
            static_cast<uint8_t*>(t.v)[i + c] = static_cast<uint8_t>(vc[c]);
          } else {
            static_cast<float*>(t.m)[i + c] = m[4 * j + c];
            static_cast<float*>(t.v)[i + c] = v[4 * j + c];
          }
        }
    }
  }
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
