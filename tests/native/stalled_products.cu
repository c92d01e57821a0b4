// The dense products' kernels with an epilogue that stalls for longer than the
// waits' limit, so that the MMA issuer's and the producers' bounded waits run out: the
// status word is set, every role leaves, and the kernel ends.  No copy is in flight by
// then (they take microseconds, the limit is a millisecond or more), no address is out
// of range, and the stall itself is bounded.
#include <cstdio>

#include "dense.cuh"
#include "terms.cuh"

namespace moe {

void set_last_error(const char* msg) { std::fprintf(stderr, "%s\n", msg); }

namespace {

struct EpiStall {
  struct Args {
    uint64_t stall_ns;
  };
  static __device__ __forceinline__ void stall(const Args& a) {
    const uint64_t t0 = globaltimer_ns();
    for (int i = 0; i < 1000000 && globaltimer_ns() - t0 < a.stall_ns; ++i) __nanosleep(1000);
    __syncwarp();
  }
  // dense.cuh
  static __device__ __forceinline__ void run(const Args& a, const dense::Problem&, const dense::Tile&, const dense::EpiWarp&,
                                             const dense::Maps&) {
    stall(a);
  }
  // terms.cuh
  static __device__ __forceinline__ void ahead(const Args&, const dense::Tile&, const dense::EpiWarp&, int, int) {}
  template <class M>
  static __device__ __forceinline__ void run(const Args& a, const dense::Tile&, const dense::EpiWarp&, int, int, const M&,
                                             float (&)[128]) {
    stall(a);
  }
};

constexpr int kRows = 6 * 256, kK = 512;   // six tiles for one pair, eight K blocks (four pieces)
constexpr int kSide = 512;                 // a chain's matrix: three units a pair of a cluster of eight

// Rows [2 rows][k] of fp16 in boxes of 64 x 64, as both operands of a product.
int32_t operands(CUtensorMap* m, int index, const void* at, int rows, int k, terms::Problem* p) {
  if (dense::make_map(m, at, dense::Elem::kF16, 2 * rows, k, k, 64, 64) != MOE_OK) return 1;
  p->a.map = p->b.map = index;
  p->a.lo = p->b.lo = rows;
  p->batch = p->splits = 1;
  p->kb = p->kb_split = k / dense::kBK;
  return 0;
}

int run(int which, void* mem, int32_t* status, uint64_t limit_ns, uint64_t stall_ns, int sms, cudaStream_t s) {
  int n;
  if (which == 0) {
    dense::Maps maps;
    dense::Launch<EpiStall::Args> l = {};
    if (dense::make_map(&maps.m[0], mem, dense::Elem::kBf16, kRows, kK, kK, dense::kBK, 128) != MOE_OK ||
        dense::make_map(&maps.m[1], mem, dense::Elem::kBf16, 256, kK, kK, dense::kBK, 128) != MOE_OK)
      return 1;
    l.status = status;
    l.timeout_ns = limit_ns;
    l.problems = 1;
    l.maps = 2;
    l.p[0] = dense::make_problem({256, 1, kK / dense::kBK}, kRows, 256, kK / dense::kBK, 0, false, 1, false);
    l.e[0].stall_ns = stall_ns;
    if (dense::resident_pairs<EpiStall>(sms, &n) != cudaSuccess) return 2;
    return dense::launch<EpiStall>(maps, l, 1, s) == cudaSuccess ? 0 : 3;
  }
  if (which == 1) {
    terms::Maps maps;
    terms::Launch<EpiStall::Args> l = {};
    l.status = status;
    l.timeout_ns = limit_ns;
    l.problems = 1;
    l.maps = 2;
    maps.m[0] = CUtensorMap{};
    if (operands(&maps.m[1], 1, mem, kRows, kK, &l.p[0])) return 1;
    l.p[0].tiles_m = l.p[0].per_matrix = kRows / 256;
    l.p[0].tiles_n = 1;
    l.e[0].stall_ns = stall_ns;
    if (terms::resident_pairs<EpiStall>(sms, &n) != cudaSuccess) return 2;
    return terms::launch<EpiStall>(maps, l, 1, s) == cudaSuccess ? 0 : 3;
  }
  terms::ChainMaps maps;
  terms::Chain<EpiStall::Args> l = {};
  l.status = status;
  l.timeout_ns = limit_ns;
  l.maps = 2;
  l.phases = l.problems = 2;
  l.groups = 1;
  l.mp[0] = kSide;
  l.end[0] = 1;
  l.end[1] = 2;
  maps.m[0] = CUtensorMap{};
  for (int i = 0; i < 2; ++i) {
    if (operands(&maps.m[1], 1, mem, kSide, kSide, &l.p[i])) return 1;
    l.e[i].stall_ns = stall_ns;
  }
  if (terms::resident_chains<EpiStall>(8, &n) != cudaSuccess || n < 1) return 2;
  return terms::launch_chain<EpiStall>(maps, l, 8, 1, s) == cudaSuccess ? 0 : 3;
}

}  // namespace
}  // namespace moe

// which: 0 dense_kernel, 1 terms_kernel, 2 chain_kernel; mem: 4 MB of zeros.
extern "C" int stalled_product(int which, void* mem, int32_t* status, uint64_t limit_ns, uint64_t stall_ns, int sms,
                               void* stream) {
  return moe::run(which, mem, status, limit_ns, stall_ns, sms, static_cast<cudaStream_t>(stream));
}
