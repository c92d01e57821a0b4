"""A dense product's producer whose operand may be copied ahead of the grid wait: it comes to that wait before any
bounded one, so that no limit runs while the kernel before still does; and it copies what another producer copies, in
the same order.  The producer's source is compiled for the host, its instructions are noted instead of issued."""
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "precision_moe_grouped_gb300", "csrc")

HEAD = r"""
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
using std::min; using std::max;
#define __device__
#define __host__
#define __forceinline__ inline
struct { int x = 0; } threadIdx;
struct CUtensorMap { int id; };
constexpr int32_t kDevTimeout = 1;
void note(const char* what, int a = 0, int b = 0, int c = 0) { std::printf("%s %d %d %d\n", what, a, b, c); }
uint64_t* bars;
uint32_t cluster_addr(const void* p, uint32_t) { return uint32_t((uint64_t*)p - bars) * 8; }
void griddep_wait() { note("grid"); }
bool mbar_wait_warp(uint64_t* b, uint32_t parity, uint64_t, int32_t*, int32_t, volatile int32_t*) {
  note("wait", int(b - bars), int(parity));
  return true;
}
void mbar_arrive_expect_tx(uint64_t* b, uint32_t n) { note("expect", int(b - bars), int(n)); }
uint8_t* memory;
void tma_load_2d_pair(void* dst, const CUtensorMap*, int x, int y, uint32_t) { note("load", int((uint8_t*)dst - memory), x, y); }
struct Args {};
"""
MAIN = r"""
int main(int, char** v) {
  const int stages = atoi(v[1]), early = atoi(v[2]), rank = atoi(v[3]), kb = atoi(v[4]), tiles = atoi(v[5]);
  uint64_t bar[64];
  uint8_t mem[16];
  bars = bar; memory = mem;
  Maps maps = {};
  Launch<Args> l = {};
  l.problems = 1; l.tiles = tiles; l.stages = stages; l.slot = 32768;
  Problem& p = l.p[0];
  p.bn = p.b_step = 256; p.b_rank = 128; p.tiles_m = 1; p.tiles_n = tiles; p.per_matrix = tiles; p.splits = 1;
  p.kb = p.kb_split = kb;
  int32_t none = 0;
  if (early) produce<true, true>(maps, l, mem, bar, bar + kMaxStages, rank, 0, 1, &none);
  else produce<true, false>(maps, l, mem, bar, bar + kMaxStages, rank, 0, 1, &none);
}
"""


def cut(text, start):
    """From `start` to the end of its braces, and a semicolon."""
    i = text.index(start)
    depth, at = 0, text.index("{", i)
    for k in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[k], 0)
        if depth == 0:
            return text[i:k + 1] + (";" if text[k + 1] == ";" else "")
    raise AssertionError("unbalanced")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    text = open(os.path.join(CSRC, "dense.cuh")).read()
    constants = "\n".join(re.findall(r"^constexpr int \w+ = [^;]*;", text, re.M))
    parts = [cut(text, s) for s in ("template <int N>\nstruct MapList", "struct Problem {", "struct Tile {",
                                    "template <typename Args>\nstruct Launch {", "template <typename L>\n__device__ __forceinline__ Tile",
                                    "template <bool IS_A, bool EARLY, class L>\n__device__ __forceinline__ void produce")]
    parts.insert(1, "using Maps = MapList<kMaxMaps>;")
    source = HEAD + re.sub(r"asm volatile\(.*?\);", "", constants + "\n" + "\n".join(parts))
    source = re.sub(r"#pragma unroll[^\n]*", "", source)
    d = tmp_path_factory.mktemp("producer")
    exe = str(d / "a")
    subprocess.run(["g++", "-std=c++17", "-x", "c++", "-", "-o", exe], input=source + MAIN, text=True, check=True)

    def run(*args):
        out = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, check=True).stdout
        return [(w, *map(int, n)) for w, *n in (line.split() for line in out.splitlines())]

    return run


@pytest.mark.parametrize("stages", [6, 9])
@pytest.mark.parametrize("rank", [0, 1])
@pytest.mark.parametrize("kb,tiles", [(1, 1), (2, 2), (3, 2), (9, 1), (10, 1), (5, 7), (64, 3), (1, 0)])
def test_no_bounded_wait_ahead_of_the_grid_wait(program, stages, rank, kb, tiles):
    late, early = program(stages, 0, rank, kb, tiles), program(stages, 1, rank, kb, tiles)
    copies = lambda events: [e for e in events if e[0] in ("load", "expect")]        # noqa: E731
    assert copies(early) == copies(late) and sum(e[0] == "load" for e in early) == kb * tiles
    grid = [i for i, e in enumerate(early) if e[0] == "grid"]
    assert len(grid) == 1
    assert not any(e[0] == "wait" for e in early[:grid[0]])
    # as many copies ahead as there are slots, and behind it the waits of the other producer
    assert sum(e[0] == "load" for e in early[:grid[0]]) == min(stages, kb * tiles)
    assert not any(e[0] == "grid" for e in late)                                      # (the kernel has waited)
    waits = [e for e in late if e[0] == "wait"]
    assert [e for e in early if e[0] == "wait"] == waits[min(stages, kb * tiles):]
