"""The eviction's search on the CPU: the device functions as they stand in
fos_kv.hip, compiled for the host with every thread of a workgroup as a fiber. A
wave runs as far as it can before the next one gets a turn, in a given order of the
waves, so a word of LDS that one wave writes while another still has to read it is
read wrong here every time. The moves found have to be those of a plain search."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

from operator_reference import gen

HERE = os.path.dirname(os.path.abspath(__file__))
KERNELS = os.path.join(os.path.dirname(HERE), "nvfp4_adaptive_block_amd", "csrc", "fos_kv.hip")
PARTS = (r"constexpr int kThreads = 1024.*?;\n", r"__device__ __forceinline__ uint32_t order_of.*?\n}\n",
         r"struct Digit \{.*?\n};\n", r"template <int BINS>\n__device__ Digit find_digit.*?\n}\n",
         r"template <int BATCH>\n__device__ int find_moves.*?\n}\n")
HOST = """
#include <stdint.h>
#include <string.h>
#include <ucontext.h>
#include <algorithm>
#include <vector>
#define __device__
#define __forceinline__ inline
using std::min;
struct int2 { int x, y; };
struct Index { int x; } threadIdx;
struct KvEvictArgs { int budget, sinks, recent; };
struct Cut { int n; float* acc; int2* moves; };

constexpr int kLanes = 64, kAll = 1024;
enum State { kRuns, kAtWave, kAtBarrier, kDone };
struct Fiber { ucontext_t at; State state; std::vector<char> stack; };
Fiber fibers[kAll];
ucontext_t scheduler;
unsigned long long voted[kAll / kLanes];
int given[kAll], wave_sum[kAll];
void wait_as(State s) {
  const int t = threadIdx.x;
  fibers[t].state = s;
  swapcontext(&fibers[t].at, &scheduler);
  threadIdx.x = t;
}
void __syncthreads() { wait_as(kAtBarrier); }
// Operations over a wave: what each lane gives is seen by all once all have come here.
int wave_scan(int v) {
  const int t = threadIdx.x;
  given[t] = v;
  wait_as(kAtWave);
  int sum = 0;
  for (int i = t / kLanes * kLanes; i <= t; i++) sum += given[i];
  wait_as(kAtWave);
  return sum;
}
unsigned long long __ballot(int v) {
  const int t = threadIdx.x;
  given[t] = v != 0;
  wait_as(kAtWave);
  unsigned long long m = 0;
  for (int i = 0; i < kLanes; i++) m |= (unsigned long long)given[t / kLanes * kLanes + i] << i;
  wait_as(kAtWave);
  return m;
}
int __popcll(unsigned long long v) { return __builtin_popcountll(v); }
int atomicAdd(int* p, int v) { const int old = *p; *p += v; return old; }
uint32_t __float_as_uint(float v) { uint32_t u; memcpy(&u, &v, 4); return u; }
float __uint_as_float(uint32_t u) { float v; memcpy(&v, &u, 4); return v; }
struct Rsrc { const float* at; int bytes; };
Rsrc __builtin_amdgcn_make_buffer_rsrc(float* p, short, int bytes, int) { return Rsrc{p, bytes}; }
uint32_t __builtin_amdgcn_raw_buffer_load_b32(Rsrc r, int at, int, int) {
  return at + 4 <= r.bytes ? __float_as_uint(r.at[at / 4]) : 0u;
}
uint32_t __builtin_amdgcn_mbcnt_lo(uint32_t m, uint32_t v) {
  const int lane = threadIdx.x % kLanes;
  return v + __builtin_popcount(lane >= 32 ? m : m & ((1u << lane) - 1));
}
uint32_t __builtin_amdgcn_mbcnt_hi(uint32_t m, uint32_t v) {
  const int lane = threadIdx.x % kLanes;
  return v + (lane > 32 ? __builtin_popcount(m & ((1u << (lane - 32)) - 1)) : 0);
}

SEARCH

KvEvictArgs args;
Cut cut;
int hist[2048], share[2 * kWaves + 4], holes[kAll], batch;
void thread() {
  const int t = threadIdx.x;
  holes[t] = batch == 8 ? find_moves<8>(args, cut, hist, share) : find_moves<32>(args, cut, hist, share);
  fibers[t].state = kDone;
  swapcontext(&fibers[t].at, &scheduler);
}

// The number of moves; -1 where waves wait for each other for good or differ in it.
extern "C" int search(int n, int budget, int sinks, int recent, float* acc, int* moves, int of_batch, const int* order) {
  args = KvEvictArgs{budget, sinks, recent};
  cut = Cut{n, acc, (int2*)moves};
  batch = of_batch;
  for (int& s : share) s = -12345;
  for (int t = 0; t < kAll; t++) {
    Fiber& f = fibers[t];
    f.stack.resize(32768);
    getcontext(&f.at);
    f.at.uc_stack.ss_sp = f.stack.data();
    f.at.uc_stack.ss_size = f.stack.size();
    f.at.uc_link = &scheduler;
    makecontext(&f.at, thread, 0);
    f.state = kRuns;
  }
  auto all = [&](int from, int to, State s) {
    for (int t = from; t < to; t++)
      if (fibers[t].state != s) return false;
    return true;
  };
  while (!all(0, kAll, kDone)) {
    bool ran = false;
    for (int i = 0; i < kAll / kLanes && !ran; i++) {
      const int first = order[i] * kLanes;
      if (all(first, first + kLanes, kAtWave))
        for (int t = first; t < first + kLanes; t++) fibers[t].state = kRuns;
      for (int t = first; t < first + kLanes; t++)
        if (fibers[t].state == kRuns) {
          ran = true;
          threadIdx.x = t;
          swapcontext(&scheduler, &fibers[t].at);
        }
    }
    if (ran) continue;
    if (!all(0, kAll, kAtBarrier)) return -1;
    for (Fiber& f : fibers) f.state = kRuns;
  }
  for (int t = 1; t < kAll; t++)
    if (holes[t] != holes[0]) return -1;
  return holes[0];
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    kernels = open(KERNELS).read()
    parts = [re.search(p, kernels, re.S) for p in PARTS]
    assert all(parts), "the search's functions are not where they were"
    folder = tmp_path_factory.mktemp("search")
    source, lib = str(folder / "search.cpp"), str(folder / "search.so")
    with open(source, "w") as f:
        f.write(HOST.replace("SEARCH", "\n".join(p.group(0) for p in parts)))
    subprocess.run(["g++", "-std=c++17", "-O1", "-w", "-shared", "-fPIC", source, "-o", lib], check=True)
    return ctypes.CDLL(lib).search


def plain(acc, n, budget, sinks, recent):
    """(from, to) of each move."""
    keep = budget - recent
    best = sorted(range(sinks, n - recent), key=lambda i: (math.isnan(acc[i]), -acc[i] if acc[i] == acc[i] else 0.0, i))
    kept = set(range(sinks)) | set(best[:keep - sinks])
    return list(zip((i for i in range(keep, n - recent) if i in kept), (i for i in range(keep) if i not in kept)))


def check(host, acc, n, budget, sinks, recent):
    want = plain(acc.tolist(), n, budget, sinks, recent)
    for batch in (8, 32):
        for order in (range(16), range(15, -1, -1), [5, 2, 0, 9, 1, 15, 3, 4, 6, 7, 8, 10, 11, 12, 13, 14]):
            moves = (ctypes.c_int * (2 * max(1, budget - recent)))()
            held = (ctypes.c_float * n)(*acc.tolist())
            got = host(n, budget, sinks, recent, held, moves, batch, (ctypes.c_int * 16)(*order))
            assert got == len(want), (batch, list(order))
            assert list(zip(moves[0:2 * got:2], moves[1:2 * got:2])) == want, (batch, list(order))


@pytest.mark.parametrize("n,budget,sinks,recent", [
    (2, 1, 0, 0), (20, 9, 0, 0), (80, 50, 4, 12), (132, 70, 4, 0), (200, 100, 10, 33), (1088, 1024, 4, 128),
    (1100, 600, 0, 100), (1700, 300, 4, 17)])
def test_distinct_weights(host, n, budget, sinks, recent):
    """Middles of one to many rows, without ties: waves whose stretch is empty run ahead."""
    acc = (torch.randperm(n, generator=gen(n)) + 1).float() * 2.0 ** -9
    check(host, acc, n, budget, sinks, recent)


@pytest.mark.parametrize("n,budget,sinks,recent", [(80, 50, 4, 12), (700, 300, 4, 50), (1700, 900, 4, 17)])
def test_equal_weights(host, n, budget, sinks, recent):
    """Ties that are cut: the lower index stays."""
    acc = torch.randint(0, 5, (n,), generator=gen(n + 1)).float()
    acc[::7], acc[3::11] = math.nan, -math.inf
    check(host, acc, n, budget, sinks, recent)
