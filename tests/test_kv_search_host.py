"""Searches of the key/value cache's kernels on the CPU: the device functions as they
stand in the sources, compiled for the host with every thread as a fiber.

The eviction's: a wave runs as far as it can before the next one gets a turn, in a given
order of the waves, so a word of LDS that one wave writes while another still has to read
it is read wrong here every time. The moves found have to be those of a plain search.

Those for a tile's or a token's sequence: every row in one tile, and no offsets, bad
ones among them, that lead out of the rows."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

from operator_reference import gen

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "nvfp4_adaptive_block_amd", "csrc")
EVICT = (r"constexpr int kThreads = 1024.*?;\n", r"__device__ __forceinline__ uint32_t order_of.*?\n}\n",
         r"struct Digit \{.*?\n};\n", r"template <int BINS>\n__device__ Digit find_digit.*?\n}\n",
         r"template <int BATCH>\n__device__ int find_moves.*?\n}\n")
ROWS = (r"struct GroupTile \{.*?\n};\n", r"template <int ROWS>\n__device__ __forceinline__ GroupTile search_group_tile.*?\n}\n",
        r"__device__ __forceinline__ int first_end_behind.*?\n}\n")
HOST = """
#include <stdint.h>
#include <string.h>
#include <ucontext.h>
#include <algorithm>
#include <vector>
#define __device__
#define __forceinline__ inline
using std::max;
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
int __builtin_amdgcn_readlane(int v, int lane) {
  const int t = threadIdx.x;
  given[t] = v;
  wait_as(kAtWave);
  const int got = given[t / kLanes * kLanes + lane];
  wait_as(kAtWave);
  return got;
}
int __ffsll(unsigned long long v) { return __builtin_ffsll(v); }
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

void start(int threads, void (*run)()) {
  for (int t = 0; t < threads; t++) {
    Fiber& f = fibers[t];
    f.stack.resize(32768);
    getcontext(&f.at);
    f.at.uc_stack.ss_sp = f.stack.data();
    f.at.uc_stack.ss_size = f.stack.size();
    f.at.uc_link = &scheduler;
    makecontext(&f.at, run, 0);
    f.state = kRuns;
  }
}
bool all(int from, int to, State s) {
  for (int t = from; t < to; t++)
    if (fibers[t].state != s) return false;
  return true;
}
// One wave as far as it can; whether any lane ran.
bool run_wave(int first) {
  bool ran = false;
  if (all(first, first + kLanes, kAtWave))
    for (int t = first; t < first + kLanes; t++) fibers[t].state = kRuns;
  for (int t = first; t < first + kLanes; t++)
    if (fibers[t].state == kRuns) {
      ran = true;
      threadIdx.x = t;
      swapcontext(&scheduler, &fibers[t].at);
    }
  return ran;
}
void done() {
  const int t = threadIdx.x;
  fibers[t].state = kDone;
  swapcontext(&fibers[t].at, &scheduler);
}
"""
EVICT_HOST = """
KvEvictArgs args;
Cut cut;
int hist[2048], share[2 * kWaves + 4], holes[kAll], batch;
void thread() {
  const int t = threadIdx.x;
  holes[t] = batch == 8 ? find_moves<8>(args, cut, hist, share) : find_moves<32>(args, cut, hist, share);
  done();
}

// The number of moves; -1 where waves wait for each other for good or differ in it.
extern "C" int search(int n, int budget, int sinks, int recent, float* acc, int* moves, int of_batch, const int* order) {
  args = KvEvictArgs{budget, sinks, recent};
  cut = Cut{n, acc, (int2*)moves};
  batch = of_batch;
  for (int& s : share) s = -12345;
  start(kAll, thread);
  while (!all(0, kAll, kDone)) {
    bool ran = false;
    for (int i = 0; i < kAll / kLanes && !ran; i++) ran = run_wave(order[i] * kLanes);
    if (ran) continue;
    if (!all(0, kAll, kAtBarrier)) return -1;
    for (Fiber& f : fibers) f.state = kRuns;
  }
  for (int t = 1; t < kAll; t++)
    if (holes[t] != holes[0]) return -1;
  return holes[0];
}
"""
ROWS_HOST = """
const int32_t *offs, *values;
int groups, rows, tile, per, shift, token;
GroupTile found[kLanes];
int first[kLanes];
void thread() {
  const int t = threadIdx.x;
  found[t] = shift == 4 ? search_group_tile<4>(offs, groups, rows, tile, per, values)
                        : search_group_tile<7>(offs, groups, rows, tile, per, values);
  first[t] = first_end_behind(offs, groups, token);
  done();
}
// start, end, group, tile and value of a tile; the first end behind a token. false: lanes differ.
extern "C" bool search(const int32_t* o, const int32_t* v, int G, int M, int of_tile, int of_per, int of_shift, int of_token,
                       int* out) {
  offs = o, values = v, groups = G, rows = M, tile = of_tile, per = of_per, shift = of_shift, token = of_token;
  start(kLanes, thread);
  for (int turns = 0; !all(0, kLanes, kDone); turns++)
    if (turns > 1000 || !run_wave(0)) return false;
  for (int t = 1; t < kLanes; t++)
    if (first[t] != first[0] || memcmp(&found[t], &found[0], sizeof found[0])) return false;
  memcpy(out, &found[0], sizeof found[0]);
  out[5] = first[0];
  return true;
}
"""


def build(folder, source, parts, host):
    text = open(os.path.join(CSRC, source)).read()
    found = [re.search(p, text, re.S) for p in parts]
    assert all(found), "the search's functions are not where they were"
    source, lib = str(folder / "search.cpp"), str(folder / "search.so")
    with open(source, "w") as f:
        f.write(HOST + "\n".join(p.group(0) for p in found) + host)
    subprocess.run(["g++", "-std=c++17", "-O1", "-w", "-shared", "-fPIC", source, "-o", lib], check=True)
    return ctypes.CDLL(lib).search


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return build(tmp_path_factory.mktemp("evict"), "fos_kv.hip", EVICT, EVICT_HOST)


@pytest.fixture(scope="module")
def rows_host(tmp_path_factory):
    search = build(tmp_path_factory.mktemp("rows"), "fos_rows.h", ROWS, ROWS_HOST)
    search.restype = ctypes.c_bool
    return search


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


def tile_of(search, offs, values, M, tile, per, shift, token=0):
    out = (ctypes.c_int * 6)()
    o, v = ((ctypes.c_int * len(t))(*t) for t in (offs, values))
    assert search(o, v, len(offs), M, tile, per, shift, token, out), (tile, token)
    return list(out)


@pytest.mark.parametrize("shift", [4, 7])
@pytest.mark.parametrize("per", [1, 3, 40])
@pytest.mark.parametrize("G", [1, 2, 63, 64, 65, 128, 129, 700])
def test_every_row_is_in_one_tile(rows_host, G, per, shift):
    g = gen(G + per)
    kind = torch.rand(G, generator=g)
    new = torch.where(kind < 0.5, 0, torch.where(kind < 0.9, 1, torch.randint(0, 80, (G,), generator=g)))
    new[G // 2:G // 2 + 70] = 0  # a long run of groups without rows
    new[-1] = 1
    offs = new.cumsum(0).tolist()
    M = offs[-1] + 5
    values = torch.randint(0, 1000, (G,), generator=g).tolist()
    starts, ends = [0] + offs, offs + [M]
    want = {(b, t) for b in range(G + 1) for t in range(-(-((ends[b] - starts[b]) * per) >> shift))}
    got = []
    for tile in range((M * per >> shift) + G + 1):
        start, end, b, t, value, _ = tile_of(rows_host, offs, values, M, tile, per, shift)
        if b >= 0:
            assert (start, end, value) == (starts[b], ends[b], values[b] if b < G else 0)
            got.append((b, t))
    assert len(got) == len(want) and set(got) == want


@pytest.mark.parametrize("G", [1, 2, 63, 64, 65, 700, 5000])
def test_the_sequence_of_a_token(rows_host, G):
    new = torch.randint(0, 3, (G,), generator=gen(G))
    offs = new.cumsum(0).tolist()
    M = offs[-1] + 3
    for token in sorted({0, 1, M // 3, M // 2, M - 4, M - 3, M - 1} & set(range(M))):
        want = next((b for b, e in enumerate(offs) if e > token), G)
        assert tile_of(rows_host, offs, [0] * G, M, 0, 1, 4, token)[5] == want


@pytest.mark.parametrize("G", [1, 2, 64, 65, 300])
def test_bad_offsets_lead_nowhere(rows_host, G):
    """Any numbers: the search ends, with rows that there are and a group that there is."""
    g, M, per = gen(G), 500, 3
    for kind in range(4):
        offs = torch.randint(-2 ** 31, 2 ** 31, (G,), generator=g) if kind else torch.randint(-20, 600, (G,), generator=g)
        if kind == 2:
            offs = offs.sort().values
        if kind == 3:
            offs = offs.sort(descending=True).values
        for tile in range(0, (M * per >> 4) + G + 1, 7):
            start, end, b, t, _, first = tile_of(rows_host, offs.tolist(), [0] * G, M, tile, per, 4, tile % M)
            assert b == -1 or (0 <= b <= G and 0 <= start < end <= M and 0 <= t and 16 * t < (end - start) * per)
            assert 0 <= first <= G
