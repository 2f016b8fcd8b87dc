"""Which kernel a product's size takes, asked of the host's plan: the sizes of
test_gpu_operator_paths.py reach every instance, and more steps of K than a wave
has in flight. Also the plan's own bounds."""
import ctypes
import os
import subprocess

import pytest

import test_gpu_operator_paths as paths

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """
#include "fos_plan.h"
extern "C" void plan(int64_t M, int64_t N, int64_t K, int64_t G, int64_t* out) {
  const fos::Plan p = fos::plan(M, N, K, G);
  const int nt = fos::stream_columns(p.m_tiles, N);
  out[0] = p.stream, out[1] = p.bm, out[2] = p.splits, out[3] = p.m_tiles, out[4] = nt;
  out[5] = fos::stream_waves(p.bm / 16, nt) * fos::stream_depth(p.bm / 16, nt);
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "nvfp4_adaptive_block_amd", "csrc"), str(d / "plan.cpp"), "-o",
                    str(d / "plan.so")], check=True)
    fn = ctypes.CDLL(str(d / "plan.so")).plan
    fn.argtypes = [ctypes.c_int64] * 4 + [ctypes.POINTER(ctypes.c_int64)]

    def ask(M, N, K, G=0):
        out = (ctypes.c_int64 * 6)()
        fn(M, N, K, G, out)
        return dict(zip(("stream", "bm", "splits", "m_tiles", "nt", "in_flight"), out))
    return ask


def reaches_stream(p, K, mt, nt):
    """Two full turns of every wave's stages, and a part of a step."""
    return p["stream"] and (p["bm"], p["nt"]) == (16 * mt, nt) and K // 128 > 2 * p["in_flight"] and K % 128


def test_every_stream_instance_is_tested(plan):
    assert set(paths.STREAM) == {(mt, nt) for mt in (1, 2, 3, 4) for nt in (1, 2, 4)}
    for (mt, nt), (M, N, K) in paths.STREAM.items():
        assert reaches_stream(plan(M, N, K), K, mt, nt), (mt, nt)
        assert M % 16 or mt == 1
        assert N % (16 * nt)


def test_every_grouped_stream_instance_is_tested(plan):
    assert set(paths.GROUPED) == {(mt, nt) for mt in (1, 2, 3) for nt in (1, 2, 4)}
    for (mt, nt), (offs, N, K) in paths.GROUPED.items():
        assert offs == sorted(offs) and offs[-1] < paths.GROUPED_ROWS  # a tail of zeros
        assert reaches_stream(plan(paths.GROUPED_ROWS, N, K, len(offs)), K, mt, nt), (mt, nt)


def test_every_tile_form_is_tested(plan):
    for (bm, splits), (M, N, K) in paths.TILES.items():
        p = plan(M, N, K)
        assert (p["stream"], p["bm"], p["splits"]) == (0, bm, splits), (M, N, K, p)
        assert K % 128 and N % 256 and M % bm
    assert {bm for bm, s in paths.TILES if s == 1} == {bm for bm, s in paths.TILES if s > 1} == {64, 128}
    for bm, (offs, M, N, K) in paths.GROUPED_TILES.items():
        p = plan(M, N, K, len(offs))
        assert (p["stream"], p["bm"], p["splits"]) == (0, bm, 1), (M, N, K, p)
    assert set(paths.GROUPED_TILES) == {64, 128}


def test_plans_are_complete(plan):
    """Over a spread of sizes: tiles cover the rows of any groups, and no more
    than eight parts of K with two steps each."""
    for M in (1, 15, 16, 17, 48, 64, 65, 129, 1000, 70000):
        for N in (1, 255, 4096, 14336):
            for K in (16, 144, 4096):
                for G in (0, 1, 3, 64, 5000):
                    p = plan(M, N, K, G)
                    assert p["bm"] in ((16, 32, 48, 64) if p["stream"] else (64, 128))
                    parts = min(G + 1, M) if G else 1
                    # one row in each part but one, which has the rest
                    worst = parts - 1 + -(-(M - parts + 1) // p["bm"])
                    assert p["m_tiles"] >= worst
                    assert 1 <= p["splits"] <= 8 and (p["splits"] == 1 or (not G and K // 128 >= 2 * p["splits"]))
