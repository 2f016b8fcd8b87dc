"""The product's kernels one by one: sizes that the host's plan sends to every
instance of the stream and the tile kernel, with more steps of K than a wave
has in flight, and to the join of parts of K (test_operator_paths_host.py
asserts that they go there). GPU only."""
from functools import lru_cache

import numpy as np
import pytest
import torch

import nvfp4_adaptive_block_amd as fos
import operator_reference as ref
from operator_reference import DTYPES, assert_within, decode_nvfp4, gen
from test_gpu_operators import (assert_guard, check_balance, cuda, grouped_reference, guarded, make_w, make_x)

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "fp16", "e4m3", "nvfp4_row"]

# (row tiles, column tiles of a stream workgroup): M, N, K
STREAM = {(1, 1): (1, 70, 8336), (2, 1): (24, 70, 8336), (3, 1): (40, 70, 2192), (4, 1): (63, 70, 2192),
          (1, 2): (9, 7190, 4240), (2, 2): (24, 7190, 4240), (3, 2): (40, 7190, 2192), (4, 2): (63, 7190, 2192),
          (1, 4): (16, 14350, 2192), (2, 4): (24, 14350, 2192), (3, 4): (40, 14350, 2192), (4, 4): (63, 14350, 2192)}
# the same by group: offsets, N, K (the last rows are the tail's)
FEW, SOME, MANY = [5, 5, 30, 31, 47] + [60 + 5 * i for i in range(18)] + [148], [20, 21, 60, 100, 100, 139], [33, 33, 110, 149]
GROUPED = {(1, 1): (FEW, 70, 8336), (1, 2): (FEW, 300, 4240), (1, 4): (FEW, 500, 2192), (2, 1): (SOME, 70, 8336),
           (2, 2): (SOME, 1000, 4240), (2, 4): (SOME, 2000, 2192), (3, 1): (MANY, 70, 2192),
           (3, 2): (MANY, 1000, 2192), (3, 4): (MANY, 2000, 2192)}
GROUPED_ROWS = 150
# (rows of a tile, parts of K): M, N, K
TILES = {(64, 1): (2050, 1500, 528), (128, 1): (4100, 3000, 528), (64, 8): (150, 2051, 4208), (128, 5): (4100, 515, 4112)}
# rows of a tile: offsets, M, N, K
GROUPED_TILES = {64: ([100, 100, 390], 400, 300, 656), 128: ([4101, 8100], 8200, 1300, 528)}


@lru_cache(maxsize=2)
def weight(N, K, gran="tensor", G=None):
    return make_w(N, K, N + K, gran, G)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", STREAM.values())
def test_stream_instances(M, N, K, kind):
    x, xv, xg = make_x(kind, M, K, M + 1)
    w, wv = weight(N, K, "row")
    y, raw = guarded((M, N), torch.float32)
    fos.fos_linear(x, w, out=y, x_gran=xg, w_gran="row")
    want, bound = ref.linear(xv.cuda(), wv.cuda())
    assert_within(y, want.cpu(), bound.cpu(), f"{kind} {M}x{N}x{K}")
    assert_guard(raw)
    again = fos.fos_linear(x, w, out_dtype=torch.float32, x_gran=xg, w_gran="row")
    assert torch.equal(again, y)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("offs,N,K", GROUPED.values())
def test_grouped_stream_instances(offs, N, K, kind):
    M, G = GROUPED_ROWS, len(offs)
    x, xv, xg = make_x(kind, M, K, 5)
    w, wv = weight(N, K, "group", G)
    bias = torch.randn(G, N, generator=gen(6))
    y, raw = guarded((M, N), torch.float32)
    fos.fos_linear_grouped(x, w, torch.tensor(offs, dtype=torch.int32).cuda(), bias=cuda(bias), act="silu", out=y,
                           x_gran=xg, w_gran="group")
    want, bound = grouped_reference(xv, wv, offs, M, N, bias, "silu", None, torch.float32)
    assert_within(y, want, bound, f"{kind} {offs} {N}x{K}")
    assert_guard(raw)


def epilogues(x, xv, xg, w, wv, M, offs=None):
    """Every activation, and over them every output and bias type, after the
    products of one size. (The references are 64-bit products on the device.)"""
    N, K = wv.shape[-2:]
    xv, wv = xv.cuda(), wv.cuda()
    # sums around the activations' bend; a power of two, so that the weight's scale stays exact
    scale = 2.0 ** torch.log2(3.0 / (xv[:64] @ wv.view(-1, K)[:256].T).abs().mean()).round().item()
    w, wv = (w[0], w[1], w[2] * scale), wv * scale
    for i, act in enumerate(["none", "relu", "gelu", "gelu_tanh", "silu"]):
        for j, out in enumerate(["fp32", "bf16", "fp16"]):
            if M * N > 4e6 and (i + j) % 3:
                continue
            bias = res = None
            if (i + j) % 4:
                bias = torch.randn(*wv.shape[:-1], generator=gen(7)).to(DTYPES[["bf16", "fp16", "fp32"][(i + 2 * j) % 3]]).cuda()
            if (i + 2 * j) % 4:
                res = torch.randn(M, N, generator=gen(8)).to(DTYPES[out]).cuda()
            y, raw = guarded((M, N), DTYPES[out])
            if offs is None:
                fos.fos_linear(x, w, bias=bias, act=act, residual=res, out=y, x_gran=xg)
                want, bound = ref.linear(xv, wv, bias, act, res, DTYPES[out])
            else:
                o = torch.tensor(offs, dtype=torch.int32).cuda()
                fos.fos_linear_grouped(x, w, o, bias=bias, act=act, residual=res, out=y, x_gran=xg)
                want, bound = grouped_reference(xv, wv, offs, M, N, bias, act, res, DTYPES[out])
            assert_within(y, want.cpu(), bound.cpu(), f"{act} {out}, bias {bias is not None}, residual {res is not None}")
            assert_guard(raw)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", TILES.values())
def test_tile_epilogues(M, N, K, kind):
    epilogues(*make_x(kind, M, K, 11), *weight(N, K), M)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("offs,M,N,K", GROUPED_TILES.values())
def test_grouped_tile_epilogues(offs, M, N, K, kind):
    epilogues(*make_x(kind, M, K, 12), *weight(N, K, "tensor", len(offs)), M, offs)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("M,N,K", [*TILES.values(), STREAM[2, 2]])
def test_products_on_another_stream_and_in_a_graph(M, N, K, kind):
    x, _, xg = make_x(kind, M, K, 13)
    w, _ = weight(N, K)
    values = x if kind == "bf16" else x[1]  # what the replays change: the activations, or their scales
    y = fos.fos_linear(x, w, x_gran=xg)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        z = fos.fos_linear(x, w, x_gran=xg)
    s.synchronize()
    assert torch.equal(y, z)
    out = torch.empty_like(y)
    ws = torch.empty(max(1, fos.fos_linear_workspace(M, N, K)), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fos.fos_linear(x, w, out=out, workspace=ws, x_gran=xg)
    for k in range(4):
        values.mul_(0.5)
        out.fill_(float("nan"))
        ws.fill_(255)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, fos.fos_linear(x, w, x_gran=xg)), k


# more rows than the workgroups' first two turns, and the widest row
@pytest.mark.parametrize("T,E,k,dt", [(32769, 64, 4, "bf16"), (70001, 60, 2, "fp32"), (33000, 1024, 8, "fp16"),
                                      (300, 1024, 2, "fp32"), (40, 1024, 3, "bf16"), (200000, 3, 1, "fp32")])
def test_balance_of_many_tokens_and_experts(T, E, k, dt):
    logits = (torch.randn(T, E, generator=gen(T + E)) * 2).to(DTYPES[dt])
    idx = logits.float().topk(k, 1).indices
    check_balance(logits, idx, None, align=1)
    mask = torch.rand(T, generator=gen(E)) < 0.9
    check_balance(logits, idx.int(), mask)


@pytest.mark.parametrize("T,E", [(3000, 1000), (40000, 33)])
def test_balance_joins_the_same_columns_every_time(T, E):
    """The second launch's workgroups hand their columns to the one that ends
    last: two hundred calls on one workspace, other launches between them."""
    logits = torch.randn(2, T, E, generator=gen(T)).cuda()
    idx = logits.topk(2, 2).indices
    ws = torch.empty(fos.fos_balance_workspace(T, E), dtype=torch.uint8, device="cuda")
    want = [fos.fos_balance_loss(logits[i], idx[i]) for i in range(2)]
    for i in range(2):
        check_balance(logits[i].cpu(), idx[i].cpu(), None)
    got = [fos.fos_balance_loss(logits[k % 2], idx[k % 2], workspace=ws) for k in range(200)]
    for k, outs in enumerate(got):
        for a, b in zip(outs, want[k % 2]):
            assert torch.equal(a, b), k


def test_balance_sums_long_columns_in_64_bits():
    """2^24 rows of the same two logits, all sent to the first expert: the loss is
    2 coef p. p is off by the exponential's argument (half a step of |v|), exp, a
    sum and a division; in binary32 are 64 additions of rows, two of lanes, and the
    roundings of a workgroup's sum and of the loss, half a step each."""
    T, v = 2 ** 24, 2.9
    logits = torch.tensor([v, 0.0]).expand(T, 2).contiguous().cuda()
    idx = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    loss, counts, *_ = fos.fos_balance_loss(logits, idx, coef=0.5, align=1)
    assert counts.tolist() == [T, 0]
    p = 1 / (1 + np.exp(-float(np.float32(v))))
    assert abs(float(loss) / p - 1) <= (2 * v + 8 + 2 + 64 + 2 + 2) * 2.0 ** -24
