"""The operators around the quantizer against plain 64-bit references: the
product with NVFP4 weights (dense, by group), the RMS norm with an 8-bit
output, the balance loss and its gradient. GPU only."""
import numpy as np
import pytest
import torch

import nvfp4_adaptive_block_amd as fos
import operator_reference as ref
from operator_reference import DTYPES, assert_within, decode_nvfp4, gen, random_nvfp4

pytestmark = pytest.mark.gpu
GUARD = 64  # elements on each side of an output that must stay untouched


def cuda(v):
    return v.to("cuda") if isinstance(v, torch.Tensor) else tuple(t.to("cuda") for t in v)


def guarded(shape, dtype):
    """A contiguous output inside a larger buffer, and that buffer."""
    n = int(np.prod(shape))
    raw = torch.full((n + 2 * GUARD,), 77.0, device="cuda").to(dtype)
    return raw[GUARD:GUARD + n].view(shape), raw


def assert_guard(raw):
    seven = torch.tensor(77.0).to(raw.dtype).float().item()
    edge = torch.cat((raw[:GUARD], raw[-GUARD:])).float().cpu()
    assert (edge == seven).all(), "wrote outside the output"


def make_x(kind, M, K, seed, groups=None):
    """(operand on the device, its float64 values on the CPU, x_gran)."""
    g = gen(seed)
    v = torch.randn(M, K, generator=g)
    if kind in DTYPES:
        x = v.to(DTYPES[kind])
        return cuda(x), x.double(), None
    if kind == "e4m3":
        q = (v * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
        s = torch.rand(M, generator=g) * 0.1 + 0.01
        return cuda((q, s)), q.double() * s.double()[:, None], "row"
    codes, scales = random_nvfp4(M, K, seed)
    if kind == "nvfp4_row":
        s = torch.rand(M, generator=g) * 0.1 + 0.01
        return cuda((codes, scales, s)), decode_nvfp4(codes, scales) * s.double()[:, None], "row"
    s = torch.rand(1, generator=g) * 0.1 + 0.01
    return cuda((codes, scales, s)), decode_nvfp4(codes, scales) * s.double(), "tensor"


def make_w(N, K, seed, gran="tensor", G=None):
    rows = N * (G or 1)
    codes, scales = random_nvfp4(rows, K, seed)
    n = {"tensor": 1, "row": rows, "group": G}[gran]
    s = torch.rand(n, generator=gen(seed + 1)) * 0.02 + 0.005
    per_row = {"tensor": lambda: s.expand(rows), "row": lambda: s, "group": lambda: s.repeat_interleave(N)}[gran]()
    w = decode_nvfp4(codes, scales) * per_row.double()[:, None]
    if G is not None:
        codes, scales, w = codes.view(G, N, -1), scales.view(G, N, -1), w.view(G, N, K)
    return cuda((codes, scales, s)), w


SIZES = [(1, 1, 16), (1, 16, 16), (2, 3, 32), (3, 5, 48), (5, 17, 112), (15, 16, 128), (16, 64, 144), (17, 33, 256),
         (31, 64, 272), (48, 96, 512), (40, 4128, 160), (33, 70, 1104), (20, 14400, 64),
         (40, 14400, 64), (64, 14388, 80), (2, 14403, 144), (150, 1030, 2128), (90, 520, 4096), (300, 4100, 400),
         (63, 65, 528), (64, 128, 1024), (65, 130, 1040), (100, 256, 384),
         (128, 257, 640), (129, 64, 1936), (200, 511, 256), (257, 300, 2064), (384, 512, 1024), (1, 64, 14336),
         (7, 40, 7168)]
KINDS = ["bf16", "fp16", "e4m3", "nvfp4", "nvfp4_row"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear_sizes(kind, M, N, K):
    x, xv, xg = make_x(kind, M, K, M + N + K)
    gran = "row" if (M + N) % 2 else "tensor"
    w, wv = make_w(N, K, M * 3 + N, gran)
    out_dtype = DTYPES[["fp32", "bf16", "fp16"][(M + K // 16) % 3]]
    y, raw = guarded((M, N), out_dtype)
    got = fos.fos_linear(x, w, out=y, x_gran=xg, w_gran=gran)
    assert got is y
    want, bound = ref.linear(xv, wv, out_dtype=out_dtype)
    if out_dtype == torch.float16:  # sums past fp16's range become infinities
        over = want.abs() > 65000
        assert torch.isinf(got.cpu()[want.abs() > 66000]).all()
        got, want, bound = got.cpu()[~over], want[~over], bound[~over]
    assert_within(got, want, bound, f"{kind} {M}x{N}x{K}")
    assert_guard(raw)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("out,bias_dt", [("fp32", "fp32"), ("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp16")])
@pytest.mark.parametrize("M,N,K", [(3, 37, 64), (48, 64, 256), (150, 264, 512)])
def test_linear_epilogue(act, out, bias_dt, M, N, K):
    x, xv, xg = make_x("fp16", M, K, 5)
    w, wv = make_w(N, K, 6)
    scale = 3.0 / float((xv @ wv.T).abs().mean())  # sums around the activations' bend
    w = (w[0], w[1], w[2] * scale)
    wv = decode_nvfp4(w[0].cpu(), w[1].cpu()) * w[2].double().cpu()
    bias = torch.randn(N, generator=gen(7)).to(DTYPES[bias_dt])
    res = torch.randn(M, N, generator=gen(8)).to(DTYPES[out])
    want, bound = ref.linear(xv, wv, bias, act, res, DTYPES[out])
    got = fos.fos_linear(x, w, bias=cuda(bias), act=act, residual=cuda(res), out_dtype=DTYPES[out])
    assert_within(got, want, bound, act)
    want, bound = ref.linear(xv, wv, None, act, None, DTYPES[out])
    assert_within(fos.fos_linear(x, w, act=act, out_dtype=DTYPES[out]), want, bound, act + " alone")
    # the residual may be the output itself
    y = cuda(res)
    fos.fos_linear(x, w, bias=cuda(bias), act=act, residual=y, out=y)
    want, bound = ref.linear(xv, wv, bias, act, res, DTYPES[out])
    assert_within(y, want, bound, act + " in place")


# sizes that are cut into tiles of 64 and of 128 rows, in one part of K and in several
TILED = [(2050, 1500, 528, False), (3000, 4099, 528, False), (150, 2051, 4208, True), (130, 1500, 3088, True),
         (4100, 515, 4112, True)]


@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3", "nvfp4_row"])
@pytest.mark.parametrize("M,N,K,parts", TILED)
def test_linear_tiles(kind, M, N, K, parts):
    assert (fos.fos_linear_workspace(M, N, K) > 0) == parts
    x, xv, xg = make_x(kind, M, K, M + N)
    w, wv = make_w(N, K, M + K, "row")
    bias = torch.randn(N, generator=gen(9))
    out_dtype = torch.float32 if kind != "bf16" else torch.bfloat16
    res = torch.randn(M, N, generator=gen(10)).to(out_dtype)
    y, raw = guarded((M, N), out_dtype)
    ws = torch.full((fos.fos_linear_workspace(M, N, K) + 16,), 255, dtype=torch.uint8, device="cuda")
    fos.fos_linear(x, w, out=y, bias=cuda(bias), residual=cuda(res), act="relu", x_gran=xg, w_gran="row", workspace=ws)
    want, bound = ref.linear(xv, wv, bias, "relu", res, out_dtype)
    assert_within(y, want, bound, f"{kind} {M}x{N}x{K}")
    assert_guard(raw)
    assert (ws[-16:] == 255).all(), "wrote past the workspace"
    z = cuda(res)  # in place of the residual, on a workspace that the last call left
    fos.fos_linear(x, w, out=z, bias=cuda(bias), residual=z, act="relu", x_gran=xg, w_gran="row", workspace=ws)
    assert torch.equal(z.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("M,N,K", [(0, 8, 32), (8, 0, 32), (5, 9, 0)])
def test_linear_empty(M, N, K):
    x = torch.ones(M, K, dtype=torch.bfloat16, device="cuda")
    w = (torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda"),
         torch.zeros(N, K // 16, dtype=torch.uint8, device="cuda"), torch.ones(1, device="cuda"))
    bias = torch.arange(N, dtype=torch.float32, device="cuda")
    y = fos.fos_linear(x, w, bias=bias, out_dtype=torch.float32)
    assert y.shape == (M, N)
    if M and N:
        assert torch.equal(y, bias.expand(M, N))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", [4, 40, 200])
def test_linear_keeps_nonfinite_values_in_their_row_and_column(kind, M):
    N, K = 70, 304
    x, xv, xg = make_x(kind, M, K, 21)
    w, wv = make_w(N, K, 22)
    want, bound = ref.linear(xv, wv)
    w[1][3, 1] = 0x7F  # a NaN block scale: column 3
    row = M - 2
    if kind in DTYPES:
        x[row, 5] = float("nan")
        x[0, 7] = float("inf")
    elif kind == "e4m3":
        x[0].view(torch.uint8)[row, 5] = 0x7F
    else:
        x[1][row, 2] = 0x7F
    y = fos.fos_linear(x, w, out_dtype=torch.float32, x_gran=xg).cpu()
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[row] = True
    bad[:, 3] = True
    assert torch.isnan(y[bad]).all()
    if kind in DTYPES:  # inf * w: an infinity, or NaN where the weight is 0
        assert not torch.isfinite(y[0]).any()
        bad[0] = True
    assert_within(y[~bad], want[~bad], bound[~bad])


def test_linear_small_and_large_scales():
    """fp16 subnormal activations count, and the scales' product is applied to
    the sum: neither a tiny nor a huge S_dec loses the result."""
    K = 256
    x = (torch.randn(20, K, generator=gen(1)) * 2 ** -20).half()
    codes, scales = random_nvfp4(24, K, 2)
    for s in (1e-30, 1.0, 1e30):
        sd = torch.tensor([s])
        wv = decode_nvfp4(codes, scales) * sd.double()
        want, bound = ref.linear(x.double(), wv)
        got = fos.fos_linear(cuda(x), cuda((codes, scales, sd)), out_dtype=torch.float32)
        assert_within(got, want, bound, f"S_dec {s}")


@pytest.mark.parametrize("block", ["1x16", "16x16"])
def test_linear_reads_what_the_quantizer_writes(block):
    """fos_quantize -> fos_linear against the decoded tensors, both operands
    quantized; and the backward product through the columnwise operand."""
    M, N, K = 64, 96, 320
    x = torch.randn(M, K, generator=gen(31)).bfloat16().cuda()
    w = (torch.randn(N, K, generator=gen(32)) * 0.02).bfloat16().cuda()
    knobs = dict(recipe="4over6", err_metric="mse")
    xq = fos.fos_quantize(x, fos.fos_amax(x, "row"), scale_gran="row", **knobs)
    wq = fos.fos_quantize(w, fos.fos_amax(w), block=block, **knobs)
    xd = decode_nvfp4(xq[0].cpu(), xq[1].cpu()) * xq[2].cpu().double()[:, None]
    wd = decode_nvfp4(wq[0].cpu(), wq[1].cpu()) * wq[2].cpu().double()
    want, bound = ref.linear(xd, wd)
    assert_within(fos.fos_linear(xq, wq, x_gran="row", out_dtype=torch.float32), want, bound)
    if block == "1x16":
        dy = torch.randn(M, N, generator=gen(33)).bfloat16().cuda()
        wt = fos.fos_quantize_columnwise(w, fos.fos_amax(w), **knobs)
        wtd = decode_nvfp4(wt[0].cpu(), wt[1].cpu()) * wt[2].cpu().double()
        want, bound = ref.linear(dy.cpu().double(), wtd)
        assert_within(fos.fos_linear(dy, wt, out_dtype=torch.float32), want, bound)


@pytest.mark.parametrize("M,N,K", [(5, 64, 512), (64, 512, 4096), (300, 256, 1024)])
def test_linear_repeats_bit_for_bit_on_another_stream_and_in_a_graph(M, N, K):
    x, _, xg = make_x("bf16", M, K, 41)
    w, _ = make_w(N, K, 42)
    y = fos.fos_linear(x, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        z = fos.fos_linear(x, w)
    s.synchronize()
    assert torch.equal(y, z)
    out = torch.empty_like(y)
    ws = torch.empty(max(1, fos.fos_linear_workspace(M, N, K)), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fos.fos_linear(x, w, out=out, workspace=ws)
    for k in range(4):
        x.mul_(0.5)
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, fos.fos_linear(x, w)), k


# ---------------------------------------------------------------- grouped


def grouped_reference(xv, wv, offs, M, N, bias, act, res, out_dtype):
    y, b = torch.zeros(M, N, dtype=torch.float64), torch.zeros(M, N, dtype=torch.float64)
    at = 0
    for g, end in enumerate(offs):
        end = min(max(end, at), M)
        if end > at:
            y[at:end], b[at:end] = ref.linear(xv[at:end], wv[g], None if bias is None else bias[g], act,
                                              None if res is None else res[at:end], out_dtype)
        at = end
    return y, b


GROUPS = [
    (1, 16, 32, [1]),
    (10, 17, 48, [0, 3, 3, 10]),
    (64, 48, 256, [0, 0, 64, 64]),
    (40, 64, 144, [16, 16, 32]),               # a tail of 8 rows
    (70, 33, 272, [1, 2, 40, 41, 41, 69]),
    (200, 64, 512, [130, 131, 199]),
    (600, 130, 256, [0, 257, 258, 600]),
    (30, 16, 64, list(range(0, 26, 1)) * 5),   # not monotone: see the test of bad offsets
    (16, 24, 64, [0] * 70 + [3] * 60 + [16]),  # more groups than a wave has lanes
    (5, 20, 128, [0, 0, 0]),                   # every row in the tail
    (300, 300, 400, [100, 100, 290]),          # tiles of 64 rows
    (8200, 1030, 272, [4101, 8100]),
    (8200, 4099, 528, [4101, 8100]),           # tiles of 128 rows
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("M,N,K,offs", GROUPS)
def test_grouped(kind, M, N, K, offs):
    G = len(offs)
    good = all(a <= b for a, b in zip([0] + offs, offs)) and offs[-1] <= M
    x, xv, xg = make_x(kind, M, K, 51)
    gran = ["tensor", "row", "group"][(M + G) % 3]
    w, wv = make_w(N, K, 52, gran, G)
    bias = torch.randn(G, N, generator=gen(53))
    res = torch.randn(M, N, generator=gen(54))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, raw = guarded((M, N), torch.float32)
    fos.fos_linear_grouped(x, w, torch.tensor(offs, dtype=torch.int32).cuda(), bias=cuda(bias), act="relu",
                           residual=cuda(res), out=y, x_gran=xg, w_gran=gran, status=status)
    run = np.maximum.accumulate(np.minimum(offs, M)).tolist()
    want, bound = grouped_reference(xv, wv, run, M, N, bias, "relu", res, torch.float32)
    assert_within(y, want, bound)
    assert_guard(raw)
    assert int(status.item()) == (0 if good else fos.STATUS_BAD_OFFS)


@pytest.mark.parametrize("offs", [[-5, 10], [10, 4], [8, 1000], [-7, -3], [2 ** 31 - 1, 2 ** 31 - 1], [20, -2 ** 31]])
def test_grouped_bad_offsets_are_clamped_and_reported(offs):
    M, N, K = 24, 32, 64
    x, xv, _ = make_x("bf16", M, K, 61)
    w, wv = make_w(N, K, 62, "tensor", 2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, raw = guarded((M, N), torch.float32)
    fos.fos_linear_grouped(x, w, torch.tensor(offs, dtype=torch.int32).cuda(), out=y, status=status)
    run = np.maximum.accumulate(np.clip(offs, 0, M)).tolist()
    want, bound = grouped_reference(xv, wv, run, M, N, None, "none", None, torch.float32)
    assert_within(y, want, bound)
    assert_guard(raw)
    assert int(status.item()) == fos.STATUS_BAD_OFFS


def test_grouped_reads_the_grouped_quantizer():
    """router counts -> offs -> fos_quantize_grouped -> fos_linear_grouped."""
    T, E, k, N, K = 96, 6, 2, 40, 128
    logits = torch.randn(T, E, generator=gen(71)).cuda()
    idx = logits.topk(k, 1).indices
    _, counts, offs, _ = fos.fos_balance_loss(logits, idx, align=16)
    M = T * k + 16 * E
    ends, cnt = offs.tolist(), counts.tolist()
    x = torch.zeros(M, K, dtype=torch.bfloat16)
    for g in range(E):
        s = ends[g - 1] if g else 0
        x[s:s + cnt[g]] = torch.randn(cnt[g], K, generator=gen(72 + g)).bfloat16()
    x = x.cuda()
    codes, scales, _, sdec = fos.fos_quantize_grouped_fused(x, offs)
    w, wv = make_w(N, K, 79, "group", E)
    y = fos.fos_linear_grouped((codes, scales, sdec), w, offs, x_gran="group", w_gran="group",
                               out_dtype=torch.float32)
    xv = decode_nvfp4(codes.cpu(), scales.cpu())
    at = 0
    for g in range(E):
        xv[at:ends[g]] *= sdec.cpu().double()[g]
        at = ends[g]
    want, bound = grouped_reference(xv, wv, ends, M, N, None, "none", None, torch.float32)
    assert_within(y, want, bound)


# ------------------------------------------------------------------- norm


def norm_reference(x, res, w, eps):
    h = x.double() + (res.double() if res is not None else 0)
    v = w.double() * h / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    top = v.abs().amax(1)
    s = torch.where(top > 0, top / 448, torch.ones_like(top)).clamp_min(2.0 ** -126)
    return h, v, s


def check_norm(x, res, w, eps, q, s, h, y=None):
    """h is one binary32 addition and one rounding. v takes six binary32
    roundings from h (the addition, 1/rms, two products), s one more division;
    q then rounds v / s to E4M3: half a step, 2^-4 relative, or 2^-10 absolute
    among its subnormals, on a value that is itself off by the earlier steps."""
    hr, vr, sr = norm_reference(x, res, w, eps)
    f = 2.0 ** -24
    dt = x.dtype
    habs = x.double().abs() + (res.double().abs() if res is not None else 0)
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    assert_within(h, hr, (ref.half_step(dt) + f) * hr.abs() + f * habs * 2 + tiny, "h")
    s = s.cpu().double()
    rms = torch.sqrt((hr * hr).mean(1, keepdim=True) + eps)
    verr = 6 * f * vr.abs() + 2 * f * (w.double().abs() * habs / rms)
    serr = verr.amax(1) / 448 + 2 * f * sr
    assert_within(s, sr, serr, "scale")
    qv = q.cpu().double() * s[:, None]
    assert_within(qv, vr, 2.0 ** -4 * vr.abs() * (1 + 16 * f) + 2.0 ** -10 * s[:, None] + 2 * verr + 8 * f * vr.abs(),
                  "q")
    if y is not None:
        assert_within(y, vr, ref.half_step(dt) * vr.abs() + 2 * verr + tiny, "y")


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 16), (3, 7), (2, 64), (5, 255), (4, 256), (7, 264), (3, 1000), (2, 1024),
                                 (33, 2048), (9, 2056), (3, 4096), (5, 5001), (2, 8192), (3, 8200), (2, 14336),
                                 (1, 16384), (2, 16392), (1, 40000), (1, 40001)])
def test_norm_sizes(dt, M, K):
    x = (torch.randn(M, K, generator=gen(M + K)) * 2).to(DTYPES[dt])
    r = torch.randn(M, K, generator=gen(M + K + 1)).to(DTYPES[dt]) if (M + K) % 3 else None
    w = (1 + 0.3 * torch.randn(K, generator=gen(K))).to(DTYPES[["bf16", "fp16", "fp32"][K % 3]])
    y, raw = guarded((M, K), DTYPES[dt])
    q, s, h = fos.fos_rmsnorm_quantize(cuda(x), cuda(w), residual=None if r is None else cuda(r), eps=1e-5, y=y)
    check_norm(x, r, w, 1e-5, q, s, h, y)
    assert_guard(raw)
    if r is None:
        assert torch.equal(h.cpu(), x)


@pytest.mark.parametrize("K", [40, 33, 4096, 20000])
def test_norm_rows_of_zeros_extremes_and_nonfinite_values(K):
    x = torch.randn(12, K, generator=gen(3))
    x[1] = 0
    x[2] = 0
    x[2, K // 2] = 1e-20     # squares far below binary32
    x[3] *= 1e25             # squares far above it
    x[4, 1] = float("nan")
    x[5, 2] = float("inf")
    x[6, 3] = -float("inf")
    x[7] *= 1e-12
    w = torch.ones(K)
    w[0] = 0
    q, s, h = fos.fos_rmsnorm_quantize(cuda(x), cuda(w), eps=0.0 if K == 40 else 1e-30)
    q8, s = q.view(torch.uint8).cpu(), s.cpu()
    for i in (4, 5, 6):
        assert torch.isnan(s[i]) and (q8[i] == 0x7F).all()
    if K != 40:  # a row of zeros: with eps = 0 it is 0 / 0
        assert s[1] == 1 and (q8[1] == 0).all()
    else:
        assert torch.isnan(s[1])
    fine = [0, 2, 3, 7, 8, 9, 10, 11]
    check_norm(x[fine], None, w, 0.0 if K == 40 else 1e-30, q[fine].cpu(), s[fine], x[fine])


@pytest.mark.parametrize("K", [48, 1001])
def test_norm_in_place_of_its_inputs(K):
    x = torch.randn(9, K, generator=gen(4)).bfloat16()
    r = torch.randn(9, K, generator=gen(5)).bfloat16()
    w = torch.ones(K).bfloat16()
    want = fos.fos_rmsnorm_quantize(cuda(x), cuda(w), residual=cuda(r))
    for which in ("x", "r"):
        xd, rd = cuda(x), cuda(r)
        got = fos.fos_rmsnorm_quantize(xd, cuda(w), residual=rd, h=xd if which == "x" else rd)
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_norm_feeds_the_product():
    M, K, N = 24, 256, 40
    x = torch.randn(M, K, generator=gen(6)).bfloat16()
    r = torch.randn(M, K, generator=gen(7)).bfloat16()
    q, s, h = fos.fos_rmsnorm_quantize(cuda(x), torch.ones(K, device="cuda"), residual=cuda(r))
    w, wv = make_w(N, K, 8)
    want, bound = ref.linear(q.cpu().double() * s.cpu().double()[:, None], wv)
    assert_within(fos.fos_linear((q, s), w, out_dtype=torch.float32), want, bound)


# ---------------------------------------------------------------- balance


def balance_reference(logits, idx, mask, coef, align, dloss):
    T, E = logits.shape
    v = logits.double()
    live = torch.ones(T, dtype=torch.bool) if mask is None else mask.bool()
    p = torch.softmax(v, 1)
    p = torch.where(torch.isinf(v).all(1, keepdim=True) & (v.amax(1, keepdim=True) < 0), torch.zeros_like(p), p)
    p = p[live]
    counts = torch.zeros(E, dtype=torch.int64)
    hit = idx[live].flatten().long()
    hit = hit[(hit >= 0) & (hit < E)]
    counts.index_add_(0, hit, torch.ones_like(hit))
    n, C = max(1, int(live.sum())), max(1, int(counts.sum()))
    slope = coef * E * counts.double() / (C * n)
    grad = torch.zeros(T, E, dtype=torch.float64)
    grad[live] = dloss * p * (slope - (p @ slope)[:, None])
    size = dloss * p * (slope + (p @ slope)[:, None])  # what the difference is made of
    mag = torch.zeros(T, E, dtype=torch.float64)
    mag[live] = size
    offs = torch.cumsum((counts + align - 1) // align * align, 0)
    return (slope * p.sum(0)).sum(), counts.int(), offs.int(), slope, grad, mag


def check_balance(logits, idx, mask, coef=0.01, align=16, status=None):
    m = None if mask is None else cuda(mask)
    loss, counts, offs, slope = fos.fos_balance_loss(cuda(logits), cuda(idx), coef=coef, mask=m, align=align,
                                                     status=status)
    d = torch.tensor([0.75])
    grad = fos.fos_balance_loss_backward(cuda(d), cuda(logits), slope, mask=m)
    wl, wc, wo, ws, wg, mag = balance_reference(logits, idx, mask, coef, align, 0.75)
    assert torch.equal(counts.cpu(), wc) and torch.equal(offs.cpu(), wo)
    f = 2.0 ** -24
    # a probability: the difference from the maximum (off by half a step of up
    # to |v|, which exp turns into a relative error; past 104 it is 0), exp, a
    # sum of E terms, a division; the loss adds its column sums of up to 1024
    # rows in binary32
    v = logits.double()
    v = v[torch.isfinite(v)]
    perr = (min(2 * float(v.abs().max()), 104) + 8 + np.sqrt(logits.shape[1])) * f if v.numel() else f
    assert abs(float(loss) - float(wl)) <= (perr + 64 * f) * float(wl) + 1e-38
    assert_within(slope, ws, 2 * f * ws)
    dt = logits.dtype
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    assert_within(grad, wg, (3 * perr + 8 * f) * mag + ref.half_step(dt) * wg.abs() * (1 + 2.0 ** -10) + tiny, "grad")
    return loss, counts, offs, slope, grad


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (7, 60, 4), (33, 64, 6), (64, 65, 1), (100, 128, 8),
                                   (257, 200, 3), (1000, 256, 8), (129, 257, 2), (65, 512, 4), (50, 1000, 2),
                                   (4097, 16, 2), (9000, 33, 1)])
def test_balance(dt, T, E, k):
    logits = (torch.randn(T, E, generator=gen(T + E)) * 3).to(DTYPES[dt])
    idx = logits.float().topk(k, 1).indices
    idx[torch.rand(T, k, generator=gen(T)) < 0.1] = -1
    check_balance(logits, idx if E % 2 else idx.int(), None, align=[1, 16, 128][T % 3])
    mask = torch.rand(T, generator=gen(E)) < 0.7
    check_balance(logits, idx, mask)
    check_balance(logits, idx, mask.to(torch.uint8) * 2)


def test_balance_without_tokens():
    for T in (0, 5):
        logits = torch.randn(T, 12, generator=gen(1))
        idx = torch.zeros(T, 2, dtype=torch.int64)
        mask = torch.zeros(T, dtype=torch.bool)
        loss, counts, offs, slope, grad = check_balance(logits, idx, mask)
        assert float(loss) == 0 and not counts.any() and not offs.any() and not grad.any()
    logits = torch.randn(6, 12, generator=gen(2))
    loss, counts, *_ = check_balance(logits, torch.full((6, 3), -1), None)
    assert float(loss) == 0 and not counts.any()


def test_balance_masked_experts_empty_rows_and_nonfinite_values():
    inf = float("inf")
    logits = torch.randn(40, 70, generator=gen(9))
    logits[:, 7] = -inf              # an expert switched off
    logits[4] = -inf                 # a row that has no expert left
    logits[5] = torch.finfo(torch.float32).min
    logits[6, 1:] = -inf
    mask = torch.ones(40, dtype=torch.bool)
    mask[10], mask[11] = False, False
    logits[10] = float("nan")        # masked rows are not read
    logits[11] = inf
    idx = logits.nan_to_num(0.0).topk(2, 1).indices
    *_, grad = check_balance(logits, idx, mask)
    assert not grad[4].any() and not grad[10].any() and not grad[11].any()
    off = torch.arange(40) != 5      # row 5 was given a finite value there
    assert not grad.cpu()[off, 7].any()
    logits[20, 3] = float("nan")     # a live one shows
    m = cuda(mask)
    loss, counts, offs, slope = fos.fos_balance_loss(cuda(logits), cuda(idx), mask=m)
    grad = fos.fos_balance_loss_backward(torch.ones(1, device="cuda"), cuda(logits), slope, mask=m).cpu()
    assert torch.isnan(loss).all() and torch.isnan(grad[20]).all()
    assert torch.isfinite(grad[torch.arange(40) != 20]).all()


def test_balance_bad_indices_are_ignored_and_reported():
    logits = torch.randn(20, 9, generator=gen(10))
    idx = logits.topk(2, 1).indices
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    check_balance(logits, idx, None, status=status)
    assert int(status.item()) == 0
    idx[3, 0], idx[4, 1], idx[5, 0] = 9, -2, 2 ** 40 + 1
    check_balance(logits, idx, None, status=status)
    assert int(status.item()) == fos.STATUS_BAD_INDEX
    # one in a masked row is not looked at
    status.zero_()
    mask = torch.ones(20, dtype=torch.bool)
    mask[3:6] = False
    check_balance(logits, idx, mask, status=status)
    assert int(status.item()) == 0


def test_balance_gradient_against_differences():
    """Central differences of the 64-bit loss: the formula itself."""
    logits = torch.randn(6, 10, generator=gen(11)).double()
    idx = logits.topk(2, 1).indices
    mask = torch.tensor([True, True, False, True, True, True])
    step = 1e-4
    num = torch.zeros_like(logits)
    for t in range(6):
        for e in range(10):
            up, down = logits.clone(), logits.clone()
            up[t, e] += step
            down[t, e] -= step
            num[t, e] = (balance_reference(up, idx, mask, 0.5, 1, 1.0)[0]
                         - balance_reference(down, idx, mask, 0.5, 1, 1.0)[0]) / (2 * step)
    x = logits.float().cuda()
    m = cuda(mask)
    slope = fos.fos_balance_loss(x, cuda(idx), coef=0.5, mask=m, align=1)[3]
    grad = fos.fos_balance_loss_backward(torch.ones(1, device="cuda"), x, slope, mask=m)
    # differences: third derivatives (below 1) times step^2 / 6; logits rounded to binary32
    assert_within(grad, num, torch.full_like(num, 1e-7))


def test_balance_repeats_bit_for_bit_and_in_a_graph():
    T, E = 3000, 256
    logits = torch.randn(T, E, generator=gen(12)).bfloat16().cuda()
    idx = logits.float().topk(4, 1).indices
    first = fos.fos_balance_loss(logits, idx)
    ws = torch.empty(fos.fos_balance_workspace(T, E), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(t) for t in first]
    grad = torch.empty_like(logits)
    d = torch.ones(1, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        fos.fos_balance_loss(logits, idx, loss=outs[0], counts=outs[1], offs=outs[2], slope=outs[3], workspace=ws)
        fos.fos_balance_loss_backward(d, logits, outs[3], out=grad)
    for k in range(4):
        logits.mul_(0.75)
        ws.fill_(255)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = fos.fos_balance_loss(logits, idx)
        for a, b in zip(outs, want):
            assert torch.equal(a, b), k
        assert torch.equal(grad, fos.fos_balance_loss_backward(d, logits, want[3])), k


# ---------------------------------------------------- refusals of the binding


def test_python_refusals():
    x = torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")
    w, _ = make_w(8, 32, 1)
    g, _ = make_w(8, 32, 1, "tensor", 2)
    offs = torch.tensor([2, 4], dtype=torch.int32, device="cuda")
    one = torch.ones(1, device="cuda")
    bad = [
        (fos.fos_linear, (x.float(), w), {}), (fos.fos_linear, (x.t(), w), {}), (fos.fos_linear, (x[0], w), {}),
        (fos.fos_linear, (x[:, :16].contiguous(), w), {}), (fos.fos_linear, (x, (w[0][:, :8], w[1], w[2])), {}),
        (fos.fos_linear, (x, (w[0], w[1][:, :1].contiguous(), w[2])), {}), (fos.fos_linear, (x, w), {"act": "tanh"}),
        (fos.fos_linear, (x, w), {"w_gran": "row"}), (fos.fos_linear, (x, w), {"w_gran": "group"}),
        (fos.fos_linear, (x, w), {"bias": one}), (fos.fos_linear, (x, w), {"residual": x}),
        (fos.fos_linear, (x, w), {"out_dtype": torch.int8}), (fos.fos_linear, (x, w), {"out": x}),
        (fos.fos_linear, (x, w), {"bias": torch.ones(8)}), (fos.fos_linear, (x, (w[0], w[1], one.double())), {}),
        (fos.fos_linear, ((x.to(torch.float8_e4m3fn), one), w), {}), (fos.fos_linear, (x, g), {}),
        (fos.fos_linear, ((x, one, one, one), w), {}), (fos.fos_linear, ((x, one), w), {}),
        (fos.fos_linear_grouped, (x, w, offs), {}), (fos.fos_linear_grouped, (x, g, offs.long()), {}),
        (fos.fos_linear_grouped, (x, g, offs[:1].contiguous()), {}), (fos.fos_linear_grouped, (x, g, offs.cpu()), {}),
        (fos.fos_rmsnorm_quantize, (x, one), {}), (fos.fos_rmsnorm_quantize, (x.to(torch.int16), x[0]), {}),
        (fos.fos_rmsnorm_quantize, (x, x[0]), {"residual": x.half()}), (fos.fos_rmsnorm_quantize, (x, x[0]), {"q": x}),
        (fos.fos_rmsnorm_quantize, (x, x[0]), {"h": x.float()}), (fos.fos_rmsnorm_quantize, (x[0], x[0]), {}),
        (fos.fos_balance_loss, (x, offs), {}), (fos.fos_balance_loss, (x, torch.zeros(3, 2, device="cuda")), {}),
        (fos.fos_balance_loss, (x, torch.zeros(4, 2, device="cuda")), {}),
        (fos.fos_balance_loss, (x, torch.zeros(4, 2, device="cuda").int()), {"mask": torch.ones(4, device="cuda")}),
        (fos.fos_balance_loss, (x, torch.zeros(4, 2, device="cuda").int()), {"counts": torch.ones(32, device="cuda")}),
        (fos.fos_balance_loss_backward, (one, x, one), {}), (fos.fos_balance_loss_backward, (x, x, x[0].float()), {}),
    ]
    for fn, args, kw in bad:
        with pytest.raises(ValueError):
            fn(*args, **kw)
    with pytest.raises(fos.FosError):
        fos.fos_rmsnorm_quantize(x, x[0], eps=-1.0)
    with pytest.raises(fos.FosError):  # a view that starts off the 16-byte grid
        flat = torch.zeros(4 * 32 + 1, dtype=torch.bfloat16, device="cuda")[1:]
        fos.fos_linear(flat.view(4, 32), w)
    with pytest.raises(fos.FosError):
        fos.fos_linear(x, w, workspace=None, out=torch.zeros(40, device="cuda")[2:34].view(4, 8))


def test_workspace_and_status_are_checked():
    """Memory that the kernels write besides their outputs: on the host, with
    gaps or of another type it is refused before a launch."""
    M, N, K = 130, 1500, 3088  # in several parts of K
    need = fos.fos_linear_workspace(M, N, K)
    assert need > 0
    x = torch.randn(M, K, generator=gen(3)).bfloat16().cuda()
    w = make_w(N, K, 4)[0]
    offs = torch.tensor([M], dtype=torch.int32, device="cuda")
    w3 = (w[0][None], w[1][None], w[2])
    logits = torch.randn(8, 16, generator=gen(5)).cuda()
    idx = torch.zeros(8, 2, dtype=torch.int64, device="cuda")
    room = fos.fos_balance_workspace(8, 16)
    for bad in (lambda n: torch.empty(n, dtype=torch.uint8),
                lambda n: torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            fos.fos_linear(x, w, workspace=bad(need))
        with pytest.raises(ValueError):
            fos.fos_balance_loss(logits, idx, workspace=bad(room))
    for bad in (torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.uint8, device="cuda"),
                torch.zeros(1, dtype=torch.int64, device="cuda")):
        with pytest.raises(ValueError):
            fos.fos_linear_grouped(x, w3, offs, status=bad)
        with pytest.raises(ValueError):
            fos.fos_balance_loss(logits, idx, status=bad)
    with pytest.raises(fos.FosError):
        fos.fos_linear(x, w, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    y = fos.fos_linear(x, w, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    assert torch.equal(y, fos.fos_linear(x, w))


# ------------------------------------------------------------------ together


@pytest.mark.parametrize("tokens,width,hidden,experts,top", [(1, 256, 320, 4, 2), (200, 256, 320, 6, 2),
                                                             (700, 512, 1024, 16, 4)])
def test_example_block(tokens, width, hidden, experts, top):
    """examples/moe_feed_forward.py against the block on unquantized values:
    two NVFP4 operands in a row are each off by about a tenth, E4M3 by a
    thirtieth, and errors of different elements are independent."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_feed_forward.py")
    spec = importlib.util.spec_from_file_location("moe_feed_forward", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    w = ex.make_weights(width, hidden, experts)
    x = torch.randn(tokens, width, generator=gen(1)).bfloat16().cuda()
    r = torch.randn(tokens, width, generator=gen(2)).bfloat16().cuda()
    out, loss, saved = ex.forward(x, r, ex.quantize_weights(w), top)
    want = ex.reference(x, r, w, top)
    h = x.float() + r.float()
    assert float((out.float() - want).norm() / (want - h).norm()) < 0.25
    y, logits, slope = saved
    idx = torch.softmax(logits, 1).topk(top, 1).indices.cpu()
    wl, *_, wg, _ = balance_reference(logits.cpu(), idx, None, 0.01, 16, 1.0)
    assert abs(float(loss) - float(wl)) < 1e-5 * float(wl)
    grad = ex.router_gradient(saved, torch.ones(1, device="cuda")).cpu().double()
    ref_grad = wg.t() @ y.cpu().double()
    assert float((grad - ref_grad).norm()) <= 1e-4 * float(ref_grad.norm()) + 1e-9
