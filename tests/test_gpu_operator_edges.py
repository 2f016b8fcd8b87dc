"""The operators around the quantizer at the edges of their ranges: values
beside a rounding's border, scales and rows near the ends of binary32, sizes
past a single launch. GPU only."""
import numpy as np
import pytest
import torch

import nvfp4_adaptive_block_amd as fos
from operator_reference import DTYPES, activate, decode_nvfp4, gen, half_step, random_nvfp4
from test_gpu_operators import check_norm, cuda, make_w

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- norm


def e4m3_middles():
    """The values halfway between two neighbouring E4M3 magnitudes."""
    codes = torch.arange(0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    return (codes[1:] + codes[:-1]) / 2


@pytest.mark.parametrize("form", ["packed", "row", "wide"])
def test_norm_codes_at_the_middle_of_two(form):
    """q is E4M3 of v / s, the quotient rounded once. Rows of ones have rms 1,
    so v is the weight: multiples of the row's scale that lie on the middle of
    two codes, or one step of binary32 beside it, and the row's maximum."""
    for seed in range(12):
        # (the last rows of scales near the least and the largest that binary32 has)
        size = {9: 2.0 ** -116, 10: 2.0 ** -80, 11: 2.0 ** 127}.get(seed, 1.0)
        top = (torch.rand(1, generator=torch.Generator().manual_seed(seed)) + 0.5) * size
        v = (e4m3_middles() * (top / 448).double()).float()
        v = torch.cat([top, v, torch.nextafter(v, torch.zeros(())), torch.nextafter(v, top.expand_as(v)), -v])
        w = v.repeat({"packed": 1, "row": 3, "wide": 70}[form])
        w = torch.cat([w, torch.zeros(-len(w) % 8)]) if seed % 2 else w
        K = len(w)
        assert (8 <= K <= 512, 512 < K <= 32768, K > 32768)[["packed", "row", "wide"].index(form)]
        x = torch.ones(5, K, device="cuda")
        y = torch.empty_like(x)
        q, s, _ = fos.fos_rmsnorm_quantize(x, w.cuda(), eps=0.0, y=y)
        y, s = y.cpu(), s.cpu()
        assert torch.equal(y, w.expand(5, K)) and torch.equal(s, (top / 448).expand(5))
        want = (y / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(q.cpu().view(torch.uint8), want.view(torch.uint8)), seed


@pytest.mark.parametrize("K", [40, 999, 40000])
def test_norm_keeps_the_sign_of_zeros(K):
    x = torch.randn(4, K, generator=gen(K))
    x[:, ::3], x[:, 1::3] = -0.0, 0.0
    x[1, 2::3] = -1e-30  # quotients that round to zero
    x[1, 2] = 1.0
    q, s, _ = fos.fos_rmsnorm_quantize(cuda(x), torch.ones(K, device="cuda"))
    q = q.cpu().view(torch.uint8)
    assert (q[:, ::3] == 0x80).all() and (q[:, 1::3] == 0).all() and (q[1, 5::3] == 0x80).all()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("K", [40, 999, 40000])
def test_norm_rows_whose_rms_is_near_the_ends_of_binary32(dt, K):
    """With eps = 0 a row of subnormals has a reciprocal rms past binary32's
    largest value, and a row of the largest values one among its subnormals:
    the result is of order 1 in both."""
    x = torch.randn(6, K, generator=gen(K)).clamp(-3, 3)
    x[0] *= 2.0 ** -129
    x[1] *= 2.0 ** -131
    x[2, 1:] = 0             # one subnormal in a row of zeros
    x[2, 0] = 2.0 ** -131
    x[3] *= 2.0 ** 126
    x[4] = 3.38e38
    x = x.to(DTYPES[dt])
    w = 1 + 0.3 * torch.randn(K, generator=gen(1))
    y = torch.empty(6, K, dtype=DTYPES[dt], device="cuda")
    q, s, h = fos.fos_rmsnorm_quantize(cuda(x), cuda(w), eps=0.0, y=y)
    assert torch.isfinite(s).all()
    check_norm(x, None, w, 0.0, q.cpu(), s, x, y)


@pytest.mark.parametrize("M,K", [(2 ** 21 + 5, 9), (3 * 2 ** 21, 3), (2 ** 26 + 3, 4)])
def test_norm_of_more_rows_than_a_launch_has(M, K):
    """Rows on both sides of every 2^21 against the reference, and no row left out."""
    g = torch.Generator("cuda")
    g.manual_seed(K)
    x = torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16)
    res = torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16) if K == 9 else None
    w = 1 + 0.3 * torch.randn(K, generator=gen(2))
    s = torch.full((M,), float("nan"), device="cuda")
    y = torch.full_like(x, float("nan"))
    q, s, h = fos.fos_rmsnorm_quantize(x, w.cuda(), residual=res, eps=1e-5, scale=s, y=y)
    assert torch.isfinite(s).all() and torch.isfinite(y).all()
    near = torch.cat([torch.arange(max(0, at - 20), min(M, at + 20)) for at in [*range(0, M, 2 ** 21), M]]).cuda()
    pick = lambda t: None if t is None else t[near].cpu()
    check_norm(pick(x), pick(res), w, 1e-5, q.view(torch.uint8)[near].cpu().view(torch.float8_e4m3fn), pick(s), pick(h),
               pick(y))


# ---------------------------------------------------------------- product


@pytest.mark.parametrize("grouped", [False, True])
def test_product_of_no_rows(grouped):
    """What the norm and the quantizer return for no tokens goes into the
    product as for some."""
    K, N = 64, 24
    offs = torch.zeros(2, dtype=torch.int32, device="cuda")
    w = make_w(N, K, 1, "tensor", 2 if grouped else None)[0]
    for rows in (0, 5):
        x = torch.ones(rows, K, dtype=torch.bfloat16, device="cuda")
        q, s, _ = fos.fos_rmsnorm_quantize(x, torch.ones(K, device="cuda"))
        codes = (torch.zeros(rows, K // 2, dtype=torch.uint8, device="cuda"),
                 torch.zeros(rows, K // 16, dtype=torch.uint8, device="cuda"), torch.ones(rows, device="cuda"))
        for operand, gran in (((q, s), None), (codes, "row")):
            if grouped:
                y = fos.fos_linear_grouped(operand, w, offs, x_gran=gran)
            else:
                y = fos.fos_linear(operand, w, x_gran=gran)
            assert y.shape == (rows, N)


def test_product_with_no_columns():
    x = torch.ones(3, 64, dtype=torch.bfloat16, device="cuda")
    w = make_w(0, 64, 1, "row")[0]
    assert fos.fos_linear(x, w, w_gran="row").shape == (3, 0)


def scaled_rows(kind, M, K, seed):
    """Quantized rows whose scales are near the ends of binary32's range: (operand, unscaled
    values, scales). Every sixth row is zero, and every sixth holds one small value."""
    g = gen(seed)
    s = torch.tensor([1e-25, 1e-23, 1e25, 1e19, 1.0, 1e25]).repeat(M // 6 + 1)[:M].contiguous()
    if kind == "e4m3":
        q = (torch.randn(M, K, generator=g) * 60).clamp(-448, 448)
        q[2::6] = 0
        q[3::6] = 0
        q[3::6, 1] = 2.0 ** -9
        q = q.to(torch.float8_e4m3fn)
        return (q, s), q.double(), s.double()
    codes, scales = random_nvfp4(M, K, seed)
    scales[2::6] = 0
    scales[3::6] = 0
    scales[3::6, 0] = 1
    codes[3::6, :8] = 0
    codes[3::6, 0] = 0x10  # the second value is the smallest
    return (codes, scales, s), decode_nvfp4(codes, scales), s.double()


def assert_scaled(y, x, sx, w, sw):
    """y = (x w^T) sx sw in float32: the sum in any order (as in operator_reference),
    the product of the scales applied to it, one rounding; past the range, an infinity."""
    y = y.cpu().double()
    v = x @ w.T
    S = (x.abs() @ w.abs().T) * sx[:, None] * sw
    v = v * sx[:, None] * sw
    bound = (4 * x.shape[1] ** 0.5 + 8) * 2.0 ** -24 * S + 2.0 ** -23 * v.abs() + 2.0 ** -149
    top = torch.finfo(torch.float32).max
    over, fits = v.abs() - bound > top, v.abs() + bound < top
    assert not torch.isnan(y).any()
    assert torch.equal(y[over], v[over].sign() * float("inf"))
    off = (y - v).abs() > bound
    assert not (off & fits).any(), (int((off & fits).sum()), y[off & fits][0], v[off & fits][0])


# few rows, tiles of 64 and of 128 rows, and K in several parts
@pytest.mark.parametrize("kind", ["e4m3", "nvfp4"])
@pytest.mark.parametrize("gran", ["tensor", "row"])
@pytest.mark.parametrize("M,N,K", [(20, 33, 256), (50, 700, 1104), (2050, 1500, 528), (3000, 4099, 272), (150, 2051, 4208)])
def test_product_of_scales_past_binary32(kind, gran, M, N, K):
    """Each scale, the sum and (mostly) the result are in binary32's range; the
    product of the two scales is not."""
    x, xv, sx = scaled_rows(kind, M, K, M)
    codes, scales = random_nvfp4(N, K, N)
    wv = decode_nvfp4(codes, scales)
    for s in (1e-20, 1e20):
        sw = torch.full((N,) if gran == "row" else (1,), s)
        if gran == "row":
            sw[::3] = 1 / s
        y = fos.fos_linear(cuda(x), cuda((codes, scales, sw)), out_dtype=torch.float32, x_gran="row", w_gran=gran)
        assert_scaled(y, xv, sx, wv, sw.double())


@pytest.mark.parametrize("M", [12, 150])
def test_product_by_group_of_scales_past_binary32(M):
    N, K = 40, 272
    x, xv, _ = scaled_rows("e4m3", M, K, 3)
    codes, scales = random_nvfp4(3 * N, K, 4)
    wv = decode_nvfp4(codes, scales)
    sx, sw = torch.tensor([1e-25, 1e25, 1e19]), torch.tensor([1e-19, 1e20, 1e20])
    ends = [0, M // 3, 2 * M // 3, M]
    y = fos.fos_linear_grouped(cuda((x[0], sx)), cuda((codes.view(3, N, -1), scales.view(3, N, -1), sw)),
                               torch.tensor(ends[1:], dtype=torch.int32).cuda(), out_dtype=torch.float32,
                               x_gran="group", w_gran="group")
    for g in range(3):
        rows = slice(ends[g], ends[g + 1])
        assert_scaled(y[rows], xv[rows], sx[g].double().expand(ends[g + 1] - ends[g]), wv[g * N:(g + 1) * N],
                      sw[g].double())


# how far an activation of v may be off, in half steps of binary32: what its
# instructions round, and the rounding of the exponential's argument (1.5 half
# steps of the argument, for gelu_tanh 5 more in u)
ACTIVATION_STEPS = {"none": lambda v: 0 * v, "relu": lambda v: 0 * v, "silu": lambda v: 6 + 1.5 * v.abs(),
                    "gelu": lambda v: 16 + 1.5 * v * v,
                    "gelu_tanh": lambda v: 6 + 6.5 * 1.6 * (v.abs() + 0.045 * v.abs() ** 3)}


@pytest.mark.parametrize("out", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("M,N,K", [(3, 4100, 32), (2050, 1500, 528), (150, 2051, 4208)])
def test_activations_of_exact_values(M, N, K, out):
    """The product of zeros and a bias: the activation of a known value, relative
    to the result, for small results too (past 1e-36 they may be zero)."""
    x = torch.zeros(M, K, dtype=torch.float16, device="cuda")
    w = make_w(N, K, 1)[0]
    v = torch.cat([torch.linspace(-12, 8, N - 60), torch.logspace(-30, 2, 30), -torch.logspace(-30, 2, 30)])
    for act, steps in ACTIVATION_STEPS.items():
        y = fos.fos_linear(x, w, bias=cuda(v), act=act, out_dtype=DTYPES[out]).cpu()
        assert torch.equal(y, y[:1].expand(M, N))
        want = activate(act, v.double())
        if act == "gelu_tanh":  # (1 + tanh u) / 2 without its cancellation
            want = v.double() * torch.sigmoid(2 * (2 / np.pi) ** 0.5 * (v.double() + 0.044715 * v.double() ** 3))
        err = steps(v.double()) * 2.0 ** -24 * want.abs() + 1e-36
        tiny = torch.finfo(DTYPES[out]).smallest_normal * torch.finfo(DTYPES[out]).eps
        bound = err + half_step(DTYPES[out]) * (want.abs() + err) * (out != "fp32" or act != "none") + tiny
        off = (y[0].double() - want).abs() > bound
        assert not off.any(), (act, v[off][:4], y[0][off][:4], want[off][:4])


def test_an_empty_status_is_refused():
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    x = torch.ones(3, 32, dtype=torch.bfloat16, device="cuda")
    w = make_w(8, 32, 1, "tensor", 1)[0]
    with pytest.raises(ValueError, match="status"):
        fos.fos_linear_grouped(x, w, torch.tensor([9], dtype=torch.int32, device="cuda"), status=none)
    with pytest.raises(ValueError, match="status"):
        fos.fos_balance_loss(x, torch.full((3, 1), 99, device="cuda"), status=none)


@pytest.mark.parametrize("M,N", [(0, 16), (5, 0), (0, 0)])
def test_offsets_are_reported_where_there_is_nothing_to_write(M, N):
    G, K = 70, 32
    x = torch.ones(M, K, dtype=torch.bfloat16, device="cuda")
    w = (torch.zeros(G, N, K // 2, dtype=torch.uint8, device="cuda"),
         torch.zeros(G, N, K // 16, dtype=torch.uint8, device="cuda"), torch.ones(1, device="cuda"))
    for offs, bad in (([0] * G, False), ([0] * (G - 1) + [M], False), ([0] * 66 + [M + 1] + [M] * 3, True),
                      ([-1] + [M] * (G - 1), True)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o = torch.tensor(offs, dtype=torch.int32, device="cuda")
        assert fos.fos_linear_grouped(x, w, o, status=status).shape == (M, N)
        assert int(status.item()) == (fos.STATUS_BAD_OFFS if bad else 0), offs
        fos.fos_linear_grouped(x, w, o)


# ---------------------------------------------------------------- balance


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T", [0, 40, 3000])
def test_balance_loss_is_in_the_graph_of_its_logits(dt, masked, T):
    E = 33
    x = torch.randn(T, 16, generator=gen(1)).cuda()
    w = torch.randn(E, 16, generator=gen(2)).cuda().requires_grad_()
    mask = cuda(torch.rand(T, generator=gen(3)) < 0.7) if masked else None
    logits = (x @ w.t()).to(DTYPES[dt])
    idx = logits.detach().float().topk(2, 1).indices
    loss, counts, offs, slope = fos.fos_balance_loss(logits, idx, coef=0.5, mask=mask)
    assert loss.requires_grad and not (counts.requires_grad or offs.requires_grad or slope.requires_grad)
    with torch.no_grad():
        plain = fos.fos_balance_loss(logits, idx, coef=0.5, mask=mask)
    assert not plain[0].requires_grad
    for a, b in zip((loss, counts, offs, slope), plain):
        assert torch.equal(a.detach(), b)
    # beside another loss of the same logits, its gradient is the explicit call's
    other = (logits.float() ** 2).sum()
    (other + 0.75 * loss.sum()).backward()
    d = fos.fos_balance_loss_backward(torch.full((1,), 0.75, device="cuda"), logits.detach(), slope, mask=mask)
    both = logits.detach().requires_grad_()
    (both.float() ** 2).sum().backward()
    want = ((both.grad + d).float().t() @ x) if T else torch.zeros_like(w)
    assert (w.grad - want).abs().max() <= 4 * half_step(DTYPES[dt]) * (want.abs().max() + 1)
    leaf = logits.detach().requires_grad_()
    got, = torch.autograd.grad(fos.fos_balance_loss(leaf, idx, coef=0.5, mask=mask)[0], leaf,
                               torch.full((1,), 0.75, device="cuda"))
    assert got.dtype == leaf.dtype and torch.equal(got, d)


def test_balance_loss_keeps_its_slope_for_the_backward_pass():
    """The caller's buffers are written again before the first call's backward pass;
    a loss that is such a buffer is outside the graph."""
    logits = torch.randn(2, 50, 20, generator=gen(4)).cuda()
    idx = logits.topk(3, 2).indices
    slope, counts = torch.empty(20, device="cuda"), torch.empty(20, dtype=torch.int32, device="cuda")
    leaves, losses = [logits[i].clone().requires_grad_() for i in range(2)], []
    for leaf, i in zip(leaves, idx):
        out = fos.fos_balance_loss(leaf, i, slope=slope, counts=counts)
        assert out[3] is slope or out[3].data_ptr() == slope.data_ptr()
        losses.append(out[0])
    for leaf, loss, i in zip(leaves, losses, idx):
        loss.backward()
        s = fos.fos_balance_loss(leaf.detach(), i)[3]
        one = torch.ones(1, device="cuda")
        assert torch.equal(leaf.grad, fos.fos_balance_loss_backward(one, leaf.detach(), s))
    assert torch.equal(slope, s)
    buffer = torch.empty(1, device="cuda")
    assert fos.fos_balance_loss(leaves[0], idx[0], loss=buffer)[0] is buffer and not buffer.requires_grad


def test_balance_loss_and_its_gradient_in_a_graph():
    T, E = 3000, 64
    leaf = torch.randn(T, E, generator=gen(5)).cuda().requires_grad_()
    idx = leaf.detach().topk(2, 1).indices
    one = torch.ones(1, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss = fos.fos_balance_loss(leaf, idx)[0]
        grad, = torch.autograd.grad(loss, leaf, one)
    for k in range(4):
        with torch.no_grad():
            leaf.mul_(0.75)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        plain = leaf.detach()
        want = fos.fos_balance_loss(plain, idx)
        assert torch.equal(loss.detach(), want[0]), k
        assert torch.equal(grad, fos.fos_balance_loss_backward(one, plain, want[3])), k
