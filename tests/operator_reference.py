"""Plain 64-bit references of the operators around the quantizer, on the CPU,
and the error bounds that their tests use."""
import math

import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def gen(seed):
    g = torch.Generator("cpu")
    g.manual_seed(seed)
    return g


def half_step(dtype):
    """The largest relative error of one rounding to `dtype`."""
    return torch.finfo(dtype).eps / 2


def decode_nvfp4(codes, scales):
    """float64 values of codes [..., K/2] and E4M3 scales [..., K/16], without S_dec."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    v = torch.where(c >= 8, -E2M1[c & 7], E2M1[c & 7])
    return v * scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)


def random_nvfp4(rows, K, seed):
    """Random codes and finite, mostly middling E4M3 scales (zeros among them)."""
    g = gen(seed)
    codes = torch.randint(0, 256, (rows, K // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(0x28, 0x48, (rows, K // 16), generator=g, dtype=torch.uint8)
    odd = torch.rand(rows, K // 16, generator=g)
    scales[odd < 0.05] = 0
    scales[odd > 0.98] = 0x7E  # 448, the largest
    scales[(odd > 0.95) & (odd < 0.98)] = 0x01  # 2^-9, the smallest
    return codes, scales


def activate(name, v):
    if name == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if name == "gelu":
        return 0.5 * v * torch.special.erfc(-v / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if name == "silu":
        return v / (1 + torch.exp(-v))
    return v


def linear(x, w, bias=None, act="none", residual=None, out_dtype=torch.float32):
    """(y, bound): the product in float64 and how far a kernel may be off.

    A sum of K products in binary32, in any order, is off by a random walk of K
    roundings of partial sums no larger than S = sum |x w|: four standard
    steps, 4 sqrt(K) 2^-24 S, plus 2^-23 S for the joins. The scales, the bias,
    the activation (slope at most 1.13, own error at most eight half steps of
    its argument) and the residual each add a few half steps of binary32; the
    output is rounded once."""
    x, w = x.double(), w.double()
    K = x.shape[-1]
    v = x @ w.transpose(-1, -2)
    S = x.abs() @ w.abs().transpose(-1, -2)
    err = (4 * math.sqrt(max(K, 1)) + 8) * 2.0 ** -24 * S
    if bias is not None:
        v = v + bias.double()
        err = err + 2.0 ** -24 * (v.abs() + bias.double().abs())
    a = activate(act, v)
    err = 1.13 * err + 8 * 2.0 ** -24 * v.abs() + 1e-30
    if residual is not None:
        a = a + residual.double()
        err = err + 2.0 ** -24 * a.abs()
    # subnormal outputs round to a fixed step
    tiny = torch.finfo(out_dtype).smallest_normal * torch.finfo(out_dtype).eps
    return a, err + half_step(out_dtype) * (a.abs() + err) + tiny


def assert_within(got, want, bound, what=""):
    got = got.double().cpu()
    assert got.shape == want.shape, (got.shape, want.shape)
    bad = ~((got - want).abs() <= bound)
    bad &= ~(torch.isnan(got) & torch.isnan(want))
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got {got[i].item()!r}, "
                             f"want {want[i].item()!r} within {bound[i].item():.3g}")
