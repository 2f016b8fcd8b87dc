"""Cases of the inference and routing operators next to the NVFP4 quantizer,
their plain form in elementary torch operations, and what each pass has to
move and compute.

The operators, along a mixture-of-experts feed-forward block on NVFP4 weights:

  norm      h = x + r;  y = w * h / sqrt(mean(h^2) + eps);  per row
            s = max|y| / 448 (1 for a row of zeros), q = E4M3(y / s).
            Returns q, s and h.
  balance   p = softmax(logits) per unmasked token; c_e = assignments to
            expert e; f_e = c_e / sum(c); P_e = mean over tokens of p_e;
            loss = coef * E * sum_e f_e P_e; offs = running sum of c_e rounded
            up to the alignment. With the gradient
            dl_te = dloss * coef * E / n * p_te * (f_e - sum_j f_j p_tj).
  linear    y = act(S_x[m] * S_w[n] * sum_k x[m,k] w[n,k] + bias[n]) + res[m,n]
            with w in NVFP4 (E2M1 codes, an E4M3 scale per 16 values along k, a
            float32 scale) and x in bf16, fp16, E4M3 with a scale per row, or
            NVFP4.
  grouped   the same for G experts at once: rows [offs[g-1], offs[g]) of x take
            weight g; rows past the last offset come out as zero.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
FLOATS = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6
COEF = 0.01
ALIGN = 16


def listed():
    return [
        # one token of a decode step through the norm before a block: latency
        {"name": "norm_token", "op": "norm", "M": 1, "K": 4096, "dtype": "bf16"},
        # the activations of a training or prefill step (8192 tokens)
        {"name": "norm_prefill", "op": "norm", "M": 8192, "K": 4096, "dtype": "bf16"},
        # a ragged batch of rows of odd width, where no row but the first is aligned
        {"name": "norm_odd", "op": "norm", "M": 1531, "K": 5001, "dtype": "fp16"},
        # the router of a decode step: a few tokens, loss and gradient
        {"name": "balance_small", "op": "balance", "T": 37, "E": 64, "k": 4, "dtype": "fp32", "masked": 0.0},
        # the router of a training step: 65536 tokens, an eighth of them padding
        {"name": "balance_train", "op": "balance", "T": 65536, "E": 256, "k": 8, "dtype": "bf16", "masked": 0.125},
        # one token against a feed-forward weight: the time to stream the weight
        {"name": "linear_token", "op": "linear", "M": 1, "N": 4096, "K": 14336, "x": "bf16", "out": "bf16",
         "act": "none", "bias": False, "res": True},
        # a batch of sequences in decode, with the 8-bit rows that the norm writes
        {"name": "linear_batch", "op": "linear", "M": 48, "N": 14336, "K": 4096, "x": "e4m3", "out": "fp16",
         "act": "gelu", "bias": True, "res": False},
        # a ragged prompt, odd output width, a depth that ends inside every tile
        {"name": "linear_odd", "op": "linear", "M": 1003, "N": 5003, "K": 2064, "x": "fp16", "out": "fp32",
         "act": "silu", "bias": True, "res": True},
        # a long prompt on 16-bit activations
        {"name": "linear_prefill", "op": "linear", "M": 8192, "N": 4096, "K": 4096, "x": "bf16", "out": "bf16",
         "act": "gelu", "bias": True, "res": False},
        # a training-sized product of two quantized operands (the largest case)
        {"name": "linear_nvfp4", "op": "linear", "M": 8192, "N": 4096, "K": 14336, "x": "nvfp4", "out": "bf16",
         "act": "none", "bias": False, "res": True},
        # the experts of a decode step: 16 tokens of 4 experts each over 64 experts
        {"name": "experts_decode", "op": "grouped", "M": 64, "N": 2048, "K": 7168, "G": 64, "x": "bf16",
         "out": "bf16", "act": "silu", "bias": False, "res": False},
        # the experts of a prefill step, uneven groups and a padded tail
        {"name": "experts_prefill", "op": "grouped", "M": 16384, "N": 2048, "K": 7168, "G": 64, "x": "e4m3",
         "out": "bf16", "act": "none", "bias": True, "res": False},
    ]


def _size(rng, lo, hi, step=1, even=0.5):
    """A size between lo and hi, even over its logarithm: a power of two, or
    an odd multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    v = 2 ** round(math.log2(v)) if rng.random() < even else step * (int(v / step) | 1)
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["norm", "balance", "linear", "linear", "grouped"])
    if op == "norm":
        M, K = _size(rng, 1, 16384), _size(rng, 64, 16384)
        while M * K > 8192 * 8192:
            M = max(1, M // 2)
        return {"op": op, "M": M, "K": K, "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "balance":
        E = _size(rng, 4, 512)
        return {"op": op, "T": _size(rng, 1, 65536), "E": E, "k": rng.randint(1, min(8, E)),
                "dtype": rng.choice(["bf16", "fp32"]), "masked": rng.choice([0.0, 0.1, 0.5])}
    grouped = op == "grouped"
    step = rng.choice([16, 128, 512])
    case = {"op": op, "M": _size(rng, 1, 8192), "N": _size(rng, 64, 4096 if grouped else 16384, rng.choice([1, 64])),
            "K": _size(rng, max(256, step), 8192 if grouped else 16384, step),
            "x": rng.choice(["bf16", "fp16", "e4m3", "nvfp4"]), "out": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
            "act": rng.choice(["none", "relu", "gelu", "silu"]), "bias": rng.random() < 0.5,
            "res": rng.random() < 0.5}
    if grouped:
        case["G"] = _size(rng, 2, 64)
        while case["G"] * case["N"] * case["K"] > 64 * 2048 * 7168:
            case["G"] = max(2, case["G"] // 2)
    while case["M"] * case["N"] * case["K"] > 8192 * 4096 * 14336:
        case["M"] = max(1, case["M"] // 2)
    return case


def work(case):
    """Each input read once and each output written once; two operations per
    multiply-add, a handful per element where there is no contraction."""
    if case["op"] == "norm":
        n, b = case["M"] * case["K"], BYTES[case["dtype"]]
        return {"bytes": n * (3 * b + 1) + case["K"] * b + 4 * case["M"], "flops": 8 * n}
    if case["op"] == "balance":
        T, E, k, b = case["T"], case["E"], case["k"], BYTES[case["dtype"]]
        live = int(round(T * (1 - case["masked"])))
        # the loss needs every logit before the first gradient; one reading of
        # them is what cannot be done without, since a chip can hold them
        return {"bytes": live * E * b + T * E * b + live * k * 8 + T + 16 * E, "flops": 16 * live * E}
    M, N, K, G = case["M"], case["N"], case["K"], case.get("G", 1)
    # experts that have a row: the mean under prepare()'s uneven choice
    weights = G * (1 - 2 * (G - 1) * (2 * G - 1) / ((2 * G - 2 + M) * (2 * G - 1 + M))) if G > 1 else 1
    x = {"bf16": 2 * K, "fp16": 2 * K, "e4m3": K + 4, "nvfp4": K // 2 + K // 16 + 4}[case["x"]]
    out = BYTES[case["out"]]
    b = M * x + weights * (N * K // 2 + N * K // 16 + 4) + M * N * out * (2 if case["res"] else 1)
    return {"bytes": b + (weights * N * out if case["bias"] else 0), "flops": 2 * M * N * K}


# ------------------------------------------------------------------ inputs


def _to_nvfp4(v):
    """(codes, scales, decode scale) of rows v under one float32 scale: block
    amax to the largest E2M1 value, E4M3 block scales, round to nearest."""
    rows, K = v.shape
    top = v.abs().amax().clamp_min(1e-30)
    sdec = top / (6.0 * 448.0)
    b = v.view(rows, K // 16, 16)
    s8 = (b.abs().amax(-1) / (6.0 * sdec)).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float() * sdec
    t = b / torch.where(s > 0, s, torch.ones_like(s))[..., None]
    a = t.abs()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code += (t < 0).to(torch.uint8) * 8
    code = code.view(rows, K // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), s8.view(torch.uint8), sdec.reshape(1)


def _activations(case, gen):
    """x as the operator takes it: a tensor, (E4M3 values, row scales) or
    (codes, block scales, decode scale)."""
    M, K = case["M"], case["K"]
    v = torch.randn(M, K, generator=gen, device=DEV)
    if case["x"] in FLOATS:
        return v.to(FLOATS[case["x"]])
    if case["x"] == "e4m3":
        s = (v.abs().amax(1) / 448.0).clamp_min(1e-30)
        return (v / s[:, None]).to(torch.float8_e4m3fn), s
    return _to_nvfp4(v)


def prepare(case, seed):
    gen = torch.Generator(DEV)
    gen.manual_seed(seed * 7919 + 17)
    if case["op"] == "norm":
        M, K, dt = case["M"], case["K"], FLOATS[case["dtype"]]
        # a residual stream: rows of different size, a few large channels
        x = torch.randn(M, K, generator=gen, device=DEV)
        r = torch.randn(M, K, generator=gen, device=DEV) * (1 + 4 * torch.rand(M, 1, generator=gen, device=DEV))
        r[:, torch.randint(0, K, (max(1, K // 512),), generator=gen, device=DEV)] *= 12.0
        w = 1 + 0.2 * torch.randn(K, generator=gen, device=DEV)
        return {"case": case, "x": x.to(dt), "r": r.to(dt), "w": w.to(dt)}
    if case["op"] == "balance":
        T, E, k = case["T"], case["E"], case["k"]
        logits = torch.randn(T, E, generator=gen, device=DEV) * 1.5 + torch.randn(E, generator=gen, device=DEV)
        logits = logits.to(FLOATS[case["dtype"]])
        idx = (logits.float() + 1e-4 * torch.rand(T, E, generator=gen, device=DEV)).topk(k, dim=1).indices
        # a token that its expert had no room for is not assigned
        idx = torch.where(torch.rand(T, k, generator=gen, device=DEV) < 0.02, torch.full_like(idx, -1), idx)
        mask = None
        if case["masked"]:
            mask = torch.rand(T, generator=gen, device=DEV) >= case["masked"]
        return {"case": case, "logits": logits, "idx": idx.contiguous(), "mask": mask,
                "dloss": torch.full((1,), 0.5, device=DEV)}
    M, N, K, G = case["M"], case["N"], case["K"], case.get("G", 1)
    out = FLOATS[case["out"]]
    st = {"case": case, "x": _activations(case, gen),
          "w": _to_nvfp4(torch.randn(G * N, K, generator=gen, device=DEV) * 0.02),
          "bias": (torch.randn(G, N, generator=gen, device=DEV) * 0.1).to(out) if case["bias"] else None,
          "res": torch.randn(M, N, generator=gen, device=DEV).to(out) if case["res"] else None}
    if case["op"] == "grouped":
        # tokens choose experts unevenly; about a sixteenth of the rows is an
        # over-allocated tail (none where there are fewer rows than that)
        r = np.random.default_rng(seed * 7919 + 17)
        live = M - M // 16 if M >= 256 else M
        counts = r.multinomial(live, r.dirichlet(np.full(G, 2.0)))
        st["offs"] = torch.from_numpy(np.cumsum(counts).astype(np.int32)).to(DEV)
        st["most"] = int(counts.max())
        c, s, d = st["w"]
        st["w"] = (c.view(G, N, K // 2), s.view(G, N, K // 16), d)
        st["first"] = torch.arange(max(1, st["most"]), device=DEV)
    elif st["bias"] is not None:
        st["bias"] = st["bias"].view(N)
    return st


# -------------------------------------------------------------- plain form


def _values(codes, scales):
    """float32 values of NVFP4 codes and block scales, without the tensor's scale."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).view(*codes.shape[:-1], -1, 16)
    return (table[c.int()] * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _plain_x(x):
    """float32 values of the activations and what each row is multiplied with."""
    if isinstance(x, torch.Tensor):
        return x.float(), 1.0
    if len(x) == 2:
        return x[0].float(), x[1][:, None]
    return _values(x[0], x[1]), x[2]


def _plain_act(name, v):
    if name == "relu":
        return v.clamp_min(0)
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * (1 / math.sqrt(2.0))))
    return v


def _plain_norm(st):
    h = st["x"].float() + st["r"].float()
    y = st["w"].float() * (h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS))
    top = y.abs().amax(1)
    s = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    return {"q": (y / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), "s": s, "h": h.to(st["x"].dtype)}


def _plain_balance(st):
    T, E = st["logits"].shape
    mask = st["mask"] if st["mask"] is not None else torch.ones(T, dtype=torch.bool, device=DEV)
    v = st["logits"].float()
    p = torch.exp(v - v.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True) * mask[:, None]
    hit = torch.where(mask[:, None], st["idx"], torch.full_like(st["idx"], -1))
    counts = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    counts.index_add_(0, hit.flatten() + 1, torch.ones(hit.numel(), dtype=torch.int32, device=DEV))
    counts = counts[1:]
    n = mask.sum().clamp_min(1)
    slope = COEF * E * counts.double() / counts.sum().clamp_min(1) / n
    loss = (slope * p.sum(0, dtype=torch.float64)).sum().float()
    slope = slope.float()
    grad = st["dloss"] * p * (slope - (p * slope).sum(1, keepdim=True))
    offs = torch.cumsum((counts + ALIGN - 1) // ALIGN * ALIGN, 0).int()
    return {"loss": loss.reshape(1), "counts": counts, "offs": offs, "grad": grad.to(st["logits"].dtype)}


def _plain_linear(st):
    case = st["case"]
    x, sx = _plain_x(st["x"])
    v = (x @ _values(st["w"][0], st["w"][1]).t()) * (sx * st["w"][2])
    if st["bias"] is not None:
        v = v + st["bias"].float()
    v = _plain_act(case["act"], v)
    if st["res"] is not None:
        v = v + st["res"].float()
    return {"y": v.to(FLOATS[case["out"]])}


def _plain_grouped(st):
    """The groups padded to the largest, one batched product, and back."""
    case, offs = st["case"], st["offs"].long()
    M, N = case["M"], case["N"]
    x, sx = _plain_x(st["x"])
    x = x * (sx * st["w"][2])
    start = torch.cat((offs.new_zeros(1), offs[:-1]))
    rows = start[:, None] + st["first"]
    live = rows < offs[:, None]
    v = torch.matmul(x[rows.clamp_max(M - 1)], _values(st["w"][0], st["w"][1]).transpose(1, 2))
    if st["bias"] is not None:
        v = v + st["bias"].float()[:, None]
    v = _plain_act(case["act"], v)
    y = torch.zeros(M + 1, N, device=DEV)
    y[torch.where(live, rows, torch.full_like(rows, M)).flatten()] = v.flatten(0, 1)
    y = y[:M]
    if st["res"] is not None:
        y = y + st["res"].float() * (torch.arange(M, device=DEV) < offs[-1])[:, None]
    return {"y": y.to(FLOATS[case["out"]])}


# --------------------------------------------------------------------- run


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        plain = {"norm": _plain_norm, "balance": _plain_balance, "linear": _plain_linear, "grouped": _plain_grouped}
        return plain[op](st)
    import nvfp4_adaptive_block_amd as fos

    if op == "norm":
        q, s, h = fos.fos_rmsnorm_quantize(st["x"], st["w"], residual=st["r"], eps=EPS)
        return {"q": q, "s": s, "h": h}
    if op == "balance":
        loss, counts, offs, slope = fos.fos_balance_loss(st["logits"], st["idx"], coef=COEF, mask=st["mask"],
                                                         align=ALIGN)
        grad = fos.fos_balance_loss_backward(st["dloss"], st["logits"], slope, mask=st["mask"])
        return {"loss": loss, "counts": counts, "offs": offs, "grad": grad}
    more = {"bias": st["bias"], "act": case["act"], "residual": st["res"], "out_dtype": FLOATS[case["out"]]}
    if op == "linear":
        return {"y": fos.fos_linear(st["x"], st["w"], **more)}
    return {"y": fos.fos_linear_grouped(st["x"], st["w"], st["offs"], **more)}


# ------------------------------------------------------------------- exact


def _decoded64(codes, scales):
    """float64 values from the formats' definitions: sign, exponent, mantissa."""
    c = torch.stack((codes % 16, codes // 16), -1).flatten(-2).to(torch.int32)
    e, m = (c // 2) % 4, c % 2
    v = torch.where(e == 0, 0.5 * m.double(), torch.exp2(e.double() - 1) * (1 + 0.5 * m.double()))
    v = torch.where(c >= 8, -v, v)
    s = scales.to(torch.int32)
    e, m = (s // 8) % 16, (s % 8).double()
    b = torch.where(e == 0, m * 2.0 ** -9, torch.exp2(e.double() - 7) * (1 + m / 8))
    return v * b.repeat_interleave(16, -1)


def _exact_act(name, v):
    if name == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return v * 0.5 * torch.erfc(-v * math.sqrt(0.5))
    return v


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        h = st["x"].double() + st["r"].double()
        y = st["w"].double() * h / torch.sqrt((h ** 2).sum(1, keepdim=True) / case["K"] + EPS)
        s = y.abs().max(1).values / 448
        s[s == 0] = 1
        return {"q": y / s[:, None], "s": s, "h": h}  # before their roundings
    if case["op"] == "balance":
        T, E = case["T"], case["E"]
        live = torch.ones(T, device=DEV).double() if st["mask"] is None else st["mask"].double()
        p = torch.softmax(st["logits"].double(), 1)
        experts = torch.arange(E, device=DEV)
        c = sum((live[:, None] * (st["idx"][:, j:j + 1] == experts)).sum(0) for j in range(case["k"]))
        f, n = c / max(1.0, float(c.sum())), max(1.0, float(live.sum()))
        P = (p * live[:, None]).sum(0) / n
        loss = COEF * E * (f * P).sum()
        g = float(st["dloss"]) * COEF * E / n * live[:, None] * p * (f - (p @ f)[:, None])
        counts = c.round().to(torch.int32)
        return {"loss": loss.reshape(1), "counts": counts,
                "offs": torch.cumsum(torch.ceil(c / ALIGN) * ALIGN, 0).to(torch.int32), "grad": g}
    x = st["x"]
    if isinstance(x, torch.Tensor):
        x = x.double()
    elif len(x) == 2:
        x = x[0].double() * x[1].double()[:, None]
    else:
        x = _decoded64(x[0], x[1]) * x[2].double()
    M, N, G = case["M"], case["N"], case.get("G", 1)
    ends = st["offs"].tolist() if case["op"] == "grouped" else [M]
    codes, scales = st["w"][0].reshape(G, N, -1), st["w"][1].reshape(G, N, -1)
    y = torch.zeros(M, N, dtype=torch.float64, device=DEV)
    at = 0
    for g, end in enumerate(ends):
        if end > at:
            v = x[at:end] @ (_decoded64(codes[g], scales[g]) * st["w"][2].double()).T
            if st["bias"] is not None:
                v += st["bias"].reshape(G, N)[g].double()
            v = _exact_act(case["act"], v)
            if st["res"] is not None:
                v += st["res"][at:end].double()
            y[at:end] = v
            at = end
    return {"y": y}
