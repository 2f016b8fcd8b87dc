"""A mixture-of-experts feed-forward block on NVFP4 weights, end to end on the
library's operators:

  norm      h = x + residual, its RMS norm as E4M3 rows (and in 16 bits for the router)
  router    logits, the k best experts of each token, the load-balance loss, the
            tokens per expert and the padded group offsets
  experts   the token rows packed by expert, times each expert's up projection
            with SiLU, quantized to NVFP4 per group, times its down projection
  shared    one dense expert beside them: up projection with GELU, down
            projection with h added in the epilogue
  backward  the balance loss's gradient into the router's weight

    python examples/moe_feed_forward.py [--tokens 512] [--width 1024] [--hidden 2048] [--experts 8] [--top 2]

prints how far the block is from the same block on unquantized weights and
activations, and its time per pass.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_adaptive_block_amd as fos  # noqa: E402

ALIGN = 16  # rows per expert are padded to this, as the grouped quantizer wants
KNOBS = dict(recipe="4over6", err_metric="mse")


def make_weights(width, hidden, experts, seed=0, device="cuda"):
    g = torch.Generator(device)
    g.manual_seed(seed)

    def rand(*shape):
        return (torch.randn(*shape, generator=g, device=device) * shape[-1] ** -0.5).bfloat16()

    return {"norm": (1 + 0.1 * torch.randn(width, generator=g, device=device)).bfloat16(),
            "router": rand(experts, width).float(), "up": rand(experts, hidden, width),
            "down": rand(experts, width, hidden), "shared_up": rand(hidden, width), "shared_down": rand(width, hidden)}


def quantize_weights(w):
    """Each matrix as (codes, scales, sdec): an expert's rows are quantized in
    one flattened call under one scale for all experts."""
    out = dict(w)
    for name in ("up", "down", "shared_up", "shared_down"):
        flat = w[name].flatten(0, -2)
        codes, scales, sdec = fos.fos_quantize(flat, fos.fos_amax(flat), **KNOBS)
        lead = w[name].shape[:-1]
        out[name] = (codes.view(*lead, -1), scales.view(*lead, -1), sdec)
    return out


def pack(idx, counts, offs):
    """Row of the packed tensor for each (token, choice), experts in order,
    each expert's rows in token order from its padded start."""
    flat = idx.flatten()
    order = flat.argsort(stable=True)
    first = torch.cumsum(counts, 0) - counts               # of each expert, unpadded
    start = torch.cat((offs.new_zeros(1), offs[:-1]))      # padded
    rank = torch.arange(flat.numel(), device=flat.device) - first[flat[order]]
    rows = torch.empty_like(flat)
    rows[order] = start[flat[order]] + rank
    return rows.view_as(idx)


def forward(x, residual, w, top):
    """Returns (output, balance loss, what backward needs)."""
    T, width = x.shape
    experts = w["router"].shape[0]
    y = torch.empty_like(x)
    q, s, h = fos.fos_rmsnorm_quantize(x, w["norm"], residual=residual, y=y)

    logits = y.float() @ w["router"].t()
    gates, idx = torch.softmax(logits, 1).topk(top, 1)
    loss, counts, offs, slope = fos.fos_balance_loss(logits, idx, align=ALIGN)

    rows = pack(idx, counts, offs)
    room = T * top + ALIGN * experts  # what any choice of experts can need
    token = torch.arange(T, device=x.device).repeat_interleave(top)
    xq = torch.zeros(room, width, dtype=torch.uint8, device=x.device)
    xs = torch.ones(room, device=x.device)
    xq[rows.flatten()] = q.view(torch.uint8)[token]
    xs[rows.flatten()] = s[token]

    up = fos.fos_linear_grouped((xq.view(torch.float8_e4m3fn), xs), w["up"], offs, act="silu")
    codes, scales, _, sdec = fos.fos_quantize_grouped_fused(up, offs, **KNOBS)
    down = fos.fos_linear_grouped((codes, scales, sdec), w["down"], offs, x_gran="group")
    mixed = (down[rows].float() * gates[..., None]).sum(1)

    shared = fos.fos_linear((q, s), w["shared_up"], act="gelu")
    out = fos.fos_linear(shared, w["shared_down"], residual=h)
    return (out.float() + mixed).to(x.dtype), loss, (y, logits, slope)


def router_gradient(saved, dloss):
    """The balance loss's gradient with respect to the router's weight."""
    y, logits, slope = saved
    return fos.fos_balance_loss_backward(dloss, logits, slope).t() @ y.float()


def reference(x, residual, w, top):
    """The same block in float32 on the unquantized weights."""
    h = x.float() + residual.float()
    y = w["norm"].float() * h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6)
    p = torch.softmax(y.bfloat16().float() @ w["router"].t(), 1)
    gates, idx = p.topk(top, 1)
    mixed = torch.zeros_like(h)
    for e in range(w["router"].shape[0]):
        t, c = (idx == e).nonzero(as_tuple=True)
        v = torch.nn.functional.silu(y[t] @ w["up"][e].float().t()) @ w["down"][e].float().t()
        mixed.index_add_(0, t, v * gates[t, c, None])
    shared = torch.nn.functional.gelu(y @ w["shared_up"].float().t()) @ w["shared_down"].float().t()
    return h + shared + mixed


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 512), ("width", 1024), ("hidden", 2048), ("experts", 8), ("top", 2)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    w = make_weights(a.width, a.hidden, a.experts)
    wq = quantize_weights(w)
    x = torch.randn(a.tokens, a.width, device="cuda").bfloat16()
    residual = torch.randn(a.tokens, a.width, device="cuda").bfloat16()
    out, loss, saved = forward(x, residual, wq, a.top)
    grad = router_gradient(saved, torch.ones(1, device="cuda"))
    want = reference(x, residual, w, a.top)
    h = x.float() + residual.float()
    off = float((out.float() - want).norm() / (want - h).norm())
    for _ in range(3):
        forward(x, residual, wq, a.top)
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(20):
        forward(x, residual, wq, a.top)
    torch.cuda.synchronize()
    print(f"tokens {a.tokens} width {a.width} hidden {a.hidden} experts {a.experts} top {a.top}: "
          f"relative error of the block's update {off:.4f}, balance loss {float(loss):.5f}, "
          f"router gradient norm {float(grad.norm()):.3e}, {(time.perf_counter() - start) / 20 * 1e6:.0f} us a pass")


if __name__ == "__main__":
    main()
