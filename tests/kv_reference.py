"""A paged NVFP4 key/value cache on the CPU for the tests: random caches with
stale rows around the live ones, 64-bit references, and the error bounds of the
kernels' arithmetic."""
import math

import torch

from operator_reference import DTYPES, decode_nvfp4, gen, half_step, random_nvfp4

E24 = 2.0 ** -24


class Cache:
    """B sequences of lens tokens in shuffled pages of P rows for H heads of D
    values. What lies outside the sequences is NaN scales and infinities, and table
    entries past a sequence's pages are no pages."""

    def __init__(self, lens, H, D, P, seed=0, W=None, sizes=None):
        g = gen(seed)
        self.lens, self.H, self.D, self.P, self.B = list(lens), H, D, P, len(lens)
        used = [-(-n // P) for n in lens]
        self.W = W or max(1, max(used))
        self.pages = sum(used) + 2
        order = torch.randperm(self.pages, generator=g).tolist()
        self.table = torch.full((self.B, self.W), -7, dtype=torch.int32)
        self.table[:, 1::2] = 2 ** 30
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = torch.tensor(order[at:at + u], dtype=torch.int32)
            at += u
        live = torch.zeros(self.pages, P, dtype=torch.bool)
        for b, n in enumerate(lens):
            for i in range(used[b]):
                live[self.table[b, i], :min(P, n - i * P)] = True
        live = live[:, None, :].expand(-1, H, -1)
        self.sides = []
        for side in range(2):
            codes, scales = random_nvfp4(self.pages * H * P, D, seed + 17 * side + 1)
            sdec = torch.exp(0.7 * torch.randn(self.pages * H * P, generator=g))
            sdec *= (0.02 if side == 0 else 0.01) if sizes is None else sizes[side]
            if side == 1:  # rows of zeros, as the append writes them
                zero = torch.rand(self.pages * H * P, generator=g) < 0.03
                codes[zero], scales[zero], sdec[zero] = 0, 0, 0.0
            codes, scales = codes.view(self.pages, H, P, D // 2), scales.view(self.pages, H, P, D // 16)
            sdec = sdec.view(self.pages, H, P)
            scales[~live] = 0x7F
            sdec[~live] = math.nan
            sdec[:, :, ::3][~live[:, :, ::3]] = math.inf
            self.sides.append((codes, scales, sdec))

    def on_device(self):
        """(k_cache, v_cache, table, lens) on the device."""
        k, v = (tuple(t.cuda() for t in side) for side in self.sides)
        return k, v, self.table.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda()

    def rows(self, side, b, n=None):
        """(values without S_dec [H, n, D], S_dec [H, n]) of sequence b in float64."""
        n = self.lens[b] if n is None else n
        page = self.table[b, : -(-n // self.P)].long()
        c, s, d = (t[page].transpose(0, 1).flatten(1, 2)[:, :n] for t in self.sides[side])
        return decode_nvfp4(c.contiguous(), s.contiguous()), d.double()


def queries(T, Hq, D, dtype, seed, size=1.0):
    return (size * torch.randn(T, Hq, D, generator=gen(seed))).to(DTYPES[dtype])


def scores(cache, q, new, b, start, causal, scale):
    """(s [Hq, n, L], -inf where a key is not seen; its error; G) of sequence b."""
    n, L, G = new[b], cache.lens[b], q.shape[1] // cache.H
    kv, kd = cache.rows(0, b)
    k = (kv * kd[..., None]).repeat_interleave(G, 0)
    x = q[start:start + n].double().transpose(0, 1)
    s = scale * (x @ k.transpose(1, 2))
    size = abs(scale) * (x.abs() @ k.abs().transpose(1, 2))
    # the sum of D products in binary32, in any order (a random walk of four standard
    # steps); S_dec, scale and the power of two onto it; the exponent's difference from m
    # and its base-2 logarithm: six roundings of at most the largest score
    err = (4 * math.sqrt(cache.D) + 8) * E24 * size
    # bf16 queries in fp16: what lies below 2^-32 of the largest is off by 2^-40 of it
    err = err + abs(scale) * 2.0 ** -40 * x.abs().amax(-1, keepdim=True) * k.abs().sum(-1)[:, None]
    seen = torch.ones(n, L, dtype=torch.bool)
    if causal:
        seen = torch.arange(L)[None] < (L - n + torch.arange(n) + 1)[:, None]
    top = torch.where(seen, s.abs(), torch.zeros_like(s)).amax(-1, keepdim=True) if L else torch.zeros(s.shape[0], n, 1)
    err = err + 6 * E24 * top
    return s.masked_fill(~seen, -math.inf), err, G


def attention(cache, q, new, causal=True, scale=None):
    """(out, its bound, lse, its bound) for packed queries q [T, Hq, D] on the CPU,
    new[b] of them sequence b's; rows behind the last sequence are empty."""
    scale = cache.D ** -0.5 if scale is None else scale
    T, Hq, D = q.shape
    out, bound = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    lse, lb = torch.full((T, Hq), -math.inf, dtype=torch.float64), torch.zeros(T, Hq, dtype=torch.float64)
    at = 0
    for b, n in enumerate(new):
        L = cache.lens[b]
        if n and L:
            s, err, G = scores(cache, q, new, b, at, causal, scale)
            vv, vd = (t.repeat_interleave(G, 0) for t in cache.rows(1, b))
            z = torch.logsumexp(s, -1)
            w = torch.exp(s - z.clamp_min(-1e300)[..., None])
            o = (w * vd[:, None]) @ vv
            size = (w * vd[:, None]) @ vv.abs()
            # weights: the scores' errors, three steps of the exponential; the sums of L terms
            ew = torch.where(w > 0, err, torch.zeros_like(err)).amax(-1) + 3 * 2.0 ** -23
            # m lies within 7 of max_j z_j + log2 max(S_j, 2^-90), so for a weight that counts |z_j - m|
            # is at most the largest |log2 max(S_j, 2^-90)| and 7: it is rounded when it is taken
            # (2^-24 of it), between parts (2^-24), and as log2 of the sum of L such (a step, 2^-23)
            far = vd.clamp_min(2.0 ** -90).log2().abs().amax(-1) + 7 + math.log2(L)
            ew = ew + 4 * E24 * math.log(2) * far[:, None]
            es = (4 * math.sqrt(L) + 16) * E24
            # weights times S_dec in fp16: half a step of fp16, 2^-11, or below fp16's normal range
            # 2^-25 of the unit 2^m. m is the running maximum of z_j + log2 max(S_j, 2^-90), so in the
            # result's terms, after the division by sum_j 2^(z_j - m), the unit is at most
            # max_j w_j max(S_j, 2^-90): a row of zeros (S = 0) has no size, but its weight counts
            floor = 2.0 ** -25 * (w * vd[:, None].clamp_min(2.0 ** -90)).amax(-1)[..., None] * vv.abs().sum(1)[:, None]
            e = size * (2 * ew + 2 ** -11 + es)[..., None] + floor
            tiny = torch.finfo(q.dtype).smallest_normal * torch.finfo(q.dtype).eps
            e = e + half_step(q.dtype) * (o.abs() + e) + tiny
            out[at:at + n], bound[at:at + n] = o.transpose(0, 1), e.transpose(0, 1)
            lse[at:at + n] = z.T
            lb[at:at + n] = (ew + es + 8 * E24 * z.abs().clamp(max=1e30)).T
        at += n
    return out, bound, lse, lb


def weights(cache, q, new, lse, causal=True, scale=None):
    """(sums [B, H, W P], bound) that the weights call adds, with the lse given."""
    scale = cache.D ** -0.5 if scale is None else scale
    acc = torch.zeros(cache.B, cache.H, cache.W * cache.P, dtype=torch.float64)
    bound = torch.zeros_like(acc)
    at = 0
    for b, n in enumerate(new):
        L = cache.lens[b]
        if n and L:
            s, err, G = scores(cache, q, new, b, at, causal, scale)
            z = lse[at:at + n].double().T[..., None]
            w = torch.where(z > -math.inf, torch.exp(s - z), torch.zeros_like(s))
            # the scores' errors, lse in base 2 (two roundings), three steps of the
            # exponential, and the sum over the rows
            e = w * (err + 2 * E24 * z.abs().clamp(max=1e30) + 3 * 2.0 ** -23)
            acc[b, :, :L] = w.reshape(cache.H, G * n, L).sum(1)
            bound[b, :, :L] = e.reshape(cache.H, G * n, L).sum(1) + (4 * math.sqrt(n * G) + 8) * E24 * acc[b, :, :L]
        at += n
    return acc, bound


def evict(cache, acc, budget, sinks, recent):
    """Per sequence and head the index that each kept row comes from; the new acc."""
    keep, came = budget - recent, {}
    new = acc.clone()
    for b, n in enumerate(cache.lens):
        if n <= budget:
            continue
        for h in range(cache.H):
            a = acc[b, h].tolist()
            rank = [(-math.inf if math.isnan(v) else v) for v in a]
            nan = [math.isnan(v) for v in a]
            middle = sorted(range(sinks, n - recent), key=lambda i: (nan[i], -rank[i], i))
            kept = set(range(sinks)) | set(middle[: keep - sinks])
            free = [i for i in range(keep) if i not in kept]
            moved = [i for i in range(keep, n - recent) if i in kept]
            assert len(free) == len(moved)
            src = list(range(keep)) + list(range(n - recent, n))
            for f, m in zip(free, moved):
                src[f] = m
            came[b, h] = src
            new[b, h, :budget] = acc[b, h, src]
            new[b, h, budget:n] = 0.0
    return came, new
