"""The key/value cache's calls where they can go wrong: what the plain tests of
test_gpu_kv.py do not reach. GPU only."""
import math

import pytest
import torch

import kv_reference as ref
import nvfp4_adaptive_block_amd as fos
from operator_reference import DTYPES, assert_within, gen, half_step
from test_gpu_kv import (DIMS, LONG, WIDE, assert_guard, attend, check_append, check_attention, check_evict, check_weights,
                         ends, guarded, oracle_rows, rows_like, same)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- evict


@pytest.mark.parametrize("middle", [1, 2, 33, 63, 64, 65, 96, 127, 128])
def test_evict_short_middles(middle):
    """Few rows to choose from, no two weights alike: waves without a row of their own."""
    def distinct(shape):
        order = torch.stack([torch.randperm(shape[-1], generator=gen(i)) for i in range(shape[0] * shape[1])])
        return ((order + 1).float() * 2.0 ** -7).view(shape)

    n, sinks, recent = middle + 24, 4, 20
    for budget in sorted({sinks + recent, n - 1, sinks + recent + middle // 2}):
        check_evict([n, n + 1], 64, 64, 16, budget, sinks, recent, seed=middle, acc=distinct)


@pytest.mark.parametrize("budget", [40, 1200])
def test_evict_bad_lengths(budget):
    """In one launch and in three: lengths past the table are cut to it, negative ones are empty."""
    H, D, P, W = 2, 32, 64, 60
    cache = ref.Cache([W * P, 30, W * P], H, D, P, seed=9)
    acc = torch.rand(3, H, W * P, generator=gen(10))
    results = []
    for lens in ([W * P, 0, W * P], [2 ** 31 - 1, -1, W * P + 1], [W * P + 7, -2 ** 31, W * P]):
        kc, vc, table, _ = cache.on_device()
        acc_d = acc.cuda()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        n = torch.tensor(lens, dtype=torch.int32).cuda()
        new = fos.fos_kv_evict(acc_d, kc, vc, table, n, budget, sinks=2, recent=30, status=status)
        assert int(status.item()) == (fos.STATUS_BAD_CACHE if results else 0)
        assert new.tolist() == [budget, 0, budget]
        results.append([acc_d, *kc, *vc])
    for got in results[1:]:
        assert all(same(a, b) for a, b in zip(got, results[0]))


# ------------------------------------------------------------------ append


def test_append_to_lengths_past_the_table(orc):
    """They are taken as the table's end, as the attention takes them: the new rows are its last."""
    H, D, P = 2, 64, 16
    x = rows_like((9, H, D), "bf16", 7).cuda()
    offs = torch.tensor([4, 4, 9], dtype=torch.int32).cuda()
    table = torch.tensor([[2, 0], [1, 3], [4, 5]], dtype=torch.int32).cuda()
    codes, scales, sdec, _ = oracle_rows(orc, x.cpu())
    for lens in ([32, 0, 32], [33, 0, 10 ** 9], [2 ** 31 - 1, 0, 40]):
        kc, vc = (fos.fos_kv_cache(6, H, P, D) for _ in range(2))
        status = torch.zeros(1, dtype=torch.int32).cuda()
        fos.fos_kv_append(x, x, offs, kc, vc, table, torch.tensor(lens, dtype=torch.int32).cuda(), status=status)
        assert int(status.item()) == (0 if max(lens) == 32 else fos.STATUS_BAD_CACHE)
        want = [torch.zeros_like(t).cpu() for t in kc]
        for b, start, n, page in ((0, 0, 4, 0), (2, 4, 5, 5)):
            for i in range(n):
                r = (start + i) * H
                for w, o in zip(want, (codes, scales, sdec)):
                    w[page, :, P - n + i] = torch.from_numpy(o[r:r + H])
        for side in (kc, vc):
            assert all(same(t, w) for t, w in zip(side, want))


@pytest.mark.parametrize("length", [33, -1, -2 ** 31])
def test_append_reports_lengths_of_sequences_without_new_rows(length):
    kc, vc = (fos.fos_kv_cache(4, 2, 16, 64) for _ in range(2))
    table = torch.arange(4, dtype=torch.int32).view(2, 2).cuda()
    x = torch.ones(3, 2, 64, device="cuda")
    for bad in (False, True):
        status = torch.zeros(1, dtype=torch.int32).cuda()
        lens = torch.tensor([3, length if bad else 32], dtype=torch.int32).cuda()
        fos.fos_kv_append(x, x, torch.tensor([3, 3], dtype=torch.int32).cuda(), kc, vc, table, lens, status=status)
        assert int(status.item()) == (fos.STATUS_BAD_CACHE if bad else 0)


def test_append_bad_offsets():
    """Reported; no row goes outside the pages that the table names, or the outputs."""
    H, D, P, T = 2, 64, 16, 70
    x = rows_like((T, H, D), "fp16", 8).cuda()
    table = torch.tensor([[1, 2, 5], [3, 6, 7]], dtype=torch.int32).cuda()
    lens = torch.tensor([48, 40], dtype=torch.int32).cuda()
    for offs in ([T - 1, T - 2], [2, T + 5], [-1, T], [2 ** 31 - 1, -2 ** 31], [-2 ** 31, 2 ** 31 - 1], [T, 0]):
        kc, vc = (fos.fos_kv_cache(9, H, P, D) for _ in range(2))
        for side in (kc, vc):
            for t in side:
                t.fill_(77)
        ko, raw = guarded((T, H, D), x.dtype)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        fos.fos_kv_append(x, x, torch.tensor(offs, dtype=torch.int32).cuda(), kc, vc, table, lens, k_out=ko, status=status)
        assert int(status.item()) & fos.STATUS_BAD_OFFS
        assert_guard(raw)
        for side in (kc, vc):
            for t in side:
                assert (t[[0, 4, 8]] == 77).all()


@pytest.mark.parametrize("B,most", [(300, 2), (5000, 2), (5000, 5)])
def test_append_to_many_sequences(orc, B, most):
    """A token here and there: sequences far apart in one wave."""
    g = gen(B)
    new = torch.where(torch.rand(B, generator=g) < 0.1, torch.randint(1, most, (B,), generator=g), 0)
    lens = (new + torch.randint(0, 5, (B,), generator=g)).tolist()
    check_append(orc, lens, new.tolist(), 1, 32, 16, "bf16", seed=B, tail=2)


# --------------------------------------------------------------- attention


def poison(cache, side, pos, what, block):
    """A row of the first head of the first sequence with a NaN block scale or an S_dec of `what`."""
    page, slot = int(cache.table[0, pos // cache.P]), pos % cache.P
    if what == "scale":
        cache.sides[side][1][page, 0, slot, block] = 0xFF if block % 2 else 0x7F
    else:
        cache.sides[side][2][page, 0, slot] = float(what)


@pytest.mark.parametrize("what", ["scale", "nan", "-nan", "inf"])
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("dtype,n,max_len", [("bf16", 7, 0), ("fp16", 24, 2000), ("bf16", 60, LONG), ("fp16", 60, LONG)])
def test_attention_rows_that_are_not_numbers(dtype, n, max_len, D, what):
    """A value row with a NaN reaches the queries that see it, in the block that it is in, and
    no others; the same for keys, whose queries are NaN as a whole."""
    G, L = 3, 150
    bad = [(L - 1, 0), (L - 5, D // 16 - 1), (L - n + 2, 1)]  # (place, block) of three of the new tokens
    cache = ref.Cache([L, 40], 2, D, 16, seed=D + n, W=WIDE if max_len == LONG else None)
    for pos, block in bad:  # whatever random rows hold there, a size that counts
        page, slot = int(cache.table[0, pos // 16]), pos % 16
        for _, scales, sdec in cache.sides:
            scales[page, 0, slot], sdec[page, 0, slot] = 0x38, 0.02
    q, new = ref.queries(2 * n, 2 * G, D, dtype, D + 1), [n, n]
    want, bound, want_lse, lse_bound = ref.attention(cache, q, new)
    keep = [tuple(t.clone() for t in side) for side in cache.sides]
    for side in (1, 0):
        cache.sides = [tuple(t.clone() for t in s) for s in keep]
        hit = torch.zeros(2 * n, 2 * G, D, dtype=torch.bool)
        for pos, block in bad:
            poison(cache, side, pos, what, block)
            where = slice(16 * block, 16 * block + 16) if what == "scale" and side == 1 else slice(None)
            hit[pos - (L - n):n, :G, where] = True
        out, lse, status = attend(cache, q, new, max_len=max_len)
        out, lse = out.cpu(), lse.cpu()
        assert status == 0
        whole, none = hit.all(-1), want_lse == -math.inf
        assert_within(out[~hit], want[~hit], bound[~hit], "out")
        assert torch.equal(lse == -math.inf, none)
        rest = ~whole & ~none
        assert_within(lse[rest], want_lse[rest], lse_bound[rest], "lse")
        if what != "inf":
            assert torch.isnan(out[hit]).all()
        elif side == 1:
            assert not torch.isfinite(out[hit]).any()
        if side == 0 and what != "inf":
            assert torch.isnan(lse[whole]).all()


@pytest.mark.parametrize("what", ["scale", "nan"])
@pytest.mark.parametrize("H,lens,new", [(30, [150, 33, 5], [80, 30, 5]), (2, [2500, 700], [60, 90])])
def test_attention_rows_that_are_not_numbers_in_tiles_of_many_heads_and_in_parts(H, lens, new, what):
    """Tiles whose keys are in one part, and in several, of which the last has the rows."""
    D = 64
    cache = ref.Cache(lens, H, D, 16, seed=H, W=None if H == 30 else WIDE)
    q = ref.queries(sum(new) + 3, H * 8 if H == 30 else 8, D, "bf16", H + 1)
    want, bound, want_lse, lse_bound = ref.attention(cache, q, new)
    G, L, n = q.shape[1] // H, lens[0], new[0]
    hit = torch.zeros(q.shape, dtype=torch.bool)
    for pos, block in ((L - 1, 0), (L - 33, 3)):
        poison(cache, 1, pos, what, block)
        hit[pos - (L - n):n, :G, slice(16 * block, 16 * block + 16) if what == "scale" else slice(None)] = True
    out, lse, _ = attend(cache, q, new, max_len=0 if H == 30 else LONG)
    out, lse = out.cpu(), lse.cpu()
    assert torch.isnan(out[hit]).all()
    assert_within(out[~hit], want[~hit], bound[~hit], "out")
    some = want_lse > -math.inf
    assert_within(lse[some], want_lse[some], lse_bound[some], "lse")


@pytest.mark.parametrize("n,max_len", [(3, 0), (60, LONG)])
def test_attention_a_nan_that_all_see(n, max_len):
    """In an early row, in a page's last place, and where some keys of the step are not there."""
    L, D = 130, 128
    cache = ref.Cache([L], 2, D, 16, seed=5, W=WIDE if max_len else None)
    for pos in (0, 47, L - n - 1):
        poison(cache, 1, pos, "scale", 2)
    cache.table[0, 1] = -1  # keys 16 to 31
    q = ref.queries(n, 4, D, "bf16", 6)
    for causal in (True, False):
        out, lse, _ = attend(cache, q, [n], causal=causal, max_len=max_len)
        nan = torch.isnan(out.cpu())
        assert nan[:, :2, 32:48].all() and not nan[:, 2:].any()
        assert not nan[:, :2, :32].any() and not nan[:, :2, 48:].any() and torch.isfinite(lse).all()


def one_row(sides, page, slot, values):
    """A row of block scales and S_dec of 1: values 0 and 1."""
    codes = (2 * values[0::2] + 32 * values[1::2]).to(torch.uint8)
    sides[0][page, 0, slot], sides[1][page, 0, slot], sides[2][page, 0, slot] = codes, 0x38, 1.0


def many_small_weights(B, G, N, dtype):
    """(out, lse, its value without rounding, the few keys' part of it, their values) of a few keys far
    ahead of very many. All sequences share one's pages, so that each workgroup walks over all keys."""
    D, P, a = 32, 2 ** 16, 18.5  # a query gives the few keys a weight e^a times the others'
    half = torch.arange(D) < D // 2
    k, v = (fos.fos_kv_cache(N // P, 1, P, D, device="cpu") for _ in range(2))
    one_row(k, slice(None), slice(None), torch.zeros(D, dtype=torch.int32))
    one_row(v, slice(None), slice(None), (~half).int())
    few = [0, 32, 64, 96]  # in the first step of each wave
    for pos in few:
        one_row(k, 0, pos, (torch.arange(D) < 1).int())
        one_row(v, 0, pos, half.int())
    k, v = (tuple(t.cuda() for t in side) for side in (k, v))
    table = torch.arange(N // P, dtype=torch.int32).expand(B, -1).contiguous().cuda()
    lens = torch.full((B,), N, dtype=torch.int32).cuda()
    q = torch.zeros(B, G, D, dtype=DTYPES[dtype])
    q[..., 0] = a
    if B > 1:
        assert fos.fos_kv_attention_workspace(B, G, B, N // P, 1, P, D) == 0  # one part
    out, lse = fos.fos_kv_attention(q.cuda(), ends([1] * B), k, v, table, lens, scale=1.0, causal=False)
    small = (N - len(few)) * math.exp(-a)
    part = len(few) / (len(few) + small)
    score = 6 * ref.E24 * a + 3 * 2.0 ** -23  # six roundings of a score of at most a log2 e, the exponential
    return out, lse, a + math.log(len(few) + small), part, half, score


MANY = [(2304, 1, 2 ** 20), (512, 64, 2 ** 18), (1, 4, 2 ** 20)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B,G,N", MANY)
def test_attention_sum_of_many_small_weights(B, G, N, dtype):
    """A step's weights are added up before they meet what a lane has: a wave of four has
    N / 128 steps of 32 keys, one of 32 rows N / 64 of 64, and each addition is off by half a step
    of binary32 at most, 2^-24 of the sum."""
    _, lse, want, _, _, score = many_small_weights(B, G, N, dtype)
    err = score + (N / (64 if G > 48 else 128) + 64) * ref.E24
    assert ((lse.cpu().double() - want).abs() < err).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B,G,N", MANY)
def test_attention_values_of_many_small_weights(B, G, N, dtype):
    """What very many small weights have together counts beside a few large ones."""
    out, _, _, part, half, score = many_small_weights(B, G, N, dtype)
    want = torch.where(half, part, 1 - part).double().expand(B, G, -1)
    # a weight in fp16: half a step, 2^-11, or below fp16's normal range 2^-25 where the few keys'
    # are 2^8 or more; then the sums of both, an addition a step as above and up to two for the
    # products; the result
    steps = N / (64 if G > 48 else 128) + 64
    bound = want * (2 * score + 2.0 ** -11 + 3 * steps * ref.E24) + (1 - part) / math.exp(-18.5) * 2.0 ** -33
    bound = bound + half_step(out.dtype) * (want + bound)
    assert_within(out, want, bound, "out")


@pytest.mark.parametrize("size_q,size_k,scale", [(2.0 ** -108, 2.0 ** 106, 0.125), (2.0 ** -115, 2.0 ** 112, 0.125),
                                                 (2.0 ** 110, 2.0 ** -112, 0.125), (1.0, 2.0 ** 110, 2.0 ** -115),
                                                 (2.0 ** -100, 1.0, 2.0 ** 96), (1.0, 0.02, 0.125)])
def test_scores_between_rows_of_opposite_sizes(size_q, size_k, scale):
    """Scores of ordinary size from queries, keys and scales that are not: no product on the way
    leaves binary32's range. Attention of few rows and of many, whose queries have a power of two
    each or one for all; weights of 32 rows and of 256."""
    for G, n, max_len in ((3, 2, 0), (4, 25, LONG), (2, 200, 0)):
        cache = ref.Cache([230, 210], 2, 64, 16, seed=31, sizes=(size_k, 0.01), W=WIDE if max_len else None)
        q = ref.queries(2 * n, 2 * G, 64, "bf16", 32)
        for spread in (1.0, 2.0 ** -11):  # rows of one size and of two
            q[::3] *= spread
            x = (q.double() * size_q).bfloat16()
            check_attention(cache, x, [n, n], scale=scale, max_len=max_len)
            if not max_len:
                check_weights(cache, x, [n, n], scale=scale)


@pytest.mark.parametrize("scale", [3e38, -3e38, 2.0 ** -140, 1e-45])
def test_scales_at_the_end_of_the_range(scale):
    """The largest and the smallest scale that float32 has."""
    cache = ref.Cache([50, 9], 2, 64, 16, seed=33, sizes=(0.02, 0.01))
    size = 1 / abs(scale) if abs(scale) > 1 else 2.0 ** 120
    q = (ref.queries(4, 4, 64, "bf16", 34).double() * size).bfloat16()
    check_attention(cache, q, [2, 2], scale=scale)


@pytest.mark.parametrize("n,max_len", [(1, 0), (60, LONG)])
def test_small_values_beside_a_large_one(n, max_len):
    """bf16 queries go through fp16 times a power of two: a value of eight bits down to 2^-32 of the
    row's largest is exact, and where rows of 2^-8 of the tile's largest share theirs, too, as long
    as it is 2^-32 of the tile's. A key that has only the small value's place shows it."""
    D, small = 64, (1 + 2.0 ** -7) * 2.0 ** -32
    L = max(n, 40)
    cache = ref.Cache([L], 1, D, 16, seed=41, W=WIDE if max_len else None)
    for t in cache.sides[0]:
        t.zero_()
    cache.sides[0][2].fill_(1.0)
    cache.sides[0][1].fill_(0x38)
    at = int(cache.table[0, 0])
    cache.sides[0][0][at, 0, 0, 0] = 0x20  # the first key: 1 in the second place
    q = torch.zeros(n, 2, D, dtype=torch.bfloat16)
    q[..., 0] = 1.0
    q[:, 1, 0] = 2.0 ** -8
    q[..., 1] = small
    assert (q[..., 1].double() == small).all()
    scale = 2.0 ** 34
    want, bound, want_lse, _ = ref.attention(cache, q, [n], scale=scale)
    out, lse, _ = attend(cache, q, [n], scale=scale, max_len=max_len)
    # exact queries: the score's and the sums' roundings alone (a score of 4, L weights)
    err = (6 * 4 + 4 * math.sqrt(L) + 40) * ref.E24
    assert ((lse.cpu().double() - want_lse).abs() < err).all()
    assert_within(out, want, bound, "out")
    if not max_len:
        acc = torch.zeros(1, 1, cache.W * 16, device="cuda")
        k, v, table, lens = cache.on_device()
        fos.fos_kv_weights(q.cuda(), ends([n]), k, table, lens, lse, acc, scale=scale)
        sums, _ = ref.weights(cache, q, [n], lse.cpu(), scale=scale)
        assert ((acc.cpu().double() - sums).abs() <= 2 * n * err * sums).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", DIMS)
def test_attention_short_caches_of_many_sequences(D, dtype):
    """As many tiles as CUs, each walking over a whole cache, and more."""
    for B, whole in ((32, D <= 192), (33, False)):
        lens = torch.randint(0, 290, (B,), generator=gen(D)).tolist()
        lens[3], lens[4], lens[5] = 290, 1, 0
        cache = ref.Cache(lens, 8, D, 16, seed=D)
        need = fos.fos_kv_attention_workspace(B, 16, B, cache.W, 8, 16, D)
        assert need == 0 if whole else need > 0
        check_attention(cache, ref.queries(B, 16, D, dtype, D + 1), [1] * B)


@pytest.mark.parametrize("B,G,most", [(257, 3, 3), (700, 2, 2), (700, 16, 9), (4200, 1, 2)])
def test_attention_batches_of_many_sequences(B, G, most):
    """Their sequences are found by search: ragged ones, a long run without new tokens, and a tail.
    Tiles of 16 rows and, with sixteen query heads and up to eight tokens each, of 128."""
    g = gen(B + G)
    new = torch.randint(0, most, (B,), generator=g)
    new[B // 2:B // 2 + 90] = 0
    lens = new + torch.randint(0, 40, (B,), generator=g)
    cache = ref.Cache(lens.tolist(), 1, 32, 16, seed=B)
    T = int(new.sum())
    q = ref.queries(T + 3, G, 32, "bf16", B)
    if G == 16:
        assert T * G > 48 * B
    check_attention(cache, q, new.tolist())
    k, v, table, lens_d = cache.on_device()
    good = new.cumsum(0).int()
    for at, bad in ((B // 3, -1), (B - 1, T + 9), (0, 2 ** 31 - 1), (B - 2, -2 ** 31)):
        offs = good.clone()
        offs[at] = bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, raw = guarded(q.shape, q.dtype)
        fos.fos_kv_attention(q.cuda(), offs.cuda(), k, v, table, lens_d, out=out, status=status)
        assert int(status.item()) == fos.STATUS_BAD_OFFS
        assert_guard(raw)


# ----------------------------------------------------------------- weights


def add_weights(cache, q, offs, lse, causal=True):
    """(acc after the call, acc before it, status)."""
    k, v, table, lens = cache.on_device()
    start = torch.rand(cache.B, cache.H, cache.W * cache.P, generator=gen(1)).cuda()
    acc, raw = guarded(start.shape, torch.float32)
    acc.copy_(start)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fos.fos_kv_weights(q.cuda(), torch.tensor(offs, dtype=torch.int32).cuda(), k, table, lens, lse.cuda(), acc,
                       causal=causal, status=status)
    assert_guard(raw)
    return acc.cpu(), start.cpu(), int(status.item())


def check_sums(acc, want, bound):
    """What is past float32's range has become an infinity."""
    over = want > 3.5e38
    assert (acc[over] == math.inf).all()
    assert_within(acc[~over], want[~over], bound[~over], "acc")


@pytest.mark.parametrize("n,G", [(2, 3), (16, 2), (17, 2), (100, 4)])
def test_weights_bad_cache(n, G):
    """32 rows staged and 256. Pages that are none add nothing to their keys; lengths past the
    table end with it, negative ones have no keys."""
    cache = ref.Cache([64, 50], 2, 64, 16, seed=61)
    q = ref.queries(2 * n, 2 * G, 64, "bf16", 62)
    lse = 3 + torch.rand(2 * n, 2 * G, generator=gen(63))  # any: the sums are of exp(s - lse)
    keep = cache.table.clone()
    want, bound = ref.weights(cache, q, [n, n], lse, causal=False)
    parts = -(-n * G // 32)
    for bad in (cache.pages, -1, -2 ** 31, 2 ** 31 - 1):
        cache.table = keep.clone()
        cache.table[0, 1], cache.table[1, 3] = bad, -1  # keys 16 to 31, and 48 and 49
        acc, start, status = add_weights(cache, q, [n, 2 * n], lse, causal=False)
        assert status == 0
        gone = torch.zeros_like(acc, dtype=torch.bool)
        gone[0, :, 16:32] = gone[1, :, 48:] = True
        assert same(acc[gone], start[gone])
        total = want + start.double()
        check_sums(acc[~gone], total[~gone], (bound + ref.E24 * parts * total.abs())[~gone])
    cache.table = keep
    for lens, taken in (([64, -5], [64, 0]), ([10 ** 6, 50], [64, 50]), ([2 ** 31 - 1, -2 ** 31], [64, 0])):
        cache.lens = lens
        acc, start, status = add_weights(cache, q, [n, 2 * n], lse)
        assert status == fos.STATUS_BAD_CACHE
        cache.lens = taken
        sums, bound = ref.weights(cache, q, [n, n], lse)
        total = sums + start.double()
        check_sums(acc, total, bound + ref.E24 * parts * total.abs())
        for b, length in enumerate(taken):
            assert same(acc[b, :, length:], start[b, :, length:])


@pytest.mark.parametrize("n,G", [(4, 2), (60, 3)])
def test_weights_bad_offsets(n, G):
    cache = ref.Cache([64, 50], 2, 64, 16, seed=64)
    q = ref.queries(n, 2 * G, 64, "bf16", 65)
    lse = 3 + torch.rand(n, 2 * G, generator=gen(66))
    for offs in ([n - 1, n - 2], [2, n + 5], [-1, n], [2 ** 31 - 1, -2 ** 31]):
        acc, start, status = add_weights(cache, q, offs, lse)
        assert status == fos.STATUS_BAD_OFFS
        assert same(acc[1, :, 50:], start[1, :, 50:])


# ---------------------------------------------------------------- together


@pytest.mark.parametrize("B", [2, 300])
def test_calls_without_tokens_report_what_is_bad(B):
    cache = ref.Cache([33] * B, 2, 64, 16, seed=51)
    k, v, table, lens = cache.on_device()
    none = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    acc = torch.zeros(B, 2, cache.W * 16, device="cuda")

    def calls(offs, lens):
        yield lambda **kw: fos.fos_kv_append(none, none, offs, k, v, table, lens, **kw)
        yield lambda **kw: fos.fos_kv_attention(none, offs, k, v, table, lens, **kw)
        yield lambda **kw: fos.fos_kv_weights(none, offs, k, table, lens, none[..., 0].float(), acc, **kw)

    zeros = [0] * B
    late = lambda t, x: t[:-1] + [x]
    for offs, lengths, want in ((zeros, [33] * B, 0), (late(zeros, 1), [33] * B, fos.STATUS_BAD_OFFS),
                                (late(zeros, -1), [33] * B, fos.STATUS_BAD_OFFS),
                                (zeros, late([33] * B, 49), fos.STATUS_BAD_CACHE),
                                (late(zeros, 3), late([33] * B, -1), fos.STATUS_BAD_OFFS | fos.STATUS_BAD_CACHE)):
        o, n = (torch.tensor(t, dtype=torch.int32).cuda() for t in (offs, lengths))
        for call in calls(o, n):
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            call(status=status)
            call()
            assert int(status.item()) == want
    assert not acc.any()
