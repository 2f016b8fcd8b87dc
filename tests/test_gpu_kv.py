"""The NVFP4 key/value cache against plain references: the append bit for bit
against the quantizer's oracle, attention and its weights against 64-bit
references, the eviction row by row. GPU only."""
import math

import numpy as np
import pytest
import torch

import kv_reference as ref
import nvfp4_adaptive_block_amd as fos
from operator_reference import DTYPES, assert_within, gen
from synthdata import raw_bits

pytestmark = pytest.mark.gpu
DIMS = [32, 64, 96, 128, 192, 256]
LONG = 10 ** 6  # an expected length, past any table's: with a table of WIDE pages 49 rows to a
WIDE = 2 ** 14  # sequence go in tiles of 128


def ends(new):
    return torch.tensor(np.cumsum(new).astype(np.int32)).cuda()


def same(a, b):
    return torch.equal(a.cpu().contiguous().view(torch.uint8), b.cpu().contiguous().view(torch.uint8))


def guarded(shape, dtype, pad=64):
    raw = torch.full((int(np.prod(shape)) + 2 * pad,), 77.0, device="cuda").to(dtype)
    return raw[pad:-pad].view(shape), raw


def assert_guard(raw, pad=64):
    edge = torch.cat((raw[:pad], raw[-pad:])).float()
    assert (edge == torch.tensor(77.0).to(raw.dtype).float().item()).all(), "wrote outside the output"


def assert_tiles(cache, q):
    """The rule by which the rows go in tiles of 128."""
    rows = len(q) * q.shape[1] // cache.H // cache.B
    assert rows > 48 and -(-rows // 16) * cache.B * cache.H * -(-cache.W * cache.P // 128) > 2048


def attend(cache, q, new, **kw):
    """(out, lse, status) of the packed queries, into guarded outputs."""
    if kw.get("max_len") == LONG and cache.W == WIDE:
        assert_tiles(cache, q)
    k, v, table, lens = cache.on_device()
    out, raw = guarded(q.shape, q.dtype)
    lse, raw_l = guarded(q.shape[:2], torch.float32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = fos.fos_kv_attention(q.cuda(), ends(new), k, v, table, lens, out=out, lse=lse, status=status, **kw)
    assert got[0] is out and got[1] is lse
    assert_guard(raw)
    assert_guard(raw_l)
    return out, lse, int(status.item())


def check_attention(cache, q, new, causal=True, scale=None, **kw):
    out, lse, status = attend(cache, q, new, causal=causal, scale=scale, **kw)
    want, bound, want_lse, lse_bound = ref.attention(cache, q, new, causal, scale)
    assert status == 0
    empty = want_lse == -math.inf
    assert torch.equal(lse.cpu() == -math.inf, empty)
    assert (out.cpu()[empty] == 0).all()
    if q.dtype == torch.float16:  # results past fp16's range become infinities
        over = want.abs() > 65000
        assert torch.isinf(out.cpu()[want.abs() > 66000]).all()
        assert_within(out.cpu()[~over], want[~over], bound[~over], "out")
    else:
        assert_within(out, want, bound, "out")
    assert_within(lse.cpu()[~empty], want_lse[~empty], lse_bound[~empty], "lse")
    return out, lse


# ------------------------------------------------------------------ append


def oracle_rows(orc, x, **knobs):
    """(codes, scales, sdec, values) of rows x by the oracle, S_dec of zeros 0."""
    rows = x.reshape(-1, x.shape[-1]).contiguous()
    name = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}[x.dtype]
    amax = orc.amax(raw_bits(rows), name, "row")
    kw = dict(recipe="4over6", err_metric="mse", err_prec="exact", bound=448)
    kw.update(knobs)
    o = orc.quantize(raw_bits(rows), name, amax, scale_gran="row", **kw)
    y = orc.qdq(raw_bits(rows), name, amax, scale_gran="row", **kw)
    sdec = np.where(amax == 0, np.float32(0), o["sdec"])
    return o["codes"], o["scales"], sdec, y


def rows_like(shape, dtype, seed):
    """Rows of different size, zeros, tiny and huge rows, NaN and infinities."""
    g = gen(seed)
    x = torch.randn(*shape, generator=g) * torch.exp(2 * torch.randn(*shape[:-1], 1, generator=g))
    x = x.to(DTYPES[dtype])
    flat = x.view(-1, shape[-1])
    n = flat.shape[0]
    if n >= 8:
        flat[1] = 0
        flat[2] *= 1e-30 if dtype != "fp16" else 1e-4
        flat[3, 5] = math.nan
        flat[4, 7] = math.inf
        flat[5] = math.nan
        flat[6] = torch.tensor([6.0, 4.0, 2.5, -5.0] * (shape[-1] // 4)).to(x.dtype)
        flat[7, 1:] = -0.0
    return x


def check_append(orc, lens, new, H, D, P, dtype, seed=0, tail=0, **knobs):
    cache = ref.Cache(lens, H, D, P, seed)
    T = sum(new) + tail
    wide = rows_like((T, 3 * H, D), dtype, seed + 3).cuda()
    k, v = wide[:, H:2 * H], wide[:, 2 * H:]
    sides = [tuple(t.clone() for t in side) for side in cache.sides]
    kc, vc, table, lens_d = cache.on_device()
    ko, raw_k = guarded((T, H, D), k.dtype)
    vo, raw_v = guarded((T, H, D), k.dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fos.fos_kv_append(k, v, ends(new), kc, vc, table, lens_d, k_out=ko, v_out=vo, status=status, **knobs)
    assert int(status.item()) == 0
    for x, got, out, side in ((k, kc, ko, sides[0]), (v, vc, vo, sides[1])):
        codes, scales, sdec, y = oracle_rows(orc, x.cpu(), **knobs)
        at = 0
        for b, n in enumerate(new):
            for i in range(n):
                pos = lens[b] - n + i
                page, slot = int(cache.table[b, pos // P]), pos % P
                r = (at + i) * H
                side[0][page, :, slot] = torch.from_numpy(codes[r:r + H])
                side[1][page, :, slot] = torch.from_numpy(scales[r:r + H])
                side[2][page, :, slot] = torch.from_numpy(sdec[r:r + H])
            at += n
        for a, w in zip(got, side):  # what was not written is as it was
            assert same(a, w)
        want = np.array(y).reshape(T, H, D)
        want[at:] = 0
        assert np.array_equal(raw_bits(out.cpu().contiguous()), want)
    assert_guard(raw_k)
    assert_guard(raw_v)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D", DIMS)
def test_append(orc, D, dtype):
    check_append(orc, [70, 16, 1, 33, 0, 128], [7, 16, 1, 3, 0, 100], 3, D, 16, dtype, seed=D, tail=2)


@pytest.mark.parametrize("knobs", [dict(recipe="nvfp4"), dict(err_metric="mae"), dict(err_prec="fp16", bound=256),
                                   dict(err_metric="mae", err_prec="fp16", err_order="seq"), dict(err_order="seq")])
def test_append_knobs(orc, knobs):
    check_append(orc, [90, 41], [60, 41], 2, 128, 48, "bf16", seed=5, **knobs)


@pytest.mark.parametrize("lens,new,H,P", [([1], [1], 1, 16), ([64, 65, 63], [1, 1, 1], 8, 64), ([300], [300], 5, 64),
                                          ([5] * 130, [0, 1] * 65, 1, 16)])
def test_append_batches(orc, lens, new, H, P):
    check_append(orc, lens, new, H, 64, P, "bf16", seed=len(lens))


def test_append_is_the_quantizer():
    """The same rows through fos_amax, fos_quantize and fos_qdq."""
    x = torch.randn(40, 4, 128, generator=gen(1)).bfloat16().cuda()
    kc, vc = (fos.fos_kv_cache(1, 4, 48, 128) for _ in range(2))
    table, lens = torch.zeros(1, 1, dtype=torch.int32).cuda(), torch.tensor([40], dtype=torch.int32).cuda()
    ko, vo = fos.fos_kv_append(x, -x, lens, kc, vc, table, lens, values=True)
    for rows, cache, out in ((x, kc, ko), (-x, vc, vo)):
        flat = rows.flatten(0, 1).contiguous()
        amax = fos.fos_amax(flat, "row")
        codes, scales, sdec = fos.fos_quantize(flat, amax, scale_gran="row")
        held = [t[0, :, :40].transpose(0, 1).flatten(0, 1) for t in cache]
        assert same(held[0], codes) and same(held[1], scales) and same(held[2], sdec)
        assert same(out.flatten(0, 1), fos.fos_qdq(flat, amax, scale_gran="row"))
    y = x.clone()  # the outputs may be the inputs
    fos.fos_kv_append(y, -x, lens, kc, vc, table, lens, k_out=y)
    assert same(y, ko)


def test_append_bad_places(orc):
    """Pages that are none and lengths below the new rows: reported, nothing else written."""
    H, D, P = 2, 64, 16
    kc, vc = (fos.fos_kv_cache(3, H, P, D) for _ in range(2))
    table = torch.tensor([[0, -1], [1, 3], [2, 2]], dtype=torch.int32).cuda()
    lens = torch.tensor([20, 18, 2], dtype=torch.int32).cuda()
    offs = torch.tensor([6, 8, 13], dtype=torch.int32).cuda()  # places 14-19, 16-17, -3-1
    x = rows_like((13, H, D), "bf16", 4).cuda()
    for write_status in (True, False):
        status = torch.zeros(1, dtype=torch.int32).cuda() if write_status else None
        fos.fos_kv_append(x, x, offs, kc, vc, table, lens, status=status)
        if write_status:
            assert int(status.item()) == fos.STATUS_BAD_CACHE
    codes, scales, sdec, _ = oracle_rows(orc, x.cpu())
    want = torch.zeros(3, H, P, D // 2, dtype=torch.uint8)
    for token, page, slot in ((0, 0, 14), (1, 0, 15), (11, 2, 0), (12, 2, 1)):
        want[page, :, slot] = torch.from_numpy(codes[token * H:token * H + H])
    assert same(kc[0], want) and same(vc[0], want)


# --------------------------------------------------------------- attention

LENGTHS = [1, 0, 15, 16, 17, 31, 32, 33, 63, 100, 129]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", DIMS)
def test_attention_one_token(D, dtype):
    cache = ref.Cache(LENGTHS, 2, D, 16, seed=D)
    new = [1] * len(LENGTHS)
    check_attention(cache, ref.queries(len(new), 6, D, dtype, D + 1), new)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 8, 16, 17, 40])
@pytest.mark.parametrize("P,dtype", [(16, "bf16"), (48, "fp16"), (256, "bf16")])
def test_attention_groups(G, P, dtype):
    lens, new = [37, 5, 260, 64], [1, 2, 3, 0]
    cache = ref.Cache(lens, 2, 64, P, seed=G)
    check_attention(cache, ref.queries(sum(new), 2 * G, 64, dtype, G + 1, 3.0), new)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("max_len", [0, LONG])
def test_attention_many_tokens(D, dtype, causal, max_len):
    """Prompts, chunks behind a prefix, sequences without new tokens, a padded tail,
    and more new tokens than the cache has: their first see no key."""
    lens, new = [150, 300, 40, 0, 33], [150, 70, 0, 3, 47]
    cache = ref.Cache(lens, 2, D, 32, seed=D + 7, W=WIDE if max_len else None)
    check_attention(cache, ref.queries(sum(new) + 5, 4, D, dtype, D, 2.0), new, causal, max_len=max_len)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attention_whole_tiles(D, dtype, causal):
    """Heads enough for tiles whose keys are not in parts."""
    cache = ref.Cache([150, 33, 5], 30, D, 16, seed=D)
    new = [80, 30, 5]
    assert_tiles(cache, ref.queries(118, 240, 1, dtype, 0))
    assert fos.fos_kv_attention_workspace(118, 240, 3, cache.W, 30, 16, D) == 0
    check_attention(cache, ref.queries(118, 240, D, dtype, D), new, causal)


@pytest.mark.parametrize("H,G,n,L", [(1, 1, 1, 5000), (2, 4, 1, 3001), (1, 8, 5, 2500), (3, 2, 130, 1111), (1, 4, 600, 600),
                                     (8, 4, 33, 700), (1, 1, 257, 900)])
@pytest.mark.parametrize("max_len", [0, 100, LONG])
def test_attention_splits(H, G, n, L, max_len):
    """Whatever the caller expects the length to be."""
    cache = ref.Cache([L, L // 3 + n], H, 128, 64, seed=L, W=WIDE if max_len == LONG and n * G > 48 else None)
    check_attention(cache, ref.queries(2 * n, H * G, 128, "bf16", n), [n, n], max_len=max_len)


def test_attention_wide_table_of_a_short_cache():
    """A table for far longer sequences than there are."""
    cache = ref.Cache([70, 3], 2, 128, 16, seed=3, W=3000)
    check_attention(cache, ref.queries(2, 8, 128, "bf16", 4), [1, 1])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,max_len", [(1, 0), (40, 0), (40, LONG)])
def test_attention_extreme_rows(n, max_len, dtype):
    """Value rows of very different size, among them one that is huge where its weight
    is tiny and rows of zeros with the largest weight; queries of any size and scale."""
    cache = ref.Cache([200], 2, 128, 64, seed=8, W=WIDE if max_len else None)
    sd = cache.sides[1][2]
    where = [(int(cache.table[0, p // 64]), p % 64) for p in (3, 77, 150)]
    for i, (page, slot) in enumerate(where):
        sd[page, :, slot] = [2.0 ** 18, 2.0 ** -40, 0.0][i]
    q = ref.queries(n, 4, 128, dtype, 9)
    # the row of zeros gets nearly all of the first head's weight
    kv, kd = cache.rows(0, 0)
    q[:, 0] = (8 * kv[0, 150] / kv[0, 150].norm()).to(q.dtype)
    q[:, 1] *= 1e-3 if dtype == "fp16" else 1e-25
    q[:, 2] *= 30
    check_attention(cache, q, [n], max_len=max_len)
    check_attention(cache, q, [n], scale=-0.03, max_len=max_len)
    check_attention(cache, q, [n], scale=0.0, max_len=max_len)
    if dtype == "bf16":
        q[:, 3] *= 1e20
        check_attention(cache, q, [n], scale=1e-21, max_len=max_len)


@pytest.mark.parametrize("apart", [2.0 ** -7, 2.0 ** -12, 0.0])
@pytest.mark.parametrize("size", [1e-18, 1.0, 1e6])
def test_attention_tile_of_rows_of_two_sizes(size, apart):
    """Rows near enough for one power of two and too far for it, and rows of zeros."""
    cache = ref.Cache([200], 2, 64, 16, seed=26, W=WIDE)
    q = ref.queries(70, 4, 64, "bf16", 27)
    q[::3] *= apart
    check_attention(cache, q * size, [70], scale=0.125 / size, max_len=LONG)


@pytest.mark.parametrize("size_k,size_v", [(1e-20, 1e-25), (1e3, 1e8), (1e15, 1e25)])
def test_attention_sizes_of_the_cache(size_k, size_v):
    cache = ref.Cache([100, 40], 2, 64, 16, seed=10, sizes=(size_k, size_v))
    check_attention(cache, ref.queries(7, 4, 64, "bf16", 11), [4, 3], scale=0.02 / size_k)
    cache = ref.Cache([100, 40], 2, 64, 16, seed=10, sizes=(size_k, size_v), W=WIDE)
    check_attention(cache, ref.queries(90, 4, 64, "bf16", 11), [60, 30], scale=0.02 / size_k, max_len=LONG)


@pytest.mark.parametrize("n,max_len", [(1, 0), (50, 0), (50, LONG)])
def test_attention_not_a_number(n, max_len):
    """A query with a NaN or an infinity is NaN; others are as without it."""
    cache = ref.Cache([90], 2, 128, 16, seed=12, W=WIDE if max_len else None)
    q = ref.queries(n, 4, 128, "bf16", 13)
    out, lse, _ = attend(cache, q, [n], max_len=max_len)
    bad = q.clone()
    bad[0, 1, 77] = math.nan
    bad[n - 1, 2, 3] = math.inf
    got, got_lse, _ = attend(cache, bad, [n], max_len=max_len)
    hit = torch.zeros(n, 4, dtype=torch.bool)
    hit[0, 1] = hit[n - 1, 2] = True
    assert torch.isnan(got.cpu()[hit]).all() and torch.isnan(got_lse.cpu()[hit]).all()
    assert same(got[~hit.cuda()], out[~hit.cuda()]) and same(got_lse[~hit.cuda()], lse[~hit.cuda()])


@pytest.mark.parametrize("n,max_len", [(1, 0), (3, 0), (60, 0), (60, LONG)])
def test_attention_strides_and_repeats(n, max_len):
    """Queries inside wider rows; the same bits again, on any workspace and another stream."""
    cache = ref.Cache([400, 77], 2, 128, 64, seed=14, W=WIDE if max_len else None)
    T = 2 * n
    wide = ref.queries(T, 12, 128, "bf16", 15).cuda()
    q = wide[:, 2:10]
    k, v, table, lens = cache.on_device()
    args = (ends([n, n]), k, v, table, lens)
    out, lse = fos.fos_kv_attention(q, *args, max_len=max_len)
    again, lse2 = fos.fos_kv_attention(q.contiguous(), *args, max_len=max_len)
    assert same(out, again) and same(lse, lse2)
    need = fos.fos_kv_attention_workspace(T, 8, 2, cache.W, 2, 64, 128, max_len)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        third, _ = fos.fos_kv_attention(q, *args, workspace=ws, max_len=max_len)
    s.synchronize()
    assert same(out, third) and (ws[need:] == 255).all()


@pytest.mark.parametrize("n,max_len", [(2, 0), (60, 0), (60, LONG)])
def test_attention_bad_cache(n, max_len):
    """Pages that are none hold no keys; lengths past the table end with it."""
    cache = ref.Cache([64, 50], 2, 64, 16, seed=16, W=WIDE if max_len else None)
    q = ref.queries(2 * n, 4, 64, "bf16", 17)
    keep = cache.table.clone()
    cache.table[0, 1] = cache.pages
    cache.table[0, 3] = -1
    out, lse, _ = attend(cache, q, [n, n], causal=False, max_len=max_len)
    # the same with the two pages left out
    cache.table = keep.clone()
    cache.table[0, 1] = keep[0, 2]
    cache.lens[0] = 32
    want, bound, want_lse, lb = ref.attention(cache, q, [n, n], causal=False)
    assert_within(out, want, bound, "out")
    assert_within(lse, want_lse, lb, "lse")
    # no page at all
    cache.table[0] = -1
    cache.lens[0] = 64
    out, lse, _ = attend(cache, q, [n, n], max_len=max_len)
    assert (out[:n] == 0).all() and (lse[:n] == -math.inf).all()
    if max_len:
        return
    # lengths outside [0, W P]
    cache.table = keep
    cache.lens = [10 ** 6, -5]
    out, lse, status = attend(cache, q, [n, n], max_len=max_len)
    assert status == fos.STATUS_BAD_CACHE
    cache.lens = [64, 0]
    want, bound, want_lse, lb = ref.attention(cache, q, [n, n])
    assert_within(out, want, bound, "out")
    assert (lse[n:] == -math.inf).all()


@pytest.mark.parametrize("n,max_len", [(4, 0), (100, 0), (100, LONG)])
def test_attention_bad_offsets(n, max_len):
    cache = ref.Cache([64, 50], 2, 64, 16, seed=16, W=WIDE if max_len else None)
    k, v, table, lens = cache.on_device()
    q = ref.queries(n, 4, 64, "bf16", 17).cuda()
    for offs in ([n - 1, n - 2], [2, n + 5], [-1, n]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, raw = guarded(q.shape, q.dtype)
        fos.fos_kv_attention(q, torch.tensor(offs, dtype=torch.int32).cuda(), k, v, table, lens, out=out, status=status,
                             max_len=max_len)
        assert int(status.item()) == fos.STATUS_BAD_OFFS
        assert_guard(raw)


# ----------------------------------------------------------------- weights


def check_weights(cache, q, new, causal=True, scale=None, **kw):
    k, v, table, lens = cache.on_device()
    offs = ends(new)
    _, lse = fos.fos_kv_attention(q.cuda(), offs, k, v, table, lens, causal=causal, scale=scale)
    start = torch.rand(cache.B, cache.H, cache.W * cache.P, generator=gen(1)).cuda()
    acc, raw = guarded(start.shape, torch.float32)
    acc.copy_(start)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = fos.fos_kv_weights(q.cuda(), offs, k, table, lens, lse, acc, causal=causal, scale=scale, status=status, **kw)
    assert got is acc and int(status.item()) == 0
    assert_guard(raw)
    want, bound = ref.weights(cache, q, new, lse.cpu(), causal, scale)
    want = want + start.double().cpu()
    # rows come 32 or 256 at a time: each such part is added to what is there in binary32,
    # which rounds a total of at most the result by half a step, 2^-24 of it at most
    parts = torch.tensor([max(1, -(-n * q.shape[1] // cache.H // 32)) for n in new], dtype=torch.float64)
    assert_within(acc, want, bound + ref.E24 * parts[:, None, None] * want.abs(), "acc")
    for b, n in enumerate(cache.lens):
        assert same(acc[b, :, n:], start[b, :, n:])
    # every row's weights sum to one
    total = (acc - start).double().sum().item()
    rows = int((lse[:sum(new)] > -math.inf).sum())
    assert abs(total - rows) <= 1e-4 * max(1, rows)
    return acc


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", DIMS)
def test_weights_one_token(D, dtype):
    cache = ref.Cache(LENGTHS, 2, D, 16, seed=D)
    check_weights(cache, ref.queries(len(LENGTHS), 6, D, dtype, D + 1), [1] * len(LENGTHS))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("G,D,dtype", [(1, 64, "bf16"), (3, 128, "fp16"), (8, 96, "bf16"), (17, 32, "fp16")])
def test_weights_many_tokens(G, D, dtype, causal):
    lens, new = [150, 300, 40, 0, 33], [150, 70, 0, 3, 47]
    cache = ref.Cache(lens, 2, D, 48, seed=D + 7)
    check_weights(cache, ref.queries(sum(new) + 5, 2 * G, D, dtype, D, 2.0), new, causal)


@pytest.mark.parametrize("max_len", [0, 50, 10 ** 6])
def test_weights_long(max_len):
    cache = ref.Cache([3000, 700], 2, 128, 64, seed=20)
    check_weights(cache, ref.queries(40, 8, 128, "bf16", 21), [20, 20], max_len=max_len)


def test_weights_of_the_last_tokens():
    """The last tokens' part of q and lse: the rows that see the most."""
    cache = ref.Cache([200], 2, 64, 16, seed=22)
    q = ref.queries(50, 4, 64, "bf16", 23)
    k, v, table, lens = cache.on_device()
    _, lse = fos.fos_kv_attention(q.cuda(), ends([50]), k, v, table, lens)
    acc = torch.zeros(1, 2, cache.W * 16, device="cuda")
    fos.fos_kv_weights(q[-8:].cuda(), ends([8]), k, table, lens, lse[-8:], acc)
    want, bound = ref.weights(cache, q[-8:], [8], lse[-8:].cpu())
    assert_within(acc, want, bound, "acc")


# ------------------------------------------------------------------- evict


def check_evict(lens, H, D, P, budget, sinks, recent, seed=0, acc=None, W=None):
    cache = ref.Cache(lens, H, D, P, seed, W=W)
    shape = (cache.B, H, cache.W * P)
    acc = torch.exp(2 * torch.randn(*shape, generator=gen(seed + 1))) if acc is None else acc(shape)
    kc, vc, table, lens_d = cache.on_device()
    acc_d, raw = guarded(shape, torch.float32)
    acc_d.copy_(acc)
    need = fos.fos_kv_evict_workspace(cache.B, H, budget, recent)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    new_lens = fos.fos_kv_evict(acc_d, kc, vc, table, lens_d, budget, sinks=sinks, recent=recent, workspace=ws,
                                status=status)
    assert int(status.item()) == 0 and (ws[need:] == 255).all()
    assert new_lens.tolist() == [min(n, budget) for n in lens]
    assert_guard(raw)
    came, want_acc = ref.evict(cache, acc, budget, sinks, recent)
    assert same(acc_d, want_acc)
    for side, got in zip(cache.sides, (kc, vc)):
        got, want = [t.cpu() for t in got], [t.clone() for t in side]
        for (b, h), src in came.items():
            for i, j in enumerate(src):
                to, of = int(cache.table[b, i // P]), int(cache.table[b, j // P])
                for w, t in zip(want, side):
                    w[to, h, i % P] = t[of, h, j % P]
        for b, n in enumerate(lens):  # rows that are still in use; what is behind them is anybody's
            for i in range(min(n, budget)):
                page = int(cache.table[b, i // P])
                for w, g in zip(want, got):
                    assert same(g[page, :, i % P], w[page, :, i % P]), (b, i)


@pytest.mark.parametrize("D", DIMS)
def test_evict(D):
    check_evict([130, 70, 50, 90, 0, 71], 2, D, 16, 70, 4, 20, seed=D)


@pytest.mark.parametrize("budget,sinks,recent", [(64, 0, 0), (64, 0, 64), (64, 64, 0), (64, 4, 60), (64, 10, 33), (1, 0, 0),
                                                 (1, 0, 1), (1, 1, 0), (0, 0, 0), (150, 5, 140), (199, 4, 100)])
def test_evict_shares(budget, sinks, recent):
    check_evict([200, 65], 2, 64, 48, budget, sinks, recent, seed=budget)


@pytest.mark.parametrize("n,budget,recent", [(3000, 500, 100), (2500, 2400, 1000), (1025, 1024, 128), (5000, 4000, 70)])
def test_evict_long(n, budget, recent):
    check_evict([n], 2, 64, 64, budget, 4, recent, seed=n)


@pytest.mark.parametrize("D", DIMS)
def test_evict_many_moves(D):
    """Enough of them for launches of their own; sequences of any length beside them."""
    check_evict([2700, 1250, 1500, 40, 0, 1401], 2, D, 64, 1400, 4, 200, seed=D)


@pytest.mark.parametrize("W", [41, 300])
def test_evict_many_heads(W):
    """128 of them, with many moves, under a table of their length and a wider one."""
    check_evict([2600, 30], 64, 32, 64, 1200, 4, 40, seed=W, W=W)


ODD = [math.nan, math.inf, -math.inf, 0.0, -0.0, 1.0, 1.0000001, -1.0, 1e-40, -1e-40, 3e38]


@pytest.mark.parametrize("kind", ["zeros", "equal", "few", "odd", "sorted", "reversed"])
def test_evict_order_of_weights(kind):
    def make(shape):
        n = shape[-1]
        if kind == "zeros":
            return torch.zeros(shape)
        if kind == "equal":
            return torch.full(shape, 0.7)
        if kind == "few":
            return torch.randint(0, 3, shape, generator=gen(3)).float()
        if kind == "odd":
            return torch.tensor(ODD)[torch.randint(0, len(ODD), shape, generator=gen(4))]
        line = torch.arange(n).float() * 1e-3
        return (line if kind == "sorted" else line.flip(0)).expand(shape).contiguous()

    check_evict([300, 140], 2, 32, 16, 100, 3, 30, seed=1, acc=make)


def test_evict_bad_page():
    """A sequence with a page that is none stays as it is."""
    cache = ref.Cache([100, 100], 2, 64, 16, seed=2)
    cache.table[0, 2] = cache.pages
    acc = torch.rand(2, 2, cache.W * 16, generator=gen(3))
    kc, vc, table, lens = cache.on_device()
    acc_d = acc.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = fos.fos_kv_evict(acc_d, kc, vc, table, lens, 40, recent=8, status=status)
    assert new.tolist() == [100, 40] and int(status.item()) == fos.STATUS_BAD_CACHE
    assert same(acc_d[0], acc[0])
    for b, page in enumerate(cache.table[0]):
        if b != 2:
            assert same(kc[0][int(page)], cache.sides[0][0][int(page)])


# ---------------------------------------------------------------- together


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_decode_with_eviction(dtype):
    """Prompts, then decode steps with their weights, and an eviction when a sequence
    is a page over its budget, as a server would run them; each step's attention
    against a 64-bit one on the values that the cache holds."""
    H, G, D, P, B, W, budget = 2, 3, 64, 16, 3, 8, 96
    dt = DTYPES[dtype]
    kc, vc = (fos.fos_kv_cache(B * W, H, P, D) for _ in range(2))
    table = torch.randperm(B * W, generator=gen(0)).int().view(B, W).cuda()
    acc = torch.zeros(B, H, W * P, device="cuda")
    held = [[[], []] for _ in range(B)]  # float64 rows [H, D] of K and V, in the cache's order per head
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    g = gen(5)
    evicted = 0
    for step in range(30):
        new = [70, 30, 91] if step == 0 else [1, 2 if step % 5 == 0 else 1, 0 if step == 7 else 1]
        T = sum(new)
        qkv = torch.randn(T, (G + 2) * H, D, generator=g).to(dt).cuda()
        q, k, v = qkv[:, :G * H], qkv[:, G * H:G * H + H], qkv[:, G * H + H:]
        offs = ends(new)
        lens += torch.tensor(new, dtype=torch.int32).cuda()
        fos.fos_kv_append(k, v, offs, kc, vc, table, lens)
        out, lse = fos.fos_kv_attention(q, offs, kc, vc, table, lens)
        fos.fos_kv_weights(q, offs, kc, table, lens, lse, acc)
        snapshot = ref.Cache([int(n) for n in lens], H, D, P, W=W)
        snapshot.table, snapshot.pages = table.cpu(), B * W
        snapshot.sides = [tuple(t.cpu() for t in side) for side in (kc, vc)]
        want, bound, want_lse, lb = ref.attention(snapshot, q.cpu(), new)
        assert_within(out, want, bound, f"step {step}")
        assert_within(lse, want_lse, lb, f"step {step}")
        if int(lens.max()) >= budget + P:
            before = acc.clone()
            lens = fos.fos_kv_evict(acc, kc, vc, table, lens, budget, sinks=2, recent=40)
            assert int(lens.max()) <= budget and (acc.sum() < before.sum())
            evicted += 1
    assert evicted >= 1


def test_captured_decode_step():
    """Append, attention, weights and eviction in one graph: lengths and offsets are read
    on the device, so replays follow them."""
    H, G, D, P, B, W = 2, 4, 128, 16, 2, 16
    kc, vc = (fos.fos_kv_cache(B * W, H, P, D) for _ in range(2))
    table = torch.arange(B * W, dtype=torch.int32).view(B, W).cuda()
    acc = torch.zeros(B, H, W * P, device="cuda")
    offs = ends([1, 1])
    lens = torch.tensor([100, 47], dtype=torch.int32).cuda()
    fill = torch.randn(147, H, D, generator=gen(2)).bfloat16().cuda()
    fos.fos_kv_append(fill, fill.flip(0).contiguous(), ends([100, 47]), kc, vc, table, lens)
    qkv = torch.zeros(B, (G + 2) * H, D, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(B, G * H, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(B, G * H, device="cuda")
    ws = torch.empty(fos.fos_kv_attention_workspace(B, G * H, B, W, H, P, D), dtype=torch.uint8, device="cuda")
    ws_e = torch.empty(fos.fos_kv_evict_workspace(B, H, 102, 30), dtype=torch.uint8, device="cuda")
    cut = torch.zeros(B, dtype=torch.int32, device="cuda")

    def step():
        q, k, v = qkv[:, :G * H], qkv[:, G * H:G * H + H], qkv[:, G * H + H:]
        lens.add_(1)
        fos.fos_kv_append(k, v, offs, kc, vc, table, lens)
        fos.fos_kv_attention(q, offs, kc, vc, table, lens, out=out, lse=lse, workspace=ws)
        fos.fos_kv_weights(q, offs, kc, table, lens, lse, acc)
        fos.fos_kv_evict(acc, kc, vc, table, lens, 102, sinks=2, recent=30, new_lens=cut, workspace=ws_e)
        lens.copy_(cut)

    state = [*kc, *vc, acc, lens]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    keep = [t.clone() for t in state]
    with torch.cuda.stream(s):
        step()  # outside the graph first
    s.synchronize()
    for t, was in zip(state, keep):
        t.copy_(was)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, was in zip(state, keep):
        t.copy_(was)
    shadow = [t.clone() for t in state]
    for i in range(6):
        qkv.copy_(torch.randn(*qkv.shape, generator=gen(40 + i)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in state] + [out.clone(), lse.clone()]
        for t, was in zip(state, shadow):
            t.copy_(was)
        step()  # the same step eagerly
        want = [t.clone() for t in state] + [out.clone(), lse.clone()]
        for a, b in zip(got, want):
            assert same(a, b), i
        shadow = [t.clone() for t in state]
    assert lens.tolist() == [102, 53]


def test_cache_past_32_bits():
    """Pages behind more than 2^32 bytes of codes: the same bits as in a small pool."""
    H, P, D, pages = 16, 64, 128, 70000
    cache = ref.Cache([300, 129], H, D, P, seed=21, W=256)
    small = cache.on_device()
    up = pages - cache.pages
    far = []
    for side in small[:2]:
        big = (torch.empty(pages, H, P, D // 2, dtype=torch.uint8, device="cuda"),
               torch.empty(pages, H, P, D // 16, dtype=torch.uint8, device="cuda"),
               torch.empty(pages, H, P, device="cuda"))
        for t, b in zip(side, big):
            b[up:] = t
        far.append(big)
    assert far[0][0].numel() > 2 ** 32
    pools = [(*small, 0), (*far, small[2] + up, small[3], up)]  # stale entries stay out of range
    k = torch.randn(5, H, D, generator=gen(22)).bfloat16().cuda()
    results = []
    for kc, vc, table, lens, at in pools:
        fos.fos_kv_append(k, -k, ends([3, 2]), kc, vc, table, lens)
        got = []
        for n, max_len in ((1, 0), (60, LONG)):
            q = ref.queries(2 * n, 2 * H, D, "bf16", 23).cuda()
            if n > 1:
                assert_tiles(cache, q)
            out, lse = fos.fos_kv_attention(q, ends([n, n]), kc, vc, table, lens, max_len=max_len)
            acc = torch.zeros(2, H, cache.W * P, device="cuda")
            got += [out, lse, fos.fos_kv_weights(q, ends([n, n]), kc, table, lens, lse, acc)]
        got.append(fos.fos_kv_evict(acc, kc, vc, table, lens, 100, sinks=2, recent=30).clone())
        got += [t[at:].clone() for side in (kc, vc) for t in side]
        results.append(got)
    for a, b in zip(*results):
        assert same(a, b)


@pytest.mark.parametrize("n", [1, 60])
def test_calls_on_two_streams(n):
    """The same calls on two streams at once, each with workspaces of its own."""
    cache = ref.Cache([700, 333], 2, 128, 64, seed=24, W=128)
    kc, vc, table, lens = cache.on_device()
    q = ref.queries(2 * n, 8, 128, "bf16", 25).cuda()
    offs = ends([n, n])
    if n > 1:
        assert_tiles(cache, q)

    def calls():
        k, v = (tuple(t.clone() for t in side) for side in (kc, vc))
        acc = torch.zeros(2, 2, cache.W * 64, device="cuda")
        out, lse = fos.fos_kv_attention(q, offs, k, v, table, lens, max_len=LONG)
        fos.fos_kv_weights(q, offs, k, table, lens, lse, acc)
        cut = fos.fos_kv_evict(acc, k, v, table, lens, 300, sinks=4, recent=64)
        return [out, lse, acc, cut, *fos.fos_kv_attention(q, offs, k, v, table, cut)]

    want = calls()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(calls())
    torch.cuda.synchronize()
    for g in got:
        assert all(same(a, b) for a, b in zip(g, want))
