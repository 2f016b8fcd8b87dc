"""Refusals of the key/value cache's calls, on the host: every check runs before a
device is touched (made-up addresses stand in for buffers)."""
import ctypes

import pytest
import torch

import nvfp4_adaptive_block_amd as fos

INVALID, DTYPE, SHAPE, ALIGN, CONFIG, DEVICE = 1, 2, 3, 4, 5, 6
Q, K, S, D_, T_, L, O, Y, A, W_ = (0x10000 * i for i in range(1, 11))


class Rows(ctypes.Structure):  # fos_kv_rows
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("sdec", ctypes.c_void_p)]


class Cache(ctypes.Structure):  # fos_kv_cache
    _fields_ = [("k", Rows), ("v", Rows), ("table", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("pages", ctypes.c_int64), *((name, ctypes.c_int32) for name in "BWHPD")]


def rows(codes=K, scales=S, sdec=D_):
    return Rows(codes, scales, sdec)


def cache(k=None, v=None, table=T_, lens=L, pages=9, B=2, W=4, H=3, P=64, D=128):
    return Cache(k or rows(), v or rows(), table, lens, pages, B, W, H, P, D)


def test_the_packed_cache_is_the_structure():
    c = cache(v=rows(K + 16, S + 32, D_ + 48))
    packed = fos._KV_CACHE.pack(K, S, D_, K + 16, S + 32, D_ + 48, T_, L, 9, 2, 4, 3, 64, 128)
    assert packed == bytes(c) and len(packed) == ctypes.sizeof(Cache)


def checked(rc):
    assert rc == 0 or fos.load_library().fos_last_error()
    return rc


def append(c=None, k=Q, v=Q, dtype=0, T=5, ks=3 * 128, vs=3 * 128, offs=O, cfg=None, ko=None, vo=None, st=None):
    cfg = cfg or fos.config(scale_gran="row")
    c = c or cache()
    return checked(fos.load_library().fos_kv_append(k, v, dtype, T, ks, vs, offs, ctypes.byref(c), ctypes.byref(cfg), ko,
                                                    vo, st, None))


def attention(c=None, q=Q, dtype=0, T=5, Hq=6, qs=6 * 128, offs=O, scale=0.1, max_len=100, out=Y, lse=A, work=None,
              room=None, st=None):
    lib, c = fos.load_library(), c or cache()
    need = lib.fos_kv_attention_workspace(T, Hq, c.B, c.W, c.H, c.P, c.D, max_len)
    work = W_ if work is None else work
    return checked(lib.fos_kv_attention(q, dtype, T, Hq, qs, offs, ctypes.byref(c), scale, 1, max_len, out, lse, work,
                                        max(0, need) if room is None else room, st, None))


def weights(c=None, q=Q, dtype=0, T=5, Hq=6, qs=6 * 128, offs=O, scale=0.1, max_len=100, lse=A, acc=Y, st=None):
    c = c or cache()
    return checked(fos.load_library().fos_kv_weights(q, dtype, T, Hq, qs, offs, ctypes.byref(c), scale, 1, max_len, lse,
                                                     acc, st, None))


def evict(c=None, acc=A, budget=64, sinks=4, recent=16, new=Y, work=W_, room=None, st=None):
    lib, c = fos.load_library(), c or cache()
    need = lib.fos_kv_evict_workspace(c.B, c.H, budget, recent)
    return checked(lib.fos_kv_evict(ctypes.byref(c), acc, budget, sinks, recent, new, work,
                                    max(0, need) if room is None else room, st, None))


CALLS = [append, attention, weights, evict]


@pytest.mark.parametrize("call", CALLS)
def test_what_is_right_passes_every_check(call):
    assert call() in (0, DEVICE)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(B=0)), (INVALID, dict(W=0)), (INVALID, dict(H=0)), (INVALID, dict(P=0)), (INVALID, dict(P=-16)),
    (SHAPE, dict(P=24)), (SHAPE, dict(P=8)), (SHAPE, dict(D=0)), (SHAPE, dict(D=16)), (SHAPE, dict(D=80)),
    (SHAPE, dict(D=160)), (SHAPE, dict(D=512)), (SHAPE, dict(D=-64)), (SHAPE, dict(W=2 ** 30, P=16)),
    (SHAPE, dict(B=2 ** 20 + 1)), (SHAPE, dict(B=2 ** 20, H=8)), (SHAPE, dict(B=2 ** 20, H=4)), (INVALID, dict(pages=0)), (INVALID, dict(pages=-1)),
    (SHAPE, dict(pages=2 ** 40)), (INVALID, dict(table=0)), (INVALID, dict(lens=0)), (ALIGN, dict(table=T_ + 2)),
    (ALIGN, dict(lens=L + 1)), (INVALID, dict(k=rows(codes=0))), (INVALID, dict(k=rows(scales=0))),
    (INVALID, dict(k=rows(sdec=0))), (ALIGN, dict(k=rows(codes=K + 8))), (ALIGN, dict(k=rows(scales=S + 2))),
    (ALIGN, dict(k=rows(sdec=D_ + 4))),
])
@pytest.mark.parametrize("call", CALLS)
def test_cache_refusals(call, want, kw):
    assert call(cache(**kw)) == want


@pytest.mark.parametrize("call", [append, attention, evict])
def test_values_are_needed_where_they_are_read(call):
    assert call(cache(v=rows(codes=0))) == INVALID
    assert call(cache(v=rows(sdec=D_ + 8))) == ALIGN
    assert weights(cache(v=Rows(0, 0, 0))) in (0, DEVICE)


@pytest.mark.parametrize("want,kw", [
    (DTYPE, dict(dtype=3)), (INVALID, dict(T=-1)), (SHAPE, dict(T=2 ** 27)), (INVALID, dict(k=None)), (INVALID, dict(v=None)),
    (ALIGN, dict(k=Q + 8)), (ALIGN, dict(v=Q + 2)), (ALIGN, dict(ko=Y + 8)), (ALIGN, dict(vo=Y + 4)), (INVALID, dict(offs=None)),
    (ALIGN, dict(offs=O + 2)), (ALIGN, dict(st=A + 1)), (SHAPE, dict(ks=2 * 128)), (SHAPE, dict(vs=-3 * 128)),
    (ALIGN, dict(ks=3 * 128 + 4)), (ALIGN, dict(vs=3 * 128 + 1)), (ALIGN, dict(dtype=2, ks=3 * 128 + 2)),
    (SHAPE, dict(ks=2 ** 40)), (CONFIG, dict(cfg=fos.config(block="16x16"))), (CONFIG, dict(cfg=fos.config(bound=300))),
])
def test_append_refusals(want, kw):
    assert append(**kw) == want


@pytest.mark.parametrize("want,kw", [
    (DTYPE, dict(dtype=2)), (DTYPE, dict(dtype=-1)), (INVALID, dict(T=-1)), (SHAPE, dict(Hq=7)), (SHAPE, dict(Hq=0)),
    (SHAPE, dict(Hq=-3)), (SHAPE, dict(T=2 ** 26)), (INVALID, dict(q=None)), (ALIGN, dict(q=Q + 8)), (INVALID, dict(offs=None)),
    (ALIGN, dict(offs=O + 1)), (INVALID, dict(scale=float("nan"))), (INVALID, dict(scale=float("inf"))),
    (INVALID, dict(max_len=-1)), (SHAPE, dict(qs=5 * 128)), (ALIGN, dict(qs=6 * 128 + 2)), (ALIGN, dict(st=A + 2)),
    (ALIGN, dict(lse=A + 2)),
])
@pytest.mark.parametrize("call", [attention, weights])
def test_query_refusals(call, want, kw):
    assert call(**kw) == want


def test_attention_refusals():
    assert attention(out=None) == INVALID
    assert attention(out=Y + 8) == ALIGN
    need = fos.fos_kv_attention_workspace(1, 6, 2, 64, 3, 64, 128)
    assert need > 0
    long = dict(c=cache(W=64), T=1, max_len=0)
    assert attention(**long) in (0, DEVICE)
    assert attention(room=need - 1, **long) == INVALID
    assert attention(work=0, **long) == INVALID
    assert attention(work=W_ + 8, **long) == ALIGN
    assert attention(lse=None) in (0, DEVICE)
    assert weights(lse=None) == INVALID
    assert weights(acc=None) == INVALID
    assert weights(acc=Y + 2) == ALIGN


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(budget=-1)), (INVALID, dict(sinks=-1)), (INVALID, dict(recent=-1)), (INVALID, dict(sinks=40, recent=25)),
    (INVALID, dict(recent=65, sinks=0)), (INVALID, dict(budget=2 ** 30 + 1)), (INVALID, dict(acc=None)), (INVALID, dict(new=None)),
    (INVALID, dict(new=L)), (INVALID, dict(new=L + 4)), (INVALID, dict(new=L - 4)), (ALIGN, dict(acc=A + 2)), (ALIGN, dict(new=Y + 2)), (ALIGN, dict(st=A + 3)), (INVALID, dict(room=10)),
    (INVALID, dict(work=None)), (ALIGN, dict(work=W_ + 8)),
])
def test_evict_refusals(want, kw):
    assert evict(**kw) == want


def test_calls_without_tokens_need_no_rows():
    """A tensor without elements has no address."""
    assert append(T=0, k=None, v=None) in (0, DEVICE)
    assert attention(T=0, q=None, out=None, lse=None) in (0, DEVICE)
    assert weights(T=0, q=None, lse=None) in (0, DEVICE)


def test_workspaces():
    with pytest.raises(ValueError):
        fos.fos_kv_attention_workspace(1, 5, 1, 4, 2, 64, 128)
    with pytest.raises(ValueError):
        fos.fos_kv_attention_workspace(1, 4, 1, 4, 2, 60, 128)
    with pytest.raises(ValueError):
        fos.fos_kv_attention_workspace(1, 4, 1, 4, 2, 64, 128, -1)
    with pytest.raises(ValueError):
        fos.fos_kv_evict_workspace(1, 2, 10, 11)
    assert fos.fos_kv_evict_workspace(2, 3, 100, 40) == 2 * 3 * 60 * 8 + 2 * 3 * 4
    assert fos.fos_kv_evict_workspace(2, 3, 40, 40) == 2 * 3 * 4
    # more keys, no smaller a workspace; none where there are rows enough
    sizes = [fos.fos_kv_attention_workspace(1, 8, 1, w, 2, 64, 128) for w in (1, 8, 64, 1024)]
    assert sizes == sorted(sizes) and sizes[-1] > 0
    assert fos.fos_kv_attention_workspace(8192, 32, 1, 128, 8, 64, 128) == 0


def test_python_checks():
    """On host tensors, whose device index is -1; a cache on the host is refused."""
    k, v = (fos.fos_kv_cache(3, 2, 16, 64, device="cpu") for _ in range(2))
    table, lens = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: fos.fos_kv_attention(q, lens, k, v, table, lens),
                 lambda: fos.fos_kv_append(q, q, lens, k, v, table, lens),
                 lambda: fos.fos_kv_weights(q, lens, k, table, lens, lens, lens),
                 lambda: fos.fos_kv_evict(lens, k, v, table, lens, 4)):
        with pytest.raises(ValueError, match="on a device"):
            call()
    assert fos._kv_at(k[0], "codes", -1, (3, 2, 16, 32), torch.uint8) == k[0].data_ptr()
    for bad in ((3, 2, 16, 31), torch.uint8), ((3, 2, 16, 32), torch.int8):
        with pytest.raises(ValueError):
            fos._kv_at(k[0], "codes", -1, *bad)
    with pytest.raises(ValueError):
        fos._kv_at(k[0], "codes", 0, (3, 2, 16, 32), torch.uint8)
    with pytest.raises(ValueError):
        fos._kv_at(k[0].transpose(1, 2), "codes", -1, (3, 16, 2, 32), torch.uint8)
    with pytest.raises(ValueError, match="bf16 or fp16"):
        fos._kv_queries(q.float(), -1, 64)
    wide = torch.zeros(5, 6, 64)
    assert fos._kv_tokens(wide[:, 2:4], "k", -1, 2, 64)[1] == 6 * 64
    assert fos._kv_tokens(wide[:1, 2:4], "k", -1, 2, 64)[1] == 2 * 64
    for bad in (wide[:, ::2], wide[..., :32], wide[:, :2].transpose(0, 2), wide[:, 0]):
        with pytest.raises(ValueError):
            fos._kv_tokens(bad, "k", -1, bad.shape[1], 64)
    with pytest.raises(ValueError):
        fos._kv_tokens(wide, "k", 0, 6, 64)
