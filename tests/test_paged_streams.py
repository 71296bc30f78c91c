"""Language streams over a paged cache, without a GPU: the oracle's own pins and
the refusals of the library and of the binding."""
import ctypes

import numpy as np
import pytest

from oracle import pages as OP
from tests._util import LIB, ensure_built


@pytest.fixture(scope="module")
def lib():
    try:
        ensure_built()
    except RuntimeError as e:  # pragma: no cover
        pytest.skip("cannot build librx.so here: %s" % e)
    return ctypes.CDLL(LIB)


# ------------------------------------------------------------------- oracle
@pytest.mark.parametrize("adjacent", [False, True])
def test_rotation_keeps_lengths_and_depends_on_distance(adjacent):
    g = np.random.default_rng(0)
    freq = 100.0 ** -(np.arange(8) / 8)
    a, b = g.standard_normal((1, 1, 24)), g.standard_normal((1, 1, 24))
    at = lambda x, p: OP.rotate(x, None, 0, [[p], [2 * p]], freq, (5, 3), adjacent)[0, 0]
    np.testing.assert_allclose(at(a, 0), a[0, 0])
    np.testing.assert_allclose(np.linalg.norm(at(a, 9)), np.linalg.norm(a))
    np.testing.assert_allclose(at(a, 9)[16:], a[0, 0, 16:])
    np.testing.assert_allclose(at(a, 9) @ at(b, 4), at(a, 105) @ at(b, 100))


def test_attention_matches_a_masked_softmax():
    import torch
    g = np.random.default_rng(1)
    n, length, prefix = 4, 11, 9
    q, k, v = (g.standard_normal(s) for s in ((n, 4, 8), (length, 2, 8), (length, 2, 8)))
    ks, vs = g.standard_normal((3, 2, 8)), g.standard_normal((3, 2, 8))
    there = np.arange(length) != 5
    out, lse, _, _ = OP.attend(q, k, v, there, prefix, ks, vs)
    t = lambda x: torch.from_numpy(x)
    kk, vv = (t(np.concatenate(x)).repeat_interleave(2, 1).permute(1, 0, 2) for x in ((ks, k), (vs, v)))
    on = np.array([[True] * 3 + [there[j] and (j < prefix or j <= length - n + i) for j in range(length)] for i in range(n)])
    ref = torch.nn.functional.scaled_dot_product_attention(t(q).permute(1, 0, 2), kk, vv, attn_mask=t(on))
    np.testing.assert_allclose(out, ref.permute(1, 0, 2).numpy(), atol=1e-12)
    z = (t(q).permute(1, 0, 2) @ kk.transpose(1, 2) / 8 ** 0.5).masked_fill(~t(on), -np.inf)
    np.testing.assert_allclose(lse, torch.logsumexp(z, -1).T.numpy(), atol=1e-12)
    # Weights over all keys of all rows sum to one each; the store took the rest.
    w = OP.gather(q, lse, k, there, prefix)
    np.testing.assert_allclose(w.sum(), torch.softmax(z, -1)[..., 3:].sum().item(), atol=1e-12)
    assert np.all(w[5] == 0)


def test_eviction_keeps_the_heaviest_and_the_earlier_of_equals():
    w = np.array([0., 5, 1, 5, np.nan, 2, 5, 0, 0, 0])
    assert OP.keep(w, 1, 2, 10) == list(range(10))
    assert OP.keep(w, 1, 2, 5) == [0, 1, 3, 8, 9]
    assert OP.keep(w, 0, 0, 4) == [1, 3, 5, 6]
    assert OP.keep(w, 2, 1, 9) == [0, 1, 2, 3, 5, 6, 7, 8, 9]
    assert OP.keep(w, 1, 2, 3) == [0, 8, 9]


def test_plan_of_row_tiles(lib):
    """The closed form that numbers a batch's key tiles against a count."""
    from partitioned_kv_cache_gb300 import rx
    g = np.random.default_rng(2)
    for _ in range(3000):
        G = 1 << int(g.integers(0, 8))
        a = 128 // G
        n, shared = int(g.integers(1, 40 if g.random() < 0.5 else 900)), int(g.integers(0, 5))
        length = n + int(g.integers(0, 300)) if g.random() < 0.7 else int(g.integers(0, 900))
        prefix = int(g.integers(0, 900)) if g.random() < 0.3 else 0
        R, keys = -(-n // a), int(g.choice([64, 128]))
        tiles = [shared + -(-max(1, OP.seen(min(n, (r + 1) * a) - 1, n, length, prefix)) // keys) for r in range(R)]
        r = int(g.integers(0, R + 1))
        before, row_tile = rx.page_plan(n, length, prefix, shared, G, keys, r)
        assert before == sum(tiles[:r])
        assert row_tile == (r if r < R else -1)


# ----------------------------------------------------------------- refusals
def _buf(n=1 << 16):
    b = ctypes.create_string_buffer(n + 256)
    return b, ctypes.addressof(b) + (-ctypes.addressof(b)) % 256


def _pages(rx, p, **kw):
    a = dict(k=p, v=p + 4096, weight=p + 8192, table=p + 8448, n_pages=1, page=16, max_pages=2, B=2)
    a.update(kw)
    return rx.RxPages(*(a[n] for n in ("k", "v", "weight", "table", "n_pages", "page", "max_pages", "B")))


def _heads(rx, p, **kw):
    a = dict(freq=p + 8704, q_weight=None, k_weight=None, Hq=2, Hkv=1, D=64, n_axes=1, sections=(32, 0, 0, 0), adjacent=0, eps=1e-6)
    a.update(kw)
    a["sections"] = (ctypes.c_int * 4)(*a["sections"])
    return rx.RxHeads(*(a[n] for n in ("freq", "q_weight", "k_weight", "Hq", "Hkv", "D", "n_axes", "sections", "adjacent", "eps")))


BAD_PAGES = [dict(page=8), dict(page=48), dict(page=512), dict(n_pages=0), dict(max_pages=0), dict(B=-1), dict(B=1025),
             dict(k=None), dict(v=None), dict(table=None), dict(n_pages=(1 << 31) - 1, page=256, B=1)]


def test_rotation_refuses_bad_arguments(lib):
    from partitioned_kv_cache_gb300 import rx
    keep, p = _buf()
    x, q, k, v, pos = p + 16384, p + 20480, p + 24576, p + 28672, p + 9216
    f = rx._lib.rx_rotate_heads

    def call(stride=256, N=3, heads=None, x=x, pos=pos, q=q, k=k, v=v):
        return f(x, stride, N, ctypes.byref(heads or _heads(rx, p)), pos, q, k, v, None)
    assert call(N=0) == 0
    assert call(N=-1) == -1
    assert call(stride=248) == -1 and call(stride=257) == -1
    assert f(x, 256, 3, None, pos, q, k, v, None) == -1
    for bad in (dict(Hq=0), dict(Hkv=0), dict(n_axes=0), dict(n_axes=5), dict(adjacent=2), dict(eps=-1.0), dict(eps=float("nan")),
                dict(sections=(12, 0, 0, 0)), dict(sections=(40, 0, 0, 0)), dict(sections=(-8, 16, 0, 0), n_axes=2), dict(freq=None)):
        assert call(heads=_heads(rx, p, **bad)) == -1, bad
    assert call(heads=_heads(rx, p, D=96)) == -6
    for name, at in (("x", x), ("q", q), ("k", k), ("v", v), ("pos", pos)):
        assert call(**{name: None}) == -1, name
        assert call(**{name: at + 2}) == -1, name
    assert call(q=x) == -1 and call(k=q) == -1 and call(v=pos) == -1 and call(N=1 << 30) == -1
    fp = rx._lib.rx_rotate_heads_paged
    qs, held, nl, ov = p + 12288, p + 12352, p + 12416, p + 12480

    def paged(N=3, pages=None, q_start=qs, held=held, new_len=nl, overflow=ov, q=q):
        return fp(x, 256, N, ctypes.byref(_heads(rx, p)), pos, q, ctypes.byref(pages or _pages(rx, p)), q_start, held, new_len,
                  overflow, None)
    assert paged(pages=_pages(rx, p, B=0)) == 0
    for bad in BAD_PAGES:
        assert paged(pages=_pages(rx, p, **bad)) == -1, bad
    assert paged(q_start=None) == -1 and paged(held=None) == -1 and paged(held=held + 2) == -1
    assert paged(new_len=held) == -1 and paged(overflow=qs) == -1 and paged(q=p) == -1
    assert paged(pages=_pages(rx, p, v=p + 1024)) == -1
    del keep


def test_attention_and_weights_refuse_bad_arguments(lib):
    from partitioned_kv_cache_gb300 import rx
    keep, p = _buf()
    q, out, lse, ws, qs, ln = p + 16384, p + 20480, p + 24576, p + 28672, p + 12288, p + 12352

    def attend(N=3, Hq=2, Hkv=1, D=64, pages=None, q=q, q_start=qs, length=ln, prefix=None, out=out, lse=lse, ws=ws, size=1 << 12):
        return rx._lib.rx_attend_pages(None, 0, q, N, Hq, Hkv, D, ctypes.byref(pages or _pages(rx, p)), q_start, length, prefix, out,
                                       lse, ws, size, None)

    def weigh(N=3, Hq=2, Hkv=1, D=64, pages=None, q=q, q_start=qs, length=ln, prefix=None, out=p + 32768, lse=lse, decay=1.0, ws=None,
              size=0):
        return rx._lib.rx_weigh_pages(q, lse, N, Hq, Hkv, D, ctypes.byref(pages or _pages(rx, p)), q_start, length, prefix, decay,
                                      out, ws, size, None)
    for call in (attend, weigh):
        assert call(N=0) == 0 and call(pages=_pages(rx, p, B=0)) == 0
        for bad in BAD_PAGES:
            assert call(pages=_pages(rx, p, **bad)) == -1, bad
        assert call(N=-1) == -1 and call(Hq=3, Hkv=2) == -1 and call(Hkv=0) == -1 and call(N=1 << 30) == -1
        assert call(Hq=6) == -6 and call(Hq=256) == -6 and call(D=80) == -6
        for name, at in (("q", q), ("q_start", qs), ("length", ln)):
            assert call(**{name: None}) == -1, name
            assert call(**{name: at + 2}) == -1, name
        assert call(prefix=ln + 2) == -1
        assert call(out=q) == -1 and call(out=p) == -1 and call(lse=lse + 2) == -1
    assert attend(out=None) == -1 and attend(ws=None) == -1 and attend(ws=ws + 16) == -1
    assert attend(lse=out) == -1 and attend(ws=out) == -1 and attend(ws=q) == -1
    assert weigh(lse=None) == -1 and weigh(decay=-1.0) == -1 and weigh(decay=float("nan")) == -1 and weigh(decay=float("inf")) == -1
    assert weigh(out=None, pages=_pages(rx, p, weight=None)) == -1 and weigh(pages=_pages(rx, p, weight=None)) == -1
    assert weigh(out=p + 8192 + 4) == -1 and weigh(out=p + 4096) == -1
    n = ctypes.c_longlong()
    f = rx._lib.rx_attend_pages_workspace
    assert f(1, 2, 1, 64, None) == -1 and f(-1, 2, 1, 64, ctypes.byref(n)) == -1 and f(1, 3, 2, 64, ctypes.byref(n)) == -1
    assert f(1, 6, 1, 64, ctypes.byref(n)) == -6 and f(1, 2, 1, 32, ctypes.byref(n)) == -6
    assert weigh(ws=ws + 16, size=64) == -1 and weigh(ws=q, size=64) == -1 and weigh(ws=p + 32768, size=64) == -1
    f = rx._lib.rx_weigh_pages_workspace
    assert f(1, 2, 1, None) == -1 and f(-1, 2, 1, ctypes.byref(n)) == -1 and f(1, 3, 2, ctypes.byref(n)) == -1
    assert f(1, 6, 1, ctypes.byref(n)) == -6
    del keep


def test_eviction_refuses_bad_arguments(lib):
    from partitioned_kv_cache_gb300 import rx
    keep, p = _buf()
    ln, kept, nl, ov, to = p + 12352, p + 16384, p + 12416, p + 12480, p + 12544

    def call(pages=None, Hkv=1, D=64, length=ln, sink=1, recent=2, budget=8, to=None, to_pages=0, new_len=nl, kept=kept, overflow=ov):
        return rx._lib.rx_evict_pages(ctypes.byref(pages or _pages(rx, p)), Hkv, D, length, sink, recent, budget, to, to_pages, new_len,
                                      kept, overflow, None)
    assert call(pages=_pages(rx, p, B=0)) == 0
    for bad in BAD_PAGES + [dict(weight=None)]:
        assert call(pages=_pages(rx, p, **bad)) == -1, bad
    assert call(D=32) == -6 and call(Hkv=0) == -1
    assert call(sink=-1) == -1 and call(recent=-1) == -1 and call(budget=0) == -1 and call(sink=6, recent=3) == -1
    assert call(length=None) == -1 and call(kept=None) == -1 and call(length=ln + 2) == -1 and call(to=to) == -1
    assert call(to=p + 8448, to_pages=2) == -1         # the pages' own table
    assert call(kept=p) == -1 and call(new_len=ln + 4) == -1 and call(overflow=ln) == -1 and call(kept=to, to=to, to_pages=2) == -1
    del keep


def test_binding_refuses_shapes_and_types(lib):
    import torch
    from partitioned_kv_cache_gb300 import rx
    z, bf, i32, f32 = torch.zeros, torch.bfloat16, torch.int32, torch.float32
    k, table, w = z(3, 16, 1, 64, dtype=bf), z(2, 2, dtype=i32), z(3, 16, 1)
    pages = rx.Pages(k, k.clone(), table, w)
    q, qs, ln, lse = z(5, 2, 64, dtype=bf), z(3, dtype=i32), z(2, dtype=i32), z(5, 2)
    # (the heads' own tensors are checked when they are made)
    with pytest.raises(ValueError, match="freq"):
        rx.Heads(2, 1, 64, z(32))
    heads = rx.Heads.__new__(rx.Heads)
    heads.Hq, heads.Hkv, heads.D, heads.axes, heads.width, heads._device = 2, 1, 64, 1, 256, 0
    x, pos = z(5, 256, dtype=bf), z(1, 5, dtype=i32)
    with pytest.raises(ValueError, match="axes"):
        rx.Heads(2, 1, 64, z(40), (8,) * 5)
    with pytest.raises(ValueError, match="pairs"):
        rx.Heads(2, 1, 64, z(32), (16, 8))
    with pytest.raises(ValueError, match="x must have shape"):
        rx.rotate_heads(x[:, :192], heads, pos)
    with pytest.raises(TypeError, match="x must be"):
        rx.rotate_heads(x.float(), heads, pos)
    with pytest.raises(ValueError, match="contiguous"):
        rx.rotate_heads(z(256, 5, dtype=bf).t(), heads, pos)
    with pytest.raises(ValueError, match="current device"):
        rx.rotate_heads(x, heads, pos)
    with pytest.raises(ValueError, match="q must have"):
        rx.attend_pages(q[0], pages, qs, ln)
    c = rx.Cache.__new__(rx.Cache)
    c._h = None
    with pytest.raises(ValueError, match="closed"):
        c.attend_pages(0, q, pages, qs, ln)
    with pytest.raises(ValueError, match="heads"):
        rx.attend_pages(z(5, 2, 128, dtype=bf), pages, qs, ln)
    with pytest.raises(ValueError, match="q_start"):
        rx.attend_pages(q, pages, qs[:2], ln)
    with pytest.raises(ValueError, match="length"):
        rx.attend_pages(q, pages, qs, z(3, dtype=i32))
    with pytest.raises(ValueError, match="pages.v"):
        rx.attend_pages(q, rx.Pages(k, k[:2], table, w), qs, ln)
    with pytest.raises(ValueError, match="pages.weight"):
        rx.attend_pages(q, rx.Pages(k, k, table, w[:2]), qs, ln)
    with pytest.raises(ValueError, match="CUDA"):
        rx.attend_pages(q, pages, qs, ln)
    with pytest.raises(ValueError, match="lse"):
        rx.weigh_pages(q, lse[:4], pages, qs, ln)
    with pytest.raises(ValueError, match="no weight"):
        rx.weigh_pages(q, lse, rx.Pages(k, k, table), qs, ln)
    with pytest.raises(ValueError, match="out"):
        rx.weigh_pages(q, lse, pages, qs, ln, out=z(3, 16, 2))
    with pytest.raises(ValueError, match="no weight"):
        rx.evict_pages(rx.Pages(k, k, table), ln, 4)
    with pytest.raises(ValueError, match="to must have"):
        rx.evict_pages(pages, ln, 4, to=z(3, 2, dtype=i32))
    with pytest.raises(ValueError, match="kept"):
        rx.evict_pages(pages, ln, 4, kept=z(2, 1, 5, dtype=i32))
