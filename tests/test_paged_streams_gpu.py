"""Language streams over a paged cache: norm and rotation of heads, attention,
gathered weight and eviction, against the fp64 oracle, and the four together.

Every pool is filled with NaN wherever no stream holds a key, so whatever reads
a place that it should not read shows.

Tolerances.  A bf16 rounding is within 2^-8 of the value.
Rotation: fp32 steps (norm, cosine, products) are within 2^-20 of |a| + |b| of
the pair; then one rounding.
Attention: a weight alpha_j enters its product with V with one rounding (2^-8
of it), the output is rounded once, and the fp32 steps move a weight by less
than 2^-11 of itself: |got - ref| <= (2^-8 + 2^-11) spread + 2^-8 |ref| + 1e-30,
spread = sum_j alpha_j |v_j|.  A score is a sum of D products in fp32, each
addition off by at most 2^-23 of the sum of magnitudes so far: err_s = (D + 2)
2^-23 reach with reach = max_j sum_i |q_i k_ji| / sqrt(D).  lse is off by at
most err_s, the exponentials' and the logarithm's 2^-20, and 2^-22 of itself.
Gathered weight: a term exp(s - lse) is off by err_s, by the rounding of lse
and of the exponent (2^-22 of their size) and by 2^-20, relative to itself.
"""
import numpy as np
import pytest

from oracle import pages as OP
from partitioned_kv_cache_gb300 import workload as W
from tests._util import dev, ensure_built, host64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rx():
    ensure_built()
    from partitioned_kv_cache_gb300 import rx as m
    return m


def _int(a):
    import torch
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _bits(g, shape, scale=1.0):
    return W.to_bf16_bits(scale * g.standard_normal(shape, dtype=np.float32))


f64 = W.bf16_bits_to_f64
NAN = 0x7FC0


class Pool:
    """A pool of pages whose unused places hold NaN, with tables in random order."""

    def __init__(self, g, lens, page, Hkv, D, extra=1, spare=2):
        self.page, self.Hkv, self.D, self.lens = page, Hkv, D, list(lens)
        counts = [-(-n // page) for n in lens]
        self.n_pages = sum(counts) + spare
        order = list(g.permutation(self.n_pages))
        width = max(1, max(counts, default=1)) + extra
        self.table = np.full((len(lens), width), -7, np.int64)
        for b, c in enumerate(counts):
            self.table[b, :c] = [order.pop() for _ in range(c)]
        self.free = order
        self.k = np.full((self.n_pages * page, Hkv, D), NAN, np.uint16)
        self.v = self.k.copy()
        self.w = np.full((self.n_pages * page, Hkv), np.nan, np.float32)

    def rows(self, b, n=None, table=None):
        t = (self.table if table is None else table)[b]
        return np.array([t[j // self.page] * self.page + j % self.page for j in range(self.lens[b] if n is None else n)], np.int64)

    def fill(self, g, scale=1.0):
        for b, n in enumerate(self.lens):
            r = self.rows(b)
            self.k[r], self.v[r] = _bits(g, (n, self.Hkv, self.D), scale), _bits(g, (n, self.Hkv, self.D))
            self.w[r] = g.random((n, self.Hkv), dtype=np.float32)
        return self

    def pages(self, rx, table=None):
        import torch
        shape = (self.n_pages, self.page, self.Hkv, self.D)
        return rx.Pages(dev(self.k).view(shape), dev(self.v).view(shape), _int(self.table if table is None else table),
                        torch.from_numpy(self.w.copy()).cuda().view(shape[:3]))


def _starts(new):
    return np.concatenate([[0], np.cumsum(new)])


def _same(t, bits):
    np.testing.assert_array_equal(t.contiguous().view(-1).view(__import__("torch").int16).cpu().numpy().view(np.uint16), bits.reshape(-1))


# ---------------------------------------------------------------- rotation
def _rotated(x, Hq, Hkv, wq, wk, eps, pos, freq, sections, adjacent):
    """Oracle's q, k, v and the tolerances of q and k; x [N][Hq+2Hkv][D] float64."""
    out = []
    for part, w in ((x[:, :Hq], wq), (x[:, Hq:Hq + Hkv], wk)):
        y = OP.rotate(part, w, eps, pos, freq, sections, adjacent)
        n = OP.rotate(part, w, eps, pos, freq, (), adjacent)           # normed, not turned
        R2 = sum(sections)
        tol = 2.0 ** -8 * np.abs(y) + 2.0 ** -20 * np.abs(n) + 1e-37
        one, two = (slice(0, 2 * R2, 2), slice(1, 2 * R2, 2)) if adjacent else (slice(0, R2), slice(R2, 2 * R2))
        both = 2.0 ** -20 * (np.abs(n[..., one]) + np.abs(n[..., two]))
        tol[..., one] += both
        tol[..., two] += both
        out += [y, tol]
    return out


ROTATIONS = [  # N, Hq, Hkv, D, sections, adjacent, norms
    (1, 1, 1, 64, (32,), False, ""),
    (5, 8, 1, 256, (128,), False, "qk"),
    (7, 8, 1, 256, (44, 42, 42), True, "qk"),
    (33, 32, 8, 128, (16, 16), False, "k"),
    (9, 3, 2, 128, (0, 8, 0, 24), True, "q"),
    (4, 2, 2, 64, (8,), False, ""),
    (6, 2, 1, 64, (0,), False, "qk"),
    (1300, 4, 1, 64, (10, 11, 11), False, "qk"),      # four tokens a CTA
]


@pytest.mark.parametrize("N,Hq,Hkv,D,sections,adjacent,norms", ROTATIONS)
def test_rotation_of_dense_heads(rx, N, Hq, Hkv, D, sections, adjacent, norms):
    import torch
    g = np.random.default_rng(N + D)
    H, pad = Hq + 2 * Hkv, 24
    x = _bits(g, (N, H * D + pad), 3.0)
    freq = (10000.0 ** -(np.arange(sum(sections)) / max(1, sum(sections)))).astype(np.float32)
    pos = g.integers(0, 5000, (len(sections), N))
    wq, wk = (g.standard_normal(D, dtype=np.float32) if n in norms else None for n in "qk")
    cuda = lambda a: None if a is None else torch.from_numpy(a).cuda()
    heads = rx.Heads(Hq, Hkv, D, cuda(freq), sections, cuda(wq), cuda(wk), 1e-6, adjacent)
    xd = dev(x)[:, :H * D]                                   # rows apart
    q, k, v = rx.rotate_heads(xd, heads, _int(pos))
    yq, tq, yk, tk = _rotated(f64(x[:, :H * D]).reshape(N, H, D), Hq, Hkv, wq, wk, 1e-6, pos, freq, sections, adjacent)
    assert np.all(np.abs(host64(q) - yq) <= tq)
    assert np.all(np.abs(host64(k) - yk) <= tk)
    _same(v, np.ascontiguousarray(x[:, :H * D].reshape(N, H, D)[:, Hq + Hkv:]))


def test_rotation_at_far_positions_and_over_bf16s_range(rx):
    """Angles to 2^31 (fp32 products would be off by whole turns), and rows of
    every magnitude through the norm."""
    import torch
    g = np.random.default_rng(3)
    N, D = 64, 64
    freq = np.array([1.0, 0.7, 1e-3, 6.25, 123.4, 2.0 ** -20, 3.1415927, 0.0] * 4, np.float32)
    pos = np.concatenate([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 6, 2 ** 24 + 1], g.integers(-2 ** 31, 2 ** 31, N - 7)])
    x = W.to_bf16_bits(g.standard_normal((N, 3, D), dtype=np.float32) * 2.0 ** g.integers(-60, 60, (N, 1, 1)).astype(np.float32))
    heads = rx.Heads(1, 1, D, torch.from_numpy(freq).cuda())
    q, k, _ = rx.rotate_heads(dev(x).view(N, -1), heads, _int(pos))
    # The angle in exact arithmetic: integers times 24-bit numbers, reduced in turns with Python's integers.
    from fractions import Fraction
    pi = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
    turn = np.empty((N, 32))
    for n in range(N):
        for i in range(32):
            a = Fraction(int(pos[n])) * Fraction(float(freq[i]))
            turn[n, i] = float(a - 2 * pi * round(a / (2 * pi)))
    y = f64(x)
    for got, part in ((q, y[:, :1]), (k, y[:, 1:2])):
        a, b, c, s = part[..., :32], part[..., 32:], np.cos(turn)[:, None], np.sin(turn)[:, None]
        ref = np.concatenate([a * c - b * s, b * c + a * s], -1)
        # The angle's own error: 2^-31 turns, and 2^-53 of freq / 2 pi times the position.
        size = np.abs(a) + np.abs(b)
        ang = 2 * np.pi * 2.0 ** -31 + np.abs(pos[:, None].astype(float)) * np.maximum(freq, 1) * 2.0 ** -52
        tol = 2.0 ** -8 * np.abs(ref) + np.concatenate([(2.0 ** -20 + ang[:, None]) * size] * 2, -1) + 1e-37
        assert np.all(np.abs(host64(got) - ref) <= tol)


def test_rotation_where_an_angles_error_shows(rx):
    """Positions at which a pair turns by nearly half a turn or a whole one: a sine
    near zero is the angle's own error and nothing else.  The error: a 32-bit
    fraction of a turn rounded to fp32, 2^-26 + 2^-32 of a turn, and for each position
    the rounding of freq / 2 pi, freq 2^-52 radians, of its fraction, 2^-64 of a turn,
    and of a negative one's distance from a whole turn, 2^-54."""
    import torch
    from fractions import Fraction
    D, R2 = 64, 32
    freq = np.array([1.0, 0.7, 6.25, 123.4, -1.0, -0.003] + [10000.0 ** -(i / 26) for i in range(26)], np.float32)
    two_pi = 2 * Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
    g = np.random.default_rng(5)
    pos = [355, 104348, 5419351, 80143857, 245850922, 411557987, -411557987, 2 ** 31 - 1, -2 ** 31]
    many = g.integers(-2 ** 31, 2 ** 31, 400000)
    for f in freq:   # of many positions those whose sine is smallest
        pos += [int(p) for p in many[np.argsort(np.abs(np.sin(many * np.float64(f))))[:4]]]
    N = len(pos)
    turn = np.empty((N, R2))
    for n, p in enumerate(pos):
        for i, f in enumerate(freq):
            a = Fraction(p) * Fraction(float(f))
            turn[n, i] = float(a - two_pi * round(a / two_pi))
    assert np.min(np.abs(np.sin(turn))) < 1e-8
    x = np.zeros((N, 3, D), np.float32)
    x[..., R2:] = 1                                           # (0, 1) -> (-sin, cos)
    heads = rx.Heads(1, 1, D, torch.from_numpy(freq).cuda())
    q, _, _ = rx.rotate_heads(dev(W.to_bf16_bits(x)).view(N, -1), heads, _int(pos))
    far = np.abs(np.array(pos, np.float64))[:, None]
    angle = 2 * np.pi * (2.0 ** -26 + 2.0 ** -32 + far * (2.0 ** -64 + (freq < 0) * 2.0 ** -54)) + far * np.abs(freq) * 2.0 ** -52
    got = host64(q)[:, 0]
    for ref, at in ((-np.sin(turn), slice(0, R2)), (np.cos(turn), slice(R2, D))):
        # sincospi is good to 2 of fp32's last places, the output is rounded once.
        assert np.all(np.abs(got[:, at] - ref) <= angle + (2.0 ** -8 + 2.0 ** -21) * np.abs(ref))


@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-30])
@pytest.mark.parametrize("N,Hq,Hkv,D", [(70, 2, 1, 64), (70, 1, 1, 128), (70, 1, 2, 256), (700, 3, 1, 64)])
def test_norm_over_bf16s_range(rx, eps, N, Hq, Hkv, D):
    """Heads from bf16's smallest values to its largest: squares that fp32 cannot
    hold, rows of zeros, and one large value among small ones."""
    import torch
    g = np.random.default_rng([N, D])
    H = Hq + 2 * Hkv
    x = g.standard_normal((N, H, D), dtype=np.float32).clip(-3, 3) * 2.0 ** g.integers(-133, 126, (N, H, 1)).astype(np.float32)
    x[::7, :, 5] = 2.0 ** 120
    x[1::7] = 2.0 ** -133
    if eps:
        x[2::7] = 0
    x = W.to_bf16_bits(x)
    freq = (100.0 ** -(np.arange(D // 2) / (D // 2))).astype(np.float32)
    pos = g.integers(0, 500, (1, N))
    wq, wk = (1 + 0.25 * g.standard_normal(D, dtype=np.float32) for _ in range(2))
    cuda = lambda a: torch.from_numpy(a).cuda()
    heads = rx.Heads(Hq, Hkv, D, cuda(freq), (), cuda(wq), cuda(wk), eps)
    q, k, v = rx.rotate_heads(dev(x).view(N, -1), heads, _int(pos))
    y = f64(x)
    live = np.any(y != 0, -1)
    assert eps or np.all(live)
    eps32 = float(np.float32(eps))
    yq, tq, yk, tk = _rotated(y, Hq, Hkv, wq, wk, eps32, pos, freq, (D // 2,), False)
    assert np.all(np.abs(host64(q) - yq) <= tq)
    assert np.all(np.abs(host64(k) - yk) <= tk)
    _same(v, np.ascontiguousarray(x[:, Hq + Hkv:]))


@pytest.mark.parametrize("page,held,new", [
    (16, [0], [1]),
    (16, [0, 15, 16, 31], [1, 1, 1, 2]),
    (64, [0, 5, 63, 200, 7], [3, 0, 70, 1, 129]),
    (256, [255, 256, 0], [2, 1, 300]),
])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 256), (4, 2, 64)])
def test_rotation_into_pages(rx, page, held, new, Hq, Hkv, D):
    """Every byte of the pools, places that nothing was written to among them."""
    import torch
    g = np.random.default_rng(page + sum(new))
    pool = Pool(g, [h + n for h, n in zip(held, new)], page, Hkv, D)
    start = _starts(new) + 2                                 # two tokens before and three behind are nobody's
    N, H = start[-1] + 3, Hq + 2 * Hkv
    x, pos = _bits(g, (N, H * D)), g.integers(0, 999, (1, N))
    freq = (100.0 ** -(np.arange(D // 2) / (D // 2))).astype(np.float32)
    heads = rx.Heads(Hq, Hkv, D, torch.from_numpy(freq).cuda())
    pages, hd = pool.pages(rx), _int(held)
    new_len, over = _int([-1] * len(held)), _int([0])
    q = torch.full((N, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    rx.rotate_heads_paged(dev(x), heads, _int(pos), pages, _int(start), hd, q=q, new_len=new_len, overflow=over)
    _, k, v = rx.rotate_heads(dev(x), heads, _int(pos))      # bit for bit the dense call's
    q2 = rx.rotate_heads(dev(x), heads, _int(pos))[0]
    kb, vb = (t.view(torch.int16).cpu().numpy().view(np.uint16) for t in (k, v))
    want_k, want_v, want_w = pool.k.copy(), pool.v.copy(), pool.w.copy()
    for b, (h, n) in enumerate(zip(held, new)):
        r = pool.rows(b)[h:h + n]
        want_k[r], want_v[r], want_w[r] = kb[start[b]:start[b] + n], vb[start[b]:start[b] + n], 0
    _same(pages.k, want_k)
    _same(pages.v, want_v)
    np.testing.assert_array_equal(pages.weight.cpu().numpy().reshape(want_w.shape), want_w)
    assert torch.equal(q[2:N - 3], q2[2:N - 3])
    assert torch.all(q[:2] == 7) and torch.all(q[N - 3:] == 7)
    assert new_len.tolist() == [h + n for h, n in zip(held, new)] and over.item() == 0 and hd.tolist() == held


def test_rotation_drops_what_has_no_place(rx):
    """Full tables, lengths out of range, entries that name no page."""
    import torch
    g = np.random.default_rng(8)
    Hq, Hkv, D, page = 2, 1, 64, 16
    pool = Pool(g, [32, 32, 32, 32, 20], page, Hkv, D, extra=0)
    pool.table[3, 1] = pool.n_pages
    held, new = [30, -1, 33, 14, 3], [5, 2, 2, 4, 0]
    start = _starts(new)
    x = _bits(g, (start[-1], 4 * D))
    heads = rx.Heads(Hq, Hkv, D, torch.ones(32, device="cuda"))
    pos = _int(g.integers(0, 99, start[-1]))
    pages, new_len, over = pool.pages(rx), _int([9] * 5), _int([0])
    rx.rotate_heads_paged(dev(x), heads, pos, pages, _int(start), _int(held), new_len=new_len, overflow=over)
    k = rx.rotate_heads(dev(x), heads, pos)[1].view(torch.int16).cpu().numpy().view(np.uint16)
    want = pool.k.copy()
    for b, count in ((0, 2), (3, 2)):
        r = [pool.table[b][(held[b] + t) // page] * page + (held[b] + t) % page for t in range(count)]
        want[r] = k[start[b]:start[b] + count]
    _same(pages.k, want)
    assert new_len.tolist() == [32, -1, 33, 18, 3] and over.item() == 1


# --------------------------------------------------------------- attention
def _store(rx, g, Hq, Hkv, D, P, N, F, pushed, spare=0, L=1):
    """A cache with P pinned tokens and `pushed` frames; the keys its window holds."""
    c = rx.Cache(L, Hq, Hkv, D, P, N, F, 1, spare_slot=spare)
    pk, pv = _bits(g, (L, P, Hkv, D)), _bits(g, (L, P, Hkv, D))
    if P:
        c.pin_prefix(dev(pk), dev(pv))
    frames = [(_bits(g, (L, F, Hkv, D)), _bits(g, (L, F, Hkv, D))) for _ in range(pushed)]
    for k, v in frames:
        c.push_frame(dev(k), dev(v))
    last = frames[-N:]
    ks, vs = (np.concatenate([f64(p)] + [f64(f[i]) for f in last], 1) for i, p in enumerate((pk, pv)))
    return c, ks, vs


def _err_s(D, reach):
    return (D + 2) * 2.0 ** -23 * reach


def _check_attention(out, lse, ref, ref_lse, spread, reach):
    tol = (2.0 ** -8 + 2.0 ** -11) * spread + 2.0 ** -8 * np.abs(ref) + 1e-30
    assert np.all(np.isfinite(out))
    assert np.all(np.abs(out - ref) <= tol), np.max(np.abs(out - ref) / tol)
    none = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(lse), none)
    off = np.abs(np.where(none, 0, lse) - np.where(none, 0, ref_lse))
    assert np.all(off <= _err_s(ref.shape[-1], reach) + 2.0 ** -20 + 2.0 ** -22 * np.where(none, 0, np.abs(ref_lse)))


def _attend_case(rx, g, pool, new, Hq, prefix=None, cache=None, ks=None, vs=None, layer=0, lens=None, there=None, edge=1):
    """One call against the oracle; rows of tokens in no stream stay as they are."""
    import torch
    lens = pool.lens if lens is None else lens
    start = _starts(new) + edge
    N = start[-1] + edge
    q = _bits(g, (N, Hq, pool.D))
    out = torch.full((N, Hq, pool.D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((N, Hq), 7.0, device="cuda")
    args = (dev(q), pool.pages(rx), _int(start), _int(lens))
    kw = dict(prefix=None if prefix is None else _int(prefix), out=out, lse=lse)
    if cache is None:
        rx.attend_pages(*args, **kw)
    else:
        cache.attend_pages(layer, *args, **kw)
    o, e = host64(out), lse.double().cpu().numpy()
    if edge:
        for rows in (slice(0, edge), slice(N - edge, N)):
            assert np.all(o[rows] == 7) and np.all(e[rows] == 7)
    for b, n in enumerate(new):
        if not n:
            continue
        length = min(max(lens[b], 0), pool.table.shape[1] * pool.page)
        names = np.array([0 <= pool.table[b][j // pool.page] < pool.n_pages for j in range(length)], bool)
        r = np.where(names, pool.rows(b, length), 0)
        k, v = f64(pool.k[r]), f64(pool.v[r])
        k[~names], v[~names] = 0, 0
        s = slice(start[b], start[b] + n)
        got = OP.attend(f64(q[s]), k, v, names, 0 if prefix is None else prefix[b], None if ks is None else ks[layer],
                        None if vs is None else vs[layer])
        _check_attention(o[s], e[s], *got)
    return q, start, o, e


HEADS = [(8, 1, 256), (8, 2, 128), (4, 4, 64), (128, 1, 64), (2, 1, 128), (1, 1, 256)]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("page", [16, 64])
def test_attention_of_single_tokens(rx, Hq, Hkv, D, page):
    g = np.random.default_rng(Hq + D + page)
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200]
    _attend_case(rx, g, Pool(g, lens, page, Hkv, D).fill(g), [1] * len(lens), Hq)


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("page", [32, 128])
def test_attention_of_chunks(rx, Hq, Hkv, D, page):
    """Chunks of every length around a row tile's tokens, with and without keys
    before them, an idle stream among them."""
    g = np.random.default_rng(Hq + D + page)
    a = 128 // (Hq // Hkv)
    new = [min(n, 70) for n in (1, a, a + 1, max(1, a - 1), 0, 2 * a + 3, 5)]
    lens = [n + h for n, h in zip(new, (0, 0, 60, 1, 33, 130, 59))]
    _attend_case(rx, g, Pool(g, lens, page, Hkv, D).fill(g), new, Hq)


@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 1, 256, 16), (8, 2, 128, 64), (4, 4, 64, 256)])
def test_attention_with_a_prefix(rx, Hq, Hkv, D, page):
    g = np.random.default_rng(D)
    new = [40, 33, 1, 65, 20]
    lens = [40, 90, 70, 65, 30]
    _attend_case(rx, g, Pool(g, lens, page, Hkv, D).fill(g), new, Hq, prefix=[40, 64, 1000, 33, -5])


@pytest.mark.parametrize("P,N,F,pushed,spare", [(0, 3, 50, 0, 0), (37, 3, 100, 2, 0), (64, 2, 64, 5, 0), (100, 3, 64, 7, 1), (5, 2, 128, 1, 1)])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 256), (8, 2, 128), (4, 4, 64)])
def test_attention_over_the_store_and_pages(rx, P, N, F, pushed, spare, Hq, Hkv, D):
    g = np.random.default_rng(P + D)
    cache, ks, vs = _store(rx, g, Hq, Hkv, D, P, N, F, pushed, spare, L=2)
    new, lens = [1, 30, 0, 17], [20, 130, 9, 17]
    pool = Pool(g, lens, 64, Hkv, D).fill(g)
    for layer in range(2):
        _attend_case(rx, g, pool, new, Hq, cache=cache, ks=ks, vs=vs, layer=layer, prefix=[0, 100, 5, 17] if layer else None)
    assert cache.check_device_error() == 0
    cache.close()


def test_rows_without_keys(rx):
    """Empty streams, more new tokens than keys, a table that names no page: zeros
    and lse -infinity where nothing is seen; with a store, the store alone."""
    g = np.random.default_rng(5)
    Hq, Hkv, D = 8, 1, 256
    pool = Pool(g, [0, 3, 40, 70, 64], 16, Hkv, D).fill(g)
    pool.table[2] = -1
    pool.table[3, 1], pool.table[3, 4] = pool.n_pages, -3        # holes, one in the last tile
    new = [2, 5, 3, 20, 1]
    _, start, out, lse = _attend_case(rx, g, pool, new, Hq)
    assert np.all(out[start[0]:start[1]] == 0) and np.all(np.isneginf(lse[start[0]:start[1]]))
    assert np.all(np.isneginf(lse[start[1]:start[1] + 2])) and np.all(np.isneginf(lse[start[2]:start[3]]))
    cache, ks, vs = _store(rx, g, Hq, Hkv, D, 30, 2, 40, 3)
    _attend_case(rx, g, pool, new, Hq, cache=cache, ks=ks, vs=vs)
    cache.close()


def test_lengths_and_ranges_out_of_bounds_are_clamped(rx):
    import torch
    g = np.random.default_rng(6)
    pool = Pool(g, [48, 48, 48], 16, 1, 64, extra=0).fill(g)
    _attend_case(rx, g, pool, [1, 2, 1], 2, lens=[-4, 1000, 48])
    # Ranges beyond N, and ranges that run backwards, hold no tokens.
    q, out = dev(_bits(g, (4, 2, 64))), torch.full((4, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    rx.attend_pages(q, pool.pages(rx), _int([3, 1, 1, 99]), _int([48] * 3), out=out)
    o = host64(out)
    assert np.all(o[0] == 7) and np.all(np.isfinite(o)) and not np.any(o[1:] == 7)


@pytest.mark.parametrize("D,Hq,Hkv", [(256, 8, 1), (128, 4, 2), (64, 4, 4)])
@pytest.mark.parametrize("what", [np.inf, -np.inf, np.nan])
def test_values_that_are_not_finite_stay_with_the_rows_that_see_them(rx, D, Hq, Hkv, what):
    """A chunk's token 10 has a bad value, its token 20 a bad key, a place behind
    the stream's end both: rows before them are as without them."""
    g = np.random.default_rng(D)
    n, held = 40, 50
    pool = Pool(g, [held + n], 16, Hkv, D).fill(g)
    q = _bits(g, (n, Hq, D))
    bad = W.to_bf16_bits(np.array([what], np.float32))[0]
    ref = OP.attend(f64(q), f64(pool.k[pool.rows(0)]), f64(pool.v[pool.rows(0)]), np.ones(held + n, bool), 0)
    pool.v[pool.rows(0)[held + 10], Hkv - 1, 3] = bad
    pool.k[pool.rows(0)[held + 20], Hkv - 1, 5] = bad
    out, lse = rx.attend_pages(dev(q), pool.pages(rx), _int([0, n]), _int([held + n]), lse=True)
    o, e = host64(out), lse.double().cpu().numpy()
    G = Hq // Hkv
    _check_attention(o[:10], e[:10], *(x[:10] for x in ref))
    first = Hkv - 1
    _check_attention(o[:, :first * G], e[:, :first * G], *(x[:, :first * G] for x in ref))
    assert not np.any(np.isfinite(o[10:, first * G:, 3]))
    if np.isnan(what):
        assert np.all(np.isnan(o[20:, first * G:])) and np.all(np.isnan(e[20:, first * G:]))


@pytest.mark.parametrize("D,Hq,Hkv", [(256, 8, 1), (128, 4, 2), (64, 4, 4)])
@pytest.mark.parametrize("what", [np.inf, np.nan])
@pytest.mark.parametrize("n,held", [(40, 50), (1, 700), (200, 9000)])
def test_values_have_no_part_in_lse(rx, D, Hq, Hkv, what, n, held):
    """Values that are not finite, at places that some rows of a tile see and some
    do not and at places that all see: lse, which is of the scores alone, is bit
    for bit as without them, and so is what is gathered by it."""
    import torch
    g = np.random.default_rng([D, n])
    pool = Pool(g, [held + n, 60], 16, Hkv, D).fill(g)
    q = dev(_bits(g, (n + 60, Hq, D)))
    args = (_int([0, n, n + 60]), _int([held + n, 60]))
    clean = pool.pages(rx)
    ref, ref_lse = rx.attend_pages(q, clean, *args, lse=True)
    bad = W.to_bf16_bits(np.array([what], np.float32))[0]
    pool.v[pool.rows(0)[[3, held + n - 1]], :, 3] = bad
    pool.v[pool.rows(1)[7], Hkv - 1, 1] = bad
    pages = pool.pages(rx)
    out, lse = rx.attend_pages(q, pages, *args, lse=True)
    assert torch.equal(lse, ref_lse) and torch.all(torch.isfinite(lse))
    assert not torch.any(torch.isfinite(out[:n, :, 3])) and not torch.any(torch.isfinite(out[n + 7:, Hq - 1, 1]))
    assert torch.equal(out[n:n + 7], ref[n:n + 7])
    rx.weigh_pages(q, lse, pages, *args)
    rx.weigh_pages(q, ref_lse, clean, *args)
    r = np.concatenate([pool.rows(0), pool.rows(1)])
    a, b = (p.weight.view(-1, Hkv).cpu().numpy()[r] for p in (pages, clean))
    assert np.all(np.isfinite(a)) and np.array_equal(a, b)


@pytest.mark.parametrize("D,Hq,Hkv", [(256, 8, 1), (128, 4, 2), (64, 4, 4)])
def test_infinite_keys(rx, D, Hq, Hkv):
    """A key with an infinity: rows to whose queries it is opposite get a score of
    -infinity and are as without it; the others, +infinity, are not finite."""
    import torch
    g = np.random.default_rng(D)
    n, held = 30, 100
    pool = Pool(g, [held + n], 32, Hkv, D).fill(g)
    q = f64(_bits(g, (n, Hq, D)))
    q[..., 5] = np.where(np.arange(n)[:, None] % 2, 1, -1) * (1 + np.abs(q[..., 5]))
    bits = W.to_bf16_bits(q.astype(np.float32))
    there = np.ones(held + n, bool)
    at = [40, held + 12]
    there[at] = False
    ref = OP.attend(f64(bits), f64(pool.k[pool.rows(0)]), f64(pool.v[pool.rows(0)]), there, 0)
    pool.k[pool.rows(0)[at], :, 5] = W.to_bf16_bits(np.array([np.inf], np.float32))[0]
    out, lse = rx.attend_pages(dev(bits), pool.pages(rx), _int([0, n]), _int([held + n]), lse=True)
    o, e = host64(out), lse.double().cpu().numpy()
    _check_attention(o[::2], e[::2], *(x[::2] for x in ref))
    assert not np.any(np.isfinite(o[1::2])) and not np.any(np.isfinite(e[1::2]))


@pytest.mark.parametrize("Hq,Hkv,D,lens,new", [
    (8, 1, 256, [20000], [1]),                    # one stream over all SMs
    (8, 1, 256, [9000, 100, 5000], [1, 1, 8]),
    (8, 8, 128, [7001, 3], [1, 1]),
    (4, 1, 64, [3000] * 20, [1] * 20),
])
def test_attention_over_long_streams(rx, Hq, Hkv, D, lens, new):
    """Units cut into many parts, few parts and none."""
    g = np.random.default_rng(sum(lens))
    _attend_case(rx, g, Pool(g, lens, 64, Hkv, D).fill(g), new, Hq, edge=0)


def test_as_many_streams_as_a_call_takes(rx):
    """1024 streams, a third of them idle, lengths from 0 on."""
    g = np.random.default_rng(14)
    lens = [int(x) for x in g.integers(0, 70, 1024)]
    new = [min(n, int(x)) for n, x in zip(lens, g.integers(0, 3, 1024))]
    pool = Pool(g, lens, 16, 1, 64).fill(g)
    _attend_case(rx, g, pool, new, 2)
    _weigh_case(rx, g, pool, new, 2)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_outputs_aligned_to_16_bytes_only(rx, D):
    import torch
    g = np.random.default_rng(15)
    pool = Pool(g, [300, 40], 32, 1, D).fill(g)
    args = (dev(_bits(g, (50, 4, D))), pool.pages(rx), _int([0, 20, 50]), _int([300, 40]))
    ref = rx.attend_pages(*args)
    buf = torch.full((50 * 4 * D + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[8:8 + 50 * 4 * D].view(50, 4, D)
    assert out.data_ptr() % 32 == 16
    rx.attend_pages(*args, out=out)
    assert torch.equal(out, ref) and torch.all(buf[:8] == 7) and torch.all(buf[-8:] == 7)


def test_large_scores_and_far_apart_maxima(rx):
    """Scores to some hundreds: the running maximum is renewed all along the
    stream, in cut units too."""
    g = np.random.default_rng(11)
    Hq, Hkv, D = 8, 1, 128
    pool = Pool(g, [4000, 300], 32, Hkv, D).fill(g)
    r = pool.rows(0)
    pool.k[r] = W.to_bf16_bits((f64(pool.k[r]) * np.linspace(0, 30, len(r))[:, None, None]).astype(np.float32))
    _attend_case(rx, g, pool, [20, 300], Hq)


def test_full_size_chunks_give_the_same_bits_twice(rx):
    """Thousands of row tiles: a second call, beside other work, gives the same
    bits, and a sample of rows agrees with the oracle."""
    import torch
    g = np.random.default_rng(12)
    Hq, Hkv, D = 8, 1, 256
    lens, new = [2048, 3000, 2905, 5001, 4097], [2048, 1500, 2048, 777, 2000]
    pool = Pool(g, lens, 64, Hkv, D).fill(g)
    start = _starts(new)
    q = _bits(g, (start[-1], Hq, D))
    args = (dev(q), pool.pages(rx), _int(start), _int(lens))
    first = rx.attend_pages(*args, lse=True)
    for _ in range(4):
        again = rx.attend_pages(*args, lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    o, e = host64(first[0]), first[1].double().cpu().numpy()
    for b in range(5):
        k, v = f64(pool.k[pool.rows(b)]), f64(pool.v[pool.rows(b)])
        for t in (0, 1, new[b] // 2, new[b] - 17, new[b] - 1):
            length = lens[b] - new[b] + t + 1
            got = OP.attend(f64(q[start[b] + t:start[b] + t + 1]), k[:length], v[:length], np.ones(length, bool), 0)
            _check_attention(o[start[b] + t:start[b] + t + 1], e[start[b] + t:start[b] + t + 1], *got)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("one_cta,n", [(True, 300_000), (False, 4_000_005)])
def test_sums_over_very_many_keys(rx, D, one_cta, n):
    """Hundreds of thousands of keys in one CTA, units whole and cut, over pages that
    the table names again and again; values of one sign, where an accumulator that
    drops its last places is always off to the same side.  16384 keys are 1024
    additions of 16 products, each of which costs up to two last places, 2^-22, of the
    sum so far, on average half of the whole: 2^-13 of the result at most; longer sums
    are closed in fp32.  The outputs' own rounding
    and the weights' average out over the heads: a mean over 152 x 64 outputs that are
    off by up to 2^-9 has a deviation of 1.2e-5, over 2 x 64 1e-4, and is held to five
    times that."""
    import torch
    H = torch.cuda.get_device_properties(0).multi_processor_count if one_cta else 2
    torch.manual_seed(D)
    page, each = 256, 4                                            # the second half's keys are larger
    k = torch.randn(2 * each, page, H, D, device="cuda") * torch.tensor([0.5] * each + [1.5] * each, device="cuda")[:, None, None, None]
    k, v = k.bfloat16(), (0.5 + 0.5 * torch.rand(2 * each, page, H, D, device="cuda")).bfloat16()
    q = torch.randn(1, H, D, device="cuda").bfloat16()
    slots = torch.arange(-(-n // page), device="cuda")
    table = (slots % each + each * (slots >= len(slots) // 2)).to(torch.int32)
    out, lse = rx.attend_pages(q, rx.Pages(k, v, table[None]), _int([0, 1]), _int([n]), lse=True)
    times = torch.bincount(table[:-1].long(), minlength=2 * each).double()[:, None].repeat(1, page)
    times[table[-1].long(), :n - (len(slots) - 1) * page] += 1
    z = torch.einsum("hd,khd->hk", q[0].double(), k.view(-1, H, D).double()) / D ** 0.5 + times.view(-1).log()
    ref = torch.einsum("hk,khd->hd", torch.softmax(z, -1), v.view(-1, H, D).double())
    off = (out[0].double() - ref) / ref
    assert off.abs().max().item() <= 2.0 ** -8 + 2.0 ** -8 + 2.0 ** -11
    assert abs(off.mean().item()) <= 2.0 ** -13 + (2.0 ** -14 if one_cta else 2.0 ** -11)
    reach = (q[0].double().abs() * k.view(-1, H, D).double().abs()).sum(-1).max().item() / D ** 0.5
    ref_lse = torch.logsumexp(z, -1)
    assert torch.all((lse[0].double() - ref_lse).abs() <= _err_s(D, reach) + 2.0 ** -20 + 2.0 ** -22 * ref_lse.abs())


def test_pools_beyond_32_bits(rx):
    """Places whose bytes lie beyond 2^32 in the pool: rotation, attention,
    weight and eviction."""
    import torch
    g = np.random.default_rng(13)
    Hq, Hkv, D, page = 2, 1, 256, 256
    n_pages = (1 << 33) // (page * D * 2) + 4
    k, v = (torch.zeros((n_pages, page, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w = torch.zeros((n_pages, page, Hkv), device="cuda")
    table = _int([[n_pages - 1, 0, n_pages - 2]])
    n = 520
    pages = rx.Pages(k, v, table, w)
    x, pos = _bits(g, (n, 4 * D)), np.arange(n)
    heads = rx.Heads(Hq, Hkv, D, torch.ones(8, device="cuda") * 0.01)
    q = rx.rotate_heads_paged(dev(x), heads, _int(pos), pages, _int([0, n]), _int([0]))
    _, kk, vv = rx.rotate_heads(dev(x), heads, _int(pos))
    at = lambda p: torch.cat([p[n_pages - 1], p[0], p[n_pages - 2]])[:n]
    assert torch.equal(at(k), kk) and torch.equal(at(v), vv)
    out, lse = rx.attend_pages(q[-1:].contiguous(), pages, _int([0, 1]), _int([n]), lse=True)
    ref = OP.attend(host64(q[-1:]), host64(kk), host64(vv), np.ones(n, bool), 0)
    _check_attention(host64(out), lse.double().cpu().numpy(), *ref)
    rx.weigh_pages(q[-1:].contiguous(), lse, pages, _int([0, 1]), _int([n]))
    _check_weight(at(w).cpu().numpy(), OP.gather(host64(q[-1:]), lse.double().cpu().numpy(), host64(kk), np.ones(n, bool), 0), D,
                  ref[3].max(), np.abs(ref[1]).max())
    before = at(w).clone()
    kept = rx.evict_pages(pages, _int([n]), 300, sink=2, recent=10)
    want = OP.keep(before[:, 0].cpu().numpy(), 2, 10, 300)
    assert kept[0, 0].tolist() == want and torch.equal(at(k)[:300], kk[want]) and torch.equal(at(v)[:300], vv[want])


# ------------------------------------------------------------------ weight
def _check_weight(got, ref, D, reach, size):
    """size: the largest |lse|."""
    rel = _err_s(D, reach) + 2.0 ** -22 * (size + reach) + 2.0 ** -20
    assert np.all(np.abs(got - ref) <= rel * ref + 1e-30), np.max(np.abs(got - ref) / (rel * ref + 1e-30))


def _weigh_case(rx, g, pool, new, Hq, prefix=None, decay=1.0, apart=False, cache=None, ks=None, vs=None):
    import torch
    start = _starts(new) + 1
    N = start[-1] + 1
    q = _bits(g, (N, Hq, pool.D))
    pages, sd, ld = pool.pages(rx), _int(start), _int(pool.lens)
    pf = None if prefix is None else _int(prefix)
    call = rx.attend_pages if cache is None else lambda *a, **k: cache.attend_pages(0, *a, **k)
    lse = torch.full((N, Hq), np.nan, device="cuda")
    call(dev(q), pages, sd, ld, prefix=pf, lse=lse)
    to = torch.full_like(pages.weight, 5.0) if apart else None
    got = rx.weigh_pages(dev(q), lse, pages, sd, ld, prefix=pf, decay=decay, out=to)
    assert got is (to if apart else pages.weight)
    got = got.cpu().numpy().reshape(pool.w.shape)
    want = np.full_like(pool.w, 5.0) if apart else pool.w.copy()
    e = lse.double().cpu().numpy()
    touched = np.zeros(len(want), bool)
    for b, n in enumerate(new):
        if not n or not pool.lens[b]:
            continue
        names = np.array([0 <= pool.table[b][j // pool.page] < pool.n_pages for j in range(pool.lens[b])], bool)
        r = np.where(names, pool.rows(b), 0)
        k = f64(pool.k[r])
        k[~names] = 0
        s = slice(start[b], start[b] + n)
        ref = OP.gather(f64(q[s]), e[s], k, names, 0 if prefix is None else prefix[b])
        reach = np.max(np.abs(k).sum(-1)) * np.max(np.abs(f64(q[s]))) / np.sqrt(pool.D)
        old = decay * pool.w[r].astype(np.float64) if decay else 0 * ref
        size = np.max(np.abs(e[s][np.isfinite(e[s])]), initial=0)
        rel = _err_s(pool.D, reach) + 2.0 ** -22 * (size + reach) + 2.0 ** -20
        g_, r_ = got[r][names], (old + ref)[names]
        tol = rel * ref[names] + 2.0 ** -23 * np.abs(r_) + 1e-30
        assert np.all(np.abs(g_ - r_) <= tol), np.max(np.abs(g_ - r_) / tol)
        touched[r[names]] = True
    np.testing.assert_array_equal(got[~touched], want[~touched])


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("page", [16, 128])
def test_weight_of_single_tokens_and_chunks(rx, Hq, Hkv, D, page):
    g = np.random.default_rng(Hq + D + page)
    new = [1, 1, 0, 9, 70, 33]
    lens = [1, 130, 40, 9, 200, 129]
    _weigh_case(rx, g, Pool(g, lens, page, Hkv, D).fill(g), new, Hq)
    _weigh_case(rx, g, Pool(g, lens, page, Hkv, D).fill(g), new, Hq, prefix=[0, 5, 9, 9, 150, 128], decay=0.25, apart=True)


def test_weight_with_pages_that_are_not_named_and_rows_that_see_nothing(rx):
    g = np.random.default_rng(5)
    pool = Pool(g, [0, 3, 40, 70, 64], 16, 1, 128).fill(g)
    pool.table[2] = -1
    pool.table[3, 1] = pool.n_pages
    _weigh_case(rx, g, pool, [2, 5, 3, 20, 1], 8)


@pytest.mark.parametrize("lens,new,Hq,Hkv,D,page,prefix,decay", [
    ([400], [300], 8, 1, 256, 64, None, 0.5),             # fewer keys than CTAs have: every share is a part
    ([130, 700], [127, 260], 4, 1, 64, 16, [60, 300], 1.0),
    ([900, 0, 333, 1500], [450, 7, 0, 600], 16, 2, 128, 32, [0, 0, 9, 1500], 0.0),
    ([0, 640, 50], [2, 640, 33], 32, 1, 64, 256, None, 1.0),
])
def test_weight_of_chunks_that_several_ctas_share(rx, lens, new, Hq, Hkv, D, page, prefix, decay):
    """Few keys and many rows: a block of keys is cut between row tiles."""
    g = np.random.default_rng([lens[0], Hq])
    pool = Pool(g, lens, page, Hkv, D).fill(g)
    pool.table[-1][min(2, len(pool.table[-1]) - 1)] = -1
    assert rx.weigh_pages_workspace(sum(new), Hq, Hkv) > 0
    _weigh_case(rx, g, pool, new, Hq, prefix=prefix, decay=decay, apart=prefix is not None)


def test_weight_without_decay_does_not_read_the_old(rx):
    g = np.random.default_rng(6)
    pool = Pool(g, [100, 20], 32, 2, 64).fill(g)
    pool.w[:] = np.nan
    _weigh_case(rx, g, pool, [3, 20], 4, decay=0.0)


def test_weight_beside_the_store(rx):
    """What the store took is not counted: weights and the store's share sum to
    the number of rows."""
    g = np.random.default_rng(7)
    cache, ks, vs = _store(rx, g, 8, 1, 256, 40, 2, 64, 2)
    _weigh_case(rx, g, Pool(g, [90, 33], 64, 1, 256).fill(g), [5, 33], 8, cache=cache, ks=ks, vs=vs)
    cache.close()


def test_weight_of_long_chunks_gives_the_same_bits_twice(rx):
    import torch
    g = np.random.default_rng(8)
    lens, new = [3000, 1200], [700, 1200]
    pool = Pool(g, lens, 64, 2, 128).fill(g)
    start = _starts(new)
    q = dev(_bits(g, (start[-1], 8, 128)))
    pages = pool.pages(rx)
    lse = rx.attend_pages(q, pages, _int(start), _int(lens), lse=True)[1]
    one, two = (rx.weigh_pages(q, lse, pages, _int(start), _int(lens), decay=0.5, out=torch.zeros_like(pages.weight)) for _ in range(2))
    assert torch.equal(one, two)
    for b in range(2):   # every row's weights sum to one: a stream's to rows x heads of the group
        got = (one.view(-1, 2)[pool.rows(b)].double() - 0.5 * pages.weight.view(-1, 2)[pool.rows(b)].double()).sum(0)
        np.testing.assert_allclose(got.cpu().numpy(), new[b] * 4, rtol=1e-4)


def test_weight_of_a_prefix_that_streams_share(rx):
    """A call for each stream: those without new tokens leave the shared pages alone."""
    import torch
    g = np.random.default_rng(17)
    Hq, Hkv, D, page = 8, 2, 128, 32
    pool = Pool(g, [200, 150], page, Hkv, D).fill(g)
    pool.table[1, :2] = pool.table[0, :2]                    # 64 places
    pool.w[:] = 0
    new = [20, 33]
    q = _bits(g, (sum(new), Hq, D))
    pages, ln = pool.pages(rx), _int(pool.lens)
    lse = rx.attend_pages(dev(q), pages, _int([0, 20, 53]), ln, lse=True)[1]
    for start in ([0, 20, 20], [20, 20, 53]):
        rx.weigh_pages(dev(q), lse, pages, _int(start), ln)
    got = pages.weight.cpu().numpy().reshape(pool.w.shape)
    want, e = np.zeros(pool.w.shape), lse.double().cpu().numpy()
    rel = 0.0
    for b, s in enumerate((slice(0, 20), slice(20, 53))):
        r = pool.rows(b)
        k = f64(pool.k[r])
        want[r] += OP.gather(f64(q[s]), e[s], k, np.ones(len(r), bool), 0)
        reach = np.max(np.abs(k).sum(-1)) * np.max(np.abs(f64(q[s]))) / np.sqrt(D)
        rel = max(rel, _err_s(D, reach) + 2.0 ** -22 * (np.max(np.abs(e[s])) + reach) + 2.0 ** -20)
    assert np.all(np.abs(got - want) <= (rel + 2.0 ** -23) * want)


@pytest.mark.parametrize("what", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 256), (8, 2, 128), (4, 4, 64), (128, 1, 64)])
@pytest.mark.parametrize("new,lens", [
    ([1, 1, 1, 1], [130, 40, 77, 300]),           # decoding streams side by side
    ([40, 9, 33, 150], [90, 20, 33, 400]),
    ([300, 3, 260], [500, 200, 700]),             # blocks of keys that several CTAs share
])
def test_weight_is_of_the_streams_own_rows(rx, what, Hq, Hkv, D, new, lens):
    """Queries of the next stream and of tokens in no stream that are not finite:
    the other streams' weights are bit for bit as without them."""
    import torch
    g = np.random.default_rng([D, new[0]])
    pool = Pool(g, lens, 32, Hkv, D).fill(g)
    start = _starts(new) + 2
    N = start[-1] + 5
    q = _bits(g, (N, Hq, D))
    bad = q.copy()
    value = W.to_bf16_bits(np.array([what], np.float32))[0]
    for rows in (slice(0, 2), slice(start[1], start[2]), slice(start[-1], N)):
        bad[rows, :, 3] = value
    got = []
    for bits in (q, bad):
        pages = pool.pages(rx)
        args = (pages, _int(start), _int(lens))
        _, lse = rx.attend_pages(dev(bits), *args, lse=torch.zeros((N, Hq), device="cuda"))
        rx.weigh_pages(dev(bits), lse, *args, decay=0.5)
        got.append((pages.weight.cpu().numpy().reshape(pool.w.shape), lse.cpu().numpy()))
    for b in range(len(new)):
        if b == 1:
            continue
        np.testing.assert_array_equal(got[1][1][start[b]:start[b + 1]], got[0][1][start[b]:start[b + 1]])
        assert np.all(np.isfinite(got[0][0][pool.rows(b)]))
        np.testing.assert_array_equal(got[1][0][pool.rows(b)], got[0][0][pool.rows(b)])


@pytest.mark.parametrize("what", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 256), (8, 2, 128), (4, 4, 64)])
def test_weight_is_of_the_rows_that_see_the_key(rx, what, Hq, Hkv, D):
    """A chunk's token 10 whose query is not finite, its lse NaN or what the
    attention makes of it: keys behind token 10, which it does not see, weigh bit
    for bit what they weigh without it.  With lse -infinity it weighs nothing
    anywhere."""
    import torch
    g = np.random.default_rng(D)
    n, held, t = 200, 150, 10
    pool = Pool(g, [held + n], 16, Hkv, D).fill(g)
    q = _bits(g, (n, Hq, D))
    bad = q.copy()
    bad[t, :, 5] = W.to_bf16_bits(np.array([what], np.float32))[0]
    pages = pool.pages(rx)
    args = (pages, _int([0, n]), _int([held + n]))
    def weigh(bits, lse):
        return rx.weigh_pages(dev(bits), lse, *args, decay=0.0, out=torch.zeros_like(pages.weight)).cpu().numpy().reshape(pool.w.shape)
    lse = rx.attend_pages(dev(q), *args, lse=True)[1]
    lse_bad = rx.attend_pages(dev(bad), *args, lse=True)[1]
    lse_nan, lse_low = lse.clone(), lse.clone()
    lse_nan[t], lse_low[t] = float("nan"), -3.2e38
    clean = weigh(q, lse)
    hidden = pool.rows(0)[held + t + 1:]
    assert np.all(np.isfinite(clean[hidden]))
    for e in (lse_bad, lse_nan, lse_low):
        np.testing.assert_array_equal(weigh(bad, e)[hidden], clean[hidden])
        np.testing.assert_array_equal(weigh(q, e)[hidden], clean[hidden])
    assert np.all(np.isnan(weigh(q, lse_nan)[pool.rows(0)[:held + t + 1]]))
    off = lse.clone()
    off[t] = -float("inf")
    np.testing.assert_array_equal(weigh(bad, off), weigh(q, off))
    assert np.all(np.isfinite(weigh(bad, off)[pool.rows(0)]))


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 256), (8, 2, 128), (2, 2, 64)])
@pytest.mark.parametrize("new,lens", [([1, 1, 1], [130, 40, 77]), ([40, 9, 150], [90, 20, 400])])
def test_weight_of_a_key_that_no_row_can_weigh(rx, Hq, Hkv, D, new, lens):
    """An infinite key whose scores are all -infinity in its stream, and would be
    +infinity in the others: it gathers nothing, and the lse stays finite."""
    g = np.random.default_rng([D, new[0]])
    pool = Pool(g, lens, 32, Hkv, D).fill(g)
    start = _starts(new) + 1
    N = start[-1] + 1
    q = np.abs(f64(_bits(g, (N, Hq, D)))) + 1
    q[start[0]:start[1], :, 5] *= -1
    q = W.to_bf16_bits(q.astype(np.float32))
    pool.k[pool.rows(0)[17], :, 5] = W.to_bf16_bits(np.array([np.inf], np.float32))[0]
    pages = pool.pages(rx)
    args = (pages, _int(start), _int(lens))
    _, lse = rx.attend_pages(dev(q), *args, lse=True)
    rx.weigh_pages(dev(q), lse, *args, decay=0.5)
    got = pages.weight.cpu().numpy().reshape(pool.w.shape)
    assert np.all(np.isfinite(lse[1:N - 1].cpu().numpy()))
    np.testing.assert_array_equal(got[pool.rows(0)[17]], np.float32(0.5) * pool.w[pool.rows(0)[17]])
    assert all(np.all(np.isfinite(got[pool.rows(b)])) for b in range(len(new)))


# ---------------------------------------------------------------- eviction
def _evict_case(rx, pool, sink, recent, budget, copy, alias=False, table_to=None):
    import torch
    pages = pool.pages(rx)
    B, ln = len(pool.lens), _int(pool.lens)
    to = None
    tab = pool.table
    if copy:
        counts = [-(-min(n, budget) // pool.page) for n in pool.lens]
        tab = np.full((B, max(1, max(counts))), -1, np.int64)
        free = list(pool.free)
        for b, c in enumerate(counts):
            tab[b, :c] = [free.pop() for _ in range(c)]
        to = _int(tab)
    new_len, over = ln if alias else _int([-9] * B), _int([0])
    kept = rx.evict_pages(pages, ln, budget, sink=sink, recent=recent, to=to, new_len=new_len, overflow=over)
    want = [pool.k.copy(), pool.v.copy(), pool.w.copy()]
    want_kept = np.full((B, pool.Hkv, budget), -1)
    flagged = 0
    for b, n in enumerate(pool.lens):
        for h in range(pool.Hkv):
            names = np.array([0 <= pool.table[b][j // pool.page] < pool.n_pages for j in range(n)], bool)
            src = np.where(names, pool.rows(b), 0)
            keep = OP.keep(np.where(names, pool.w[src, h], np.nan), sink, recent, budget)
            want_kept[b, h, :len(keep)] = keep
            for i, j in enumerate(keep):
                d = tab[b][i // pool.page]
                if not copy and i == j:
                    continue
                if not names[j] or not 0 <= d < pool.n_pages:
                    flagged = 1
                    continue
                for new, old in zip(want, (pool.k, pool.v, pool.w)):
                    new[d * pool.page + i % pool.page, h] = old[src[j], h]
    np.testing.assert_array_equal(kept.cpu().numpy(), want_kept)
    _same(pages.k, want[0])
    _same(pages.v, want[1])
    np.testing.assert_array_equal(pages.weight.cpu().numpy().reshape(want[2].shape), want[2])
    assert new_len.tolist() == [min(n, budget) for n in pool.lens] and over.item() == flagged


@pytest.mark.parametrize("Hkv,D,page", [(1, 256, 64), (3, 128, 16), (2, 64, 256)])
@pytest.mark.parametrize("sink,recent,budget", [(0, 0, 1), (0, 0, 40), (4, 10, 64), (3, 0, 33), (0, 64, 64), (2, 60, 63), (1, 5, 129)])
@pytest.mark.parametrize("copy", [False, True])
def test_eviction(rx, Hkv, D, page, sink, recent, budget, copy):
    g = np.random.default_rng(Hkv + budget)
    pool = Pool(g, [0, 1, budget, budget + 1, 65, 130, 400], page, Hkv, D, spare=60).fill(g)
    _evict_case(rx, pool, sink, recent, budget, copy, alias=not copy)


@pytest.mark.parametrize("copy", [False, True])
def test_eviction_of_equal_negative_and_odd_weights(rx, copy):
    g = np.random.default_rng(4)
    pool = Pool(g, [300] * 6, 32, 2, 64, spare=40).fill(g)
    r = [pool.rows(b) for b in range(6)]
    pool.w[r[0]] = 1.0                                             # all equal: the earliest stay
    pool.w[r[1]] = g.choice([0.0, -0.0, 1.0], (300, 2))            # zeros of both signs are equal
    pool.w[r[2]] = g.choice([np.nan, np.inf, -np.inf, 3.0, -3.0, 1e-42], (300, 2))
    pool.w[r[3]] = np.nan
    pool.w[r[4]] = -g.random((300, 2), dtype=np.float32)
    pool.w[r[5]] = 2.0 ** -149 * g.integers(0, 5, (300, 2))        # subnormals
    _evict_case(rx, pool, 3, 7, 100, copy)


def test_eviction_of_long_streams(rx):
    """More candidates than the selection keeps at hand, many equal."""
    g = np.random.default_rng(9)
    pool = Pool(g, [30000, 24600], 256, 1, 64, spare=250).fill(g)
    r = pool.rows(1)
    pool.w[r] = g.integers(0, 4, (len(r), 1)).astype(np.float32)
    for copy in (False, True):
        _evict_case(rx, pool, 4, 1000, 20000, copy)


@pytest.mark.parametrize("copy", [False, True])
def test_eviction_with_pages_that_are_not_named(rx, copy):
    g = np.random.default_rng(10)
    pool = Pool(g, [100, 100, 100], 16, 2, 64, spare=40).fill(g)
    pool.table[0, 2] = -1            # its keys rank last and are not missed
    pool.table[1, 0] = pool.n_pages  # sinks that are kept all the same
    _evict_case(rx, pool, 2, 5, 64, copy)


@pytest.mark.parametrize("copy", [False, True])
def test_eviction_reports_every_kept_key_without_a_page(rx, copy):
    """A kept key in a page that is not named sets the flag whether it would move
    or stay: a sink, a key of a stream that is short enough to keep all.  A key
    that goes anyway does not."""
    import torch
    g = np.random.default_rng(16)
    budget, sink, recent, page = 64, 20, 5, 16

    def flag(lens, hole, entry=-1):
        pool = Pool(g, lens, page, 2, 64, spare=20).fill(g)
        pool.w[:] = np.where(np.isnan(pool.w), pool.w, 1.0)            # equal: the earliest stay
        if hole is not None:
            pool.table[hole] = entry
        to, tab = None, pool.table
        if copy:
            tab = np.array([[pool.free[5 * b + i] for i in range(4)] for b in range(len(lens))])
            to = _int(tab)
        over, new_len = _int([0]), _int([-1] * len(lens))
        pages = pool.pages(rx)
        kept = rx.evict_pages(pages, _int(lens), budget, sink=sink, recent=recent, to=to, new_len=new_len, overflow=over)
        assert torch.equal(kept, rx.evict_pages(pool.pages(rx), _int(lens), budget, sink=sink, recent=recent, to=to))
        assert new_len.tolist() == [min(n, budget) for n in lens]
        return over.item()

    assert flag([64, 100], None) == 0 and flag([0, 1], None) == 0
    assert flag([30, 3], (0, 1)) == 1                       # short streams keep all where it is
    assert flag([3, 30], (1, 0), 10 ** 6) == 1
    assert flag([64, 3], (0, 3)) == 1                       # as many keys as the budget
    assert flag([100, 40], (0, 0)) == 1                     # sinks, and weights that stay in front
    assert flag([40, 200], (1, 6)) == 0                     # keys 96 to 111 go
    assert flag([40, 3], (0, 3)) == 0                       # no key lies there


# ------------------------------------------------------------ run together
def test_a_captured_step_of_all_four(rx):
    """Two layers; each step rotates and stores a step's tokens, attends over
    the store and the pages, gathers weight and, when streams have outgrown the
    budget, evicts, all in one captured graph that is replayed while lengths
    grow and fall on the device.  Followed step by step in 64 bits from the
    kernels' own bf16 keys."""
    import torch
    g = np.random.default_rng(21)
    L, Hq, Hkv, D, page, budget, sink, recent, T = 2, 8, 2, 64, 16, 40, 2, 6, 3
    B, cap = 3, 4
    cache, ks, vs = _store(rx, g, Hq, Hkv, D, 20, 2, 30, 3, L=L)
    n_pages = B * cap
    kp, vp = (torch.full((L, n_pages, page, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w = torch.full((L, n_pages, page, Hkv), float("nan"), device="cuda")
    table = _int(g.permutation(n_pages).reshape(B, cap))
    held = _int([0, 30, 38])
    for b in range(B):                                    # what the streams hold before the first step
        for j in range(held[b].item()):
            at = table[b, j // page].item(), j % page
            for layer in range(L):
                for pool in (kp, vp):
                    pool[layer, at[0], at[1]] = torch.from_numpy(g.standard_normal((Hkv, D), dtype=np.float32)).cuda().to(torch.bfloat16)
                w[layer, at[0], at[1]] = 0.1
    now = torch.empty_like(held)
    new = [3, 1, 2]
    start = _int(_starts(new))
    N = sum(new)
    x = torch.empty((L, N, (Hq + 2 * Hkv) * D), dtype=torch.bfloat16, device="cuda")
    pos = torch.empty((1, N), dtype=torch.int32, device="cuda")
    freq = (100.0 ** -(np.arange(D // 2) / (D // 2))).astype(np.float32)
    qw = torch.from_numpy(1 + 0.1 * g.standard_normal(D, dtype=np.float32)).cuda()
    heads = rx.Heads(Hq, Hkv, D, torch.from_numpy(freq).cuda(), (), qw, qw)
    outs = [torch.empty((N, Hq, D), dtype=torch.bfloat16, device="cuda") for _ in range(L)]
    qs = [torch.empty_like(outs[0]) for _ in range(L)]
    lses = [torch.empty((N, Hq), device="cuda") for _ in range(L)]
    kept = [torch.empty((B, Hkv, budget), dtype=torch.int32, device="cuda") for _ in range(L)]

    def step():
        for layer in range(L):
            pages = rx.Pages(kp[layer], vp[layer], table, w[layer])
            rx.rotate_heads_paged(x[layer], heads, pos, pages, start, held, q=qs[layer], new_len=now)
            cache.attend_pages(layer, qs[layer], pages, start, now, out=outs[layer], lse=lses[layer])
            rx.weigh_pages(qs[layer], lses[layer], pages, start, now, decay=0.9)
            rx.evict_pages(pages, now, budget, sink=sink, recent=recent, kept=kept[layer], new_len=held if layer == L - 1 else None)

    def feed(i):
        x.copy_(torch.from_numpy(np.random.default_rng(100 + i).standard_normal(tuple(x.shape), dtype=np.float32)))
        pos.copy_(torch.arange(N, dtype=torch.int32) + 7 * i)

    saved = [t.clone() for t in (kp, vp, w, held)]
    feed(0)
    step()                                                 # (loads everything before the capture)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, s in zip((kp, vp, w, held), saved):
        t.copy_(s)
    tab, st = table.cpu().numpy(), _starts(new)
    rows = lambda b, n: [tab[b][j // page] * page + j % page for j in range(n)]
    flat = lambda t, layer: t[layer].reshape(n_pages * page, Hkv, -1)
    lens = held.tolist()
    for i in range(8):
        feed(i)
        before = [[host64(flat(p, layer)) for p in (kp, vp)] + [flat(w, layer).double().cpu().numpy()[..., 0]] for layer in range(L)]
        graph.replay()
        torch.cuda.synchronize()
        after = [min(n + m, cap * page) for n, m in zip(lens, new)]
        for layer in range(L):
            y = host64(x[layer]).reshape(N, Hq + 2 * Hkv, D)
            qw64 = qw.double().cpu().numpy()
            yq, tq, yk, tk = _rotated(y, Hq, Hkv, qw64, qw64, 1e-6, pos.cpu().numpy(), freq, (D // 2,), False)
            q = host64(qs[layer])
            assert np.all(np.abs(q - yq) <= tq)
            _, kd, vd = (host64(t) for t in rx.rotate_heads(x[layer], heads, pos))
            assert np.all(np.abs(kd - yk) <= tk)
            kb, vb, wb = before[layer]
            e = lses[layer].double().cpu().numpy()
            k_now, v_now, w_now = host64(flat(kp, layer)), host64(flat(vp, layer)), flat(w, layer).double().cpu().numpy()[..., 0]
            for b in range(B):
                s = slice(st[b], st[b] + new[b])
                at = rows(b, after[b])
                k = np.concatenate([kb[at[:lens[b]]], kd[s]])
                v = np.concatenate([vb[at[:lens[b]]], vd[s]])
                ref = OP.attend(q[s], k, v, np.ones(after[b], bool), 0, ks[layer], vs[layer])
                _check_attention(host64(outs[layer])[s], e[s], *ref)
                old = 0.9 * np.concatenate([wb[at[:lens[b]]], np.zeros((new[b], Hkv))])
                gathered = OP.gather(q[s], e[s], k, np.ones(after[b], bool), 0)
                keep = kept[layer][b].cpu().numpy()
                n = min(after[b], budget)
                for h in range(Hkv):
                    kh = keep[h][:n]
                    assert np.all(keep[h][n:] == -1) and np.all(np.diff(kh) > 0)
                    full = old[:, h] + gathered[:, h]
                    # Weights within their tolerance of the cut may fall on either side; the others may not.
                    np.testing.assert_allclose(w_now[at[:n], h], full[kh], rtol=1e-4)
                    np.testing.assert_array_equal(k_now[at[:n], h], k[kh, h])
                    np.testing.assert_array_equal(v_now[at[:n], h], v[kh, h])
                    if after[b] > budget:
                        gone = np.setdiff1d(np.arange(after[b]), kh)
                        middle = kh[(kh >= sink) & (kh < after[b] - recent)]
                        assert full[middle].min() >= full[gone].max() * (1 - 1e-4)
                        assert np.all(gone >= sink) and np.all(gone < after[b] - recent)
        lens = [min(n, budget) for n in after]
        assert held.tolist() == lens and now.tolist() == after
    assert lens == [27, 38, 40] or max(lens) == budget
    assert cache.check_device_error() == 0
    cache.close()


def test_two_captured_calls_of_one_cache_replayed_side_by_side(rx):
    """Each call has a workspace of its own: graphs on two streams do not meet."""
    import torch
    g = np.random.default_rng(22)
    Hq, Hkv, D = 8, 1, 256
    cache, ks, vs = _store(rx, g, Hq, Hkv, D, 64, 2, 64, 2)
    cases = []
    for lens in ([5000], [3000, 2000]):
        pool = Pool(g, lens, 64, Hkv, D).fill(g)
        n = len(lens)
        args = (dev(_bits(g, (n, Hq, D))), pool.pages(rx), _int(range(n + 1)), _int(lens))
        ref = cache.attend_pages(0, *args, lse=True)
        out, lse = torch.zeros_like(ref[0]), torch.zeros_like(ref[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(10):
                cache.attend_pages(0, *args, out=out, lse=lse)
        cases.append((graph, out, lse, ref, torch.cuda.Stream(), args))
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, *_, s, _ in cases:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for _, out, lse, ref, *_ in cases:
            assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
            out.zero_()
            lse.zero_()
    cache.close()


def test_calls_of_one_cache_side_by_side_beside_pushes(rx):
    """A ring with a spare slot; two calls on streams of their own, and a push that
    publishes between them while other work holds SMs, so that some of the first
    call's CTAs start after all that: every call's rows are those of one window, the
    one before the push or the one after it."""
    import torch
    g = np.random.default_rng(31)
    Hq, Hkv, D, N, F, steps = 8, 1, 256, 3, 128, 6
    frames = [tuple(dev(_bits(g, (1, F, Hkv, D))) for _ in range(2)) for _ in range(steps + 1)]
    caches = [rx.Cache(1, Hq, Hkv, D, 0, N, F, 1, spare_slot=1) for _ in range(2)]
    calls = []
    for lens, new in (([6000] * 8, [2048] * 8), ([2500, 30], [1, 1])):   # the first takes some 0.5 ms
        pool = Pool(g, lens, 64, Hkv, D).fill(g)
        calls.append((dev(_bits(g, (sum(new), Hq, D))), pool.pages(rx), _int(_starts(new)), _int(lens)))
    refs = []                                       # by window, one call after the other
    for f in frames:
        caches[0].push_frame(*f)
        refs.append([caches[0].attend_pages(0, *c, lse=True) for c in calls])
    # 64 CTAs for 0.8 ms.
    V = 1 << 25
    p, draft, none, r = torch.rand(8, 1, V, device="cuda"), _int(np.zeros((8, 0))), torch.rand(8, 0, device="cuda"), torch.rand(8, device="cuda")
    caches[1].push_frame(*frames[0])
    streams = [torch.cuda.Stream(priority=p) for p in (0, -1, -1, 0)]   # the push gets its places before the first call's rest
    for s, c in zip(streams, calls + calls):        # (loads everything)
        caches[1].attend_pages(0, *c, stream=s)
    rx.verify_drafts(p, None, draft, none, r, stream=streams[3])
    torch.cuda.synchronize()
    for i in range(steps):
        rx.verify_drafts(p, None, draft, none, r, stream=streams[3])
        one = caches[1].attend_pages(0, *calls[0], lse=True, stream=streams[0])
        caches[1].push_frame_async(*frames[i + 1], streams[2], streams[1])
        streams[1].wait_stream(streams[2])
        two = caches[1].attend_pages(0, *calls[1], lse=True, stream=streams[1])
        torch.cuda.synchronize()
        for call, got in enumerate((one, two)):
            assert any(torch.equal(got[0], refs[w][call][0]) and torch.equal(got[1], refs[w][call][1]) for w in (i, i + 1)), (i, call)
    assert caches[1].get_state()[2] == steps + 1
    for c in caches:
        assert c.check_device_error() == 0
        c.close()


def test_two_captured_calls_of_a_cache_with_a_spare_slot(rx):
    """Graphs of one cache replayed side by side follow its window, pushes between
    the replays."""
    import torch
    g = np.random.default_rng(32)
    Hq, Hkv, D, F = 8, 2, 128, 64
    cache, _, _ = _store(rx, g, Hq, Hkv, D, 64, 2, F, 1, spare=1)
    cases = []
    for lens in ([3000], [1500, 700]):
        pool = Pool(g, lens, 64, Hkv, D).fill(g)
        n = len(lens)
        args = (dev(_bits(g, (n, Hq, D))), pool.pages(rx), _int(range(n + 1)), _int(lens))
        out, lse = cache.attend_pages(0, *args, lse=True)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(5):
                cache.attend_pages(0, *args, out=out, lse=lse)
        cases.append((graph, out, lse, torch.cuda.Stream(), args))
    for _ in range(5):
        cache.push_frame(*(dev(_bits(g, (1, F, Hkv, D))) for _ in range(2)))
        refs = [cache.attend_pages(0, *c[4], lse=True) for c in cases]
        for _, out, lse, _, _ in cases:
            out.zero_()
            lse.zero_()
        torch.cuda.synchronize()
        for graph, _, _, s, _ in cases:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for (_, out, lse, _, _), ref in zip(cases, refs):
            assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    assert cache.check_device_error() == 0
    cache.close()


def test_calls_on_another_stream(rx):
    """stream= orders a call on that stream, its own outputs allocated there."""
    import torch
    g = np.random.default_rng(23)
    pool = Pool(g, [300, 200], 32, 2, 128).fill(g)
    q = dev(_bits(g, (3, 8, 128)))
    args = (pool.pages(rx), _int([0, 2, 3]), _int([300, 200]))
    ref = rx.attend_pages(q, *args, lse=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(10):
            big = big @ big * 1e-3
        late = torch.empty_like(q).copy_(q)          # written behind the products
    out, lse = rx.attend_pages(late, *args, lse=True, stream=s)
    got = rx.weigh_pages(late, lse, *args, decay=0.0, out=torch.empty_like(args[0].weight), stream=s)
    s.synchronize()
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    want = rx.weigh_pages(q, ref[1], *args, decay=0.0, out=torch.empty_like(args[0].weight))
    r = torch.from_numpy(np.concatenate([pool.rows(0), pool.rows(1)])).cuda()
    assert torch.equal(got.view(-1, 2)[r], want.view(-1, 2)[r])


def test_a_wait_that_runs_out_is_reported(rx):
    import torch
    g = np.random.default_rng(24)
    cache, ks, vs = _store(rx, g, 8, 1, 256, 64, 2, 64, 2)
    pool = Pool(g, [100], 64, 1, 256).fill(g)
    args = (dev(_bits(g, (2, 8, 256))), pool.pages(rx), _int([0, 2]), _int([100]))
    ref = cache.attend_pages(0, *args)
    cache.debug_inject_timeout(16)
    bad = cache.attend_pages(0, *args)
    assert cache.check_device_error() & 8
    assert torch.isnan(bad).any()
    assert torch.equal(cache.attend_pages(0, *args), ref)
    assert cache.check_device_error() == 0
    cache.close()


def test_workspace_too_small_or_cache_of_other_heads_is_refused(rx):
    import torch
    g = np.random.default_rng(25)
    pool = Pool(g, [20], 16, 1, 64).fill(g)
    args = (dev(_bits(g, (1, 2, 64))), pool.pages(rx), _int([0, 1]), _int([20]))
    need = rx.attend_pages_workspace(1, 2, 1, 64)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    rx.attend_pages(*args, workspace=ws)
    with pytest.raises(rx.RxError, match="workspace"):
        rx.attend_pages(*args, workspace=ws[:need - 1])
    assert rx.weigh_pages_workspace(1, 2, 1) == 0
    n = 900
    q, lse = dev(_bits(g, (n, 2, 64))), torch.zeros((n, 2), device="cuda")
    need = rx.weigh_pages_workspace(n, 2, 1)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    late = (q, lse, args[1], _int([0, n]), _int([20]))
    rx.weigh_pages(*late, workspace=ws)
    with pytest.raises(rx.RxError, match="workspace"):
        rx.weigh_pages(*late, workspace=ws[:need - 1])
    cache = rx.Cache(1, 4, 1, 64, 0, 1, 1, 1)
    with pytest.raises(rx.RxError, match="heads"):
        cache.attend_pages(0, *args)
    with pytest.raises(rx.RxError, match="layer"):
        cache.attend_pages(1, *args)
    cache.close()


def test_empty_calls(rx):
    import torch
    g = np.random.default_rng(26)
    pool = Pool(g, [20], 16, 1, 64).fill(g)
    pages = pool.pages(rx)
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert rx.attend_pages(none, pages, _int([0, 0]), _int([20])).shape == (0, 2, 64)
    rx.weigh_pages(none, torch.empty((0, 2), device="cuda"), pages, _int([0, 0]), _int([20]))
    heads = rx.Heads(2, 1, 64, torch.ones(32, device="cuda"))
    new_len = _int([-1])
    x, pos = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"), _int([])
    assert rx.rotate_heads_paged(x, heads, pos, pages, _int([0, 0]), _int([20]), new_len=new_len).shape == (0, 2, 64)
    assert new_len.tolist() == [20] and rx.rotate_heads(x, heads, pos)[1].shape == (0, 1, 64)
    np.testing.assert_array_equal(pages.weight.cpu().numpy().reshape(pool.w.shape), pool.w)
