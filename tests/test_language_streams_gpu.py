"""Language streams over 8-bit tails: append, attention, verification of
drafts, against the fp64 oracle, and the three run together.

Tolerances of the attention.  A weight alpha_j enters its product with V as at
most one rounding to bf16 (2^-8 relative), the output is rounded once to bf16
(2^-8 of its value), and the fp32 steps (scores, exponentials, sums, merges)
move a weight by less than 2^-12 of itself at these sizes: a score is a sum of
D <= 256 products with |s| below 40, off by at most 40 * 256 * 2^-24 in the
worst case.  So |got - ref| <= (2^-8 + 2^-11) * spread + 2^-8 * |ref| with
spread = sum_j alpha_j |v_j|, plus 1e-30 for zeros.
"""
import numpy as np
import pytest

from oracle import streams as OS
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


def _codes(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().view(torch.float8_e4m3fn)


def _u8(t):
    import torch
    return t.view(torch.uint8).cpu().numpy()


def _tails(g, B, cap, Hkv, D):
    """Quantised random tails: codes, exponent bytes and the values they stand for."""
    f = W.bf16_bits_to_f64
    out = []
    for _ in range(2):
        codes, byte = OS.quantise(f(_bits(g, (B, cap, Hkv, D))))
        out += [codes, byte]
    return out   # kc, ke, vc, ve


# ------------------------------------------------------------------ append
def _append_case(rx, xk, xv, cap, lens, new=None, T_none=False):
    """Append bf16 bits xk, xv [B][T][Hkv][D] and compare every byte of the
    tails, places that nothing was written to among them."""
    import torch
    B, T, Hkv, D = xk.shape
    kt = torch.full((B, cap, Hkv, D), 0x5A, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    vt = torch.full((B, cap, Hkv, D), 0x33, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    ke = torch.full((B, cap, Hkv), 7, dtype=torch.uint8, device="cuda")
    ve = torch.full((B, cap, Hkv), 9, dtype=torch.uint8, device="cuda")
    nl, ov = _int([-5] * B), _int([0])
    tl = _int(lens)
    rx.tail_append_quant(kt, vt, ke, ve, tl, dev(xk), dev(xv), n_new=None if new is None else _int(new), new_len=nl,
                         overflow=ov)
    torch.cuda.synchronize()
    n = [T] * B if new is None else [min(max(x, 0), T) for x in new]
    over = 0
    for got_c, got_e, x, fill, fe in ((kt, ke, xk, 0x5A, 7), (vt, ve, xv, 0x33, 9)):
        want_c, want_e = np.full((B, cap, Hkv, D), fill, np.uint8), np.full((B, cap, Hkv), fe, np.uint8)
        codes, byte = OS.quantise(W.bf16_bits_to_f64(x))
        for b in range(B):
            if not 0 <= lens[b] <= cap:
                over |= n[b] > 0
                continue
            m = min(n[b], cap - lens[b])
            over |= m < n[b]
            want_c[b, lens[b]:lens[b] + m] = codes[b, :m]
            want_e[b, lens[b]:lens[b] + m] = byte[b, :m]
        np.testing.assert_array_equal(got_e.cpu().numpy(), want_e)
        np.testing.assert_array_equal(_u8(got_c), want_c)
    want_len = [min(ln + k, cap) if 0 <= ln <= cap else ln for ln, k in zip(lens, n)]
    assert nl.tolist() == want_len
    assert tl.tolist() == list(lens)
    assert ov.item() == int(over)


@pytest.mark.parametrize("B,T,Hkv,D,cap,lens,new", [
    (1, 1, 1, 64, 1, [0], None),
    (3, 1, 1, 256, 32, [0, 31, 32], None),                 # the last one is full
    (5, 4, 2, 128, 9, [0, 3, 6, 9, 7], [4, 0, 4, 1, 2]),   # one overflows in part
    (4, 7, 3, 64, 40, [-1, 41, 5, 0], [7, 7, 99, -3]),     # lengths and counts out of range
    (2, 33, 8, 256, 50, [1, 17], [33, 32]),
    (9, 5, 1, 128, 21, [0, 1, 2, 3, 4, 5, 6, 7, 8], [5, 4, 3, 2, 1, 0, 1, 2, 3]),
])
def test_append_stores_codes_and_exponents(rx, B, T, Hkv, D, cap, lens, new):
    g = np.random.default_rng(B * 100 + T)
    _append_case(rx, _bits(g, (B, T, Hkv, D)), _bits(g, (B, T, Hkv, D), 30.0), cap, lens, new)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_over_the_whole_range_of_bf16(rx, D):
    """Vectors of every magnitude, ties, zeros of both signs, subnormals, the
    largest value, infinities and NaN."""
    g = np.random.default_rng(D)
    x = _bits(g, (2, 254, 1, D))
    e = np.arange(254, dtype=np.uint32)[None, :, None, None]          # exponent field of each vector's largest
    drop = g.integers(0, 20, x.shape).astype(np.uint32)
    x = ((x & 0x807F) | (np.maximum(e.astype(np.int64) - drop, 0) << 7).astype(np.uint32)).astype(np.uint16)
    x[0, :, 0, 3] = (np.arange(254) << 7) | g.integers(90, 102, 254)   # tops around 1.75 * 2^k
    x[1, 0] = 0
    x[1, 1] = 0x8000
    x[1, 2, 0, 5] = 0x7F80      # inf
    x[1, 3, 0, D - 1] = 0xFF80  # -inf
    x[1, 4, 0, 0] = 0x7FC0      # NaN
    x[1, 5, 0, 1] = 0x7F7F      # the largest bf16
    x[1, 6] = 1                 # the smallest subnormal
    _append_case(rx, x, x[::-1].copy(), 260, [0, 3])


def test_append_follows_lengths_on_the_device_in_a_graph(rx):
    import torch
    g = np.random.default_rng(3)
    B, T, Hkv, D, cap = 2, 2, 1, 64, 9
    xk, xv = _bits(g, (B, T, Hkv, D)), _bits(g, (B, T, Hkv, D))
    kt = torch.zeros((B, cap, Hkv, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    vt, ke = kt.clone(), torch.zeros((B, cap, Hkv), dtype=torch.uint8, device="cuda")
    ve, tl, nl = ke.clone(), _int([0, 3]), _int([0, 0])
    dk, dv = dev(xk), dev(xv)
    rx.tail_append_quant(kt, vt, ke, ve, tl, dk, dv, new_len=nl)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rx.tail_append_quant(kt, vt, ke, ve, tl, dk, dv, new_len=nl)
        tl.copy_(nl)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert tl.tolist() == [4, 7]
    codes, byte = OS.quantise(W.bf16_bits_to_f64(xk))
    got = _u8(kt)
    np.testing.assert_array_equal(got[0, 0:4], np.concatenate([codes[0], codes[0]]))
    np.testing.assert_array_equal(got[1, 3:7], np.concatenate([codes[1], codes[1]]))
    np.testing.assert_array_equal(ke.cpu().numpy()[1, 3:7], np.concatenate([byte[1], byte[1]]))


# --------------------------------------------------------------- attention
class Store:
    """A one-layer store and its keys in oracle form."""

    def __init__(self, rx, g, Hq, Hkv, D, P, N, F, cap, req, pushes, spare=0, layers=1):
        f = W.bf16_bits_to_f64
        self.Hq, self.Hkv, self.D, self.cap = Hq, Hkv, D, cap
        self.cache = rx.Cache(layers, Hq, Hkv, D, P, N, F, 4, cap, req, spare)
        pk, pv = _bits(g, (layers, P, Hkv, D)), _bits(g, (layers, P, Hkv, D))
        self.cache.pin_prefix(dev(pk), dev(pv))
        fk, fv = [], []
        for _ in range(pushes):
            k, v = _bits(g, (layers, F, Hkv, D)), _bits(g, (layers, F, Hkv, D))
            self.cache.push_frame(dev(k), dev(v))
            fk.append(k)
            fv.append(v)
        self.k = [f(np.concatenate([pk[i]] + [x[i] for x in fk[-N:]])) for i in range(layers)]
        self.v = [f(np.concatenate([pv[i]] + [x[i] for x in fv[-N:]])) for i in range(layers)]


def _check(got, ref, spread):
    bound = (2.0 ** -8 + 2.0 ** -11) * spread + 2.0 ** -8 * np.abs(ref) + 1e-30
    off = np.abs(got - ref)
    assert np.all(np.isfinite(got))
    assert np.all(off <= bound), "worst %.3f of the bound" % np.max(off / bound)


def _attend(rx, st, g, lens, new, T, layer=0, tails=None, garbage=True):
    """Run a batch and check every row; rows past n_new keep their bits."""
    import torch
    B = len(lens)
    kc, ke, vc, ve = tails if tails is not None else _tails(g, B, st.cap, st.Hkv, st.D)
    q = _bits(g, (B, T, st.Hq, st.D))
    kd, vd, ked, ved = kc.copy(), vc.copy(), ke.copy(), ve.copy()
    if garbage:   # whatever lies behind a tail's end: NaN codes and any exponent
        for b in range(B):
            kd[b, lens[b]:], vd[b, lens[b]:] = 0x7F, 0xFF
            ked[b, lens[b]:] = g.integers(0, 256, ked[b, lens[b]:].shape)
            ved[b, lens[b]:] = g.integers(0, 256, ved[b, lens[b]:].shape)
    out = torch.full((B, T, st.Hq, st.D), -3.0, dtype=torch.bfloat16, device="cuda")
    args = (dev(q), _codes(kd), _codes(vd), torch.from_numpy(ked).cuda(), torch.from_numpy(ved).cuda(), _int(lens))
    res = st.cache.attend_streams_quant(layer, *args, n_new=None if new is None else _int(new), out=out)
    assert res is out
    got = host64(out)
    again = st.cache.attend_streams_quant(layer, *args, n_new=None if new is None else _int(new), out=out.clone())
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))   # the same bits every time
    for b in range(B):
        n = T if new is None else min(max(new[b], 0), T)
        k, v = OS.dequantise(kc[b, :lens[b]], ke[b, :lens[b]]), OS.dequantise(vc[b, :lens[b]], ve[b, :lens[b]])
        ref, spread = OS.stream_attention(W.bf16_bits_to_f64(q[b, :n]), st.k[layer], st.v[layer], k, v)
        _check(got[b, :n], ref, spread)
        assert np.all(got[b, n:] == -3.0)
    assert st.cache.check_device_error() == 0
    return args, out


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 256), (8, 2, 128), (4, 4, 64), (2, 1, 64), (32, 1, 128), (128, 1, 64),
                                      (1, 1, 256), (16, 8, 256)])
@pytest.mark.parametrize("T,lens,new", [
    (1, [0, 1, 130], None),
    (3, [3, 64, 129, 300], [3, 1, 2, 0]),
])
def test_attention_head_layouts(rx, Hq, Hkv, D, T, lens, new):
    g = np.random.default_rng(Hq * 1000 + D + T)
    st = Store(rx, g, Hq, Hkv, D, 20, 2, 48, 301, len(lens) * T, pushes=3)
    _attend(rx, st, g, lens, new, T)


@pytest.mark.parametrize("lens", [[31, 32, 33], [63, 64, 65], [127, 128, 129], [255, 256, 257], [511, 512, 513],
                                  [1023, 1025, 1500], [0, 0, 0], [1, 1500, 0]])
@pytest.mark.parametrize("D", [64, 256])
def test_attention_tail_lengths(rx, lens, D):
    g = np.random.default_rng(lens[1] + D)
    st = Store(rx, g, 8, 1, D, 64, 1, 64, 1500, 6, pushes=1)
    _attend(rx, st, g, lens, [1, 2, 1] if lens[0] else None, 2)


@pytest.mark.parametrize("T,Hq,Hkv,D", [(5, 8, 1, 256), (8, 8, 1, 128), (9, 8, 1, 256), (16, 8, 1, 64), (17, 16, 2, 128),
                                        (40, 8, 1, 256), (130, 1, 1, 64)])
def test_attention_drafts_and_prompts_are_causal(rx, T, Hq, Hkv, D):
    """Several query tokens: each sees its own tail up to itself; T * G crosses
    one and several tiles of query rows."""
    g = np.random.default_rng(T)
    st = Store(rx, g, Hq, Hkv, D, 30, 2, 64, 400, 3 * T, pushes=1)
    _attend(rx, st, g, [T, 400, T + 61], [T, T, max(1, T - 3)], T)


def test_attention_prompt_longer_than_its_tail(rx):
    """More query tokens than keys: the first rows see no tail key."""
    g = np.random.default_rng(7)
    st = Store(rx, g, 8, 1, 64, 5, 1, 16, 40, 12, pushes=1)
    _attend(rx, st, g, [2, 0], None, 6)


@pytest.mark.parametrize("P,pushes,spare,F", [(0, 0, 0, 16), (0, 1, 0, 16), (7, 0, 0, 64), (40, 5, 1, 64),
                                              (64, 4, 1, 128), (3, 3, 0, 100)])
def test_attention_store_states(rx, P, pushes, spare, F):
    """No prefix, no frame, a partly and a fully filled window, a spare slot."""
    g = np.random.default_rng(P + pushes)
    st = Store(rx, g, 8, 1, 128, P, 3, F, 70, 8, pushes=pushes, spare=spare)
    _attend(rx, st, g, [0, 1, 70, 33], [1, 1, 2, 2], 2)


def test_attention_second_layer(rx):
    g = np.random.default_rng(17)
    st = Store(rx, g, 8, 1, 256, 64, 8, 256, 32, 16, pushes=8, layers=3)
    _attend(rx, st, g, [0, 2, 4, 6, 8, 10, 12, 14, 16, 18, 20, 22, 24, 26, 28, 30], None, 1, layer=2)


def test_attention_many_streams_of_odd_lengths(rx):
    g = np.random.default_rng(18)
    st = Store(rx, g, 4, 2, 64, 10, 1, 32, 250, 200, pushes=1)
    lens = [int(x) for x in g.integers(0, 251, 67)]
    new = [int(min(max(1, x), y)) for x, y in zip(g.integers(0, 4, 67), np.maximum(lens, 1))]
    _attend(rx, st, g, lens, new, 2)


def test_attention_outliers_far_apart(rx):
    """Scales that differ by many powers of two between neighbouring tokens."""
    g = np.random.default_rng(19)
    st = Store(rx, g, 8, 1, 256, 16, 1, 16, 300, 4, pushes=1)
    f = W.bf16_bits_to_f64
    kx = f(_bits(g, (2, 300, 1, 256)))
    vx = f(_bits(g, (2, 300, 1, 256))) * 2.0 ** g.integers(-30, 30, (2, 300, 1, 1))
    kx *= 2.0 ** g.integers(-6, 1, (2, 300, 1, 1))
    kc, ke = OS.quantise(kx)
    vc, ve = OS.quantise(vx)
    _attend(rx, st, g, [300, 211], [2, 2], 2, tails=(kc, ke, vc, ve))


def test_attention_score_range(rx):
    """Scores that grow along the tail by hundreds: the running maximum moves
    at every tile, and early keys vanish."""
    g = np.random.default_rng(20)
    st = Store(rx, g, 2, 1, 64, 4, 1, 16, 700, 4, pushes=1)
    f = W.bf16_bits_to_f64
    kc, ke = OS.quantise(f(_bits(g, (2, 700, 1, 64))) * np.linspace(0.01, 6, 700)[None, :, None, None])
    vc, ve = OS.quantise(f(_bits(g, (2, 700, 1, 64))))
    _attend(rx, st, g, [700, 650], None, 2, tails=(kc, ke, vc, ve))


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 256), (32, 8, 128), (4, 4, 64)])
@pytest.mark.parametrize("P,pushes,T", [(2, 0, 1), (5, 1, 3), (0, 1, 8)])
def test_attention_weights_are_not_rounded_to_16_bits(rx, Hq, Hkv, D, P, pushes, T):
    """Few keys, so that roundings of the weights do not average out, and a
    bound without a bf16 rounding of them: 2^-11 of a weight for the tails'
    terms, 2^-12 for the fp32 steps, and 2^-8 of the output for its own."""
    import torch
    g = np.random.default_rng(50 + D + P)
    B = 24
    st = Store(rx, g, Hq, Hkv, D, P, 1, 16, 40, B * T, pushes=pushes)
    kc, ke, vc, ve = _tails(g, B, 40, Hkv, D)
    lens = [int(x) for x in g.integers(T, T + 3, B)]
    q = _bits(g, (B, T, Hq, D))
    got = host64(st.cache.attend_streams_quant(0, dev(q), _codes(kc), _codes(vc), torch.from_numpy(ke).cuda(),
                                               torch.from_numpy(ve).cuda(), _int(lens)))
    for b in range(B):
        ref, spread = OS.stream_attention(W.bf16_bits_to_f64(q[b]), st.k[0], st.v[0],
                                          OS.dequantise(kc[b, :lens[b]], ke[b, :lens[b]]),
                                          OS.dequantise(vc[b, :lens[b]], ve[b, :lens[b]]))
        bound = (2.0 ** -11 + 2.0 ** -12) * spread + 2.0 ** -8 * np.abs(ref) + 1e-30
        off = np.abs(got[b] - ref)
        assert np.all(off <= bound), "worst %.3f of the bound" % np.max(off / bound)


@pytest.mark.parametrize("T", [1, 2, 8])
def test_attention_weights_over_a_tail_keep_12_bits(rx, T):
    """Two keys whose values nearly cancel, so that the output's own rounding is
    small beside the weights' errors: three e4m3 terms are within 2^-12 of a
    weight (2^-4 of a remainder each), the fp32 steps at scores below 8 within
    2^-16."""
    import torch
    g = np.random.default_rng(70 + T)
    B, D, f = 120, 64, W.bf16_bits_to_f64
    st = Store(rx, g, 8, 1, D, 0, 1, 16, 8, B * T, pushes=0)
    kc, ke = OS.quantise(f(_bits(g, (B, 8, 1, D))))
    v = np.ones((B, 8, 1, D))
    v[:, 1:] = -2.0 ** g.integers(-3, 4, (B, 7, 1, D)) * (1 + g.integers(0, 8, (B, 7, 1, D)) / 8)   # e4m3 holds them
    vc, ve = OS.quantise(v)
    lens = [T + 1] * B
    q = _bits(g, (B, T, 8, D), 0.5)
    got = host64(st.cache.attend_streams_quant(0, dev(q), _codes(kc), _codes(vc), torch.from_numpy(ke).cuda(),
                                               torch.from_numpy(ve).cuda(), _int(lens)))
    near = 0
    for b in range(B):
        ref, spread = OS.stream_attention(f(q[b]), st.k[0], st.v[0], OS.dequantise(kc[b, :T + 1], ke[b, :T + 1]),
                                          OS.dequantise(vc[b, :T + 1], ve[b, :T + 1]))
        bound = (2.0 ** -12 + 2.0 ** -16) * spread + 2.0 ** -8 * np.abs(ref)
        near += np.sum(np.abs(ref) < 0.02 * spread)
        off = np.abs(got[b] - ref)
        assert np.all(off <= bound), "worst %.3f of the bound" % np.max(off / bound)
    assert near > 300


@pytest.mark.parametrize("T", [1, 4, 8])
@pytest.mark.parametrize("power", [18, 23, 24, 25, 26, 28, 31])
def test_attention_large_scores(rx, T, power):
    """Scores of 2^power (in units of log 2) whose order is plain, and values
    of very different scales: two keys share the top score, every other key is
    at half of it or less, so the output is the mean of their two values."""
    import torch
    g = np.random.default_rng(power)
    D, n, f = 256, 300, W.bf16_bits_to_f64
    st = Store(rx, g, 8, 1, D, 16, 1, 16, n, 2 * T, pushes=1)
    # q . k / sqrt(D) / log 2 = 2^a * 2^b * c * 256 / 16 / log 2 for q = 2^a, k = 2^b c
    a = (power - 4) // 2
    b = power - 4 - a
    q = np.full((2, T, 8, D), 2.0 ** a, np.float32)
    c = g.choice([0.5, 0.25, -1.0], (2, n, 1, 1)) * np.ones(D)
    c[0, [40, 200]] = c[1, [130, 131]] = 1.0
    kc, ke = OS.quantise(c * 2.0 ** b)
    scale = g.integers(-40, 41, (2, 1, 1, 1)) + g.integers(-5, 6, (2, n, 1, 1))
    vc, ve = OS.quantise(f(_bits(g, (2, n, 1, D))) * 2.0 ** scale)
    out = st.cache.attend_streams_quant(0, dev(W.to_bf16_bits(q)), _codes(kc), _codes(vc), torch.from_numpy(ke).cuda(),
                                        torch.from_numpy(ve).cuda(), _int([n, n]))
    got = host64(out)
    for b in range(2):
        ref, spread = OS.stream_attention(q[b].astype(np.float64), st.k[0], st.v[0], OS.dequantise(kc[b], ke[b]),
                                          OS.dequantise(vc[b], ve[b]))
        _check(got[b], ref, spread)


@pytest.mark.parametrize("Hq,Hkv,D", [(6, 3, 128), (14, 7, 64), (320, 320, 64), (40, 20, 256)])
def test_attention_head_counts(rx, Hq, Hkv, D):
    """Head counts that do not divide the GPU's SMs, and more heads than CTAs."""
    g = np.random.default_rng(Hkv)
    st = Store(rx, g, Hq, Hkv, D, 6, 1, 16, 400, 9, pushes=1)
    _attend(rx, st, g, [400, 129, 5], [3, 1, 2], 3)


def test_attention_more_streams_than_threads_of_a_cta(rx):
    g = np.random.default_rng(27)
    st = Store(rx, g, 2, 1, 64, 4, 1, 16, 140, 500, pushes=1)
    lens = [int(x) for x in g.integers(0, 141, 500)]
    _attend(rx, st, g, lens, None, 1)


@pytest.mark.parametrize("D", [64, 256])
def test_attention_few_new_tokens_in_a_wide_batch(rx, D):
    """Streams with one, all and some of 40 query tokens: row tiles without rows."""
    g = np.random.default_rng(28)
    st = Store(rx, g, 8, 1, D, 10, 1, 16, 260, 160, pushes=1)
    _attend(rx, st, g, [260, 40, 133, 1], [1, 40, 17, 0], 40)


@pytest.mark.parametrize("T", [1, 2, 4, 8])
@pytest.mark.parametrize("gap", [6.0, 9.7, 12.5])
def test_attention_many_small_weights_beside_a_large_one(rx, T, gap):
    """One key `gap` nats above 16000 equal ones: together these weigh up to
    40 times as much, or far less; their share must not be rounded away."""
    g = np.random.default_rng(29)
    n, D = 16000, 64
    st = Store(rx, g, 8, 1, D, 0, 1, 16, n, T, pushes=0)
    f = W.bf16_bits_to_f64
    k = np.zeros((1, n, 1, D))
    k[0, 7777] = gap / np.sqrt(D)      # against q = 1: gap nats
    kc, ke = OS.quantise(f(W.to_bf16_bits(k.astype(np.float32))))
    vc, ve = OS.quantise(f(_bits(g, (1, n, 1, D))) + 0.25)
    import torch
    q = np.ones((1, T, 8, D), np.float32)
    out = st.cache.attend_streams_quant(0, dev(W.to_bf16_bits(q)), _codes(kc), _codes(vc), torch.from_numpy(ke).cuda(),
                                        torch.from_numpy(ve).cuda(), _int([n]))
    ref, spread = OS.stream_attention(q[0].astype(np.float64), st.k[0], st.v[0], OS.dequantise(kc[0], ke[0]), OS.dequantise(vc[0], ve[0]))
    _check(host64(out)[0], ref, spread)


@pytest.mark.parametrize("T", [1, 8])
def test_attention_very_many_small_weights_beside_a_large_one(rx, T):
    """One key 16.7 nats above 196607 equal ones, on so many heads that a CTA
    reads all of a head's keys, or half of them, one after the other.  Each of
    these weighs a little less than half of what a weight can be told apart
    by, so all of them are lost beside the large one: of 16384 keys that is
    16384 * e^-16.7 * 2 = 0.0018, of all 0.022, and the bound is 0.0085 (the
    large key's values are 1 or -1, the others' 2)."""
    import torch
    g = np.random.default_rng(42)
    n, D, H = 196608, 64, 152
    st = Store(rx, g, 8 * H, H, D, 0, 1, 16, n, T, pushes=0)
    k = np.zeros((1, D))
    k[0] = 2.0
    k[0, :23] = 2.25                      # against q = 1: (41 * 2 + 23 * 2.25) / 8 = 16.72 nats
    sign = np.where(g.random((1, D)) < 0.5, -1.0, 1.0)
    (kc, ke), (vc, ve), (sc, se) = OS.quantise(k), OS.quantise(sign), OS.quantise(np.full((1, D), 2.0))
    kt = torch.zeros((1, n, H, D), dtype=torch.uint8, device="cuda")
    kx = torch.zeros((1, n, H), dtype=torch.uint8, device="cuda")
    vt = torch.from_numpy(sc).cuda().view(1, 1, 1, D).repeat(1, n, H, 1)
    vx = torch.full((1, n, H), int(se[0]), dtype=torch.uint8, device="cuda")
    kt[0, 7777], kx[0, 7777] = torch.from_numpy(kc).cuda(), int(ke[0])
    vt[0, 7777], vx[0, 7777] = torch.from_numpy(vc).cuda(), int(ve[0])
    q = torch.ones((1, T, 8 * H, D), dtype=torch.bfloat16, device="cuda")
    out = st.cache.attend_streams_quant(0, q, kt.view(torch.float8_e4m3fn), vt.view(torch.float8_e4m3fn), kx, vx, _int([n]))
    got = host64(out)[0]
    for t in range(T):
        others = (n - T + t) * np.exp(-np.sum(OS.dequantise(kc, ke)) / np.sqrt(D))
        ref = (sign[0] + 2.0 * others) / (1 + others)
        spread = (1 + 2.0 * others) / (1 + others)
        for h in range(8 * H):
            _check(got[t, h], ref, spread * np.ones(D))
    assert st.cache.check_device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,D,T", [(8, 1, 256, 1), (32, 2, 64, 8), (16, 2, 128, 1)])
def test_attention_tails_of_several_segments(rx, Hq, Hkv, D, T):
    """More keys of one stream in a CTA's run than are summed under one pair of
    references: 160 streams' worth of the GPU's runs in one, a second stream of
    an odd length behind it, and scores that grow and fall along the tail."""
    import torch
    g = np.random.default_rng(43)
    H, n = 160, 16384 * 2 + 77
    G = Hq // Hkv
    st = Store(rx, g, H * G, H, D, 3, 1, 16, n, 2 * T, pushes=1)
    tails = []
    for scale in (np.sin(np.arange(n) / 9000.0)[None, :, None, None] + 1.5, 1.0):
        codes, byte = OS.quantise((g.standard_normal((2, n, 1, D)) * scale).astype(np.float32).astype(np.float64))
        tails += [codes, byte]
    kc, ke, vc, ve = (np.ascontiguousarray(x) for x in tails)
    lens = [n, 16384 + 130]
    on = lambda x: torch.from_numpy(x).cuda().expand(2, n, H, *x.shape[3:]).contiguous()
    q1 = W.to_bf16_bits(0.3 * g.standard_normal((2, T, 1, G, D), dtype=np.float32))
    q = dev(np.ascontiguousarray(np.broadcast_to(q1, (2, T, H, G, D))).reshape(2, T, H * G, D))
    out = st.cache.attend_streams_quant(0, q, on(kc).view(torch.float8_e4m3fn), on(vc).view(torch.float8_e4m3fn), on(ke),
                                        on(ve), _int(lens))
    got = host64(out).reshape(2, T, H, G, D)
    for b in range(2):
        for h in (0, 1, 80, H - 1):
            ref, spread = OS.stream_attention(W.bf16_bits_to_f64(q1[b, :, 0]), st.k[0][:, h:h + 1], st.v[0][:, h:h + 1],
                                              OS.dequantise(kc[b, :lens[b]], ke[b, :lens[b]]),
                                              OS.dequantise(vc[b, :lens[b]], ve[b, :lens[b]]))
            _check(got[b, :, h], ref, spread)
    assert st.cache.check_device_error() == 0


def test_attention_wait_that_runs_out_is_reported(rx):
    g = np.random.default_rng(31)
    st = Store(rx, g, 8, 1, 64, 16, 1, 16, 200, 4, pushes=1)
    kc, ke, vc, ve = _tails(g, 2, 200, 1, 64)
    import torch
    args = (dev(_bits(g, (2, 2, 8, 64))), _codes(kc), _codes(vc), torch.from_numpy(ke).cuda(), torch.from_numpy(ve).cuda(),
            _int([200, 31]))
    good = st.cache.attend_streams_quant(0, *args)
    st.cache.debug_inject_timeout(1024)
    st.cache.attend_streams_quant(0, *args)
    assert st.cache.check_device_error() == 8
    again = st.cache.attend_streams_quant(0, *args)
    assert st.cache.check_device_error() == 0
    assert torch.equal(good, again)


def test_the_tails_take_one_cta_an_sm_of_workspace(rx):
    """What a cache with language streams holds for the tails' partials: units
    of 64 rows for one CTA an SM and the batch's own rows, (D + 2) fp32 each."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    torch.cuda.synchronize()

    def held(tail_cap):
        free = torch.cuda.mem_get_info()[0]
        c = rx.Cache(1, 8, 1, 256, 64, 1, 64, 4, tail_cap, 16)
        used = free - torch.cuda.mem_get_info()[0]
        c.close()
        return used
    held(32)
    need = (64 * sms + 2 * 16 * 8) * (256 + 2) * 4
    assert held(32) - held(0) <= need + (4 << 20)   # whole pages of 2 MiB


def test_attention_refusals(rx):
    import torch
    g = np.random.default_rng(32)
    st = Store(rx, g, 8, 1, 64, 16, 1, 16, 40, 4, pushes=1)
    kc, ke, vc, ve = _tails(g, 3, 40, 1, 64)
    kt, vt, ke, ve = _codes(kc), _codes(vc), torch.from_numpy(ke).cuda(), torch.from_numpy(ve).cuda()
    q = dev(_bits(g, (3, 1, 8, 64)))
    call = st.cache.attend_streams_quant
    with pytest.raises(rx.RxError) as e:
        call(1, q, kt, vt, ke, ve, _int([1, 2, 3]))                       # layer
    assert e.value.status == -2
    with pytest.raises(rx.RxError) as e:
        call(0, dev(_bits(g, (3, 2, 8, 64))), kt, vt, ke, ve, _int([1, 2, 3]))   # 6 query tokens > max_req = 4
    assert e.value.status == -3
    with pytest.raises(rx.RxError) as e:
        call(0, q, kt, vt, ke, ve, _int([1, 2, 3]), out=q)                # out is q
    assert e.value.status == -1
    with pytest.raises(ValueError, match="tail_len"):
        call(0, q, kt, vt, ke, ve, torch.tensor([1, 2, 3], dtype=torch.int32))   # host memory
    with pytest.raises(TypeError, match="k_tail"):
        call(0, q, kt.view(torch.uint8), vt, ke, ve, _int([1, 2, 3]))
    small = rx.Cache(1, 8, 1, 64, 16, 1, 16, 4)                            # no language streams
    with pytest.raises(rx.RxError) as e:
        small.attend_streams_quant(0, q, kt[:, :0], vt[:, :0], ke[:, :0], ve[:, :0], _int([1, 2, 3]))
    assert e.value.status == -3
    empty = call(0, q[:0], kt[:0], vt[:0], ke[:0], ve[:0], _int([]))
    assert empty.shape == (0, 1, 8, 64)


def test_nan_tokens_reach_only_the_rows_that_see_them(rx):
    import torch
    g = np.random.default_rng(21)
    T, D = 3, 128
    st = Store(rx, g, 8, 1, D, 16, 1, 16, 200, 3 * T, pushes=1)
    kc, ke, vc, ve = _tails(g, 3, 200, 1, D)
    lens = [150, 200, 90]
    ve[0, 148], vc[0, 148] = 255, 0      # seen by query tokens 1 and 2 of stream 0
    ke[1, 199], kc[1, 199] = 255, 0      # seen by query token 2 of stream 1
    q = dev(_bits(g, (3, T, 8, D)))
    out = st.cache.attend_streams_quant(0, q, _codes(kc), _codes(vc), torch.from_numpy(ke).cuda(),
                                        torch.from_numpy(ve).cuda(), _int(lens))
    nan = torch.isnan(out).cpu().numpy()
    want = np.zeros((3, T, 8, D), bool)
    want[0, 1:] = want[1, 2] = True
    np.testing.assert_array_equal(nan, want)


def test_attention_places_beyond_32_bits(rx):
    """The third stream's tail starts past 2^31 bytes."""
    import torch
    g = np.random.default_rng(22)
    cap, D, B = (1 << 22) + 5, 256, 3
    st = Store(rx, g, 8, 1, D, 16, 1, 16, cap, 2 * B, pushes=1)
    kt = torch.full((B, cap, 1, D), 0x7F, dtype=torch.uint8, device="cuda")
    vt = torch.full((B, cap, 1, D), 0xFF, dtype=torch.uint8, device="cuda")
    ke = torch.full((B, cap, 1), 255, dtype=torch.uint8, device="cuda")
    ve = ke.clone()
    kc, kb, vc, vb = _tails(g, B, 400, 1, D)
    lens = [10, 399, 400]
    for b in range(B):
        for t, c in ((kt, kc), (vt, vc), (ke, kb), (ve, vb)):
            t[b, :lens[b]] = torch.from_numpy(c[b, :lens[b]]).cuda()
    q = _bits(g, (B, 2, 8, D))
    out = st.cache.attend_streams_quant(0, dev(q), kt.view(torch.float8_e4m3fn), vt.view(torch.float8_e4m3fn), ke, ve,
                                        _int(lens))
    got = host64(out)
    for b in range(B):
        ref, spread = OS.stream_attention(W.bf16_bits_to_f64(q[b]), st.k[0], st.v[0],
                                          OS.dequantise(kc[b, :lens[b]], kb[b, :lens[b]]),
                                          OS.dequantise(vc[b, :lens[b]], vb[b, :lens[b]]))
        _check(got[b], ref, spread)
    # ... and the append writes there.
    xk, xv = _bits(g, (B, 2, 1, D)), _bits(g, (B, 2, 1, D))
    rx.tail_append_quant(kt.view(torch.float8_e4m3fn), vt.view(torch.float8_e4m3fn), ke, ve,
                         _int([cap - 2, cap - 2, cap - 2]), dev(xk), dev(xv))
    codes, byte = OS.quantise(W.bf16_bits_to_f64(xk))
    np.testing.assert_array_equal(kt[2, cap - 2:].cpu().numpy(), codes[2])
    np.testing.assert_array_equal(ke[2, cap - 2:].cpu().numpy(), byte[2])


def test_attention_long_tail(rx):
    """One stream with a tail of 20000 tokens beside short ones."""
    g = np.random.default_rng(23)
    st = Store(rx, g, 8, 1, 64, 64, 1, 64, 20000, 9, pushes=1)
    kc, ke, vc, ve = _tails(g, 1, 20000, 1, 64)
    tails = [np.concatenate([x, x[:, ::-1], x]) for x in (kc, ke, vc, ve)]
    _attend(rx, st, g, [20000, 3, 777], [3, 3, 1], 3, tails=tails)


def test_attention_graph_follows_growing_tails(rx):
    import torch
    g = np.random.default_rng(24)
    B, D, cap = 3, 256, 300
    st = Store(rx, g, 8, 1, D, 16, 2, 64, cap, B, pushes=2)
    kc, ke, vc, ve = _tails(g, B, cap, 1, D)
    q = _bits(g, (B, 1, 8, D))
    out = torch.zeros((B, 1, 8, D), dtype=torch.bfloat16, device="cuda")
    tl = _int([0, 0, 0])
    args = (dev(q), _codes(kc), _codes(vc), torch.from_numpy(ke).cuda(), torch.from_numpy(ve).cuda(), tl)
    st.cache.attend_streams_quant(0, *args, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.cache.attend_streams_quant(0, *args, out=out)
    for lens in ([0, 1, 300], [299, 128, 7], [5, 0, 0]):
        tl.copy_(_int(lens))
        graph.replay()
        got = host64(out)
        for b in range(B):
            ref, spread = OS.stream_attention(W.bf16_bits_to_f64(q[b]), st.k[0], st.v[0],
                                              OS.dequantise(kc[b, :lens[b]], ke[b, :lens[b]]),
                                              OS.dequantise(vc[b, :lens[b]], ve[b, :lens[b]]))
            _check(got[b], ref, spread)


def test_attention_outside_a_capture_is_refused(rx):
    """A call on another stream while one of this cache is being captured: it
    is refused, the capture goes on, and both work once it has ended."""
    import torch
    g = np.random.default_rng(28)
    st = Store(rx, g, 8, 1, 64, 16, 1, 16, 40, 4, pushes=1)
    kc, ke, vc, ve = _tails(g, 2, 40, 1, 64)
    q = dev(_bits(g, (2, 1, 8, 64)))
    args = (q, _codes(kc), _codes(vc), torch.from_numpy(ke).cuda(), torch.from_numpy(ve).cuda(), _int([40, 13]))
    first = st.cache.attend_streams_quant(0, *args)
    outs = [torch.zeros_like(first) for _ in range(3)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.cache.attend_streams_quant(0, *args, out=outs[0])
        with pytest.raises(rx.RxError) as e:
            st.cache.attend_streams_quant(0, *args, out=outs[2], stream=side)
        assert e.value.status == -7
        st.cache.attend_streams_quant(0, *args, out=outs[1])
    graph.replay()
    torch.cuda.synchronize()
    st.cache.attend_streams_quant(0, *args, out=outs[2], stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs)


def test_a_push_within_an_attention_call_changes_none_of_its_rows(rx):
    """Ring with a spare slot: a batch whose query tiles take many waves of CTAs,
    and a push on another stream that publishes its frame in the middle.  All
    rows see the window before the push, or all of them the one after it."""
    import torch
    g = np.random.default_rng(60)
    B, T, Hq, Hkv, D, N, F = 16, 256, 64, 8, 64, 8, 256
    cache = rx.Cache(1, Hq, Hkv, D, 64, N, F, 4, 64, B * T, 1)
    draw = lambda *shape: torch.from_numpy(g.standard_normal(shape, dtype=np.float32)).to(torch.bfloat16).cuda()
    cache.pin_prefix(draw(1, 64, Hkv, D), draw(1, 64, Hkv, D))
    for _ in range(N):
        cache.push_frame(draw(1, F, Hkv, D), draw(1, F, Hkv, D))
    tail = torch.zeros((B, 64, Hkv, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    exps = torch.zeros((B, 64, Hkv), dtype=torch.uint8, device="cuda")
    none = _int([0] * B)
    q = torch.randn((B, T, Hq, D), generator=torch.Generator(device="cuda").manual_seed(60), device="cuda").to(torch.bfloat16)
    attend = lambda out, s=None: cache.attend_streams_quant(0, q, tail, tail, exps, exps, none, out=out, stream=s)
    before, after = torch.empty_like(q), torch.empty_like(q)
    attend(before)
    torch.cuda.synchronize()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    attend(before)
    end.record()
    torch.cuda.synchronize()
    ms = start.elapsed_time(end)
    prod, cons = torch.cuda.Stream(priority=-1), torch.cuda.Stream()
    got = [torch.empty_like(q) for _ in range(8)]
    frames = [(draw(1, F, Hkv, D), draw(1, F, Hkv, D)) for _ in got]
    torch.cuda.synchronize()
    for i, (out, (fk, fv)) in enumerate(zip(got, frames)):
        attend(before)
        torch.cuda.synchronize()
        with torch.cuda.stream(prod):
            torch.cuda._sleep(int(ms * 1e6 * 1.9 * (i + 1) / 9))     # cycles: into the call that follows
        cache.push_frame_async(fk, fv, prod, cons)
        attend(out, cons)
        torch.cuda.synchronize()
        attend(after)
        torch.cuda.synchronize()
        assert not torch.equal(before, after)
        assert torch.equal(out, before) or torch.equal(out, after), i
    assert cache.check_device_error() == 0
    cache.close()


@pytest.mark.parametrize("spare", [0, 1])
def test_attention_graph_follows_the_ring(rx, spare):
    """A captured call sees the frames that are pushed between its replays."""
    import torch
    g = np.random.default_rng(61 + spare)
    B, T, D, N = 3, 2, 128, 3
    st = Store(rx, g, 8, 1, D, 20, N, 64, 50, B * T, pushes=0, spare=spare)
    kc, ke, vc, ve = _tails(g, B, 50, 1, D)
    lens = [2, 50, 31]
    q = _bits(g, (B, T, 8, D))
    args = (dev(q), _codes(kc), _codes(vc), torch.from_numpy(ke).cuda(), torch.from_numpy(ve).cuda(), _int(lens))
    out = torch.empty((B, T, 8, D), dtype=torch.bfloat16, device="cuda")
    st.cache.attend_streams_quant(0, *args, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.cache.attend_streams_quant(0, *args, out=out)
    f = W.bf16_bits_to_f64
    frames = []
    for _ in range(N + 3):
        fk, fv = _bits(g, (1, 64, 1, D)), _bits(g, (1, 64, 1, D))
        st.cache.push_frame(dev(fk), dev(fv))
        frames.append((f(fk[0]), f(fv[0])))
        graph.replay()
        got = host64(out)
        k, v = (np.concatenate([x] + [y[i] for y in frames[-N:]]) for i, x in enumerate((st.k[0], st.v[0])))
        for b in range(B):
            ref, spread = OS.stream_attention(f(q[b]), k, v, OS.dequantise(kc[b, :lens[b]], ke[b, :lens[b]]),
                                              OS.dequantise(vc[b, :lens[b]], ve[b, :lens[b]]))
            _check(got[b], ref, spread)
    assert st.cache.check_device_error() == 0


def test_attention_on_the_legacy_stream_beside_a_capture_is_refused(rx):
    """The capturing stream waits on the legacy one (it is no torch stream, but
    one made by cudaStreamCreate): a call there is refused with the same status,
    and the capture goes on."""
    import ctypes
    import torch
    g = np.random.default_rng(45)
    st = Store(rx, g, 8, 1, 64, 16, 1, 16, 40, 4, pushes=1)
    kc, ke, vc, ve = _tails(g, 2, 40, 1, 64)
    q = dev(_bits(g, (2, 1, 8, 64)))
    args = (q, _codes(kc), _codes(vc), torch.from_numpy(ke).cuda(), torch.from_numpy(ve).cuda(), _int([40, 13]))
    first = st.cache.attend_streams_quant(0, *args)
    outs = [torch.zeros_like(first) for _ in range(3)]
    legacy = torch.cuda.default_stream()
    assert legacy.cuda_stream == 0
    cudart = ctypes.CDLL([line.split()[-1] for line in open("/proc/self/maps") if "libcudart.so" in line][0])
    made = ctypes.c_void_p()
    assert cudart.cudaStreamCreate(ctypes.byref(made)) == 0
    blocking = torch.cuda.ExternalStream(made.value)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=blocking):
        st.cache.attend_streams_quant(0, *args, out=outs[0])
        with pytest.raises(rx.RxError) as e:
            st.cache.attend_streams_quant(0, *args, out=outs[2], stream=legacy)
        assert e.value.status == -7
        st.cache.attend_streams_quant(0, *args, out=outs[1])
    graph.replay()
    torch.cuda.synchronize()
    st.cache.attend_streams_quant(0, *args, out=outs[2], stream=legacy)
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs)
    del graph
    assert cudart.cudaStreamDestroy(made) == 0


def test_a_cache_collected_within_a_capture_leaves_it_whole(rx):
    """The garbage collector may run at any place, within a capture too."""
    import gc
    import torch
    g = np.random.default_rng(44)
    st = Store(rx, g, 8, 1, 64, 16, 1, 16, 40, 4, pushes=1)
    kc, ke, vc, ve = _tails(g, 2, 40, 1, 64)
    q = dev(_bits(g, (2, 1, 8, 64)))
    args = (q, _codes(kc), _codes(vc), torch.from_numpy(ke).cuda(), torch.from_numpy(ve).cuda(), _int([40, 13]))
    first = st.cache.attend_streams_quant(0, *args)
    out = torch.zeros_like(first)
    gc.collect()
    free = torch.cuda.mem_get_info()[0]
    cycle = [rx.Cache(1, 8, 1, 256, 1024, 1, 64, 4)]
    cycle.append(cycle)
    assert torch.cuda.mem_get_info()[0] < free
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        st.cache.attend_streams_quant(0, *args, out=out)
        del cycle
        gc.collect()
        st.cache.attend_streams_quant(0, *args, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, out)
    assert rx._parked
    rx.Cache(1, 8, 1, 64, 16, 1, 16, 4).close()
    assert not rx._parked


def test_attention_shares_the_exchange_area(rx):
    """The suffix's and the batch's attention in front of and behind it, and all
    of them in one captured graph: they use one exchange area, which the store's
    kernel writes from a stream of the cache."""
    import torch
    g = np.random.default_rng(46)
    B, T, D, cap, S = 12, 4, 256, 200, 51
    cache = rx.Cache(1, 8, 1, D, 64, 8, 256, S, cap, B * T)
    pk, pv = _bits(g, (1, 64, 1, D)), _bits(g, (1, 64, 1, D))
    cache.pin_prefix(dev(pk), dev(pv))
    for _ in range(8):
        cache.push_frame(dev(_bits(g, (1, 256, 1, D))), dev(_bits(g, (1, 256, 1, D))))
    kc, ke, vc, ve = _tails(g, B, cap, 1, D)
    lens = [int(x) for x in g.integers(T, cap + 1, B)]
    held = _int(lens)
    tails = (_codes(kc), _codes(vc), torch.from_numpy(ke).cuda(), torch.from_numpy(ve).cuda(), held)
    q8 = dev(_bits(g, (B, T, 8, D)))
    qs, ks, vs = dev(_bits(g, (S, 8, D))), dev(_bits(g, (S, 1, D))), dev(_bits(g, (S, 1, D)))
    qb = dev(_bits(g, (B, 1, 8, D)))
    k16, v16 = (torch.from_numpy(OS.dequantise(c, e)).to(torch.bfloat16).cuda() for c, e in ((kc, ke), (vc, ve)))
    order = "8s8b8bs8s"
    run = {"8": lambda o: cache.attend_streams_quant(0, q8, *tails, out=o),
           "s": lambda o: cache.attend_suffix(0, qs, ks, vs, out=o),
           "b": lambda o: cache.attend_batch(0, None, (qb, k16, v16, held), out_lang=o)}
    like = {"8": q8, "s": qs, "b": qb}
    alone = {}
    for k in "8sb":
        alone[k] = torch.zeros_like(like[k])
        run[k](alone[k])
        torch.cuda.synchronize()
    outs = [torch.zeros_like(like[k]) for k in order]
    for k, o in zip(order, outs):
        run[k](o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, alone[k]) for k, o in zip(order, outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for k, o in zip(order, outs):
            run[k](o)
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, alone[k]) for k, o in zip(order, outs))
    assert cache.check_device_error() == 0
    cache.close()


@pytest.mark.parametrize("B,T,lo,hi", [(32, 1, 1, 16000), (64, 8, 8000, 16384)])
def test_attention_at_full_size(rx, B, T, lo, hi):
    """Long dialogues and the largest drafts, at the sizes they are measured at."""
    import torch
    g = np.random.default_rng(47)
    D, cap, P = 256, 16384, 256
    st = Store(rx, g, 8, 1, D, P, 8, 256, cap, B * T, pushes=8)
    gen = torch.Generator(device="cuda").manual_seed(47)

    def tails():   # normal values of a random scale, as codes and exponents
        code = torch.randn((B, cap, 1, D), generator=gen, device="cuda").mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn)
        return code, torch.randint(119, 122, (B, cap, 1), generator=gen, device="cuda", dtype=torch.uint8)
    (kt, ke), (vt, ve) = tails(), tails()
    lens = [lo + (hi - lo) * ((7 * b) % B) // (B - 1) for b in range(B)]
    q = _bits(g, (B, T, 8, D), 0.2)
    got = host64(st.cache.attend_streams_quant(0, dev(q), kt, vt, ke, ve, _int(lens)))
    for b in list(range(0, B, 21)) + [B - 1]:
        k, v = (OS.dequantise(_u8(c[b, :lens[b]]), e[b, :lens[b]].cpu().numpy()) for c, e in ((kt, ke), (vt, ve)))
        ref, spread = OS.stream_attention(W.bf16_bits_to_f64(q[b]), st.k[0], st.v[0], k, v)
        _check(got[b], ref, spread)
    assert st.cache.check_device_error() == 0


def test_calls_with_their_outputs_given_allocate_nothing(rx):
    import torch
    g = np.random.default_rng(48)
    st = Store(rx, g, 8, 1, 128, 16, 1, 64, 300, 12, pushes=1)
    kc, ke, vc, ve = _tails(g, 3, 300, 1, 128)
    tails = (_codes(kc), _codes(vc), torch.from_numpy(ke).cuda(), torch.from_numpy(ve).cuda())
    q, xk, xv = dev(_bits(g, (3, 4, 8, 128))), dev(_bits(g, (3, 4, 1, 128))), dev(_bits(g, (3, 4, 1, 128)))
    out, held, now = torch.empty_like(q), _int([0, 100, 290]), _int([0, 0, 0])

    def step():
        rx.tail_append_quant(*tails, held, xk, xv, new_len=now)
        st.cache.attend_streams_quant(0, q, *tails, now, out=out)
    step()
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0], torch.cuda.memory_allocated(), torch.cuda.memory_stats()["allocation.all.allocated"]
    for _ in range(5):
        step()
    torch.cuda.synchronize()
    assert before == (torch.cuda.mem_get_info()[0], torch.cuda.memory_allocated(),
                      torch.cuda.memory_stats()["allocation.all.allocated"])


def test_attention_on_another_stream(rx):
    import torch
    g = np.random.default_rng(25)
    st = Store(rx, g, 8, 1, 64, 16, 1, 16, 40, 4, pushes=1)
    kc, ke, vc, ve = _tails(g, 2, 40, 1, 64)
    q = dev(_bits(g, (2, 1, 8, 64)))
    args = (q, _codes(kc), _codes(vc), torch.from_numpy(ke).cuda(), torch.from_numpy(ve).cuda(), _int([40, 13]))
    here = st.cache.attend_streams_quant(0, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there = torch.empty_like(here)
    st.cache.attend_streams_quant(0, *args, out=there, stream=side)
    fresh = st.cache.attend_streams_quant(0, *args, stream=side)   # allocated there
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(here, there) and torch.equal(here, fresh)


def test_attention_agrees_with_the_16_bit_tails(rx):
    """Tails whose values e4m3 holds exactly: the same answer as rx_attend_batch
    on 16-bit tails, within both calls' roundings."""
    import torch
    g = np.random.default_rng(26)
    B, D, cap = 16, 256, 32
    st = Store(rx, g, 8, 1, D, 64, 8, 256, cap, B, pushes=9)
    kc, ke, vc, ve = _tails(g, B, cap, 1, D)
    lens = [int(x) for x in g.integers(0, 31, B)]
    q = dev(_bits(g, (B, 1, 8, D)))
    k16 = torch.from_numpy(OS.dequantise(kc, ke)).to(torch.bfloat16).cuda()
    v16 = torch.from_numpy(OS.dequantise(vc, ve)).to(torch.bfloat16).cuda()
    _, want = st.cache.attend_batch(0, None, (q, k16, v16, _int(lens)))
    got = st.cache.attend_streams_quant(0, q, _codes(kc), _codes(vc), torch.from_numpy(ke).cuda(),
                                        torch.from_numpy(ve).cuda(), _int(lens))
    # attend_batch rounds weights, partials and output: 3 * 2^-8 of spread <= max|v| < 6 there, 2 here.
    assert (got.float() - want.float()).abs().max().item() <= 5 * 2.0 ** -8 * 6


# ------------------------------------------------------------ verification
def _verify(rx, p, q, draft, u, r, n, dtype, lens=True):
    import torch
    B, T1, V = p.shape
    T = T1 - 1
    pt = torch.from_numpy(p).to(dtype).cuda()
    qt = None if q is None else torch.from_numpy(q).to(dtype).cuda()
    tl = _int(np.arange(B) * 3)
    got = rx.verify_drafts(pt, qt, _int(np.reshape(draft, (B, T))), torch.from_numpy(u).cuda(), torch.from_numpy(r).cuda(),
                           n_draft=None if n is None else _int(n), tail_len=tl if lens else None)
    tokens, count = got[0].cpu().numpy(), got[1].cpu().numpy()
    p64 = pt.double().cpu().numpy()
    q64 = None if q is None else qt.double().cpu().numpy()
    for b in range(B):
        m = T if n is None else min(n[b], T)
        if m < 0:
            want, a = [], -1
        else:
            want, a = OS.verify(p64[b], None if q is None else q64[b], draft[b], u[b].astype(np.float64), float(r[b]), m)
        assert count[b] == a, (b, count[b], a)
        assert tokens[b].tolist() == want + [-1] * (T + 1 - len(want)), b
    if lens:
        assert got[2].tolist() == [3 * b + 1 + int(count[b]) for b in range(B)]
    else:
        assert got[2] is None


def _softmax(x):
    x = np.exp(x - x.max(-1, keepdims=True))
    return (x / x.sum(-1, keepdims=True)).astype(np.float32)


@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (3, 2, 2), (5, 1, 31), (4, 3, 33), (7, 8, 1000), (6, 4, 1023), (2, 33, 257),
                                   (16, 7, 50257), (3, 2, 151936), (9, 5, 4100), (64, 4, 515), (2, 3, 257153)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("with_q", [True, False])
def test_verify_accepts_and_draws(rx, B, T, V, dtype, with_q):
    import torch
    g = np.random.default_rng(B * 10000 + V)
    z = g.standard_normal((B, T + 1, V)) * 2
    p = _softmax(z)
    q = _softmax(z[:, :T] + 0.5 * g.standard_normal((B, T, V))) if with_q else None
    draft = np.argmax(z[:, :T] + g.gumbel(size=(B, T, V)), -1)
    n = [int(x) for x in g.integers(-1, T + 2, B)]
    _verify(rx, p, q, draft, g.random((B, T), dtype=np.float32), g.random(B, dtype=np.float32), n, getattr(torch, dtype))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_verify_without_drafts_samples(rx, dtype):
    import torch
    g = np.random.default_rng(5)
    p = _softmax(g.standard_normal((70, 1, 777)) * 3)
    r = g.random(70, dtype=np.float32)
    r[0], r[1] = 0.0, np.float32(1 - 2.0 ** -24)
    _verify(rx, p, None, np.zeros((70, 0), np.int64), np.zeros((70, 0), np.float32), r, None, getattr(torch, dtype), lens=False)


def test_verify_edges(rx):
    """Equal distributions, drafts without probability, tokens out of range,
    NaN and infinite entries, rows without any weight."""
    import torch
    g = np.random.default_rng(6)
    B, T, V = 12, 3, 300
    p = _softmax(g.standard_normal((B, T + 1, V)))
    q = _softmax(g.standard_normal((B, T, V)))
    draft = g.integers(0, V, (B, T))
    u, r = g.random((B, T), dtype=np.float32), g.random(B, dtype=np.float32)
    q[0] = p[0, :T]                                   # equal: accepted whatever u < 1 is
    p[1, 0, draft[1, 0]] = 0                          # p = 0: refused
    q[2, 0, draft[2, 0]] = 0                          # q = 0 < p: accepted
    draft[3, 1], draft[4, 0], draft[5, 2] = -1, V, 1 << 30
    u[6] = 0                                          # accepted wherever p > 0
    p[7, 0], q[7, 0] = 0.5 * q[7, 0], q[7, 0]         # no positive difference: drawn from p
    u[7, 0] = np.float32(0.99)
    p[8, 0, 5], p[8, 0, 9] = np.nan, np.inf
    p[9, 0] = 0                                       # nothing at all
    p[10, 0, :] = 0
    p[10, 0, V - 1] = 1                               # all weight on the last
    r[11] = 0
    _verify(rx, p, q, draft, u, r, None, torch.float32)
    _verify(rx, p, None, draft, u, r, [T, T, 0, 1, 2, T, T, 0, 0, 0, 0, -7], torch.float32)


@pytest.mark.parametrize("V", [300, 5000, 40000, 257153])
def test_verify_weights_far_apart(rx, V):
    """Few tokens with weight, in different CTAs' and warps' parts, and
    thresholds at the ends: never a token without weight."""
    import torch
    at = sorted({0, 5, V // 3, V // 2 + 1, V - 7, V - 1})
    rows, r = [], []
    for i in at:
        p = np.zeros(V, np.float32)
        p[i] = 1
        rows += [p, p]
        r += [0.0, 1 - 2.0 ** -24]
    for i, j in zip(at, at[1:]):
        p = np.zeros(V, np.float32)
        p[i], p[j] = 0.25, 0.75
        rows += [p] * 4
        r += [0.0, 0.25 - 2.0 ** -26, 0.25, 1 - 2.0 ** -24]
    p = np.stack(rows)[:, None]
    n = len(rows)
    _verify(rx, p, None, np.zeros((n, 0), np.int64), np.zeros((n, 0), np.float32), np.array(r, np.float32), None,
            torch.float32)


def test_verify_probabilities_near_the_smallest_number(rx):
    """u * q(x) and p(x) within a few steps of 2^-149 of each other, where the
    product's rounding error is no fp32 number."""
    import torch
    g = np.random.default_rng(41)
    B, T, V = 256, 1, 40
    p, q = _softmax(g.standard_normal((B, T + 1, V))), _softmax(g.standard_normal((B, T, V)))
    draft = g.integers(0, V, (B, T))
    m, k = g.integers(1, 9, B), g.integers(0, 6, B)
    at = np.arange(B)
    q[at, 0, draft[:, 0]] = (m * 2.0 ** -149).astype(np.float32)
    p[at, 0, draft[:, 0]] = (k * 2.0 ** -149).astype(np.float32)
    u, r = g.random((B, T), dtype=np.float32), g.random(B, dtype=np.float32)
    near = np.abs(u[:, 0].astype(np.float64) * m - k) < 0.5
    assert near.sum() > 20 and ((u[:, 0].astype(np.float64) * m < k) & near).sum() > 5
    _verify(rx, p, q, draft, u, r, None, torch.float32)


@pytest.mark.parametrize("seed", [0, 3])
def test_verify_sums_over_many_terms(rx, seed):
    """A row of 2^26 terms whose threshold lies between tokens of 2^-43 of the
    total.  The terms before it are alike in every lane of the kernel, so that
    the lanes' rounding errors add up instead of cancelling; those after it add
    without rounding.  Every number is an integer of 2^-45, and r = 1/2 falls
    into the middle of the 2001 small tokens, with 2^-44 of the total to either
    side.  Sums that are off by 2^-46 move the threshold by a quarter of that
    (half of the total is the terms before it, and it moves by half as much)."""
    import torch
    g = np.random.default_rng(seed)
    V, half, small, unit = 1 << 26, 1 << 25, 2001, 2.0 ** -45
    base = np.exp(2.5 * g.standard_normal(4096)).astype(np.float32)
    base = np.maximum(np.float32(2.0 ** -21), base / np.float32(2.0 ** 6))   # 24 bits of at least 2^-21: integers of 2^-45
    steps = np.tile(base, half // 4096 // 128)
    first = np.repeat(steps, 128)                                  # each value at 128 places: one per lane, four terms a load
    total = 128 * (half // 4096 // 128) * sum(int(x) for x in base.astype(np.float64) / unit)
    w = float(2.0 ** round(np.log2(total * unit)) * 2.0 ** -42)    # a small token, 2^-43 of the total
    assert (w / unit).is_integer()
    row = np.zeros(V, np.float32)
    row[:half] = first
    row[half:half + small] = w
    rest = V - half - small - 4
    c = 2.0 ** np.floor(np.log2(total * unit / rest))
    row[half + small:half + small + rest] = c
    left = total - rest * int(c / unit)                            # in up to three pieces of 24 bits
    for i in range(4):
        bits = max(0, left.bit_length() - 24)
        piece = (left >> bits) << bits
        row[V - 4 + i] = piece * unit
        left -= piece
    assert left == 0
    p = torch.from_numpy(row).cuda().view(1, 1, V)
    none = torch.zeros((1, 0), dtype=torch.int32, device="cuda")
    tokens, n, _ = rx.verify_drafts(p, None, none, none.float(), torch.full((1,), 0.5, device="cuda"))
    assert n.item() == 0
    assert tokens.item() == half + small // 2


@pytest.mark.parametrize("V", [5000, 10000, 60000])
def test_verify_clusters_beside_other_work(rx, V):
    """Clusters of 2, 4 and 8 CTAs whose CTAs start at different times, because
    other kernels hold SMs: every call gives what it gives alone, idle slots
    and rows without any difference among them."""
    import torch
    g = np.random.default_rng(V)
    B, T = 24, 2
    p = _softmax(g.standard_normal((B, T + 1, V)))
    q = _softmax(g.standard_normal((B, T, V)))
    q[3] = p[3, :T]
    p[4, 0], q[4, 0] = 0.5 * q[4, 0], q[4, 0]
    u, r = g.random((B, T), dtype=np.float32), g.random(B, dtype=np.float32)
    n = [T] * B
    n[5] = n[23] = -1
    draft = g.integers(0, V, (B, T))
    _verify(rx, p, q, draft, u, r, n, torch.float32)
    args = [torch.from_numpy(x).cuda() for x in (p, q)] + [_int(draft), torch.from_numpy(u).cuda(), torch.from_numpy(r).cuda()]
    n = _int(n)
    want = rx.verify_drafts(*args, n_draft=n)
    side = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    got = []
    for _ in range(40):
        with torch.cuda.stream(side):
            busy @ busy
        got.append(rx.verify_drafts(*args, n_draft=n))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for a in got for x, y in zip(a[:2], want))


@pytest.mark.parametrize("V", [4099, 32000, 151936])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_verify_does_not_depend_on_the_batch(rx, V, dtype):
    """The batch's size sets the CTAs of a stream and with them the order of the
    sums: the same rows give the same tokens whatever stands beside them."""
    import torch
    g = np.random.default_rng(49)
    T, most = 2, 160
    z = g.standard_normal((8, T + 1, V)) * 2
    p = torch.from_numpy(_softmax(z)).to(getattr(torch, dtype)).cuda()
    q = torch.from_numpy(_softmax(z[:, :T] + 0.5 * g.standard_normal((8, T, V)))).to(p.dtype).cuda()
    draft = _int(np.argmax(z[:, :T] + g.gumbel(size=(8, T, V)), -1))
    u = torch.from_numpy(g.random((8, T), dtype=np.float32)).cuda()
    r = torch.from_numpy(g.random(8, dtype=np.float32)).cuda()
    at = torch.arange(most, device="cuda") % 8
    want = None
    for B in (8, 1, 20, 40, 80, most):
        i = at[:B]
        tokens, n, _ = rx.verify_drafts(p[i], q[i], draft[i], u[i], r[i])
        if want is None:
            want = tokens, n
        assert torch.equal(tokens, want[0][i]) and torch.equal(n, want[1][i])


def test_verify_lengths_in_place_and_graph(rx):
    import torch
    g = np.random.default_rng(8)
    B, T, V = 4, 2, 100
    p, q = _softmax(g.standard_normal((B, T + 1, V))), _softmax(g.standard_normal((B, T, V)))
    args = (torch.from_numpy(p).cuda(), torch.from_numpy(q).cuda(), _int(g.integers(0, V, (B, T))),
            torch.rand((B, T), device="cuda"), torch.rand((B,), device="cuda"))
    tl = _int([0, 10, 20, 30])
    _, n, _ = rx.verify_drafts(*args, tail_len=tl, new_len=tl)
    n = n.tolist()
    assert tl.tolist() == [10 * b + 1 + n[b] for b in range(B)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rx.verify_drafts(*args, tail_len=tl, new_len=tl)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert tl.tolist() == [10 * b + 4 * (1 + n[b]) for b in range(B)]


# ------------------------------------------------------------- run together
def test_streams_decode_with_drafts(rx):
    """Four steps of append, attention on every layer and verification, with
    the lengths kept on the device throughout, beside frames that arrive."""
    import torch
    g = np.random.default_rng(30)
    L, B, T, Hq, Hkv, D, cap, V = 2, 3, 4, 8, 1, 128, 64, 500
    st = Store(rx, g, Hq, Hkv, D, 32, 2, 64, cap, B * T, pushes=2, layers=L)
    kt = [torch.full((B, cap, Hkv, D), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(L)]
    vt = [x.clone() for x in kt]
    ke = [torch.full((B, cap, Hkv), 255, dtype=torch.uint8, device="cuda") for _ in range(L)]
    ve = [x.clone() for x in ke]
    length, total = _int([0, 0, 0]), _int([0, 0, 0])
    held = [[(np.zeros((0, Hkv, D)), np.zeros((0, Hkv, D))) for _ in range(B)] for _ in range(L)]
    kept = [0] * B
    for step in range(4):
        n = [T, 1 + step % T, T - 1]               # the last token and up to T - 1 drafts
        new = _int(n)
        for i in range(L):
            xk, xv, q = (_bits(g, (B, T, h, D)) for h in (Hkv, Hkv, Hq))
            rx.tail_append_quant(kt[i], vt[i], ke[i], ve[i], length, dev(xk), dev(xv), n_new=new, new_len=total)
            out = host64(st.cache.attend_streams_quant(i, dev(q), kt[i], vt[i], ke[i], ve[i], total, n_new=new))
            for b in range(B):
                k, v = (np.concatenate([held[i][b][j][:kept[b]], OS.dequantise(*OS.quantise(W.bf16_bits_to_f64(x[b, :n[b]])))])
                        for j, x in enumerate((xk, xv)))
                held[i][b] = (k, v)
                ref, spread = OS.stream_attention(W.bf16_bits_to_f64(q[b, :n[b]]), st.k[i], st.v[i], k, v)
                _check(out[b, :n[b]], ref, spread)
        z = g.standard_normal((B, T, V))
        p, qd = _softmax(z), _softmax(z[:, :T - 1] + 0.3 * g.standard_normal((B, T - 1, V)))
        draft = np.argmax(z[:, :T - 1] + g.gumbel(size=(B, T - 1, V)), -1)
        u, r = g.random((B, T - 1), dtype=np.float32), g.random(B, dtype=np.float32)
        tokens, count, _ = rx.verify_drafts(torch.from_numpy(p).cuda(), torch.from_numpy(qd).cuda(), _int(draft),
                                            torch.from_numpy(u).cuda(), torch.from_numpy(r).cuda(),
                                            n_draft=_int([x - 1 for x in n]), tail_len=length, new_len=length)
        for b in range(B):
            want, a = OS.verify(p[b].astype(np.float64), qd[b].astype(np.float64), draft[b], u[b].astype(np.float64), float(r[b]), n[b] - 1)
            assert count[b].item() == a and tokens[b, :a + 1].tolist() == want
            kept[b] += 1 + a
        assert length.tolist() == kept
    assert max(kept) > 4
    st.cache.close()
