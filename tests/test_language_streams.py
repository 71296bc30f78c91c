"""Language streams over 8-bit tails, without a GPU: the oracle's own pins and
the refusals of the library and of the binding."""
import ctypes

import numpy as np
import pytest

from oracle import streams as OS
from tests._util import LIB, ensure_built


@pytest.fixture(scope="module")
def lib():
    try:
        ensure_built()
    except RuntimeError as e:  # pragma: no cover
        pytest.skip("cannot build librx.so here: %s" % e)
    return ctypes.CDLL(LIB)


# ------------------------------------------------------------------- oracle
def test_e4m3_codes_match_torch():
    import torch
    every = torch.arange(256, dtype=torch.uint8)
    np.testing.assert_array_equal(OS.e4m3_decode(every.numpy()), every.view(torch.float8_e4m3fn).double().numpy())
    x = np.concatenate([np.linspace(-448, 448, 9001), 2.0 ** np.arange(-12, 8), 0.0625 + 2.0 ** -7 * np.arange(20)])
    x = x.astype(np.float32)
    np.testing.assert_array_equal(OS.e4m3_encode(x.astype(np.float64)),
                                  torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_quantised_vectors_use_the_top_of_the_range():
    g = np.random.default_rng(0)
    x = g.standard_normal((50, 64)) * 2.0 ** g.integers(-40, 40, (50, 1))
    codes, byte = OS.quantise(x)
    back = OS.dequantise(codes, byte)
    top = np.abs(OS.e4m3_decode(codes)).max(-1)
    assert np.all((top >= 224) & (top <= 448))
    step = 2.0 ** -10 * 2.0 ** (byte.astype(np.float64) - 127)
    assert np.all(np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), step[:, None]))


def test_verify_keeps_the_targets_distribution():
    """Over all (u, r) the first token is distributed as p: the total over a
    fine grid, for a draft from each possible token weighted by q."""
    p = np.array([[0.5, 0.2, 0.3], [1, 0, 0]])
    q = np.array([[0.2, 0.6, 0.2]])
    grid = (np.arange(60) + 0.5) / 60
    got = np.zeros(3)
    for x in range(3):
        for u in grid:
            for r in grid:
                tokens, _ = OS.verify(p, q, [x], [u], r, 1)
                got[tokens[0]] += q[0, x] / len(grid) ** 2
    np.testing.assert_allclose(got, p[0], atol=0.02)   # the grid's cells are 1/60 wide


# ----------------------------------------------------------------- refusals
def _buf(n=1 << 14):
    b = ctypes.create_string_buffer(n + 64)
    return b, ctypes.addressof(b) + (-ctypes.addressof(b)) % 64


def test_append_refuses_bad_arguments(lib):
    from partitioned_kv_cache_gb300 import rx
    keep, p = _buf()
    f = rx._lib.rx_tail_append_quant
    good = dict(kt=p, vt=p + 256, ke=p + 512, ve=p + 528, tl=p + 544, nl=p + 560, kn=p + 1024, vn=p + 2048, nn=None,
                B=1, T=1, cap=4, Hkv=1, D=64, ov=None)

    def call(**kw):
        a = dict(good, **kw)
        return f(a["kt"], a["vt"], a["ke"], a["ve"], a["tl"], a["nl"], a["kn"], a["vn"], a["nn"], a["B"], a["T"], a["cap"],
                 a["Hkv"], a["D"], a["ov"], None)
    assert call(B=-1) == -1
    assert call(T=0) == -1
    assert call(cap=0) == -1
    assert call(Hkv=0) == -1
    assert call(T=(1 << 28) + 1) == -1
    assert call(B=1 << 20, T=1 << 13) == -1
    assert call(D=96) == -6
    assert call(B=0) == 0
    for name in ("kt", "vt", "ke", "ve", "tl", "kn", "vn"):
        assert call(**{name: None}) == -1, name
    for name in ("kt", "vt", "kn", "vn"):
        assert call(**{name: good[name] + 8}) == -1, name
    for name in ("tl", "nl"):
        assert call(**{name: good[name] + 2}) == -1, name
    assert call(nl=good["tl"]) == -1
    assert call(nn=p + 576, nl=p + 576) == -1
    assert call(vt=good["kt"]) == -1               # K and V in one place
    assert call(ve=good["ke"] + 3) == -1
    assert call(kn=good["vt"] + 128) == -1         # new values inside a tail
    assert call(ov=good["tl"]) == -1
    del keep


def test_attention_refuses_a_null_handle(lib):
    from partitioned_kv_cache_gb300 import rx
    assert rx._lib.rx_attend_streams_quant(None, 0, ctypes.byref(rx.RxQuantStreams()), None) == -1
    assert rx._lib.rx_attend_streams_quant(None, 0, None, None) == -1


def test_verify_refuses_bad_arguments(lib):
    from partitioned_kv_cache_gb300 import rx
    keep, p = _buf()
    f = rx._lib.rx_verify_drafts
    good = dict(p=p, q=p + 512, t=0, d=p + 1024, u=p + 1056, r=p + 1088, n=None, B=2, T=2, V=8, tl=p + 1120,
                tok=p + 1152, na=p + 1184, nl=p + 1216)

    def call(**kw):
        a = dict(good, **kw)
        return f(a["p"], a["q"], a["t"], a["d"], a["u"], a["r"], a["n"], a["B"], a["T"], a["V"], a["tl"], a["tok"], a["na"],
                 a["nl"], None)
    assert call(B=-1) == -1
    assert call(T=-1) == -1
    assert call(V=0) == -1
    assert call(V=(1 << 28) + 1) == -1
    assert call(t=2) == -1
    assert call(B=0) == 0
    for name in ("p", "r", "tok", "na", "d", "u"):
        assert call(**{name: None}) == -1, name
    assert call(tl=None) == -1                     # new_len without tail_len
    assert call(p=p + 2) == -1
    assert call(d=good["d"] + 2) == -1
    assert call(tok=good["d"]) == -1               # outputs over inputs or each other
    assert call(na=good["r"]) == -1
    assert call(na=good["tok"]) == -1
    assert call(nl=good["tl"] + 4) == -1           # neither the same array nor apart
    assert call(tok=good["tl"]) == -1
    assert call(na=good["p"] + 64) == -1
    del keep


def test_binding_refuses_shapes_and_types(lib):
    import torch
    from partitioned_kv_cache_gb300 import rx
    z = torch.zeros
    e4, u8, i32, bf = torch.float8_e4m3fn, torch.uint8, torch.int32, torch.bfloat16
    kt, ke = z(2, 5, 1, 64, dtype=u8).view(e4), z(2, 5, 1, dtype=u8)
    tl, x = z(2, dtype=i32), z(2, 3, 1, 64, dtype=bf)
    f = rx.tail_append_quant
    with pytest.raises(ValueError, match="v_tail"):
        f(kt, kt[:1], ke, ke, tl, x, x)
    with pytest.raises(ValueError, match="k_exp"):
        f(kt, kt, ke[:, :4], ke, tl, x, x)
    with pytest.raises(ValueError, match="v_new"):
        f(kt, kt, ke, ke, tl, x, x[:, :2])
    with pytest.raises(ValueError, match="n_new"):
        f(kt, kt, ke, ke, tl, x, x, n_new=tl[:1])
    with pytest.raises(TypeError, match="k_tail"):
        f(kt.view(u8), kt, ke, ke, tl, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        f(kt, kt, ke, ke, tl, x, x)
    c = rx.Cache.__new__(rx.Cache)
    c.cfg = rx.RxConfig(1, 8, 1, 64, 16, 4, 32, 51, 5, 6, 0)
    c._h = None
    q = z(2, 3, 8, 64, dtype=bf)
    with pytest.raises(ValueError, match="k_tail"):
        c.attend_streams_quant(0, q, kt[:, :4], kt, ke, ke, tl)
    with pytest.raises(ValueError, match="q"):
        c.attend_streams_quant(0, q[:, :, :4], kt, kt, ke, ke, tl)
    with pytest.raises(ValueError, match="out"):
        c.attend_streams_quant(0, q, kt, kt, ke, ke, tl, out=q[:1])
    with pytest.raises(ValueError, match="contiguous"):
        c.attend_streams_quant(0, q.transpose(0, 1).contiguous().transpose(0, 1), kt, kt, ke, ke, tl)
    p, d, u, r = z(2, 4, 9), z(2, 3, dtype=i32), z(2, 3), z(2)
    with pytest.raises(ValueError, match="p must"):
        rx.verify_drafts(p[:, :3], None, d, u, r)
    with pytest.raises(ValueError, match="q must"):
        rx.verify_drafts(p, p, d, u, r)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        rx.verify_drafts(p.half(), None, d, u, r)
    with pytest.raises(ValueError, match="tail_len"):
        rx.verify_drafts(p, None, d, u, r, new_len=z(2, dtype=i32))
    with pytest.raises(ValueError, match="CUDA"):
        rx.verify_drafts(p, None, d, u, r)


# ------------------------------------------------------------ cluster starts
@pytest.mark.parametrize("name,write", [("verify_drafts.cu", "st_cluster_f64("), ("adarmsnorm.cu", "cluster_peer(")])
def test_peers_have_started_before_their_shared_memory_is_written(name, write):
    """A kernel that stores into its cluster's shared memory arrives on the
    cluster's barrier early and waits for it in front of the first store."""
    import os
    import re
    from tests._util import ROOT
    src = open(os.path.join(ROOT, "partitioned_kv_cache_gb300", "csrc", name)).read()
    src = re.sub(r"//[^\n]*", "", src)
    kernel = [k for k in src.split("__global__")[1:] if write in k]
    assert len(kernel) == 1
    at = [kernel[0].find(x) for x in ("cluster_arrive_started();", "cluster_wait_started();", write)]
    assert -1 < at[0] < at[1] < at[2], at


# ------------------------------------- the SMs of the store and of the tails
SMS = 152


def test_stream_partition_leaves_the_tails_their_share(lib):
    """Whatever the sizes, the tails' grid gets at least three quarters of the
    SMs that its part of the work is worth, and what runs beside it fits."""
    from partitioned_kv_cache_gb300 import rx
    for units in range(1, 201):
        for t_max in (0, 1, 6, 33, 36, 132, 500, 5000):
            for tail_tiles in (0, 1, 16, 300, 2304, 2432, 8192, 10 ** 5, 10 ** 7):
                splits, tail_sms = rx.choose_stream_partition(t_max, units, tail_tiles, SMS)
                assert 1 <= splits <= max(1, min(t_max, 32))
                assert tail_sms == SMS or tail_sms == SMS - splits * units
                store = units * t_max
                share = SMS * 2 * tail_tiles / (store + 2 * tail_tiles + 1)
                assert 1 <= tail_sms and tail_sms >= 0.75 * share - 1, (units, t_max, tail_tiles, splits, tail_sms)


@pytest.mark.parametrize("name,units,t_max,tail_tiles,want", [
    ("64/8 heads of 128, 72 x 4 tokens, 8448 keys, tails of 512", 144, 132, 2304, (1, 152)),
    ("8 prompts of 302 tokens, 8448 keys, tails of 1024", 151, 132, 2432, (1, 152)),
    ("16 tokens, 2112 keys, tails of 32", 1, 33, 16, (17, 135)),
    ("16 x 5 tokens, 8448 keys, tails of 2048", 5, 132, 256, (17, 67)),
    ("7 x 3 tokens, 32/8 heads of 128, 337 keys, tails of 1001", 8, 6, 448, (3, 128)),
    ("32 tokens, 2112 keys, tails of 16384", 2, 33, 4096, (11, 130)),
    ("64 x 8 tokens, 2304 keys, tails of 16384", 32, 36, 8192, (2, 152)),
    ("64 tokens, 8448 keys, tails of 4096", 4, 132, 2048, (19, 152)),
])
def test_stream_partition_choices(lib, name, units, t_max, tail_tiles, want):
    from partitioned_kv_cache_gb300 import rx
    assert rx.choose_stream_partition(t_max, units, tail_tiles, SMS) == want, name


def test_stream_partition_refuses_sizes_out_of_range(lib):
    from partitioned_kv_cache_gb300 import rx
    for a in ((-1, 1, 1, 152, 32), (1, 0, 1, 152, 32), (1, 1, -1, 152, 32), (1, 1, 1, 0, 32), (1, 1, 1, 152, 0),
              ((1 << 20) + 1, 1, 1, 152, 32), (1, (1 << 20) + 1, 1, 152, 32), (1, 1, (1 << 48) + 1, 152, 32)):
        with pytest.raises(rx.RxError):
            rx.choose_stream_partition(*a)


# --------------------------------------------------- caches that are collected
def test_a_cache_is_freed_once_and_not_within_a_capture(lib, monkeypatch):
    """A cache that is collected while the current stream is being captured is
    freed when the next one is made; one whose freeing fails is not freed twice."""
    from partitioned_kv_cache_gb300 import rx
    freed, capturing, status = [], [False], [0]

    def destroy(h):
        freed.append(h)
        return status[0]
    monkeypatch.setattr(rx._lib, "rx_cache_destroy", destroy)
    monkeypatch.setattr(rx, "_capturing", lambda: capturing[0])

    def cache(h):
        c = rx.Cache.__new__(rx.Cache)
        c._h = h
        return c
    c = cache(1)
    del c
    assert freed == [1]
    capturing[0] = True
    c = cache(2)
    del c
    rx._free_parked()
    assert freed == [1]
    capturing[0] = False
    rx._free_parked()
    rx._free_parked()
    assert freed == [1, 2]
    status[0] = -4
    c = cache(3)
    with pytest.raises(rx.RxError):
        c.close()
    del c
    assert freed == [1, 2, 3]
