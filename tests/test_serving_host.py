"""Refusals of the serving entry points, and their plain forms against hand-made cases (CPU only)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import fp8, serving

FAKE = 0x100000  # never dereferenced: every call below fails its checks, or has nothing to do


def _strides(n, *values):
    return (ctypes.c_longlong * n)(*(values or [64] * n))


def _nr(lib, **kw):
    a = dict(norm=1, eps=1e-6, q_weight=None, k_weight=None, weight_dtype=lib.SAGE_FP32, cos_sin=FAKE, n_pos=16, rot=64,
             interleaved=0)
    a.update(kw)
    return lib.SageNormRope(**a)


def _rows(lib, nr=None, **kw):
    a = dict(q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, st=_strides(12), pos=FAKE, ps=0, B=1, N=4, Hq=2, Hkv=2, d=64,
             dtype=lib.SAGE_FP16)
    a.update(kw)
    nr = _nr(lib) if nr is None else nr
    return lib.capi.sage_qk_norm_rope(a["q"], a["k"], a["qo"], a["ko"], a["st"], a["pos"], a["ps"], a["B"], a["N"],
                                      a["Hq"], a["Hkv"], a["d"], a["dtype"], None if nr == "null" else ctypes.byref(nr),
                                      None)


def _cache(lib, **kw):
    a = dict(k8=FAKE, ks=FAKE, v8=FAKE, vs=FAKE, num_pages=4, page_size=64, Hkv=2, d=64)
    a.update(kw)
    return lib.SageKVCache(**a)


def _append(lib, cache=None, nr=None, **kw):
    a = dict(q=None, k=FAKE, v=FAKE, qo=None, st=_strides(8), table=FAKE, ts=4, mp=4, lens=FAKE, cu=FAKE, mean=None, T=4,
             B=2, Hq=0, dtype=lib.SAGE_FP16)
    a.update(kw)
    c = _cache(lib) if cache is None else cache
    return lib.capi.sage_cache_append(None if c == "null" else ctypes.byref(c), a["q"], a["k"], a["v"], a["qo"], a["st"],
                                      a["table"], a["ts"], a["mp"], a["lens"], a["cu"], a["mean"], a["T"], a["B"],
                                      a["Hq"], a["dtype"], None if nr is None else ctypes.byref(nr), None)


def _gather(lib, cache=None, **kw):
    a = dict(table=FAKE, ts=4, mp=4, cu=FAKE, starts=None, mean=None, ko=FAKE + (1 << 32), vo=FAKE + (2 << 32), T=4, B=2,
             dtype=lib.SAGE_FP16)
    a.update(kw)
    c = _cache(lib) if cache is None else cache
    return lib.capi.sage_cache_gather(ctypes.byref(c), a["table"], a["ts"], a["mp"], a["cu"], a["starts"], a["mean"],
                                      a["ko"], a["vo"], a["T"], a["B"], a["dtype"], None)


def _decode(lib, cache=None, **kw):
    a = dict(q=FAKE, qb=128, qh=64, table=FAKE, ts=4, mp=4, lens=FAKE, out=FAKE + (1 << 32), B=2, Hq=4, n=100,
             dtype=lib.SAGE_FP16)
    a.update(kw)
    c = _cache(lib) if cache is None else cache
    return lib.capi.sage_attn_decode(a["q"], a["qb"], a["qh"], ctypes.byref(c), a["table"], a["ts"], a["mp"], a["lens"],
                                     a["out"], a["B"], a["Hq"], a["n"], a["dtype"], 0.0, None)


@pytest.fixture
def no_device(lib):
    """The device check reports an sm_90: a call that passes its argument checks ends there."""
    lib.capi.sage_test_inject(90, 0)
    yield lib.SAGE_ERR_ARCH
    lib.capi.sage_test_inject(0, 0)


def test_norm_rope_argument_checks(lib, no_device):
    E = lib.SAGE_ERR_INVALID_ARG
    assert _rows(lib) == no_device
    assert _rows(lib, k=None, ko=None, Hkv=0) == no_device and _rows(lib, pos=None) == no_device
    assert _rows(lib, dtype=lib.SAGE_FP32) == lib.SAGE_ERR_UNSUPPORTED and _rows(lib, dtype=9) == E
    for kw in (dict(q=None), dict(qo=None), dict(ko=None), dict(B=-1), dict(N=-1), dict(Hq=0), dict(Hkv=0), dict(d=0),
               dict(d=257), dict(Hq=70000), dict(st=None), dict(st=_strides(12, *[-1] * 12)), dict(ps=-1),
               dict(pos=FAKE + 2), dict(q=FAKE + 1), dict(N=2 ** 31 - 1, B=2 ** 31 - 1, Hq=65535),
               dict(N=2 ** 31 - 1, Hq=65535), dict(N=2 ** 20, st=_strides(12, *[2 ** 40] * 12)),
               dict(st=_strides(12, *[2 ** 41] * 12))):
        assert _rows(lib, **kw) == E, kw
    for kw in (dict(eps=-1.0), dict(eps=float("nan")), dict(rot=3), dict(rot=66), dict(rot=0), dict(n_pos=0),
               dict(q_weight=FAKE, weight_dtype=5), dict(norm=0, q_weight=FAKE), dict(cos_sin=FAKE + 2),
               dict(k_weight=FAKE + 2)):
        assert _rows(lib, nr=_nr(lib, **kw)) == E, kw
    assert _rows(lib, nr="null") == E
    assert _rows(lib, N=0) == lib.SAGE_OK and _rows(lib, B=0) == lib.SAGE_OK


def test_cache_argument_checks(lib, no_device):
    E = lib.SAGE_ERR_INVALID_ARG
    assert _append(lib) == no_device and _gather(lib) == no_device and _decode(lib) == no_device
    for kw in (dict(k8=None), dict(ks=None), dict(v8=None), dict(vs=None), dict(k8=FAKE + 8), dict(v8=FAKE + 1),
               dict(ks=FAKE + 2), dict(num_pages=0), dict(Hkv=0), dict(d=0), dict(d=257), dict(page_size=8),
               dict(page_size=48), dict(page_size=2048), dict(page_size=0)):
        c = _cache(lib, **kw)
        assert (_append(lib, c), _gather(lib, c), _decode(lib, c)) == (E, E, E), kw
    for kw in (dict(table=None), dict(table=FAKE + 2), dict(ts=-1), dict(mp=0), dict(ts=3)):  # rows shorter than max_pages
        assert (_append(lib, **kw), _gather(lib, **kw), _decode(lib, **kw)) == (E, E, E), kw
    assert _append(lib, "null") == E


def test_append_gather_decode_argument_checks(lib, no_device):
    E, U = lib.SAGE_ERR_INVALID_ARG, lib.SAGE_ERR_UNSUPPORTED
    for f in (_append, _gather, _decode):
        assert f(lib, dtype=lib.SAGE_FP32) == U and f(lib, dtype=-1) == E and f(lib, B=-1) == E
    for kw in (dict(k=None), dict(v=None), dict(lens=None), dict(lens=FAKE + 2), dict(cu=FAKE + 1), dict(mean=FAKE + 2),
               dict(T=-1), dict(cu=None), dict(k=FAKE + 1), dict(st=None),
               dict(q=FAKE, qo=FAKE, Hq=4)):                                    # q without norm or rotation
        assert _append(lib, **kw) == E, kw
    assert _append(lib, cu=None, T=2) == no_device
    assert _append(lib, nr=_nr(lib), q=FAKE, qo=FAKE, Hq=4) == no_device
    assert _append(lib, nr=_nr(lib), q=FAKE, qo=None, Hq=4) == E and _append(lib, nr=_nr(lib, rot=65)) == E
    assert _append(lib, T=0) == lib.SAGE_OK and _gather(lib, T=0) == lib.SAGE_OK and _decode(lib, B=0) == lib.SAGE_OK
    for kw in (dict(cu=None), dict(ko=None), dict(vo=None), dict(ko=FAKE), dict(ko=FAKE + (2 << 32) + 2), dict(T=-1),
               dict(starts=FAKE + 3), dict(vo=FAKE + (2 << 32) + 1)):
        assert _gather(lib, **kw) == E, kw
    for kw in (dict(q=None), dict(out=None), dict(lens=None), dict(Hq=3), dict(Hq=0), dict(n=-1), dict(out=FAKE + 8),
               dict(qb=-1), dict(qh=-1), dict(B=70000), dict(q=FAKE + 1)):
        assert _decode(lib, **kw) == E, kw


@pytest.mark.parametrize("array", ["k8", "ks", "v8", "vs"])
def test_decode_refuses_an_output_inside_the_cache(lib, no_device, array):
    at = {name: FAKE + ((i + 2) << 32) for i, name in enumerate(("k8", "ks", "v8", "vs"))}
    rows = 4 * 2 * 64                                          # pages, kv heads, page_size
    size = rows * (64 if array in ("k8", "v8") else 4)
    out_bytes = 2 * 4 * 64 * 2
    for out, want in ((at[array], lib.SAGE_ERR_INVALID_ARG), (at[array] + size - 2, lib.SAGE_ERR_INVALID_ARG),
                      (at[array] - out_bytes + 2, lib.SAGE_ERR_INVALID_ARG),
                      (at[array] + size, no_device), (at[array] - out_bytes, no_device)):
        assert _decode(lib, _cache(lib, **at), out=out) == want, (array, out - at[array])


def test_decode_reports_a_failed_workspace(lib):
    try:
        lib.capi.sage_test_inject(100, 1)  # one long sequence: split, so it needs a workspace
        assert _decode(lib, _cache(lib, num_pages=2000), mp=2000, ts=2000, n=100000, B=1) == lib.SAGE_ERR_OOM
    finally:
        lib.capi.sage_test_inject(0, 0)


def test_python_layer_refuses_host_tensors(lib):
    q = torch.zeros(2, 4, 64, dtype=torch.float16)
    ints = torch.zeros(2, dtype=torch.int32)
    cache = lib.sage_kv_cache(4, 4, 64, 16, device="cpu")
    assert cache["k8"].shape == (4, 4, 16, 64) and cache["vs"].shape == (4, 4, 16)
    assert lib.sage_kv_cache(1, 1, 40, 16, device="cpu")["v8"].shape[-1] == 48
    for call in (lambda: lib.sage_qk_norm_rope(q, q), lambda: lib.sage_cache_append(cache, q, q, ints[:, None], ints),
                 lambda: lib.sage_cache_gather(cache, ints[:, None], ints, 2, 64),
                 lambda: lib.sage_attn_decode(q, cache, ints[:, None], ints, 10)):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------------------------------ the oracle's own pins
def test_oracle_norm_rope_on_a_hand_made_row():
    # row (3, 4): mean square 12.5; a quarter turn maps (a, b) to (-b, a)
    table = np.array([[1.0, 0.0], [0.0, 1.0]], np.float32)
    x = np.array([[[3.0, 4.0]], [[3.0, 4.0]]])
    y, _ = serving.norm_rope(x, True, 0.0, None, table, np.array([0, 1]), False)
    n = np.array([3.0, 4.0]) / np.sqrt(12.5)
    assert np.allclose(y[0, 0], n, rtol=1e-15) and np.allclose(y[1, 0], [-n[1], n[0]], rtol=1e-15)
    y, _ = serving.norm_rope(np.arange(1.0, 7.0)[None, None], False, 0.0, None, np.array([[0, 0, 1, 1]], np.float32),
                             np.array([0]), False)
    assert y[0, 0].tolist() == [-3, -4, 1, 2, 5, 6]        # channels 4, 5 pass
    y, _ = serving.norm_rope(np.arange(1.0, 7.0)[None, None], False, 0.0, None, np.array([[0, 0, 1, 1]], np.float32),
                             np.array([0]), True)
    assert y[0, 0].tolist() == [-2, 1, -4, 3, 5, 6]


def test_oracle_codes_on_hand_made_rows():
    k = np.array([[127, -127, 0.5, 1.5], [0, 0, 0, 0], [1e-31, 0, 0, 0], [np.inf, 1, 2, 3], [1, np.nan, 0, 0]], np.float32)
    c, s = serving.k_codes(k)
    assert c.tolist() == [[127, -127, 0, 2], [0] * 4, [0] * 4, [0] * 4, [0] * 4]
    assert s[0] == 1 and s[1] == 0 and s[2] == 0 and np.isnan(s[3]) and np.isnan(s[4])
    v, t = serving.v_codes(np.array([[448, -448, 0, 2.0 ** -9]], np.float32))
    assert fp8.decode(v).tolist() == [[448, -448, 0, 2.0 ** -9]] and t[0] == 1
    a, b = serving.read(c[:1], s[:1], v, t, k_mean=np.ones(4, np.float32))
    assert a.tolist() == [[128, -126, 1, 3]] and b.tolist() == [[448, -448, 0, 2.0 ** -9]]


def test_oracle_decode_is_softmax_attention():
    r = np.random.RandomState(0)
    q, k, v = r.randn(4, 8), r.randn(6, 2, 8), r.randn(6, 2, 8)
    out, spread, _ = serving.decode(q, k, v, 0.3)
    for h in range(4):
        w = [np.exp(0.3 * sum(q[h, c] * k[j, h // 2, c] for c in range(8))) for j in range(6)]
        for c in range(8):
            assert abs(out[h, c] - sum(w[j] * v[j, h // 2, c] for j in range(6)) / sum(w)) < 1e-12
    assert (spread >= np.abs(out)).all()
    assert serving.decode(q, k[:0], v[:0], 0.3)[0].tolist() == np.zeros((4, 8)).tolist()
