"""Outputs of the head-row calls that overlap what the call reads, another output or themselves are refused before
anything is launched; slices side by side of one fused tensor are not.  (CPU only: the device check reports a B200, so that a
call that is not refused ends at its launch, with a CUDA error.)"""
import ctypes
import itertools

import pytest
import torch

FAKE = 0x10000000  # never dereferenced
FAR = 1 << 40


@pytest.fixture
def launched(lib):
    if torch.cuda.is_available():
        pytest.skip("the calls that pass would be launched on addresses that do not exist")
    lib.capi.sage_test_inject(100, 0)
    yield lib.SAGE_ERR_CUDA
    lib.capi.sage_test_inject(0, 0)


class View:
    """Element offset and (batch, token, head) strides and extents."""

    def __init__(self, at, strides, sizes):
        self.at, self.strides, self.sizes = at, strides, sizes

    @property
    def ptr(self):
        return FAKE + 2 * self.at

    def places(self, d):
        out = []
        for i in itertools.product(*(range(n) for n in self.sizes)):
            first = self.at + sum(x * s for x, s in zip(i, self.strides))
            out += range(first, first + d)
        return out


def _rows(lib, q, k, qo, ko, d):
    nr = lib.SageNormRope(1, 1e-6, None, None, lib.SAGE_FP32, None, 0, 0, 0)
    none = View(0, (0, 0, 0), (0, 0, 0))
    st = (ctypes.c_longlong * 12)(*(x for v in (q, k or none, qo, ko or none) for x in v.strides))
    return lib.capi.sage_qk_norm_rope(q.ptr, k.ptr if k else None, qo.ptr, ko.ptr if ko else None, st, None, 0, q.sizes[0],
                                      q.sizes[1], q.sizes[2], k.sizes[2] if k else 0, d, lib.SAGE_FP16, ctypes.byref(nr), None)


def _append(lib, q, k, v, qo, d, **arrays):
    a = dict(k8=FAKE + FAR, ks=FAKE + 2 * FAR, v8=FAKE + 3 * FAR, vs=FAKE + 4 * FAR)
    a.update(arrays)
    c = lib.SageKVCache(a["k8"], a["ks"], a["v8"], a["vs"], 4, 16, k.sizes[2], d)
    nr = lib.SageNormRope(1, 1e-6, None, None, lib.SAGE_FP32, None, 0, 0, 0)
    st = (ctypes.c_longlong * 8)(*(x for w in (q, k, v, qo) for x in w.strides[1:]))
    T = q.sizes[1]
    return lib.capi.sage_cache_append(ctypes.byref(c), q.ptr, k.ptr, v.ptr, qo.ptr, st, FAKE, 4, 4, FAKE, FAKE, None, T, 2,
                                      q.sizes[2], lib.SAGE_FP16, ctypes.byref(nr), None)


def _contiguous(at, B, N, H, d, layout="NHD"):
    return View(at, (N * H * d, H * d, d) if layout == "NHD" else (H * N * d, d, N * d), (B, N, H))


@pytest.mark.parametrize("B,N", [(1, 1), (1, 5), (3, 1), (3, 5)])
def test_slices_of_one_fused_tensor_go_in_place(lib, launched, B, N):
    Hq, Hkv, d = 4, 2, 8
    H = Hq + 2 * Hkv
    for strides in ((N * H * d, H * d, d), (H * N * d, d, N * d)):            # [tokens][heads] and [heads][tokens]
        q = View(0, strides, (B, N, Hq))
        k = View(Hq * strides[2], strides, (B, N, Hkv))
        assert _rows(lib, q, k, q, k, d) == launched and _rows(lib, k, q, k, q, d) == launched
    # each head's q and k next to each other; and as the two halves of wider channels
    for step in (3 * d, 2 * d):
        strides = (N * Hq * step, Hq * step, step)
        q, k = View(0, strides, (B, N, Hq)), View(d, strides, (B, N, Hq))
        assert _rows(lib, q, k, q, k, d) == launched
    # other memory
    far = _contiguous(1 << 30, B, N, Hq, d), _contiguous(1 << 31, B, N, Hkv, d)
    assert _rows(lib, q, _contiguous(1 << 20, B, N, Hkv, d), *far, d) == launched
    if B == 1:
        rows = (0, H * d, d)
        q, k, v = (View(at * d, rows, (1, N, n)) for at, n in ((0, Hq), (Hq, Hkv), (Hq + Hkv, Hkv)))
        assert _append(lib, q, k, v, q, d) == launched and _append(lib, q, k, v, far[0], d) == launched


def test_overlapping_outputs_are_refused(lib, launched):
    E, B, N, Hq, Hkv, d = lib.SAGE_ERR_INVALID_ARG, 2, 5, 4, 2, 8
    q, k = _contiguous(0, B, N, Hq, d), _contiguous(1 << 20, B, N, Hkv, d)
    qo, ko = _contiguous(1 << 30, B, N, Hq, d), _contiguous(1 << 31, B, N, Hkv, d)
    assert _rows(lib, q, k, qo, ko, d) == launched and _rows(lib, q, None, qo, None, d) == launched
    at = lambda v, n: View(v.at + n, v.strides, v.sizes)  # noqa: E731
    for args in ((q, k, at(k, 0), ko), (q, k, at(q, d), ko), (q, k, at(q, N * Hq * d), ko), (q, None, at(q, 1), None),
                 (q, k, qo, at(qo, 3)), (q, k, qo, q), (q, q, q, ko), (q, q, q, q),
                 (q, k, qo, _contiguous(q.at + B * N * Hq * d - 1, B, N, Hkv, d)),
                 (q, None, _contiguous(0, B, N, Hq, d, "HND"), None),         # the same memory in another order
                 (q, None, View(1 << 30, (N * Hq * d, d, d), (B, N, Hq)), None),           # tokens over heads
                 (q, None, View(1 << 30, (0, Hq * d, d), (B, N, Hq)), None),
                 (q, None, View(1 << 30, (N * Hq * d, Hq * d, d - 1), (B, N, Hq)), None)):
        assert _rows(lib, *args, d) == E
    t = [View(i << 20, (0, H * d, d), (1, N, H)) for i, H in enumerate((Hq, Hkv, Hkv, Hq))]
    assert _append(lib, *t, d) == launched
    for qo in (t[1], t[2], at(t[0], d), at(t[1], Hkv * d * N - 1), View(t[0].at, (0, d, d * N), (1, N, Hq))):
        assert _append(lib, t[0], t[1], t[2], View(qo.at, qo.strides, (1, N, Hq)), d) == E
    codes, scales = 4 * Hkv * 16 * 16, 4 * Hkv * 16 * 4                          # dc = 16
    base, size = FAKE + (1 << 36), N * Hq * d * 2
    qo = View((base - FAKE) // 2, t[3].strides, t[3].sizes)
    for name, n in (("k8", codes), ("ks", scales), ("v8", codes), ("vs", scales)):
        for start, want in ((base, E), (base + size - 16, E), (base - n + 16, E), (base + size, launched), (base - n, launched)):
            assert _append(lib, t[0], t[1], t[2], qo, d, **{name: start}) == want


def test_no_overlapping_views_pass(lib, launched):
    """Small random views: what shares a place is refused, whatever its strides; in place is not."""
    import random
    r, passed = random.Random(0), 0
    for _ in range(3000):
        B, N, Hq, Hkv, d = r.randint(1, 2), r.randint(1, 3), r.randint(1, 3), r.randint(1, 2), r.randint(1, 3)
        row = r.randint(1, 14)
        view = lambda H: View(r.randint(0, 30), r.choice([(r.randint(0, 40), row, r.randint(0, 6)),  # noqa: E731
                                                          (N * row, row, d), (r.randint(0, 40), r.randint(0, 14), row)]), (B, N, H))
        q, k, qo, ko = view(Hq), view(Hkv), view(Hq), view(Hkv)
        if r.random() < 0.3:
            qo = q
        if r.random() < 0.3:
            ko = k
        places = [v.places(d) for v in (q, k, qo, ko)]
        bad = len(set(places[2])) < len(places[2]) or len(set(places[3])) < len(places[3]) or \
            bool(set(places[2]) & set(places[3])) or bool(set(places[2]) & set(places[1])) or \
            bool(set(places[3]) & set(places[0])) or (places[2] != places[0] and bool(set(places[2]) & set(places[0]))) or \
            (places[3] != places[1] and bool(set(places[3]) & set(places[1])))  # (the same places in order: in place)
        got = _rows(lib, q, k, qo, ko, d)
        assert got in (launched, lib.SAGE_ERR_INVALID_ARG)
        assert not bad or got != launched, (vars(q), vars(k), vars(qo), vars(ko), d)
        passed += got == launched
    assert passed > 50
