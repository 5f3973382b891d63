"""The serving operators on the GPU against plain 64-bit forms (oracle/serving.py): head norm and rotation, the paged
cache's write and read, one-token attention, and a run of them together.  Tolerances: tests/_serving.py."""
import math

import numpy as np
import pytest
import torch

from oracle import attention, serving
from tests import _serving as S

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


# ------------------------------------------------------------------------------------------ norm and rotation
ROWS = [  # layout, B, N, Hq, Hkv, d, rot, dtype, norm, weights, interleaved
    ("HND", 1, 1, 1, 1, 64, 64, F16, True, "same", False),
    ("NHD", 2, 5, 4, 2, 128, 128, BF16, True, "fp32", False),
    ("HND", 3, 17, 3, 1, 96, 48, F16, True, "none", False),      # part of the head rotated
    ("NHD", 1, 9, 2, 2, 256, 256, BF16, True, "same", True),
    ("HND", 2, 7, 5, 5, 80, 80, F16, False, "none", False),      # rotation alone; a half of 40 channels
    ("NHD", 2, 6, 2, 1, 40, 40, BF16, True, "same", False),      # halves of 20: the scalar path
    ("HND", 1, 8, 2, 2, 37, 10, F16, True, "fp32", True),        # an odd head size
    ("NHD", 1, 4, 3, 3, 1, 0, BF16, True, "same", False),        # one channel, no rotation
    ("packed", 1, 13, 6, 2, 128, 64, F16, True, "same", True),
    ("packed", 1, 400, 32, 8, 128, 128, BF16, True, "same", False),  # groups of four heads
    ("HND", 2, 1000, 9, 3, 64, 64, F16, True, "fp32", False),    # groups of four, the last of one head
    ("packed", 1, 3, 2, 2, 130, 2, BF16, True, "same", False),
    ("NHD", 1, 2400, 32, 32, 40, 20, F16, True, "fp32", False),  # rotated channels that are no multiple of eight,
    ("HND", 2, 1201, 32, 32, 48, 20, BF16, True, "same", True),  # four heads at a time
]


def _rows_case(case):
    layout, B, N, Hq, Hkv, d, rot, dt, norm, weights, inter = case
    if layout == "packed":
        rows = S.heads((N, Hq + 2 * Hkv, d), dt, 1).cuda()
        q, k = rows[:, :Hq], rows[:, Hq:Hq + Hkv]
    else:
        shape = (lambda H: (B, H, N, d)) if layout == "HND" else (lambda H: (B, N, H, d))
        q, k = S.heads(shape(Hq), dt, 1).cuda(), S.heads(shape(Hkv), dt, 2, 3.0).cuda()
    wt = {"none": None, "same": dt, "fp32": torch.float32}[weights]
    w = [None if wt is None else (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(3 + i))).to(wt).cuda()
         for i in range(2)]
    pos = np.random.RandomState(5).randint(0, 500, (B, N)).astype(np.int32)
    table = S.rope_table(500, rot) if rot else None
    return q, k, w, pos, table


def _tokens(t, layout):
    """(B, N, H, d) of any layout."""
    return t[None] if t.dim() == 3 else t.transpose(1, 2) if layout == "HND" else t


@pytest.mark.parametrize("case", ROWS, ids=lambda c: f"{c[0]}_b{c[1]}_n{c[2]}_h{c[3]}_{c[4]}_d{c[5]}_rot{c[6]}")
def test_norm_rope(lib, case):
    layout, B, N, Hq, Hkv, d, rot, dt, norm, weights, inter = case
    q, k, w, pos, table = _rows_case(case)
    cs = None if table is None else torch.from_numpy(table).cuda()
    pt = torch.from_numpy(pos if layout != "packed" else pos[0]).cuda() if rot else None
    lay = "HND" if layout == "HND" else "NHD"
    kw = dict(tensor_layout=lay, norm=norm, eps=1e-5, interleaved=inter)
    qo, ko = lib.sage_qk_norm_rope(q, k, pt, cs, w[0], w[1], **kw)
    lib.sage_check_status()
    for got, x, wt in ((qo, q, w[0]), (ko, k, w[1])):
        for b in range(B):
            S.check_norm_rope(_tokens(got, layout)[b], _tokens(x, layout)[b], dt, norm, 1e-5, wt, table, pos[b], inter)
    # q alone; and in place, on the caller's own (strided) tensors
    q2, none = lib.sage_qk_norm_rope(q, None, pt, cs, w[0], None, **kw)
    assert none is None and torch.equal(S.bits(q2), S.bits(qo))
    a, b = lib.sage_qk_norm_rope(q, k, pt, cs, w[0], w[1], q_out=q, k_out=k, **kw)
    lib.sage_check_status()
    assert a is q and b is k and torch.equal(S.bits(q), S.bits(qo)) and torch.equal(S.bits(k), S.bits(ko))


def test_norm_rope_default_positions_and_misaligned_rows(lib):
    table = torch.from_numpy(S.rope_table(50, 64)).cuda()
    x = S.heads((2, 3, 50, 64), F16, 1).cuda()
    a, _ = lib.sage_qk_norm_rope(x, None, None, table)
    b, _ = lib.sage_qk_norm_rope(x, None, torch.arange(50, dtype=torch.int32, device="cuda"), table)
    # the same rows from an odd address, through the scalar path, by an output of other strides
    wide = torch.zeros((2, 3, 50, 67), dtype=F16, device="cuda")
    wide[..., 3:] = x
    out = torch.full((2, 3, 50, 65), 7.0, dtype=F16, device="cuda")
    c, _ = lib.sage_qk_norm_rope(wide[..., 3:], None, None, table, q_out=out[..., :64])
    lib.sage_check_status()
    assert torch.equal(S.bits(a), S.bits(b))
    for bb in range(2):
        S.check_norm_rope(_tokens(c, "HND")[bb], _tokens(x, "HND")[bb], F16, True, 1e-6, None, S.rope_table(50, 64),
                          np.arange(50), False)
    assert (out[..., 64] == 7).all()


def test_norm_rope_bad_position_leaves_its_token_alone(lib):
    table = torch.from_numpy(S.rope_table(8, 64)).cuda()
    x = S.heads((5, 4, 64), F16, 1).cuda()
    pos = torch.tensor([0, 8, 3, -1, 7], dtype=torch.int32, device="cuda")
    out = torch.full_like(x, 7.0)
    lib.sage_qk_norm_rope(x, None, pos, table, q_out=out)
    with pytest.raises(lib.SageError) as e:
        lib.sage_check_status()
    assert e.value.status == lib.SAGE_ERR_INVALID_ARG
    good = [0, 2, 4]
    S.check_norm_rope(out[good], x[good], F16, True, 1e-6, None, S.rope_table(8, 64), pos.cpu().numpy()[good], False)
    assert (out[[1, 3]] == 7).all()


def test_norm_rope_special_values(lib):
    x = torch.zeros((6, 1, 64), dtype=BF16, device="cuda")
    x[1, 0, 3] = math.nan
    x[2, 0, 5] = math.inf
    x[3] = 1e-30            # the squares vanish: eps alone under the root
    x[4] = 3e38             # the squares overflow: the row becomes zeros, as in fp32
    y, _ = lib.sage_qk_norm_rope(x, None, eps=1e-6)
    lib.sage_check_status()
    assert (y[0] == 0).all() and y[1].isnan().all()
    assert y[2, 0, 5].isnan() and (y[2, 0, :5] == 0).all()
    assert (y[3].float() / 1e-27 - 1).abs().max() < 2.0 ** -6 and (y[4] == 0).all()


# ------------------------------------------------------------------------------------------ the cache
WRITES = [  # d, Hkv, page, lengths before, new tokens, dtype, k_mean
    (64, 2, 16, [0, 5, 16, 31], [1, 11, 16, 40], F16, False),
    (128, 8, 64, [0, 100], [300, 1], BF16, True),
    (96, 3, 32, [7], [90], F16, True),
    (40, 2, 16, [0, 3, 0], [20, 0, 33], BF16, False),   # padded channels; a sequence with nothing new
    (256, 1, 128, [130], [130], F16, True),
    (33, 2, 16, [1, 2], [17, 3], F16, True),             # the scalar path
    (16, 1, 1024, [1020], [10], BF16, False),
    (128, 8, 64, [10] * 3, [500, 700, 1000], F16, False),  # groups of four heads
]


def _write_case(case, seed=0):
    d, Hkv, ps, hist, new, dt, mean = case
    T = sum(new)
    k, v = S.heads((T, Hkv, d), dt, seed + 1), S.heads((T, Hkv, d), dt, seed + 2, 2.0)
    km = torch.randn((Hkv, d), generator=torch.Generator().manual_seed(seed + 3)) * 2 if mean else None
    lens = [h + n if n else h for h, n in zip(hist, new)]
    table, pages = S.page_table(lens, ps, seed + 4, extra=2)
    cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
    return k, v, km, lens, table, pages, cu


def _slots(cache, table, b, positions):
    ps = cache["ks"].shape[2]
    pos = torch.as_tensor(positions)
    page, slot = table[b].long()[pos // ps].cuda(), (pos % ps).cuda()
    return {n: cache[n][page, :, slot].cpu().numpy() for n in cache}


@pytest.mark.parametrize("case", WRITES, ids=lambda c: f"d{c[0]}_h{c[1]}_page{c[2]}")
def test_cache_write_and_read_bit_for_bit(lib, case):
    d, Hkv, ps, hist, new, dt, mean = case
    k, v, km, lens, table, pages, cu = _write_case(case)
    cache = S.poison(lib, pages, Hkv, d, ps)
    kmd = km.cuda() if mean else None
    # strided k and v (one fused tensor), two rows behind the last sequence
    T = sum(new)
    rows = torch.full((T + 2, 2 * Hkv, d), math.nan, dtype=dt)
    rows[:T, :Hkv], rows[:T, Hkv:] = k, v
    rows = rows.cuda()
    assert lib.sage_cache_append(cache, rows[:, :Hkv], rows[:, Hkv:], table.cuda(),
                                 torch.tensor(lens, dtype=torch.int32).cuda(), cu.cuda(), k_mean=kmd) is None
    lib.sage_check_status()
    want_k8, want_ks = serving.k_codes(S.np32(k), None if km is None else km.numpy())
    want_v8, want_vs = serving.v_codes(S.np32(v))
    written = torch.zeros(cache["ks"].shape, dtype=torch.bool)
    for b, n in enumerate(new):
        if not n:
            continue
        pos = np.arange(hist[b], hist[b] + n)
        got = _slots(cache, table, b, pos)
        at = slice(int(cu[b]), int(cu[b + 1]))
        assert (got["k8"][..., :d] == want_k8[at]).all() and (got["k8"][..., d:] == 0).all()
        assert (got["v8"][..., :d] == want_v8[at]).all() and (got["v8"][..., d:] == 0).all()
        assert (got["ks"] == want_ks[at]).all() and (got["vs"] == want_vs[at]).all()
        written[table[b].long()[torch.as_tensor(pos // ps)], :, torch.as_tensor(pos % ps)] = True
    rest = ~written.cuda()  # every other slot is as it was
    assert cache["ks"][rest].isnan().all() and cache["vs"][rest].isnan().all()
    assert (cache["k8"][rest] == 127).all() and (cache["v8"][rest] == 0x7F).all()
    # what was written, read back; two rows behind the last sequence stay as they were
    for out_dt in (F16, BF16):
        ko = torch.full((T + 2, Hkv, d), 7.0, dtype=out_dt, device="cuda")
        vo = ko.clone()
        lib.sage_cache_gather(cache, table.cuda(), cu.cuda(), T + 2, d, out_dt,
                              starts=torch.tensor(hist, dtype=torch.int32).cuda(), k_mean=kmd, k_out=ko, v_out=vo)
        lib.sage_check_status()
        rk, rv = serving.read(want_k8, want_ks, want_v8, want_vs, None if km is None else km.numpy())
        assert torch.equal(S.bits(ko[:T]), S.bits(torch.from_numpy(rk).to(out_dt).cuda()))
        assert torch.equal(S.bits(vo[:T]), S.bits(torch.from_numpy(rv).to(out_dt).cuda()))
        assert (ko[T:] == 7).all() and (vo[T:] == 7).all()


def test_cache_special_rows(lib):
    d, dt = 64, BF16
    k, v = S.heads((7, 1, d), dt, 1), S.heads((7, 1, d), dt, 2)
    k[0] = 0
    k[1, 0, 9] = math.nan
    k[2, 0, 1] = -math.inf
    k[3] = 1e-38               # below 2^-100: stored as zeros
    k[4] = 2.0 ** -100         # the smallest that is kept
    k[5, 0, 0] = 3e38
    v[0] = -0.0
    v[1, 0, 0] = math.inf
    v[2] = 2e-38
    v[5, 0, 3] = -3e38
    cache = S.poison(lib, 1, 1, d, 16)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    lib.sage_cache_append(cache, k.cuda(), v.cuda(), table, torch.tensor([7], dtype=torch.int32).cuda(),
                          torch.tensor([0, 7], dtype=torch.int32).cuda())
    lib.sage_check_status()
    for want, names in ((serving.k_codes(S.np32(k)), ("k8", "ks")), (serving.v_codes(S.np32(v)), ("v8", "vs"))):
        assert (cache[names[0]][0, 0, :7].cpu().numpy() == want[0][:, 0]).all()
        assert np.array_equal(cache[names[1]][0, 0, :7].cpu().numpy(), want[1][:, 0], equal_nan=True)


FUSED = [  # d, rot, Hq, Hkv, dtype, norm, interleaved, k_mean, lengths before, new
    (128, 128, 32, 8, F16, True, False, False, [500, 3, 77], None),           # a decode step: one token each
    (128, 64, 8, 2, BF16, True, True, True, [0, 40], [200, 9]),
    (80, 80, 6, 3, F16, False, False, True, [15], [33]),
    (40, 40, 4, 2, BF16, True, False, False, [0, 1], [5, 17]),                 # the scalar path
    (256, 128, 4, 4, F16, True, False, False, [9], [20]),
    (64, 0, 4, 1, F16, True, False, False, [0], [30]),                        # norm alone
    (40, 20, 16, 8, BF16, True, False, True, [0, 50], [2000, 700]),           # halves of 10, four heads at a time
    (128, 128, 32, 8, F16, True, False, True, [0, 100], [700, 400]),          # groups of four heads
]


@pytest.mark.parametrize("case", FUSED, ids=lambda c: f"d{c[0]}_rot{c[1]}_h{c[2]}_{c[3]}_new{c[9]}")
def test_cache_write_with_norm_and_rotation(lib, case):
    d, rot, Hq, Hkv, dt, norm, inter, mean, hist, new = case
    ps, step = 16, new is None
    new = new or [1] * len(hist)
    k, v, km, lens, table, pages, cu = _write_case((d, Hkv, ps, hist, new, dt, mean), 7)
    T = sum(new)
    rows = torch.cat([S.heads((T, Hq, d), dt, 9), k, v], 1).cuda()
    q, kd, vd = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    w = [(1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(3 + i))).to(dt) if norm else None for i in (0, 1)]
    wd = [x.cuda() if norm else None for x in w]
    table_cs = S.rope_table(max(lens), rot) if rot else None
    cs = torch.from_numpy(table_cs).cuda() if rot else None
    cache = S.poison(lib, pages, Hkv, d, ps)
    qo = lib.sage_cache_append(cache, kd, vd, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                               None if step else cu.cuda(), q=q, cos_sin=cs, q_weight=wd[0], k_weight=wd[1], norm=norm,
                               eps=1e-5, interleaved=inter, k_mean=km.cuda() if mean else None)
    lib.sage_check_status()
    pos = np.concatenate([np.arange(h, h + n) for h, n in zip(hist, new)])
    S.check_norm_rope(qo, q, dt, norm, 1e-5, w[0], table_cs, pos, inter)
    # the same q through sage_qk_norm_rope, bit for bit
    q2, _ = lib.sage_qk_norm_rope(q, None, torch.from_numpy(pos.astype(np.int32)).cuda() if rot else None, cs, wd[0], None,
                                  norm=norm, eps=1e-5, interleaved=inter)
    assert torch.equal(S.bits(q2), S.bits(qo))
    y, mag = serving.norm_rope(S.np32(k), norm, 1e-5, None if w[1] is None else S.np32(w[1]), table_cs, pos, inter)
    if mean:
        y, mag = y - km.numpy(), mag + np.abs(km.numpy())
    want_v8, want_vs = serving.v_codes(S.np32(v))
    for b, n in enumerate(new):
        got, at = _slots(cache, table, b, np.arange(hist[b], lens[b])), slice(int(cu[b]), int(cu[b + 1]))
        assert (got["v8"][..., :d] == want_v8[at]).all() and (got["vs"] == want_vs[at]).all()
        top = mag[at].max(-1, keepdims=True)
        ks = got["ks"].astype(np.float64)[..., None]
        assert (np.abs(ks[..., 0] * 127 - np.abs(y[at]).max(-1)) <= 2.0 ** -18 * top[..., 0]).all()
        err = np.abs(got["k8"][..., :d] * ks - y[at])
        assert (err <= ks / 2 + 2.0 ** -17 * top).all()


def test_append_decode_batch_with_empty_slots(lib):
    # one token per sequence; length 0 is an empty slot: nothing of it is written or reported
    lens = [3, 0, 1, 16, 0]
    table, pages = S.page_table(lens, 16, 0)
    cache = S.poison(lib, pages, 2, 64, 16)
    k, v = S.heads((5, 2, 64), F16, 1), S.heads((5, 2, 64), F16, 2)
    q, qo = S.heads((5, 4, 64), F16, 3).cuda(), torch.full((5, 4, 64), 7.0, dtype=F16, device="cuda")
    lib.sage_cache_append(cache, k.cuda(), v.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), q=q,
                          norm=True, q_out=qo)
    lib.sage_check_status()
    assert int((~cache["ks"].isnan()).sum()) == 3 * 2 and (qo[[1, 4]] == 7).all() and not (qo[[0, 2, 3]] == 7).any()


@pytest.mark.parametrize("bad", ["page", "negative page", "position", "long", "offsets", "table end"])
def test_append_and_gather_skip_and_report_bad_places(lib, bad):
    lens, new = [20, 40], [4, 6]
    table, pages = S.page_table(lens, 16, 0)
    cu = [0, 4, 10]
    if bad == "page":
        table[1, 2] = pages
    elif bad == "negative page":
        table[1, 2] = -1
    elif bad == "position":
        lens[1] = 3                      # six new tokens in a sequence of three
    elif bad == "long":
        lens[1] = 49 + 16                # beyond the table's three pages
    elif bad == "offsets":
        cu = [0, 12, 10]                 # decreasing
    else:
        table = table[:, :2].contiguous()  # positions 34 .. 39 are on the third page
    cache = S.poison(lib, pages, 2, 64, 16)
    k = S.heads((10, 2, 64), F16, 1).cuda()
    cud, ld, td = (torch.as_tensor(x, dtype=torch.int32).cuda() for x in (cu, lens, table))
    lib.sage_cache_append(cache, k, k.clone(), td, ld, cud)
    with pytest.raises(lib.SageError) as e:
        lib.sage_check_status()
    assert e.value.status == lib.SAGE_ERR_INVALID_ARG
    if bad != "offsets":                 # the good sequence is written, nothing of the bad one but valid positions
        got = _slots(cache, table, 0, np.arange(16, 20))
        assert (got["k8"] == serving.k_codes(S.np32(k[:4]))[0]).all()
        assert int((~cache["ks"].isnan()).sum()) == 2 * (4 + (3 if bad == "position" else 0))
    ko = torch.full((10, 2, 64), 7.0, dtype=F16, device="cuda")
    vo = ko.clone()
    starts = torch.tensor([16, 60 if bad in ("position", "long") else 34], dtype=torch.int32).cuda()
    lib.sage_cache_gather(cache, td, cud, 10, 64, F16, starts=starts, k_out=ko, v_out=vo)
    with pytest.raises(lib.SageError) as e:
        lib.sage_check_status()
    assert e.value.status == lib.SAGE_ERR_INVALID_ARG
    if bad != "offsets":
        assert not (ko[:4] == 7).any() and (ko[4:] == 7).all() and (vo[4:] == 7).all()


# ------------------------------------------------------------------------------------------ one-token attention
def _decode_setup(lib, lens, Hkv, d, ps, seed=0, k_amp=1.0, v_amp=1.0):
    seqs = S.random_sequences(lens, Hkv, d, seed, k_amp, v_amp)
    table, pages = S.page_table(lens, ps, seed, extra=1)
    cache = S.poison(lib, pages, Hkv, d, ps)
    S.fill(cache, table, lens, *seqs, d)
    return seqs, table.cuda(), cache, torch.tensor(lens, dtype=torch.int32).cuda()


DECODE = [  # d, Hq, Hkv, page, lengths, dtype
    (64, 1, 1, 16, [0, 1, 2, 15, 16, 17, 31, 33], F16),
    (128, 8, 2, 64, [63, 64, 65, 127, 128, 129, 0, 300], BF16),
    (128, 32, 8, 64, [1000], F16),
    (128, 4, 4, 16, [515, 3], F16),
    (96, 6, 2, 32, [100, 257], BF16),
    (80, 14, 2, 16, [77, 500], F16),        # seven heads to a kv head
    (40, 2, 2, 16, [50], BF16),
    (20, 3, 1, 128, [130], F16),
    (1, 2, 1, 16, [40], F16),
    (256, 16, 1, 64, [200, 1], F16),        # sixteen heads: two tiles
    (160, 9, 1, 256, [300], BF16),          # a tile of eight and one of one
    (256, 4, 2, 1024, [1025, 90], BF16),
    (64, 64, 2, 16, [33], BF16),            # four tiles
    (128, 32, 8, 64, [2049, 5000, 1], F16),  # split and joined, next to short ones
    (37, 5, 5, 16, [90, 16], F16),          # an odd head size
    (64, 16, 16, 16, [1, 500, 0, 300] * 10, F16),           # more pairs than CTAs run at a time, none split
    (128, 16, 16, 64, [700, 1, 0, 1500, 513, 64] * 6, BF16),  # shares of several short sequences
    (256, 8, 8, 16, [900, 3, 0, 2000] * 4, F16),
    (48, 6, 3, 32, [3000, 700], BF16),      # a CTA to each unit
]


@pytest.mark.parametrize("case", DECODE, ids=lambda c: f"d{c[0]}_h{c[1]}_{c[2]}_page{c[3]}_n{c[4][0]}")
def test_decode(lib, case):
    d, Hq, Hkv, ps, lens, dt = case
    seqs, table, cache, ld = _decode_setup(lib, lens, Hkv, d, ps)
    q = S.heads((len(lens), Hq, d), dt, 1).cuda()
    for bound in (max(lens), max(lens) + 1000):  # (more chunks than the sequences have)
        out = lib.sage_attn_decode(q, cache, table, ld, bound)
        lib.sage_check_status()
        S.check_decode(out, q, seqs, lens, 1 / math.sqrt(d))
    # a wide margin of scales: peaked and flat softmax
    for scale in (4.0, 1e-3):
        out = lib.sage_attn_decode(q, cache, table, ld, max(lens), sm_scale=scale)
        lib.sage_check_status()
        S.check_decode(out, q, seqs, lens, scale, f"scale {scale}")


def test_decode_strided_and_misaligned_queries(lib):
    lens, Hq, Hkv, d = [70, 30], 8, 2, 128
    seqs, table, cache, ld = _decode_setup(lib, lens, Hkv, d, 16)
    rows = S.heads((2, Hq + 3, d + 1), F16, 1).cuda()
    a = rows[:, 1:1 + Hq, 1:]                       # odd address, odd head stride
    b = S.heads((2, Hq + 2, d), F16, 2).cuda()[:, 2:]  # slice of a fused projection
    wide = torch.full((3, 2, 5), 0, dtype=torch.int32, device="cuda")
    wide[0, :, :table.shape[1]] = table[:, :5]
    for q in (a, b):
        out = lib.sage_attn_decode(q, cache, wide[0, :, :table.shape[1]], ld, 70)
        lib.sage_check_status()
        S.check_decode(out, q.contiguous(), seqs, lens, 1 / math.sqrt(d))


def test_decode_shared_pages_and_many_splits_agree(lib):
    # sixteen sequences over one prefix, of different lengths; every way of splitting it
    n, Hkv, Hq, d = 4000, 2, 8, 64
    seqs, table, cache, _ = _decode_setup(lib, [n], Hkv, d, 16)
    lens = [1 + (n - 1) * i // 15 for i in range(16)]
    q = S.heads((16, Hq, d), BF16, 1).cuda()
    many = table.expand(16, -1)
    with pytest.raises(lib.SageError):              # rows that overlap in memory: a stride of 0 < max_pages
        lib.sage_attn_decode(q, cache, many, torch.tensor(lens, dtype=torch.int32).cuda(), n)
    many = many.contiguous()
    out = lib.sage_attn_decode(q, cache, many, torch.tensor(lens, dtype=torch.int32).cuda(), n)
    lib.sage_check_status()
    S.check_decode(out, q, tuple([x[0]] * 16 for x in seqs), lens, 1 / 8)
    for b in (0, 7, 15):  # alone (other chunks): the same to the tolerance
        one = lib.sage_attn_decode(q[b:b + 1], cache, many[b:b + 1], torch.tensor([lens[b]], dtype=torch.int32).cuda(), n)
        S.check_decode(one, q[b:b + 1], tuple([x[0]] for x in seqs), [lens[b]], 1 / 8)
    again = lib.sage_attn_decode(q, cache, many, torch.tensor(lens, dtype=torch.int32).cuda(), n)
    assert torch.equal(S.bits(out), S.bits(again))


def test_decode_extreme_scales_and_values(lib):
    d, Hkv, ps = 64, 1, 16
    n = 200
    r = np.random.RandomState(0)
    k8, ks = serving.k_codes(r.randn(n, 1, d).astype(np.float32))
    # values whose scales span 2^80: each matters where its weight is large
    amp = np.exp2(r.randint(-60, 20, (n, 1, 1))).astype(np.float32)
    v8, vs = serving.v_codes((r.randn(n, 1, d) * amp).astype(np.float32))
    vs[5] = 0.0  # a value of zeros
    v8[5] = 0
    table, pages = S.page_table([n], ps, 0)
    cache = S.poison(lib, pages, Hkv, d, ps)
    S.fill(cache, table, [n], [k8], [ks], [v8], [vs], d)
    ld = torch.tensor([n], dtype=torch.int32).cuda()
    q = S.heads((1, 3, d), BF16, 1).cuda()
    for scale in (0.125, 3.0, 40.0):
        out = lib.sage_attn_decode(q, cache, table.cuda(), ld, n, sm_scale=scale)
        lib.sage_check_status()
        S.check_decode(out, q, ([k8], [ks], [v8], [vs]), [n], scale)
    # all values zero, all keys zero
    cache["vs"].zero_()
    assert (lib.sage_attn_decode(q, cache, table.cuda(), ld, n) == 0).all()
    k0 = np.zeros_like(k8)
    S.fill(cache, table, [n], [k0], [ks], [v8], [vs], d)
    out = lib.sage_attn_decode(q, cache, table.cuda(), ld, n)
    S.check_decode(out, q, ([k0], [ks], [v8], [vs]), [n], 0.125)
    lib.sage_check_status()


@pytest.mark.parametrize("which", ["ks", "vs"])
@pytest.mark.parametrize("n,at", [(40, 0), (40, 39), (3000, 1700)])
def test_decode_nan_token_makes_its_head_nan_and_no_other(lib, which, n, at):
    lens = [n, 50]
    seqs, table, cache, ld = _decode_setup(lib, lens, 2, 64, 16)
    page, slot = int(table[0, at // 16]), at % 16
    cache[which][page, 1, slot] = math.nan
    q = S.heads((2, 8, 64), F16, 1).cuda()
    out = lib.sage_attn_decode(q, cache, table, ld, max(lens))
    lib.sage_check_status()
    assert out[0, 4:].isnan().all()
    clean = [x.copy() for x in (seqs[0][0], seqs[1][0], seqs[2][0], seqs[3][0])]
    S.check_decode(out[1:], q[1:], tuple(x[1:] for x in seqs), lens[1:], 0.125)
    ok = S.np32(out[0, :4])
    ref, _, _ = serving.decode(S.np32(q[0]).astype(np.float64), clean[0] * clean[1].astype(np.float64)[..., None],
                               serving.fp8.decode(clean[2]) * clean[3].astype(np.float64)[..., None], 0.125)
    assert np.abs(ok - ref[:4]).max() < 2e-3


@pytest.mark.parametrize("bad", ["negative", "over max_seqlen", "over table"])
def test_decode_reports_bad_lengths_with_zeros(lib, bad):
    seqs, table, cache, ld = _decode_setup(lib, [40, 33], 1, 64, 16)
    q = S.heads((2, 2, 64), F16, 1).cuda()
    ld[0] = {"negative": -1, "over max_seqlen": 41, "over table": 16 * table.shape[1] + 1}[bad]
    bound = 40 if bad != "over table" else 10000
    out = lib.sage_attn_decode(q, cache, table, ld, bound, out=torch.full_like(q, 7.0))
    with pytest.raises(lib.SageError) as e:
        lib.sage_check_status()
    assert e.value.status == lib.SAGE_ERR_INVALID_ARG and (out[0] == 0).all()
    S.check_decode(out[1:], q[1:], tuple(x[1:] for x in seqs), [33], 0.125)


def test_decode_leaves_out_keys_on_bad_pages(lib):
    seqs, table, cache, ld = _decode_setup(lib, [64], 1, 64, 16)
    table[0, 2] = 1 << 30
    q = S.heads((1, 2, 64), F16, 1).cuda()
    out = lib.sage_attn_decode(q, cache, table, ld, 64)
    with pytest.raises(lib.SageError):
        lib.sage_check_status()
    keep = np.r_[0:32, 48:64]
    S.check_decode(out, q, tuple([x[0][keep]] for x in seqs), [48], 0.125)


def test_decode_empty_batch_and_zero_bound(lib):
    cache = lib.sage_kv_cache(2, 2, 64, 16)
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.ones((3, 4, 64), dtype=F16, device="cuda")
    assert lib.sage_attn_decode(q[:0], cache, torch.zeros((0, 2), **i32), torch.zeros(0, **i32), 10).shape == (0, 4, 64)
    out = lib.sage_attn_decode(q, cache, torch.full((3, 2), -1, **i32), torch.zeros(3, **i32), 0)
    lib.sage_check_status()
    assert (out == 0).all()


def test_offsets_past_32_bits(lib):
    """A cache whose codes, and whose rows' byte offsets, pass 2^32: pages at its far end."""
    d, Hkv, ps = 256, 8, 1024
    pages = (1 << 32) // (d * Hkv * ps) + 4          # 2052 pages, 4.3 GB of codes each for K and V
    cache = dict(k8=torch.empty((pages, Hkv, ps, d), dtype=torch.int8, device="cuda"),
                 v8=torch.empty((pages, Hkv, ps, d), dtype=torch.uint8, device="cuda"),
                 ks=torch.empty((pages, Hkv, ps), device="cuda"), vs=torch.empty((pages, Hkv, ps), device="cuda"))
    lens, new = [1030, 700], [40, 700]
    table = torch.tensor([[pages - 1, pages - 2], [pages - 3, -1]], dtype=torch.int32).cuda()
    T = sum(lens)
    k, v = S.heads((T, Hkv, d), BF16, 1).cuda(), S.heads((T, Hkv, d), BF16, 2).cuda()
    cu = torch.tensor([0, 1030, 1730], dtype=torch.int32).cuda()
    ld = torch.tensor(lens, dtype=torch.int32).cuda()
    lib.sage_cache_append(cache, k, v, table, ld, cu)
    ko, vo = lib.sage_cache_gather(cache, table, cu, T, d, BF16)
    lib.sage_check_status()
    k8, ks = serving.k_codes(S.np32(k))
    v8, vs = serving.v_codes(S.np32(v))
    rk, rv = serving.read(k8, ks, v8, vs)
    assert torch.equal(S.bits(ko), S.bits(torch.from_numpy(rk).to(BF16).cuda()))
    assert torch.equal(S.bits(vo), S.bits(torch.from_numpy(rv).to(BF16).cuda()))
    q = S.heads((2, Hkv, d), BF16, 3).cuda()
    out = lib.sage_attn_decode(q, cache, table, ld, 1030)
    lib.sage_check_status()
    S.check_decode(out, q, tuple([x[:1030], x[1030:]] for x in (k8, ks, v8, vs)), lens, 1 / 16)


# ------------------------------------------------------------------------------------------ streams and graphs
def test_decode_on_another_stream_and_two_at_once(lib):
    lens = [5000, 3]
    seqs, table, cache, ld = _decode_setup(lib, lens, 2, 64, 16)
    qs = [S.heads((2, 4, 64), F16, i).cuda() for i in range(2)]
    want = [lib.sage_attn_decode(q, cache, table, ld, 5000) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        got = []
        for s, q in zip(streams, qs):
            with torch.cuda.stream(s):
                got.append(lib.sage_attn_decode(q, cache, table, ld, 5000))
        torch.cuda.synchronize()
        assert all(torch.equal(S.bits(a), S.bits(b)) for a, b in zip(got, want))
    lib.sage_check_status()


def test_decode_step_captured_and_replayed(lib):
    """A decode step (append with norm and rotation, attention) in a graph: replays follow lengths and tokens that the
    caller writes into the captured buffers; two graphs in flight on two streams keep apart."""
    Hq, Hkv, d, ps, steps = 8, 2, 64, 16, 20
    hist = [30, 1500]
    table, pages = S.page_table([h + steps for h in hist], ps, 0)
    td, cs = table.cuda(), torch.from_numpy(S.rope_table(2000, d)).cuda()
    rows = S.heads((steps, 2, Hq + 2 * Hkv, d), F16, 1).cuda()
    seqs = S.random_sequences(hist, Hkv, d, 3)

    def state():
        cache = S.poison(lib, pages, Hkv, d, ps)
        S.fill(cache, table, hist, *seqs, d)
        return cache, torch.tensor(hist, dtype=torch.int32).cuda(), rows[0].clone(), torch.empty((2, Hq, d), dtype=F16,
                                                                                                device="cuda")

    def step(cache, lens, x, out):
        q = lib.sage_cache_append(cache, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], td, lens, q=x[:, :Hq], cos_sin=cs, norm=True)
        lib.sage_attn_decode(q, cache, td, lens, 2000, out=out)

    want, st = [], state()
    for i in range(steps):
        st[1].add_(1)
        st[2].copy_(rows[i])
        step(*st)
        want.append(st[3].clone())
    lib.sage_check_status()
    two = [state(), state()]
    graphs = []
    for s in two:
        s[1].add_(1)
        step(*s)  # warm-up: the first token (written again by the first replay)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            step(*s)
        s[1].sub_(1)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in two]
    torch.cuda.synchronize()
    for i in range(steps):
        for s, g, stream in zip(two, graphs, streams):
            with torch.cuda.stream(stream):
                s[1].add_(1)
                s[2].copy_(rows[i])
                g.replay()
        torch.cuda.synchronize()
        for s in two:
            assert torch.equal(S.bits(s[3]), S.bits(want[i])), i
    lib.sage_check_status()


@pytest.mark.parametrize("captured", [False, True])
def test_calls_see_what_the_work_just_before_them_wrote(lib, captured):
    """The kernels are set up while the work before them ends: lengths, queries and cache rows that it writes (a copy, a
    torch kernel, an append) are seen all the same.  Two states in turn, many times."""
    Hq, Hkv, d, ps = 8, 2, 128, 64
    lens = [[3000, 40, 700, 0], [200, 2900, 1, 1500]]
    table, pages = S.page_table([3000, 2900, 700, 1500], ps, 0)
    td = table.cuda()
    seqs = S.random_sequences([3000, 2900, 700, 1500], Hkv, d, 1)
    cache = S.poison(lib, pages, Hkv, d, ps)
    S.fill(cache, table, [3000, 2900, 700, 1500], *seqs, d)
    ld = [torch.tensor(x, dtype=torch.int32).cuda() for x in lens]
    rows = [S.heads((4, Hq + 2 * Hkv, d), F16, i).cuda() for i in range(2)]
    cu = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32).cuda()
    lens_now, rows_now, out = torch.empty_like(ld[0]), torch.empty_like(rows[0]), torch.empty((4, Hq, d), dtype=F16,
                                                                                             device="cuda")
    ko, vo = (torch.empty((4, Hkv, d), dtype=F16, device="cuda") for _ in range(2))

    def step(i):
        lens_now.copy_(ld[i])
        torch.mul(rows[i], 1.0, out=rows_now)
        q = lib.sage_cache_append(cache, rows_now[:, Hq:Hq + Hkv], rows_now[:, Hq + Hkv:], td, lens_now, q=rows_now[:, :Hq],
                                  norm=True)
        lib.sage_attn_decode(q, cache, td, lens_now, 3000, out=out)
        torch.sub(lens_now, 1, out=lens_now)
        lib.sage_cache_gather(cache, td, cu, 4, d, starts=lens_now.clamp(min=0), k_out=ko, v_out=vo)

    runs = [lambda i=i: step(i) for i in range(2)]
    want = []
    for i in (0, 1, 0, 1):  # (the appended rows settle in the first round)
        step(i)
        torch.cuda.synchronize()
        want.append([t.clone() for t in (out, ko, vo)])
    if captured:
        graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
        for i, g in enumerate(graphs):
            with torch.cuda.graph(g, stream=torch.cuda.Stream()):
                step(i)
        runs = [g.replay for g in graphs]
    got = []
    for _ in range(100):
        for i in range(2):
            runs[i]()
            got.append([t.clone() for t in (out, ko, vo)])
    lib.sage_check_status()
    for n, ts in enumerate(got):
        for a, b in zip(ts, want[2 + n % 2]):
            assert torch.equal(S.bits(a), S.bits(b)), n


# ------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("dt,mean", [(F16, False), (BF16, True)])
def test_prompt_chunk_and_steps_together(lib, dt, mean):
    """A prompt, a chunk behind it, and decode steps, as a server runs them; every answer against exact attention over
    the dequantized cache (decode) or over what the attention call was given (prompt, chunk)."""
    Hq, Hkv, d, ps = 8, 2, 128, 64
    n1, n2, steps = [200, 131, 90], [64, 1, 33], 3
    B = 3
    total = [a + b + steps for a, b in zip(n1, n2)]
    table, pages = S.page_table(total, ps, 0)
    td = table.cuda()
    cache = S.poison(lib, pages, Hkv, d, ps)
    cs = torch.from_numpy(S.rope_table(max(total), d)).cuda()
    w = [(1 + 0.2 * torch.randn(d, generator=torch.Generator().manual_seed(i))).to(dt).cuda() for i in range(2)]
    km = torch.randn((Hkv, d), generator=torch.Generator().manual_seed(9)).cuda() if mean else None
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    kw = dict(cos_sin=cs, q_weight=w[0], k_weight=w[1], norm=True, k_mean=km)

    def qkv(T, seed):
        r = S.heads((T, Hq + 2 * Hkv, d), dt, seed).cuda()
        return r[:, :Hq], r[:, Hq:Hq + Hkv], r[:, Hq + Hkv:]

    # prompts: written to the cache; attention over the 16-bit keys
    cu1 = i32([0] + list(np.cumsum(n1)))
    q, k, v = qkv(sum(n1), 1)
    qn = lib.sage_cache_append(cache, k, v, td, i32(n1), cu1, q=q, **kw)
    pos = torch.cat([torch.arange(n) for n in n1]).to(torch.int32).cuda()
    qr, kr = lib.sage_qk_norm_rope(q, k, pos, cs, w[0], w[1])
    assert torch.equal(S.bits(qr), S.bits(qn))
    o1 = lib.sage_attn_varlen(qn, kr, v.contiguous(), cu1, cu1, max(n1), max(n1), True, pv_dtype="fp16")
    # chunks: written, then attention over the whole prefix read back
    cu2, lens2 = i32([0] + list(np.cumsum(n2))), [a + b for a, b in zip(n1, n2)]
    cuk = i32([0] + list(np.cumsum(lens2)))
    q2, k2, v2 = qkv(sum(n2), 2)
    qn2 = lib.sage_cache_append(cache, k2, v2, td, i32(lens2), cu2, q=q2, **kw)
    kc, vc = lib.sage_cache_gather(cache, td, cuk, sum(lens2), d, dt, k_mean=km)
    o2 = lib.sage_attn_varlen(qn2, kc, vc, cu2, cuk, max(n2), max(lens2), True, pv_dtype="fp16")
    lib.sage_check_status()
    for o, qq, kk, vv, cq, ck in ((o1, qn, kr, v, cu1, cu1), (o2, qn2, kc, vc, cu2, cuk)):
        ref = attention.attention_varlen_f64(*(t.contiguous().cpu() for t in (qq, kk, vv)), cq.cpu().numpy(),
                                             ck.cpu().numpy(), True, 1 / math.sqrt(d))
        a, b = S.np32(o).astype(np.float64).ravel(), ref.ravel()
        assert a @ b / math.sqrt((a @ a) * (b @ b)) >= 0.999
    # the first rows of the prefix read back are the prompt's keys, to the codes' half step
    y = S.np32(kr[:n1[0]]) - (S.np32(km) if mean else 0)
    half = np.abs(y).max(-1, keepdims=True) / 127 / 2
    assert (np.abs(S.np32(kc[:n1[0]]) - S.np32(kr[:n1[0]])) <= half + 2 * S.U[dt] * (np.abs(S.np32(kr[:n1[0]])) + 1e-2)
            + 2.0 ** -14).all()
    # steps
    lens = lens2
    for i in range(steps):
        lens = [n + 1 for n in lens]
        q3, k3, v3 = qkv(B, 10 + i)
        qn3 = lib.sage_cache_append(cache, k3, v3, td, i32(lens), q=q3, **kw)
        out = lib.sage_attn_decode(qn3, cache, td, i32(lens), max(total))
        lib.sage_check_status()
        seqs = [[], [], [], []]
        for b in range(B):
            got = _slots(cache, table, b, np.arange(lens[b]))
            for s, name in zip(seqs, ("k8", "ks", "v8", "vs")):
                s.append(got[name])
        S.check_decode(out, qn3, seqs, lens, 1 / math.sqrt(d), f"step {i}")


# ------------------------------------------------------------------------------------------ refusals, checked build
def test_python_layer_refuses(lib):
    x = torch.zeros((2, 4, 64), dtype=F16, device="cuda")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = lib.sage_kv_cache(4, 4, 64, 16)
    table, lens, cu = i32(2, 2), i32(2), i32(3)
    cs = torch.zeros((8, 64), device="cuda")
    w = torch.zeros(64, dtype=F16, device="cuda")
    bad = [
        lambda: lib.sage_qk_norm_rope(x.double(), None), lambda: lib.sage_qk_norm_rope(x, x.bfloat16()),
        lambda: lib.sage_qk_norm_rope(x, x[:1]), lambda: lib.sage_qk_norm_rope(x[0], None),
        lambda: lib.sage_qk_norm_rope(x.transpose(1, 2), None), lambda: lib.sage_qk_norm_rope(x, x, lens, None),
        lambda: lib.sage_qk_norm_rope(x, x, lens.long(), cs), lambda: lib.sage_qk_norm_rope(x, x, i32(3), cs),
        lambda: lib.sage_qk_norm_rope(x, x, lens, cs.half()), lambda: lib.sage_qk_norm_rope(x, x, q_weight=w[:3]),
        lambda: lib.sage_qk_norm_rope(x, x, q_weight=w, norm=False),
        lambda: lib.sage_qk_norm_rope(x, x, q_weight=w, k_weight=w.float()),
        lambda: lib.sage_qk_norm_rope(x[None], None, tensor_layout="NDH"), lambda: lib.sage_qk_norm_rope(x, None, k_out=x),
        lambda: lib.sage_qk_norm_rope(x, None, q_out=x[:1]),
        lambda: lib.sage_cache_append(cache, x, x, table, lens.long()),
        lambda: lib.sage_cache_append(cache, x[:1], x[:1], table, lens),
        lambda: lib.sage_cache_append(cache, x[:, :2], x[:, :2], table, lens),
        lambda: lib.sage_cache_append(cache, x[..., :40], x[..., :40], table, lens),
        lambda: lib.sage_cache_append(cache, x, x, table, lens, cu[:2]),
        lambda: lib.sage_cache_append(cache, x, x, table.t(), lens),
        lambda: lib.sage_cache_append(cache, x, x, table, lens, k_mean=torch.zeros((4, 64), dtype=F16, device="cuda")),
        lambda: lib.sage_cache_append(cache, x, x, table, lens, q_out=x),
        lambda: lib.sage_cache_append({**cache, "ks": cache["ks"][:2]}, x, x, table, lens),
        lambda: lib.sage_cache_append({**cache, "v8": cache["v8"].char()}, x, x, table, lens),
        lambda: lib.sage_cache_gather(cache, table, cu, 4, 64, torch.float64),
        lambda: lib.sage_cache_gather(cache, table, cu, 4, 64, k_out=x),
        lambda: lib.sage_cache_gather(cache, table, lens, 4, 64), lambda: lib.sage_cache_gather(cache, table, cu, 4, 96),
        lambda: lib.sage_attn_decode(x[None], cache, table, lens, 4), lambda: lib.sage_attn_decode(x, cache, table[:1], lens, 4),
        lambda: lib.sage_attn_decode(x, cache, table, lens, 4, out=x.transpose(0, 1)),
        lambda: lib.sage_qk_norm_rope(x, None, q_out=x[:, :1].expand(2, 4, 64)),  # an output that overlaps itself
        lambda: lib.sage_qk_norm_rope(x, None, None, cs[:0]), lambda: lib.sage_attn_decode(x, cache, table, lens, 1 << 40),
        lambda: lib.sage_attn_decode(None, cache, table, lens, 4), lambda: lib.sage_cache_gather(cache, table, cu, -1, 64),
    ]
    accepted = []
    for i, f in enumerate(bad):
        try:
            f()
            accepted.append(i)
        except ValueError:
            pass
    assert not accepted
    for f in (lambda: lib.sage_qk_norm_rope(x.float(), None), lambda: lib.sage_cache_gather(cache, table, cu, 4, 64, torch.float32)):
        with pytest.raises(lib.SageError) as e:           # fp32: the library's answer, as for sage_attn
            f()
        assert e.value.status == lib.SAGE_ERR_UNSUPPORTED
    with pytest.raises(lib.SageError):                    # three heads for four of the cache
        lib.sage_attn_decode(x[:, :3], cache, table, lens, 4)
    with pytest.raises(lib.SageError):                    # the answer over the question
        lib.sage_attn_decode(x, cache, table, lens, 4, out=x)
    with pytest.raises(lib.SageError):                    # a rotation of more channels than a head has
        lib.sage_qk_norm_rope(x, x, lens, torch.zeros((8, 66), device="cuda"))
    with pytest.raises(lib.SageError):
        lib.sage_attn_decode(x, lib.sage_kv_cache(4, 4, 64, 48), table, lens, 4)


def test_narrowed_output_skips_and_reports_decode_stores(lib):
    # the extent ends inside the second sequence's output: its bytes stay, the first ones are the normal result
    checked = lib.load_checked()
    lens = [600, 700]
    _, table, cache, ld = _decode_setup(lib, lens, 2, 64, 16)
    q = S.heads((2, 4, 64), F16, 1).cuda()
    want = lib.sage_attn_decode(q, cache, table, ld, 700)
    lib.sage_check_status()
    out, limit = torch.full_like(q, 7.0), 4 * 64 * 2 + 100
    saved, lib.capi = lib.capi, checked
    checked.sage_test_out_limit(limit)
    try:
        lib.sage_attn_decode(q, cache, table, ld, 700, out=out)
        assert checked.sage_check_status(torch.cuda.current_stream().cuda_stream) == lib.SAGE_ERR_BOUNDS
    finally:
        checked.sage_test_out_limit(0)
        lib.capi = saved
    assert torch.equal(S.bits(out)[:limit], S.bits(want)[:limit])
    assert torch.equal(S.bits(out)[limit:], S.bits(torch.full_like(q, 7.0))[limit:])


def test_checked_build_serving_matches(lib):
    checked = lib.load_checked()
    d, Hq, Hkv, ps, lens, new = 96, 6, 2, 16, [40, 3000], [7, 33]
    seqs, table, cache, ld = _decode_setup(lib, lens, Hkv, d, ps)
    cu = torch.tensor([0, 7, 40], dtype=torch.int32).cuda()
    rows = S.heads((40, Hq + 2 * Hkv, d), F16, 1).cuda()
    cs = torch.from_numpy(S.rope_table(3000, d)).cuda()

    def run():
        c = {n: t.clone() for n, t in cache.items()}
        q, k = rows[:, :Hq], rows[:, Hq:Hq + Hkv]
        qo = lib.sage_cache_append(c, k, rows[:, Hq + Hkv:], table, ld, cu, q=q, cos_sin=cs, norm=True)
        qr, kr = lib.sage_qk_norm_rope(q, k, None, cs)
        ko, vo = lib.sage_cache_gather(c, table, torch.tensor([0, 40, 3040], dtype=torch.int32).cuda(), 3040, d)
        out = lib.sage_attn_decode(qo[:2], c, table, ld, 3000)
        return [qo, qr, kr, ko, vo, out, *c.values()]

    want = run()
    lib.sage_check_status()
    saved = lib.capi
    lib.capi = checked
    try:
        got = run()
        assert checked.sage_check_status(torch.cuda.current_stream().cuda_stream) == lib.SAGE_OK
    finally:
        lib.capi = saved
    assert all(torch.equal(S.bits(a), S.bits(b)) for a, b in zip(got, want))
