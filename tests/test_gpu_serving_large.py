"""Head rows and the read back at sizes where a group of lanes takes four heads at a time (coded keys two), with head counts that
are no multiple of four, and writes so large that every CTA takes a share of each kind.  The checks are those of the small
cases; that a case is large enough is computed here from its sizes."""
import pytest
import torch

from tests import test_gpu_serving as small

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
SMS = 148


def _chunks(heads, at_a_time):
    return -(-heads // at_a_time)


def _lanes(d):
    return 8 if d <= 64 else 16 if d <= 128 else 32


def _four(tokens, heads, d):
    """Whether groups of four heads still give every SM 2048 threads: then a group takes four."""
    return d % 8 == 0 and tokens * sum(_chunks(h, 4) for h in heads) * _lanes(d) >= SMS * 2048


def _rounds(tokens, d, at_a_time):
    return -(-tokens // (128 // _lanes(d))) * sum(_chunks(h, n) for h, n in at_a_time)


SHARED = 8 * SMS * 6  # more rounds: each CTA works on all kinds

ROWS = [  # as of the small ones: layout, B, N, Hq, Hkv, d, rot, dtype, norm, weights, interleaved
    ("packed", 1, 6400, 6, 3, 128, 128, F16, True, "same", False),
    ("NHD", 2, 1600, 10, 7, 256, 64, BF16, True, "fp32", True),
    ("HND", 1, 7600, 9, 5, 64, 0, BF16, True, "same", False),
    ("NHD", 1, 5000, 5, 5, 96, 48, F16, True, "none", False),
]


@pytest.mark.parametrize("case", ROWS, ids=lambda c: f"{c[0]}_n{c[2]}_h{c[3]}_{c[4]}_d{c[5]}_rot{c[6]}")
def test_norm_rope(lib, case):
    _, B, N, Hq, Hkv, d = case[:6]
    assert _four(B * N, (Hq, Hkv), d)
    small.test_norm_rope(lib, case)


WRITES = [  # d, Hkv, page, lengths before, new tokens, dtype, k_mean; read back by four heads; shares of each kind
    (256, 3, 64, [5, 0, 100], [2500, 0, 2300], BF16, True, False, False),
    (128, 5, 16, [0, 33], [6000, 4000], F16, False, True, False),
    (256, 7, 128, [0, 77], [3000, 2000], F16, True, True, True),
]


@pytest.mark.parametrize("case", WRITES, ids=lambda c: f"d{c[0]}_h{c[1]}_page{c[2]}")
def test_cache_write_and_read_bit_for_bit(lib, case):
    d, Hkv, _, _, new, _, _, read, shared = case
    T = sum(new)
    assert _four(T, (Hkv, Hkv), d) and _four(T, (Hkv,), d) == read
    assert (_rounds(T, d, ((Hkv, 2), (Hkv, 4))) > SHARED) == shared
    small.test_cache_write_and_read_bit_for_bit(lib, case[:7])


FUSED = [  # d, rot, Hq, Hkv, dtype, norm, interleaved, k_mean, lengths before, new; shares of each kind
    (128, 128, 9, 5, F16, True, False, True, [0, 100], [1800, 1500], False),
    (256, 128, 5, 3, BF16, True, True, False, [3], [5800], True),
    (128, 128, 9, 5, F16, True, False, False, [0], [7200], True),
]


@pytest.mark.parametrize("case", FUSED, ids=lambda c: f"d{c[0]}_rot{c[1]}_h{c[2]}_{c[3]}_new{c[9]}")
def test_cache_write_with_norm_and_rotation(lib, case):
    d, _, Hq, Hkv, _, _, _, _, _, new, shared = case
    T = sum(new)
    assert _four(T, (Hq, Hkv, Hkv), d)
    assert (_rounds(T, d, ((Hq, 4), (Hkv, 2), (Hkv, 4))) > SHARED) == shared
    small.test_cache_write_with_norm_and_rotation(lib, case[:10])
