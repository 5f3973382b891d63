"""One-token attention with one key far above a long flat tail: the tail's keys weigh nothing one by one, and much together.

The weights of P V are fp16 above 2^-36 of a warp's largest: a key is off by 2^-36 of that weight at most, n / 4 keys of a warp
(a CTA's four warps share a sequence out evenly) by n 2^-38 max p |v| together.  With the values below that is under a quarter of
the term n / 8 2^-24 spread that S.check_decode takes for the fp32 sums (spread >= the tail's share >= n 2^-gap / 4, or p |v| of
the dominant key), for gaps up to 35."""
import math

import numpy as np
import pytest
import torch

from oracle import serving
from tests import _serving as S

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("gap,at", [(20.0, 0), (25.01, 0), (25.01, 100000), (28.0, 0)])
def test_a_dominant_key_and_a_long_flat_tail(lib, gap, at, dt):
    n, B, d, ps = 131072, 512, 64, 1024  # as many sequences (over the same pages) as keep a whole one in a CTA
    k8, ks = np.zeros((n, 1, d), np.int8), np.zeros((n, 1), np.float32)
    k8[at], ks[at] = 127, gap * math.log(2) / (127 * d / math.sqrt(d))  # queries of ones: `gap` powers of two above score 0
    v = np.ones((n, 1, d), np.float32)
    v[at, 0, 1:32], v[at, 0, 32:] = 0, 1 / 16
    v8, vs = serving.v_codes(v)
    table, pages = S.page_table([n], ps, 0)
    cache = S.poison(lib, pages, 1, d, ps)
    S.fill(cache, table, [n], [k8], [ks], [v8], [vs], d)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    q = torch.ones((B, 8, d), dtype=dt, device="cuda")
    out = lib.sage_attn_decode(q, cache, table.cuda().expand(B, -1).contiguous(), lens, n)
    lib.sage_check_status()
    some = [0, B - 1]
    S.check_decode(out[some], q[some], tuple([x] * len(some) for x in (k8, ks, v8, vs)), [n] * len(some), 1 / math.sqrt(d))
