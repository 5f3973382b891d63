"""The serving operators at the ends of their ranges of sizes."""
import pytest
import torch

from tests import _serving as S

pytestmark = pytest.mark.gpu

F16 = torch.float16


def test_decode_more_pairs_than_units_can_be_counted(lib):
    """65535 sequences of 3300 kv heads under a bound of 600 keys: so many pairs that the unit of work grows (its number stays
    below 2^31) until nothing is split.  Every output is written: the one value that is seen, or zero."""
    B, H = 65535, 3300
    assert B * H * (2 + 8) >= 2 ** 31 > B * H * (1 + 8)  # (two units of keys and eight of a pair's own time; one and eight)
    cache = lib.sage_kv_cache(1, H, 1, 1024)
    k = S.heads((1, H, 1), F16, 0).cuda()
    v = S.heads((1, H, 1), F16, 1).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    one = torch.ones(1, **i32)
    lib.sage_cache_append(cache, k, v, torch.zeros((1, 1), **i32), one)
    _, seen = lib.sage_cache_gather(cache, torch.zeros((1, 1), **i32), torch.tensor([0, 1], **i32), 1, 1)
    lens = torch.zeros(B, **i32)
    lens[::1000] = 1
    q = S.heads((1, H, 1), F16, 2).cuda().expand(B, H, 1)
    out = torch.full((B, H, 1), 7.0, dtype=F16, device="cuda")
    lib.sage_attn_decode(q, cache, torch.zeros((B, 1), **i32), lens, 600, out=out)
    lib.sage_check_status()
    assert torch.equal(out[::1000], seen.expand(len(out[::1000]), H, 1))
    out[::1000] = 0
    assert not out.any()
