"""sage_check_status with flags of several kernels: one report, and nothing left behind."""
import pytest
import torch

from tests import _serving as S

pytestmark = pytest.mark.gpu

F16 = torch.float16


def _flag_rows(lib):
    x = S.heads((2, 4, 64), F16, 0).cuda()
    lib.sage_qk_norm_rope(x, None, torch.tensor([0, 9], dtype=torch.int32).cuda(), torch.ones((8, 64), device="cuda"))


def _flag_decode(lib):
    cache = lib.sage_kv_cache(1, 1, 64, 16)
    zero = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    lib.sage_attn_decode(S.heads((1, 1, 64), F16, 0).cuda(), cache, zero, zero[0] - 1, 16)


def _flag_packed(lib):
    x = S.heads((8, 1, 64), F16, 0).cuda()
    cu = torch.tensor([0, 5, 3], dtype=torch.int32).cuda()
    lib.sage_attn_varlen(x, x, x, cu, cu, 8, 8)


@pytest.mark.parametrize("flags", [(_flag_rows,), (_flag_decode,), (_flag_packed,), (_flag_rows, _flag_decode, _flag_packed)])
def test_reported_once(lib, flags):
    lib.sage_check_status()
    for _ in range(2):
        for f in flags:
            f(lib)
        with pytest.raises(lib.SageError) as e:
            lib.sage_check_status()
        assert e.value.status == lib.SAGE_ERR_INVALID_ARG
        lib.sage_check_status()


@pytest.mark.parametrize("cu", [[0, -5], [0, 4, -1], [2, 0], [3, 3], [-1, 10], [0, 11], [0, 5, 3]])
def test_offset_tables_that_tokens_meet_are_reported(lib, cu):
    """Offsets that end below 0, or behind the tokens, or do not begin with 0, or fall: no place is written for what they
    say, and the call is reported, whichever token finds out."""
    T, B = 10, len(cu) - 1
    cache = S.poison(lib, 2 * B, 1, 64, 16)
    table = torch.arange(2 * B, dtype=torch.int32, device="cuda").view(B, 2)
    k = S.heads((T, 1, 64), F16, 0).cuda()
    cud, lens = torch.tensor(cu, dtype=torch.int32).cuda(), torch.full((B,), 12, dtype=torch.int32, device="cuda")
    for call in (lambda: lib.sage_cache_append(cache, k, k, table, lens, cud),
                 lambda: lib.sage_cache_gather(cache, table, cud, T, 64)):
        call()
        with pytest.raises(lib.SageError) as e:
            lib.sage_check_status()
        assert e.value.status == lib.SAGE_ERR_INVALID_ARG


def test_tokens_behind_the_last_sequence_are_no_fault(lib):
    cache = S.poison(lib, 1, 1, 64, 16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    k = S.heads((10, 1, 64), F16, 0).cuda()
    for cu, lens in ((i32(0, 0), i32(0)), (i32(0, 4), i32(4))):
        lib.sage_cache_append(cache, k, k, i32(0)[None], lens, cu)
        lib.sage_cache_gather(cache, i32(0)[None], cu, 10, 64)
        lib.sage_check_status()
    assert int((~cache["ks"].isnan()).sum()) == 4
