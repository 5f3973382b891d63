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
