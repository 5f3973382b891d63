"""What follows a serving call in the stream, directly and without a synchronization: it sees the call's outputs and may
overwrite what the call read.  Results of calls in a row against those of the same calls with the device waited
for in between, bit for bit, eager and captured."""
import pytest
import torch

from tests import _serving as S

pytestmark = pytest.mark.gpu

F16 = torch.float16


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("B,n,bound", [(1, 100, 4096), (1, 200, 4096), (4, 256, 1024), (64, 50, 32768), (4, 600, 4096)])
def test_short_sequences_under_a_large_bound(lib, B, n, bound, captured):
    """The attention is launched for the bound, with a join; with short sequences no pair of the batch needs it (but in the
    last case).  Directly behind it its output is read by a dependent launch, and the rows that it read are overwritten."""
    Hq, Hkv, d, ps = 32, 8, 128, 64
    table, pages = S.page_table([bound] * B, ps, 0)
    td = table.cuda()
    cache = S.poison(lib, pages, Hkv, d, ps)
    ld = torch.full((B,), n, dtype=torch.int32, device="cuda")
    cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    rows = [S.heads((B * n, 2 * Hkv, d), F16, i).cuda() for i in range(2)]
    q = S.heads((B, Hq, d), F16, 5).cuda()

    def step(i, between):
        lib.sage_cache_append(cache, rows[i][:, :Hkv], rows[i][:, Hkv:], td, ld, cu)
        between()
        out = lib.sage_attn_decode(q, cache, td, ld, bound)
        between()
        normed, _ = lib.sage_qk_norm_rope(out, None)
        between()
        lib.sage_cache_append(cache, rows[1 - i][:, :Hkv], rows[1 - i][:, Hkv:], td, ld, cu)
        return out, normed

    want = [step(i, torch.cuda.synchronize) for i in range(2)]
    lib.sage_check_status()
    assert not torch.equal(want[0][0], want[1][0])
    runs = [lambda i=i: step(i, lambda: None) for i in range(2)]
    if captured:
        graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
        for i, g in enumerate(graphs):
            with torch.cuda.graph(g, stream=torch.cuda.Stream()):
                outs.append(step(i, lambda: None))

        def replay(i):
            graphs[i].replay()
            return outs[i]
        runs = [lambda i=i: replay(i) for i in range(2)]
    got = []
    for _ in range(50):
        for i in range(2):
            got.append([t.clone() for t in runs[i]()])
    lib.sage_check_status()
    for j, ts in enumerate(got):
        for a, b in zip(ts, want[j % 2]):
            assert torch.equal(S.bits(a), S.bits(b)), j


def test_a_packed_batch_without_keys_before_other_calls(lib):
    """Queries that see no key get zeros, and the passes behind the first have nothing to do: the call's workspace, and the
    queries that the first pass reads, belong to the next call only when that pass has ended."""
    H, d, n = 16, 128, 8192
    q = S.heads((4 * n, H, d), F16, 0).cuda()
    none = torch.zeros((1, H, d), dtype=F16, device="cuda")  # a row that no sequence owns
    cu = torch.arange(0, 4 * n + 1, n, dtype=torch.int32, device="cuda")
    x = [S.heads((1, H, 1024, d), F16, i).cuda() for i in range(1, 4)]
    want = lib.sage_attn(*x)
    torch.cuda.synchronize()
    for _ in range(20):
        zeros = lib.sage_attn_varlen(q, none, none, cu, torch.zeros_like(cu), n, 0)
        got = lib.sage_attn(*x)
        assert torch.equal(S.bits(got), S.bits(want)) and not zeros.any()
    lib.sage_check_status()
