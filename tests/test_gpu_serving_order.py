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
