"""What the decoding entry points promise at their limits: the order of their work, values at the
ends of their types' ranges, scales of any size, and how far results may be off."""
import math

import pytest
import torch

from tests import decode_ref as R
from tests.test_gpu_decode import _no_device_error, fill, gen, lc, make_batch, make_cache  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- the order of the work

@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("new,group,length", [(1, 4, 100), (1, 1, 1), (16, 2, 90), (20, 1, 128), (0, 4, 50)])
def test_attention_is_done_when_its_last_kernel_is(lc, new, group, length, captured):  # noqa: F811
    """Calls whose tiles have one chunk each, so that no part is joined: many of them, one behind the
    other with one workspace and one output, and a reader of the output behind each."""
    D, heads, steps = 64, 3, 48
    q_start, kv_len, table, n_pages = make_batch([(new, length), (new, max(length // 2, new)), (new, new)], 32, 3)
    cache = make_cache(lc, n_pages, heads, 32, D, 4)
    fill(lc, cache, q_start, kv_len, table, 5)
    rows = 3 * new + 1
    qs = [torch.randn(rows, heads * group, D, generator=gen(6 + i), device="cuda").to(torch.bfloat16) for i in range(3)]
    max_new = max(new, 1)
    out, lse = torch.zeros_like(qs[0]), torch.zeros(rows, heads * group, device="cuda")
    ws = lc.kv8_attention_workspace(qs[0], cache, table, max_new)
    want = []
    for q in qs:
        lc.kv8_attention(q, cache, q_start, kv_len, table, max_new, out=out, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        want.append((out.clone(), lse.clone()))
    assert new == 0 or not torch.equal(want[0][1], want[1][1])  # (over one token out is its value, whatever q)
    seen = [torch.zeros(steps, *t.shape, dtype=t.dtype, device="cuda") for t in (out, lse)]

    def chain():
        for i in range(steps):
            lc.kv8_attention(qs[i % 3], cache, q_start, kv_len, table, max_new, out=out, lse=lse, workspace=ws)
            seen[0][i].copy_(out)
            seen[1][i].copy_(lse)

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            chain()
        for t in seen:
            t.zero_()
        graph.replay()
        graph.replay()
    else:
        chain()
    torch.cuda.synchronize()
    for i in range(steps):
        assert torch.equal(seen[0][i], want[i % 3][0]) and torch.equal(seen[1][i], want[i % 3][1]), i
