"""Calls at the limits of the operators around the loop: rows without pages for them, nothing to do at all,
many requests of which few have rows, groups of heads that fill no half."""
import math

import pytest
import torch

from tests import loop_ref as R
from tests.test_gpu_cross import check, i32, make
from tests.test_gpu_pages import count, make_caches, pool, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lc():
    import __graft_entry__
    __graft_entry__.build()
    import draft_block_candidate_gb300 as lc
    lc.device_error()
    return lc


@pytest.fixture(autouse=True)
def _no_device_error(lc):
    yield
    assert lc.device_error() == 0


@pytest.mark.parametrize("batch,beams,cols,page,new,spare", [
    (1, 4, 3, 16, 40, 3), (3, 5, 9, 32, 70, 6), (40, 16, 5, 16, 64, 100), (2, 32, 300, 16, 30, 20), (1, 3, 260, 16, 1500, 60)])
def test_grow_leaves_a_refused_row_as_it_was(lc, batch, beams, cols, page, new, spare):
    """Any negative entry is none, and a row without pages for all its tokens keeps the one it had."""
    g = torch.Generator().manual_seed(cols)
    refs, table, kv_len = pool(batch, beams, cols, page, spare, cols, capacity=cols + new // page + 2)
    refs[(refs == 0).nonzero()[spare:]] = 1  # (pages of others)
    none = -torch.randint(1, 50, table.shape, generator=g, dtype=torch.int32)
    none[torch.rand(table.shape, generator=g) < 0.1] = -(1 << 31)
    table = torch.where(table < 0, none, table)
    add = torch.randint(0, new + 1, kv_len.shape, generator=g, dtype=torch.int32)
    flat = table.view(batch * beams, -1)
    want = R.grow(refs, flat, kv_len.flatten(), add.flatten(), page)
    assert not want[3].all()
    refs, table = refs.cuda(), table.cuda()
    tail, granted = lc.kv8_grow(refs, table, kv_len.cuda(), add.cuda(), page, new)
    assert same(refs, want[0]) and same(table.view(batch * beams, -1), want[1])
    assert same(tail.flatten(), want[2]) and same(granted.flatten(), want[3])


def test_adjust_without_rows_or_tokens(lc):
    f32 = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    words = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    for x in (f32(0, 100), f32(4, 0, 100), f32(0, 3, 100)):
        assert lc.adjust_logits(x) is x
        assert lc.adjust_logits(x, mask=words, mask_index=e) is x
        assert lc.adjust_logits(x, mask=words[:0]) is x
        assert lc.adjust_logits(x, history=e.view(0, 1), seen=e, presence=f32(0), bias_ids=e.view(0, 2), bias_values=f32(0, 2)) is x
        out = torch.empty_like(x)
        assert lc.adjust_logits(x, out=out) is out
    x = f32(3, 0)
    assert lc.adjust_logits(x, mask=words[:, :0]) is x


def test_adjust_takes_what_lies_between_the_rows(lc):
    """What is read may lie behind a row's last token, but not among those that are written."""
    g = torch.Generator(device="cuda").manual_seed(3)
    buf = torch.zeros(8, 1024, dtype=torch.bfloat16, device="cuda")
    x = buf[:, :1000]
    x.copy_(torch.randn(8, 1000, generator=g, device="cuda"))
    history = torch.randint(0, 1000, (2, 40), generator=g, device="cuda", dtype=torch.int32)
    seen, penalty = i32(3, 40, 0, 7, 22, 40, 1, 39), torch.tensor([0.5, 1.5], device="cuda")
    want = lc.adjust_logits(x, history=history, seen=seen, presence=penalty, out=torch.empty_like(x))
    raw = buf.view(torch.uint8).flatten()
    there = raw[3 * 2048 + 2000:][:32].view(torch.int32)
    there.copy_(seen)
    lc.adjust_logits(x, history=history, seen=there, presence=penalty)
    assert torch.equal(x, want) and torch.equal(there, seen)
    for at in (3 * 2048 + 1996, 3 * 2048 + 2020, 0):
        with pytest.raises(lc.LilicorrError):
            lc.adjust_logits(x, history=history, seen=raw[at:][:32].view(torch.int32), presence=penalty)


def test_pages_without_rows(lc):
    refs = torch.ones(5, dtype=torch.int32, device="cuda")
    for lead in ((0,), (4, 0), (0, 3)):
        table, n = torch.zeros(*lead, 6, dtype=torch.int32, device="cuda"), torch.zeros(lead, dtype=torch.int32, device="cuda")
        tail, granted = lc.kv8_grow(refs, table, n, n, 16, 1)
        assert tail.shape == granted.shape == lead
        lc.kv8_free(refs, table, n, 16)
        caches = make_caches(lc, 1, 5, 1, 16, 32, 1)
        assert lc.kv8_compact(caches, refs, [table]).tolist() == [5]
    assert refs.tolist() == [1] * 5


def test_cross_without_states(lc):
    """Keys and values of no states: rows of requests have out 0 and lse -inf, whoever asks for states is reported."""
    q = torch.randn(6, 4, 64, device="cuda").to(torch.bfloat16)
    k = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    check(lc, q, k, k, i32(0, 2, 5), i32(0, 0), i32(0, 0), 3)
    new, lse = lc.cross_attention(q, k, k, i32(0, 2, 5), i32(0, 0), i32(0, 0), 3, lse=True)
    assert not new.any() and bool((lse == R.NEG).all())
    for start, length in ((0, 1), (1, 0), (-1, 1), (-1, 0), (0, -1)):
        out = torch.full_like(q, 7)
        lc.cross_attention(q, k, k, i32(0, 2, 5), i32(start, 0), i32(length, 0), 3, out=out)
        assert lc.device_error() == 1 << 26
        assert bool((out[:2] == 7).all()) and not out[2:5].any() and bool((out[5] == 7).all())


@pytest.mark.parametrize("rows", [1, 129])
@pytest.mark.parametrize("D", [64, 128])
def test_cross_sums_keep_small_weights_beside_a_heavy_one(lc, rows, D):
    """Weights below half a step of the heavy one's, which come to 2^-8 of it together: the sum of a row takes
    128 of them at a time, so it is off by (T / 128 + 8) 2^-24 at most, and its logarithm, with the score's
    2^-22 and a few roundings below 2^-20, too.  As many requests as keep each tile on one part of the GPU."""
    T, batch, score = 65536, 304, 16.75  # (a product that bf16 and f32 hold: 8 times that, by 1 / 8)
    k = torch.zeros(T, 1, D, dtype=torch.bfloat16, device="cuda")
    k[0, 0, 0] = score
    v = torch.ones_like(k)
    q = torch.zeros(batch * rows, 1, D, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 8
    start = torch.zeros(batch, dtype=torch.int32, device="cuda")
    q_start = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * rows
    out, lse = lc.cross_attention(q, k, v, q_start, start, start + T, rows, scale=0.125, lse=True)
    assert bool(((out.double() - 1).abs() <= 2.0 ** -8 + (T / 128 + 8) * 2.0 ** -24).all())
    want = score + torch.log1p((T - 1) * torch.tensor(-score).double().exp()).item()
    assert (lse.double() - want).abs().max() <= (T / 128 + 8) * 2.0 ** -24 + 2.0 ** -22 * score + 2.0 ** -24 * want + 2.0 ** -20


MANY = 1 << 20


def sparse(rows, lens, device="cuda"):
    """(q_start, lengths) of 2^20 requests of which a few, far apart, have rows."""
    at = torch.linspace(0, MANY - 1, len(rows)).long()
    n, t = torch.zeros(MANY, dtype=torch.long), torch.zeros(MANY, dtype=torch.int32)
    n[at], t[at] = torch.tensor(rows), torch.tensor(lens, dtype=torch.int32)
    return at, torch.cat([torch.zeros(1, dtype=torch.long), n.cumsum(0)]).int().to(device), t.to(device)


def test_cross_many_requests_without_rows(lc):
    """Runs of work that go on behind hundreds of thousands of requests without any."""
    rows, lens = [2, 300, 1, 3], [70000, 129, 1, 90000]
    q, k, v, few_start, kv_start, kv_len = make(list(zip(rows, lens)), 2, 2, 64, 5)
    at, q_start, length = sparse(rows, lens)
    start = torch.zeros(MANY, dtype=torch.int32, device="cuda")
    start[at.cuda()] = kv_start
    want = lc.cross_attention(q, k, v, few_start, kv_start, kv_len, 300)
    assert torch.equal(lc.cross_attention(q, k, v, q_start, start, length, 300), want)


@pytest.mark.parametrize("new", [2, 40])
def test_cache_attention_many_requests_without_rows(lc, new):
    rows, lens, cols = [new, 1, new - 1], [31900, 128, 30000], 250
    cache = make_caches(lc, 1, 500, 4, 128, 64, 2)[0]
    for t in (cache.k, cache.v):  # (no NaN among the codes)
        b = t.view(torch.uint8)
        b[(b & 127) == 127] = 3
    q = torch.randn(sum(rows), 4, 64, device="cuda").to(torch.bfloat16)
    at, q_start, length = sparse(rows, lens)
    pages = torch.randperm(500, generator=torch.Generator().manual_seed(1)).int().cuda()
    small = torch.stack([pages[:cols], pages[:cols].flip(0), pages[cols:2 * cols]])
    table = torch.full((MANY, cols), -1, dtype=torch.int32, device="cuda")
    table[at.cuda()] = small
    want = lc.kv8_attention(q, cache, i32(0, *torch.tensor(rows).cumsum(0).tolist()), i32(*lens), small, new)
    assert torch.equal(lc.kv8_attention(q, cache, q_start, length, table, new), want)


def test_cross_tiles_that_take_longer_than_a_wait(lc):
    """A CTA's first tile holds the places of q of its second one for more than a second."""
    n, rows = 144 << 20, 228 * 256
    k, v = (torch.full((n, 1, 8), x, dtype=torch.bfloat16, device="cuda") for x in (0.0, 1.0))
    q = torch.ones(rows, 1, 8, dtype=torch.bfloat16, device="cuda")
    out, lse = lc.cross_attention(q, k, v, i32(0, rows), i32(0), i32(n), rows, lse=True)
    # The tensor cores drop what a product has 2^-25 below the first bit of the sum that it is added to: weights of 1
    # are added up exactly to 2^26, and from there on not at all.
    assert bool(((out >= (1 - 2.0 ** -8) * 2.0 ** 26 / n) & (out <= 1)).all())
    assert (lse.double() - math.log(n)).abs().max() <= (n / 128 + 8) * 2.0 ** -24


def test_cache_attention_tiles_that_take_longer_than_a_wait(lc):
    """The outputs of a tile are waited for while its tokens are gone over."""
    D, page = 32, 128
    n, rows = 140 << 20, 228 * 128
    cache = lc.KV8Cache(1, 1, page, D)
    cache.k.view(torch.uint8).fill_(0)
    cache.v.view(torch.uint8).fill_(0x38)  # 1
    cache.k_scale.fill_(1)
    cache.v_scale.fill_(1)
    table = torch.zeros(1, n // page, dtype=torch.int32, device="cuda")
    q = torch.ones(rows, 1, D, dtype=torch.bfloat16, device="cuda")
    out, lse = lc.kv8_attention(q, cache, i32(0, rows), i32(n), table, rows, lse=True)
    assert bool(((out >= (1 - 2.0 ** -8) * 2.0 ** 26 / n) & (out <= 1)).all())  # (as above)
    seen = torch.arange(n - rows + 1, n + 1, device="cuda").double()
    assert (lse[:, 0].double() - seen.log()).abs().max() <= (n / 16 + 40) * 2.0 ** -24


@pytest.mark.parametrize("group", [43, 47, 65, 95])
@pytest.mark.parametrize("D,scale", [(64, 0.2), (64, -0.3), (128, 0.1), (80, -0.15)])
def test_cross_groups_whose_tokens_straddle_halves_and_tiles(lc, group, D, scale):
    check(lc, *make([(9, 300), (1, 40), (13, 129), (0, 7), (3, 1), (6, 700)], 2, group, D, group), 13, scale=scale)


@pytest.mark.parametrize("group", [1, 4, 3])
def test_cross_requests_of_the_same_states_under_a_negative_scale(lc, group):
    q, k, v, *_ = make([(5, 300), (140, 200), (9, 100)], 2, group, 64, group)
    check(lc, q, k, v, i32(0, 5, 145, 154), i32(7, 7, 60), i32(290, 290, 237), 140, scale=-0.25)


def test_grow_and_the_append_that_takes_its_tails_replayed(lc):
    """Captured together and replayed for three tokens: forked rows leave a shared tail page, whose tokens go with them."""
    page, D, heads, beams = 16, 32, 2, 3

    def state():
        table = torch.full((beams, 4), -1, dtype=torch.int32, device="cuda")
        table[:, 0] = 2
        refs, n = count(table.cpu(), 12).cuda(), torch.full((beams,), 14, dtype=torch.int32, device="cuda")
        return refs, table, n, make_caches(lc, 1, 12, heads, page, D, 9)[0]

    one, q_start = torch.ones(beams, dtype=torch.int32, device="cuda"), i32(*range(beams + 1))
    ws = lc.kv8_pages_workspace(12, beams)
    kv = torch.randn(3, 2, beams, heads, D, device="cuda").to(torch.bfloat16)

    def step(refs, table, n, cache, k, v, out):
        lc.kv8_grow(refs, table, n, one, page, 1, out=out, workspace=ws)
        n.add_(1)
        lc.kv8_append(cache, k, v, q_start, n, table, 1, tail_src=out[0])

    runs = []
    for captured in (False, True):
        s = state()
        k, v = torch.empty_like(kv[0, 0]), torch.empty_like(kv[0, 0])
        out = torch.empty(beams, dtype=torch.int32, device="cuda"), torch.empty(beams, dtype=torch.bool, device="cuda")
        if captured:
            spare = state()
            step(*spare, k, v, out)
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                step(*s, k, v, out)
        tails = []
        for i in range(3):
            k.copy_(kv[i, 0]), v.copy_(kv[i, 1])
            gr.replay() if captured else step(*s, k, v, out)
            tails.append(out[0].tolist())
            assert out[1].all()
        assert tails == [[2] * beams, [-1] * beams, [-1] * beams]
        runs.append(s)
    (ra, ta, na, ca), (rb, tb, nb, cb) = runs
    assert torch.equal(ra, rb) and torch.equal(ta, tb) and na.tolist() == nb.tolist() == [17] * beams
    assert ta.tolist() == [[0, 2, -1, -1], [1, 4, -1, -1], [3, 5, -1, -1]]  # (page 2 fell free at the first token)
    for x, y in zip((ca.k, ca.v, ca.k_scale, ca.v_scale), (cb.k, cb.v, cb.k_scale, cb.v_scale)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("mask_alone", [False, True])
def test_adjust_more_rows_than_a_grid_holds_side_by_side(lc, inplace, mask_alone):
    rows, V = 70001, 37
    g = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn(rows, V, generator=g, device="cuda")
    masks = torch.randint(-(1 << 31), 1 << 31, (3, 2), generator=g, device="cuda").int()
    index = torch.randint(-1, 3, (rows,), generator=g, device="cuda").int()
    allowed = ((masks[:, :, None] >> torch.arange(32, device="cuda")) & 1).view(3, 64)[:, :V].bool()
    allowed = torch.cat([allowed, torch.ones(1, V, dtype=torch.bool, device="cuda")])[index.long()]
    kw, want = {}, x.double()
    if not mask_alone:
        history = torch.randint(0, V, (rows, 3), generator=g, device="cuda").int()
        seen = torch.randint(0, 4, (rows,), generator=g, device="cuda").int()
        kw = dict(history=history, seen=seen, frequency=torch.rand(rows, generator=g, device="cuda"))
        there = torch.arange(3, device="cuda") < seen[:, None]
        want = want - torch.zeros_like(want).scatter_add_(1, history.long(), there.double()) * kw["frequency"].double()[:, None]
    want = torch.where(allowed, want, R.NEG)
    got = lc.adjust_logits(x, mask=masks, mask_index=index, out=None if inplace else torch.empty_like(x), **kw)
    assert (got is x) == inplace
    inside = allowed & want.isfinite()
    assert bool((got[~inside] == R.NEG).all())
    # a sum of at most two terms of up to 3 x 1 and 6 in all, off by 2^-46 of each, rounded once
    assert ((got.double() - want).abs()[inside] <= 2.0 ** -24 * want.abs()[inside] + 2.0 ** -42).all()


@pytest.mark.parametrize("layers,n_tables", [(1, 19), (35, 3), (17, 8), (16, 9)])
def test_compact_more_tables_and_caches_than_a_launch_takes(lc, layers, n_tables):
    n = 60
    g = torch.Generator().manual_seed(layers)
    caches = make_caches(lc, layers, n, 1, 16, 32, 3)
    pages = torch.randperm(n, generator=g)[:31].int()
    flat = torch.full((n_tables * 20,), -1, dtype=torch.int32)
    flat[torch.randperm(flat.numel(), generator=g)[:31]] = pages
    tables = [t.clone() for t in flat.view(n_tables, 2, 10)]
    refs = count(flat, n)
    wrefs, wtab, moves, live = R.compact(refs, tables)
    want = [[t.clone() for t in (c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale)] for c in caches]
    for parts in want:
        for t in parts:
            for a, b in moves:
                t[b] = t[a]
    refs, tables = refs.cuda(), [t.cuda() for t in tables]
    assert lc.kv8_compact(caches, refs, tables).tolist() == [live]
    assert same(refs, wrefs) and all(same(t, w) for t, w in zip(tables, wtab))
    for c, w in zip(caches, want):
        assert all(torch.equal(x, y) for x, y in zip((c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale), w))
