"""The pages of the 8-bit cache that sequences share, against the plain forms in loop_ref: whole
numbers and moved bytes, equal to the last bit."""
import pytest
import torch

from tests import loop_ref as R

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


def count(table, n_pages):
    return torch.bincount(table[table >= 0].long(), minlength=n_pages).to(torch.int32)


def pool(batch, beams, cols, page, spare, seed, capacity=None):
    """(refs, table, kv_len) on the CPU: beams of a batch entry share a part of their pages."""
    g = torch.Generator().manual_seed(seed)
    n = batch * beams * cols + spare
    order = torch.randperm(n, generator=g).to(torch.int32)
    table = torch.full((batch, beams, capacity or cols + 3), -1, dtype=torch.int32)
    kv_len = torch.zeros(batch, beams, dtype=torch.int32)
    at = 0
    for b in range(batch):
        length = int(torch.randint(0, cols * page + 1, (1,), generator=g))
        held = -(-length // page)
        shared = int(torch.randint(0, held + 1, (1,), generator=g))
        table[b, :, :shared] = order[at:at + shared]
        at += shared
        for j in range(beams):
            table[b, j, shared:held] = order[at:at + held - shared]
            at += held - shared
        kv_len[b] = length
    return count(table, n), table, kv_len


def same(got, want):
    return torch.equal(got.cpu(), want)


@pytest.mark.parametrize("batch,beams,cols", [(1, 1, 1), (2, 3, 5), (3, 4, 130), (5, 7, 20), (2, 16, 129), (1, 32, 300), (4, 9, 1)])
def test_fork_matches_reference(lc, batch, beams, cols):
    refs, table, _ = pool(batch, beams, cols, 16, 5, cols)
    parent = torch.randint(0, beams, (batch, beams), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    want = R.fork(refs, table, parent)
    refs, table = refs.cuda(), table.cuda()
    lc.kv8_fork(refs, table, parent.cuda())
    assert same(refs, want[0]) and same(table, want[1])
    assert same(refs, count(want[1], refs.shape[0]))


def test_fork_strided_tables_and_bad_parents(lc):
    refs, table, _ = pool(3, 4, 40, 16, 5, 2)
    wide = torch.full((3, 6, table.shape[2] + 9), 77, dtype=torch.int32).cuda()
    view = wide[:, 1:5, 2:2 + table.shape[2]]
    view.copy_(table)
    parent = torch.tensor([[1, 0, 9, -1], [3, 3, 3, 3], [0, 1, 2, 3]], dtype=torch.int32)
    want = R.fork(refs, table, parent)
    refs = refs.cuda()
    lc.kv8_fork(refs, view, parent.cuda())
    assert lc.device_error() == 1 << 24
    assert same(refs, want[0]) and same(view, want[1])
    assert bool((wide[:, 0] == 77).all()) and bool((wide[:, 5] == 77).all()) and bool((wide[:, :, :2] == 77).all())


@pytest.mark.parametrize("batch,beams,cols,page,new", [
    (1, 1, 1, 16, 1), (1, 4, 16, 64, 1), (3, 5, 9, 32, 16), (7, 3, 40, 16, 200), (2, 32, 6, 128, 17), (40, 16, 5, 16, 64), (300, 4, 3, 64, 1),
    (1, 1, 260, 16, 4096)])
@pytest.mark.parametrize("spare", [0, 3, 100, 3000])
def test_grow_matches_reference(lc, batch, beams, cols, page, new, spare):
    """Rows that share pages or hold reserved ones, some without new tokens; pools that do not suffice."""
    g = torch.Generator().manual_seed(cols + spare)
    refs, table, kv_len = pool(batch, beams, cols, page, spare, cols + spare, capacity=cols + new // page + 2)
    kv_len = (kv_len - torch.randint(0, page + 5, kv_len.shape, generator=g, dtype=torch.int32)).clamp_min(0)
    add = torch.randint(0, new + 1, kv_len.shape, generator=g, dtype=torch.int32)
    add[0, 0] = new
    flat = table.view(batch * beams, -1)
    want = R.grow(refs, flat, kv_len.flatten(), add.flatten(), page)
    refs, table = refs.cuda(), table.cuda()
    tail, granted = lc.kv8_grow(refs, table, kv_len.cuda(), add.cuda(), page, new)
    assert tail.shape == granted.shape == kv_len.shape and granted.dtype == torch.bool
    assert same(refs, want[0]) and same(table.view(batch * beams, -1), want[1])
    assert same(tail.flatten(), want[2]) and same(granted.flatten(), want[3])


def test_grow_all_sharers_of_a_tail_leave_it(lc):
    """The page that they copy from is not dealt out in the same call, and is free in the next."""
    table = torch.tensor([[[0, 2, -1]] * 3], dtype=torch.int32)
    refs = count(table, 8)
    kv_len, one = torch.full((1, 3), 20, dtype=torch.int32).cuda(), torch.ones(1, 3, dtype=torch.int32).cuda()
    refs, table = refs.cuda(), table.cuda()
    tail, granted = lc.kv8_grow(refs, table, kv_len, one, 16, 1)
    assert tail.tolist() == [[2, 2, 2]] and granted.all()
    assert table.tolist() == [[[0, 1, -1], [0, 3, -1], [0, 4, -1]]]
    assert refs.tolist() == [3, 1, 0, 1, 1, 0, 0, 0]
    tail, granted = lc.kv8_grow(refs, table, kv_len + 1, one * 12, 16, 12)  # 21 + 12 = 33: a third column
    assert tail.tolist() == [[-1, -1, -1]] and table[0, :, 2].tolist() == [2, 5, 6]


def test_grow_rows_out_of_range_are_left_and_reported(lc):
    table = torch.tensor([[0, -1], [-1, -1], [1, 9], [2, -1], [3, 4]], dtype=torch.int32).cuda()
    before = table.clone()
    refs = torch.tensor([1, 1, 1, 1, 1, 0, 0, 0], dtype=torch.int32).cuda()
    keep = refs.clone()
    kv = torch.tensor([-1, 3, 20, 10, 30], dtype=torch.int32).cuda()
    new = torch.tensor([1, 1, 1, 9, 3], dtype=torch.int32).cuda()
    tail, granted = lc.kv8_grow(refs, table, kv, new, 16, 8)
    assert lc.device_error() == (1 << 26 | 1 << 25)
    assert not granted.any() and tail.tolist() == [-1] * 5
    assert torch.equal(table, before) and torch.equal(refs, keep)


def test_grow_a_large_pool_with_few_free_pages(lc):
    n = 300000
    refs = torch.ones(n, dtype=torch.int32)
    free = torch.tensor([7, 4096, 150001, 299998, 299999])
    refs[free] = 0
    table = torch.full((6, 4), -1, dtype=torch.int32)
    new = torch.tensor([16, 0, 17, 1, 1, 0], dtype=torch.int32)
    zero = torch.zeros(6, dtype=torch.int32)
    want = R.grow(refs, table, zero, new, 16)
    refs, table = refs.cuda(), table.cuda()
    _, granted = lc.kv8_grow(refs, table, zero.cuda(), new.cuda(), 16, 32)
    assert granted.all() and same(refs, want[0]) and same(table, want[1])
    assert sorted(table[table >= 0].tolist()) == free.tolist()


@pytest.mark.parametrize("batch,beams,cols,page", [(1, 1, 1, 16), (3, 4, 30, 16), (2, 5, 300, 64), (9, 2, 4, 128)])
def test_free_matches_reference(lc, batch, beams, cols, page):
    g = torch.Generator().manual_seed(cols)
    refs, table, kv_len = pool(batch, beams, cols, page, 4, cols + 1)
    keep = (torch.rand(kv_len.shape, generator=g) * (kv_len + 40)).int()
    keep[0, 0] = 0
    want = R.free(refs, table.view(batch * beams, -1), keep.flatten(), page)
    refs, table = refs.cuda(), table.cuda()
    lc.kv8_free(refs, table, keep.cuda(), page)
    assert same(refs, want[0]) and same(table.view(batch * beams, -1), want[1])
    lc.kv8_free(refs, table, torch.zeros_like(keep).cuda(), page)
    assert not refs.any() and bool((table == -1).all())


def test_free_reports_what_nobody_holds(lc):
    table = torch.tensor([[0, 1, 50], [2, -1, -1]], dtype=torch.int32).cuda()
    refs = torch.tensor([1, 0, 1], dtype=torch.int32).cuda()
    lc.kv8_free(refs, table, torch.tensor([0, -1], dtype=torch.int32).cuda(), 16)
    assert lc.device_error() == (1 << 25 | 1 << 26)
    assert refs.tolist() == [0, 0, 1] and table.tolist() == [[-1, -1, -1], [2, -1, -1]]


def make_caches(lc, layers, n, heads, page, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in range(layers):
        c = lc.KV8Cache(n, heads, page, D)
        for t in (c.k, c.v):
            t.view(torch.uint8).copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
        for t in (c.k_scale, c.v_scale):
            t.copy_(torch.rand(t.shape, generator=g, device="cuda") + 0.5)
        out.append(c)
    return out


def parts(c):
    return c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale


@pytest.mark.parametrize("heads,page,D", [(1, 16, 32), (3, 16, 64), (2, 64, 128), (5, 128, 32), (7, 32, 128)])
@pytest.mark.parametrize("layers", [1, 3, 18])
def test_copy_moves_every_layer(lc, heads, page, D, layers):
    n = 23
    caches = make_caches(lc, layers, n, heads, page, D, 3)
    order = torch.randperm(n, generator=torch.Generator().manual_seed(layers))
    src, dst = order[:9].int().cuda(), order[9:18].int().cuda()
    src[4] = -1
    dst[6] = -7
    src[2] = src[1]  # one page to two places
    moves = [(a, b) for a, b in zip(src.tolist(), dst.tolist()) if a >= 0 and b >= 0]
    want = []
    for c in caches:
        keep = [t.clone() for t in parts(c)]
        for t in keep:
            for a, b in moves:
                t[b] = t[a]
        want.append(keep)
    lc.kv8_copy(caches, src, dst)
    for c, w in zip(caches, want):
        assert all(torch.equal(a, b) for a, b in zip(parts(c), w))


def test_copy_into_other_caches_and_bad_pages(lc):
    a, b = make_caches(lc, 2, 10, 2, 16, 64, 1), make_caches(lc, 2, 6, 2, 16, 64, 2)
    src, dst = torch.tensor([9, 3, 12, 1], dtype=torch.int32).cuda(), torch.tensor([0, 5, 1, 6], dtype=torch.int32).cuda()
    want = [[t.clone() for t in parts(c)] for c in b]
    for c, w in zip(a, want):
        for t, s in zip(w, parts(c)):
            t[0], t[5] = s[9], s[3]
    lc.kv8_copy(a, src, dst, into=b)
    assert lc.device_error() == 1 << 25
    for c, w in zip(b, want):
        assert all(torch.equal(x, y) for x, y in zip(parts(c), w))


def test_copy_of_pages_behind_32_bits(lc):
    """Pages whose first vector of 16 bytes is the 2^31-th and further."""
    n = (1 << 35) // (8 * 128 * 128) + 40
    c = lc.KV8Cache(n, 8, 128, 128)
    low, high = [3, 4, 5], [n - 40, n - 39, n - 1]
    g = torch.Generator(device="cuda").manual_seed(7)
    for t in parts(c):
        for p in low + [n - 20]:
            t[p] = torch.randint(0, 200, t[p].shape, generator=g, device="cuda").to(t.dtype)
    src, dst = torch.tensor(low + [n - 20], dtype=torch.int32).cuda(), torch.tensor(high + [6], dtype=torch.int32).cuda()
    lc.kv8_copy([c], src, dst)
    for t in parts(c):
        for p, q in zip(src.tolist(), dst.tolist()):
            assert torch.equal(t[p], t[q])


@pytest.mark.parametrize("n,held,layers", [(1, 0, 1), (1, 1, 1), (2, 1, 1), (40, 11, 2), (300, 150, 3), (300, 299, 1), (5000, 40, 17), (128, 0, 1)])
@pytest.mark.parametrize("inplace", [False, True])
def test_compact_matches_reference(lc, n, held, layers, inplace):
    g = torch.Generator().manual_seed(n + held)
    caches = make_caches(lc, layers, n, 2, 16, 32, 5)
    a, b = torch.full((6, 30), -1, dtype=torch.int32), torch.full((2, 3, 60), -1, dtype=torch.int32)
    pages = torch.randperm(n, generator=g)[:held].int()
    flat = torch.cat([a.flatten(), b.flatten()])
    at = torch.randperm(flat.numel(), generator=g)
    flat[at[:held]] = pages
    if held:  # some are held twice
        flat[at[held:held + 40]] = pages[torch.randint(0, held, (40,), generator=g)]
    a, b = flat[:180].view(6, 30).clone(), flat[180:].view(2, 3, 60).clone()
    refs = count(flat, n)
    wrefs, wtab, moves, live = R.compact(refs, [a, b])
    want = []
    for c in caches:
        keep = [t.clone() for t in parts(c)]
        for t in keep:
            for x, y in moves:
                t[y] = t[x]
        want.append(keep)
    refs, a, b = refs.cuda(), a.cuda(), b.cuda()
    if inplace:
        got = lc.kv8_compact(caches, refs, [a, b])
        ro, ao, bo = refs, a, b
    else:
        ro, ao, bo = torch.full_like(refs, 9), torch.full_like(a, 9), torch.full_like(b, 9)
        keep = refs.clone(), a.clone(), b.clone()
        got = lc.kv8_compact(caches, refs, [a, b], out=(ro, [ao, bo]))
        assert all(torch.equal(x, y) for x, y in zip((refs, a, b), keep))
    assert got.tolist() == [live]
    assert same(ro, wrefs) and same(ao, wtab[0]) and same(bo, wtab[1])
    for c, w in zip(caches, want):
        assert all(torch.equal(x, y) for x, y in zip(parts(c), w))


def test_compact_reports_entries_of_free_pages(lc):
    caches = make_caches(lc, 1, 8, 1, 16, 32, 5)
    table = torch.tensor([[6, 5, 99]], dtype=torch.int32).cuda()
    refs = torch.tensor([0, 0, 0, 0, 0, 0, 1, 0], dtype=torch.int32).cuda()
    lc.kv8_compact(caches, refs, [table])
    assert lc.device_error() == 1 << 25
    assert table.tolist() == [[0, 5, 99]] and refs.tolist() == [1] + [0] * 7


def test_pages_on_another_stream_and_replayed(lc):
    """fork, grow and free of one step, captured, replayed over other contents."""
    refs, table, kv_len = pool(4, 6, 20, 16, 400, 9)
    parent = torch.randint(0, 6, (4, 6), generator=torch.Generator().manual_seed(4), dtype=torch.int32)
    new = torch.full_like(kv_len, 16)
    keep = kv_len + 5

    def plain(refs, table, parent):
        refs, table = R.fork(refs, table, parent)
        refs, flat, tail, ok = R.grow(refs, table.view(24, -1), kv_len.flatten(), new.flatten(), 16)
        refs, flat = R.free(refs, flat, keep.flatten(), 16)
        return refs, flat.view_as(table), tail, ok

    d = [t.cuda() for t in (refs, table, parent, kv_len, new, keep)]
    tail, ok = torch.empty_like(d[3]), torch.empty(4, 6, dtype=torch.bool, device="cuda")
    ws = lc.kv8_pages_workspace(refs.shape[0], 24)

    def step(stream=None):
        lc.kv8_fork(d[0], d[1], d[2], stream=stream)
        lc.kv8_grow(d[0], d[1], d[3], d[4], 16, 16, out=(tail, ok), workspace=ws, stream=stream)
        lc.kv8_free(d[0], d[1], d[5], 16, stream=stream)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    step(st)
    st.synchronize()
    refs, table, wt, wo = plain(refs, table, parent)
    assert same(d[0], refs) and same(d[1], table) and same(tail.flatten(), wt) and same(ok.flatten(), wo)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step()
    for seed in (5, 6, 7):
        parent = torch.randint(0, 6, (4, 6), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
        d[2].copy_(parent)
        gr.replay()
        refs, table, wt, wo = plain(refs, table, parent)
        assert same(d[0], refs) and same(d[1], table) and same(tail.flatten(), wt) and same(ok.flatten(), wo)
