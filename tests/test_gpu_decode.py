"""Beam selection and reordering, the 8-bit cache's writer and its attention, against the
float64 forms in decode_ref."""
import math

import pytest
import torch

from tests import decode_ref as R

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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ----------------------------------------------------------------------------- beam_select

LSE_TOL = 1e-5  # the logit pass's contract for a log-partition


def check_select(got, logits, scores, n_out, finished=None, pad_id=0):
    """Outputs against the sorted candidates: two whose exact scores differ by less than twice
    the log-partition's tolerance may stand in either order; scores within that tolerance and
    half a float step."""
    every, outs = R.select(logits, scores, n_out, finished, pad_id)
    score, token, parent = (t.cpu() for t in got)
    assert score.shape == token.shape == parent.shape == (logits.shape[0], n_out)
    for b, (cand, want) in enumerate(zip(every, outs)):
        exact = {(p, t): s for s, p, t, _ in cand}
        seen = set()
        for j, (ws, wp, wt) in enumerate(want):
            s, t, p = float(score[b, j]), int(token[b, j]), int(parent[b, j])
            if ws == R.NEG:
                assert (s, t, p) == (R.NEG, pad_id, 0)
                continue
            assert (p, t) in exact, (b, j, p, t)
            assert (p, t) not in seen
            seen.add((p, t))
            assert abs(exact[(p, t)] - ws) <= 2 * LSE_TOL
            assert abs(s - exact[(p, t)]) <= LSE_TOL + 2.0 ** -24 * abs(s)


@pytest.mark.parametrize("batch,beams,V,n_out,dtype", [
    (1, 1, 1, 1, torch.float32), (1, 1, 3, 8, torch.bfloat16), (2, 3, 5, 4, torch.float32),
    (3, 4, 1001, 8, torch.bfloat16), (2, 32, 333, 32, torch.float32), (5, 7, 32003, 31, torch.bfloat16),
    (1, 4, 151936, 8, torch.bfloat16), (30, 5, 4097, 17, torch.float32), (128, 2, 257, 2, torch.bfloat16),
    (40, 3, 1024, 31, torch.bfloat16), (9, 32, 1023, 32, torch.float32), (3, 4, 1025, 30, torch.bfloat16), (2, 1, 20, 32, torch.float32),
    (7, 5, 95, 16, torch.bfloat16), (5, 2, 127, 4, torch.float32), (2, 2, 1, 1, torch.bfloat16), (3, 1, 33, 2, torch.bfloat16)])
def test_select_matches_reference(lc, batch, beams, V, n_out, dtype):
    g = gen(batch * 7 + V)
    x = (torch.randn(batch, beams, V, generator=g, device="cuda") * 2).to(dtype)
    s = torch.randn(batch, beams, generator=g, device="cuda") * 2 - 20
    check_select(lc.beam_select(x, s, n_out), x, s, n_out)


def test_select_dead_finished_masked_and_nan_rows(lc):
    g = gen(3)
    x = torch.randn(4, 6, 700, generator=g, device="cuda")
    s = torch.randn(4, 6, generator=g, device="cuda") - 5
    done = torch.zeros(4, 6, dtype=torch.bool, device="cuda")
    s[0, 1:] = -math.inf                  # first step: one live beam
    x[0, 1:] = math.nan                   # a dead beam's logits are not read
    x[1, 2] = -math.inf                   # a mask that leaves nothing
    x[1, 3, 5:] = -math.inf               # ... and one that leaves five tokens
    x[1, :, 100:] = -math.inf
    done[2] = torch.tensor([1, 0, 0, 1, 0, 0], device="cuda")
    x[2, 0] = math.inf
    x[2, 3] = math.nan                    # a finished beam's are not read either
    s[3] = -math.inf                      # nothing left at all
    s[2, 4] = math.nan                    # a NaN score is dead
    check_select(lc.beam_select(x, s, 9, finished=done, pad_id=77), x, s, 9, done, 77)
    done[:] = True
    check_select(lc.beam_select(x, s, 8, finished=done, pad_id=-3), x, s, 8, done, -3)


@pytest.mark.parametrize("V,dtype", [(90, torch.bfloat16), (1024, torch.bfloat16), (130, torch.float32), (5000, torch.bfloat16)])
def test_select_short_rows_dead_finished_and_not_finite(lc, V, dtype):
    """Rows with a NaN or +inf have no candidates, like those of a dead beam."""
    x = torch.randn(3, 5, V, generator=gen(V), device="cuda").to(dtype)
    s = torch.randn(3, 5, generator=gen(2), device="cuda") - 3
    done = torch.zeros(3, 5, dtype=torch.bool, device="cuda")
    done[0, 1] = done[1, 4] = True
    x[0, 2, 10:] = -math.inf
    x[1, 0] = -math.inf
    x[2, 1:] = -math.inf
    x[2, 1:, 3:6] = 0.5
    y, t = x.clone(), s.clone()
    y[0, 0, V - 1] = math.nan
    y[1, 3, 7] = math.inf
    y[1, 2] = math.nan
    t[0, 0] = t[1, 3] = t[1, 2] = -math.inf
    check_select(lc.beam_select(x, s, 32, finished=done, pad_id=5), x, s, 32, done, 5)
    for a, b in zip(lc.beam_select(y, s, 32, finished=done), lc.beam_select(x, t, 32, finished=done)):
        assert torch.equal(a, b)


def test_select_ties_go_to_the_lowest_beam_and_token(lc):
    x = torch.zeros(2, 4, 1024, device="cuda", dtype=torch.bfloat16)
    s = torch.full((2, 4), -1.5, device="cuda")
    s[1] = torch.tensor([-2.0, -1.0, -1.0, -3.0])
    score, token, parent = (t.cpu() for t in lc.beam_select(x, s, 20))
    assert parent[0].tolist() == [0] * 20 and token[0].tolist() == list(range(20))
    assert parent[1].tolist() == [1] * 20 and token[1].tolist() == list(range(20))
    x[0, :, 3:] = -math.inf
    score, token, parent = (t.cpu() for t in lc.beam_select(x, s, 20))
    assert parent[0].tolist() == [0] * 3 + [1] * 3 + [2] * 3 + [3] * 3 + [0] * 8
    assert token[0].tolist() == [0, 1, 2] * 4 + [0] * 8


def test_select_strided_rows_and_odd_offsets(lc):
    g = gen(5)
    full = torch.randn(3 * 4 * 2100 + 5, generator=g, device="cuda").to(torch.bfloat16)
    x = full[3:3 + 3 * 4 * 2100].view(3, 4, 2100)[:, :, :2049]
    s = torch.randn(3, 4, generator=g, device="cuda")
    check_select(lc.beam_select(x, s, 6), x, s, 6)


def test_select_replays_in_graphs_that_have_their_own_workspaces(lc):
    g = gen(6)
    xs = [torch.randn(1, 4, 5000 + 96 * i, generator=g, device="cuda") for i in range(2)]
    s = torch.randn(1, 4, generator=g, device="cuda")
    want = [[t.clone() for t in lc.beam_select(x, s, 8)] for x in xs]
    graphs, outs = [], []
    for x in xs:
        ws = lc.beam_select_workspace(x, 8)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(lc.beam_select(x, s, 8, workspace=ws))
        graphs.append((gr, ws))
    for _ in range(3):
        for gr, _ws in graphs:
            gr.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))


# ---------------------------------------------------------------------------- beam_reorder

@pytest.mark.parametrize("beams", [1, 2, 4, 7, 8, 16, 31, 32])
@pytest.mark.parametrize("inplace", [False, True])
def test_reorder_moves_every_state(lc, beams, inplace):
    g = gen(beams)
    batch = 3
    cap = torch.randn(batch, beams, 2, 50, 24, generator=g, device="cuda").to(torch.bfloat16)
    states = [torch.randint(0, 1 << 30, (batch, beams, 37), generator=g, device="cuda", dtype=torch.int32),
              torch.randint(0, 255, (batch, beams, 13), generator=g, device="cuda", dtype=torch.uint8),
              torch.randn(batch, beams, generator=g, device="cuda"),
              torch.randn(batch, beams, 5, 3, generator=g, device="cuda").to(torch.bfloat16),
              torch.randn(batch, beams, 515, generator=g, device="cuda", dtype=torch.float64),
              cap[:, :, :, :33],
              torch.randn(beams, batch, 9, generator=g, device="cuda").transpose(0, 1)]
    parent = torch.randint(0, beams, (batch, beams), generator=g, device="cuda", dtype=torch.int32)
    behind = cap[:, :, :, 33:].clone()
    row = torch.arange(batch, device="cuda")[:, None]
    want = [s[row, parent.long()].clone() for s in states]
    keep = [s.clone() for s in states]
    if inplace:
        got = lc.beam_reorder(states, parent)
        assert all(a is b for a, b in zip(got, states))
    else:
        into = [torch.zeros_like(s) for s in states]
        got = lc.beam_reorder(states, parent, out=into)
        assert all(torch.equal(a, b) for a, b in zip(states, keep))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(cap[:, :, :, 33:], behind)


def test_reorder_many_states_and_empty_ones(lc):
    g = gen(9)
    states = [torch.randn(2, 3, 1 + i, generator=g, device="cuda") for i in range(37)]
    states.insert(5, torch.empty(2, 3, 0, device="cuda"))
    parent = torch.tensor([[2, 2, 0], [1, 0, 1]], dtype=torch.int32, device="cuda")
    row = torch.arange(2, device="cuda")[:, None]
    want = [s[row, parent.long()].clone() for s in states]
    assert all(torch.equal(a, b) for a, b in zip(lc.beam_reorder(states, parent), want))


def test_reorder_bad_parent_keeps_the_row_and_is_reported(lc):
    s = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4).clone()
    parent = torch.tensor([[3, 9, -1, 0], [1, 1, 2, 2]], dtype=torch.int32, device="cuda")
    lc.beam_reorder([s], parent)
    assert s.tolist() == [[3, 1, 2, 0], [5, 5, 6, 6]]
    assert lc.device_error() == 1 << 24


def test_reorder_offsets_beyond_32_bits(lc):
    full = torch.zeros(2, 2, (1 << 31) // 2 + 16, dtype=torch.bfloat16, device="cuda")  # rows of 2 GiB
    full[:, 0, -16:] = 1
    full[:, 1, -16:] = 2
    parent = torch.tensor([[1, 1], [1, 0]], dtype=torch.int32, device="cuda")
    lc.beam_reorder([full], parent)
    assert full[:, :, -16:].float().mean(-1).tolist() == [[2, 2], [2, 1]]
    assert int(full[:, :, :64].count_nonzero()) == 0


# -------------------------------------------------------------------------------- the cache

def make_cache(lc, n_pages, heads, page, D, seed, garbage=True):
    """A cache whose every row holds garbage, NaN codes among it."""
    c = lc.KV8Cache(n_pages, heads, page, D)
    if garbage:
        g = gen(seed)
        for t in (c.k, c.v):
            t.view(torch.uint8).copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
        for t in (c.k_scale, c.v_scale):
            t.copy_(torch.exp2(torch.randint(-3, 3, t.shape, generator=g, device="cuda").float()))
    return c


def make_batch(seqs, page, seed, spare=2, cols=None):
    """q_start, kv_len and a block table of pages in no order for [(new, length)]."""
    counts = [-(-ln // page) for _, ln in seqs]
    n_pages = sum(counts) + spare
    ids = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    cols = cols or max(max(counts), 1)
    table = torch.full((len(seqs), cols), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = ids[at:at + c]
        at += c
    q_start = torch.tensor([0] + [n for n, _ in seqs]).cumsum(0).to(torch.int32)
    kv_len = torch.tensor([ln for _, ln in seqs], dtype=torch.int32)
    return q_start.cuda(), kv_len.cuda(), table.cuda(), n_pages


def same_codes(a, b):
    """Codes equal; NaN codes of either sign are one value."""
    a, b = a.cpu().to(torch.float32), b.cpu().to(torch.float32)
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


def check_append(lc, cache, k, v, q_start, kv_len, table, max_new, tail_src=None):
    want = [R.append(p, s, x, q_start.cpu(), kv_len.cpu(), table.cpu(), tail_src)
            for p, s, x in ((cache.k, cache.k_scale, k), (cache.v, cache.v_scale, v))]
    lc.kv8_append(cache, k, v, q_start, kv_len, table, max_new,
                  tail_src=None if tail_src is None else tail_src.cuda())
    for (p, s), gp, gs in zip(want, (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
        assert torch.equal(gs.cpu(), s)
        assert same_codes(gp, p)


SEQS = [[(1, 1)], [(1, 5), (1, 64), (1, 65), (1, 16), (1, 17)], [(5, 5), (0, 40), (16, 100), (33, 33), (130, 300)],
        [(128, 128), (1, 129), (64, 192), (200, 201)], [(0, 0), (7, 7)]]


@pytest.mark.parametrize("page,D", [(16, 32), (16, 128), (32, 64), (64, 128), (128, 32), (128, 128)])
@pytest.mark.parametrize("seqs", SEQS)
def test_append_matches_reference(lc, page, D, seqs):
    heads = 3
    q_start, kv_len, table, n_pages = make_batch(seqs, page, len(seqs))
    cache = make_cache(lc, n_pages, heads, page, D, 4)
    g = gen(D + page)
    rows = int(q_start[-1]) + 2  # two rows behind the last sequence
    packed = torch.randn(rows, 2, heads + 1, D, generator=g, device="cuda") * 3
    packed = (packed * torch.exp2(torch.randint(-20, 20, (rows, 1, 1, 1), generator=g, device="cuda").float())).to(torch.bfloat16)
    check_append(lc, cache, packed[:, 0, :heads], packed[:, 1, 1:], q_start, kv_len, table, max(max(n for n, _ in seqs), 1))


def test_append_extremes(lc):
    """Zeros, subnormals, the largest bf16, infinities and NaN; 448 * 2^k exactly and one step above."""
    q_start, kv_len, table, n_pages = make_batch([(9, 9)], 16, 1)
    cache = make_cache(lc, n_pages, 8, 16, 32, 2)
    x = torch.zeros(9, 8, 32, device="cuda")
    x[:, 1] = 1e-40
    x[:, 2, 3] = 3.3895313892515355e38
    x[2, 3, 1], x[3, 3, 2], x[4, 3, 3], x[4, 3, 4] = math.inf, -math.inf, math.nan, 2.0
    x[:, 4] = 448.0 * 2.0 ** -7
    x[:, 5] = 450.0 * 2.0 ** -7
    x[:, 6] = math.inf
    x[:, 7] = math.nan
    x = x.to(torch.bfloat16)
    check_append(lc, cache, x, -x, q_start, kv_len, table, 9)


def test_append_one_by_one_and_at_once_are_the_same(lc):
    """Power-of-two scales: moving codes to a larger scale is exact for values of e4m3's normal range."""
    g = gen(11)
    n, page, heads, D = 70, 32, 2, 64
    x = torch.randn(n, heads, D, generator=g, device="cuda")
    x = (torch.sign(x) * (x.abs() + 0.5) * torch.linspace(0.25, 4, n, device="cuda")[:, None, None]).to(torch.bfloat16)
    q_start, kv_len, table, n_pages = make_batch([(n, n)], page, 1)
    a, b = make_cache(lc, n_pages, heads, page, D, 3), make_cache(lc, n_pages, heads, page, D, 3)
    lc.kv8_append(a, x, x, q_start, kv_len, table, n)
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for i in range(n):
        ln = torch.tensor([i + 1], dtype=torch.int32, device="cuda")
        lc.kv8_append(b, x[i:i + 1], x[i:i + 1], one, ln, table, 1)
    assert torch.equal(a.k_scale, b.k_scale) and torch.equal(a.v_scale, b.v_scale)
    assert torch.equal(a.k.view(torch.uint8), b.k.view(torch.uint8))


def test_append_forks_a_shared_tail_page(lc):
    """Three beams continue one sequence of 37 tokens: each copies the tail page's rows into its own."""
    page, heads, D = 16, 2, 64
    g = gen(12)
    cache = make_cache(lc, 12, heads, page, D, 5)
    x = torch.randn(37, heads, D, generator=g, device="cuda").to(torch.bfloat16)
    base = torch.tensor([[4, 7, 1, -1]], dtype=torch.int32, device="cuda")
    check_append(lc, cache, x, x * 2, torch.tensor([0, 37], dtype=torch.int32, device="cuda"),
                 torch.tensor([37], dtype=torch.int32, device="cuda"), base, 37)
    table = torch.tensor([[4, 7, 1, -1], [4, 7, 2, -1], [4, 7, 9, 3]], dtype=torch.int32, device="cuda")
    table[0, 2] = 5
    y = torch.randn(16, heads, D, generator=g, device="cuda").to(torch.bfloat16) * 9
    q_start = torch.tensor([0, 1, 2, 16], dtype=torch.int32, device="cuda")
    kv_len = torch.tensor([38, 38, 51], dtype=torch.int32, device="cuda")
    check_append(lc, cache, y, y / 3, q_start, kv_len, table, 14, tail_src=torch.tensor([1, 1, 1], dtype=torch.int32))


def test_append_reports_bad_pages_and_lengths(lc):
    page, heads, D = 16, 1, 32
    cache = make_cache(lc, 6, heads, page, D, 5)
    before = cache.k.view(torch.uint8).clone()
    x = torch.randn(12, heads, D, device="cuda").to(torch.bfloat16)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.tensor([[6, 0], [-1, 0], [1, 2], [3, 4]], dtype=torch.int32, device="cuda")
    lc.kv8_append(cache, x, x, i32(0, 3, 6, 9, 12), i32(3, 3, 2, 33), table, 3)  # two bad pages, len < n, len > cols * page
    assert torch.equal(cache.k.view(torch.uint8), before)
    assert lc.device_error() == (1 << 25 | 1 << 26)
    lc.kv8_append(cache, x, x, i32(0, 4, 2, 13, 13), i32(4, 4, 4, 4), table[[2, 2, 2, 2]], 3)  # over max_new, decreasing, behind total
    assert torch.equal(cache.k.view(torch.uint8), before)
    assert lc.device_error() == 1 << 26


def test_append_at_the_end_of_the_longest_table(lc):
    """Positions next to 2^31, and a bound on the new tokens that reaches beyond them."""
    page, D = 128, 32
    cols = ((1 << 31) - 1 - 256) // page
    table = torch.zeros(1, cols, dtype=torch.int32, device="cuda")
    table[0, -2:] = torch.tensor([2, 1], dtype=torch.int32)
    cache = lc.KV8Cache(3, 1, page, D)
    n = page + 40
    x = torch.randn(n, 1, D, generator=gen(3), device="cuda").to(torch.bfloat16)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    lc.kv8_append(cache, x, x, i32(0, n), i32(cols * page - 5), table, 1 << 24)
    near = lc.KV8Cache(3, 1, page, D)
    lc.kv8_append(near, x, x, i32(0, n), i32(2 * page - 5), i32(2, 1)[None], n)
    for a, b in ((cache.k, near.k), (cache.v, near.v), (cache.k_scale, near.k_scale)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and int(b.view(torch.uint8).count_nonzero()) > 0


# ----------------------------------------------------------------------------- kv8_attention

def fill(lc, cache, q_start, kv_len, table, seed, spread=0):
    """Write every sequence's tokens (all of them) into the cache, and zero nothing else."""
    g = gen(seed)
    ln = kv_len.cpu()
    total = int(ln.sum())
    k = torch.randn(max(total, 1), cache.kv_heads, cache.head_dim, generator=g, device="cuda")
    v = torch.randn(max(total, 1), cache.kv_heads, cache.head_dim, generator=g, device="cuda")
    if spread:
        e = torch.randint(-spread, spread + 1, (max(total, 1), cache.kv_heads, 1), generator=g, device="cuda").float()
        v = v * torch.exp2(e)
    starts = torch.cat([torch.zeros(1, dtype=torch.int64), ln.long().cumsum(0)]).to(torch.int32).cuda()
    if total:
        lc.kv8_append(cache, k.to(torch.bfloat16), v.to(torch.bfloat16), starts, kv_len, table, int(ln.max()))


def check_attention(lc, q, cache, q_start, kv_len, table, max_new, scale=None, **kw):
    total, q_heads, D = q.shape
    out = torch.full((total, q_heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((total, q_heads), 7.0, device="cuda")
    got, gl = lc.kv8_attention(q, cache, q_start, kv_len, table, max_new, scale=scale, out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    want, wl, to, tl = R.attention(q, cache.k, cache.v, cache.k_scale, cache.v_scale, q_start.cpu(),
                                   kv_len.cpu(), table, D ** -0.5 if scale is None else scale)
    rows = torch.zeros(total, dtype=torch.bool)
    rows[int(q_start[0]):int(q_start[-1])] = True
    got, gl = got.cpu().double(), gl.cpu().double()
    assert bool((got[~rows] == 7).all()) and bool((gl[~rows] == 7).all())
    compare(got[rows], want[rows], to[rows])
    compare(gl[rows], wl[rows], tl[rows])


def compare(got, want, tol):
    odd = ~torch.isfinite(want)
    assert torch.equal(got[odd].nan_to_num(123.0), want[odd].nan_to_num(123.0))
    off = (got - want).abs()[~odd] - tol[~odd]
    assert off.numel() == 0 or bool((off <= 0).all()), float(off.max())


ATT = [
    # D, page, kv heads, group, [(new, length)]
    (128, 64, 1, 1, [(1, 1)]), (128, 64, 2, 4, [(1, 1000)]), (128, 16, 1, 8, [(1, 63), (1, 64), (1, 65), (0, 9), (1, 2)]),
    (64, 32, 3, 5, [(1, 31), (1, 700), (1, 1)]), (32, 128, 2, 3, [(1, 129), (1, 17)]), (128, 128, 1, 16, [(1, 333)]),
    (64, 16, 1, 1, [(16, 16), (16, 200), (3, 3), (1, 77)]), (128, 64, 2, 8, [(16, 300), (16, 16), (5, 64)]),
    (128, 32, 1, 7, [(64, 64), (64, 130), (2, 2), (33, 99)]), (32, 16, 2, 4, [(9, 50), (1, 1), (20, 21)]),
    (64, 64, 8, 1, [(1, 5), (0, 0), (1, 1)]), (128, 64, 1, 4, [(1, 4100)]), (64, 128, 1, 2, [(40, 2050)]),
]


@pytest.mark.parametrize("D,page,heads,group,seqs", ATT)
def test_attention_matches_reference(lc, D, page, heads, group, seqs):
    q_start, kv_len, table, n_pages = make_batch(seqs, page, D + len(seqs))
    cache = make_cache(lc, n_pages, heads, page, D, 21)
    fill(lc, cache, q_start, kv_len, table, 22)
    g = gen(23)
    rows = int(q_start[-1]) + 3
    packed = torch.randn(rows, heads * group + 2, D, generator=g, device="cuda").to(torch.bfloat16)
    check_attention(lc, packed[:, 1:-1], cache, q_start, kv_len, table, max(max(n for n, _ in seqs), 1))


@pytest.mark.parametrize("new,group", [(1, 4), (16, 2), (16, 8)])
def test_attention_rows_that_see_nothing(lc, new, group):
    """Lengths of zero, and more new tokens than cached ones: out 0 and lse -inf, no NaN."""
    seqs = [(new, 0), (new, max(new - 1, 0)), (new, new // 2), (new, 40)]
    q_start, kv_len, table, n_pages = make_batch(seqs, 16, 3)
    cache = make_cache(lc, n_pages, 1, 16, 128, 31)
    fill(lc, cache, q_start, kv_len, table, 32)
    q = torch.randn(4 * new, group, 128, generator=gen(33), device="cuda").to(torch.bfloat16)
    check_attention(lc, q, cache, q_start, kv_len, table, new)


@pytest.mark.parametrize("D,new,group", [(128, 16, 8), (64, 5, 1), (32, 16, 3)])
def test_attention_nan_and_infinity_stay_where_they_are_seen(lc, D, new, group):
    """NaN in a late token's key or value reaches the rows that see it and no other; a NaN or
    infinite query reaches its own row alone."""
    seqs = [(new, 70), (new, new)]
    q_start, kv_len, table, n_pages = make_batch(seqs, 16, 5)
    cache = make_cache(lc, n_pages, 2, 16, D, 41)
    fill(lc, cache, q_start, kv_len, table, 42)
    for b, ln in ((0, 70), (1, new)):
        t = ln - 2  # seen by the last two tokens
        cache.v.view(torch.uint8)[int(table[b, t // 16]), 0, t % 16, 3] = 0x7F
        cache.k.view(torch.uint8)[int(table[b, (ln - 1) // 16]), 1, (ln - 1) % 16, 5] = 0xFF
    q = torch.randn(2 * new, 2 * group, D, generator=gen(43), device="cuda").to(torch.bfloat16)
    q[1, 0, 4] = math.nan
    q[2, 2 * group - 1, 1] = math.inf
    check_attention(lc, q, cache, q_start, kv_len, table, new)


def test_attention_value_scales_far_apart(lc):
    q_start, kv_len, table, n_pages = make_batch([(1, 300), (16, 190)], 16, 6)
    cache = make_cache(lc, n_pages, 2, 16, 64, 51)
    fill(lc, cache, q_start, kv_len, table, 52, spread=12)
    q = torch.randn(17, 6, 64, generator=gen(53), device="cuda").to(torch.bfloat16)
    check_attention(lc, q, cache, q_start, kv_len, table, 16)


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** 100])
def test_attention_queries_of_any_size(lc, size):
    q_start, kv_len, table, n_pages = make_batch([(2, 100)], 32, 6)
    cache = make_cache(lc, n_pages, 1, 32, 64, 61)
    fill(lc, cache, q_start, kv_len, table, 62)
    q = torch.randn(2, 4, 64, generator=gen(63), device="cuda").to(torch.bfloat16)
    check_attention(lc, (q.float() * size).to(torch.bfloat16), cache, q_start, kv_len, table, 2, scale=0.125 / size)


def test_attention_pages_beyond_32_bits(lc):
    """A pool of more than 2^32 bytes: pages at its end."""
    n_pages = (1 << 32) // (8 * 128 * 128) + 6
    cache = lc.KV8Cache(n_pages, 8, 128, 128)
    kv_len = torch.tensor([200, 90], dtype=torch.int32, device="cuda")
    table = torch.tensor([[n_pages - 1, n_pages - 3], [n_pages - 2, 0]], dtype=torch.int32, device="cuda")
    q_start = torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda")
    fill(lc, cache, q_start, kv_len, table, 72)
    q = torch.randn(3, 8, 128, generator=gen(73), device="cuda").to(torch.bfloat16)
    small = lc.KV8Cache.from_tensors(*(t[-3:].clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)))
    out, lse = lc.kv8_attention(q, cache, q_start, kv_len, table, 2, lse=True)
    near = torch.where(table > 0, table - (n_pages - 3), 0).to(torch.int32)
    want, wl = lc.kv8_attention(q, small, q_start, kv_len, near, 2, lse=True)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    check_attention(lc, q, small, q_start, kv_len, near, 2)


def test_attention_reports_bad_pages_and_lengths(lc):
    cache = make_cache(lc, 4, 1, 16, 64, 1, garbage=False)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.randn(6, 2, 64, device="cuda").to(torch.bfloat16)
    table = torch.tensor([[0, 4], [-7, 1], [0, 1]], dtype=torch.int32, device="cuda")
    out = lc.kv8_attention(q, cache, i32(0, 1, 2, 3), i32(32, 17, 3), table, 1)
    assert lc.device_error() == 1 << 25 and bool(torch.isfinite(out.float()).all())
    out = lc.kv8_attention(q, cache, i32(0, 1, 2, 3), i32(33, -1, 3), table[[2, 2, 2]], 1)
    assert lc.device_error() == 1 << 26 and bool((out[:2] == 0).all())
    out = lc.kv8_attention(q, cache, i32(0, 4, 2, 9), i32(3, 3, 3), table[[2, 2, 2]], 2)
    assert lc.device_error() == 1 << 26 and bool((out == 0).all())


def test_attention_same_bits_in_graphs_and_on_another_stream(lc):
    q_start, kv_len, table, n_pages = make_batch([(4, 900), (4, 33), (2, 64)], 64, 8)
    cache = make_cache(lc, n_pages, 2, 64, 128, 81)
    fill(lc, cache, q_start, kv_len, table, 82)
    q = torch.randn(10, 8, 128, generator=gen(83), device="cuda").to(torch.bfloat16)
    want, wl = lc.kv8_attention(q, cache, q_start, kv_len, table, 4, lse=True)
    ws = [lc.kv8_attention_workspace(q, cache, table, 4) for _ in range(2)]
    outs, graphs = [], []
    for w in ws:
        o, l = torch.zeros_like(want), torch.zeros_like(wl)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            lc.kv8_attention(q, cache, q_start, kv_len, table, 4, out=o, lse=l, workspace=w)
        outs.append((o, l))
        graphs.append(gr)
    for gr in graphs:
        for _ in range(2):
            gr.replay()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs.append(lc.kv8_attention(q, cache, q_start, kv_len, table, 4, lse=True, stream=side))
    side.synchronize()
    for o, l in outs:
        assert torch.equal(o, want) and torch.equal(l, wl)


@pytest.mark.parametrize("new,group,D,page", [(1, 4, 128, 64), (1, 12, 128, 16), (1, 2, 64, 32), (16, 8, 128, 64), (4, 8, 32, 128)])
def test_attention_many_stages_give_the_same_bits_every_time(lc, new, group, D, page):
    """Long runs of copies through the rings, from pages all over a large pool."""
    seqs = [(new, 200 + (i * 977) % 9000) for i in range(40)]
    q_start, kv_len, table, n_pages = make_batch(seqs, page, 7)
    heads = 4
    wide = -(-(1 << 28) // (heads * page * D))  # a pool of 2^28 values, the pages in use spread over it
    spread = torch.randperm(max(wide, n_pages), generator=torch.Generator().manual_seed(1))[:n_pages].to(torch.int32).cuda()
    table = torch.where(table >= 0, spread[table.clamp_min(0).long()], table).contiguous()
    cache = lc.KV8Cache(max(wide, n_pages), heads, page, D)
    fill(lc, cache, q_start, kv_len, table, 17)
    q = torch.randn(40 * new, heads * group, D, generator=gen(18), device="cuda").to(torch.bfloat16)
    want, wl = lc.kv8_attention(q, cache, q_start, kv_len, table, new, lse=True)
    for _ in range(25):
        out, lse = lc.kv8_attention(q, cache, q_start, kv_len, table, new, lse=True)
        assert torch.equal(out, want) and torch.equal(lse, wl)
    for b in (3, 39):
        one = torch.tensor([0, new], dtype=torch.int32, device="cuda")
        check_attention(lc, q[b * new:(b + 1) * new, :group].contiguous(), lc.KV8Cache.from_tensors(*(
            t[:, :1].contiguous() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale))),
            one, kv_len[b:b + 1], table[b:b + 1], new)


@pytest.mark.parametrize("new,group,heads", [(16, 8, 4), (17, 1, 12), (1, 4, 8)])
def test_attention_many_short_sequences(lc, new, group, heads):
    """Tiles of a chunk or two, so that a CTA's roles are at several of them at once; sequences
    without tokens among them."""
    seqs = [(0, 30) if i % 7 == 3 else (0, 0) if i % 11 == 5 else (new, new + (i * 37) % 240) for i in range(200)]
    q_start, kv_len, table, n_pages = make_batch(seqs, 16, 12)
    cache = make_cache(lc, n_pages, heads, 16, 64, 13)
    fill(lc, cache, q_start, kv_len, table, 14)
    scale = torch.exp2(torch.randint(-20, 20, (int(q_start[-1]), heads * group, 1), generator=gen(15), device="cuda").float())
    q = (torch.randn(int(q_start[-1]), heads * group, 64, generator=gen(16), device="cuda") * scale).to(torch.bfloat16)
    check_attention(lc, q, cache, q_start, kv_len, table, new)
    want = lc.kv8_attention(q, cache, q_start, kv_len, table, new)
    for _ in range(30):
        assert torch.equal(lc.kv8_attention(q, cache, q_start, kv_len, table, new), want)


@pytest.mark.parametrize("heads", [1, 3, 8, 24, 50, 90])
@pytest.mark.parametrize("new,group", [(1, 3), (2, 7), (19, 2), (16, 8)])
def test_attention_tiles_in_any_number_of_parts(lc, heads, new, group):
    q_start, kv_len, table, n_pages = make_batch([(new, 2900 + new)], 128, 3)
    cache = make_cache(lc, n_pages, heads, 128, 32, 4)
    fill(lc, cache, q_start, kv_len, table, 5)
    q = torch.randn(new, heads * group, 32, generator=gen(6), device="cuda").to(torch.bfloat16)
    check_attention(lc, q, cache, q_start, kv_len, table, new)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30])
@pytest.mark.parametrize("new,group", [(2, 2), (20, 2)])
def test_attention_of_any_scale(lc, new, group, scale):
    q_start, kv_len, table, n_pages = make_batch([(new, 150), (new, 20)], 32, 3)
    cache = make_cache(lc, n_pages, 2, 32, 64, 4)
    fill(lc, cache, q_start, kv_len, table, 5)
    q = torch.randn(2 * new, 2 * group, 64, generator=gen(6), device="cuda").to(torch.bfloat16)
    check_attention(lc, q, cache, q_start, kv_len, table, new, scale=scale)


def test_calls_at_once_on_two_streams(lc):
    """Selection, append and attention of two batches, each on a stream of its own."""
    side = [torch.cuda.Stream() for _ in range(2)]
    work = []
    for s in range(2):
        seqs = [(4 + 12 * s, 300 + 900 * i) for i in range(6)]
        q_start, kv_len, table, n_pages = make_batch(seqs, 64, s)
        cache = make_cache(lc, n_pages, 2, 64, 128, s, garbage=False)
        fill(lc, cache, q_start, kv_len, table, 30 + s)
        rows = int(q_start[-1])
        q = torch.randn(rows, 8, 128, generator=gen(s), device="cuda").to(torch.bfloat16)
        kv = torch.randn(rows, 2, 128, generator=gen(40 + s), device="cuda").to(torch.bfloat16)
        logits, scores = torch.randn(3, 4, 40000 + s, generator=gen(50 + s), device="cuda"), torch.zeros(3, 4, device="cuda")
        call = lambda st, q=q, kv=kv, cache=cache, a=q_start, b=kv_len, t=table, n=seqs[0][0], x=logits, y=scores: (  # noqa: E731
            lc.kv8_append(cache, kv, kv, a, b, t, n, stream=st), lc.kv8_attention(q, cache, a, b, t, n, lse=True, stream=st),
            lc.beam_select(x, y, 5, stream=st))
        torch.cuda.synchronize()
        work.append((call, call(None)))
    torch.cuda.synchronize()
    for _ in range(10):
        got = [call(st) for st, (call, _) in zip(side, work)]
        torch.cuda.synchronize()
        for g, (_, want) in zip(got, work):
            assert all(torch.equal(a, b) for a, b in zip(g[1] + g[2], want[1] + want[2]))


def test_attention_scores_that_rise_by_any_amount(lc):
    """Keys that grow along the sequence: maxima move in every chunk, by little and by more than
    f16 or f32 weights could hold."""
    for rise in (0.02, 0.5, 40.0, 600.0):
        for new, group in ((1, 4), (8, 4)):
            n = 700
            q_start, kv_len, table, n_pages = make_batch([(new, n), (new, n - 130)], 32, 9)
            cache = make_cache(lc, n_pages, 1, 32, 64, 10)
            g = gen(11)
            q = torch.randn(2 * new, group, 64, generator=g, device="cuda").to(torch.bfloat16)
            dir_ = q.float().mean((0, 1))
            at = torch.arange(n, device="cuda", dtype=torch.float32)
            k = (torch.randn(n, 1, 64, generator=g, device="cuda") + (at * rise / n)[:, None, None] * dir_).to(torch.bfloat16)
            v = torch.randn(n, 1, 64, generator=g, device="cuda").to(torch.bfloat16)
            starts = torch.tensor([0, n, 2 * n - 130], dtype=torch.int32, device="cuda")
            lc.kv8_append(cache, torch.cat([k, k[:n - 130]]), torch.cat([v, v[:n - 130]]), starts, kv_len, table, n)
            check_attention(lc, (q.float() * 4).to(torch.bfloat16), cache, q_start, kv_len, table, new)


# ------------------------------------------------------------------------- used together

def test_beam_decoding_with_the_cache(lc):
    """Beam search of one layer over the 8-bit cache: prompt append, then per step attention,
    logits, selection, reordering of tables and histories, and an append that forks the tail
    pages.  A reference keeps every beam's pages apart, in the same order of appends."""
    torch.manual_seed(0)
    batch, beams, V, heads, group, D, page, steps, plen = 2, 3, 500, 2, 4, 64, 16, 21, 29
    H = heads * group * D
    g = gen(90)
    mk = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 0.08).to(torch.bfloat16)  # noqa: E731
    emb, wq, wk, wv, wo = mk(V, H), mk(H, H), mk(H, heads * D), mk(H, heads * D), mk(H, V)
    emb = emb * 12
    project = lambda tok: (emb[tok] @ wq, emb[tok] @ wk, emb[tok] @ wv)  # noqa: E731
    cols = -(-(plen + steps) // page)
    rows = batch * beams
    n_pages = batch * cols + rows * steps
    cache = make_cache(lc, n_pages, heads, page, D, 91)
    free = list(range(n_pages))
    # the prompt, once for each batch entry
    prompt = torch.randint(0, V, (batch, plen), generator=g, device="cuda")
    table = torch.full((batch, beams, cols), -1, dtype=torch.int32, device="cuda")
    ptab = torch.tensor([[free.pop(0) for _ in range(-(-plen // page))] for _ in range(batch)], dtype=torch.int32, device="cuda")
    _, k, v = project(prompt.reshape(-1))
    starts = torch.arange(0, batch * plen + 1, plen, dtype=torch.int32, device="cuda")
    lens = torch.full((batch,), plen, dtype=torch.int32, device="cuda")
    lc.kv8_append(cache, k.view(-1, heads, D), v.view(-1, heads, D), starts, lens, ptab, plen)
    table[:, :, :ptab.shape[1]] = ptab[:, None]
    # the reference: every row's pages of its own, as codes
    ref = {(b, j): [(cache.k[ptab[b].long()].cpu(), cache.k_scale[ptab[b].long()].cpu()),
                    (cache.v[ptab[b].long()].cpu(), cache.v_scale[ptab[b].long()].cpu())]
           for b in range(batch) for j in range(beams)}
    scores = torch.full((batch, beams), -math.inf, device="cuda")
    scores[:, 0] = 0
    token = prompt[:, -1:].expand(batch, beams).contiguous()
    history = torch.zeros(batch, beams, steps, dtype=torch.int32, device="cuda")
    one = torch.arange(rows + 1, dtype=torch.int32, device="cuda")
    for step in range(steps):
        ln = plen + step
        q, k, v = project(token.reshape(-1))
        if step:  # the chosen tokens' keys and values, into pages of the beams' own
            at = (ln - 1) // page
            fork = torch.full((rows,), -1, dtype=torch.int32)
            if (ln - 1) % page:
                fork = table[:, :, at].reshape(-1).cpu().clone()
            for b in range(batch):
                for j in range(beams):
                    table[b, j, at] = free.pop(0)
            kv_len = torch.full((rows,), ln, dtype=torch.int32, device="cuda")
            lc.kv8_append(cache, k.view(rows, heads, D), v.view(rows, heads, D), one, kv_len,
                          table.view(rows, cols), 1, tail_src=fork.cuda())
            for b in range(batch):
                for j in range(beams):
                    new = []
                    for (p, s), x in zip(ref[b, j], (k, v)):
                        if p.shape[0] <= at:
                            p = torch.cat([p.view(torch.uint8), torch.zeros(1, heads, page, D, dtype=torch.uint8)]).view(torch.float8_e4m3fn)
                            s = torch.cat([s, torch.ones(1, heads)])
                        new.append(R.append(p, s, x.view(rows, heads, D)[b * beams + j:b * beams + j + 1], [0, 1], [ln],
                                            torch.arange(p.shape[0])[None]))
                    ref[b, j] = new
        kv_len = torch.full((rows,), ln, dtype=torch.int32, device="cuda")
        out = lc.kv8_attention(q.view(rows, heads * group, D), cache, one, kv_len, table.view(rows, cols), 1)
        if step in (0, 3, 4, steps - 1):
            for b in range(batch):
                for j in range(beams):
                    (kp, ks), (vp, vs) = ref[b, j]
                    ids = table[b, j, :kp.shape[0]].long()
                    full = ln // page
                    assert same_codes(cache.k[ids][:full], kp[:full]) and torch.equal(cache.k_scale[ids].cpu(), ks)
                    r = b * beams + j
                    want, _, to, _ = R.attention(q.view(rows, heads * group, D)[r:r + 1], kp, vp, ks, vs, [0, 1], [ln],
                                                 torch.arange(kp.shape[0])[None], D ** -0.5)
                    compare(out[r:r + 1].cpu().double(), want, to)
        logits = ((out.view(rows, H) + emb[token.reshape(-1)]) @ wo).view(batch, beams, V)
        got = lc.beam_select(logits, scores, beams)
        check_select(got, logits, scores, beams)
        scores, new_token, parent = got
        before = (table.clone(), history.clone())
        lc.beam_reorder([table, history], parent)
        row = torch.arange(batch, device="cuda")[:, None]
        assert torch.equal(table, before[0][row, parent.long()]) and torch.equal(history, before[1][row, parent.long()])
        history[:, :, step] = new_token
        ref = {(b, j): ref[b, int(parent[b, j])] for b in range(batch) for j in range(beams)}
        token = new_token.long()
    assert bool((scores[:, :-1] >= scores[:, 1:]).all()) and bool(torch.isfinite(scores).all())
