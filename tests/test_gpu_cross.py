"""Attention over states of another length against the float64 form in loop_ref, within the roundings
that the kernel makes (derived there)."""
import math

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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def make(seqs, heads, group, D, seed, spare=3):
    """q, k, v and the requests' places for [(rows, states)]; states lie in another order than rows."""
    g = gen(seed)
    rows = sum(n for n, _ in seqs) + 2  # two rows behind the last request
    q = torch.randn(rows, heads * group, D, generator=g, device="cuda").to(torch.bfloat16)
    kv = torch.randn(sum(t for _, t in seqs) + spare, 2, heads, D, generator=g, device="cuda").to(torch.bfloat16)
    q_start = torch.tensor([0] + [n for n, _ in seqs]).cumsum(0).int().cuda()
    at, start = 0, [0] * len(seqs)
    for b in reversed(range(len(seqs))):
        start[b] = at
        at += seqs[b][1]
    return q, kv[:, 0], kv[:, 1], q_start, i32(*start), i32(*[t for _, t in seqs])


def check(lc, q, k, v, q_start, kv_start, kv_len, max_new, scale=None, **kw):
    total, q_heads, D = q.shape
    scale = 1 / math.sqrt(D) if scale is None else scale
    out = torch.full((total, q_heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((total, q_heads), 7.0, device="cuda")
    got = lc.cross_attention(q, k, v, q_start, kv_start, kv_len, max_new, scale=scale, out=out, lse=lse, **kw)
    assert got[0] is out and got[1] is lse
    want, wl, to, tl = R.cross(q, k, v, q_start, kv_start, kv_len, scale)
    o, n = out.cpu().double(), lse.cpu().double()
    outside = wl.isnan()
    assert bool((o[outside] == 7).all()) and bool((n[outside] == 7).all())
    inside = ~outside
    empty = inside & (wl == R.NEG)
    assert bool((o[empty] == 0).all()) and bool((n[empty] == R.NEG).all())
    some = inside & ~empty
    assert not o[inside].isnan().any()
    assert ((o - want).abs()[some] <= to[some]).all(), ((o - want).abs() - to)[some].max()
    assert ((n - wl).abs()[some] <= tl[some]).all()
    return out, lse


SEQS = [[(1, 1)], [(1, 128)], [(1, 129)], [(4, 1500)], [(3, 5), (0, 40), (16, 100), (2, 0), (33, 33), (130, 300)], [(256, 256), (257, 129), (1, 1000)],
        [(1, 15), (1, 16), (1, 17), (1, 127), (1, 255), (1, 257)], [(600, 700)], [(2, 20000), (1, 3)]]


@pytest.mark.parametrize("seqs", SEQS)
@pytest.mark.parametrize("heads,group,D", [(1, 1, 64), (2, 4, 128), (3, 1, 32), (2, 5, 80), (1, 3, 8), (2, 2, 96), (1, 16, 128)])
def test_cross_matches_reference(lc, seqs, heads, group, D):
    check(lc, *make(seqs, heads, group, D, len(seqs) + D), max(n for n, _ in seqs))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads,group", [(40, 1), (2, 3)])
def test_cross_tiles_of_one_and_two_halves_in_turn(lc, heads, group, D):
    """Second halves that hold a few rows, over many chunks, and tiles of one half's rows between them."""
    seqs = [(129, 3000), (3, 100), (140, 1500), (33, 64), (161, 2500), (5, 700), (1, 1), (192, 1000), (250, 1800), (128, 300), (130, 129)]
    check(lc, *make(seqs, heads, group, D, D + heads), 250)


@pytest.mark.parametrize("group", [7, 50, 97, 100, 128, 130])
@pytest.mark.parametrize("scale", [0.2, -0.3])
def test_cross_groups_that_fill_no_half(lc, group, scale):
    """Halves of whole tokens (7, 97, 100), halves that split tokens (50, 130), and q with its signs turned over."""
    check(lc, *make([(5, 300), (1, 40), (9, 129), (0, 7), (4, 1)], 1, group, 64, group), 9, scale=scale)


@pytest.mark.parametrize("D", [80, 128])
def test_cross_long_rows_of_three_to_a_head(lc, D):
    check(lc, *make([(170, 700), (84, 300), (85, 129), (3, 90)], 2, 3, D, D), 170)


def test_cross_many_short_requests(lc):
    seqs = [(1 + i % 5, (i * 37) % 200) for i in range(300)]
    check(lc, *make(seqs, 2, 2, 64, 3), 5)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.5, 1e-3])
def test_cross_scales_of_any_sign(lc, D, scale):
    check(lc, *make([(5, 300), (140, 90)], 2, 2, D, 4), 140, scale=scale)


@pytest.mark.parametrize("D", [64, 128])
def test_cross_growing_scores_move_the_reference(lc, D):
    """Scores that climb by far more than the reference's slack, chunk by chunk, and fall again."""
    q, k, v, *rest = make([(20, 1000), (200, 900)], 1, 2, D, 6)
    k = k * torch.linspace(0.1, 12, k.shape[0], device="cuda").to(torch.bfloat16)[:, None, None]
    check(lc, q, k, v, *rest, 200)
    check(lc, q, k.flip(0), v, *rest, 200)


def test_cross_heavy_state_beside_many(lc):
    """Many small weights beside a heavy one keep what they hold together."""
    q, k, v, *rest = make([(3, 9000)], 1, 1, 64, 7)
    k, v = k.clone(), v.clone()
    k[:] = 0
    q[:, :, 0] = 8
    k[4000, 0, 0] = 9  # its weight is e^9 of any other's
    v[:] = 1
    v[4000] = -1
    check(lc, q, k, v, *rest, 3)


@pytest.mark.parametrize("D", [64, 128])
def test_cross_what_lies_behind_the_states_has_no_influence(lc, D):
    q, k, v, q_start, kv_start, kv_len = make([(5, 100), (150, 333), (2, 16)], 2, 2, D, 8, spare=200)
    k, v = k.clone(), v.clone()
    want = lc.cross_attention(q, k, v, q_start, kv_start, kv_len, 150)
    held = torch.zeros(k.shape[0], dtype=torch.bool, device="cuda")
    for s, n in zip(kv_start.tolist(), kv_len.tolist()):
        held[s:s + n] = True
    k[~held], v[~held] = math.nan, math.nan
    got = lc.cross_attention(q, k, v, q_start, kv_start, kv_len, 150)
    assert torch.equal(got, want)
    # the same with a request's neighbours NaN
    k[:], v[:] = math.nan, math.inf
    g = make([(5, 100), (150, 333), (2, 16)], 2, 2, D, 8, spare=200)
    s, n = int(kv_start[1]), int(kv_len[1])
    k[s:s + n], v[s:s + n] = g[1][s:s + n], g[2][s:s + n]
    got = lc.cross_attention(q, k, v, q_start, kv_start, kv_len, 150)
    r0, r1 = int(q_start[1]), int(q_start[2])
    assert torch.equal(got[r0:r1], want[r0:r1])


def test_cross_infinities_and_nan_where_they_are_seen(lc):
    q, k, v, *rest = make([(4, 200), (3, 50)], 1, 1, 64, 9)
    k, v, q = k.clone(), v.clone(), q.clone()
    s0 = int(rest[1][0])
    v[s0 + 7, 0, 5] = math.nan
    out = lc.cross_attention(q, k, v, *rest, 4).cpu()
    assert bool(out[:4, 0, 5].isnan().all()) and not out[:4, 0, :5].isnan().any() and not out[4:].isnan().any()
    v[s0 + 7, 0, 5] = 0
    q[1, 0, 3] = math.nan
    out, lse = (t.cpu() for t in lc.cross_attention(q, k, v, *rest, 4, lse=True))
    assert bool(out[1].isnan().all()) and bool(lse[1].isnan().all())
    assert not out[0].isnan().any() and not out[2:].isnan().any()


def test_cross_layouts(lc):
    """Heads before tokens, rows inside wider ones, shared states, a padded batch."""
    g = gen(10)
    B, T, heads, group, D = 3, 90, 2, 3, 64
    kv = torch.randn(2, B, heads, T, D, generator=g, device="cuda").to(torch.bfloat16)
    lens = i32(90, 17, 0)
    q = torch.randn(heads * group, 12, D + 8, generator=g, device="cuda").to(torch.bfloat16)[:, :, :D].transpose(0, 1)
    q_start = i32(0, 4, 8, 12)
    padded = [x.transpose(1, 2).reshape(B * T, heads, D) for x in kv]
    want = check(lc, q, *padded, q_start, i32(0, T, 2 * T), lens, 4)
    one = [x[0].transpose(0, 1) for x in kv]  # [T, heads, D] with heads outermost
    got = check(lc, q, *one, q_start, i32(0, 0, 5), i32(90, 90, 30), 4)
    assert torch.equal(got[0][:4], want[0][:4])
    new = lc.cross_attention(q, *padded, q_start, i32(0, T, 2 * T), lens, 4)
    assert torch.equal(new, want[0])


def test_cross_requests_out_of_range_are_left_out_and_reported(lc):
    q, k, v, q_start, kv_start, kv_len = make([(2, 30), (2, 30), (2, 30), (2, 30), (2, 30)], 1, 1, 64, 11)
    want = lc.cross_attention(q, k, v, q_start, kv_start, kv_len, 2)
    out = torch.full_like(want, 7)
    kv_start[1], kv_len[2], kv_start[3] = -1, -5, k.shape[0] - 29
    lc.cross_attention(q, k, v, q_start, kv_start, kv_len, 2, out=out)
    assert lc.device_error() == 1 << 26
    assert torch.equal(out[:2], want[:2]) and torch.equal(out[8:10], want[8:10]) and bool((out[2:8] == 7).all())
    out.fill_(7)
    lc.cross_attention(q, k, v, q_start, kv_start, kv_len, 1, out=out)  # more rows than max_new
    assert lc.device_error() == 1 << 26
    assert bool((out == 7).all())


def test_cross_repeats_to_the_last_bit(lc):
    a = make([(4, 3000), (300, 2000), (1, 5000)], 4, 2, 128, 12)
    want = lc.cross_attention(*a, 300, lse=True)
    for _ in range(5):
        got = lc.cross_attention(*a, 300, lse=True)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_cross_streams_and_graphs_with_their_own_workspaces(lc):
    cases = [make([(4, 700), (9, 65)], 2, 2, 64, 13), make([(1, 3000)], 4, 1, 128, 14)]
    want = [lc.cross_attention(*c, 9) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    ws = [lc.cross_attention_workspace(c[0], c[1], 9) for c in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [lc.cross_attention(*c, 9, workspace=w, stream=s) for c, w, s in zip(cases, ws, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for c, w in zip(cases, ws):
        out = torch.zeros_like(c[0])
        lc.cross_attention(*c, 9, workspace=w, out=out)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            lc.cross_attention(*c, 9, workspace=w, out=out)
        graphs.append(gr)
        outs.append(out)
    for c in cases:  # other contents and lengths
        c[0].mul_(0.5)
        c[5].sub_(3)
    want = [lc.cross_attention(*c, 9) for c in cases]
    for gr in graphs + graphs[::-1]:
        gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_cross_offsets_beyond_32_bits(lc):
    """States behind 2^31 elements and 2^32 bytes."""
    D, heads = 128, 8
    n = (1 << 31) // (heads * D) + 300
    k, v = (torch.zeros(n, heads, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, kk, vv, *_ = make([(3, 200)], heads, 1, D, 15)
    k[-200:], v[-200:] = kk[:200], vv[:200]
    out = lc.cross_attention(q, k, v, i32(0, 3), i32(n - 200), i32(200), 3)
    want = lc.cross_attention(q, kk, vv, i32(0, 3), i32(0), i32(200), 3)
    assert torch.equal(out, want)
