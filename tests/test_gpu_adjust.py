"""Penalties, biases and masks on logits against the float64 form in loop_ref.

Tolerance: a value is kept as a pair of floats.  A product or quotient is a pair, off by 2^-47 of itself (its
low part, 2^-24 of it, is rounded, and so is the quotient's remainder times a reciprocal); a sum of pairs
adds their low parts, each at most 2^-23 of the sum so far, with two roundings of 2^-24: 2^-46 of the terms'
magnitudes for each of the terms.  Then it is rounded once, by half a step of the type.  A token that nothing
touches is bit for bit the logit."""
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


def make_mask(n, V, density, g):
    words = -(-V // 32)
    bits = torch.rand(n, words, 32, generator=g, device="cuda") < density
    return (bits.long() << torch.arange(32, device="cuda")).sum(-1).to(torch.int32)


def make(rows, V, dtype, groups, cap, n_bias, masks, seed):
    g = gen(seed)
    x = (torch.randn(rows, V, generator=g, device="cuda") * 4).to(dtype)
    kw = {}
    if cap:
        kw["history"] = torch.randint(-2, V + 2, (groups, cap), generator=g, device="cuda", dtype=torch.int32)
        kw["history"][:, ::3] = kw["history"][:, :1].clamp(0, V - 1)  # one token again and again
        kw["seen"] = torch.randint(0, cap + 1, (rows,), generator=g, device="cuda", dtype=torch.int32)
        kw["seen"][0], kw["seen"][-1] = 0, cap
        kw["counted_from"] = torch.randint(0, cap, (groups,), generator=g, device="cuda", dtype=torch.int32)
        kw["repetition"] = 0.5 + torch.rand(groups, generator=g, device="cuda") * 1.5
        kw["presence"] = torch.randn(groups, generator=g, device="cuda")
        kw["frequency"] = torch.randn(groups, generator=g, device="cuda")
    if n_bias:
        kw["bias_ids"] = torch.randint(-1, V + 1, (groups, n_bias), generator=g, device="cuda", dtype=torch.int32)
        kw["bias_ids"][:, -1] = kw["bias_ids"][:, 0]  # one listed twice
        kw["bias_values"] = torch.randn(groups, n_bias, generator=g, device="cuda") * 5
    if masks:
        kw["mask"] = make_mask(masks, V, 0.5, g)
        kw["mask"][0] = 0  # nothing is left
        kw["mask_index"] = torch.randint(-1, masks, (rows,), generator=g, device="cuda", dtype=torch.int32)
        kw["mask_index"][-1] = 0
    return x, kw


def check(got, x, kw):
    want, mag = R.adjust(x, **kw)
    y = got.cpu().double()
    nan = want.isnan()  # (what passes the type's largest is infinite, in 64 bits it need not be)
    assert torch.equal(y.isnan(), nan)
    inf = torch.isinf(want.to(x.dtype)) | nan
    assert torch.equal(y[inf & ~nan], want.to(x.dtype).double()[inf & ~nan])
    assert not torch.isinf(y[~inf]).any()
    half = torch.finfo(x.dtype).eps / 2
    terms = 4 + (kw["bias_ids"].shape[1] if "bias_ids" in kw else 0)
    assert ((y - want).abs()[~inf] <= (half * want.abs() + terms * 2.0 ** -46 * mag + 2.0 ** -133)[~inf]).all()
    same = (want == x.cpu().double()) & ~inf  # what nothing moved
    assert torch.equal(got.cpu()[same], x.cpu()[same])


@pytest.mark.parametrize("rows,V,groups,cap,n_bias,masks", [
    (1, 1, 1, 3, 2, 1), (2, 7, 1, 9, 0, 0), (4, 31, 2, 20, 3, 2), (3, 32, 3, 0, 5, 0), (6, 33, 2, 64, 1, 3), (5, 1000, 5, 300, 64, 2),
    (4, 8191, 2, 500, 7, 2), (3, 8192, 1, 0, 0, 2), (8, 8193, 2, 1500, 33, 4), (2, 16391, 1, 40, 0, 0), (16, 32003, 1, 700, 3, 3),
    (2, 151936, 2, 2000, 300, 2), (2, 500, 1, 5000, 1024, 1), (70, 96, 7, 50, 4, 5)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inplace", [False, True])
def test_adjust_matches_reference(lc, rows, V, groups, cap, n_bias, masks, dtype, inplace):
    x, kw = make(rows, V, dtype, groups, cap, n_bias, masks, rows * 31 + V)
    keep = x.clone()
    if inplace:
        got = lc.adjust_logits(x, **kw)
        assert got is x
    else:
        into = torch.full_like(x, 7)
        got = lc.adjust_logits(x, out=into, **kw)
        assert got is into and torch.equal(x, keep)
    check(got, keep, kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [32768, 32767, 65536])
def test_adjust_every_token_seen(lc, dtype, V):
    x, kw = make(3, V, dtype, 3, 70000, 9, 2, V)
    for h in kw["history"]:  # all of them, at places that differ from row to row
        at = torch.randperm(70000, device="cuda", generator=gen(4))[:V]
        h[at] = torch.randperm(V, device="cuda", generator=gen(5)).to(torch.int32)
    kw["seen"][1] = 70000
    check(lc.adjust_logits(x, out=torch.empty_like(x), **kw), x, kw)


@pytest.mark.parametrize("which", [("repetition",), ("repetition", "presence")])
@pytest.mark.parametrize("V", [8192, 8193, 16385])
def test_adjust_more_different_tokens_than_a_list_holds(lc, which, V):
    x, kw = make(2, V, torch.float32, 2, 20000, 40, 0, V)
    for h in kw["history"]:
        h[:V] = torch.randperm(V, device="cuda", generator=gen(6)).to(torch.int32)
    kw["seen"][:] = torch.tensor([V, 20000])
    kw = {k: v for k, v in kw.items() if k in ("history", "seen", "bias_ids", "bias_values") + which}
    keep = x.clone()
    check(lc.adjust_logits(x, **kw), keep, kw)


@pytest.mark.parametrize("which", ["repetition", "presence", "frequency", "seen"])
def test_adjust_each_penalty_alone(lc, which):
    x, kw = make(4, 300, torch.float32, 2, 100, 0, 0, 5)
    kw = {k: v for k, v in kw.items() if k in ("history", "seen", which)}
    check(lc.adjust_logits(x, out=torch.empty_like(x), **kw), x, kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("off_in,off_out", [(0, 0), (1, 1), (3, 0), (0, 5), (7, 2)])
def test_adjust_strided_rows_at_any_offset(lc, dtype, off_in, off_out):
    """Rows off the 16-byte grid, input and output differently; what lies between the rows stays."""
    V, stride = 9001, 9013
    x, kw = make(6, V, dtype, 3, 200, 9, 2, 8)
    a, b = (torch.full((6 * stride + 16,), 3.0, dtype=dtype, device="cuda") for _ in range(2))
    view = lambda t, off: t[off:off + 6 * stride].view(2, 3, stride)[..., :V]  # noqa: E731
    src, dst = view(a, off_in), view(b, off_out)
    src.copy_(x.view(2, 3, V))
    got = lc.adjust_logits(src, out=dst, **kw)
    check(got.reshape(6, V), x, kw)
    behind = b[off_out:off_out + 6 * stride].view(6, stride)[:, V:]
    assert bool((behind == 3).all()) and bool((b[:off_out] == 3).all()) and bool((b[off_out + 6 * stride:] == 3).all())
    lc.adjust_logits(src, **kw)
    assert torch.equal(src, got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_adjust_infinities_nan_and_the_lowest_value(lc, dtype):
    """Masked places may hold anything; what is not masked follows the formula."""
    V = 70
    x = torch.randn(3, V, device="cuda").to(dtype)
    low = torch.finfo(dtype).min
    x[:, 0], x[:, 1], x[:, 2], x[:, 3] = math.nan, math.inf, -math.inf, low
    mask = torch.full((3, 3), -1, dtype=torch.int32, device="cuda")
    mask[0, 0] = ~0b1111
    hist = torch.tensor([[0, 1, 2, 3, 4, 4]], dtype=torch.int32, device="cuda")
    seen = torch.tensor([6, 6, 0], dtype=torch.int32, device="cuda")
    rho, freq = torch.tensor([1.25], device="cuda"), torch.tensor([0.5], device="cuda")
    y = lc.adjust_logits(x, hist, seen, repetition=rho, frequency=freq, mask=mask, out=torch.empty_like(x)).cpu()
    assert bool((y[0, :4] == -math.inf).all())
    assert math.isnan(y[1, 0]) and y[1, 1] == math.inf and y[1, 2] == -math.inf and y[1, 3] == -math.inf
    assert torch.equal(y[2].nan_to_num(9), x[2].cpu().nan_to_num(9))
    keep = x.cpu()
    lc.adjust_logits(x, mask=mask)
    assert bool((x[0, :4] == -math.inf).all()) and torch.equal(x[0, 4:].cpu(), keep[0, 4:])
    assert torch.equal(x[1:].cpu().nan_to_num(9), keep[1:].nan_to_num(9))


def test_adjust_cancelling_terms_keep_their_bits(lc):
    """A count of thousands against a bias of the same size, which leave 2^-10 of themselves: one rounding."""
    x = torch.tensor([[1.0009765625, 2.0]], device="cuda")
    hist = torch.zeros(1, 30000, dtype=torch.int32, device="cuda")
    freq = torch.tensor([0.1], device="cuda")
    seen = torch.tensor([30000], dtype=torch.int32, device="cuda")
    bias = torch.tensor([[3000.0]], device="cuda")
    kw = dict(history=hist, seen=seen, frequency=freq, bias_ids=torch.zeros(1, 1, dtype=torch.int32, device="cuda"), bias_values=bias)
    got = lc.adjust_logits(x, out=torch.empty_like(x), **kw)
    want = float(x[0, 0]) - float(freq[0].double()) * 30000 + 3000.0
    assert abs(float(got[0, 0]) - want) <= 2.0 ** -24 * abs(want) + 5 * 2.0 ** -46 * 6001
    assert float(got[0, 1]) == 2.0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_adjust_values_near_the_ends_of_the_type(lc, dtype):
    """Products that overflow, sums that come back from there, subnormals, exact zeros, odd penalties."""
    V = 64
    x = torch.zeros(4, V, device="cuda")
    x[0] = torch.linspace(-3.3e38, 3.3e38, V)
    x[1] = torch.linspace(-1, 1, V) * 1e-38
    x[2] = 5.0
    x[3] = torch.linspace(-9, 9, V)
    x = x.to(dtype)
    hist = torch.arange(V, dtype=torch.int32, device="cuda").expand(4, V).contiguous()
    kw = dict(history=hist, seen=torch.full((4,), V, dtype=torch.int32, device="cuda"),
              repetition=torch.tensor([1.5, 1.5, 1.0, 1e-3], device="cuda"), presence=torch.tensor([-2e38, 0, 5.0, 0], device="cuda"),
              bias_ids=hist[:, :8].contiguous(), bias_values=torch.full((4, 8), 0.25, device="cuda"))
    check(lc.adjust_logits(x, out=torch.empty_like(x), **kw), x, kw)


@pytest.mark.parametrize("rho", [3.4e38, -2.9e38, 1.3e30, 1.1e30, 1.2e-38, 1e-40, 0.0])
def test_adjust_penalties_near_the_ends_of_their_type(lc, rho):
    """Logits whose quotient, or product, is an ordinary number again: its bits are all there."""
    V = 512
    x = torch.logspace(-38, 38, V, device="cuda") * torch.where(torch.arange(V, device="cuda") % 2 == 0, 1.0, -1.0)
    hist = torch.arange(V, dtype=torch.int32, device="cuda")[None]
    rep = torch.tensor([rho], device="cuda")
    got = lc.adjust_logits(x[None].contiguous(), out=torch.empty(1, V, device="cuda"), history=hist,
                           seen=torch.tensor([V], dtype=torch.int32, device="cuda"), repetition=rep)[0]
    want = torch.where(x > 0, x.double() / rep.double(), x.double() * rep.double())
    far = want.abs() >= 2.0 ** 128 * (1 - 2.0 ** -25)  # rounded to an infinity
    assert torch.equal(got[far].double(), torch.sign(want[far]) * math.inf)
    # a product or quotient by itself, off by 2^-46 of its size, rounded once (by half of the smallest step below 2^-126)
    near = want[~far]
    assert ((got[~far].double() - near).abs() <= near.abs() * (2.0 ** -24 + 2.0 ** -46) + 2.0 ** -150).all()


def test_adjust_ties_of_bf16_are_told_by_the_whole_sum(lc):
    """Sums a hair above and below a bf16 tie, by less than a float's step: rounded to their own side."""
    tie = 1 + 2.0 ** -8  # between 1 and 1 + 2^-7
    x = torch.full((3, 2), 1.0, device="cuda").to(torch.bfloat16)
    ids = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    bias = torch.tensor([[2.0 ** -8, 2.0 ** -40], [2.0 ** -8, -2.0 ** -40], [2.0 ** -8, 0.0]], device="cuda")
    got = lc.adjust_logits(x, bias_ids=ids, bias_values=bias)
    assert tie == 1.00390625 and got[:, 0].tolist() == [1.0078125, 1.0, 1.0] and got[:, 1].tolist() == [1.0] * 3


def test_adjust_rows_out_of_range_are_left_out_and_reported(lc):
    x, kw = make(4, 100, torch.float32, 4, 10, 0, 2, 3)
    kw["seen"] = torch.tensor([3, 11, -1, 10], dtype=torch.int32, device="cuda")
    kw["mask_index"] = torch.tensor([0, 1, 1, -5], dtype=torch.int32, device="cuda")
    into = torch.full_like(x, 5)
    lc.adjust_logits(x, out=into, **kw)
    assert lc.device_error() == 1 << 26
    assert bool((into[1:3] == 5).all()) and bool((into[0] == -math.inf).all())
    kw["seen"].fill_(2)
    kw["mask_index"][2] = 2
    into.fill_(5)
    lc.adjust_logits(x, out=into, **kw)
    assert lc.device_error() == 1 << 31
    assert bool((into[2] == 5).all()) and not bool((into[3] == 5).any())


def test_adjust_shapes_streams_and_replays(lc):
    """Any leading shape; another stream; a captured call replayed with other contents."""
    x, kw = make(24, 5000, torch.bfloat16, 6, 100, 4, 3, 21)
    shaped = x.view(3, 2, 4, 5000)
    want = lc.adjust_logits(x, out=torch.empty_like(x), **kw)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = torch.empty_like(shaped)
    lc.adjust_logits(shaped, out=got, stream=st, **kw)
    st.synchronize()
    assert torch.equal(got.view_as(want), want)
    into = torch.empty_like(x)
    lc.adjust_logits(x, out=into, **kw)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        lc.adjust_logits(x, out=into, **kw)
    y, kw2 = make(24, 5000, torch.bfloat16, 6, 100, 4, 3, 22)
    x.copy_(y)
    for k in kw:
        kw[k].copy_(kw2[k])
    gr.replay()
    torch.cuda.synchronize()
    check(into, y, kw2)


def test_adjust_offsets_beyond_32_bits(lc):
    """Rows whose element offsets pass 2^31 and whose byte offsets pass 2^32."""
    V, rows = 1 << 20, 2300
    x = torch.zeros(rows, V, dtype=torch.bfloat16, device="cuda")
    hist = torch.tensor([[V - 1, 5]], dtype=torch.int32, device="cuda").expand(rows, 2).contiguous()
    seen = torch.full((rows,), 2, dtype=torch.int32, device="cuda")
    lc.adjust_logits(x, hist, seen, presence=torch.arange(rows, device="cuda").float())
    want = -torch.arange(rows, device="cuda").to(torch.bfloat16)
    assert torch.equal(x[:, V - 1], want) and torch.equal(x[:, 5], want)
    assert int(x[:, 6:V - 1].count_nonzero()) == 0


def test_adjusted_logits_feed_selection_and_the_logit_pass(lc):
    """A mask that leaves three tokens leaves three candidates; one that leaves none, none."""
    x, kw = make(6, 3000, torch.float32, 2, 50, 3, 0, 33)
    mask = torch.zeros(6, -(-3000 // 32), dtype=torch.int32, device="cuda")
    mask[0] = -1
    mask[1, 2], mask[2, 90] = 0b1011, 1
    y = lc.adjust_logits(x.view(2, 3, 3000), mask=mask, out=torch.empty(2, 3, 3000, device="cuda"), **kw)
    scores = torch.zeros(2, 3, device="cuda")
    s, token, parent = (t.cpu() for t in lc.beam_select(y, scores, 32))
    pairs = set(zip(parent[0].tolist(), token[0].tolist()))
    assert {(1, 64), (1, 65), (1, 67), (2, 2880)} <= pairs
    assert s[1].tolist() == [-math.inf] * 32
