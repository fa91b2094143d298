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


# ------------------------------------------------------------------ how far attention may be off

HELD = 9  # log2 of what the kernel for more than 16 rows holds a weight of 1 at; the one for fewer, 14


def exact_attention(q, cache, q_start, kv_len, table, scale, held):
    """(out, lse, tolerance of out, tolerance of lse) in float64 for the rows of the sequences, in order.

    With p the softmax weights, D the head dimension, T the tokens a row sees and m the row's largest score:
      * a score is off by at most e: an f32 sum of 2 D products and one f32 fma, (2 D + 4) 2^-24 (scale sum|q k|);
        q to 2^-17 of its row's largest value, 2^-17 max|q| (scale sum|k|); f32's roundings of the score, of m and of
        their difference, 2^-22 |score|; and the logarithm of the value scale, 2^-22 + 2^-23 |log2|;
      * the reciprocal of the value scale and exp2 are off by 2^-22 each, their products by 2^-24: 2^-20;
      * a weight is rounded to f16: by 2^-11 of its value, or where it is subnormal by 2^-25 of what it is held at, 2^held
        times what it is of a weight that the row has;
      * f32 sums over T tokens in runs of 16, and their joining: (T / 16 + 40) 2^-24 of sum p |v|;
      * out is rounded to bf16: half a step, 2^-8 of its value; lse to f32 after a logarithm and a product, 2^-20 in all."""
    D, page, heads = q.shape[2], cache.page, cache.kv_heads
    group = q.shape[1] // heads
    kp, vp, ks, vs, table = (t.cpu() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale, table))
    outs, lses, tos, tls = [], [], [], []
    q = q.cpu().double()
    for b in range(len(kv_len)):
        q0, n, ln = int(q_start[b]), int(q_start[b + 1] - q_start[b]), int(kv_len[b])
        ids = table[b, :-(-ln // page)].long()
        o, l, to, tl = (torch.zeros(n, heads, group, *s, dtype=torch.float64) for s in ((D,), (), (D,), ()))
        for h in range(heads):
            code = [(p.view(torch.uint8)[ids, h].view(p.dtype).double().reshape(-1, D)[:ln],
                     s[ids, h].double().repeat_interleave(page)[:ln, None]) for p, s in ((kp, ks), (vp, vs))]
            (ck, sk), (cv, sv) = code
            k, v = ck * sk, cv * sv
            for i in range(n):
                t = ln - n + i + 1
                x = q[q0 + i, h * group:(h + 1) * group]
                s = (x @ k[:t].T) * scale
                mag = (x.abs() @ k[:t].abs().T) * abs(scale)
                qk = x.abs().amax(1, keepdim=True) * k[:t].abs().sum(1)[None] * abs(scale)
                e = ((2 * D + 4) * 2.0 ** -24 * mag + 2.0 ** -17 * qk + 2.0 ** -22 * s.abs()).amax(1)
                e = e + 2.0 ** -22 + 2.0 ** -23 * float(torch.log2(sv[:t]).abs().max())
                norm = torch.logsumexp(s, 1)
                p = torch.exp(s - norm[:, None])
                pv = p @ v[:t].abs()
                low = 2.0 ** (-25 - held) * (p * sv[:t, 0]).amax(1, keepdim=True) * cv[:t].abs().sum(0)[None]
                o[i, h], l[i, h] = p @ v[:t], norm
                to[i, h] = (2.0 ** -8 * o[i, h].abs() + (1 + 2.0 ** -8) * (
                    (2 * e[:, None] + 2.0 ** -11 + 2.0 ** -20 + (t / 16 + 40) * 2.0 ** -24) * pv + low))
                tl[i, h] = e + (t / 16 + 40) * 2.0 ** -24 + 2.0 ** -24 * norm.abs() + 2.0 ** -20
        for a, x in zip((outs, lses, tos, tls), (o, l, to, tl)):
            a.append(x.reshape(n, heads * group, *x.shape[3:]))
    return [torch.cat(a) for a in (outs, lses, tos, tls)]


def within(got, exact):
    """Whether (out, lse) are within their tolerances."""
    for name, x, want, tol in zip(("out", "lse"), got, exact[:2], exact[2:]):
        off = ((x.cpu().double() - want).abs() / tol.clamp_min(1e-300)).nan_to_num(math.inf)
        assert float(off.max()) <= 1, (name, float(off.max()))


@pytest.mark.parametrize("where", ["first", "last"])
@pytest.mark.parametrize("D,new,group,length,batch", [
    (128, 8, 4, 32768, 1), (128, 8, 4, 32768, 20), (64, 16, 2, 32768, 20), (32, 16, 2, 32768, 20), (128, 16, 8, 3000, 20),
    (128, 1, 4, 32768, 1), (128, 1, 4, 32768, 40), (64, 1, 16, 9000, 80)])
def test_attention_beside_a_heavy_token(lc, D, new, group, length, batch, where):  # noqa: F811
    """A token that holds from 1 % to all of a row's weight, with a value of zero, and the others nearly alike:
    what the output has is their share, many weights that are small beside the heavy one.  One sequence, whose
    tokens are dealt to many CTAs, and as many over the same pages as give each CTA whole tiles."""
    heads = 8
    q_start, kv_len, table, n_pages = make_batch([(new, length)], 64, 3)
    cache = make_cache(lc, n_pages, heads, 64, D, 4)
    g = gen(D + new)
    u = torch.sign(torch.randn(D, generator=g, device="cuda"))
    k = 0.02 * torch.randn(length, heads, D, generator=g, device="cuda")
    v = 1 + 0.5 * torch.randn(length, heads, D, generator=g, device="cuda")
    at = 0 if where == "first" else length - new  # (the block's first token is seen by all its rows)
    k[at], v[at] = u, 0
    starts = torch.tensor([0, length], dtype=torch.int32, device="cuda")
    lc.kv8_append(cache, k.to(torch.bfloat16), v.to(torch.bfloat16), starts, kv_len, table, length)
    top = torch.linspace(math.log(length) - 4.6, math.log(length) + 4.6, new * heads * group, device="cuda")  # its scores
    q = (top.view(new, heads * group, 1) * u * D ** -0.5).to(torch.bfloat16)
    want = exact_attention(q, cache, q_start.cpu(), kv_len.cpu(), table, D ** -0.5, 14 if new * group <= 16 else HELD)
    starts = new * torch.arange(batch + 1, dtype=torch.int32, device="cuda")
    out, lse = lc.kv8_attention(q.repeat(batch, 1, 1), cache, starts, kv_len.repeat(batch), table.repeat(batch, 1), new, lse=True)
    for b in range(batch):
        within((out[b * new:(b + 1) * new], lse[b * new:(b + 1) * new]), want)
    off = (out.cpu().double().view(batch, -1) - want[0].view(1, -1)).norm(dim=1) / want[0].norm()
    assert float(off.max()) <= 2.0 ** -8


TIGHT = [
    # D, page, kv heads, group, [(new, length)]
    (128, 64, 2, 4, [(1, 1000), (1, 77)]), (64, 32, 3, 5, [(1, 31), (1, 700), (1, 1)]), (32, 128, 2, 3, [(1, 129), (4, 90)]),
    (128, 128, 1, 16, [(1, 333)]), (128, 16, 2, 8, [(2, 5000), (1, 9)]), (64, 64, 8, 1, [(9, 2100)]), (32, 16, 1, 13, [(1, 4000)]),
    (128, 64, 2, 8, [(16, 300), (16, 16), (5, 64)]), (64, 16, 4, 4, [(16, 2000), (9, 130)]), (32, 16, 2, 24, [(9, 500), (20, 21)]),
    (128, 32, 8, 7, [(64, 64), (64, 1300)]), (128, 128, 1, 1, [(17, 5000), (1, 1)])]


@pytest.mark.parametrize("size,spread", [(1.0, 0), (8.0, 0), (2.0, 9)])
@pytest.mark.parametrize("D,page,heads,group,seqs", TIGHT)
def test_attention_is_off_by_its_own_roundings_alone(lc, D, page, heads, group, seqs, size, spread):  # noqa: F811
    """Flat and peaked softmaxes, values of one size and of many, against what each kernel rounds."""
    q_start, kv_len, table, n_pages = make_batch(seqs, page, D + len(seqs))
    cache = make_cache(lc, n_pages, heads, page, D, 21)
    fill(lc, cache, q_start, kv_len, table, 22, spread)
    q = (size * torch.randn(int(q_start[-1]), heads * group, D, generator=gen(23), device="cuda")).to(torch.bfloat16)
    max_new = max(n for n, _ in seqs)
    exact = exact_attention(q, cache, q_start.cpu(), kv_len.cpu(), table, D ** -0.5, 14 if max_new * group <= 16 else HELD)
    within(lc.kv8_attention(q, cache, q_start, kv_len, table, max_new, lse=True), exact)
