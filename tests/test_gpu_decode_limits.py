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


# ---------------------------------------------------------------------------- scales of any size

def any_scales(cache, seed, low, high):
    """Scales spread over 2^low .. 2^high that are no powers of two."""
    g = gen(seed)
    for t in (cache.k_scale, cache.v_scale):
        t.copy_(torch.exp2(low + (high - low) * torch.rand(t.shape, generator=g, device="cuda")))


@pytest.mark.parametrize("k_range,v_range", [((-1, 1), (-1, 1)), ((-3, 0), (-60, -56)), ((-9, -1), (-60, 3)), ((-2, 1), (-70, -64)),
                                             ((-126, -100), (-12, 20)), ((-2, 0), (60, 100))])
@pytest.mark.parametrize("D,page,heads,group,seqs", [TIGHT[i] for i in (0, 2, 3, 7, 8, 9)])
def test_attention_with_scales_of_any_size(lc, D, page, heads, group, seqs, k_range, v_range):  # noqa: F811
    q_start, kv_len, table, n_pages = make_batch(seqs, page, D + len(seqs))
    cache = make_cache(lc, n_pages, heads, page, D, 21)
    fill(lc, cache, q_start, kv_len, table, 22)
    any_scales(cache, 24, *k_range)
    k_scale = cache.k_scale.clone()
    any_scales(cache, 25, *v_range)
    cache.k_scale.copy_(k_scale)
    q = torch.randn(int(q_start[-1]), heads * group, D, generator=gen(23), device="cuda").to(torch.bfloat16)
    max_new = max(n for n, _ in seqs)
    # codes are of magnitudes up to 448: scores of some units where the keys' scales allow it
    scale = 2.0 ** -(6 + k_range[1]) / D ** 0.5
    exact = exact_attention(q, cache, q_start.cpu(), kv_len.cpu(), table, scale, 14 if max_new * group <= 16 else HELD)
    within(lc.kv8_attention(q, cache, q_start, kv_len, table, max_new, scale=scale, lse=True), exact)


@pytest.mark.parametrize("size", [2.0 ** -6, 1.0, 2.0 ** 9])
@pytest.mark.parametrize("fork", [False, True])
@pytest.mark.parametrize("page,D", [(16, 32), (32, 128), (128, 64)])
def test_append_to_pages_with_scales_of_any_size(lc, page, D, fork, size):  # noqa: F811
    """Tail pages whose scales are no powers of two, kept where they hold the new rows and outgrown where not: scales are exact, and
    a code, new, kept or moved, stands for its value to half a step (2^-4 of it, or 2^-10 of the scale) and f32's rounding."""
    heads, before, n = 3, page + 5, page + 4
    seqs = [(n, before + n), (2, before + 2)]
    q_start, kv_len, table, n_pages = make_batch(seqs, page, 7, spare=4)
    cache = make_cache(lc, n_pages, heads, page, D, 8)
    any_scales(cache, 9, -3, 3)
    table_cpu = table.cpu()
    tails = [int(table_cpu[b, 1]) for b in range(2)]
    source, tail_src = list(tails), None
    if fork:
        free = sorted(set(range(n_pages)) - set(table_cpu.flatten().tolist()))
        source = free[:2]
        tail_src = torch.tensor(source, dtype=torch.int32, device="cuda")
    # tail pages without NaN codes
    for t in (cache.k, cache.v):
        raw = t.view(torch.uint8)
        raw[source] = torch.where((raw[source] & 0x7F) == 0x7F, 0x31, raw[source])
    old = [(c.view(torch.uint8).clone(), s.clone()) for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
    g = gen(10)
    x = [(size * 100 * torch.randn(n + 2, heads, D, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2)]
    lc.kv8_append(cache, *x, q_start, kv_len, table, n, tail_src=tail_src)
    value = lambda raw: raw.view(torch.float8_e4m3fn).double()  # noqa: E731
    for (codes, scales), (raw, was), new in zip(((cache.k, cache.k_scale), (cache.v, cache.v_scale)), old, x):
        for b, (k, total) in enumerate(seqs):
            rows = new[int(q_start[b]):int(q_start[b]) + k].cpu().double()
            for at in range(before // page, -(-total // page)):
                lo, hi = max(before, at * page), min(total, (at + 1) * page)
                dst, src = int(table_cpu[b, at]), source[b] if at * page < before else None
                for h in range(heads):
                    got, now = value(codes.view(torch.uint8)[dst, h].cpu()), float(scales[dst, h])
                    part = rows[lo - before:hi - before, h]
                    need = R.page_scale(float(part.abs().max()))
                    assert now == (need if src is None else max(need, float(was[src, h])))
                    want = torch.zeros(0, D, dtype=torch.float64)
                    if src is not None:
                        had = raw[src, h, :lo - at * page].cpu()
                        want = value(had) * float(was[src, h])
                        if now == float(was[src, h]):
                            assert torch.equal(codes.view(torch.uint8)[dst, h, :lo - at * page].cpu(), had)
                    want = torch.cat([want, part])
                    off = (got[:want.shape[0]] * now - want).abs()
                    assert bool((off <= torch.maximum(2.0 ** -4 * want.abs(), torch.tensor(2.0 ** -10 * now)) + 2.0 ** -22 * want.abs()).all())


# ----------------------------------------------------------------- selection at the ends of the types

LSE_TOL = 1e-5  # the logit pass's contract for a log-partition


def exact_select(x, s, done):
    """Per batch entry the scores of all candidates in float64, [beams, V + 1] (-inf: none; a finished beam's own is the last)."""
    x, s, done = x.cpu().double(), s.cpu().double(), done.cpu()
    out = torch.full((*x.shape[:2], x.shape[2] + 1), -math.inf, dtype=torch.float64)
    for i in range(x.shape[0]):
        for j in range(x.shape[1]):
            row = x[i, j]
            if not float(s[i, j]) > -math.inf:
                continue
            if done[i, j]:
                out[i, j, -1] = s[i, j]
            elif not bool((row.isnan() | (row == math.inf)).any()) and bool((row > -math.inf).any()):
                # (the largest is taken off first: beside it the logarithm of the sum can be far below a rounding)
                rest = row - row.max()
                out[i, j, :-1] = s[i, j] + (rest - torch.log(torch.exp(rest).sum()))
    return out


def check_candidates(got, x, s, n_out, done=None, pad_id=0):
    """As many candidates as there are, each at a place where its score belongs."""
    done = torch.zeros(x.shape[:2], dtype=torch.bool) if done is None else done
    score, token, parent = (t.cpu() for t in got)
    for i, all_ in enumerate(exact_select(x, s, done)):
        best = torch.sort(all_.flatten(), descending=True).values
        seen = set()
        for k in range(n_out):
            at, value = (int(parent[i, k]), int(token[i, k])), float(score[i, k])
            if k >= best.numel() or best[k] == -math.inf:
                assert (at, value) == ((0, pad_id), -math.inf), (i, k)
                continue
            exact = float(all_[at[0], -1 if done[i, at[0]] else at[1]])
            assert exact > -math.inf and at not in seen and (not done[i, at[0]] or at[1] == pad_id), (i, k, at)
            seen.add(at)
            tol = LSE_TOL + 2.0 ** -24 * abs(exact)
            assert abs(value - exact) <= tol and abs(exact - float(best[k])) <= 2 * tol, (i, k, at)


BF16_MIN, F32_MIN = torch.finfo(torch.bfloat16).min, torch.finfo(torch.float32).min
SIZES = [(2, 90, torch.bfloat16), (2, 1000, torch.float32), (2, 5001, torch.bfloat16), (3, 20000, torch.float32), (40, 3001, torch.bfloat16)]


@pytest.mark.parametrize("mask", [-1e4, -1e9, -2.0 ** 31, -1e10, -1e20, -1e30, BF16_MIN, F32_MIN])
@pytest.mark.parametrize("batch,V,dtype", SIZES)
def test_select_with_finite_masks(lc, batch, V, dtype, mask):  # noqa: F811
    """Tokens masked with a finite value of any size, alone, in long runs and all but a few."""
    if mask == F32_MIN and dtype == torch.bfloat16:
        mask = BF16_MIN
    g = gen(V)
    x = torch.randn(batch, 5, V, generator=g, device="cuda") * 2
    s = torch.randn(batch, 5, generator=g, device="cuda") - 5
    x[:, 1, :V // 2] = mask
    x[:, 2, V // 3:] = mask
    x[:, 3] = mask
    x[:, 3, V - 2], x[:, 3, V // 2] = 0.5, -0.25
    x[:, 4, ::3] = mask
    x = x.to(dtype)
    check_candidates(lc.beam_select(x, s, 32), x, s, 32)
    few = x[:, 3:4].contiguous()
    check_candidates(lc.beam_select(few, s[:, 3:4].contiguous(), 8), few, s[:, 3:4], 8)


@pytest.mark.parametrize("mask", [-1e4, -2.0 ** 31, -1e10, -1e20, -1e30, BF16_MIN])
@pytest.mark.parametrize("batch,V,dtype", [(1, 151936, torch.bfloat16), (1, 9001, torch.float32), (60, 5001, torch.bfloat16)])
def test_log_partitions_with_finite_masks(lc, batch, V, dtype, mask):  # noqa: F811
    x = torch.randn(batch, 4, V, generator=gen(V), device="cuda") * 2
    x[:, 1, :V // 2] = mask
    x[:, 2, V // 3:] = mask
    x[:, 3] = mask
    x[:, 3, V - 2] = 0.5
    x = x.to(dtype)
    ids, values, lse = lc.topk_lse(x, 4)
    rows = x[:, 1:].double()
    assert float((lse.double() - torch.logsumexp(rows, -1)).abs().max()) <= LSE_TOL
    assert torch.equal(values[..., 0].double(), rows.amax(-1))
    assert torch.equal(rows.gather(-1, ids.long()), values.double())


@pytest.mark.parametrize("value", [-2.0 ** 29, -1.2e9, -2e9, -2.9e9, -1e10, -1e20, F32_MIN, -math.inf])
@pytest.mark.parametrize("batch,V,dtype", [(1, 40000, torch.bfloat16), (2, 9001, torch.float32), (60, 5001, torch.bfloat16)])
def test_log_partitions_of_rows_masked_throughout(lc, batch, V, dtype, value):  # noqa: F811
    """There the log-partition rounds to the largest logit; a NaN is still one."""
    if value == F32_MIN and dtype == torch.bfloat16:
        value = BF16_MIN
    x = torch.full((batch, 4, V), value, device="cuda").to(dtype)
    x[:, 2, 7] = max(value / 2, F32_MIN)
    x[0, 3, V // 2] = math.nan
    ids, values, lse = lc.topk_lse(x, 2)
    want = torch.logsumexp(x[:, 1:].double(), -1)
    assert bool(torch.isnan(lse[0, 2])) and torch.equal(lse[:, :2].double().isinf(), want[:, :2].isinf())
    fin = torch.isfinite(want)
    assert float(((lse.double() - want).abs()[fin] / want.abs()[fin]).max() if fin.any() else 0) <= 2.0 ** -24 + 2.0 ** -40
    shards = torch.stack([lc.topk_lse_shard(x[..., :V // 2], 0, 2), lc.topk_lse_shard(x[..., V // 2:], V // 2, 2)])
    _, _, merged = lc.topk_lse_merge(shards, 2)
    assert torch.equal(merged.view(batch, 3)[fin], lse[fin])



@pytest.mark.parametrize("value", [-2.0 ** 30, -1.5e9, -2.0 ** 31, -1e10, -1e20, -1e30, BF16_MIN, F32_MIN, 2.0 ** 30, 1e10, 3e38])
@pytest.mark.parametrize("batch,V,dtype", SIZES)
def test_select_rows_whose_largest_logit_is_of_any_size(lc, batch, V, dtype, value):  # noqa: F811
    """All of a row masked with a finite value; a few tokens next to it or as far below as the type goes; rows of which
    some token is NaN or infinite; and what a dead or finished beam has of them."""
    if value == F32_MIN and dtype == torch.bfloat16:
        value = BF16_MIN
    g = gen(V + 1)
    x = torch.randn(batch, 8, V, generator=g, device="cuda") * 2
    s = torch.randn(batch, 8, generator=g, device="cuda") - 5
    done = torch.zeros(batch, 8, dtype=torch.bool, device="cuda")
    x[:, 1] = value
    x[:, 2] = value * (1 + 2.0 ** -6 * torch.randint(0, 3, (batch, V), generator=g, device="cuda")).clamp_max(1 if abs(value) > 1e38 else 2)
    x[:, 3] = min(value, F32_MIN * 0.99)
    x[:, 3, 5:V:7] = value
    x[:, 4:] = value
    x[0, 4, V // 2] = math.nan
    x[-1, 4, V - 1] = math.inf
    x[:, 5, 3:] = -math.inf
    s[:, 6] = -math.inf
    done[:, 7] = True
    x = x.to(dtype)
    check_candidates(lc.beam_select(x, s, 32, finished=done, pad_id=9), x, s, 32, done, 9)
    s[:, 0] = -math.inf
    check_candidates(lc.beam_select(x, s, 20, finished=done, pad_id=9), x, s, 20, done, 9)
    alone = x[:, 1:2].contiguous()
    check_candidates(lc.beam_select(alone, s[:, 1:2].contiguous(), 5), alone, s[:, 1:2], 5)


@pytest.mark.parametrize("V,dtype,same", [(32000, torch.bfloat16, True), (151936, torch.bfloat16, True), (5004, torch.float32, True),
                                          (904, torch.bfloat16, True), (780, torch.float32, True), (32003, torch.bfloat16, False),
                                          (9999, torch.float32, False), (151935, torch.bfloat16, False)])
def test_select_among_beams_that_are_alike(lc, V, dtype, same):  # noqa: F811
    """Beams of equal logits and scores.  Rows that begin at the same place of a 16-byte line have equal log-partitions, so
    their candidates stand by (logit, beam, token); elsewhere those of one beam do, and beams come in
    either order where their scores are within the log-partition's tolerance of one another."""
    beams, n_out = 4, 30
    row = (torch.randn(3, 1, V, generator=gen(V), device="cuda") * 3).to(dtype)
    x = row.expand(3, beams, V).contiguous()
    s = torch.full((3, beams), -7.25, device="cuda")
    got = lc.beam_select(x, s, n_out)
    check_candidates(got, x, s, n_out)
    score, token, parent = (t.cpu() for t in got)
    for i in range(3):
        value = row[i, 0].cpu().float()
        best = sorted(range(V), key=lambda t: (-float(value[t]), t))[:n_out]
        if same:
            want = sorted(((-float(value[t]), j, t) for t in best for j in range(beams)))[:n_out]
            assert list(zip(parent[i].tolist(), token[i].tolist())) == [(j, t) for _, j, t in want]
        for j in range(beams):
            mine = token[i][parent[i] == j].tolist()
            assert mine == best[:len(mine)]


# ------------------------------------------------------------------- numbers that do not fit

@pytest.mark.parametrize("wrap", [1 << 32, -(1 << 32), 1 << 40])
def test_numbers_over_32_bits_are_refused(lc, wrap):  # noqa: F811
    """Not cut down to their low bits, with which the call would leave out sequences."""
    q_start, kv_len, table, n_pages = make_batch([(4, 20), (1, 3)], 16, 1)
    cache = make_cache(lc, n_pages, 1, 16, 32, 2)
    x = torch.randn(5, 1, 32, device="cuda").to(torch.bfloat16)
    before = [t.clone() for t in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale)]
    for call in (lambda n: lc.kv8_append(cache, x, x, q_start, kv_len, table, n), lambda n: lc.kv8_attention(x, cache, q_start, kv_len, table, n),
                 lambda n: lc.kv8_attention_workspace(x, cache, table, n),
                 lambda n: lc.beam_select_workspace(torch.zeros(1, 2, 50, device="cuda"), n),
                 lambda n: lc.beam_select(torch.zeros(1, 2, 50, device="cuda"), torch.zeros(1, 2, device="cuda"), n),
                 lambda n: lc.beam_select(torch.zeros(1, 2, 50, device="cuda"), torch.zeros(1, 2, device="cuda"), 2, pad_id=n)):
        with pytest.raises(ValueError):
            call(4 + wrap)
    for a, b in zip(before, (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale)):
        assert torch.equal(a, b)


def test_select_writes_its_scores_over_those_it_was_given(lc):  # noqa: F811
    """A loop that keeps one tensor of scores: each entry's are read before its own are written."""
    x = torch.randn(200, 6, 5000, generator=gen(1), device="cuda")
    s = torch.randn(200, 6, generator=gen(2), device="cuda") - 3
    want = lc.beam_select(x, s, 6)
    got = lc.beam_select(x, s, 6, out=(s, torch.empty_like(want[1]), torch.empty_like(want[2])))
    assert got[0] is s and all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------- a captured step, replayed

@pytest.mark.parametrize("new,group", [(1, 4), (5, 4)])
def test_a_captured_step_follows_what_its_tensors_hold(lc, new, group):  # noqa: F811
    """Append, attention, selection and reordering as one graph: replays take the lengths, tables, rows and scores that
    are there then, and leave what the calls made one by one leave."""
    batch, beams, heads, D, page, V, steps = 2, 3, 2, 64, 16, 900, 9
    rows = batch * beams
    total = 70 + new * steps
    _, _, table, n_pages = make_batch([(0, total)] * rows, page, 5)
    w = torch.randn(heads * group * D, V, generator=gen(6), device="cuda") * 0.3
    feed = torch.randn(steps, rows * new, heads * (group + 2), D, generator=gen(7), device="cuda").to(torch.bfloat16)

    def state():
        cache = make_cache(lc, n_pages, heads, page, D, 8, garbage=False)
        length = torch.tensor([70 - 11 * i for i in range(rows)], dtype=torch.int32, device="cuda")
        fill(lc, cache, None, length, table, 9)
        return dict(cache=cache, length=length, starts=new * torch.arange(rows + 1, dtype=torch.int32, device="cuda"), x=feed[0].clone(),
                    scores=torch.zeros(batch, beams, device="cuda"), history=torch.arange(batch * beams * 7, device="cuda").view(batch, beams, 7))

    def step(s):
        s["length"].add_(new)
        q, k, v = s["x"].split([heads * group, heads, heads], dim=1)
        lc.kv8_append(s["cache"], k, v, s["starts"], s["length"], table, new)
        out, lse = lc.kv8_attention(q, s["cache"], s["starts"], s["length"], table, new, lse=True)
        last = out.view(rows, new, heads * group * D)[:, -1].float()
        score, token, parent = lc.beam_select((last @ w).view(batch, beams, V), s["scores"], beams)
        s["scores"].copy_(score)
        lc.beam_reorder([s["history"]], parent)
        return out, lse, score, token, parent

    one, many = state(), state()
    want = []
    for i in range(steps):
        one["x"].copy_(feed[i])
        want.append([t.clone() for t in step(one)] + [one["history"].clone()])
    graph = torch.cuda.CUDAGraph()
    held = [t.clone() for t in (many["length"], many["scores"], many["history"])]
    with torch.cuda.graph(graph):
        got = step(many)
    for t, h in zip((many["length"], many["scores"], many["history"]), held):
        assert torch.equal(t, h)  # (a capture runs nothing)
    for i in range(steps):
        many["x"].copy_(feed[i])
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip((*got, many["history"]), want[i])), i
    for a, b in zip((one["cache"].k, one["cache"].v, one["cache"].k_scale), (many["cache"].k, many["cache"].v, many["cache"].k_scale)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
