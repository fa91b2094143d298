"""The operators of a decoding loop used together: beams of a constrained search share the pages of an
8-bit cache and the states of an encoder, on the device throughout."""
import math

import pytest
import torch

from tests import decode_ref as D
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


def test_constrained_beam_decoding_over_shared_pages_and_states(lc):
    """Each step: attention over the cache and over the encoder's states, logits, penalties and a grammar,
    selection, fork of tables, histories by beam_reorder, pages for the next token, append, and now and then a
    compaction.  A reference keeps every beam's pages apart, in the same order of appends."""
    torch.manual_seed(0)
    batch, beams, V, heads, group, dim, page, steps, plen = 2, 3, 500, 2, 4, 64, 16, 24, 29
    rows, width = batch * beams, heads * group * dim
    g = torch.Generator(device="cuda").manual_seed(90)
    mk = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 0.08).to(torch.bfloat16)  # noqa: E731
    emb, wq, wk, wv, wo = mk(V, width) * 12, mk(width, width), mk(width, heads * dim), mk(width, heads * dim), mk(width, V)
    enc_len = [150, 33]
    enc = mk(sum(enc_len), 2, heads, dim) * 10
    project = lambda tok: (emb[tok] @ wq, emb[tok] @ wk, emb[tok] @ wv)  # noqa: E731
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cols, n_pages = -(-(plen + steps) // page), 40
    cache = lc.KV8Cache(n_pages, heads, page, dim)
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    table = torch.full((batch, beams, cols), -1, dtype=torch.int32, device="cuda")
    # the prompt, in the first beam's row; then all beams go on from it
    prompt = torch.randint(0, V, (batch, plen), generator=g, device="cuda")
    first = torch.zeros(batch, beams, dtype=torch.int32, device="cuda")
    new = first.clone()
    new[:, 0] = plen
    tail, granted = lc.kv8_grow(refs, table, first, new, page, plen)
    assert granted.all() and bool((tail == -1).all())
    _, k, v = project(prompt.reshape(-1))
    starts, lens = i32(*range(0, batch * plen + 1, plen)), i32(*[plen] * batch)
    lc.kv8_append(cache, k.view(-1, heads, dim), v.view(-1, heads, dim), starts, lens, table[:, 0].contiguous(), plen)
    lc.kv8_fork(refs, table, first)
    ids = table[:, 0, :-(-plen // page)].long().cpu()
    ref = {(b, j): [(cache.k[ids[b].cuda()].cpu(), cache.k_scale[ids[b].cuda()].cpu()), (cache.v[ids[b].cuda()].cpu(), cache.v_scale[ids[b].cuda()].cpu())]
           for b in range(batch) for j in range(beams)}
    scores = torch.full((batch, beams), -math.inf, device="cuda")
    scores[:, 0] = 0
    token = prompt[:, -1:].expand(batch, beams).contiguous()
    history = torch.full((batch, beams, plen + steps), -1, dtype=torch.int32, device="cuda")
    history[:, :, :plen] = prompt[:, None].int()
    seen, length = torch.full((rows,), plen, dtype=torch.int32, device="cuda"), torch.full((batch, beams), plen, dtype=torch.int32, device="cuda")
    one, by_request = i32(*range(rows + 1)), i32(*range(0, rows + 1, beams))
    enc_start = i32(0, enc_len[0])
    # two grammars, turn by turn: the lower half of the vocabulary with three more tokens, and every third token
    allow = torch.zeros(2, V, dtype=torch.bool)
    allow[0, :V // 2] = True
    allow[0, [400, 450, 499]] = True
    allow[1, ::3] = True
    bits = torch.zeros(2, -(-V // 32) * 32, dtype=torch.long)
    bits[:, :V] = allow.long()
    mask = (bits.view(2, -1, 32) << torch.arange(32)).sum(-1).to(torch.int32).cuda()
    for step in range(steps):
        q, _, _ = project(token.reshape(-1))
        q = q.view(rows, heads * group, dim)
        flat = table.view(rows, cols)
        out = lc.kv8_attention(q, cache, one, length.view(-1), flat, 1)
        want, _, tol, _ = D.attention(q, cache.k, cache.v, cache.k_scale, cache.v_scale, one.cpu(), length.view(-1).cpu(), flat, 1 / math.sqrt(dim))
        assert ((out.cpu().double() - want).abs() <= tol).all()
        # a request's beams read its encoder's states side by side
        over = lc.cross_attention(q, enc[:, 0], enc[:, 1], by_request, enc_start, i32(*enc_len), beams)
        want, _, tol, _ = R.cross(q, enc[:, 0], enc[:, 1], by_request, enc_start, i32(*enc_len), 1 / math.sqrt(dim))
        assert ((over.cpu().double() - want).abs() <= tol).all()
        logits = ((out + over).reshape(rows, width) @ wo).float()
        raw = logits.clone()
        kw = dict(history=history.view(rows, -1), seen=seen, counted_from=torch.full((rows,), plen, dtype=torch.int32, device="cuda"),
                  repetition=torch.full((rows,), 1.1, device="cuda"), frequency=torch.full((rows,), 0.1, device="cuda"),
                  mask=mask, mask_index=torch.full((rows,), step % 2, dtype=torch.int32, device="cuda"))
        lc.adjust_logits(logits, **kw)
        want, mag = R.adjust(raw, **kw)
        inf = torch.isinf(want)
        assert torch.equal(torch.isinf(logits.cpu()), inf)
        assert ((logits.cpu().double() - want).abs()[~inf] <= (2.0 ** -24 * want.abs() + 4 * 2.0 ** -46 * mag + 1e-40)[~inf]).all()
        scores, token, parent = lc.beam_select(logits.view(batch, beams, V), scores, beams)
        assert bool(allow[step % 2][token.cpu().long().flatten()].all())
        lc.beam_reorder([history], parent)
        history.view(rows, -1).scatter_(1, seen.view(rows, 1).long(), token.reshape(rows, 1))
        seen += 1
        # fork, room for the token, and the token; the reference's own pages
        lc.kv8_fork(refs, table, parent)
        tail, granted = lc.kv8_grow(refs, table, length, torch.ones_like(length), page, 1)
        assert granted.all()
        length += 1
        _, k, v = project(token.reshape(-1).long())
        k, v = k.view(rows, heads, dim), v.view(rows, heads, dim)
        lc.kv8_append(cache, k, v, one, length.view(-1), table.view(rows, cols), 1, tail_src=tail.view(-1))
        ln = plen + step + 1
        old, ref = ref, {}
        for b in range(batch):
            for j in range(beams):
                ref[b, j] = []
                for (p, s), x in zip(old[b, int(parent[b, j])], (k, v)):
                    if p.shape[0] * page < ln:
                        p = torch.cat([p.view(torch.uint8), torch.zeros(1, heads, page, dim, dtype=torch.uint8)]).view(torch.float8_e4m3fn)
                        s = torch.cat([s, torch.ones(1, heads)])
                    ref[b, j].append(D.append(p, s, x[b * beams + j:b * beams + j + 1], [0, 1], [ln], torch.arange(p.shape[0])[None]))
        if step % 7 == 3:
            live = lc.kv8_compact([cache], refs, [table])
            assert int(live) == int((refs > 0).sum()) and bool((refs[:int(live)] > 0).all())
        held = table[table >= 0].long()
        assert torch.equal(refs, torch.bincount(held, minlength=n_pages).int())
        for (b, j), pair in ref.items():
            row = table[b, j, :-(-ln // page)].long()
            assert bool((row >= 0).all())
            for (p, s), gp, gs in zip(pair, (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
                for h in range(heads):
                    at = torch.arange(len(row))
                    assert torch.equal(D.gather(gp.cpu(), gs.cpu(), row.cpu(), ln, h), D.gather(p, s, at, ln, h))
    # the sequences end
    lc.kv8_free(refs, table, torch.zeros_like(length), page)
    assert not refs.any() and bool((table == -1).all())


def test_calls_at_once_on_two_streams(lc):
    """Every operator in two streams at a time, each with its own tensors and workspaces, gives what it gives alone."""
    def work(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randn(40, 20000, generator=g, device="cuda")
        hist = torch.randint(0, 20000, (40, 3000), generator=g, device="cuda", dtype=torch.int32)
        seen = torch.randint(0, 3000, (40,), generator=g, device="cuda", dtype=torch.int32)
        table = torch.randint(0, 3000, (30, 4, 60), generator=g, device="cuda", dtype=torch.int32)
        refs = torch.bincount(table.flatten().long(), minlength=5000).int()
        parent = torch.randint(0, 4, (30, 4), generator=g, device="cuda", dtype=torch.int32)
        length = torch.full((30, 4), 16 * 50 + 3, dtype=torch.int32, device="cuda")
        q = torch.randn(200, 8, 64, generator=g, device="cuda").to(torch.bfloat16)
        kv = torch.randn(3000, 2, 4, 64, generator=g, device="cuda").to(torch.bfloat16)
        at = torch.tensor([0, 100, 200], dtype=torch.int32, device="cuda")
        start, lens = torch.tensor([0, 900], dtype=torch.int32, device="cuda"), torch.tensor([900, 2100], dtype=torch.int32, device="cuda")
        ws, pws = lc.cross_attention_workspace(q, kv[:, 0], 100), lc.kv8_pages_workspace(5000, 120)
        out, tail, ok = torch.zeros_like(q), torch.empty_like(length), torch.empty(30, 4, dtype=torch.bool, device="cuda")
        y = torch.empty_like(x)

        def run(stream):
            lc.adjust_logits(x, hist, seen, frequency=torch.ones(40, device="cuda"), out=y, stream=stream)
            lc.kv8_fork(refs, table, parent, stream=stream)
            lc.kv8_grow(refs, table, length, torch.full_like(length, 2), 16, 2, out=(tail, ok), workspace=pws, stream=stream)
            lc.kv8_free(refs, table, length, 16, stream=stream)
            lc.cross_attention(q, kv[:, 0], kv[:, 1], at, start, lens, 100, out=out, workspace=ws, stream=stream)
        return run, (y, refs, table, tail, ok, out)

    want = []
    for seed in (1, 2):
        run, got = work(seed)
        for _ in range(3):
            run(None)
        want.append([t.clone() for t in got])
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = [work(seed) for seed in (1, 2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for (run, _), st in zip(both, streams):
            with torch.cuda.stream(st):
                run(st)
    torch.cuda.synchronize()
    for (_, got), w in zip(both, want):
        assert all(torch.equal(a, b) for a, b in zip(got, w))
