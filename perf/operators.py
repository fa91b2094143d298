"""The decoding operators next to the rerank, as they are measured: their cases, a plain form
of each in elementary torch operations, the framework's calls, and their values in 64 bits.

  select    beam search's choice over beams and vocabulary from one step's logits
  reorder   per-beam states gathered by the chosen parents
  append    new keys and values into a paged cache of 8-bit values (e4m3) with one
            power-of-two scale for each page (block of tokens) and key/value head
  attend    attention of each sequence's last tokens over that cache
"""
import math

import torch

own = False

NEG = float("-inf")
SCALE_MIN_EXP = -60  # the smallest page scale is 2^-60
E4M3_MAX = 448.0


# --------------------------------------------------------------------------------- cases

def listed():
    return [
        # one request, four hypotheses, twice as many candidates for the caller's stop rules
        dict(name="select_single", op="select", batch=1, beams=4, vocab=151936, out=8, dtype="bf16", done=0),
        # f32 logits, odd sizes: rows start off the 16-byte grid; some beams have finished
        dict(name="select_f32_odd", op="select", batch=9, beams=5, vocab=32003, out=7, dtype="f32", done=1),
        # a full serving batch of wide searches
        dict(name="select_large", op="select", batch=128, beams=16, vocab=151936, out=32, dtype="bf16", done=1),
        # token history and block tables of a small batch: latency
        dict(name="reorder_small", op="reorder", batch=4, beams=4, kind="tables", length=129, heads=1, dim=1),
        # contiguous bf16 caches of 8 requests' beams, the used part of a larger capacity
        dict(name="reorder_large", op="reorder", batch=8, beams=8, kind="cache", length=1000, heads=8, dim=128),
        # one token for each sequence of a batch: every tail page grows by a row
        dict(name="append_token", op="append", batch=64, new=1, before=4000, heads=8, page=64, dim=128, ragged=1),
        # a drafted block of 16 for each sequence, small pages and heads
        dict(name="append_block", op="append", batch=256, new=16, before=500, heads=4, page=16, dim=64, ragged=1),
        # prompts of up to 4,096 tokens
        dict(name="append_prompt", op="append", batch=16, new=4096, before=0, heads=8, page=64, dim=128, ragged=1),
        # one short request, one token: latency
        dict(name="attend_single", op="attend", batch=1, new=1, length=1000, heads=8, group=4, page=64, dim=128, ragged=0),
        # two long contexts, one token each: few rows over a long axis
        dict(name="attend_long", op="attend", batch=2, new=1, length=131072, heads=8, group=8, page=64, dim=128, ragged=1),
        # a serving batch of single tokens over ragged contexts
        dict(name="attend_batch", op="attend", batch=128, new=1, length=8192, heads=8, group=4, page=64, dim=128, ragged=1),
        # the committed block of 16 checked for a batch: causal among its own tokens
        dict(name="attend_block", op="attend", batch=64, new=16, length=4096, heads=8, group=8, page=64, dim=128, ragged=1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: an operator, its sizes over their ranges, the batch cut where it would cost more than the largest listed case."""
    op = rng.choice(["select", "reorder", "append", "attend", "attend"])
    if op == "select":
        c = dict(op=op, batch=_log(rng, 1, 128), beams=rng.randint(1, 32), vocab=_log(rng, 40, 160000),
                 out=rng.randint(1, 32), dtype=rng.choice(["bf16", "bf16", "f32"]), done=rng.randint(0, 1))
    elif op == "reorder":
        c = dict(op=op, batch=_log(rng, 1, 64), beams=rng.randint(1, 32), kind=rng.choice(["tables", "cache"]),
                 length=_log(rng, 1, 4096), heads=rng.choice([1, 2, 8]), dim=rng.choice([32, 64, 80, 128]))
    elif op == "append":
        c = dict(op=op, batch=_log(rng, 1, 256), new=_log(rng, 1, 4096), before=rng.choice([0, _log(rng, 1, 4096)]),
                 heads=rng.choice([1, 2, 3, 8]), page=rng.choice([16, 32, 64, 128]), dim=rng.choice([32, 64, 128]),
                 ragged=rng.randint(0, 1))
    else:
        c = dict(op=op, batch=_log(rng, 1, 128), new=rng.choice([1, 1, 1, rng.randint(2, 8), 16, rng.randint(9, 64)]),
                 length=_log(rng, 1, 131072), heads=rng.choice([1, 2, 4, 8]), group=rng.choice([1, 2, 3, 4, 5, 8, 16]),
                 page=rng.choice([16, 32, 64, 128]), dim=rng.choice([32, 64, 128]), ragged=rng.randint(0, 1),
                 uneven=rng.randint(0, 1))
    top = {}
    for x in listed():
        w = work(x)
        top[x["op"]] = max(top.get(x["op"], 0), w["bytes"] + w["flops"] / 200)
    while (lambda w: w["bytes"] + w["flops"] / 200)(work(c)) > top[op]:
        name = "batch" if c["batch"] > 1 else "length"
        c[name] = max(1, c[name] * 3 // 4)
    return c


def _spread(n, lo, hi, ragged):
    """n whole numbers: hi for each, or spread over lo..hi with both ends among them."""
    if not ragged or n == 1:
        return [hi] * n
    return [hi if i == 0 else lo if i == 1 else lo + int((hi - lo) * ((i * 0.6180339887) % 1.0)) for i in range(n)]


def _lengths(case):
    """(new tokens, cached tokens after them) of each sequence: a matter of the case, not of the seed."""
    b, n = case["batch"], case["new"]
    if case["op"] == "append":
        new = _spread(b, 1, n, case["ragged"] and n > 64)
        before = _spread(b, case["before"] // 2, case["before"], case["ragged"])
        return new, [x + y for x, y in zip(new, before)]
    new = _spread(b, 1, n, case.get("uneven"))  # a drawn case's sequences may bring different numbers of tokens
    total = _spread(b, max(n, case["length"] // 8), max(n, case["length"]), case["ragged"])
    return new, total


def work(case):
    op = case["op"]
    if op == "select":
        rows = case["batch"] * case["beams"]
        es = 4 if case["dtype"] == "f32" else 2
        # finished beams (one in eight where there are any) have no logits to read
        live = rows - len(_done_rows(case))
        return {"bytes": live * case["vocab"] * es + rows * 5 + case["batch"] * case["out"] * 12, "flops": 4.0 * live * case["vocab"]}
    if op == "reorder":
        w = case["beams"]
        parents = w * (1 - (1 - 1 / w) ** w)  # distinct ones, as drawn evenly
        return {"bytes": case["batch"] * (parents + w) * sum(math.prod(s) * e for s, e in _state_shapes(case)), "flops": 0}
    new, total = _lengths(case)
    h, d, page = case["heads"], case["dim"], case["page"]
    if op == "append":
        pages = sum(-(-t // page) - (t - n) // page for n, t in zip(new, total))
        # the new rows once in, once out as 8 bits, a scale and a table entry for each page
        return {"bytes": sum(new) * h * d * 2 * (2 + 1) + pages * (h * 16 + 4), "flops": sum(new) * h * d * 4.0}
    q = h * case["group"]
    pages = sum(-(-t // page) for t in total)
    pairs = sum(sum(t - n + i + 1 for i in range(n)) for n, t in zip(new, total))
    return {"bytes": sum(total) * h * d * 2 + pages * (h * 8 + 4) + sum(new) * q * (d * 4 + 4), "flops": 4.0 * d * q * pairs}


# ------------------------------------------------------------------------------- prepare

def _done_rows(case):
    rows = case["batch"] * case["beams"]
    return [r for r in range(rows) if case["done"] and r % 8 == 5]


def _state_shapes(case):
    """(shape behind [batch, beams], bytes an element) of each state of a reorder case."""
    t = case["length"]
    if case["kind"] == "tables":  # token history, block table, lengths
        return [((t,), 4), ((-(-t // 16),), 4), ((), 4)]
    return [((case["heads"], t, case["dim"]), 2)] * 4  # keys and values of two layers


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 7)
    dev = "cuda"
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    s = dict(case)
    op, b = case["op"], case["batch"]
    if op == "select":
        w, v = case["beams"], case["vocab"]
        # a decoder's logits: a broad body, a peaked head of falling candidates at places of their own
        x = rnd(b, w, v).mul_(1.5)
        n = min(v, 64)
        at = torch.randint(0, v, (b, w, 1), generator=g, device=dev)
        at = (at + torch.arange(n, device=dev) * (v // n)) % v
        peak = 9.0 - 1.1 * torch.log(torch.arange(1, n + 1, device=dev, dtype=torch.float32))
        x.scatter_(2, at, (peak + 0.3 * rnd(b, w, n)))
        s["logits"] = x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
        s["scores"] = -torch.rand(b, w, generator=g, device=dev).mul_(6.0) - 20.0
        done = torch.zeros(b * w, dtype=torch.bool, device=dev)
        if _done_rows(case):
            done[torch.tensor(_done_rows(case), device=dev)] = True
        s["done"] = done.view(b, w)
        s["pad"] = 0
        if own:
            import draft_block_candidate_gb300 as lc
            s["workspace"] = lc.beam_select_workspace(s["logits"], case["out"])
        return s
    if op == "reorder":
        w = case["beams"]
        s["parent"] = torch.randint(0, w, (b, w), generator=g, device=dev, dtype=torch.int32)
        s["states"], s["into"] = [], []
        for shape, size in _state_shapes(case):
            if size == 4:
                t = torch.randint(0, 1 << 20, (b, w, *shape), generator=g, device=dev, dtype=torch.int32)
                s["states"].append(t)
                s["into"].append(torch.zeros_like(t))
            else:  # the used part of a cache whose capacity is a quarter larger
                heads, length, dim = shape
                full = rnd(b, w, heads, length + length // 4 + 8, dim).to(torch.bfloat16)
                s["states"].append(full[:, :, :, :length])
                s["into"].append(torch.zeros_like(full)[:, :, :, :length])
        return s
    new, total = _lengths(case)
    h, d, page = case["heads"], case["dim"], case["page"]
    counts = [-(-t // page) for t in total]
    cols = max(counts)
    n_pages = sum(counts) + 3
    order = torch.randperm(n_pages, generator=g, device=dev)[:sum(counts)].to(torch.int32)
    table = torch.full((b, cols), -1, dtype=torch.int32, device=dev)
    held = torch.arange(cols, device=dev)[None] < torch.tensor(counts, device=dev)[:, None]
    table[held] = order
    s["table"] = table
    s["kv_len"] = torch.tensor(total, dtype=torch.int32, device=dev)
    ends = torch.tensor([0] + new, device=dev).cumsum(0)
    s["q_start"] = ends.to(torch.int32)
    rows = sum(new)
    s["max_new"] = max(new)
    # pages as an earlier append left them: codes of normal values, scales about 2^-6 .. 2^-8
    code = lambda: (rnd(n_pages, h, page, d) * 112).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)  # noqa: E731
    scale = lambda: torch.exp2(torch.randint(-8, -5, (n_pages, h), generator=g, device=dev).float())  # noqa: E731
    s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"] = code(), code(), scale(), scale()
    if op == "append":
        s["k"] = (rnd(rows, h, d) * torch.exp(0.5 * rnd(1, h, d))).to(torch.bfloat16)
        s["v"] = rnd(rows, h, d).to(torch.bfloat16)
    else:
        # two rows behind the last sequence, as a padded batch has them: their output stays as it was
        s["q"] = rnd(rows + 2, h * case["group"], d).to(torch.bfloat16)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(rows + 2, h * case["group"], device=dev)
        s["scale"] = 1.0 / math.sqrt(d)
    if own:
        import draft_block_candidate_gb300 as lc
        s["cache"] = lc.KV8Cache.from_tensors(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
        if op == "attend":
            s["workspace"] = lc.kv8_attention_workspace(s["q"], s["cache"], s["table"], s["max_new"])
    return s


# ----------------------------------------------------------------------------------- run

def run(s):
    op = s["op"]
    if own:
        import draft_block_candidate_gb300 as lc
        if op == "select":
            return lc.beam_select(s["logits"], s["scores"], s["out"], finished=s["done"], pad_id=s["pad"],
                                  workspace=s["workspace"])
        if op == "reorder":
            return lc.beam_reorder(s["states"], s["parent"], out=s["into"])
        if op == "append":
            lc.kv8_append(s["cache"], s["k"], s["v"], s["q_start"], s["kv_len"], s["table"], s["max_new"])
            return s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]
        return lc.kv8_attention(s["q"], s["cache"], s["q_start"], s["kv_len"], s["table"], s["max_new"],
                                scale=s["scale"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return {"select": _select, "reorder": _reorder, "append": _append, "attend": _attend}[op](s)


def _select(s):
    """score(i, v) = scores[i] + logits[i, v] - logsumexp(logits[i]): the `out` best by (score, then the lowest i * vocab + v)."""
    x, m = s["logits"], s["out"]
    b, w, v = x.shape
    xd = x.double()  # a candidate's rank is decided by differences far below 32 bits' rounding of a score
    top = xd.amax(-1, keepdim=True)
    lse = top + torch.log(torch.exp(xd - top).sum(-1, keepdim=True))
    # the best of each beam: equal logits by the lower token, through whole keys that have no equals
    bits = (x.float() + 0.0).view(torch.int32).long()
    key = (torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF)) << 32) + (v - 1 - torch.arange(v, device=x.device))
    k = min(m, v)
    token = v - 1 - (torch.topk(key, k, dim=-1).values & 0xFFFFFFFF)
    del key, bits
    score = s["scores"].double()[..., None] + (xd.gather(-1, token) - lse)
    # a finished beam goes on as itself, with the pad token and its score
    first = torch.arange(k, device=x.device) == 0
    score = torch.where(s["done"][..., None], torch.where(first, s["scores"].double()[..., None], NEG), score)
    token = torch.where(s["done"][..., None], s["pad"], token)
    score = torch.where(score > NEG, score, NEG)
    score, at = torch.sort(score.reshape(b, w * k), dim=-1, descending=True, stable=True)
    n = min(m, w * k)
    out = torch.full((b, m), NEG, device=x.device)
    out[:, :n] = score[:, :n].float()
    ids = torch.full((b, m), s["pad"], dtype=torch.int32, device=x.device)
    parent = torch.zeros(b, m, dtype=torch.int32, device=x.device)
    there = out[:, :n] > NEG
    ids[:, :n] = torch.where(there, token.reshape(b, w * k).gather(-1, at[:, :n]), s["pad"]).int()
    parent[:, :n] = torch.where(there, at[:, :n] // k, 0).int()
    return out, ids, parent


def _reorder(s):
    row = torch.arange(s["parent"].shape[0], device=s["parent"].device)[:, None]
    p = s["parent"].long()
    return [into.copy_(t[row, p]) for t, into in zip(s["states"], s["into"])]


def _page_scale(amax):
    """The smallest power of two s >= 2^-60 with amax / s <= 448 = 0.875 * 2^9."""
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, SCALE_MIN_EXP).clamp_min(SCALE_MIN_EXP))


def _append(s):
    page = s["k_pages"].shape[2]
    start, total = s["q_start"].long(), s["kv_len"].long()
    before = total - (start[1:] - start[:-1])
    cols = (s["max_new"] + page - 2) // page + 1
    dev = total.device
    at = before[:, None] // page + torch.arange(cols, device=dev)  # [batch, cols]: the pages that grow
    touched = (at * page < total[:, None]) & (total > before)[:, None]
    ids = s["table"].long().gather(1, at.clamp_max(s["table"].shape[1] - 1))[touched]
    pos = (at[..., None] * page + torch.arange(page, device=dev))[touched]  # [pages, page]
    lo, hi = (t[:, None].expand_as(at)[touched][:, None] for t in (before, total))
    fresh = (pos >= lo) & (pos < hi)
    old = pos < lo
    src = (start[:-1, None].expand_as(at)[touched][:, None] + pos - lo).clamp(0, s["k"].shape[0] - 1)
    for x, pages, scales in ((s["k"], s["k_pages"], s["k_scale"]), (s["v"], s["v_pages"], s["v_scale"])):
        rows = x[src].float().transpose(1, 2)  # [pages, heads, page, dim]
        there, kept = fresh[:, None, :, None], old[:, None, :, None]
        size = torch.where(there & torch.isfinite(rows), rows.abs(), 0).amax((2, 3))
        was = scales[ids]
        now = torch.maximum(_page_scale(size), torch.where(old.any(-1)[:, None], was, 0))
        had = pages.view(torch.uint8)[ids]
        moved = (had.view(torch.float8_e4m3fn).float() * (was / now)[..., None, None]).to(torch.float8_e4m3fn)
        coded = (rows / now[..., None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        both = torch.where(there, coded.view(torch.uint8), torch.where(kept, moved.view(torch.uint8), had))
        pages.view(torch.uint8)[ids] = both
        scales[ids] = now
    return s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]


def _attend(s):
    """softmax(scale * q k^T) v; the i-th of n new tokens sees the first length - n + i + 1 cached ones."""
    dev = s["q"].device
    start, total, n_max = s["q_start"].long(), s["kv_len"].long(), s["max_new"]
    b = total.shape[0]
    d = s["q"].shape[-1]
    h = s["k_pages"].shape[1]
    row = start[:-1, None] + torch.arange(n_max, device=dev)
    there = row < start[1:, None]
    q = s["q"][row.clamp_max(s["q"].shape[0] - 1)].float()  # [b, n, heads * group, d]
    group = q.shape[2] // h
    q = q.reshape(b, n_max, h, group, d).permute(0, 2, 3, 1, 4).reshape(b, h, group * n_max, d)
    ids = s["table"].long().clamp_min(0)

    def whole(pages, scales):
        x = pages.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float() * scales[ids][..., None, None]
        return x.transpose(1, 2).reshape(b, h, -1, d)  # [b, heads, tokens, d]

    score = torch.matmul(q, whole(s["k_pages"], s["k_scale"]).transpose(-1, -2)).mul_(s["scale"])
    seen = total[:, None] - (start[1:] - start[:-1])[:, None] + torch.arange(n_max, device=dev) + 1
    seen = seen[:, None, :].expand(b, group, n_max).reshape(b, 1, group * n_max, 1)
    score.masked_fill_(torch.arange(score.shape[-1], device=dev) >= seen, NEG)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top > NEG, top, 0)).exp_()
    mass = p.sum(-1, keepdim=True)
    o = torch.matmul(p, whole(s["v_pages"], s["v_scale"])) / torch.where(mass > 0, mass, 1)
    lse = (torch.log(mass) + top)[..., 0]
    o = o.reshape(b, h, group, n_max, d).permute(0, 3, 1, 2, 4).reshape(b, n_max, h * group, d)
    lse = lse.reshape(b, h, group, n_max).permute(0, 3, 1, 2).reshape(b, n_max, h * group)
    s["out"][row[there]] = o[there].to(s["out"].dtype)
    s["lse"][row[there]] = lse[there]
    return s["out"], s["lse"]


# --------------------------------------------------------------------------------- exact

def exact(case, seed):
    """The same outputs in 64 bits, sequence by sequence; None where it would take too long."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "reorder":
        return [torch.stack([x[i, rows.tolist()].double() for i, rows in enumerate(s["parent"])]) if x.dtype == torch.bfloat16
                else None for x in s["states"]] if case["kind"] == "cache" else None
    if op == "append":
        if case["batch"] * case["new"] > 70000:
            return None
        return _append_exact(case, s)
    if op == "select":
        return _select_exact(s)
    return _attend_exact(case, s)


def _select_exact(s):
    b, w, v = s["logits"].shape
    out = torch.full((b, s["out"]), NEG, dtype=torch.float64, device="cuda")
    for i in range(b):
        rows = torch.log_softmax(s["logits"][i].double(), -1) + s["scores"][i].double()[:, None]
        rows[s["done"][i]] = NEG
        flat = torch.cat([rows.flatten(), s["scores"][i].double()[s["done"][i]]])
        best = torch.topk(flat, min(s["out"], flat.numel())).values
        out[i, :best.numel()] = best
    return out, None, None


def _append_exact(case, s):
    """Scales are exact; a stored code is within half a step of e4m3, so what it holds has no 64-bit value of its own."""
    page = case["page"]
    new, total = _lengths(case)
    steps = torch.arange(SCALE_MIN_EXP, 125, device="cuda").double()
    holds = E4M3_MAX * torch.exp2(steps)  # the largest value that each scale can hold
    got = []
    for x, scales in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
        out = scales.double().clone()
        mag = x.double().abs().amax(-1)  # [rows, heads]
        at = 0
        for i, (n, t) in enumerate(zip(new, total)):
            for p in range((t - n) // page, -(-t // page)):
                lo, hi = max(t - n, p * page), min(t, (p + 1) * page)
                a = mag[at + lo - (t - n):at + hi - (t - n)].amax(0)
                need = torch.exp2(steps[torch.searchsorted(holds, a)])
                ids = s["table"][i, p].long()
                out[ids] = torch.maximum(need, out[ids]) if p * page < t - n else need
            at += n
        got.append(out)
    return None, None, got[0], got[1]


def _attend_exact(case, s):
    new, total = _lengths(case)
    page, h, g, d = case["page"], case["heads"], case["group"], case["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for i, (n, t) in enumerate(zip(new, total)):
        ids = s["table"][i, :-(-t // page)].long()
        q = s["q"][at:at + n].double().view(n, h, g, d)
        for j in range(h):
            k, v = (torch.mul(p.view(torch.uint8)[ids, j].view(torch.float8_e4m3fn).double(), c[ids, j].double()[:, None, None])
                    .reshape(-1, d)[:t] for p, c in ((s["k_pages"], s["k_scale"]), (s["v_pages"], s["v_scale"])))
            x = (q[:, j].reshape(n * g, d) @ k.T) * s["scale"]
            late = torch.arange(t, device="cuda")[None] > (t - n + torch.arange(n, device="cuda"))[:, None]
            x = x.view(n, g, t).masked_fill(late[:, None], NEG)
            norm = torch.logsumexp(x, -1)
            lse[at:at + n, j * g:(j + 1) * g] = norm
            out[at:at + n, j * g:(j + 1) * g] = (torch.exp(x - norm[..., None]).reshape(n * g, t) @ v).view(n, g, d)
        at += n
    return out, lse
