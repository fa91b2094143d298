"""The operators of a decoding loop around its cache and its logits, as they are measured: their
cases, a plain form of each in elementary torch operations, the framework's calls, and their
values in 64 bits.

  adjust   penalties for repeated tokens, biases and grammar masks on logits
  step     pages of a cache in one step of a loop: hypotheses fork, grow (a shared last page is
           replaced by one of their own) and give back what was rejected or finished
  copy     the contents of pages, to other pages, in every layer's cache
  compact  live pages moved to the front of every layer's cache, tables and counts with them
  cross    attention of each request's rows (beams, a drafted block) over states of another length
"""
import math

import torch

own = False

NEG = float("-inf")


# --------------------------------------------------------------------------------- cases

def listed():
    return [
        # one request's drafted block of 16: its rows share a history and see more of it row by row; every
        # penalty, some biases and a few grammars; f32 logits of an odd vocabulary, whose rows start off the
        # 16-byte grid: latency
        dict(name="adjust_block_f32", op="adjust", batch=1, group=16, vocab=32003, dtype="f32", history=1000, bias=5, masks=3,
             inplace=0),
        # a serving batch with long histories
        dict(name="adjust_large", op="adjust", batch=256, group=1, vocab=151936, dtype="bf16", history=4096, bias=64, masks=16,
             inplace=0),
        # grammars alone, written into the logits where they lie
        dict(name="adjust_mask", op="adjust", batch=128, group=4, vocab=151936, dtype="bf16", history=0, bias=0, masks=32,
             inplace=1),
        # one request of four beams, a token each
        dict(name="step_small", op="step", batch=1, beams=4, length=1000, cols=64, page=64, new=1, spare=64),
        # a batch of wide searches that check drafted blocks of 16, over tables of long contexts
        dict(name="step_large", op="step", batch=64, beams=16, length=16000, cols=512, page=64, new=16, spare=4096),
        # two pages of one layer: a prefix that goes on in two ways
        dict(name="copy_small", op="copy", layers=1, heads=8, page=64, dim=128, pages=2, pool=64),
        # a batch's pages in four layers' caches
        dict(name="copy_large", op="copy", layers=4, heads=8, page=64, dim=128, pages=2048, pool=4224),
        # half of a pool of four layers is live, strewn over it
        dict(name="compact_large", op="compact", layers=4, heads=8, page=64, dim=128, pool=4096, batch=64, cols=48),
        # a small pool of one layer
        dict(name="compact_small", op="compact", layers=1, heads=8, page=64, dim=128, pool=64, batch=4, cols=7),
        # one request's four beams, a token each, over 1,500 states
        dict(name="cross_single", op="cross", batch=1, new=4, length=1500, heads=16, group=1, dim=64, ragged=0),
        # a batch of requests of four beams over ragged states; grouped heads
        dict(name="cross_batch", op="cross", batch=128, new=4, length=4096, heads=8, group=4, dim=128, ragged=1),
        # whole prompts over a long encoder's states
        dict(name="cross_long", op="cross", batch=8, new=2048, length=4096, heads=8, group=4, dim=128, ragged=1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: an operator, its sizes over their ranges, cut where it would cost more than the largest listed case."""
    op = rng.choice(["adjust", "adjust", "step", "copy", "compact", "cross", "cross"])
    if op == "adjust":
        c = dict(op=op, batch=_log(rng, 1, 256), group=rng.choice([1, 1, 4, rng.randint(2, 16)]), vocab=_log(rng, 40, 160000),
                 dtype=rng.choice(["bf16", "bf16", "f32"]), history=_log(rng, 1, 32768), bias=rng.choice([0, _log(rng, 1, 300)]),
                 masks=rng.choice([0, rng.randint(1, 32)]), inplace=0)
        if rng.random() < 0.25:
            c.update(history=0, bias=0, masks=rng.randint(1, 32), inplace=1)
    elif op == "step":
        c = dict(op=op, batch=_log(rng, 1, 64), beams=rng.randint(1, 32), length=_log(rng, 1, 30000), page=rng.choice([16, 32, 64, 128]),
                 new=rng.choice([1, 1, 16, rng.randint(2, 64)]), spare=0)
        c["cols"] = (c["length"] + c["new"]) // c["page"] + rng.randint(1, 40)
        c["spare"] = 2 * c["batch"] * c["beams"] * (c["new"] // c["page"] + 2) + rng.randint(0, 500)
    elif op == "copy":
        n = _log(rng, 1, 2048)
        c = dict(op=op, layers=rng.randint(1, 4), heads=rng.choice([1, 2, 3, 8]), page=rng.choice([16, 32, 64, 128]),
                 dim=rng.choice([32, 64, 128]), pages=n, pool=2 * n + rng.randint(0, 100))
    elif op == "compact":
        c = dict(op=op, layers=rng.randint(1, 4), heads=rng.choice([1, 2, 3, 8]), page=rng.choice([16, 32, 64, 128]),
                 dim=rng.choice([32, 64, 128]), pool=_log(rng, 2, 4096), batch=_log(rng, 1, 64), cols=_log(rng, 1, 48))
    else:
        c = dict(op=op, batch=_log(rng, 1, 128), new=rng.choice([1, 4, 16, rng.randint(2, 40), _log(rng, 40, 2048)]),
                 length=_log(rng, 1, 16384), heads=rng.choice([1, 2, 4, 8, 16]), group=rng.choice([1, 1, 2, 3, 4, 5, 8]),
                 dim=rng.choice([32, 64, 80, 96, 128]), ragged=rng.randint(0, 1))
    top = {}
    for x in listed():
        top[x["op"]] = max(top.get(x["op"], 0), _cost(x))
    name = {"copy": "pages", "compact": "pool"}.get(op, "batch")
    while _cost(c) > top[op]:
        at = name if c[name] > 1 else "length"
        c[at] = max(1, c[at] * 3 // 4)
    return c


def _cost(case):
    w = work(case)
    return w["bytes"] + w["flops"] / 200


def _spread(n, lo, hi, ragged):
    """n whole numbers: hi for each, or spread over lo..hi with both ends among them."""
    if not ragged or n == 1:
        return [hi] * n
    return [hi if i == 0 else lo if i == 1 else lo + int((hi - lo) * ((i * 0.6180339887) % 1.0)) for i in range(n)]


def _allowed(case):
    """The share of the vocabulary that each grammar leaves: a few tokens, a class of them, nearly all."""
    return [(0.0005, 0.97, 0.2)[i % 3] for i in range(case["masks"])]


def _row_mask(case):
    """Each row's mask, -1 for one in eight without a grammar where there are several."""
    rows, m = case["batch"] * case["group"], case["masks"]
    return [-1 if m > 1 and r % 8 == 3 else (r * 7 + r // m) % m for r in range(rows)]


def _prompts(case):
    """Cached tokens of each batch entry of a step."""
    return _spread(case["batch"], max(1, case["length"] // 4), case["length"], case["batch"] > 1)


def _live(case):
    """Pages in use of a pool that is compacted."""
    return max(1, min(case["pool"] // 2, case["batch"] * case["cols"]))


def _page_bytes(case):
    return case["layers"] * case["heads"] * 2 * (case["page"] * case["dim"] + 4)


def work(case):
    op = case["op"]
    if op == "adjust":
        rows, v, es = case["batch"] * case["group"], case["vocab"], 4 if case["dtype"] == "f32" else 2
        words = -(-v // 32) * 4
        small = case["batch"] * (case["history"] * 4 + case["bias"] * 8 + 16) + rows * 8 + case["masks"] * words
        if case["inplace"]:
            off = [1 - x for x in _allowed(case)]
            return {"bytes": int(sum(off[i] for i in _row_mask(case) if i >= 0) * v * es) + small, "flops": 0}
        return {"bytes": rows * v * es * 2 + small, "flops": 4.0 * rows * v}
    if op == "step":
        rows = case["batch"] * case["beams"]
        held = sum(-(-t // case["page"]) for t in _prompts(case)) * case["beams"]
        # tables and counts once in and out, lengths, parents, new and kept tokens, sources and grants
        return {"bytes": held * 8 + _step_pool(case) * 8 + rows * 21, "flops": 0}
    if op == "copy":
        return {"bytes": case["pages"] * (2 * _page_bytes(case) + 8), "flops": 0}
    if op == "compact":
        live = _live(case)
        moved = int(live * (1 - live / case["pool"]))  # of pages strewn evenly
        return {"bytes": moved * 2 * _page_bytes(case) + case["pool"] * 8 + case["batch"] * case["cols"] * 8, "flops": 0}
    h, d, n = case["heads"], case["dim"], case["new"]
    q, total = h * case["group"], sum(_states(case))
    return {"bytes": total * h * d * 4 + case["batch"] * n * q * (d * 4 + 4), "flops": 4.0 * d * q * n * total}


def _states(case):
    return _spread(case["batch"], max(1, case["length"] // 8), case["length"], case["ragged"])


def _step_pool(case):
    """Pages of a step's pool: three quarters of a prompt's pages are shared by its beams, the others each beam's own."""
    counts = [-(-t // case["page"]) for t in _prompts(case)]
    return sum(n * 3 // 4 + (n - n * 3 // 4) * case["beams"] for n in counts) + case["spare"]


# ------------------------------------------------------------------------------- prepare

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 11)
    s = dict(case)
    {"adjust": _prepare_adjust, "step": _prepare_step, "copy": _prepare_copy, "compact": _prepare_compact,
     "cross": _prepare_cross}[case["op"]](case, s, g)
    return s


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prepare_adjust(case, s, g):
    b, w, v, t = case["batch"], case["group"], case["vocab"], case["history"]
    rows, dev = b * w, "cuda"
    rand = lambda *n: torch.rand(*n, generator=g, device=dev)  # noqa: E731
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    x = torch.empty(rows, v, dtype=dtype, device=dev)
    for r in range(0, rows, 64):  # a decoder's logits: a broad body with a head of high ones
        y = torch.randn(min(64, rows - r), v, generator=g, device=dev).mul_(1.5)
        n = min(v, 64)  # (at places of their own)
        at = (torch.randint(0, v, (y.shape[0], 1), generator=g, device=dev) + torch.arange(n, device=dev) * (v // n)) % v
        y.scatter_(1, at, 9.0 - 4.0 * rand(*at.shape))
        x[r:r + 64] = y.to(dtype)
    s["logits"] = x
    s["into"] = None if case["inplace"] else torch.zeros_like(x)
    s["history"] = s["seen"] = s["from"] = s["bias_ids"] = s["bias"] = s["mask"] = s["mask_at"] = None
    s["repetition"] = s["presence"] = s["frequency"] = None
    if t:
        # token ids fall off as words do, so that histories repeat themselves
        ids = ((rand(b, t + w) * math.log(v + 1)).exp() - 1).long().clamp_(0, v - 1)
        s["history"] = ((ids * 7919) % v).to(torch.int32)
        # row j of a block sees j tokens of it
        base = _ints(_spread(b, max(1, t // 4), t, b > 1))
        s["seen"] = (base[:, None] + torch.arange(w, device=dev, dtype=torch.int32)).reshape(rows).contiguous()
        s["from"] = base // 3  # the prompt's tokens are not counted
        s["repetition"] = 1 + 0.3 * rand(b)
        s["presence"] = 0.5 * rand(b)
        s["frequency"] = 0.4 * rand(b)
    if case["bias"]:
        s["bias_ids"] = torch.randint(0, v, (b, case["bias"]), generator=g, device=dev, dtype=torch.int32)
        s["bias"] = 4 * torch.randn(b, case["bias"], generator=g, device=dev)
    if case["masks"]:
        words = -(-v // 32)
        bits = rand(case["masks"], words * 32) < torch.tensor(_allowed(case), device=dev)[:, None]
        shifted = bits.view(case["masks"], words, 32).long() << torch.arange(32, device=dev)
        s["mask"] = shifted.sum(-1).to(torch.int32)
        s["mask_at"] = _ints(_row_mask(case))


def _prepare_step(case, s, g):
    b, w, cols, page, dev = case["batch"], case["beams"], case["cols"], case["page"], "cuda"
    pool = _step_pool(case)
    order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    table = torch.full((b, w, cols), -1, dtype=torch.int32, device=dev)
    at = 0
    for i, t in enumerate(_prompts(case)):
        n = -(-t // page)
        shared = n * 3 // 4
        table[i, :, :shared] = order[at:at + shared]
        at += shared
        table[i, :, shared:n] = order[at:at + (n - shared) * w].view(w, n - shared)
        at += (n - shared) * w
    s["table"] = table
    s["refs"] = torch.bincount(table[table >= 0], minlength=pool).to(torch.int32)
    # hypotheses that survive go on as themselves, the others as one of them
    lives = torch.rand(b, w, generator=g, device=dev) < 0.6
    lives[:, 0] = True
    pick = (torch.rand(b, w, w, generator=g, device=dev) * lives[:, None]).argmax(-1)
    s["parent"] = torch.where(lives, torch.arange(w, device=dev), pick).to(torch.int32)
    before = _ints(_prompts(case))[:, None].expand(b, w).contiguous()
    s["before"] = before
    s["new"], s["max_new"] = torch.full_like(before, case["new"]), case["new"]
    taken = torch.randint(1, case["new"] + 1, (b, w), generator=g, device=dev, dtype=torch.int32)
    done = ~lives & (torch.arange(w, device=dev) % 4 == 1)
    s["keep"] = torch.where(done, 0, before + taken).to(torch.int32)
    s["tail"] = torch.empty_like(before)
    s["granted"] = torch.empty(b, w, dtype=torch.bool, device=dev)
    if own:
        import draft_block_candidate_gb300 as lc
        s["workspace"] = lc.kv8_pages_workspace(pool, b * w, device=dev)


def _layers(case, g):
    """Caches of random codes (none of them NaN) and scales."""
    out = []
    n, h, page, d = case["pool"], case["heads"], case["page"], case["dim"]
    for _ in range(case["layers"]):
        k, v = (torch.randint(0, 254, (n, h, page, d), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2))
        for x in (k, v):
            x.add_((x >= 127).to(torch.uint8))
        ks, vs = (torch.exp2(torch.randint(-8, -5, (n, h), generator=g, device="cuda").float()) for _ in range(2))
        out.append((k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), ks, vs))
    return out


def _prepare_copy(case, s, g):
    s["layers"] = _layers(case, g)
    order = torch.randperm(case["pool"], generator=g, device="cuda").to(torch.int32)
    s["src"], s["dst"] = order[:case["pages"]].contiguous(), order[case["pages"]:2 * case["pages"]].contiguous()
    if own:
        import draft_block_candidate_gb300 as lc
        s["caches"] = [lc.KV8Cache.from_tensors(*x) for x in s["layers"]]


def _prepare_compact(case, s, g):
    s["layers"] = _layers(case, g)
    b, cols, live, pool = case["batch"], case["cols"], _live(case), case["pool"]
    order = torch.randperm(pool, generator=g, device="cuda")[:live].to(torch.int32)
    # every live page is held by a table's entry, some by several
    flat = torch.full((b * cols,), -1, dtype=torch.int32, device="cuda")
    flat[:live] = order
    more = b * cols - live
    again = torch.randint(0, live, (more,), generator=g, device="cuda")
    flat[live:] = torch.where(torch.rand(more, generator=g, device="cuda") < 0.3, order[again], -1)
    s["table"] = flat[torch.randperm(b * cols, generator=g, device="cuda")].view(b, cols)
    s["refs"] = torch.bincount(s["table"][s["table"] >= 0], minlength=pool).to(torch.int32)
    s["refs_to"], s["table_to"] = torch.zeros_like(s["refs"]), torch.zeros_like(s["table"])
    if own:
        import draft_block_candidate_gb300 as lc
        s["caches"] = [lc.KV8Cache.from_tensors(*x) for x in s["layers"]]
        s["workspace"] = lc.kv8_pages_workspace(pool, 1, device="cuda")


def _prepare_cross(case, s, g):
    b, n, h, d, q = case["batch"], case["new"], case["heads"], case["dim"], case["heads"] * case["group"]
    total = _states(case)
    rnd = lambda *x: torch.randn(*x, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    # keys and values of a projection, side by side; a request's states lie together
    kv = rnd(sum(total), 2, h, d)
    s["k"], s["v"] = kv[:, 0], kv[:, 1]
    ends = torch.tensor([0] + total).cumsum(0)
    s["kv_start"], s["kv_len"] = _ints(ends[:-1].tolist()), _ints(total)
    s["q_start"] = _ints([i * n for i in range(b + 1)])
    # two rows behind the last request, as a padded batch has them: their output stays as it was
    s["q"] = rnd(b * n + 2, q, d)
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(b * n + 2, q, device="cuda")
    s["scale"] = 1.0 / math.sqrt(d)
    if own:
        import draft_block_candidate_gb300 as lc
        s["workspace"] = lc.cross_attention_workspace(s["q"], s["k"], n)


# ----------------------------------------------------------------------------------- run

def run(s):
    op = s["op"]
    if own:
        import draft_block_candidate_gb300 as lc
        if op == "adjust":
            return lc.adjust_logits(s["logits"], history=s["history"], seen=s["seen"], counted_from=s["from"],
                                    repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
                                    bias_ids=s["bias_ids"], bias_values=s["bias"], mask=s["mask"], mask_index=s["mask_at"],
                                    out=s["into"])
        if op == "step":
            lc.kv8_fork(s["refs"], s["table"], s["parent"])
            lc.kv8_grow(s["refs"], s["table"], s["before"], s["new"], s["page"], s["max_new"],
                        out=(s["tail"], s["granted"]), workspace=s["workspace"])
            lc.kv8_free(s["refs"], s["table"], s["keep"], s["page"])
            return s["table"], s["refs"], s["tail"], s["granted"]
        if op == "copy":
            lc.kv8_copy(s["caches"], s["src"], s["dst"])
            return s["layers"]
        if op == "compact":
            live = lc.kv8_compact(s["caches"], s["refs"], [s["table"]], out=(s["refs_to"], [s["table_to"]]),
                                  workspace=s["workspace"])
            return s["layers"], s["refs_to"], s["table_to"], live
        return lc.cross_attention(s["q"], s["k"], s["v"], s["q_start"], s["kv_start"], s["kv_len"], s["new"], scale=s["scale"],
                                  out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return {"adjust": _adjust, "step": _step, "copy": _copy, "compact": _compact, "cross": _cross}[op](s)


def _seen_counts(s):
    """How often each token is among the seen ones of a row's history, and among those that count: [rows, vocab]."""
    rows, v = s["logits"].shape
    hist = s["history"].long().repeat_interleave(rows // s["history"].shape[0], 0)
    first = s["from"].repeat_interleave(rows // s["history"].shape[0])[:, None]
    pos = torch.arange(hist.shape[1], device=hist.device)
    seen = (pos < s["seen"][:, None]) & (hist >= 0) & (hist < v)
    out = []
    for which in (seen, seen & (pos >= first)):
        out.append(torch.zeros(rows, v, device=hist.device).scatter_add_(1, hist.clamp(0, v - 1), which.float()))
    return out


def _masked(s):
    """The tokens that a row's mask does not allow: [rows, vocab]."""
    v = s["logits"].shape[1]
    token = torch.arange(v, device=s["logits"].device)
    table = (s["mask"][:, token // 32] >> (token % 32).int()) & 1 == 0
    return table[s["mask_at"].long().clamp_min(0)] & (s["mask_at"] >= 0)[:, None]


def _adjust(s):
    into = s["logits"] if s["into"] is None else s["into"]
    if s["history"] is None and s["bias"] is None:
        if s["mask"] is None:
            return into.copy_(s["logits"])
        return into.copy_(s["logits"].masked_fill(_masked(s), NEG))
    x = s["logits"].double()  # penalties and biases may all but cancel
    each = lambda t: t.repeat_interleave(x.shape[0] // t.shape[0], 0)  # noqa: E731
    if s["history"] is not None:
        seen, counted = _seen_counts(s)
        rep = each(s["repetition"]).double()[:, None]
        x = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
        x -= each(s["frequency"]).double()[:, None] * counted + each(s["presence"]).double()[:, None] * (counted > 0)
        del seen, counted
    if s["bias"] is not None:
        for i in range(s["bias"].shape[1]):  # a token may be listed twice
            x.scatter_add_(1, each(s["bias_ids"][:, i:i + 1].long()), each(s["bias"][:, i:i + 1]).double())
    if s["mask"] is not None:
        x = x.masked_fill_(_masked(s), NEG)
    return into.copy_(x)


def _step(s):
    table, refs, page = s["table"], s["refs"], s["page"]
    b, w, cols = table.shape
    n = refs.shape[0]
    count = lambda ids, by: torch.zeros(n, dtype=torch.int32, device=refs.device).index_add_(0, ids.long(), by.to(torch.int32))  # noqa: E731
    # fork: row j becomes its parent's; a row's pages gain as many holders as it has children, less one
    parent = s["parent"].long()
    row = torch.arange(b, device=refs.device)[:, None]
    chosen = torch.zeros(b, w, dtype=torch.int32, device=refs.device).scatter_add_(1, parent, torch.ones_like(s["parent"]))
    held = table >= 0
    refs += count(table[held], (chosen - 1)[..., None].expand_as(table)[held])
    table.copy_(table[row, parent])
    # grow: columns from the last token's page to the last new one's; what is missing or shared is replaced
    before, new = s["before"].reshape(-1), s["new"].reshape(-1)
    flat = table.view(b * w, cols)
    col = torch.arange(cols, device=refs.device)
    wanted = (col >= (before // page)[:, None]) & (col < (-(-(before + new) // page))[:, None]) & (new > 0)[:, None]
    want = wanted & ((flat < 0) | (refs[flat.clamp_min(0).long()] > 1))
    free = torch.nonzero(refs == 0)[:, 0].to(torch.int32)
    need = want.sum(1)
    granted = (need.cumsum(0) <= free.shape[0]) | (need == 0)
    rank = (want.reshape(-1).long().cumsum(0) - 1).view_as(flat)
    do = want & granted[:, None]
    old = torch.where(do, flat, -1)
    flat[do] = free[rank[do]]
    refs += count(flat[do], torch.ones_like(flat[do])) - count(old[old >= 0], torch.ones_like(old[old >= 0]))
    first = (before // page).clamp_max(cols - 1)[:, None]
    partial = (before % page > 0) & (new > 0)
    s["tail"].copy_(torch.where(partial, old.gather(1, first.long())[:, 0], -1).view(b, w))
    s["granted"].copy_(granted.view(b, w))
    # free: pages behind the kept tokens
    gone = (col >= (-(-s["keep"].reshape(-1) // page))[:, None]) & (flat >= 0)
    refs -= count(flat[gone], torch.ones_like(flat[gone]))
    flat[gone] = -1
    return table, refs, s["tail"], s["granted"]


def _copy(s):
    for layer in s["layers"]:
        _move(layer, s["src"].long(), s["dst"].long())
    return s["layers"]


def _move(layer, src, dst):
    for x in layer:
        y = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
        y[dst] = y[src]


def _compact(s):
    refs, table = s["refs"], s["table"]
    live = refs > 0
    n = live.sum()
    at = torch.arange(refs.shape[0], device=refs.device)
    src, dst = torch.nonzero(live & (at >= n))[:, 0], torch.nonzero(~live & (at < n))[:, 0]
    for layer in s["layers"]:
        _move(layer, src, dst)
    to = at.clone()
    to[src] = dst
    s["refs_to"].copy_(refs)
    s["refs_to"][dst] = refs[src]
    s["refs_to"][src] = 0
    s["table_to"].copy_(torch.where(table >= 0, to[table.clamp_min(0).long()], -1))
    return s["layers"], s["refs_to"], s["table_to"], n.to(torch.int32).reshape(1)


def _cross(s):
    """softmax(scale * q k^T) v over all states of a request, for each of its rows."""
    d, h, n = s["q"].shape[-1], s["k"].shape[1], s["new"]
    b = s["kv_len"].shape[0]
    group = s["q"].shape[1] // h
    longest = s["length"]
    pos = torch.arange(longest, device="cuda")
    there = pos < s["kv_len"][:, None]
    at = (s["kv_start"].long()[:, None] + pos).clamp_max(s["k"].shape[0] - 1)
    q = s["q"][:b * n].float().view(b, n, h, group, d).permute(0, 2, 3, 1, 4).reshape(b, h, group * n, d)
    k, v = (x[at].float().masked_fill_(~there[..., None, None], 0).transpose(1, 2) for x in (s["k"], s["v"]))
    o = torch.empty_like(q)
    lse = torch.empty(b, h, group * n, device="cuda")
    step = max(1, (1 << 31) // (group * n * longest * h))  # requests at a time
    for i in range(0, b, step):
        x = torch.matmul(q[i:i + step], k[i:i + step].transpose(-1, -2)).mul_(s["scale"])
        x.masked_fill_(~there[i:i + step, None, None], NEG)
        top = x.amax(-1, keepdim=True)
        p = x.sub_(top).exp_()
        mass = p.sum(-1, keepdim=True)
        o[i:i + step] = torch.matmul(p, v[i:i + step]) / mass
        lse[i:i + step] = (torch.log(mass) + top)[..., 0]
    s["out"][:b * n] = o.view(b, h, group, n, d).permute(0, 3, 1, 2, 4).reshape(b * n, h * group, d).to(s["out"].dtype)
    s["lse"][:b * n] = lse.view(b, h, group, n).permute(0, 3, 1, 2).reshape(b * n, h * group)
    return s["out"], s["lse"]


# --------------------------------------------------------------------------------- exact

def exact(case, seed):
    """The same outputs in 64 bits, row by row or head by head; None for what is moved and not computed."""
    if case["op"] == "adjust":
        return _adjust_exact(case, prepare(case, seed))
    if case["op"] == "cross":
        return _cross_exact(case, prepare(case, seed))
    return None


def _adjust_exact(case, s):
    rows, v = s["logits"].shape
    out = s["logits"].double()
    seen = None if s["seen"] is None else s["seen"].tolist()
    first = None if s["from"] is None else s["from"].tolist()
    shift = torch.arange(32, device="cuda")
    allowed = None if s["mask"] is None else ((s["mask"][..., None] >> shift) & 1).flatten(1)[:, :v].bool()
    for r in range(rows):
        i = r // case["group"]
        x = out[r]
        if s["history"] is not None:
            ids, times = torch.unique(s["history"][i, :seen[r]].long(), return_counts=True)
            rep = s["repetition"][i].double()
            x[ids] = torch.where(x[ids] > 0, x[ids] / rep, x[ids] * rep)
            ids, times = torch.unique(s["history"][i, first[i]:seen[r]].long(), return_counts=True)
            x[ids] -= s["frequency"][i].double() * times + s["presence"][i].double()
        if s["bias"] is not None:
            x.index_put_((s["bias_ids"][i].long(),), s["bias"][i].double(), accumulate=True)
        if allowed is not None and int(s["mask_at"][r]) >= 0:
            x[~allowed[int(s["mask_at"][r])]] = NEG
    return out


def _cross_exact(case, s):
    h, g, n, d = case["heads"], case["group"], case["new"], case["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for i, t in enumerate(_states(case)):
        for j in range(h):
            k, v = (x[at:at + t, j].double() for x in (s["k"], s["v"]))
            heads = slice(j * g, (j + 1) * g)
            x = torch.einsum("ngd,td->ngt", s["q"][i * n:(i + 1) * n, heads].double(), k) * s["scale"]
            norm = torch.logsumexp(x, -1)
            lse[i * n:(i + 1) * n, heads] = norm
            out[i * n:(i + 1) * n, heads] = torch.einsum("ngt,td->ngd", torch.exp(x - norm[..., None]), v)
        at += t
    return out, lse
