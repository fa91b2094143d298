"""Plain float64 forms of the decoding operators, step by step, for the tests to compare with.

Everything runs on CPU tensors; codes are torch.float8_e4m3fn values widened exactly."""
import math

import torch

NEG = -math.inf


def e4m3(codes: torch.Tensor) -> torch.Tensor:
    return codes.cpu().to(torch.float64)


def select(logits, scores, n_out, finished=None, pad_id=0):
    """Per batch entry the sorted list of all candidates [(score, parent, token)], best first,
    by (score desc, parent * V + token asc); and the filled-up outputs."""
    x = logits.cpu().to(torch.float64)
    b, w, v = x.shape
    every, outs = [], []
    for i in range(b):
        cand = []
        for j in range(w):
            s = float(scores[i, j])
            if not s > NEG:
                continue
            if finished is not None and bool(finished[i, j]):
                cand.append((s, j, pad_id, j * v))
                continue
            row = x[i, j]
            if not bool((row > NEG).any()):
                continue
            sc = s + (row - torch.logsumexp(row, 0))
            keep = torch.topk(sc, min(v, n_out + 40)).values[-1]
            for t in torch.nonzero((sc >= keep) & (sc > NEG))[:, 0].tolist():
                cand.append((float(sc[t]), j, t, j * v + t))
        cand.sort(key=lambda c: (-c[0], c[3]))
        every.append(cand)
        outs.append([c[:3] for c in cand[:n_out]] + [(NEG, 0, pad_id)] * max(0, n_out - len(cand)))
    return every, outs


def page_scale(amax: float) -> float:
    """The smallest power of two s >= 2^-60 with amax / s <= 448."""
    s = 2.0 ** -60
    while amax / s > 448.0:
        s *= 2.0
    return s


def append(pages, scales, x, q_start, kv_len, table, tail_src=None):
    """New (pages, scales) after writing rows x [total, heads, D] (any sign of NaN kept NaN)."""
    pages, scales = pages.cpu().clone(), scales.cpu().clone()
    page = pages.shape[2]
    raw = pages.view(torch.uint8)
    old_raw, old_scales = raw.clone(), scales.clone()
    x = x.cpu().to(torch.float32)
    for b in range(len(kv_len)):
        q0, n, ln = int(q_start[b]), int(q_start[b + 1] - q_start[b]), int(kv_len[b])
        if n == 0:
            continue
        before = ln - n
        for at in range(before // page, (ln + page - 1) // page):
            lo, hi = max(before, at * page), min(ln, (at + 1) * page)
            dst = int(table[b, at])
            src = dst
            if at * page < before and tail_src is not None and int(tail_src[b]) >= 0:
                src = int(tail_src[b])
            for h in range(pages.shape[1]):
                rows = x[q0 + lo - before:q0 + hi - before, h]
                fin = rows[torch.isfinite(rows)].abs()
                s = page_scale(float(fin.max()) if fin.numel() else 0.0)
                if at * page < before:
                    was = float(old_scales[src, h])
                    s = max(s, was)
                    k = lo - at * page
                    had = old_raw[src, h, :k].view(torch.float8_e4m3fn).to(torch.float32)
                    raw[dst, h, :k] = (had * (was / s)).to(torch.float8_e4m3fn).view(torch.uint8)
                code = (rows / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
                raw[dst, h, lo - at * page:hi - at * page] = code.view(torch.uint8)
                scales[dst, h] = s
    return pages, scales


def gather(pages, scales, table_row, n_tokens, head):
    """Float64 rows [n_tokens, D] of one sequence and head."""
    page, D = pages.shape[2], pages.shape[3]
    out = torch.zeros(n_tokens, D, dtype=torch.float64)
    for at in range((n_tokens + page - 1) // page):
        i = int(table_row[at])
        k = min(page, n_tokens - at * page)
        out[at * page:at * page + k] = e4m3(pages[i, head, :k]) * float(scales[i, head])
    return out


def attention(q, k_pages, v_pages, k_scale, v_scale, q_start, kv_len, table, scale):
    """(out, lse, tolerance of out, tolerance of lse), float64, rows outside the sequences NaN.

    Tolerances: with p the softmax weights and D the head dimension,
      * q is split into two e4m3 values, exactly but for 2^-17 of its row's largest; a score is
        an f32 sum of 2 D products and one f32 fma: it is off by at most
        e = (2 D + 4) 2^-24 (scale sum|q k|) + 2^-17 max|q| (scale sum|k|) + 2^-23 |score|
            + 2^-23 |log2 of the value scale|,
        and so is the lse, with one rounding of the lse and a few of exp2, log2 and their sum
        (each below 2^-21) on top;
      * a weight is off by that relative amount and by its rounding: to f16 (2^-11 of its value,
        or 2^-25 of the row's largest weight times value scale where it is f16-subnormal), or to
        f16 and then to a sum of three e5m2 values of 3 bits (2^-12 + 2^-9 of its value);
      * the f32 sums over T tokens in runs of 16: (T / 16 + 40) 2^-24 of sum p |v|;
      * out is rounded to bf16 once: half a step, 2^-8 of its value."""
    total, q_heads, D = q.shape
    heads = k_pages.shape[1]
    group = q_heads // heads
    nan = float("nan")
    out = torch.full((total, q_heads, D), nan, dtype=torch.float64)
    lse = torch.full((total, q_heads), nan, dtype=torch.float64)
    to, tl = torch.zeros_like(out), torch.zeros_like(lse)
    q = q.cpu().to(torch.float64)
    k_pages, v_pages, k_scale, v_scale, table = (t.cpu() for t in (k_pages, v_pages, k_scale, v_scale, table))
    page = k_pages.shape[2]
    for b in range(len(kv_len)):
        q0, n, ln = int(q_start[b]), int(q_start[b + 1] - q_start[b]), int(kv_len[b])
        for h in range(heads):
            if n == 0:
                continue
            k, v = gather(k_pages, k_scale, table[b], ln, h), gather(v_pages, v_scale, table[b], ln, h)
            vs = torch.tensor([float(v_scale[int(table[b, t // page]), h]) for t in range(ln)], dtype=torch.float64)
            for i in range(n):
                t = max(0, ln - n + i + 1)
                for j in range(group):
                    r, c = q0 + i, h * group + j
                    if t == 0:
                        out[r, c], lse[r, c] = 0.0, NEG
                        continue
                    s = (k[:t] @ q[r, c]) * scale
                    mag = (k[:t].abs() @ q[r, c].abs()) * abs(scale)
                    m = s.max()
                    p = torch.exp(s - m)
                    z = p.sum()
                    p = p / z
                    out[r, c] = p @ v[:t]
                    lse[r, c] = m + torch.log(z)
                    qk = k[:t].abs().sum(1) * float(q[r, c].abs().max()) * abs(scale)
                    e = float(((2 * D + 4) * 2.0 ** -24 * mag + 2.0 ** -17 * qk + 2.0 ** -23 * s.abs()
                               + 2.0 ** -23 * torch.log2(vs[:t]).abs()).max())
                    pv = p @ v[:t].abs()
                    codes = (v[:t].abs() / vs[:t, None]).sum(0)
                    to[r, c] = (2.0 ** -8 * out[r, c].abs() + (2 * e + 2.0 ** -9 + 2.0 ** -11 + (t / 16 + 40) * 2.0 ** -24) * pv
                                + 2.0 ** -25 * float((p * vs[:t]).max()) * codes + 1e-30)
                    tl[r, c] = e + 2.0 ** -24 * lse[r, c].abs() + 2.0 ** -20
    return out, lse, to, tl
