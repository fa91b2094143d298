"""Plain forms, step by step, of what a decoding loop does to logits and to the pages that sequences
share, and of attention over other states, for the tests to compare with.  Everything runs on CPU."""
import math

import torch

NEG = -math.inf


def allowed(mask_row, v: int) -> bool:
    return bool((int(mask_row[v // 32]) >> (v % 32)) & 1)


def adjust(x, history=None, seen=None, counted_from=None, repetition=None, presence=None, frequency=None, bias_ids=None,
           bias_values=None, mask=None, mask_index=None):
    """(values, sums of the terms' magnitudes) of logits x [rows, V] in 64 bits."""
    cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
    history, seen, counted_from, repetition, presence, frequency, bias_ids, bias_values, mask, mask_index = map(
        cpu, (history, seen, counted_from, repetition, presence, frequency, bias_ids, bias_values, mask, mask_index))
    y = x.cpu().double()
    rows, V = y.shape
    mag = y.abs().nan_to_num(0, 0, 0)
    groups = history.shape[0] if history is not None else bias_ids.shape[0] if bias_ids is not None else rows
    for r in range(rows):
        h = r // (rows // groups)
        if history is not None:
            n, start = int(seen[r]), 0 if counted_from is None else int(counted_from[h])
            c, g = {}, {}
            for i, t in enumerate(history[h, :n].tolist()):
                if 0 <= t < V:
                    c[t] = c.get(t, 0) + 1
                    g[t] = g.get(t, 0) + (i >= start)
            rho = 1.0 if repetition is None else float(repetition[h])
            freq = 0.0 if frequency is None else float(frequency[h])
            pres = 0.0 if presence is None else float(presence[h])
            for t in c:
                v = float(y[r, t])
                if rho != 1.0:
                    v = v / rho if v > 0 else v * rho
                if g[t]:
                    v -= freq * g[t] + pres
                y[r, t] = v
                mag[r, t] = mag[r, t] * max(rho, 1 / rho) + abs(freq) * g[t] + abs(pres)
        if bias_ids is not None:
            for t, b in zip(bias_ids[h].tolist(), bias_values[h].tolist()):
                if 0 <= t < V:
                    y[r, t] += b
                    mag[r, t] += abs(b)
        if mask is not None:
            i = r if mask_index is None else int(mask_index[r])
            if i >= 0:
                bits = (mask[i][:, None] >> torch.arange(32)) & 1
                y[r, bits.flatten()[:V] == 0] = NEG
    return y, mag


def fork(refs, table, parent):
    refs, table = refs.tolist(), table.cpu()
    batch, beams, cols = table.shape
    new = table.clone()
    for b in range(batch):
        for j in range(beams):
            p = int(parent[b, j])
            new[b, j] = table[b, p if 0 <= p < beams else j]
        for row, step in ((table, -1), (new, 1)):
            for e in row[b].flatten().tolist():
                if e >= 0:
                    refs[e] += step
    return torch.tensor(refs, dtype=torch.int32), new


def grow(refs, table, kv_len, new, page):
    """(refs, table, tail_src, granted) after every row has its pages; table [rows, cols]."""
    refs, table = refs.tolist(), table.cpu().clone()
    was = list(refs)
    free = [p for p, n in enumerate(refs) if n == 0]
    tails, granted, at = [], [], 0
    for r in range(table.shape[0]):
        n, add = int(kv_len[r]), int(new[r])
        tails.append(-1)
        cols = range(n // page, -(-(n + add) // page)) if add > 0 else range(0)
        ok = n >= 0 and add >= 0 and n + add <= table.shape[1] * page
        ok = ok and not (add > 0 and n % page and int(table[r, n // page]) < 0)
        if not ok:
            granted.append(False)
            continue
        want = [c for c in cols if int(table[r, c]) < 0 or was[int(table[r, c])] > 1]
        granted.append(not want or at + len(want) <= len(free))
        if granted[-1]:
            for k, c in enumerate(want):
                old = int(table[r, c])
                if old >= 0:
                    refs[old] -= 1
                    if c == n // page and n % page:
                        tails[-1] = old
                table[r, c] = free[at + k]
                refs[free[at + k]] = 1
        at += len(want)
    return torch.tensor(refs, dtype=torch.int32), table, torch.tensor(tails, dtype=torch.int32), torch.tensor(granted)


def free(refs, table, keep, page):
    refs, table = refs.tolist(), table.cpu().clone()
    for r in range(table.shape[0]):
        for c in range(table.shape[1]):
            if c * page >= int(keep[r]) >= 0 and int(table[r, c]) >= 0:
                refs[int(table[r, c])] -= 1
                table[r, c] = -1
    return torch.tensor(refs, dtype=torch.int32), table


def compact(refs, tables):
    """(refs, tables, moves [(from, to)], live pages)"""
    refs = refs.tolist()
    live = sum(n > 0 for n in refs)
    src = [p for p, n in enumerate(refs) if n > 0 and p >= live]
    dst = [p for p, n in enumerate(refs) if n <= 0 and p < live]
    to = dict(zip(src, dst))
    out = list(refs)
    for a, b in to.items():
        out[b], out[a] = refs[a], 0
    for p in range(live, len(out)):
        out[p] = 0
    moved = [t.cpu().clone().apply_(lambda e: to.get(e, e)) for t in tables]
    return torch.tensor(out, dtype=torch.int32), moved, list(to.items()), live


def cross(q, k, v, q_start, kv_start, kv_len, scale):
    """(out, lse, tolerance of out, tolerance of lse), float64, rows outside the requests NaN.

    Tolerances: with p the softmax weights and D the head dimension,
      * a score is an f32 sum of D exact products, and takes one f32 fma: it is off by at most
        e = (D + 4) 2^-24 (scale sum|q k|) + 2^-22 |score|, and so is the lse, with one rounding of
        the lse and a few of exp2, log2 and their sum (each below 2^-21) on top;
      * a weight is off by that relative amount, the sum of weights too, and by its rounding to bf16
        (2^-8 of its value at most), which the sum does not take;
      * the f32 sums over T states in runs of 16: (T / 16 + 40) 2^-24 of sum p |v|;
      * out is rounded to bf16 once: half a step, 2^-8 of its value at most."""
    total, q_heads, D = q.shape
    heads = k.shape[1]
    group = q_heads // heads
    out = torch.full((total, q_heads, D), math.nan, dtype=torch.float64)
    lse = torch.full((total, q_heads), math.nan, dtype=torch.float64)
    to, tl = torch.zeros_like(out), torch.zeros_like(lse)
    q, k, v = (x.cpu().double() for x in (q, k, v))
    for b in range(len(kv_len)):
        r0, r1, t0, n = int(q_start[b]), int(q_start[b + 1]), int(kv_start[b]), int(kv_len[b])
        for h in range(heads):
            rows = q[r0:r1, h * group:(h + 1) * group]
            at = (slice(r0, r1), slice(h * group, (h + 1) * group))
            if n == 0:
                out[at], lse[at] = 0.0, NEG
                continue
            kk, vv = k[t0:t0 + n, h], v[t0:t0 + n, h]
            s = rows @ kk.T * scale
            e = ((D + 4) * 2.0 ** -24 * (rows.abs() @ kk.abs().T) * abs(scale) + 2.0 ** -22 * s.abs()).amax(-1)
            lse[at] = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[at][..., None])
            out[at] = p @ vv
            pv = p @ vv.abs()
            to[at] = 2.0 ** -8 * out[at].abs() + (2 * e[..., None] + 2.0 ** -8 + (n / 16 + 40) * 2.0 ** -24) * pv + 1e-30
            tl[at] = e + 2.0 ** -24 * lse[at].abs() + 2.0 ** -20
    return out, lse, to, tl
