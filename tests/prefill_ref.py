"""Plain 64-bit implementations of the operators that bring prompts into the paged
cache: the plan of pages and rows, rotary positions, attention of packed rows."""

import math

import torch

from tests.paged_ref import entries


def plan(table, lens, free, count, keep, next_pos, n_rows, page, n_pages):
    """(table, lens, the stack of free pages, first, granted, seq, slot, pos) after the plan,
    by lists, sequence by sequence."""
    table, lens, stack = [list(r) for r in table], list(lens), list(free)
    width, seqs = len(table[0]), len(table)
    cap = width * page
    length = [min(max(n, 0), cap) for n in lens]
    for b in range(seqs):
        if keep is None or keep[b] < 0:
            continue
        length[b] = lens[b] = min(length[b], keep[b])
        j = length[b] // page
        if length[b] % page and j < width and 0 <= table[b][j] < n_pages:
            j += 1
        elif length[b] % page:
            continue
        while j < width and 0 <= table[b][j] < n_pages:
            stack.append(table[b][j])
            table[b][j] = -1
            j += 1
    first, granted, starved = [], [], False
    seq, slot, pos = [-1] * n_rows, [-1] * n_rows, [0] * n_rows
    total = 0
    for b in range(seqs):
        n = max(count[b], 0)
        first.append(total)
        ok = n > 0 and total + n <= n_rows and length[b] + n <= cap
        if ok:
            j = length[b] // page
            end = -(-(length[b] + n) // page)
            while j < end and 0 <= table[b][j] < n_pages:
                j += 1
            need = end - j
            if need > 0 and (starved or need > len(stack)):
                ok, starved = False, True
            elif need > 0:
                for i in range(j, end):
                    table[b][i] = stack.pop()
        granted.append(n if ok else 0)
        for i in range(min(n, max(0, n_rows - total))):
            seq[total + i] = b
            slot[total + i] = length[b] + i if ok else -1
            pos[total + i] = (length[b] if next_pos is None else next_pos[b]) + i
        total += n
    return table, lens, stack, first, granted, seq, slot, pos


def frequencies(dims, theta=1e7, scaling=None, factor=1.0, context=0.0, low=0.0, high=0.0):
    f = []
    for i in range(dims // 2):
        w = theta ** (-2.0 * i / dims)
        if scaling == "linear":
            w /= factor
        if scaling == "parts":
            g = min(1.0, max(0.0, (context * w / (2 * math.pi) - low) / (high - low)))
            w *= g + (1 - g) / factor
        f.append(w)
    return f


def turned(x, pos, f, layout="half", scale=1.0, transpose=False):
    """x [rows][heads][hd]: pair i of its first 2 len(f) elements turned by pos f[i]."""
    x = x.double().clone()
    n = len(f)
    ang = pos.double()[:, None] * torch.tensor(f, dtype=torch.float64, device=x.device)
    c, s = (ang.cos() * scale)[:, None], (ang.sin() * scale)[:, None] * (-1.0 if transpose else 1.0)
    a, b = (x[..., :n].clone(), x[..., n:2 * n].clone()) if layout == "half" else (x[..., 0:2 * n:2].clone(), x[..., 1:2 * n:2].clone())
    p, q = a * c - b * s, b * c + a * s
    if layout == "half":
        x[..., :n], x[..., n:2 * n] = p, q
    else:
        x[..., 0:2 * n:2], x[..., 1:2 * n:2] = p, q
    return x


def attention(q, k, v, table, lens, first, count, page, scale=None):
    """(out, mean, bound): out of the rows of the sequences (others NaN), ``mean`` the sum of
    p |v| of each output, ``bound`` the largest sum over head dims of |q k| scale."""
    rows, heads, hd = q.shape
    kv = k.shape[2]
    scale = 1 / math.sqrt(hd) if scale is None else scale
    out = torch.full(q.shape, math.nan, dtype=torch.float64, device=q.device)
    mean = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    bound, slots = 0.0, table.shape[1] * page
    for b in range(table.shape[0]):
        n, m, r0 = int(count[b]), max(0, min(int(lens[b]), slots)), int(first[b])
        if n <= 0 or r0 < 0 or r0 + n > rows:
            continue
        kk, there = entries(k, table, b, m, page)
        vv, _ = entries(v, table, b, m, page)
        sees = torch.arange(m, device=q.device) < m - n + torch.arange(n, device=q.device)[:, None] + 1
        sees = sees & there
        vv = torch.where(there[:, None, None], vv, torch.zeros_like(vv))
        kk = torch.where(there[:, None, None], kk, torch.zeros_like(kk))
        for h in range(heads):
            g = h // (heads // kv)
            x = (q[r0:r0 + n, h].double() @ kk[:, g].T) * scale
            if m:
                bound = max(bound, float((q[r0:r0 + n, h].double().abs() @ kk[:, g].abs().T).max()) * abs(scale))
            x = torch.where(sees, x, torch.full_like(x, -math.inf))
            top = x.max(1, keepdim=True).values.clamp(min=-1e300) if m else torch.zeros(n, 1, dtype=torch.float64, device=q.device)
            p = torch.exp(x - top)
            p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
            out[r0:r0 + n, h] = p @ vv[:, g]
            mean[r0:r0 + n, h] = p @ vv[:, g].abs()
    return out, mean, bound
