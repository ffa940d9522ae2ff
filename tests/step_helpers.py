"""The operators around the paged cache's attention from their definitions, in Python integers and 64-bit floats on the
CPU: rotary positions, requests that share pages, compaction, verification of drafted tokens; and their tolerances."""
import math

import numpy as np
import torch

D = 128


def pages_of(n, P):
    return (n + P - 1) // P


# ---- rotary positions ---------------------------------------------------------------------

def plain_rope(x, positions, offset, freq, axis, interleaved):
    """(rotated, tolerance) of x [tokens, heads, D] in 64 bits. positions [axes, tokens].

    Tolerance of an element of a pair (a, b), u the half step of the output type (2^-8 for bf16, 2^-24 for fp32):
      * the sine's and the cosine's error: the angle's 64-bit roundings, here and there (f / 2 pi, the product): 2^-50 |angle|;
        the fraction of a turn in 32 bits, 2 pi 2^-33, and in fp32, pi 2^-25 (half a step below 1); the functions', two steps, 2^-22;
      * the two products and the sum in fp32: 2 x 2^-24 (|a| + |b|);
      * the output's rounding: u |out|.
    """
    n = len(freq)
    u = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -24
    y = x.double().clone()
    tol = torch.zeros_like(y)
    f = torch.tensor(freq, dtype=torch.float64)
    angle = (positions.double() + offset)[torch.tensor(axis)].T * f  # [tokens, n]
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    a, b = x.double()[..., first], x.double()[..., second]
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    err = (2.0 ** -50 * angle.abs() + 2 * math.pi * 2.0 ** -33 + math.pi * 2.0 ** -25 + 2.0 ** -22)[:, None]
    t = (a.abs() + b.abs()) * (err + 2 * 2.0 ** -24)
    tol[..., first], tol[..., second] = t, t
    tol += torch.where(tol > 0, u * y.abs() + 1e-30, torch.zeros_like(tol))
    return y, tol


# ---- shared pages -------------------------------------------------------------------------

def plain_fork(src, dst, fork_len, lens, table, refs, P):
    """(code, lens, table, refs); lists in, lists out."""
    n, cols = len(lens), len(table[0])
    lens2, table2, refs2 = list(lens), [list(r) for r in table], list(refs)
    bad = len(set(dst)) != len(dst) or bool(set(src) & set(dst))
    for i, (s, d) in enumerate(zip(src, dst)):
        if not (0 <= s < n and 0 <= d < n):
            bad = True
            continue
        m = lens[s] if fork_len is None else fork_len[i]
        bad |= not 0 <= lens[s] <= cols * P or not 0 <= m <= lens[s] or lens[d] != 0
    if bad:
        return -5, lens2, table2, refs2
    for i, (s, d) in enumerate(zip(src, dst)):
        m = lens[s] if fork_len is None else fork_len[i]
        for j in range(pages_of(m, P)):
            table2[d][j] = table[s][j]
            refs2[table[s][j]] += 1
        lens2[d] = m
    return 0, lens2, table2, refs2


def plain_tables_shared(lens, n_new, table, ring, state, refs, n_slots, P):
    """(code, lens, state, q_start, slots, positions, copy_src, copy_dst, table, ring, refs); lists in, lists out."""
    n, cols, n_pages = len(lens), len(table[0]), len(ring)
    head, tail = state
    cap = cols * P
    new = [a + b for a, b in zip(lens, n_new)]

    def fail(code):
        return (code, list(lens), list(state), [0] * (n + 1), [-1] * n_slots, [0] * n_slots, [-1] * n, [-1] * n,
                [list(r) for r in table], list(ring), list(refs))

    bounds = any(a < 0 or a > cap or b < 0 for a, b in zip(lens, new))
    capacity = any(b > cap for b in new)
    fine = [0 <= a <= cap and 0 <= b <= cap for a, b in zip(lens, new)]
    # holders that let go: (page, writes, request), and what is left of the counts
    left, holders = list(refs), {}
    for r in range(n):
        if not fine[r]:
            continue
        grows = n_new[r] > 0 and lens[r] % P
        cells = [pages_of(lens[r], P) - 1] if grows else range(pages_of(new[r], P), pages_of(lens[r], P))
        for j in cells:
            p = table[r][j]
            if not 0 <= p < n_pages:
                bounds = True
                continue
            left[p] -= 1
            holders.setdefault(p, []).append((bool(grows), r))
    bounds |= any(left[p] < 0 for p in holders)
    decides = {p: max(h) for p, h in holders.items() if left[p] == 0}
    copies = [bool(fine[r] and n_new[r] > 0 and lens[r] % P and
                   decides.get(table[r][pages_of(lens[r], P) - 1]) != (True, r)) for r in range(n)]
    if bounds or head < 0 or tail < head or tail - head > n_pages:
        return fail(-5)
    if capacity:
        return fail(-2)
    back = [[table[r][j] for j in range(pages_of(new[r], P), pages_of(lens[r], P)) if decides.get(table[r][j]) == (False, r)]
            for r in range(n)]
    take = [max(0, pages_of(b, P) - pages_of(a, P)) + c for a, b, c in zip(lens, new, copies)]
    if sum(take) > tail - head or sum(max(0, x) for x in n_new) > n_slots:
        return fail(-2)
    if tail - head + sum(map(len, back)) > n_pages:
        return fail(-5)
    table, ring, refs = [list(r) for r in table], list(ring), left
    for p, (writes, _) in decides.items():
        refs[p] = int(writes)
    h, t = head, tail
    q_start, slots, pos, copy_src, copy_dst = [0], [], [], [], []
    for r in range(n):
        last = pages_of(lens[r], P) - 1
        cells = ([last] if copies[r] else []) + list(range(last + 1, pages_of(new[r], P)))
        copy_src.append(table[r][last] if copies[r] else -1)
        for j in cells:
            table[r][j] = ring[h % n_pages]
            refs[table[r][j]] = 1
            h += 1
        copy_dst.append(table[r][last] if copies[r] else -1)
        for i in range(lens[r], new[r]):
            slots.append(table[r][i // P] * P + i % P)
            pos.append(i)
        q_start.append(len(slots))
    for x in back:
        for p in x:
            ring[t % n_pages] = p
            t += 1
    rest = n_slots - len(slots)
    return 0, new, [h, t], q_start, slots + [-1] * rest, pos + [0] * rest, copy_src, copy_dst, table, ring, refs


def plain_compact(lens, table, extra, refs, ring, state, n_moves, P):
    """(code, src, dst, table, extra, refs, ring, state); lists in, lists out."""
    n_pages, cols = len(refs), len(table[0])
    live = [p for p in range(n_pages) if refs[p] > 0]
    L = len(live)
    src = [p for p in live if p >= L]
    dst = [p for p in range(L) if refs[p] <= 0]
    named = [p for r, n in enumerate(lens) if 0 <= n <= cols * P for p in table[r][:pages_of(n, P)]] + list(extra)
    code = 0
    if any(not 0 <= n <= cols * P for n in lens) or min(refs) < 0 or any(not 0 <= p < n_pages or refs[p] <= 0 for p in named):
        code = -5
    elif len(src) > n_moves:
        code = -2
    none = [-1] * n_moves
    if code:
        return code, none, none, [list(r) for r in table], list(extra), list(refs), list(ring), list(state)
    goes = dict(zip(src, dst))
    table2 = [[goes.get(p, p) if j < pages_of(n, P) else p for j, p in enumerate(row)] for row, n in zip(table, lens)]
    refs2 = [0] * n_pages
    for p in live:
        refs2[goes.get(p, p)] = refs[p]
    ring2 = list(range(L, n_pages)) + list(ring)[n_pages - L:]
    rest = [-1] * (n_moves - len(src))
    return 0, src + rest, dst + rest, table2, [goes.get(p, p) for p in extra], refs2, ring2, [0, n_pages - L]


# ---- verification of drafts ----------------------------------------------------------------

def entries(x):
    """What entries of a row count for, in 64 bits."""
    x = x.double()
    return torch.where((x > 0) & (x <= 2.0 ** 100), x, torch.zeros_like(x))


def plain_verify(tokens, n_draft, target, draft, uniform):
    """Per request (code, accepted, check): check(token) says whether the token is right.

    A draft's test is exact (48 bits of u q against p). The drawn token: sums that are held to 40 bits move a
    border by at most 2^-40 of the whole, so the first j with sum_j > u W is found between u W - 2^-40 W and u W + 2^-40 W."""
    V = target.shape[-1]
    answers = []
    for r, n in enumerate(n_draft.tolist()):
        if not 0 <= n <= tokens.shape[1]:
            answers.append((0 if n == -1 else -5, 0, lambda x: x == -1))
            continue
        code, a = 0, 0
        if any(not 0 <= x < V for x in tokens[r, :n].tolist()):
            code = -5
        if uniform is None:
            while True:
                row = target[r, a].float().clone()
                row[row.isnan()] = -math.inf
                some = ~target[r, a].float().isnan()
                best = int(torch.nonzero((row == row.max()) & some)[0]) if bool(some.any()) else -1
                if a < n and best >= 0 and int(tokens[r, a]) == best:
                    a += 1
                    continue
                break
            answers.append((code if best >= 0 else -5, a, lambda x, y=best: x == y))
            continue
        u = [min(max(x, 0.0), 1 - 2.0 ** -24) if x == x else 0.0 for x in uniform[r].tolist()]
        while a < n:
            x = int(tokens[r, a])
            if not 0 <= x < V:
                break
            q = float(entries(draft[r, a, x])) if draft is not None else 1.0
            if not u[a] * q < float(entries(target[r, a, x])):
                break
            a += 1
        p = entries(target[r, a])
        w = p
        if a < n:
            if draft is not None:
                q = entries(draft[r, a])
            else:
                q = torch.zeros(V, dtype=torch.float64)
                if 0 <= int(tokens[r, a]) < V:
                    q[int(tokens[r, a])] = 1.0
            w = (p - q).clamp(min=0)
            if not bool((w > 0).any()):
                w = p
        if not bool((w > 0).any()):
            answers.append((-5, a, lambda x: x == -1))
            continue
        sums = np.cumsum(w.numpy().astype(np.longdouble))
        want, eps = u[-1] * sums[-1], sums[-1] * np.longdouble(2.0) ** -40

        def check(x, sums=sums, want=want, eps=eps, w=w):
            return (0 <= x < len(sums) and float(w[x]) > 0 and bool(sums[x] > want - eps)
                    and (x == 0 or bool(sums[x - 1] <= want + eps)))
        answers.append((code, a, check))
    return answers
