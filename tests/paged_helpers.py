"""The paged cache's operators from their definitions, in Python integers and 64-bit
floats on the CPU, and the tolerance of the attention.

Tolerance of one output element, with w_t the exact weights, v_t the values, u the half step of
the output type (2^-8 for bf16, 2^-24 for fp32):
  * the output's own rounding: u |out|;
  * every weight is off by a factor 1 + e, numerator and denominator alike, which moves the
    output by at most 2 e sum_t w_t |v_t|. e is the sum of
      - bf16 only: the weight's rounding to bf16, 2^-8;
      - the score's error ds = (128 + 4) 2^-24 sum_i |q_i k_ti| / sqrt(d) (every product and addition
        rounds once at most, the scaling and the exponent's argument a few times): 2 ds;
      - the exponential's approximation, twice (the weight and the factor that brings it to the
        common maximum): 2 x 2^-22;
  * sums of N terms in fp32, their roundings as independent: 8 sqrt(N) 2^-24 of sum_t w_t |v_t|,
    once for the numerator and once for the denominator.
"""
import math

import torch

D = 128


def pages_of(n, P):
    return (n + P - 1) // P


def plain_tables(seq_len, n_new, table, ring, state, n_slots, P):
    """(code, seq_len, state, q_start, slot_map, positions, table, ring); lists in, lists out."""
    n, cols, n_pages = len(seq_len), len(table[0]), len(ring)
    table, ring = [list(r) for r in table], list(ring)
    head, tail = state
    cap = cols * P
    new = [a + b for a, b in zip(seq_len, n_new)]
    grow = [max(0, pages_of(b, P) - pages_of(a, P)) for a, b in zip(seq_len, new)]
    shrink = [max(0, pages_of(a, P) - pages_of(b, P)) for a, b in zip(seq_len, new)]
    code = 0
    if any(a < 0 or a > cap or b < 0 for a, b in zip(seq_len, new)) or head < 0 or tail < head \
            or tail - head > n_pages:
        code = -5
    elif any(b > cap for b in new) or sum(grow) > tail - head or sum(max(0, x) for x in n_new) > n_slots:
        code = -2
    elif tail - head + sum(shrink) > n_pages:
        code = -5
    if code:
        return code, list(seq_len), [head, tail], [0] * (n + 1), [-1] * n_slots, [0] * n_slots, table, ring
    before = [list(r) for r in table]
    h, t = head, tail
    q_start, slots, pos = [0], [], []
    for r in range(n):
        had, has = pages_of(seq_len[r], P), pages_of(new[r], P)
        for j in range(had, has):
            table[r][j] = ring[h % n_pages]
            h += 1
        for i in range(seq_len[r], new[r]):
            slots.append(table[r][i // P] * P + i % P)
            pos.append(i)
        q_start.append(len(slots))
    for r in range(n):
        for j in range(pages_of(new[r], P), pages_of(seq_len[r], P)):
            ring[t % n_pages] = before[r][j]
            t += 1
    rest = n_slots - len(slots)
    return 0, new, [h, t], q_start, slots + [-1] * rest, pos + [0] * rest, table, ring


def plain_attn(q, q_start, seq_len, table, k_pages, v_pages, prefix, L):
    """(out, tolerance) of the attention in 64 bits; rows that no request owns are NaN."""
    T, Hq, _ = q.shape
    _, H, P, _ = k_pages.shape
    G = Hq // H
    bf16 = q.dtype == torch.bfloat16
    out = torch.full((T, Hq, D), math.nan, dtype=torch.float64)
    tol = torch.zeros((T, Hq, D), dtype=torch.float64)

    def rows(pool, ids, n):
        ids = ids[:pages_of(n, P)].long()
        return pool[ids].double().permute(1, 0, 2, 3).reshape(H, -1, D)[:, :n]

    kp, vp = (rows(x, prefix, L) if L else torch.zeros((H, 0, D), dtype=torch.float64) for x in (k_pages, v_pages))
    for r in range(len(seq_len)):
        b, e, s = int(q_start[r]), int(q_start[r + 1]), int(seq_len[r])
        ks, vs = (torch.cat([x, rows(y, table[r], s)], 1) if s else x for x, y in ((kp, k_pages), (vp, v_pages)))
        for t in range(b, e):
            n = L + min(s, max(0, s - (e - b) + (t - b) + 1))
            if n == 0:
                out[t] = 0.0
                continue
            qh = q[t].double().view(H, G, D)
            sc = qh @ ks[:, :n].transpose(1, 2) / math.sqrt(D)
            w = torch.softmax(sc, -1)
            o = w @ vs[:, :n]
            mag = w @ vs[:, :n].abs()
            ds = 132 * 2.0 ** -24 * (qh.abs() @ ks[:, :n].abs().transpose(1, 2)).amax(-1, keepdim=True) / math.sqrt(D)
            err = (2.0 ** -8 if bf16 else 0.0) + 2 * ds + 2 * 2.0 ** -22
            u = 2.0 ** -8 if bf16 else 2.0 ** -24
            tt = u * o.abs() + mag * (2 * err + 2 * 8 * math.sqrt(n) * 2.0 ** -24) + 1e-30
            out[t], tol[t] = o.reshape(Hq, D), tt.reshape(Hq, D)
    return out, tol
