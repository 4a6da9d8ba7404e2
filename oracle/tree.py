"""fp64 and whole-number definitions of the operators that serve trees of drafted tokens from a paged cache.

Plain Python and numpy, one sequence, token and head at a time.
"""
import numpy as np

from oracle import paged


def ancestors(parents, t):
    """Token t and its ancestors, itself first; a parent that does not come before its child counts as -1."""
    out = []
    while t >= 0:
        out.append(t)
        p = int(parents[t])
        t = p if -1 <= p < t else -1
    return out


def plan(table, ring, held, span, kv_len, new_len, rows, page, parents=None):
    """(table, ring, held, span, kv_len, cu, slots, positions, granted) after the call; lists and nested lists."""
    table, ring, held = [list(r) for r in table], list(ring), list(held)
    P, (first, count) = len(ring), span
    want = [-(-(k + n) // page) for k, n in zip(kv_len, new_len)]
    taken, short, total, back = 0, False, [], []
    for b, (k, n) in enumerate(zip(kv_len, new_len)):
        need = want[b] - held[b]
        if need <= 0:
            back += table[b][want[b]:held[b]]
            held[b] = want[b]
            total.append(k + n)
        elif short or taken + need > count:
            short = True
            total.append(k)
        else:
            for i in range(need):
                table[b][held[b] + i] = ring[(first + taken + i) % P]
            taken += need
            held[b] = want[b]
            total.append(k + n)
    for j, pg in enumerate(back):
        ring[(first + count + j) % P] = pg
    granted = [t - k for t, k in zip(total, kv_len)]
    cu, slots, positions = [0], [-1] * rows, [0] * rows
    for b, (k, n) in enumerate(zip(kv_len, new_len)):
        for t in range(n):
            r, at = cu[-1] + t, k + t
            if total[b] == k + n:
                slots[r] = table[b][at // page] * page + at % page
            positions[r] = at if parents is None else k + len(ancestors(parents[b], t)) - 1
        cu.append(cu[-1] + n)
    return table, ring, held, [(first + taken) % P, count - taken + len(back)], total, cu, slots, positions, granted


def decode_tree(q, q_w, kp, vp, table, lens, parents, nodes, base, eps=1e-6, half=False):
    """o [B,Tq,Hq,D], lse [B,Hq,Tq] and the error bounds' factors a, m (as oracle.paged.decode_paged's)."""
    B, Tq, Hq, D = q.shape
    G = Hq // kp.shape[1]
    o, a, m = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, Tq, Hq))
    lse = np.full((B, Hq, Tq), -np.inf)
    for b in range(B):
        n, ctx = int(lens[b]), int(lens[b]) - int(nodes[b])
        if n <= 0 or ctx < 0:
            continue
        k, v = (paged.gather(x, table[b], n).astype(np.float64) for x in (kp, vp))
        for t in range(int(nodes[b])):
            line = ancestors(parents[b], t)
            see = list(range(ctx)) + [ctx + u for u in sorted(line)]
            qr = paged.rope_at(paged.rms_heads(q[b, t][None], q_w, eps), [ctx + len(line) - 1], base, half)[0]
            for h in range(Hq):
                kk, vv = k[h // G][see], v[h // G][see]
                s = kk @ qr[h] / np.sqrt(D)
                p = np.exp(s - s.max())
                z = p.sum()
                o[b, t, h] = p @ vv / z
                lse[b, h, t] = s.max() + np.log(z)
                a[b, t, h] = p @ np.abs(vv) / z
                m[b, t, h] = (np.abs(kk) @ np.abs(qr[h])).max() / np.sqrt(D)
    return o, lse, a, m


def keep(kp, vp, table, lens, nodes, path, count, page):
    """(kp, vp, lengths) after the accepted paths have moved; pools [P, H, page, D].  No tree: no path, whatever it holds."""
    kp, vp, out = kp.copy(), vp.copy(), []
    count = [c if n else 0 for c, n in zip(count, nodes)]
    for b in range(len(lens)):
        if lens[b] <= 0 or lens[b] < nodes[b]:
            out.append(max(lens[b], 0))
            continue
        ctx = lens[b] - nodes[b]
        place = lambda j: (table[b][j // page], slice(None), j % page)
        for pool in (kp, vp):
            rows = [pool[place(ctx + path[b][i])].copy() for i in range(count[b])]
            for i, r in enumerate(rows):
                pool[place(ctx + i)] = r
        out.append(ctx + count[b])
    return kp, vp, out
