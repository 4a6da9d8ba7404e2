"""fp64 definitions of the query/key norms and of the paged cache's operators.

Plain numpy, one sequence and one head at a time.  The rotation is written as a
complex product; the cached keys are taken as stored (rotated fp16, pairs side by
side).  Every function takes exact float64 values.
"""
import numpy as np


def rms_heads(x, w, eps):
    """x [..., D] -> x / sqrt(mean x^2 + eps) * w (w None: x itself)."""
    x = np.asarray(x, dtype=np.float64)
    if w is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w


def rms_heads_bwd(x, w, g, eps):
    """Gradients (dx, dw) of sum(g * rms_heads(x, w, eps)); dw summed over every row."""
    D = x.shape[-1]
    s = (x * x).mean(-1, keepdims=True) + eps
    r = 1.0 / np.sqrt(s)
    # d n_i / d x_j = w_i (delta_ij r - x_i x_j r^3 / D)
    dx = w * g * r - x * r ** 3 / D * (w * g * x).sum(-1, keepdims=True)
    dw = (g * x * r).reshape(-1, D).sum(0)
    return dx, dw


def rope_at(x, pos, base, half=False):
    """x [N, H, D] rotated at positions pos [N]; the pairs of the result lie side by
    side (the cache's order) in either input layout."""
    x = np.asarray(x, dtype=np.float64)
    D = x.shape[-1]
    z = x[..., :D // 2] + 1j * x[..., D // 2:] if half else x[..., 0::2] + 1j * x[..., 1::2]
    theta = np.power(float(base), -2.0 * np.arange(D // 2) / D)
    z = z * np.exp(1j * np.asarray(pos, dtype=np.float64)[:, None, None] * theta)
    out = np.empty_like(x)
    out[..., 0::2], out[..., 1::2] = z.real, z.imag
    return out


def places(table, pos0, cu, page):
    """(row, page, slot) of every new row of a ragged append."""
    out = []
    for b in range(len(cu) - 1):
        for i, n in enumerate(range(cu[b], cu[b + 1])):
            pos = pos0[b] + i
            out.append((n, int(table[b][pos // page]), pos % page, pos))
    return out


def gather(pool, pages, n):
    """The first n positions held by `pages` of pool [P, H, page, D] -> [H, n, D]."""
    page = pool.shape[2]
    need = -(-n // page)
    x = pool[np.asarray(pages[:need], dtype=np.int64)]
    return np.moveaxis(x, 1, 0).reshape(pool.shape[1], need * page, pool.shape[3])[:, :n]


def decode_paged(q, q_w, kp, vp, table, lens, base, eps=1e-6, half=False, prefix_pages=(), bounds=False):
    """o [B,Tq,Hq,D] and lse [B,Hq,Tq] of the newest Tq tokens of every sequence.

    bounds: also (a [B,Tq,Hq,D], m [B,Tq,Hq]): a = sum_j p_j |v_j|, the size an error
    of the weights is multiplied with, and m = max_j sum_i |q_i k_ji| / sqrt(D), the
    size a relative error of q or k is multiplied with in a logit.
    """
    B, Tq, Hq, D = q.shape
    Hkv = kp.shape[1]
    G = Hq // Hkv
    o = np.zeros(q.shape)
    lse = np.full((B, Hq, Tq), -np.inf)
    a, m = np.zeros(q.shape), np.zeros((B, Tq, Hq))
    for b in range(B):
        n = int(lens[b])
        if n <= 0:
            continue
        pages = list(prefix_pages) + list(table[b][len(prefix_pages):])
        k, v = gather(kp, pages, n).astype(np.float64), gather(vp, pages, n).astype(np.float64)
        for t in range(Tq):
            at = n - Tq + t
            if at < 0:
                continue
            qr = rope_at(rms_heads(q[b, t][None], q_w, eps), [at], base, half)[0]
            for h in range(Hq):
                kk, vv = k[h // G, :at + 1], v[h // G, :at + 1]
                s = kk @ qr[h] / np.sqrt(D)
                top = s.max()
                p = np.exp(s - top)
                z = p.sum()
                o[b, t, h] = p @ vv / z
                lse[b, h, t] = top + np.log(z)
                if bounds:
                    a[b, t, h] = p @ np.abs(vv) / z
                    m[b, t, h] = (np.abs(kk) @ np.abs(qr[h])).max() / np.sqrt(D)
    return (o, lse, a, m) if bounds else (o, lse)
