"""Plain 64-bit forms of the speculative decoding operators (numpy), shared by their tests."""
from fractions import Fraction

import numpy as np

NQ, NKV, HD, BLK = 16, 8, 128, 64
BLOCK = 131072


def lineage(parents, i):
    """Node i and its ancestors."""
    out = []
    while i >= 0:
        out.append(i)
        i = parents[i]
    return out


def random_tree(rng, n, width=12):
    return np.array([-1] + [int(rng.integers(max(0, i - width), i)) for i in range(1, n)], np.int32)


def tree_attention(q, k, v, tk, tv, parents):
    """q [n][16][128], cached k and v [keys][8][128], the nodes' own tk and tv [n][8][128] -> out [n][16][128], a bound of
    sum p |v|, and max sum |q k| / sqrt(128) of each (node, head). Only what a node sees is touched."""
    n = len(q)
    out, mag, dots = np.zeros((n, NQ, HD)), np.zeros((n, NQ, HD)), np.zeros((n, NQ))
    for i in range(n):
        line = lineage(parents, i)
        kk, vv = np.concatenate((k, tk[line])), np.concatenate((v, tv[line]))
        for h in range(NQ):
            with np.errstate(invalid="ignore"):
                z = kk[:, h // 2] @ q[i, h] / np.sqrt(HD)
                p = np.exp(z - z.max())
                p /= p.sum()
                out[i, h], mag[i, h] = p @ vv[:, h // 2], p @ np.abs(vv[:, h // 2])
                dots[i, h] = (np.abs(kk[:, h // 2]) @ np.abs(q[i, h])).max() / np.sqrt(HD)
    return out, mag, dots


def verify(tokens, parents, p, q, u, u_next):
    """One tree: p [n][V] float64, q the same or None -> (path, next token, the least distance to a border)."""
    n, path, node, near = len(tokens), [], 0, np.inf
    V = p.shape[1]
    while True:
        path.append(node)
        r, mass, c = p[node].copy(), 1.0, 0.0
        found = None
        for j in range(node + 1, n):
            x = int(tokens[j])
            if parents[j] != node or not 0 <= x < V:
                continue
            price = u[j] * mass * (q[node, x] if q is not None else 1.0)
            if price != r[x] and price > 0:
                near = min(near, abs(price - r[x]) / price)
            if price < r[x]:
                found = j
                break
            if q is not None:
                c += mass
                r = np.maximum(p[node] - c * q[node], 0)
                mass = r.sum()
            else:
                mass -= r[x]
                r[x] = 0
        if found is None:
            break
        node = found
    total = r.sum()
    if total > 0:
        cdf = np.cumsum(r)
        t = u_next * total
        near = min(near, np.abs(cdf - t)[r > 0].min() / total)
        token = int(np.argmax(cdf > t)) if (cdf > t).any() else int(np.nonzero(r)[0][-1])
    else:
        token = int(np.argmax(p[node]))
    return path, token, near


def verify_exactly(tokens, parents, p, q, u, u_next):
    """As verify for drawn drafts, of fp32 numbers, without roundings: the distance is that of two masses, of the 1 of a row."""
    whole = lambda x: int(Fraction(float(x)) * 2 ** 160)  # fp32 numbers from 2^-136 up are whole numbers of 2^-160
    n, path, node, near = len(tokens), [], 0, 1.0
    while True:
        path.append(node)
        P, Q = [whole(x) for x in p[node]], [whole(x) for x in q[node]]
        # r is in units of 2^-(160 + e), c of 2^-e, mass of 2^-m
        r, mass, m, c, e = P, 1, 0, 0, 0
        found = None
        for j in range(node + 1, n):
            if parents[j] != node:
                continue
            x = int(tokens[j])
            gap = (whole(u[j]) * Q[x] * mass << e) - (r[x] << 160 + m)
            near = min(near, abs(Fraction(gap, 1 << 320 + m + e)))
            if gap < 0:
                found = j
                break
            c, e = (c << m - e) + mass, m
            r = [max((a << e) - c * b, 0) for a, b in zip(P, Q)]
            mass, m = sum(r), 160 + e
        if found is None:
            break
        node = found
    k, total, cum, token = whole(u_next), sum(r), 0, None
    for x, y in enumerate(r):
        cum += y
        gap = (cum << 160) - k * total
        if y:
            near = min(near, abs(Fraction(gap, 1 << 320 + e)))
        if token is None and gap > 0:
            token = x
    return path, P.index(max(P)) if token is None else token, float(near)


def verify_greedy(tokens, parents, ids):
    path, node = [], 0
    while node is not None:
        path.append(node)
        last, node = node, next((j for j in range(node + 1, len(tokens)) if parents[j] == node and tokens[j] == ids[node]), None)
    return path, int(ids[last])
