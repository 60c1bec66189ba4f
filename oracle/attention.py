"""Oracle of the 8-bit path's attention in float64, row by row from the definition.

    o = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q . k_j - max),  over the keys j that the query sees
"""

import numpy as np

U32 = 2.0 ** -24                       # half a step of float32


def visible(Lq, Lk, causal):
    """Keys that each of Lq queries sees: all of Lk, or the first i + 1 + Lk - Lq."""
    n = np.full(Lq, Lk)
    return np.clip(np.arange(Lq) + 1 + Lk - Lq, 0, Lk) if causal else n


def attend(q, K, V, scale, sees, weight_error, tiny):
    """q float64 [n][D], K, V [m][D], query i sees keys 0 .. sees[i] - 1 -> (o [n][D], tau [n][D]).

    tau bounds the error of float32 arithmetic: a score is a sum of D exact products, each addition off by at
    most half a step of sum |q k|, times scale and minus the maximum (two roundings, of at most the larger
    of the scores); the exponential turns an absolute error of its argument into a relative one, and its own
    is a step.  Sums of m weights and of m products round m times at most (blocks are joined pairwise, which
    takes fewer), each by half a step of a sum of absolute values.  weight_error is the relative error of a
    weight's rounding to 16 bits, tiny what a weight may lose besides, relative to the largest."""
    o = np.zeros((len(q), V.shape[1]))
    tau = np.zeros_like(o)
    D = q.shape[1]
    for i in range(len(q)):
        m = int(sees[i])
        if m == 0:
            continue
        k, v = K[:m], V[:m]
        with np.errstate(invalid="ignore"):
            s = scale * (k @ q[i])
            w = np.exp(s - s.max())
            total = w.sum()
            o[i] = w @ v / total
            size = scale * (np.abs(k) @ np.abs(q[i]))
            arg = (D + 2) * U32 * size + 4 * U32 * np.abs(s).max()
            rel = weight_error + arg.max() + 4 * U32
            spread = w @ np.abs(v) / total
            tau[i] = (2 * rel + 2 * m * U32) * spread + tiny * np.abs(v).sum(axis=0) / total + 1e-30
    return o, tau


def attention(Q, K, V, cu_q, cu_k, causal, scale, weight_error, tiny, fill=0.0):
    """Packed sequences: Q [T][Hq][D], K, V [Tk][Hkv][D] float64 -> (o, tau) [T][Hq][D]; rows of no sequence hold fill."""
    T, Hq, D = Q.shape
    G = Hq // K.shape[1]
    o, tau = np.full(Q.shape, float(fill)), np.zeros(Q.shape)
    for a, b, c, d in zip(cu_q[:-1], cu_q[1:], cu_k[:-1], cu_k[1:]):
        sees = visible(b - a, d - c, causal)
        for h in range(Hq):
            o[a:b, h], tau[a:b, h] = attend(Q[a:b, h], K[c:d, h // G], V[c:d, h // G], scale, sees, weight_error, tiny)
    return o, tau


def gather(cache, table, n, page):
    """The n rows [n][Hkv][D] (or [n][Hkv]) of a sequence, and which of them have a page."""
    rows = np.zeros((n, cache.shape[1]) + cache.shape[3:])
    there = np.zeros(n, bool)
    for j in range(n):
        p = int(table[j // page])
        if 0 <= p < len(cache):
            rows[j], there[j] = cache[p, :, j % page], True
    return rows, there


def paged(Q, kcache, vcache, table, lengths, scale, weight_error, tiny):
    """One query a sequence: Q [B][Hq][D], caches [pages][Hkv][page][D] float64 -> (o, tau) [B][Hq][D]."""
    B, Hq, D = Q.shape
    page, G = kcache.shape[2], Hq // kcache.shape[1]
    o, tau = np.zeros(Q.shape), np.zeros(Q.shape)
    for b in range(B):
        n = int(np.clip(lengths[b], 0, table.shape[1] * page))
        K, there = gather(kcache, table[b], n, page)
        V, _ = gather(vcache, table[b], n, page)
        K, V = K[there], V[there]
        for h in range(Hq):
            oh, th = attend(Q[b, h][None], K[:, h // G], V[:, h // G], scale, [len(K)], weight_error, tiny)
            o[b, h], tau[b, h] = oh[0], th[0]
    return o, tau


def append(new, cache, table, lengths, cu, put):
    """Writes row t of new [T][Hkv]... into a copy of cache: put(destination row, new row)."""
    out = cache.copy()
    page = cache.shape[2]
    for b in range(len(lengths)):
        for t in range(max(cu[b], 0), min(cu[b + 1], len(new))):
            at = int(lengths[b]) - (int(cu[b + 1]) - t)
            if 0 <= at < table.shape[1] * page and 0 <= table[b, at // page] < len(cache):
                put(out[table[b, at // page], :, at % page], new[t])
    return out
