"""Plain references for the routing calls and the adapter products, in numpy
and 64 bits, written from the definitions in include/fp8gemm_routed.h."""
import numpy as np


def topk(x, k, renorm, scale):
    """x [T,E] float64 -> ids [T,k] int, w [T,k] float64."""
    T, E = x.shape
    ids = np.full((T, k), -1, np.int64)
    w = np.zeros((T, k))
    for t in range(T):
        ok = [e for e in range(E) if not np.isnan(x[t, e]) and x[t, e] > -np.inf]
        ok.sort(key=lambda e: (-x[t, e], e))
        if not ok:
            continue
        m = x[t, ok[0]]
        p = np.array([1.0 if x[t, e] == m else np.exp(x[t, e] - m) for e in ok])
        top = min(k, len(ok))
        ids[t, :top] = ok[:top]
        w[t, :top] = scale * p[:top] / (p[:top].sum() if renorm else p.sum())
    return ids, w


def topk_backward(x, ids, dw, renorm, scale):
    """the weights' gradient for fixed choices, by the quotient rule: with p_e
    the exponentials and Z their sum over the normalising set N,
    w_j = scale p_j / Z, d w_j / d x_e = scale (p_j [e = j] Z - p_j p_e [e in N]) / Z^2."""
    T, E = x.shape
    g = np.zeros((T, E))
    for t in range(T):
        ok = ~np.isnan(x[t]) & (x[t] > -np.inf)
        chosen = [e for e in ids[t] if e >= 0]
        if not chosen:
            continue
        p = np.where(ok, np.exp(np.where(ok, x[t], 0) - x[t][ok].max()), 0.0)
        N = np.zeros(E, bool)
        N[chosen if renorm else np.flatnonzero(ok)] = True
        Z = p[N].sum()
        for j, e in enumerate(ids[t]):
            if e < 0:
                continue
            d = -p[e] * np.where(N, p, 0.0) / Z ** 2
            d[e] += p[e] / Z
            g[t] += scale * dw[t, j] * d
    return g


def sort(ids, G, M, masked):
    """ids [S] -> row [S], then m_indices [M] and counts [G], or masked_m [G]."""
    S = len(ids)
    counts = np.array([np.sum(ids == g) for g in range(G)], np.int64)
    if masked:
        first = np.arange(G) * M
        top = first + M
    else:
        size = -(-counts // 128) * 128
        first = np.cumsum(size) - size
        top = np.full(G, M)
    row = np.full(S, -1, np.int64)
    m_indices = np.full(0 if masked else M, -1, np.int64)
    used = np.zeros(G, np.int64)
    for s in range(S):
        g = ids[s]
        if 0 <= g < G:
            r = first[g] + used[g]
            used[g] += 1
            if r < top[g]:
                row[s] = r
                if not masked:
                    m_indices[r] = g
    if masked:
        return row, np.minimum(counts, M)
    return row, m_indices, counts


def dispatch(X, row, out):
    """rows of X placed into `out` [rows, ...] (a copy is returned)."""
    out = out.copy()
    for t in range(row.shape[0]):
        for r in row[t]:
            if 0 <= r < out.shape[0]:
                out[r] = X[t]
    return out


def combine(Y, row, w):
    """(out [T,H], sum of |terms| [T,H]) in float64; w None: 1."""
    T, k = row.shape
    out = np.zeros((T, Y.shape[1]))
    mag = np.zeros_like(out)
    for t in range(T):
        for j in range(k):
            if 0 <= row[t, j] < Y.shape[0]:
                term = (1.0 if w is None else float(w[t, j])) * Y[row[t, j]]
                out[t] += term
                mag[t] += np.abs(term)
    return out, mag


def combine_backward(dout, Y, row, w, dY):
    """(dY, dw, sum of |terms| of dw): rows without a choice keep dY's contents."""
    T, k = row.shape
    dY = dY.copy()
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = row[t, j]
            if 0 <= r < Y.shape[0]:
                dY[r] = float(w[t, j]) * dout[t]
                dw[t, j] = np.dot(dout[t], Y[r])
                mag[t, j] = np.dot(np.abs(dout[t]), np.abs(Y[r]))
    return dY, dw, mag


def lora(base, X, La, Lb, ids, scale):
    """(D, sum of |h||Lb| terms, h) in float64: base [M,N] plus each row's
    adapter; an id outside [0,G) adds nothing."""
    D, mag = base.copy(), np.zeros_like(base)
    h = np.zeros((X.shape[0], La.shape[1]))
    for m, a in enumerate(ids):
        if 0 <= a < La.shape[0]:
            h[m] = float(scale[a]) * (La[a] @ X[m])
            D[m] = D[m] + Lb[a] @ h[m]
            mag[m] = np.abs(Lb[a]) @ np.abs(h[m])
    return D, mag, h
