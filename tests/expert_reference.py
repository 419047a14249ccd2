"""Plain definitions of the expert-layer operators in 64 bits (NumPy), for the tests.

Written from the formulas alone; nothing here is shared with the CUDA path."""
import numpy as np

TINY = 1e-20


def scores(z, score):
    """Scores of float64 logits [T,E]; a masked expert (-inf) has score 0, a row of them only zeros."""
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-z))
        m = z.max(1, keepdims=True)
        e = np.where(np.isneginf(z), 0.0, np.exp(z - np.where(np.isneginf(m), 0.0, m)))
        t = e.sum(1, keepdims=True)
        return e / np.where(t == 0.0, 1.0, t)


def route(z, k, score="softmax", bias=None, n_groups=1, top_groups=1, group_rank=1, renormalize=True, scale=1.0):
    """(weight float64 [T,k], index [T,k]) by sorting every row in Python."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    s = scores(z, score)
    v = z if bias is None and (group_rank == 1 or n_groups == 1) else s + (0.0 if bias is None else np.asarray(bias, np.float64))
    v = np.where(np.isneginf(z), -np.inf, v)
    index = np.full((T, k), -1, np.int64)
    weight = np.zeros((T, k))
    gs = E // n_groups
    for t in range(T):
        allowed = range(E)
        if n_groups > 1:
            rank = []
            for g in range(n_groups):
                best = sorted((x for x in v[t, g * gs:(g + 1) * gs] if x != -np.inf), reverse=True)[:group_rank]
                rank.append((-sum(best) if best else np.inf, g))
            kept = {g for _, g in sorted(rank)[:top_groups]}
            allowed = [e for e in range(E) if e // gs in kept]
        order = sorted((-v[t, e], e) for e in allowed if v[t, e] != -np.inf)[:k]
        for j, (_, e) in enumerate(order):
            index[t, j] = e
            weight[t, j] = s[t, e]
        if renormalize:
            weight[t] = weight[t] / (weight[t].sum() + TINY)
    return weight * scale, index


def route_bwd(dweight, z, index, score="softmax", renormalize=True, scale=1.0):
    """dlogits float64 by the chain rule, from the Jacobian of every row's weights."""
    z, g = np.asarray(z, np.float64), np.asarray(dweight, np.float64) * scale
    T, E = z.shape
    s = scores(z, score)
    d = np.zeros((T, E))
    for t in range(T):
        ds = np.zeros(E)
        slots = [j for j in range(index.shape[1]) if 0 <= index[t, j] < E]
        p = {j: s[t, index[t, j]] for j in slots}
        total = sum(p.values()) + TINY
        for j in slots:
            if renormalize:      # d(p_i / total) / dp_j = (i == j) / total - p_i / total^2
                ds[index[t, j]] += g[t, j] / total - sum(g[t, i] * p[i] for i in slots) / total ** 2
            else:
                ds[index[t, j]] += g[t, j]
        if score == "sigmoid":
            d[t] = s[t] * (1.0 - s[t]) * ds
        else:
            d[t] = s[t] * (ds - (s[t] * ds).sum())
    return d


def capacity(T, k, E, align):
    """The most rows that any index [T,k] can need, by spreading pairs one by one: every expert that
    has a pair costs at most align - 1 rows of padding."""
    P = T * k
    return (P + min(E, P) * (align - 1)) // align * align


def rows(index, E, align):
    """pos, src, start, count of an index [T,k] (values outside [0, E) are no pair)."""
    T, k = index.shape
    flat = index.reshape(-1).tolist()
    of = [[p for p, e in enumerate(flat) if e == x] for x in range(E)]
    start = np.zeros(E + 1, np.int64)
    src = np.full(capacity(T, k, E, align), -1, np.int64)
    pos = np.full(T * k, -1, np.int64)
    for e in range(E):
        for i, p in enumerate(of[e]):
            src[start[e] + i] = p
            pos[p] = start[e] + i
        start[e + 1] = start[e] + -(-len(of[e]) // align) * align
    return pos.reshape(T, k), src, start, np.array([len(x) for x in of])


def gather(x, src, k):
    """x[src // k] with zeros where src is -1."""
    out = np.zeros((len(src), x.shape[1]), x.dtype)
    has = src >= 0
    out[has] = x[src[has] // k]
    return out


def combine(y, pos, weight=None, residual=None):
    T, k = pos.shape
    out = np.zeros((T, y.shape[1])) if residual is None else residual.astype(np.float64).copy()
    for t in range(T):
        for j in range(k):
            if pos[t, j] >= 0:
                out[t] += (1.0 if weight is None else float(weight[t, j])) * y[pos[t, j]]
    return out


def decode_e4m3(q):
    """Values of E4M3 codes (uint8), float64."""
    q = np.asarray(q, np.uint8).astype(np.int64)
    e, m = (q >> 3) & 15, q & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((q & 127) == 127, np.nan, v)
    return np.where(q >> 7, -v, v)


def values(q, s):
    """Codes [M,C] with scales [C/128,M] -> float64 [M,C]."""
    return decode_e4m3(q) * np.repeat(np.asarray(s, np.float64).T, 128, axis=1)


def weight_values(qw, sw):
    """Codes [E N,K] with scales [E N/128,K/128] -> float64."""
    return decode_e4m3(qw) * np.repeat(np.repeat(np.asarray(sw, np.float64), 128, 0), 128, 1)


def product_fwd(x, w, start, count, E):
    """x float64 [R,K], w float64 [E N,K] -> {expert: [count,N]}."""
    N = w.shape[0] // E
    return {e: x[start[e]:start[e] + count[e]] @ w[e * N:(e + 1) * N].T for e in range(E) if count[e]}
