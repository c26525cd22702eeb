"""The routing, balance-loss and checkpoint operators from their definitions, in
64 bits on the CPU (numpy), for the tests to compare with."""
import numpy as np

EPS32 = 2.0**-24  # half a step of fp32, relative


def sigmoid(l):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-np.asarray(l, np.float64)))


def softmax(l):
    l = np.asarray(l, np.float64)
    m = l.max(axis=-1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(m == -np.inf, 0.0, np.exp(l - m))
        s = e.sum(axis=-1, keepdims=True)
        return np.where(s == 0, 0.0, e / np.where(s == 0, 1, s))


def scores(l, kind):
    return sigmoid(l) if kind == "sigmoid" else softmax(l)


def _best(a, n, among=None):
    """The n largest of a: NaN behind every number, what is not among last, ties to the lower index."""
    among = np.ones(a.shape, bool) if among is None else among
    nan = np.isnan(a)
    rank = np.where(among, np.where(nan, 1, 0), 2)
    return np.lexsort((np.arange(a.size), np.where(nan, 0.0, -a), rank))[:n]


def select(l, bias, k, score, n_group=1, topk_group=1, group_score="top2", renorm=True, scale=1.0):
    """idx [T, k] ascending and weights [T, k]."""
    l = np.asarray(l, np.float64)
    T, E = l.shape
    per = E // n_group
    idx = np.zeros((T, k), np.int32)
    p = scores(l, score)
    for t in range(T):
        a = p[t] + np.asarray(bias, np.float64) if bias is not None else l[t]
        among = np.ones(E, bool)
        if topk_group < n_group:
            by = p[t] + np.asarray(bias, np.float64) if bias is not None else (p[t] if group_score == "top2" else l[t])
            g = np.full(n_group, np.nan)
            for i in range(n_group):
                part = by[i * per:(i + 1) * per]
                part = np.sort(part[~np.isnan(part)])
                if group_score == "top2" and per > 1:
                    g[i] = part[-1] + part[-2] if part.size > 1 else np.nan
                elif part.size:
                    g[i] = part[-1]
            among = np.repeat(np.isin(np.arange(n_group), _best(g, topk_group)), per)
        idx[t] = np.sort(_best(a, k, among))
    w = weights(l, idx, score, renorm, scale)
    return idx, w


def weights(l, idx, score, renorm, scale):
    l = np.asarray(l, np.float64)
    if renorm:
        c = np.take_along_axis(l, idx.astype(np.int64), 1)
        s = softmax(c) if score == "softmax" else sigmoid(c)
        total = s.sum(1, keepdims=True)
        return scale * np.where(total == 0, 0.0, s / np.where(total == 0, 1, total))
    return scale * np.take_along_axis(scores(l, score), idx.astype(np.int64), 1)


def shares(l, score):
    p = scores(l, score)
    s = p.sum(1, keepdims=True)
    return np.where(s == 0, 0.0, p / np.where(s == 0, 1, s))


def balance(l, idx, off, alpha, score):
    """loss [n_seq], load [n_seq, E]."""
    p = shares(l, score)
    E, k = p.shape[1], idx.shape[1]
    loss, load = [], []
    for a, b in zip(off[:-1], off[1:]):
        n = b - a
        f = np.zeros(E) if n == 0 else np.bincount(idx[a:b].reshape(-1), minlength=E) * (E / (k * n))
        load.append(f)
        loss.append(0.0 if n == 0 else alpha * float((f * p[a:b].mean(0)).sum()))
    return np.array(loss), np.array(load)


def select_grad(l, idx, dw, score, renorm, scale, off=None, load=None, dloss=None, alpha=0.0):
    """dlogits [T, E], by the chain rule through the scores."""
    l = np.asarray(l, np.float64)
    T, E = l.shape
    p = scores(l, score)
    ds = np.zeros((T, E))
    if dw is not None:
        c = np.asarray(dw, np.float64) * scale
        i = idx.astype(np.int64)
        if renorm:
            s = np.take_along_axis(p, i, 1)
            S = s.sum(1, keepdims=True)
            with np.errstate(invalid="ignore", divide="ignore"):
                c = np.where(S == 0, 0.0, (c - (c * s).sum(1, keepdims=True) / S) / S)
        for t in range(T):
            np.add.at(ds[t], i[t], c[t])
    if off is not None:
        S = p.sum(1, keepdims=True)
        for q, (a, b) in enumerate(zip(off[:-1], off[1:])):
            if b > a:
                f = alpha * float(dloss[q]) * np.asarray(load[q], np.float64) / (b - a)
                Sq = np.where(S[a:b] == 0, 1, S[a:b])
                ds[a:b] += np.where(S[a:b] == 0, 0.0, (f - (f * p[a:b]).sum(1, keepdims=True) / Sq) / Sq)
    if score == "sigmoid":
        return ds * p * sigmoid(-l)
    return p * (ds - (ds * p).sum(1, keepdims=True))


TOP = {"e4m3": 448.0, "i8": 127.0}


def pack(x, fmt):
    """(values that the codes stand for in units of the scale, E8M0 bytes); x [rows, cols] float64."""
    rows, cols = x.shape
    nt = -(-cols // 128)
    u = np.zeros_like(x)
    byte = np.zeros((rows, nt), np.uint8)
    for r in range(rows):
        for i in range(nt):
            v = x[r, i * 128:(i + 1) * 128]
            if not np.isfinite(v).all():
                byte[r, i] = 255
                continue
            a = np.abs(v).max()
            e = 0
            if a > 0:
                m, e = np.frexp(a / TOP[fmt])
                e = max(int(e) - (1 if m == 0.5 else 0), -126)
            byte[r, i] = e + 127
            w = v / 2.0**e
            if fmt == "e4m3":
                step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(w), 2.0**-6))) - 3)
                u[r, i * 128:(i + 1) * 128] = np.round(w / step) * step
            else:
                u[r, i * 128:(i + 1) * 128] = np.round(w)
    return u, byte


def unpack(u, byte):
    s = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    return u * np.repeat(s, 128, axis=1)[:, :u.shape[1]]
