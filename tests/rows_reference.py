"""Operators whose rows choose their own matrices, in NumPy float64 from their
definitions (the oracle of tests/test_route_*.py and tests/test_lora_*.py; no code of
the library): a router's choice of experts, the gradient of its logits, low-rank
adapters."""
import numpy as np

SOFTMAX, SIGMOID = 0, 1


class Router:
    def __init__(self, experts, top_k, score=SOFTMAX, groups=1, top_groups=1, group_top=1, renormalize=False, scale=1.0):
        self.experts, self.top_k, self.score, self.groups = experts, top_k, score, groups
        self.top_groups, self.group_top, self.renormalize, self.scale = top_groups, group_top, renormalize, scale


def scores(l, score):
    with np.errstate(invalid="ignore", over="ignore"):
        if score == SOFTMAX:
            p = np.exp(l - l.max())
            return p / p.sum()
        return np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))


def log_scores(l, score):
    """log s, up to a constant for softmax."""
    with np.errstate(over="ignore"):
        return l if score == SOFTMAX else np.minimum(l, 0) - np.log1p(np.exp(-np.abs(l)))


def weights_of(l, chosen, r):
    """The weights of a fixed choice (a list of experts) from the logits l of a token."""
    if not len(chosen):
        return np.zeros(0)
    if not r.renormalize:
        return r.scale * scores(l, r.score)[chosen]
    q = log_scores(l[chosen], r.score)
    q = np.exp(q - q.max())
    return r.scale * q / q.sum()


def route(l, bias, r):
    """l tokens x experts float64 -> (chosen, weights, counts)."""
    T, E = l.shape
    chosen, weights = np.full((T, r.top_k), -1, np.int32), np.zeros((T, r.top_k))
    size = E // r.groups
    # without a bias the order is the logits'; sums of scores alone need the scores
    sums = r.top_groups < r.groups and r.group_top == 2 and size > 1
    for t in range(T):
        if np.isnan(l[t]).any() or (r.score == SOFTMAX and (l[t] == np.inf).any()) or (bias is not None and np.isnan(bias).any()):
            weights[t] = np.nan
            continue
        left = l[t] > -np.inf
        if bias is not None:
            left &= bias > -np.inf
        if not left.any():
            continue
        v = l[t].copy() if bias is None else scores(l[t], r.score) + bias
        if r.top_groups < r.groups:
            u = scores(l[t], r.score) if sums and bias is None else v
            worth = np.full(r.groups, -np.inf)
            for g in range(r.groups):
                mine = np.sort(u[g * size:(g + 1) * size][left[g * size:(g + 1) * size]])[::-1][:r.group_top]
                if len(mine):
                    worth[g] = mine.sum()
            best = [g for g in np.argsort(-worth, kind="stable")[:r.top_groups] if worth[g] > -np.inf]
            left &= np.isin(np.arange(E) // size, best)
        order = [e for e in np.argsort(-v, kind="stable") if left[e]][:r.top_k]
        chosen[t, :len(order)] = order
        weights[t, :len(order)] = weights_of(l[t], order, r)
    counts = np.bincount(chosen[chosen >= 0].ravel(), minlength=E)
    return chosen, weights, counts


def route_backward(l, chosen, dweights, r):
    """The gradient of the logits, and how much was summed for each (magnitudes)."""
    T, E = l.shape
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        slots = [i for i in range(chosen.shape[1]) if 0 <= chosen[t, i] < E]
        if not slots:
            continue
        e, dw = chosen[t, slots], r.scale * dweights[t, slots]
        s = scores(l[t], r.score)
        rest = scores(-l[t], SIGMOID)   # 1 - sigmoid
        if r.renormalize:
            q = log_scores(l[t][e], r.score)
            q = np.exp(q - q.max())
            q /= q.sum()
            own, m = q * (dw - (q * dw).sum()), q * (np.abs(dw) + (q * np.abs(dw)).sum())
            if r.score == SIGMOID:
                own, m = own * rest[e], m * rest[e]
        elif r.score == SOFTMAX:
            own, m = s[e] * dw, s[e] * np.abs(dw)
            d[t] -= s * own.sum()
            mag[t] += s * m.sum()
        else:
            own = s[e] * rest[e] * dw
            m = np.abs(own)
        np.add.at(d[t], e, own)
        np.add.at(mag[t], e, m)
    return d, mag


def lora(x, c, a, b, ids, ranks, scales):
    """Y = C + s (X A^T) B^T row by row (C None: zeros) and the sum of magnitudes; rows without an
    adapter keep C's."""
    rows, n = x.shape[0], b.shape[1]
    y = np.zeros((rows, n)) if c is None else c.astype(np.float64)
    mag = np.abs(y)
    for i in range(a.shape[0]):
        who = np.nonzero(ids == i)[0]
        if not len(who):
            continue
        r, s = a.shape[1] if ranks is None else int(ranks[i]), 1.0 if scales is None else float(scales[i])
        wa, wb = a[i, :r], b[i, :, :r]
        y[who] += s * ((x[who] @ wa.T) @ wb.T)
        mag[who] += abs(s) * ((np.abs(x[who]) @ np.abs(wa).T) @ np.abs(wb).T)
    return y, mag


def lora_backward(x, dy, dc, a, b, ids, ranks, scales):
    """(dX, dA, dB) and the sums of magnitudes of each."""
    dx = np.zeros(x.shape) if dc is None else dc.astype(np.float64)
    da, db = np.zeros(a.shape), np.zeros(b.shape)
    mx, ma, mb = np.abs(dx), np.zeros(a.shape), np.zeros(b.shape)
    for i in range(a.shape[0]):
        who = np.nonzero(ids == i)[0]
        if not len(who):
            continue
        r, s = a.shape[1] if ranks is None else int(ranks[i]), 1.0 if scales is None else float(scales[i])
        wa, wb, xi, di = a[i, :r], b[i, :, :r], x[who], dy[who]
        h, dh = xi @ wa.T, s * (di @ wb)
        mh, mdh = np.abs(xi) @ np.abs(wa).T, abs(s) * (np.abs(di) @ np.abs(wb))
        dx[who] += dh @ wa
        mx[who] += mdh @ np.abs(wa)
        da[i, :r], ma[i, :r] = dh.T @ xi, mdh.T @ np.abs(xi)
        db[i, :, :r], mb[i, :, :r] = s * (di.T @ h), abs(s) * (np.abs(di).T @ mh)
    return (dx, da, db), (mx, ma, mb)
