"""fp64 oracle of the operators between token ids and the expert layer: the
embedding, layer norm, the router with its balance loss, and their gradients."""
import numpy as np


def _valid(ids, V):
    ids = np.asarray(ids).reshape(-1)
    return ids, (ids >= 0) & (ids < V)


def embedding(ids, W, scale=1.0):
    flat, ok = _valid(ids, W.shape[0])
    out = np.zeros((flat.size, W.shape[1]))
    out[ok] = scale * W[flat[ok]]
    return out.reshape(*np.shape(ids), W.shape[1])


def embedding_backward(dout, ids, V, scale=1.0):
    """(dW, the sum of the sizes of its terms, the number of terms of each row)."""
    flat, ok = _valid(ids, V)
    d = dout.reshape(-1, dout.shape[-1])[ok]
    dW, size = np.zeros((V, dout.shape[-1])), np.zeros((V, dout.shape[-1]))
    np.add.at(dW, flat[ok], d)
    np.add.at(size, flat[ok], np.abs(d))
    return scale * dW, abs(scale) * size, np.bincount(flat[ok], minlength=V)


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd) of rows x [R, C]."""
    mean = x.mean(1)
    rstd = 1 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight=None):
    """(dx, dweight, dbias) for these statistics."""
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy if weight is None else dy * weight
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def scores(l, score):
    """s [T, E]; 0 for a logit of -inf, also in a row of them."""
    with np.errstate(invalid="ignore", over="ignore"):
        if score == "sigmoid":
            return np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(np.minimum(l, 0)) / (1 + np.exp(-np.abs(l)))) + 0 * np.where(
                np.isnan(l), l, 0)
        top = np.max(l, axis=1, keepdims=True, initial=-np.inf)
        e = np.exp(l - np.where(top == -np.inf, 0, top))
        total = e.sum(1, keepdims=True)
        return e / np.where(total == 0, 1, total)


def choose(l, k, score, bias=None, mask=None):
    key = l if bias is None else scores(l, score) + bias
    never = ~(l > -np.inf) | ~(key > -np.inf)
    if mask is not None:
        never = never | ~np.asarray(mask, bool)[:, None]
    key = np.where(never, -np.inf, key)
    order = np.argsort(-key, axis=1, kind="stable")[:, :k]
    ids = np.where(np.take_along_axis(never, order, 1), -1, order)
    return ids.astype(np.int32)


def _chosen(l, ids, score):
    """The chosen's s divided by a factor of the row that no score under- or overflows with, 0 for none."""
    x = np.take_along_axis(l, np.maximum(ids, 0), 1)
    x = np.where(ids >= 0, x, -np.inf)
    top = np.max(x, axis=1, keepdims=True, initial=-np.inf)
    top = np.where(top == -np.inf, 0, top)
    if score == "sigmoid":
        return np.exp(np.minimum(x, 0) - np.minimum(top, 0)) / (1 + np.exp(-np.abs(x)))
    return np.exp(x - top)


def weights(l, ids, score, normalize, scale):
    if normalize:
        v = _chosen(l, ids, score)
        total = v.sum(1, keepdims=True)
        v = v / np.where(total == 0, 1, total)
    else:
        v = np.where(ids >= 0, np.take_along_axis(scores(l, score), np.maximum(ids, 0), 1), 0)
    return scale * v


def shares(l, score):
    """p = s / sum s, with sigmoid scores also where all of a row's underflow."""
    if score == "softmax":
        return scores(l, score)
    v = np.exp(np.minimum(l, 0) - np.minimum(np.max(l, axis=1, keepdims=True), 0)) / (1 + np.exp(-np.abs(l)))
    return v / v.sum(1, keepdims=True)


def balance(l, ids, score, k):
    """(counts [E + 1], probs [E], loss)."""
    E = l.shape[1]
    some = (ids >= 0).any(1)
    N = int(some.sum())
    counts = np.append(np.bincount(ids[ids >= 0], minlength=E), N).astype(np.int32)
    if N == 0:
        return counts, np.zeros(E), 0.0
    probs = shares(l[some], score).sum(0) / N
    return counts, probs, E / (k * N) * float((counts[:E] * probs).sum())


def route_backward(l, ids, dw, score, normalize, scale, counts=None, coef=1.0):
    """(dlogits, the sum of the sizes of its terms)."""
    T, E = l.shape
    k = ids.shape[1]
    dl, size = np.zeros((T, E)), np.zeros((T, E))
    there = ids >= 0
    some = there.any(1)
    at = (np.nonzero(there)[0], ids[there])
    if dw is not None:
        g = np.where(there, scale * dw, 0)
        x = np.where(there, np.take_along_axis(l, np.maximum(ids, 0), 1), 0)
        if normalize:
            v = weights(l, ids, score, True, 1.0)
            down = 1 / (1 + np.exp(x)) if score == "sigmoid" else 1.0
            d = v * down * (g - (g * v).sum(1, keepdims=True))
            n = v * down * (np.abs(g) + (np.abs(g) * v).sum(1, keepdims=True))
            np.add.at(dl, at, d[there])
            np.add.at(size, at, n[there])
        elif score == "sigmoid":
            d = g / (1 + np.exp(-x)) / (1 + np.exp(x))
            np.add.at(dl, at, d[there])
            np.add.at(size, at, np.abs(d[there]))
        else:
            p = scores(l, score)
            pj = np.where(there, np.take_along_axis(p, np.maximum(ids, 0), 1), 0)
            G, Gn = np.zeros((T, E)), np.zeros((T, E))
            np.add.at(G, at, g[there])
            np.add.at(Gn, at, np.abs(g[there]))
            dl += p * (G - (g * pj).sum(1, keepdims=True))
            size += p * (Gn + (np.abs(g) * pj).sum(1, keepdims=True))
    if counts is not None and counts[E] > 0:
        c = coef * E / (k * float(counts[E]) ** 2) * counts[:E]
        lr = np.where(some[:, None], l, 0)
        p = shares(lr, score)
        down = 1 / (1 + np.exp(lr)) if score == "sigmoid" else 1.0
        dl += p * down * (c - (p * c).sum(1, keepdims=True))
        size += p * down * (np.abs(c) + (p * np.abs(c)).sum(1, keepdims=True))
    return dl * some[:, None], size * some[:, None]
