"""Plain implementations of embedding, routing, the exchange with experts and
dropout in 64 bits (numpy, from the formulas), shared by their tests."""
from __future__ import annotations

import numpy as np


def embedding(w, ids, scale):
    y = np.zeros((len(ids), w.shape[1]))
    held = (ids >= 0) & (ids < len(w))
    y[held] = w[ids[held]] * scale
    return y


def embedding_backward(dy, ids, V, scale):
    """dw, and the sums of its terms' magnitudes."""
    dw, mag = np.zeros((V, dy.shape[1])), np.zeros((V, dy.shape[1]))
    held = (ids >= 0) & (ids < V)
    np.add.at(dw, ids[held], dy[held] * scale)
    np.add.at(mag, ids[held], np.abs(dy[held] * scale))
    return dw, mag


def scores(z, kind):
    if kind == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-z))
    top = z.max(1, keepdims=True, initial=-np.inf)
    e = np.exp(z - np.where(np.isneginf(top), 0.0, top))
    total = e.sum(1, keepdims=True)
    return e / np.where(total > 0, total, 1.0)


def route(z, k, bias, kind, groups, top_groups, group_top, renormalise, scale):
    """(ids, weights)."""
    M, E = z.shape
    s = scores(z, kind)
    a = z.copy() if bias is None and top_groups == groups else s + (0.0 if bias is None else bias)
    a = np.where(np.isneginf(z), -np.inf, a)
    if top_groups < groups:
        per = a.reshape(M, groups, -1)
        best = -np.sort(-per, axis=2)[:, :, :group_top]
        value = np.where(np.isneginf(best[:, :, 0]), -np.inf, np.where(np.isneginf(best), 0.0, best).sum(2))
        order = np.argsort(-value, axis=1, kind="stable")[:, :top_groups]
        kept = np.zeros((M, groups), bool)
        np.put_along_axis(kept, order, True, 1)
        a = np.where(np.repeat(kept, E // groups, 1), a, -np.inf)
    ids = np.argsort(-a, axis=1, kind="stable")[:, :k]
    none = np.isneginf(np.take_along_axis(a, ids, 1))
    ids = np.where(none, -1, ids)
    return ids, route_weights(z, ids, kind, renormalise, scale)


def route_weights(z, ids, kind, renormalise, scale):
    w = np.where(ids < 0, 0.0, np.take_along_axis(scores(z, kind), np.maximum(ids, 0), 1))
    if renormalise:
        total = w.sum(1, keepdims=True)
        w = w / np.where(total > 0, total, 1.0)
    return w * scale


def route_backward(dw, z, ids, kind, renormalise, scale):
    """dlogits, and the magnitude of the terms that its formula adds."""
    M, E = z.shape
    g = np.where(ids < 0, 0.0, dw) * scale
    out, mag = np.zeros((M, E)), np.zeros((M, E))
    at = np.maximum(ids, 0)
    s = scores(z, kind)
    if renormalise:
        r = route_weights(z, ids, kind, True, 1.0)
        own, size = r * (g - (r * g).sum(1, keepdims=True)), r * (np.abs(g) + (r * np.abs(g)).sum(1, keepdims=True))
        slope = 1.0 - np.take_along_axis(s, at, 1) if kind == "sigmoid" else 1.0
        own, size = own * slope, size * slope
    else:
        own, size = g, np.abs(g)
    rows = np.arange(M)[:, None] * np.ones_like(ids)
    np.add.at(out, (rows, at), np.where(ids < 0, 0.0, own))
    np.add.at(mag, (rows, at), np.where(ids < 0, 0.0, size))
    if not renormalise:
        if kind == "sigmoid":
            out, mag = out * s * (1.0 - s), mag * s * (1.0 - s)
        else:
            out, mag = s * (out - (s * out).sum(1, keepdims=True)), s * (mag + (s * mag).sum(1, keepdims=True))
    return out, mag


def slots(ids, G):
    """(row_ptr, perm, slot) of the assignments (M, k)."""
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < G), flat, G)
    perm = np.argsort(key, kind="stable")
    row_ptr = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=G + 1)[:G])])
    slot = np.empty(flat.size, np.int64)
    slot[perm] = np.arange(flat.size)
    return row_ptr, perm, np.where(key < G, slot, -1).reshape(ids.shape)


def dispatch(x, ids, G):
    row_ptr, perm, slot = slots(ids, G)
    xs = x[perm // ids.shape[1]].copy()
    xs[row_ptr[G]:] = 0.0
    return xs, slot


def combine(h, slot, weights=None):
    """y, and the sums of its terms' magnitudes."""
    held = (slot >= 0) & (slot < len(h))
    w = np.where(held, 1.0 if weights is None else weights, 0.0)[:, :, None]
    rows = np.where(held[:, :, None], h[np.where(held, slot, 0)] if len(h) else 0.0, 0.0)
    return (w * rows).sum(1), np.abs(w * rows).sum(1)


def combine_backward(dy, h, slot, weights):
    """dh, dweights, and the sums of the latter's terms' magnitudes."""
    held = slot >= 0
    dh = np.zeros_like(h)
    rows = np.broadcast_to(np.arange(len(dy))[:, None], slot.shape)
    dh[slot[held]] = weights[held][:, None] * dy[rows[held]]
    terms = np.where(held[:, :, None], dy[:, None] * h[np.maximum(slot, 0)], 0.0)
    return dh, terms.sum(2), np.abs(terms).sum(2)


def philox(counter, key, rounds=10):
    """Philox 4x32: (n, 4) and (2,) of 32 bits, held in 64 unsigned ones."""
    c = [counter[:, i].astype(np.uint64) for i in range(4)]
    k = [np.uint64(v) for v in key]
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> half) ^ c[1] ^ k[0], b & low, (a >> half) ^ c[3] ^ k[1], a & low]
        k = [(k[0] + np.uint64(0x9E3779B9)) & low, (k[1] + np.uint64(0xBB67AE85)) & low]
    return np.stack(c, 1)


def dropout_gain(n, p, seed, call, step):
    """The factor of each of n elements: 0 or 65536 / (65536 - limit)."""
    block = np.arange(-(-n // 8), dtype=np.uint64)
    counter = np.stack([block & np.uint64(0xFFFFFFFF), block >> np.uint64(32), np.full_like(block, call),
                        np.full_like(block, step & 0xFFFFFFFF)], 1)
    words = philox(counter, (seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF))
    u = np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], 2).reshape(-1)[:n].astype(np.int64)
    limit = round(p * 65536)
    return np.where(u >= limit, 65536.0 / max(65536 - limit, 1), 0.0)
