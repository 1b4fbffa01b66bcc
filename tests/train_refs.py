"""Plain implementations of the training operators in 64 bits (numpy on the
CPU, from the formulas), shared by their tests."""
from __future__ import annotations

import numpy as np
import torch

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# half an ulp of a value held in the type, relative, and its smallest step
HALF_ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
STEP = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}


def held(a, dtype):
    """(tensor on the CPU in the type, its values in 64 bits) of an array."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(TORCH[dtype])
    return t, t.double().numpy()


def f64(t):
    return t.detach().double().cpu().numpy()


def csr(group, G):
    """Stable CSR of a group id per row; ids outside [0, G) after all others."""
    group = np.asarray(group)
    key = np.where((group >= 0) & (group < G), group, G)
    perm = np.argsort(key, kind="stable").astype(np.int32)
    row_ptr = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=G + 1)[:G])]).astype(np.int32)
    return row_ptr, perm


def grouped(x, w, group, dy=None):
    """y (and dx, dw) with, for each, the sums of the terms' magnitudes."""
    G, N, K = w.shape
    y, ay = np.zeros((len(x), N)), np.zeros((len(x), N))
    dx, adx = np.zeros_like(x), np.zeros_like(x)
    dw, adw = np.zeros_like(w), np.zeros_like(w)
    for g in range(G):
        rows = np.flatnonzero(np.asarray(group) == g)
        xg, wg = x[rows], w[g]
        y[rows], ay[rows] = xg @ wg.T, np.abs(xg) @ np.abs(wg).T
        if dy is not None:
            dg = dy[rows]
            dx[rows], adx[rows] = dg @ wg, np.abs(dg) @ np.abs(wg)
            dw[g], adw[g] = dg.T @ xg, np.abs(dg).T @ np.abs(xg)
    return (y, ay) if dy is None else (y, ay, dx, adx, dw, adw)


def norm_forward(h, x, gate, w_post, scale, w_pre, eps, kind):
    def stats(v):
        mean = v.mean(1, keepdims=True) if kind == "layer" else np.zeros((len(v), 1))
        return mean, 1.0 / np.sqrt(((v - mean) ** 2).mean(1, keepdims=True) + eps)

    mh, rh = stats(h)
    nh = (h - mh) * rh
    t = nh * w_post
    q = np.ones((len(h), 1)) if gate is None else 1.0 / (1.0 + np.exp(-gate))
    y = x + scale * q * t
    my, ry = stats(y)
    ny = (y - my) * ry
    return dict(y=y, u=ny * w_pre, nh=nh, t=t, q=q, ny=ny, rh=rh, ry=ry, stats=np.concatenate([mh, rh, my, ry], 1))


def norm_backward(dy, du, h, x, gate, w_post, scale, w_pre, eps, kind):
    """All gradients by the formulas, and for each the magnitude of the terms that
    the formulas add (dx and dh are themselves sums whose terms can cancel)."""
    f = norm_forward(h, x, gate, w_post, scale, w_pre, eps, kind)
    q, t, nh, ny = f["q"], f["t"], f["nh"], f["ny"]

    def through(d, n, r):
        out = d - n * (d * n).mean(1, keepdims=True)
        return r * (out - d.mean(1, keepdims=True) if kind == "layer" else out)

    def through_mag(d, n, r):
        out = d + np.abs(n) * (d * np.abs(n)).mean(1, keepdims=True)
        return r * (out + d.mean(1, keepdims=True) if kind == "layer" else out)

    dx = dy + through(du * w_pre, ny, f["ry"])
    mx = np.abs(dy) + through_mag(np.abs(du * w_pre), ny, f["ry"])
    mags = dict(dx=mx, dh=through_mag(mx * np.abs(scale * q * w_post), nh, f["rh"]))
    out = dict(dx=dx, dh=through(dx * scale * q * w_post, nh, f["rh"]))
    factors = dict(dgate=scale * t * q * (1.0 - q), dw_post=scale * q * nh, dscale=q * t)
    if gate is not None:
        row = gate.shape[1] != h.shape[1]
        for res, d, k in ((out, dx, factors["dgate"]), (mags, mx, np.abs(factors["dgate"]))):
            res["dgate"] = (d * k).sum(1, keepdims=True) if row else d * k
    for name in ("dw_post", "dscale"):
        out[name], mags[name] = (dx * factors[name]).sum(0), (mx * np.abs(factors[name])).sum(0)
    out["dw_pre"], mags["dw_pre"] = (du * ny).sum(0), np.abs(du * ny).sum(0)
    return out, mags


E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()   # 0 .. 448, ascending


def to_e4m3(q):
    """The e4m3 value nearest to each |q| <= 448 (ties to the even code), sign kept."""
    a = np.abs(q)
    hi = np.clip(np.searchsorted(E4M3, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    down, up = a - E4M3[lo], E4M3[hi] - a
    pick = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return np.copysign(E4M3[pick], q)


def quantise(v, root):
    """(values of the codes, scales) of float32 v, in blocks of 256."""
    f = np.float32
    codes, scales = np.empty(v.shape, np.float64), []
    for b in range(0, len(v), 256):
        x = v[b:b + 256].astype(f)
        fin = np.isfinite(x)
        top = f(np.abs(x[fin]).max()) if fin.any() else f(0)
        if top >= f(1e-30):
            scale, inv = f(top * f(1 / 448)), f(f(f(1) / top) * f(448))
        else:
            scale, inv = f(0), f(0)
        with np.errstate(invalid="ignore"):
            q = (x * inv).astype(f)
        if root and inv > 0:
            q = np.where(x > 0, np.maximum(q, f(2.0 ** -9)), q)
        c = to_e4m3(np.clip(np.where(fin, q, 0), -448, 448).astype(np.float64))
        codes[b:b + 256] = np.where(fin, c, np.nan)
        scales.append(scale)
    return codes, np.asarray(scales, f)


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, decay, grad_scale, eight):
    """One step in float32 with every operation rounded once, in the documented
    order: numpy's float32 arithmetic is exactly that.  m, v float32 (v the root
    of the second moment when ``eight``).  Returns p, m and v (or its root)."""
    f = np.float32
    with np.errstate(all="ignore"):
        g = (g.astype(f) * f(grad_scale)).astype(f)
        v = v * v if eight else v
        m = f(beta1) * m + f(1 - beta1) * g
        v = f(beta2) * v + f(1 - beta2) * (g * g)
        r = np.sqrt(v)
        denom = r * f(1 / np.sqrt(1 - beta2 ** step)) + f(eps)
        p = p * f(1 - lr * decay) - f(lr / (1 - beta1 ** step)) * (m / denom)
    return p, m, (r if eight else v)
