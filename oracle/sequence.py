"""Float64 oracle of the sequence operators, written from their formulas one token, row or class at a time.

* the gated linear recurrence over packed sequences and its gradients: h_t = f_t h_{t-1} + (1 - f_t) g_t,
  y_t = o_t h_t, f = sigmoid(zf), o = sigmoid(zo);
* the norms before and after a block with its gate and residual scale: n = z rsqrt(mean z^2 + eps) w_post,
  r = x + scale sigmoid(u) n, v = r rsqrt(mean r^2 + eps) w_pre;
* the distillation loss from a teacher's top logits: loss = w tau^2 sum_j p_j (ln p_j - ln q_{id_j}).

Rows that no sequence holds come back as NaN: no caller may use them.
"""

import numpy as np


def sigmoid(z):
    z = np.asarray(z, np.float64)
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def _tokens(off, s, reverse):
    t = range(int(off[s]), int(off[s + 1]))
    return list(reversed(t)) if reverse else list(t)


def scan_forward(off, zf, g, zo=None, h0=None, reverse=False):
    """(y [T][D], hT [S][D], h [T][D])."""
    zf, g = np.asarray(zf, np.float64), np.asarray(g, np.float64)
    S, D = len(off) - 1, zf.shape[1]
    f, fc = sigmoid(zf), sigmoid(-zf)
    h = np.full(zf.shape, np.nan)
    hT = np.zeros((S, D)) if h0 is None else np.array(h0, np.float64)
    for s in range(S):
        for t in _tokens(off, s, reverse):
            hT[s] = f[t] * hT[s] + fc[t] * g[t]
            h[t] = hT[s]
    y = h if zo is None else h * sigmoid(zo)
    return y, hT, h


def scan_backward(off, zf, g, zo, dy, h0=None, dhT=None, reverse=False):
    """dict of dzf, dg, dzo (None without zo) [T][D] and dh0 [S][D]."""
    zf, g, dy = (np.asarray(a, np.float64) for a in (zf, g, dy))
    S, D = len(off) - 1, zf.shape[1]
    _, _, h = scan_forward(off, zf, g, zo, h0, reverse)
    f, fc = sigmoid(zf), sigmoid(-zf)
    o = np.ones_like(zf) if zo is None else sigmoid(zo)
    dh0 = np.zeros((S, D)) if dhT is None else np.array(dhT, np.float64)
    dzf, dg, dzo = (np.full(zf.shape, np.nan) for _ in range(3))
    for s in range(S):
        toks = _tokens(off, s, reverse)
        for i in range(len(toks) - 1, -1, -1):
            t = toks[i]
            prev = h[toks[i - 1]] if i else (0.0 if h0 is None else np.asarray(h0, np.float64)[s])
            lam = o[t] * dy[t] + dh0[s]
            dg[t] = fc[t] * lam
            dzf[t] = f[t] * fc[t] * (prev - g[t]) * lam
            dzo[t] = dy[t] * h[t] * o[t] * (1 - o[t])
            dh0[s] = f[t] * lam
    return dict(dzf=dzf, dg=dg, dzo=None if zo is None else dzo, dh0=dh0)


def scan_step(zf, g, zo, h):
    """(y, h) of one token per row."""
    h = sigmoid(zf) * np.asarray(h, np.float64) + sigmoid(-np.asarray(zf, np.float64)) * np.asarray(g, np.float64)
    return (h if zo is None else h * sigmoid(zo)), h


def blocknorm_forward(x, z=None, u=None, w_post=None, scale=None, w_pre=None, eps=1e-6):
    """(r, v): v None without w_pre. Any of z (then u, w_post and scale too), u, w_post, scale may be None."""
    r = np.asarray(x, np.float64).copy()
    if z is not None:
        z = np.asarray(z, np.float64)
        n = z / np.sqrt((z * z).mean(1, keepdims=True) + eps)
        if w_post is not None:
            n = n * w_post
        if u is not None:
            n = n * sigmoid(u)
        r = r + (n if scale is None else n * scale)
    v = None
    if w_pre is not None:
        v = r / np.sqrt((r * r).mean(1, keepdims=True) + eps) * w_pre
    return r, v


def _norm_grad(a, t, eps):
    """Gradient of sum(t * a / rms(a)) with respect to a, row by row."""
    D = a.shape[1]
    m = np.sqrt((a * a).mean(1, keepdims=True) + eps)
    return t / m - a * (t * a).sum(1, keepdims=True) / (D * m ** 3)


def blocknorm_backward(x, z, u, w_post, scale, w_pre, dr, dv, eps=1e-6):
    """dict of dx, dz, du, dw_post, dscale, dw_pre (None where the input is). dr or dv may be None."""
    r, _ = blocknorm_forward(x, z, u, w_post, scale, None, eps)
    d = np.zeros_like(r) if dr is None else np.array(dr, np.float64)
    out = dict.fromkeys(("dz", "du", "dw_post", "dscale", "dw_pre"))
    if w_pre is not None:
        dv = np.asarray(dv, np.float64)
        d = d + _norm_grad(r, dv * w_pre, eps)
        out["dw_pre"] = (dv * r / np.sqrt((r * r).mean(1, keepdims=True) + eps)).sum(0)
    out["dx"] = d
    if z is not None:
        z = np.asarray(z, np.float64)
        zh = z / np.sqrt((z * z).mean(1, keepdims=True) + eps)
        s = 1.0 if u is None else sigmoid(u)
        wp = 1.0 if w_post is None else np.asarray(w_post, np.float64)
        sc = 1.0 if scale is None else np.asarray(scale, np.float64)
        out["dz"] = _norm_grad(z, d * s * sc * wp, eps)
        if u is not None:
            out["du"] = d * sc * zh * wp * s * (1 - s)
        if w_post is not None:
            out["dw_post"] = (d * s * sc * zh).sum(0)
        if scale is not None:
            out["dscale"] = (d * s * zh * wp).sum(0)
    return out


def distill(z, ids, t, w=None, tau=1.0):
    """(loss [N], dz [N][V]). A slot with id -1 is empty; a row of empty slots, or of weight 0, counts for nothing; in any
    other row an id outside [-1, V) makes the loss NaN and the gradient zero."""
    z, t = np.asarray(z, np.float64), np.asarray(t, np.float64)
    N, V = z.shape
    loss, dz = np.zeros(N), np.zeros((N, V))
    for n in range(N):
        wn = 1.0 if w is None else float(w[n])
        kept = [j for j, i in enumerate(ids[n]) if i != -1]
        if not kept or wn == 0.0:
            continue
        if any(not 0 <= ids[n][j] < V for j in kept):
            loss[n] = np.nan
            continue
        a = z[n] / tau
        a = a - a.max()
        lq = a - np.log(np.exp(a).sum())
        b = t[n][kept] / tau
        b = b - b.max()
        lp = b - np.log(np.exp(b).sum())
        p = np.exp(lp)
        dz[n] = np.exp(lq)
        for pj, lpj, j in zip(p, lp, kept):
            i = ids[n][j]
            if pj > 0:
                loss[n] += wn * tau * tau * pj * (lpj - lq[i])
            dz[n, i] -= pj
        dz[n] *= wn * tau
    return loss, dz
