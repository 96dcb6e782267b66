"""Float64 oracle of a sequence block's operators beside the recurrence, written from their formulas.

* linear attention with a decay for each head over packed sequences and its gradients, one token at a time:
  S_t = d S_{t-1} + k_t v_t^T, y_t = scale S_t^T q_t;
* softmax cross entropy over a vocabulary from hidden states and class weights, and its gradients, row by row;
* dropout from Philox 4x32-10, one group of eight elements at a time, in Python's integers.

Rows that no sequence holds come back as NaN: no caller may use them.
"""

import numpy as np


def _tokens(off, s, reverse):
    t = range(int(off[s]), int(off[s + 1]))
    return list(reversed(t)) if reverse else list(t)


def _states(off, H, Dk, Dv, h):
    return np.zeros((len(off) - 1, H, Dk, Dv)) if h is None else np.array(h, np.float64)


def attention_forward(off, q, k, v, decay, scale, h0=None, reverse=False):
    """(y [T][H][Dv], hT [S][H][Dk][Dv]) of q, k [T][H][Dk] and v [T][H][Dv]."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    d = np.asarray(decay, np.float64)[:, None, None]
    hT = _states(off, q.shape[1], q.shape[2], v.shape[2], h0)
    y = np.full(v.shape, np.nan)
    for s in range(len(off) - 1):
        for t in _tokens(off, s, reverse):
            hT[s] = d * hT[s] + k[t][:, :, None] * v[t][:, None, :]
            y[t] = scale * (q[t][:, :, None] * hT[s]).sum(1)
    return y, hT


def attention_backward(off, q, k, v, dy, decay, scale, h0=None, dhT=None, reverse=False):
    """dict of dq, dk, dv and dh0 [S][H][Dk][Dv]."""
    q, k, v, dy = (np.asarray(a, np.float64) for a in (q, k, v, dy))
    d = np.asarray(decay, np.float64)[:, None, None]
    state = _states(off, q.shape[1], q.shape[2], v.shape[2], h0)
    grad = _states(off, q.shape[1], q.shape[2], v.shape[2], dhT)
    dq, dk, dv = (np.full(a.shape, np.nan) for a in (q, k, v))
    for s in range(len(off) - 1):
        toks = _tokens(off, s, reverse)
        for t in toks:
            state[s] = d * state[s] + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = scale * (state[s] * dy[t][:, None, :]).sum(2)
        for t in reversed(toks):
            g = grad[s] + scale * q[t][:, :, None] * dy[t][:, None, :]
            dk[t] = (g * v[t][:, None, :]).sum(2)
            dv[t] = (g * k[t][:, :, None]).sum(1)
            grad[s] = d * g
    return dict(dq=dq, dk=dk, dv=dv, dh0=grad)


def attention_step(q, k, v, state, decay, scale):
    """(y [S][H][Dv], new states) of one token for each of S states."""
    q, k, v, state = (np.asarray(a, np.float64) for a in (q, k, v, state))
    new = np.asarray(decay, np.float64)[:, None, None] * state + k[..., None] * v[..., None, :]
    return scale * (q[..., None] * new).sum(2), new


def vocab_loss(h, W, ids, w=None):
    """(loss [N], dh [N][D], dW [V][D], p [N][V]): rows with id -1 or weight 0 count for nothing (p = 0 there)."""
    h, W = np.asarray(h, np.float64), np.asarray(W, np.float64)
    N, V = h.shape[0], W.shape[0]
    w = np.ones(N) if w is None else np.asarray(w, np.float64)
    loss, dh, dW, ps = np.zeros(N), np.zeros(h.shape), np.zeros(W.shape), np.zeros((N, V))
    for n in range(N):
        if ids[n] == -1 or w[n] == 0:
            continue
        z = W @ h[n]
        m = z.max()
        e = np.exp(z - m)
        ps[n] = e / e.sum()
        loss[n] = w[n] * (m + np.log(e.sum()) - z[ids[n]])
        g = w[n] * ps[n]
        g[ids[n]] -= w[n]
        dh[n] = g @ W
        dW += np.outer(g, h[n])
    return loss, dh, dW, ps


_M32 = 0xFFFFFFFF


def philox(counter, call, seed):
    """The four words of Philox 4x32-10 with counter (counter, call) and key seed, all 64-bit."""
    c = [counter & _M32, counter >> 32 & _M32, call & _M32, call >> 32 & _M32]
    k = [seed & _M32, seed >> 32 & _M32]
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [b >> 32 ^ c[1] ^ k[0], b & _M32, a >> 32 ^ c[3] ^ k[1], a & _M32]
        k = [k[0] + 0x9E3779B9 & _M32, k[1] + 0xBB67AE85 & _M32]
    return c


def dropout_mask(N, D, p, seed, call):
    """[N][D] of 0 and 65536 / (65536 - round(65536 p))."""
    cut = int(np.rint(float(np.float32(p)) * 65536))
    per_row = -(-D // 8)
    m = np.zeros((N, D))
    for n in range(N):
        for g in range(per_row):
            w = philox(n * per_row + g, call, seed)
            halves = [h for x in w for h in (x & 0xFFFF, x >> 16)]
            for j in range(min(8, D - 8 * g)):
                m[n, 8 * g + j] = 65536 / (65536 - cut) if halves[j] >= cut else 0.0
    return m


def dropout(x, mask, r=None):
    """r + x mask, where a dropped element adds 0 whatever it is."""
    y = np.where(mask > 0, np.asarray(x, np.float64) * mask, 0.0)
    return y if r is None else y + np.asarray(r, np.float64)
