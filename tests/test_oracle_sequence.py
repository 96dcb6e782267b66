"""Pins of the sequence operators' oracle (oracle/sequence.py): torch's autograd in float64 over separately written
forms, finite differences, and closed forms."""

import numpy as np
import pytest
import torch

from oracle import sequence as oseq


def _scan_torch(off, zf, g, zo, h0, reverse):
    """Cumulative-product form: h_t = sum_j (prod_{j < i <= t} f_i) (1 - f_j) g_j + (prod f) h0, per sequence."""
    ys, hT = [None] * zf.shape[0], []
    for s in range(len(off) - 1):
        idx = list(range(off[s], off[s + 1]))
        idx = idx[::-1] if reverse else idx
        last = h0[s]
        for n, t in enumerate(idx):
            acc = h0[s]
            for j in range(n + 1):
                acc = acc * torch.sigmoid(zf[idx[j]])
            for j in range(n + 1):
                w = 1 - torch.sigmoid(zf[idx[j]])
                for i in range(j + 1, n + 1):
                    w = w * torch.sigmoid(zf[idx[i]])
                acc = acc + w * g[idx[j]]
            last = acc
            ys[t] = torch.sigmoid(zo[t]) * acc
        hT.append(last)
    return torch.stack(ys), torch.stack(hT)


@pytest.mark.parametrize("reverse", [False, True])
def test_scan_against_autograd(reverse):
    rng = np.random.default_rng(1)
    off, D = [0, 3, 3, 8, 9], 2
    T, S = off[-1], len(off) - 1
    zf, g, zo, dy = (rng.normal(0, 1, (T, D)) for _ in range(4))
    h0, dhT = rng.normal(0, 1, (S, D)), rng.normal(0, 1, (S, D))
    leaves = [torch.tensor(a, requires_grad=True) for a in (zf, g, zo, h0)]
    y, hT = _scan_torch(off, *leaves, reverse)
    ry, rhT, _ = oseq.scan_forward(off, zf, g, zo, h0, reverse)
    assert np.allclose(ry, y.detach().numpy(), rtol=0, atol=1e-13)
    assert np.allclose(rhT, hT.detach().numpy(), rtol=0, atol=1e-13)
    ((y * torch.tensor(dy)).sum() + (hT * torch.tensor(dhT)).sum()).backward()
    got = oseq.scan_backward(off, zf, g, zo, dy, h0, dhT, reverse)
    for name, leaf in zip(("dzf", "dg", "dzo", "dh0"), leaves):
        assert np.allclose(got[name], leaf.grad.numpy(), rtol=0, atol=1e-12), name


def test_scan_finite_differences():
    rng = np.random.default_rng(2)
    off, D = [0, 4, 6], 2
    args = [rng.normal(0, 1, (6, D)) for _ in range(3)] + [rng.normal(0, 1, (2, D))]
    dy, dhT = rng.normal(0, 1, (6, D)), rng.normal(0, 1, (2, D))

    def value(a):
        y, hT, _ = oseq.scan_forward(off, *a)
        return (y * dy).sum() + (hT * dhT).sum()

    got = oseq.scan_backward(off, args[0], args[1], args[2], dy, args[3], dhT)
    _check_differences(value, args, [got[k] for k in ("dzf", "dg", "dzo", "dh0")])


def _check_differences(value, args, grads, h=1e-5):
    for k, grad in enumerate(grads):
        for i in np.ndindex(args[k].shape):
            lo, hi = [a.copy() for a in args], [a.copy() for a in args]
            lo[k][i] -= h
            hi[k][i] += h
            # central differences: h^2 truncation and 1e-16 / h rounding, both near 1e-10 for values of order ten
            assert abs((value(hi) - value(lo)) / (2 * h) - grad[i]) < 1e-7 * max(1.0, abs(grad[i])), (k, i)


def test_scan_closed_forms():
    # a constant gate and input: h_t = g (1 - f^t) + f^t h0
    T, f = 50, 0.9
    zf = np.full((T, 1), np.log(f / (1 - f)))
    _, hT, h = oseq.scan_forward([0, T], zf, np.full((T, 1), 3.0), None, np.array([[7.0]]))
    assert np.allclose(h[:, 0], 3 + 4 * f ** np.arange(1, T + 1), rtol=0, atol=1e-12)
    # gates at their ends: hold the state, or take the input
    _, hT, _ = oseq.scan_forward([0, 2], np.array([[np.inf], [np.inf]]), np.ones((2, 1)), None, np.array([[5.0]]))
    assert hT[0, 0] == 5.0
    _, hT, _ = oseq.scan_forward([0, 2], np.array([[-np.inf], [-np.inf]]), np.full((2, 1), 2.0))
    assert hT[0, 0] == 2.0


def test_step_is_the_scan_a_token_at_a_time():
    rng = np.random.default_rng(3)
    zf, g, zo = (rng.normal(0, 1, (5, 3)) for _ in range(3))
    h = rng.normal(0, 1, (1, 3))
    y, hT, _ = oseq.scan_forward([0, 5], zf, g, zo, h)
    for t in range(5):
        out, h = oseq.scan_step(zf[t:t + 1], g[t:t + 1], zo[t:t + 1], h)
        assert np.array_equal(out[0], y[t])
    assert np.array_equal(h, hT)


@pytest.mark.parametrize("parts", ["all", "no_gate", "no_scale", "pre_only", "post_only"])
def test_blocknorm_against_autograd_and_differences(parts):
    rng = np.random.default_rng(4)
    N, D, eps = 3, 5, 1e-3
    x, z, u, dr, dv = (rng.normal(0, 1, (N, D)) for _ in range(5))
    wp, sc, wn = (rng.normal(1, 0.3, D) for _ in range(3))
    if parts == "no_gate":
        u = None
    if parts == "no_scale":
        sc = None
    if parts == "pre_only":
        z = u = wp = sc = None
    if parts == "post_only":
        wn = dv = None
    names = ("x", "z", "u", "w_post", "scale", "w_pre")
    given = dict(zip(names, (x, z, u, wp, sc, wn)))
    leaves = {k: torch.tensor(a, requires_grad=True) for k, a in given.items() if a is not None}
    r = leaves["x"]
    if z is not None:
        n = leaves["z"] * torch.rsqrt(leaves["z"].square().mean(1, keepdim=True) + eps) * leaves["w_post"]
        n = n * (torch.sigmoid(leaves["u"]) if u is not None else 1) * (leaves["scale"] if sc is not None else 1)
        r = r + n
    loss = (r * torch.tensor(dr)).sum()
    if wn is not None:
        v = r * torch.rsqrt(r.square().mean(1, keepdim=True) + eps) * leaves["w_pre"]
        loss = loss + (v * torch.tensor(dv)).sum()
    loss.backward()
    rr, rv = oseq.blocknorm_forward(x, z, u, wp, sc, wn, eps)
    assert np.allclose(rr, r.detach().numpy(), rtol=0, atol=1e-13)
    assert (rv is None) == (wn is None)
    if rv is not None:
        assert np.allclose(rv, v.detach().numpy(), rtol=0, atol=1e-13)
    got = oseq.blocknorm_backward(x, z, u, wp, sc, wn, dr, dv, eps)
    for k in names:
        if k in leaves:
            assert np.allclose(got["d" + k], leaves[k].grad.numpy(), rtol=0, atol=1e-12), k
        elif k != "x":
            assert got["d" + k] is None, k
    keys = list(leaves)

    def value(a):
        kw = dict(zip(keys, a))
        r, v = oseq.blocknorm_forward(kw["x"], *(kw.get(k) for k in names[1:]), eps)
        return (r * dr).sum() + (0 if v is None else (v * dv).sum())

    _check_differences(value, [given[k] for k in keys], [got["d" + k] for k in keys])


def test_distill_against_autograd_and_closed_forms():
    rng = np.random.default_rng(5)
    N, V, k, tau = 4, 9, 3, 1.7
    z, t = rng.normal(0, 2, (N, V)), rng.normal(0, 2, (N, k))
    ids = np.stack([rng.permutation(V)[:k] for _ in range(N)])
    ids[1, 2] = -1
    ids[2, 1] = ids[2, 0]
    w = np.array([1.0, 0.5, 2.0, 0.0])
    zt = torch.tensor(z, requires_grad=True)
    total, losses = 0.0, []
    for n in range(N):
        keep = [j for j in range(k) if ids[n, j] >= 0]
        p = torch.softmax(torch.tensor(t[n, keep]) / tau, 0)
        lq = torch.log_softmax(zt[n] / tau, 0)[ids[n, keep]]
        losses.append(w[n] * tau ** 2 * (p * (p.log() - lq)).sum())
        total = total + losses[-1]
    total.backward()
    loss, dz = oseq.distill(z, ids, t, w, tau)
    assert np.allclose(loss, [float(v.detach()) for v in losses], rtol=0, atol=1e-13)
    assert np.allclose(dz, zt.grad.numpy(), rtol=0, atol=1e-13)
    _check_differences(lambda a: oseq.distill(a[0], ids, t, w, tau)[0].sum(), [z], [dz])
    # a teacher that keeps every class and equals the student: no loss, no gradient
    loss, dz = oseq.distill(z, np.tile(np.arange(V), (N, 1)), z, None, tau)
    assert np.allclose(loss, 0, atol=1e-14) and np.allclose(dz, 0, atol=1e-15)
    # one kept class: cross-entropy
    loss, _ = oseq.distill(z, ids[:, :1], t[:, :1], None, 1.0)
    assert np.allclose(loss, [-(z[n, ids[n, 0]] - np.log(np.exp(z[n]).sum())) for n in range(N)], atol=1e-13)
    # nothing kept, and a class that does not exist
    loss, dz = oseq.distill(z[:2], [[-1, -1], [0, V]], t[:2, :2])
    assert loss[0] == 0 and np.isnan(loss[1]) and not dz.any()


def test_distill_weight_zero_wins_over_a_class_that_does_not_exist():
    z, t = np.random.default_rng(4).normal(size=(3, 5)), np.zeros((3, 2))
    loss, dz = oseq.distill(z, [[9, 1], [9, 1], [-1, -1]], t, [0.0, 1.0, 1.0], 1.5)
    assert loss[0] == 0 and np.isnan(loss[1]) and loss[2] == 0 and not dz.any()
