"""GPU parity of the cross entropy over a vocabulary (mdl_vocab_loss) against the float64 oracle.

Tolerances are computed from the inputs. u = 2^-24, Z = max_c sum_d |h_d W_cd| of a row:
    a logit is a sum of D products:  dz <= (D + 2) u Z
    the sum of exponentials adds up to V of them in groups (32 a lane, then lanes, waves and tiles: below 64 + V / 1024
    roundings), each exponential off by its argument's (2 dz + |x| u, where |x| e^x < 1) and 4 u of its own; the joining
    factors 6 u a tile and group: dlse <= dz + (80 + V / 512) u + 2 u |lse|
    loss: w (dz + dlse + u (|lse| + |z_id|)), and the logarithm's and the product's own roundings
    p = e^(z - lse): p (dz + dlse + (|z - lse| + 4) u),  G = w (p - [c = id]) : that and 2 u |G|, then half a step of the type
    dh, dW: those of G times |W| or |h|, summed; (terms + 2) u of the sum of magnitudes for the product's own sum, and half a
    step of the type at the end. Pieces and slabs only regroup the same sum.
"""

import numpy as np
import pytest
import torch

from oracle import block as oblk

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
TINY = 1e-30    # products below the normal range of fp32

if torch.cuda.is_available():
    from directional_mdlstm_handwriting_amd.layer import VocabLoss

TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": U, "bf16": 2.0 ** -8}


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _inputs(seed, N, D, V, dtype, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(N, D + 3, generator=g).to(TDT[dtype]).to(DEV)[:, 1:D + 1]      # rows apart, at no round address
    W = (torch.randn(V, D, generator=g) * spread * D ** -0.5).to(TDT[dtype]).to(DEV)
    ids = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    w = torch.rand(N, generator=g) + 0.25
    if N > 2:
        ids[1] = -1
        w[2] = 0.0
    return h, W, ids.to(DEV), w.to(DEV)


def _within(name, got, ref, tol):
    err = np.abs(got - ref)
    bad = ~(err <= tol + TINY)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {err.size}, worst {np.nanmax(err / (tol + TINY)):.3g} of the tolerance"


def tolerances(h, W, ids, w, ref, dtype):
    """(loss, dh, dW) for numpy arrays; ref: the oracle's (loss, dh, dW, p)."""
    loss, dh, dW, p = ref
    V, D = W.shape
    N = h.shape[0]
    z = h @ W.T
    Z = (np.abs(h) @ np.abs(W).T).max(1)
    live = (ids >= 0) & (w != 0)
    lse = np.log(np.exp(z - z.max(1)[:, None]).sum(1)) + z.max(1)
    dz = (D + 2) * U * Z
    dlse = dz + (80 + V / 512) * U + 2 * U * np.abs(lse)
    zt = z[np.arange(N), np.maximum(ids, 0)]
    tl = live * np.abs(w) * (dz + dlse + 2 * U * (np.abs(lse) + np.abs(zt))) + 2 * U * np.abs(loss)
    aw = (live * np.abs(w))[:, None]
    hot = np.zeros((N, V))
    hot[np.arange(N)[live], ids[live]] = 1
    G = aw * np.abs(p - hot)
    # bfloat16: what is kept of a logit is q = exp(z - top) <= 1, top its tile's maximum, in half precision, whose error is
    # 2^-11 q at most, or 2^-25 below its smallest normal number; then p = q exp(top - lse), so that p is off by 2^-11 p or
    # by 2^-25 exp(top - lse) = 2^-25 of the tile's largest p. The target's p does not come from there. (The second
    # exponential is 4 U, and |z - top| + |top - lse| is |z - lse|.)
    kept = (1 - hot) * (p * 2.0 ** -11 + p.max(1)[:, None] * 2.0 ** -25 + 4 * U * p) if dtype == "bf16" else 0
    dG = aw * (p * ((dz + dlse)[:, None] + (np.abs(z - lse[:, None]) + 4) * U) + kept) + (2 * U + HALF[dtype] * 1.01) * G
    th = dG @ np.abs(W) + (V + 2) * U * (G @ np.abs(W))
    tW = dG.T @ np.abs(h) + (N + 2) * U * (G.T @ np.abs(h))
    return tl, th + HALF[dtype] * (np.abs(dh) + th), tW + HALF[dtype] * (np.abs(dW) + tW)


def check(h, W, ids, w, dtype, got):
    H, Wn, I, w_ = _np(h), _np(W), ids.cpu().numpy(), (np.ones(h.shape[0]) if w is None else _np(w))
    ref = oblk.vocab_loss(H, Wn, I, w_)
    tl, th, tW = tolerances(H, Wn, I, w_, ref, dtype)
    _within("loss", _np(got[0]), ref[0], tl)
    if got[1] is not None:
        _within("dh", _np(got[1]), ref[1], th)
        _within("dW", _np(got[2]), ref[2], tW)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D,V", [(1, 1, 1), (1, 64, 2), (5, 7, 80), (3, 50, 129), (130, 136, 700), (257, 33, 256),
                                   (64, 100, 2500), (300, 50, 80), (129, 260, 127), (1, 520, 1000), (2000, 16, 40)])
def test_values(N, D, V, dtype):
    h, W, ids, w = _inputs(N + D + V, N, D, V, dtype)
    vl = VocabLoss(N, D, V, dtype, device=DEV)
    got = [t.clone() for t in vl.run(h, W, ids, w)]
    torch.cuda.synchronize()
    check(h, W, ids, w, dtype, got)
    alone, no_h, no_W = vl.run(h, W, ids, w, want_grads=False)
    assert no_h is None and no_W is None and torch.equal(alone, got[0])
    check(h, W, ids, None, dtype, vl.run(h, W, ids))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_logits(dtype):
    """Logits of some hundreds: the maximum is taken off before any exponential, in each tile and where they are joined."""
    h, W, ids, w = _inputs(5, 40, 64, 900, dtype, spread=60.0)
    vl = VocabLoss(40, 64, 900, dtype, device=DEV)
    check(h, W, ids, w, dtype, vl.run(h, W, ids, w))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [90, 1000])
def test_confident_rows(V, dtype):
    """Targets of probability near 1, whose gradient is the small difference, and rows whose target is all but impossible."""
    N, D = 150, 96
    h, W, ids, w = _inputs(9, N, D, V, dtype, spread=6.0)
    best = torch.topk(h.float() @ W.float().t(), 2, 1).indices.int()
    ids[:100] = best[:100, 0]
    ids[100:120] = best[100:120, 1]
    vl = VocabLoss(N, D, V, dtype, device=DEV)
    check(h, W, ids, w, dtype, vl.run(h, W, ids, w))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_whole_tiles_of_impossible_classes(dtype):
    """Classes 256 to 899 some thousands below the others: their tiles' own maxima are that low too."""
    N, D, V = 300, 64, 1100
    h, W, ids, w = _inputs(10, N, D, V, dtype)
    h[:, 0] = 8.0
    W[:, 0] = 0.0
    W[256:900, 0] = -512.0
    ids[ids >= 0] %= 256
    vl = VocabLoss(N, D, V, dtype, device=DEV)
    loss, dh, dW = vl.run(h, W, ids, w)
    check(h, W, ids, w, dtype, (loss, dh, dW))
    assert (dW[256:900] == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_bad_rows_in_bfloat16(bad):
    """A NaN or infinity in one row's hidden state: NaN in its loss and gradient, in no other row's."""
    N, D, V = 300, 64, 1500
    h, W, ids, w = _inputs(12, N, D, V, "bf16")
    h = h.contiguous()
    vl = VocabLoss(N, D, V, "bf16", device=DEV)
    ref = [t.clone() for t in vl.run(h, W, ids, w)]
    h[7, 3] = bad
    loss, dh, dW = vl.run(h, W, ids, w)
    assert torch.isnan(loss[7]) and torch.isnan(dh[7]).all()
    rest = [i for i in range(N) if i != 7]
    assert torch.equal(loss[rest], ref[0][rest]) and torch.equal(dh[rest], ref[1][rest])


@pytest.mark.parametrize("dtype,N,D,V", [("bf16", 16500, 24, 8000), ("f32", 5000, 8, 9000), ("bf16", 700, 40, 60000),
                                         ("bf16", 6000, 256, 12800), ("f32", 1000, 64, 70000), ("f32", 40, 300, 9001), ("f32", 9000, 8, 9000),
                                         ("bf16", 2500, 24, 130001), ("bf16", 40000, 24, 8000), ("bf16", 3500, 512, 40000),
                                         ("bf16", 1024, 512, 50000)])
def test_pieces_and_large_tiles(dtype, N, D, V):
    """Several blocks of rows, and sizes that take the larger tiles; the reference in float64 on the device."""
    h, W, ids, w = _inputs(17, N, D, V, dtype)
    vl = VocabLoss(N, D, V, dtype, device=DEV)
    loss, dh, dW = vl.run(h, W, ids, w)
    H, Wd, wd = h.double(), W.double(), w.double() * (ids >= 0)
    ref_h, ref_W = torch.empty_like(H), torch.zeros_like(Wd)
    mag_h, mag_W = torch.empty_like(H), torch.zeros_like(Wd)
    ref_l = torch.empty_like(wd)
    eps = 0.0
    for a in range(0, N, 1000):
        x, i = H[a:a + 1000], ids[a:a + 1000].long().clamp(min=0)
        z = x @ Wd.t().contiguous()
        lse = torch.logsumexp(z, 1)
        r = torch.arange(len(i), device=DEV)
        ref_l[a:a + 1000] = wd[a:a + 1000] * (lse - z[r, i])
        g = torch.exp(z - lse[:, None])
        p = g.clone()
        g[r, i] -= 1
        g *= wd[a:a + 1000, None]
        zmax = (x.abs() @ Wd.abs().t().contiguous()).max(1).values
        dz = (D + 2) * U * zmax
        dl = dz + (80 + V / 512) * U + 2 * U * lse.abs()
        dg = wd[a:a + 1000, None] * p * ((dz + dl)[:, None] + ((z - lse[:, None]).abs() + 4) * U)
        if dtype == "bf16":  # the rounding of what is kept, as in tolerances()
            dg += wd[a:a + 1000, None] * (p * 2.0 ** -11 + p.max(1).values[:, None] * 2.0 ** -25 + 4 * U * p)
        dg += (2 * U + 1.01 * HALF[dtype]) * g.abs()
        eps = torch.cat([eps, wd[a:a + 1000] * (dz + dl + 2 * U * (lse.abs() + z[r, i].abs()))]) if a else \
            wd[a:a + 1000] * (dz + dl + 2 * U * (lse.abs() + z[r, i].abs()))
        ref_h[a:a + 1000] = g @ Wd
        mag_h[a:a + 1000] = (dg + (V + 2) * U * g.abs()) @ Wd.abs()
        ref_W += g.t().contiguous() @ x
        mag_W += (dg + (N + 2) * U * g.abs()).t().contiguous() @ x.abs()
    half = HALF[dtype]
    for name, got, ref, tol in (("loss", loss, ref_l, eps + 2 * U * ref_l.abs()),
                                ("dh", dh, ref_h, mag_h + half * (ref_h.abs() + mag_h)),
                                ("dW", dW, ref_W, mag_W + half * (ref_W.abs() + mag_W))):
        err = (got.double() - ref).abs()
        assert bool((err <= tol + TINY).all()), f"{name}: worst {float((err / (tol + TINY)).max()):.3g} of the tolerance"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_that_count_for_nothing(dtype):
    N, D, V = 200, 48, 300
    h, W, ids, w = _inputs(3, N, D, V, dtype)
    ids[10:50] = -1
    w[60:90] = 0
    vl = VocabLoss(N, D, V, dtype, device=DEV)
    ref = [t.clone() for t in vl.run(h, W, ids, w)]
    h[10:50] = float("nan")
    h[60:90] = float("inf")
    ids[60:90] = V + 7
    got = vl.run(h, W, ids, w)
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    for r in (slice(10, 50), slice(60, 90)):
        assert (got[0][r] == 0).all() and (got[1][r] == 0).all()
    # a target that is no class: NaN in its loss alone
    ids[5] = V
    ids[6] = -2
    loss, dh, dW = vl.run(h, W, ids, w)
    assert torch.isnan(loss[5:7]).all() and (dh[5:7] == 0).all()
    rest = [i for i in range(N) if i not in (5, 6)]
    assert torch.equal(loss[rest], ref[0][rest]) and torch.equal(dh[rest], ref[1][rest]) and torch.isfinite(dW).all()


def test_no_rows_and_no_targets():
    W = torch.randn(20, 12, device=DEV)
    vl = VocabLoss(0, 12, 20, "f32", device=DEV)
    loss, dh, dW = vl.run(torch.empty(0, 12, device=DEV), W, torch.empty(0, dtype=torch.int32, device=DEV))
    assert loss.numel() == 0 and dh.numel() == 0 and (dW == 0).all()
    vl = VocabLoss(9, 12, 20, "f32", device=DEV)
    loss, dh, dW = vl.run(torch.randn(9, 12, device=DEV), W, torch.full((9,), -1, dtype=torch.int32, device=DEV))
    assert (loss == 0).all() and (dh == 0).all() and (dW == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nan_logits_reach_their_rows(bad):
    """One class whose logit is NaN or +inf in one row: that row's loss and gradient, no other's loss."""
    N, D, V = 140, 16, 600
    h = torch.zeros(N, D, device=DEV)
    h[:, 0] = 1.0
    W = torch.randn(V, D, generator=torch.Generator().manual_seed(1)).to(DEV)
    ids = torch.arange(N, device=DEV, dtype=torch.int32)
    h[7, 3] = bad
    vl = VocabLoss(N, D, V, "f32", device=DEV)
    loss, dh, dW = vl.run(h, W, ids)
    assert torch.isnan(loss[7]) and torch.isnan(dh[7]).all()
    rest = [i for i in range(N) if i != 7]
    assert torch.isfinite(loss[rest]).all() and torch.isfinite(dh[rest]).all()


def test_class_ruled_out_by_minus_infinity():
    """A class of logit -inf in every row has probability 0; a row of which all are -inf is NaN."""
    N, D, V = 9, 8, 400
    h = torch.rand(N, D, device=DEV) + 0.5
    W = torch.randn(V, D, device=DEV)
    W[11] = -float("inf")
    ids = torch.full((N,), 200, dtype=torch.int32, device=DEV)
    vl = VocabLoss(N, D, V, "f32", device=DEV)
    loss = vl.run(h, W, ids, want_grads=False)[0].clone()
    keep = [c for c in range(V) if c != 11]
    ref = torch.logsumexp(h.double() @ W[keep].double().t(), 1) - h.double() @ W[200].double()
    assert torch.allclose(loss.double(), ref, rtol=1e-5, atol=1e-5)
    W[:] = -float("inf")
    assert torch.isnan(vl.run(h, W, ids, want_grads=False)[0]).all()


def test_dh_over_h():
    N, D, V = 70, 40, 150
    h, W, ids, w = _inputs(2, N, D, V, "bf16")
    h = h.contiguous()
    vl = VocabLoss(N, D, V, "bf16", device=DEV)
    ref = [t.clone() for t in vl.run(h, W, ids, w)]
    vl.dh = h
    loss, dh, dW = vl.run(h, W, ids, w)
    assert dh.data_ptr() == h.data_ptr()
    for a, b in zip((loss, dh, dW), ref):
        assert torch.equal(a, b)


def test_gradients_against_differences():
    """The oracle's losses along random directions, against the kernels' gradients."""
    N, D, V = 12, 20, 33
    h, W, ids, w = _inputs(6, N, D, V, "f32")
    loss, dh, dW = VocabLoss(N, D, V, "f32", device=DEV).run(h, W, ids, w)
    H, Wn, I, wn = _np(h), _np(W), ids.cpu().numpy(), _np(w)
    rng = np.random.default_rng(0)
    for g, base in ((dh, 0), (dW, 1)):
        e = rng.standard_normal(g.shape)
        s = 1e-4
        f = lambda t: oblk.vocab_loss(*((H + t * e, Wn) if base == 0 else (H, Wn + t * e)), I, wn)[0].sum()  # noqa: E731
        diff = (f(s) - f(-s)) / (2 * s)
        # the third derivative of the loss along e, bounded by the cubes of the logits' change: below 1e3 here, times s^2 / 6
        mag = float((np.abs(_np(g)) * np.abs(e)).sum())
        assert abs(diff - float((_np(g) * e).sum())) <= 1e3 * s * s + 200 * U * mag + 1e-9
