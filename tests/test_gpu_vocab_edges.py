"""The cross entropy over a vocabulary where a row's loss and gradient are small numbers: rows sure of their target, logits
with a large common part, classes far below the best one.

The logits are whole numbers and exact in fp32 whatever the order of their sums: the first two channels of h are (1, s) and
those of W (offset, -gap), h is zero in the others, which only dh sees. With u = 2^-24, relative to a loss or an element of G:
    an exponential: 4 u, its argument exact; in bfloat16 |x| u more for the product with log2 e, of a spread |x| <= 32 below a
    tile's maximum; a sum of up to V of them in groups: 64 + V / 1024 roundings; at most 8 joins of parts at 6 u and the
    exponential that joins the target, 4 u; logarithm, reciprocal and products 12 u: in all REL = (200 + V / 512) u
    G in bfloat16: what is kept of a logit is its exponential below its tile's maximum times 2^15 in half precision: 2^-11 of it,
    or half of 2^-24, that is 2^-40 of the maximum, below the normal range
    each value of G is rounded to the type (half a step), dh and dW are sums of (terms + 2) u and rounded once.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
TINY = 1e-36

if torch.cuda.is_available():
    from directional_mdlstm_handwriting_amd.layer import VocabLoss

TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": U, "bf16": 2.0 ** -8}
D = 12


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _inputs(seed, offset, s, gaps, dtype):
    """h [N][D], W [V][D] whose logits are offset - s[n] gaps[c]."""
    g = torch.Generator().manual_seed(seed)
    h = torch.zeros(len(s), D)
    h[:, 0], h[:, 1] = 1.0, torch.as_tensor(s, dtype=torch.float32)
    W = torch.randn(len(gaps), D, generator=g)
    W[:, 0], W[:, 1] = float(offset), -torch.as_tensor(np.float32(gaps))
    return h.to(TDT[dtype]).to(DEV), W.to(TDT[dtype]).to(DEV)


def _exact(h, W, ids, w):
    """(loss, G, largest probability of a row's other classes) in float64, without a difference of near numbers."""
    z = _np(h) @ _np(W).T
    r = np.arange(len(ids))
    zt = z[r, ids]
    other = z.copy()
    other[r, ids] = -np.inf
    top = np.maximum(other.max(1), zt)
    e, et = np.exp(other - top[:, None]), np.exp(zt - top)
    so = e.sum(1)
    with np.errstate(divide="ignore", invalid="ignore"):
        loss = np.where(zt >= top, np.log1p(so), (top - zt) + np.log(so + et))
    G = e / (so + et)[:, None]
    most = G.max(1)
    G[r, ids] = -so / (so + et)
    return w * loss, w[:, None] * G, np.abs(w) * most


def _within(name, got, ref, tol):
    err = np.abs(got - ref)
    bad = ~(err <= tol + TINY)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {err.size}, worst {np.nanmax(err / (tol + TINY)):.3g} of the tolerance"


def check(h, W, ids, w, dtype, got):
    V, half = W.shape[0], HALF[dtype]
    H, Wn = np.abs(_np(h)), np.abs(_np(W))
    loss, G, most = _exact(h, W, ids, w)
    rel = (200 + V / 512) * U
    kept = 0.0
    if dtype == "bf16":
        kept = 2.0 ** -11 * np.abs(G) + 2.0 ** -40 * most[:, None]
    dG = np.abs(G) * (rel + 1.01 * half) + kept
    A = np.abs(G)
    th = dG @ Wn + (V + 2) * U * (A @ Wn)
    tW = dG.T @ H + (len(ids) + 2) * U * (A.T @ H)
    dh, dW = G @ _np(W), G.T @ _np(h)
    _within("loss", _np(got[0]), loss, rel * np.abs(loss))
    _within("dh", _np(got[1]), dh, th + half * (np.abs(dh) + th))
    _within("dW", _np(got[2]), dW, tW + half * (np.abs(dW) + tW))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [90, 700])
def test_classes_far_below_the_best_one(V, dtype):
    """Classes 18 to 24 below the best one of their own tile, in rows that are sure of it and in rows whose target is another:
    their rows of dW are their own small numbers."""
    N = 40
    gaps = 18.0 + np.arange(V) % 7
    gaps[5] = 0.0            # the best class of each row
    gaps[7] = 2.0            # the target of the second half
    h, W = _inputs(1, 0, np.ones(N), gaps, dtype)
    ids = np.full(N, 5, np.int64)
    ids[N // 2:] = 7
    vl = VocabLoss(N, D, V, dtype, device=DEV)
    dW = _np(vl.run(h, W, torch.as_tensor(ids, dtype=torch.int32, device=DEV))[2])
    _, G, _ = _exact(h, W, ids, np.ones(N))
    ref = G.T @ _np(h)
    rest = np.array([c for c in range(V) if c not in (5, 7)])
    # the best class's own logit is 0: 2^-22 covers what is added to it in the logarithm of the sum
    tol = np.abs(G).T @ np.abs(_np(h)) * ((200 + V / 512) * U + 2.0 ** -22 + 2.01 * HALF[dtype] + (N + 2) * U)
    if dtype == "bf16":
        tol += np.abs(ref) * 2.0 ** -11 + N * 2.0 ** -40
    _within("dW", dW[rest], ref[rest], tol[rest])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,target", [(90, 0), (90, 89), (700, 300), (700, 699), (257, 256), (2, 1)])
@pytest.mark.parametrize("offset", [0, 30, 300, -300])
@pytest.mark.parametrize("gap", [10, 14, 18, 30])
def test_sure_rows(gap, offset, V, target, dtype):
    """Losses and gradients of e^-10 to e^-68 beside logits of up to some hundreds: right relative to themselves."""
    N = 33
    gaps = gap + np.arange(V) % 5.0
    gaps[target] = 0.0
    h, W = _inputs(gap + V, offset, 1 + np.arange(N) % 2, gaps, dtype)
    ids = np.full(N, target, np.int64)
    w = torch.rand(N, generator=torch.Generator().manual_seed(2)) + 0.25
    vl = VocabLoss(N, D, V, dtype, device=DEV)
    got = [t.clone() for t in vl.run(h, W, torch.as_tensor(ids, dtype=torch.int32, device=DEV), w.to(DEV))]
    check(h, W, ids, _np(w), dtype, got)
    alone = vl.run(h, W, torch.as_tensor(ids, dtype=torch.int32, device=DEV), w.to(DEV), want_grads=False)[0]
    assert torch.equal(alone, got[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [90, 700])
@pytest.mark.parametrize("offset", [0, 300, -300])
def test_rows_with_impossible_targets(offset, V, dtype):
    """Targets 10 to 32 below the best class, another one for each row, and rows between: losses of whole numbers and a
    little, targets' gradients of nearly -w."""
    N = 64
    gaps = np.arange(V) % 17.0
    h, W = _inputs(V, offset, 1 + np.arange(N) % 2, gaps, dtype)
    ids = (np.arange(N) * 13) % V
    w = np.ones(N)
    vl = VocabLoss(N, D, V, dtype, device=DEV)
    got = vl.run(h, W, torch.as_tensor(ids, dtype=torch.int32, device=DEV))
    check(h, W, ids, w, dtype, got)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 5, 300])
def test_targets_of_infinite_logits(V, dtype):
    """A target of +inf or NaN: NaN in its row's loss and gradient; of -inf: loss +inf, the target's gradient -w, none from it
    to the others; all other classes -inf: loss 0."""
    W = torch.zeros(V, 8)
    t = V - 1
    W[t, 0], W[t, 1], W[t, 2] = float("inf"), float("nan"), -float("inf")
    W[:t, 3] = -float("inf")
    # a zero beside an infinity is NaN, so each row's product is formed apart: one column of W at a time
    ids = torch.full((1,), t, dtype=torch.int32, device=DEV)
    vl = VocabLoss(1, 1, V, dtype, device=DEV)
    one = torch.ones(1, 1, dtype=TDT[dtype], device=DEV)
    out = []
    for i in range(4):
        loss, dh, dW = vl.run(one, W[:, i:i + 1].contiguous().to(TDT[dtype]).to(DEV), ids)
        out.append((float(loss[0]), dW[:, 0].float().cpu()))
    for loss, dW in out[:2]:
        assert np.isnan(loss) and torch.isnan(dW).all()
    loss, dW = out[2]
    if V == 1:
        assert np.isnan(loss)
    else:
        assert loss == float("inf") and float(dW[t]) == -1.0
        assert torch.allclose(dW[:t], torch.full((V - 1,), 1 / (V - 1)), rtol=2.0 ** -7)
    loss, dW = out[3]
    assert loss == 0.0 and (dW == 0).all()


def test_more_rows_than_a_launch_takes():
    """The loss alone of 2^23 rows over 2^15 classes, whose tiles one launch cannot count: each row as by itself, at the ends
    and around the middle, where one launch ends and the next begins."""
    N, K, V = 1 << 23, 8, 1 << 15
    print("[gpu] many rows", flush=True)
    g = torch.Generator(device=DEV).manual_seed(4)
    h = torch.randn(N, K, generator=g, device=DEV).to(torch.bfloat16)
    W = torch.randn(V, K, generator=g, device=DEV).to(torch.bfloat16)
    ids = torch.randint(0, V, (N,), generator=g, device=DEV, dtype=torch.int32)
    loss = VocabLoss(N, K, V, "bf16", device=DEV).run(h, W, ids, want_grads=False)[0]
    mid = N // 2
    at = torch.cat([torch.arange(a, b, device=DEV) for a, b in ((0, 70), (mid - 70, mid + 70), (N - 70, N))])
    z = h[at].double() @ W.double().t().contiguous()
    lse, zt = torch.logsumexp(z, 1), z[torch.arange(len(at), device=DEV), ids[at].long()]
    # a logit is a sum of 8 products, the rest as the file's other bounds, and |x| u of the exponentials' arguments
    big = (h[at].double().abs() @ W.double().abs().t().contiguous()).max(1).values
    tol = 2 * (K + 2) * U * big + (200 + V / 512 + 2 * big) * U + 2 * U * (lse - zt)
    assert bool(((loss[at].double() - (lse - zt)).abs() <= tol).all())
    assert bool(torch.isfinite(loss).all())
