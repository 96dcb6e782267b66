"""GPU parity of dropout (mdl_dropout) against the oracle's generator and float64 sums.

Masks are equal, element by element. Values: x times the scale (rounded to fp32: u = 2^-24 relative), the product u and
the sum with the residual u of what is added: 2 u |x s| + u |y|, and a bfloat16 output its half step, 2^-8.
"""

import numpy as np
import pytest
import torch

from oracle import block as oblk

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24

if torch.cuda.is_available():
    from directional_mdlstm_handwriting_amd.layer import Dropout

TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": U, "bf16": 2.0 ** -8}


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _close(name, got, ref, prod, half):
    err = np.abs(_np(got) - ref)
    tol = 2.1 * U * np.abs(prod) + U * np.abs(ref)
    bad = ~(err <= tol + half * (np.abs(ref) + tol))
    assert not bad.any(), f"{name}: {int(bad.sum())} of {err.size}"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D", [(1, 1), (1, 7), (3, 8), (5, 9), (2, 4099), (130, 50), (70, 64), (33, 129), (1100, 8)])
@pytest.mark.parametrize("p", [0.1, 0.5])
def test_values(N, D, p, dtype):
    g = torch.Generator().manual_seed(N + D)
    wide = torch.randn(N, 3 * D + 5, generator=g).to(TDT[dtype]).to(DEV)
    x, r, dy = wide[:, 1:D + 1], wide[:, D + 1:2 * D + 1], wide[:, 2 * D + 1:3 * D + 1]
    seed, call = 2 ** 63 + 12345 + N, 2 ** 40 + D
    dr = Dropout(N, D, p, dtype, seed=seed, call=call, device=DEV)
    y, y0, dx = dr.forward(x, r).clone(), dr.forward(x).clone(), dr.backward(dy)
    torch.cuda.synchronize()
    m = oblk.dropout_mask(N, D, p, seed, call)
    X, R, DY = _np(x), _np(r), _np(dy)
    _close("y", y, oblk.dropout(X, m, R), X * m, HALF[dtype])
    _close("y without r", y0, oblk.dropout(X, m), X * m, HALF[dtype])
    _close("dx", dx, oblk.dropout(DY, m), DY * m, HALF[dtype])


def test_share_of_dropped():
    """Over 2^20 elements the share that is dropped lies within six standard deviations of p, and two calls' masks agree
    as often as independent ones do."""
    N, D, p = 1024, 1024, 0.3
    dr = Dropout(N, D, p, "f32", seed=5, device=DEV)
    one = torch.ones(N, D, device=DEV)
    a = dr.forward(one).clone() > 0
    assert torch.equal(dr.forward(one) > 0, a)
    dr.advance()
    b = dr.forward(one) > 0
    n = N * D
    assert abs(float((~a).double().mean()) - p) < 6 * (p * (1 - p) / n) ** 0.5
    both = 1 - 2 * p * (1 - p)
    assert abs(float((a == b).double().mean()) - both) < 6 * (both * (1 - both) / n) ** 0.5


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place_and_nothing_dropped(dtype):
    N, D = 37, 61
    g = torch.Generator().manual_seed(1)
    x, r = (torch.randn(N, D, generator=g).to(TDT[dtype]).to(DEV) for _ in range(2))
    dr = Dropout(N, D, 0.25, dtype, seed=9, device=DEV)
    y = dr.forward(x, r).clone()
    over_x, over_r = x.clone(), r.clone()
    assert dr.forward(over_x, r, out=over_x) is over_x and torch.equal(over_x, y)
    assert torch.equal(dr.forward(x, over_r, out=over_r), y)
    none = Dropout(N, D, 0.0, dtype, device=DEV)
    assert torch.equal(none.forward(x), x)
    assert torch.equal(none.forward(x, r), (x.float() + r.float()).to(TDT[dtype]))


def test_dropped_elements_add_nothing():
    N, D = 16, 40
    x = torch.full((N, D), float("nan"), device=DEV)
    r = torch.ones(N, D, device=DEV)
    dr = Dropout(N, D, 0.5, "f32", seed=3, device=DEV)
    kept = dr.forward(r).clone() > 0
    y = dr.forward(x, r)
    assert torch.equal(torch.isnan(y), kept) and (y[~kept] == 1).all()


def test_captured_masks_follow_their_words():
    """A captured forward, backward and advance draw new masks at every replay, those of the eager calls."""
    N, D = 64, 96
    x = torch.randn(N, D, device=DEV)
    eager = Dropout(N, D, 0.2, "f32", seed=77, device=DEV)
    dr = Dropout(N, D, 0.2, "f32", seed=77, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        dr.forward(x)
        dr.backward(x)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dx = dr.forward(x), dr.backward(x)
        dr.advance()
    for _ in range(4):
        graph.replay()
        ey, edx = eager.forward(x), eager.backward(x)
        torch.cuda.synchronize()
        assert torch.equal(y, ey) and torch.equal(dx, edx)
        eager.advance()
