"""GPU parity of linear attention with a decay for each head (mdl_linattn_forward / _backward / _step) against the float64
oracle.

Tolerances are computed: the oracle run on magnitudes (all inputs and the scale replaced by their absolute values) bounds
the sum of the absolute values of everything an output adds up, m. An output is off by at most
    (r + c u) m, plus its own rounding,                                                     u = 2^-24
c: a term passes the sums over a head's channels and over the tokens up to its output (at most one rounding each for the
product and the sum, 2 (D + L)), and its decay d^e is off by up to e |ln d| u for the rounded exponent and 2 u for exp2 in
each of the factors it is formed of, of which a block contributes at most three (2 L + 2 L min(|ln d|, 1); beyond that the
term itself has vanished), and a few for the scale: c = 4 (D + L) + 2 L + 16 covers both.
r, bfloat16 only: every term meets one rounding on its way to a token's output (in the products of queries and keys, or in
the entering state): half a step, 2^-8, and the state handed on within a tile is formed of two terms of bfloat16, 2^-16
more. Last states and their gradients are of unrounded products (three terms, 2^-24): r = 0.
"""

import numpy as np
import pytest
import torch

from oracle import block as oblk

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
TINY = 1e-30    # products of fp32 numbers below the normal range

if torch.cuda.is_available():
    import directional_mdlstm_handwriting_amd as M
    from directional_mdlstm_handwriting_amd.layer import AttentionState, LinearAttention

TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": U, "bf16": 2.0 ** -8}
ROUND = {"f32": 0.0, "bf16": 2.0 ** -8 + 2.0 ** -15}


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _offsets(lens, lead=0):
    return np.concatenate([[lead], lead + np.cumsum(lens)]).astype(np.int64)


def _inputs(seed, T, S, H, Dk, Dv, dtype, h0=True):
    """Values exactly representable in the tensors' type, on the device, as column blocks of one matrix."""
    g = torch.Generator().manual_seed(seed)
    p = torch.randn(T, H * (2 * Dk + Dv), generator=g).to(TDT[dtype]).to(DEV)
    q, k, v = p[:, :H * Dk], p[:, H * Dk:2 * H * Dk], p[:, 2 * H * Dk:]
    dy = torch.randn(T, H * Dv, generator=g).to(TDT[dtype]).to(DEV)
    h = torch.randn(S, H, Dk, Dv, generator=g).to(DEV) if h0 else None
    dhT = torch.randn(S, H, Dk, Dv, generator=g).to(DEV)
    return q, k, v, dy, h, dhT


def _close(name, got, ref, tol, half):
    got = _np(got).reshape(ref.shape)
    err = np.abs(got - ref)
    lim = tol + half * (np.abs(ref) + tol) + TINY
    bad = ~(err <= lim)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {err.size}, worst {np.nanmax(err / lim):.3g} of the tolerance"


def check(off, q, k, v, dy, h0, dhT, decay, scale, reverse, dtype, got):
    """got: (y, hT, dq, dk, dv, dh0), over the rows of the sequences."""
    H = len(decay)
    T = q.shape[0]
    Q, K, V, DY = (_np(t).reshape(T, H, -1) for t in (q, k, v, dy))
    H0 = None if h0 is None else _np(h0)
    DT = None if dhT is None else _np(dhT)
    d = np.asarray(decay, np.float32).astype(np.float64)
    scale = float(np.float32(scale))
    L = int(np.diff(off).max())
    c = 4 * (max(Q.shape[2], V.shape[2]) + L) + 2 * L + 16
    absn = lambda a: None if a is None else np.abs(a)  # noqa: E731
    y, hT = oblk.attention_forward(off, Q, K, V, d, scale, H0, reverse)
    my, mh = oblk.attention_forward(off, absn(Q), absn(K), absn(V), d, abs(scale), absn(H0), reverse)
    g = oblk.attention_backward(off, Q, K, V, DY, d, scale, H0, DT, reverse)
    m = oblk.attention_backward(off, absn(Q), absn(K), absn(V), absn(DY), d, abs(scale), absn(H0), absn(DT), reverse)
    live = slice(int(off[0]), int(off[-1]))
    r, half = ROUND[dtype], HALF[dtype]
    _close("y", got[0][live], y[live].reshape(-1, y.shape[1] * y.shape[2]), (r + c * U) * my[live].reshape(-1, y.shape[1] * y.shape[2]), half)
    if got[1] is not None:
        _close("hT", got[1], hT, c * U * mh, U)
    for i, n in enumerate(("dq", "dk", "dv")):
        ref, mag = (a[n][live].reshape(live.stop - live.start, -1) for a in (g, m))
        _close(n, got[2 + i][live], ref, (r + c * U) * mag, half)
    if got[5] is not None:
        _close("dh0", got[5], g["dh0"], c * U * m["dh0"], U)


def run(off, T, H, Dk, Dv, decay, dtype, reverse, h0, seed=0, scale=None):
    q, k, v, dy, h, dhT = _inputs(seed, T, len(off) - 1, H, Dk, Dv, dtype, h0)
    at = LinearAttention(off, T, H, Dk, Dv, decay, dtype, scale=scale, reverse=reverse, device=DEV)
    y, hT = at.forward(q, k, v, h)
    dq, dk, dv, dh0 = at.backward(q, k, v, dy, h, dhT)
    torch.cuda.synchronize()
    check(off, q, k, v, dy, h, dhT, decay, at.scale, reverse, dtype, (y, hT, dq, dk, dv, dh0))
    return at


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[1], [2], [31], [64], [65], [130], [256], [257], [1, 0, 5], [700]],
                         ids=lambda v: "x".join(map(str, v)))
def test_lengths(lens, dtype):
    off = _offsets(lens)
    run(off, int(off[-1]), 2, 64, 64, [0.97, 1 - 2.0 ** -9], dtype, False, True, seed=len(lens) + lens[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("H,Dk,Dv", [(1, 1, 1), (3, 8, 16), (1, 50, 50), (2, 33, 70), (2, 128, 40), (2, 24, 100), (1, 128, 128),
                                     (2, 65, 63)])
def test_heads(H, Dk, Dv, reverse, dtype):
    """Several sequences, of which some lie in one tile of 256, some cross one or two boundaries, some are empty."""
    off = _offsets([3, 0, 200, 350, 1, 64, 0, 290], lead=5)
    run(off, int(off[-1]) + 9, H, Dk, Dv, [0.9, 0.999, 1 - 2.0 ** -5][:H], dtype, reverse, True, seed=H + Dk + Dv)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("decay", [0.0, 1e-30, 0.5, 1.0])
def test_decays(decay, reverse, dtype):
    off = _offsets([300, 70])
    run(off, 370, 1, 32, 48, [decay], dtype, reverse, True, seed=3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -2.0, 1e-3])
def test_scales_and_no_states(scale, dtype):
    off = _offsets([40, 300, 90])
    run(off, 430, 2, 64, 32, [0.95, 0.99], dtype, False, False, seed=4, scale=scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_longer_tiles(dtype):
    """Enough tokens and heads that tiles hold more than 256 tokens: 40 heads of 8 over 16000 tokens."""
    off = _offsets([9000, 1, 6999])
    H = 40
    T = 16000
    q, k, v, dy, h, dhT = _inputs(11, T, 3, H, 8, 8, dtype)
    dec = 1 - 2.0 ** -(2 + np.arange(H) % 9)
    at = LinearAttention(off, T, H, 8, 8, dec, dtype, device=DEV)
    y, hT = at.forward(q, k, v, h)
    grads = at.backward(q, k, v, dy, h, dhT)
    torch.cuda.synchronize()
    check(off, q, k, v, dy, h, dhT, dec, at.scale, False, dtype, (y, hT, *grads))


def test_rows_outside_and_other_sequences():
    """Rows in no sequence keep what they hold and reach nothing, NaN in one sequence or head stays in it."""
    off = _offsets([70, 300, 30], lead=4)
    T, H, D = 411, 2, 64
    q, k, v, dy, h, dhT = _inputs(5, T, 3, H, D, D, "bf16")
    at = LinearAttention(off, T, H, D, D, [0.9, 0.99], "bf16", device=DEV)
    ref = [t.clone() for t in (*at.forward(q, k, v, h), *at.backward(q, k, v, dy, h, dhT))]
    bad = [t.clone() for t in (q, k, v, dy)]
    for t in bad:
        t[:4] = float("nan")
        t[404:] = float("inf")
        t[100, :D] = float("nan")      # head 0 of the second sequence
    for t in (at.y, at.dq, at.dk, at.dv):
        t.fill_(7.0)
    got = [*at.forward(*bad[:3], h), *at.backward(*bad[:3], bad[3], h, dhT)]
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(got, ref)):
        if i in (1, 5):                # states [S][H]..
            assert torch.equal(a[[0, 2]], b[[0, 2]]) and torch.equal(a[1, 1], b[1, 1])
            assert not torch.isfinite(a[1, 0]).all()
        else:
            assert (a[:4] == 7).all() and (a[404:] == 7).all()
            assert torch.equal(a[4:74], b[4:74]) and torch.equal(a[374:404], b[374:404])
            assert torch.equal(a[74:374, D:], b[74:374, D:])
            assert not torch.isfinite(a[74:374, :D]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_against_differences(dtype):
    """The loss sum(y w) + sum(hT u) changes along random directions as the gradients say. In float64 through the oracle,
    whose agreement with the kernels the other tests show; the kernels' own y enters in fp32."""
    off = _offsets([37, 90])
    T, H, Dk, Dv = 127, 2, 16, 24
    g = torch.Generator().manual_seed(9)
    ten = [torch.randn(T, H * n, generator=g).to(TDT[dtype]) for n in (Dk, Dk, Dv, Dv)]
    h0, u = torch.randn(2, H, Dk, Dv, generator=g), torch.randn(2, H, Dk, Dv, generator=g)
    dec = np.float32([0.9, 0.98])
    at = LinearAttention(off, T, H, Dk, Dv, dec, dtype, device=DEV)
    q, k, v, w = (t.to(DEV) for t in ten)
    at.forward(q, k, v, h0.to(DEV))
    grads = at.backward(q, k, v, w, h0.to(DEV), u.to(DEV))
    torch.cuda.synchronize()
    Q, K, V, W = (_np(t).reshape(T, H, -1) for t in ten)
    base = (Q, K, V, _np(h0))

    def loss(q, k, v, h):
        y, hT = oblk.attention_forward(off, q, k, v, dec.astype(np.float64), at.scale, h)
        return float((y * W).sum() + (hT * _np(u)).sum())

    rng = np.random.default_rng(1)
    for i, gr in enumerate(grads):
        e = rng.standard_normal(base[i].shape)
        at_ = lambda s: [b + s * e if j == i else b for j, b in enumerate(base)]  # noqa: E731
        # the loss is a polynomial of degree one in each input alone: the central difference is exact but for rounding
        diff = (loss(*at_(0.5)) - loss(*at_(-0.5)))
        G = _np(gr).reshape(e.shape)
        tol = (4 * HALF[dtype] + 3000 * U) * float((np.abs(G) * np.abs(e)).sum())
        assert abs(diff - float((G * e).sum())) <= tol + 1e-9


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,Dk,Dv", [(1, 1, 1), (2, 64, 64), (3, 50, 70), (1, 128, 128), (2, 128, 12), (2, 9, 128)])
def test_step(H, Dk, Dv, dtype):
    S, slots = 7, 10
    q, k, v, _, _, _ = _inputs(21, S, 1, H, Dk, Dv, dtype)
    st = AttentionState(slots, H, Dk, Dv, [0.9, 0.99, 1.0][:H], dtype, device=DEV)
    g = torch.Generator().manual_seed(2)
    st.state.copy_(torch.randn(st.state.shape, generator=g))
    before = st.state.clone()
    idx = torch.tensor([3, 9, -1, 0, 5, 10, 2], dtype=torch.int32, device=DEV)     # two rows without a slot
    live = [0, 1, 3, 4, 6]
    new = before.clone()
    y = st.step(q, k, v, slots=idx, out=new).clone()
    assert torch.equal(st.state, before)
    st.step(q, k, v, slots=idx)
    torch.cuda.synchronize()
    assert torch.equal(st.state, new)
    at = idx[live].long()
    rest = [i for i in range(slots) if i not in at.tolist()]
    assert torch.equal(new[rest], before[rest])
    Q, K, V = (_np(t[live]).reshape(len(live), H, -1) for t in (q, k, v))
    d = _np(st.decay)
    sc = float(np.float32(st.scale))
    ry, rh = oblk.attention_step(Q, K, V, _np(before[at]), d, sc)
    my, mh = oblk.attention_step(np.abs(Q), np.abs(K), np.abs(V), np.abs(_np(before[at])), d, sc)
    _close("state", new[at], rh, 3 * U * mh, U)
    _close("y", y[live], ry.reshape(len(live), -1), (2 * Dk + 8) * U * my.reshape(len(live), -1), HALF[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prefix_then_steps(dtype):
    """A prefix read at once, then its states stepped token by token, gives what reading all of it at once gives."""
    H, D, T, P = 2, 64, 140, 129
    q, k, v, dy, h, dhT = _inputs(8, T, 1, H, D, D, dtype)
    dec = [0.95, 0.995]
    whole = LinearAttention([0, T], T, H, D, D, dec, dtype, device=DEV)
    y, hT = whole.forward(q, k, v, h)
    part = LinearAttention([0, P], P, H, D, D, dec, dtype, device=DEV)
    yp, hp = part.forward(q[:P], k[:P], v[:P], h)
    st = AttentionState(1, H, D, D, dec, dtype, device=DEV)
    st.state.copy_(hp)
    ys = [yp.clone()] + [st.step(q[t:t + 1], k[t:t + 1], v[t:t + 1]).clone() for t in range(P, T)]
    torch.cuda.synchronize()
    check(np.array([0, T]), q, k, v, dy, h, dhT, dec, whole.scale, False, dtype,
          (torch.cat(ys), st.state, *whole.backward(q, k, v, dy, h, dhT)))
    grads = whole.backward(q, k, v, dy, h, dhT)
    check(np.array([0, T]), q, k, v, dy, h, dhT, dec, whole.scale, False, dtype, (y, hT, *grads))
