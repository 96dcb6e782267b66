"""Linear attention where the other tests do not look: tiles of four and more blocks of 32 tokens for heads of every padded
size, rows of whole 16-byte chunks or not; inputs above zero, so that an output is the sum of its terms' magnitudes and a
wrong power of the decay shows; decays below 0 and above 1; gradients along their own direction.

The reference walks the tokens in float64 on the device. Beside each state R it keeps E, the same sum with each term
weighted by its distance in tokens: an output a^T R is off by at most
    u ((4 D + 96) a^T R + (4 |ln |d|| + 2) a^T E)   on magnitudes,   u = 2^-24
(4 D + 96: sums over a head's channels and a block's 32 tokens, and the factors within a block. Per token of distance: a
block's factor d^32 is off by 3 u |ln d| for each of its 32 tokens, in the rounded logarithm and the exponent's product, and
by 2 u, its product and the sum over 32 tokens by 34 roundings; a tile's end as a block's.) bfloat16: r = 2^-8 + 2^-15 more for
y and the gradients, as in the other tests, and each output's own rounding.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
TINY = 1e-30

if torch.cuda.is_available():
    from directional_mdlstm_handwriting_amd.layer import LinearAttention

TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": U, "bf16": 2.0 ** -8}
ROUND = {"f32": 0.0, "bf16": 2.0 ** -8 + 2.0 ** -15}


def walk(tokens, a, b, c, d, R, post, scale):
    """(out, its E, last R, its E) of R_t = b_t c_t^T + d R_{t-1}, out_t = a_t^T R_t over `tokens`; [T][H][.] float64."""
    H = a.shape[1]
    d = d.reshape(H, 1, 1)
    out, dist = torch.zeros_like(c), torch.zeros_like(c)
    E = torch.zeros_like(R)
    for t in tokens:
        if post:                   # the state of the token before
            E = d * (E + R)
            R = d * R + scale * b[t].unsqueeze(2) * c[t].unsqueeze(1)
        else:                      # the state's gradient: decayed behind the token
            R = R + scale * b[t].unsqueeze(2) * c[t].unsqueeze(1)
        out[t] = (a[t].unsqueeze(2) * R).sum(1)
        dist[t] = (a[t].unsqueeze(2) * E).sum(1)
        if not post:
            E = d * (E + R)
            R = d * R
    return out, dist, R, E


def reference(off, q, k, v, dy, d, scale, h0, dhT, reverse):
    """{name: (value, E)} of y, hT, dq, dk, dv, dh0."""
    S = len(off) - 1
    res = {n: [] for n in ("hT", "dh0")}
    out = {n: (torch.zeros_like(t), torch.zeros_like(t)) for n, t in (("y", v), ("dq", q), ("dk", k), ("dv", v))}
    for s in range(S):
        tok = list(range(int(off[s]), int(off[s + 1])))
        if reverse:
            tok.reverse()
        y, ey, R, E = walk(tok, q, k, v, d, h0[s], True, 1.0)
        dq, eq, _, _ = walk(tok, dy, v, k, d, h0[s].transpose(1, 2).contiguous(), True, 1.0)
        dv, ev, G, F = walk(tok[::-1], k, q, dy, d, dhT[s], False, scale)
        dk, ek, _, _ = walk(tok[::-1], v, dy, q, d, dhT[s].transpose(1, 2).contiguous(), False, scale)
        for n, (x, e), f in (("y", (y, ey), scale), ("dq", (dq, eq), scale), ("dv", (dv, ev), 1.0), ("dk", (dk, ek), 1.0)):
            out[n][0][tok], out[n][1][tok] = x[tok] * f, e[tok] * f
        res["hT"].append((R, E))
        res["dh0"].append((G, F))
    return {**out, **{n: (torch.stack([x for x, _ in p]), torch.stack([x for _, x in p])) for n, p in res.items()}}


def _compare(lens, H, Dk, Dv, decay, dtype, reverse, positive, seed):
    off = np.concatenate([[0], np.cumsum(lens)])
    T, S = int(off[-1]), len(lens)
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rn(*s, dt=TDT[dtype]):
        x = torch.randn(*s, generator=g, device=DEV)
        return ((x.abs() + 0.125) if positive else x).to(dt)

    p = rn(T, H * (2 * Dk + Dv))
    q, k, v = p[:, :H * Dk], p[:, H * Dk:2 * H * Dk], p[:, 2 * H * Dk:]
    dy = rn(T, H * Dv)
    h0, dhT = rn(S, H, Dk, Dv, dt=torch.float32), rn(S, H, Dk, Dv, dt=torch.float32)
    dec = torch.as_tensor(np.float32(decay), device=DEV)
    at = LinearAttention(off, T, H, Dk, Dv, dec, dtype, reverse=reverse, device=DEV)
    y, hT = at.forward(q, k, v, h0)
    got = dict(zip(("dq", "dk", "dv", "dh0"), at.backward(q, k, v, dy, h0, dhT)), y=y, hT=hT)
    torch.cuda.synchronize()
    w = [t.double().reshape(T, H, -1) for t in (q, k, v, dy)]
    d, scale = dec.double(), float(np.float32(at.scale))
    ref = reference(off, *w, d, scale, h0.double(), dhT.double(), reverse)
    mag = ref if positive and bool((d >= 0).all()) else reference(off, *(t.abs() for t in w), d.abs(), abs(scale), h0.double().abs(), dhT.double().abs(), reverse)
    kappa = 4 * torch.log(d.abs().clamp(min=1e-30)).abs().clamp(max=80) + 2
    for n, (x, _) in ref.items():
        m, e = mag[n]
        shape = (1, H, 1) if x.dim() == 3 else (1, H, 1, 1)
        r, half = (0.0, U) if n in ("hT", "dh0") else (ROUND[dtype], HALF[dtype])
        tol = r * m + U * ((4 * max(Dk, Dv) + 96) * m + kappa.reshape(shape) * e)
        err = (got[n].double().reshape(x.shape) - x).abs()
        lim = tol + half * (x.abs() + tol) + TINY
        assert bool((err <= lim).all()), f"{n}: {int((~(err <= lim)).sum())} of {err.numel()}, worst {float((err / lim).max()):.3g}"
    return at


DECAYS = 1 - 2.0 ** -np.arange(1.0, 10.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 64), (128, 64), (64, 128), (50, 50), (65, 63), (100, 100), (24, 128), (7, 9)])
def test_tiles_of_many_blocks(Dk, Dv, reverse, dtype):
    """96 heads and 900 tokens: tiles of 128 or 160 tokens, so that each buffer of a block is filled again and again."""
    H = 96
    print(f"[gpu] many blocks {Dk} {Dv} {reverse} {dtype}", flush=True)
    at = _compare([523, 377], H, Dk, Dv, DECAYS[np.arange(H) % len(DECAYS)], dtype, reverse, True, Dk + Dv)
    assert at.ws_bytes <= 2 * (900 // 96) * H * Dk * Dv * 4 + 32      # a state for each end of a tile of 96 tokens or more


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_sequences_above_zero(dtype):
    """Tiles of 320 tokens, 16 of them in a row: one power of the slowest decay too many at a tile's end is 2^-9 of what it
    brings, in fp32 many times the bound."""
    H = 40
    print(f"[gpu] long above zero {dtype}", flush=True)
    _compare([5000, 1, 2000], H, 8, 8, DECAYS[np.arange(H) % len(DECAYS)], dtype, False, True, 3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("decay", [-0.5, -0.97, -1.0, -0.0, -1e-30, 1.01, -1.01])
def test_decays_outside_zero_to_one(decay, reverse, dtype):
    """A decay tensor is taken as it is: the recurrence with a factor below 0 or above 1, over tiles and their ends."""
    print(f"[gpu] decay {decay} {reverse} {dtype}", flush=True)
    for positive in (False, True):
        _compare([301, 70, 1, 97], 1, 32, 48, [decay], dtype, reverse, positive, 5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_against_differences_along_themselves(dtype):
    """The loss sum(y w) + sum(hT u) moved along each gradient itself, where the change is the sum of the gradient's squares
    and no term cancels another: half a step of bfloat16 on the way and one at the end, twice each."""
    T, H, Dk, Dv, lens = 127, 2, 16, 24, [37, 90]
    off = np.concatenate([[0], np.cumsum(lens)])
    g = torch.Generator().manual_seed(9)
    q, k, v, w = (torch.randn(T, H * n, generator=g).to(TDT[dtype]).to(DEV) for n in (Dk, Dk, Dv, Dv))
    h0, u = (torch.randn(2, H, Dk, Dv, generator=g).to(DEV) for _ in range(2))
    dec = torch.tensor([0.9, 0.98], device=DEV)
    at = LinearAttention(off, T, H, Dk, Dv, dec, dtype, device=DEV)
    at.forward(q, k, v, h0)
    grads = at.backward(q, k, v, w, h0, u)
    torch.cuda.synchronize()
    base = [t.double().reshape(T, H, -1) for t in (q, k, v)] + [h0.double()]
    scale = float(np.float32(at.scale))

    def loss(q, k, v, h):
        total = 0.0
        for s in range(2):
            tok = range(int(off[s]), int(off[s + 1]))
            y, _, R, _ = walk(tok, q, k, v, dec.double(), h[s], True, 1.0)
            total += float((scale * y * w.double().reshape(T, H, -1)).sum() + (R * u[s].double()).sum())
        return total

    for i, G in enumerate(grads):
        e = G.double().reshape(base[i].shape)
        e = e / e.abs().max()
        # the loss is linear in each input: the difference is exact but for rounding
        diff = loss(*[b + 0.5 * e if j == i else b for j, b in enumerate(base)]) - \
            loss(*[b - 0.5 * e if j == i else b for j, b in enumerate(base)])
        want = float((G.double().reshape(e.shape) * e).sum())
        assert abs(diff - want) <= (4 * HALF[dtype] + 3000 * U) * want, i
