"""GPU parity of the norms before and after a block (mdl_blocknorm_forward / _backward) against the float64 oracle.

The tolerances are the rounding bounds of the formulas themselves (fp_bounds.Err), with a row's sums taking at most 64
additions in a row (32 elements a lane at most, 6 exchanges between lanes and 16 waves), and a column's sums the rows a
workgroup adds one after another plus the workgroups added one after another (a quarter of at most 1024), plus a half
step of the output's type."""

import numpy as np
import pytest
import torch

from fp_bounds import U, Err, assert_within
from oracle import sequence as oseq

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": U, "bf16": 2.0 ** -8}
NAMES = ("r", "v", "dx", "dz", "du", "dw_post", "dscale", "dw_pre")

if torch.cuda.is_available():
    import directional_mdlstm_handwriting_amd as M
    from directional_mdlstm_handwriting_amd.layer import BlockNorm


def _np(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def bounds(x, z, u, wp, sc, wn, dr, dv, eps, plain_exp, N):
    D = x.shape[1]
    row = 64
    col = N // 1024 + 1 + 32 + 256 + 4
    out = {}
    r = Err(x)
    if z is not None:
        z = Err(z)
        sig = ((z * z).sum(1, row, True) * (1.0 / D) + eps).rsqrt()
        zh = z * sig
        g, gc = (Err(np.ones_like(x)), Err(np.zeros_like(x))) if u is None else Err(u).sigmoid(plain_exp)
        cs = Err(np.ones(D) if sc is None else sc) * (np.ones(D) if wp is None else wp)
        r = cs * g * zh + x
        out["r"] = r
    if wn is not None:
        rho = ((r * r).sum(1, row, True) * (1.0 / D) + eps).rsqrt()
        rh = r * rho
        out["v"] = rh * wn
    if dr is None and dv is None:
        return out
    d = Err(np.zeros_like(x) if dr is None else dr)
    if wn is not None:
        t = Err(dv) * wn
        m = (t * r).sum(1, row, True) * rho * (1.0 / D)
        d = rho * (t - rh * m) + d
        out["dw_pre"] = (rh * dv).sum(0, col)
    out["dx"] = d
    if z is not None:
        k = d * g
        q = (k * zh).sum(0, col)
        p = k * cs
        m = (p * zh).sum(1, row, True) * (1.0 / D)
        out["dz"] = sig * (p - zh * m)
        out["du"] = p * zh * gc
        out["dw_post"] = q * (np.ones(D) if sc is None else sc)
        out["dscale"] = q * (np.ones(D) if wp is None else wp)
    return out


def make(seed, N, D, dtype, parts="all"):
    g = torch.Generator().manual_seed(seed)

    def rn(*s, m=0.0, k=1.0, dt=None):
        return (torch.randn(*s, generator=g) * k + m).to(dt or TDT[dtype]).to(DEV)

    t = dict(x=rn(N, D, k=2.0), z=rn(N, D), u=rn(N, D, k=1.5), w_post=rn(D, m=1.0, k=0.2, dt=torch.float32),
             scale=rn(D, m=0.3, k=0.2, dt=torch.float32), w_pre=rn(D, m=1.0, k=0.2, dt=torch.float32), dr=rn(N, D),
             dv=rn(N, D))
    drop = {"all": (), "no_gate": ("u",), "no_scale": ("scale",), "no_w_post": ("w_post",),
            "pre_only": ("z", "u", "w_post", "scale"), "post_only": ("w_pre", "dv"), "no_dr": ("dr",),
            "plain_post": ("u", "w_post", "scale", "w_pre", "dv")}[parts]
    return {k: None if k in drop else v for k, v in t.items()}


INPUTS = ("x", "z", "u", "w_post", "scale", "w_pre")


def run(bn, t):
    for b in bn._bufs.values():
        b.fill_(float("nan"))
    bn.ws.fill_(0xFF)
    fw = bn.forward(*(t[k] for k in INPUTS))
    bw = bn.backward(*(t[k] for k in INPUTS), t["dr"], t["dv"])
    torch.cuda.synchronize()
    return dict(zip(NAMES, (*fw, *bw)))


def check(t, got, eps, dtype):
    a = {k: _np(v) for k, v in t.items()}
    N = a["x"].shape[0]
    rr, rv = oseq.blocknorm_forward(*(a[k] for k in INPUTS), eps)
    ref = oseq.blocknorm_backward(*(a[k] for k in INPUTS), a["dr"], a["dv"], eps)
    ref.update(r=rr, v=rv)
    b = bounds(*(a[k] for k in INPUTS), a["dr"], a["dv"], eps, dtype == "bf16", N)
    for k in NAMES:
        if got[k] is None:
            assert ref[k] is None, k
            continue
        if k == "r" and t["z"] is None:
            assert got[k] is t["x"]
            continue
        half = U if k in ("dw_post", "dscale", "dw_pre") else HALF[dtype]
        assert_within(k, _np(got[k]), Err(ref[k], b[k].e), half)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 2, 3, 4, 5, 7, 8, 9, 16, 31, 32, 33, 50, 64, 100, 127, 128, 130, 255, 256, 257, 500,
                               512, 513, 1000, 1024, 1030, 2048, 2050, 4096, 5000, 8192, 8200, 16384])
def test_row_lengths(D, dtype):
    for N in (1, 5, 33):
        print(f"[gpu] norm N={N} D={D} {dtype}", flush=True)
        t = make(D + N, N, D, dtype)
        check(t, run(BlockNorm(N, D, dtype, device=DEV), t), 1e-6, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D", [(5000, 16), (20011, 50), (3001, 300), (1500, 2048)])
def test_many_rows(N, D, dtype):
    """More rows than the backward's workgroups hold at once."""
    print(f"[gpu] norm N={N} D={D} {dtype}", flush=True)
    t = make(N, N, D, dtype)
    bn = BlockNorm(N, D, dtype, eps=1e-5, device=DEV)
    got = {k: v.clone() for k, v in run(bn, t).items()}
    check(t, got, 1e-5, dtype)
    again = run(bn, t)
    for k in NAMES:
        assert torch.equal(got[k], again[k]), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("parts", ["no_gate", "no_scale", "no_w_post", "pre_only", "post_only", "no_dr", "plain_post"])
def test_parts(parts, dtype):
    for D in (24, 700):
        print(f"[gpu] norm {parts} D={D} {dtype}", flush=True)
        t = make(7, 13, D, dtype, parts)
        check(t, run(BlockNorm(13, D, dtype, device=DEV), t), 1e-6, dtype)


def test_no_rows():
    t = make(1, 0, 20, "f32")
    got = run(BlockNorm(0, 20, "f32", device=DEV), t)
    for k in ("dw_post", "dscale", "dw_pre"):
        assert not got[k].any()


def test_zero_rows_and_nan_rows():
    for D, dtype in ((40, "f32"), (640, "bf16")):
        t = make(2, 9, D, dtype)
        t["x"][3] = 0
        t["z"][3] = 0
        got = {k: v.clone() for k, v in run(BlockNorm(9, D, dtype, device=DEV), t).items()}
        check(t, got, 1e-6, dtype)
        assert not got["r"][3].any() and not got["v"][3].any()
        t["z"][5, D // 2] = float("nan")
        t["u"][6, 0] = float("inf")
        t["u"][7] = float("-inf")
        bad = run(BlockNorm(9, D, dtype, device=DEV), t)
        rows = [0, 1, 2, 3, 4, 8]
        for k in NAMES[:5]:
            assert torch.equal(bad[k][rows], got[k][rows]), k
            assert torch.isnan(bad[k][5].float()).any(), k
            assert not torch.isnan(bad[k][6:8].float()).any(), k
        assert torch.equal(bad["r"][7], t["x"][7])          # a closed gate leaves the residual as it was


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [6, 37, 77, 600, 2101])
def test_strides_alignment_and_in_place(D, dtype):
    N = 21
    dt = 1 if dtype == "bf16" else 0
    t = make(3, N, D, dtype)
    bn = BlockNorm(N, D, dtype, device=DEV)
    ref = {k: v.clone() for k, v in run(bn, t).items()}
    wide = torch.full((N, 3 * D + 2), 9.0, dtype=TDT[dtype], device=DEV)
    w2 = wide.clone()
    x, z, u = (wide[:, 1 + i * D:1 + (i + 1) * D] for i in range(3))
    r, v, _ = (w2[:, 1 + i * D:1 + (i + 1) * D] for i in range(3))
    for a, b in ((x, t["x"]), (z, t["z"]), (u, t["u"])):
        a.copy_(b)
    ld = wide.stride(0)
    w = (t["w_post"], t["scale"], t["w_pre"])
    M.mdl_blocknorm_forward(N, D, dt, x, ld, z, ld, u, ld, *w, 1e-6, r, v, ld)
    torch.cuda.synchronize()
    assert torch.equal(r, ref["r"]) and torch.equal(v, ref["v"])
    assert (w2[:, 0] == 9).all() and (w2[:, 1 + 2 * D:] == 9).all()
    # gradients over the inputs: dx over dr, dz over z, du over u
    w2[:, 1:1 + D].copy_(t["dr"])
    w2[:, 1 + D:1 + 2 * D].copy_(t["dv"])
    big = torch.full((N, 5 * D + 3), 9.0, dtype=TDT[dtype], device=DEV)
    b = [big[:, 1 + i * D:1 + (i + 1) * D] for i in range(5)]
    for a, k in zip(b, ("x", "z", "u", "dr", "dv")):
        a.copy_(t[k])
    ld = big.stride(0)
    gw = [torch.empty(D, device=DEV) for _ in range(3)]
    M.mdl_blocknorm_backward(N, D, dt, b[0], ld, b[1], ld, b[2], ld, *w, 1e-6, b[3], b[4], ld, b[3], b[1], b[2], ld, *gw,
                             bn.ws, bn.ws_bytes)
    torch.cuda.synchronize()
    for got, k in zip((b[3], b[1], b[2], *gw), ("dx", "dz", "du", "dw_post", "dscale", "dw_pre")):
        assert torch.equal(got, ref[k]), k
    assert (big[:, 0] == 9).all() and (big[:, 1 + 5 * D:] == 9).all()
    # the forward over its input: r over x, and v over z
    M.mdl_blocknorm_forward(N, D, dt, x, wide.stride(0), z, wide.stride(0), u, wide.stride(0), *w, 1e-6, x, z,
                            wide.stride(0))
    torch.cuda.synchronize()
    assert torch.equal(x, ref["r"]) and torch.equal(z, ref["v"])


def test_more_than_2_31_elements():
    """Rows past 2^31 elements: the last rows' results are those of a small call on them alone."""
    N, D = 1100003, 2000
    print(f"[gpu] norm N={N} D={D}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(4)
    t = make(9, 4, D, "bf16")
    for k in ("x", "z", "u", "dr", "dv"):
        t[k] = torch.randn(N, D, generator=g, device=DEV, dtype=torch.bfloat16)
    bn = BlockNorm(N, D, "bf16", device=DEV)
    got = dict(zip(NAMES, (*bn.forward(*(t[k] for k in INPUTS)),
                           *bn.backward(*(t[k] for k in INPUTS), t["dr"], t["dv"]))))
    small = {k: (v[N - 7:].contiguous() if v.dim() == 2 else v) for k, v in t.items()}
    ref = run(BlockNorm(7, D, "bf16", device=DEV), small)
    for k in NAMES[:5]:
        assert torch.equal(got[k][N - 7:], ref[k]), k


def test_more_rows_than_one_launch_takes():
    N = (1 << 28) + 5
    print(f"[gpu] norm N={N} D=1", flush=True)
    x = torch.randn(N, 1, device=DEV, dtype=torch.bfloat16)
    w = torch.full((1,), 0.5, device=DEV)
    _, v = BlockNorm(N, 1, "bf16", eps=0.25, device=DEV).forward(x, w_pre=w)
    torch.cuda.synchronize()
    for s in (slice(0, 7), slice((1 << 28) - 3, N)):
        ref = (x[s].double() * 0.5 / torch.sqrt(x[s].double() ** 2 + 0.25)).cpu().numpy()
        assert_within("v", _np(v[s]), Err(ref, 16 * U * np.abs(ref)), 2.0 ** -8)


def test_captured_backward_replays():
    N, D = 700, 96
    sets = [make(40 + i, N, D, "bf16") for i in range(2)]
    eager, held = BlockNorm(N, D, "bf16", device=DEV), BlockNorm(N, D, "bf16", device=DEV)
    buf = {k: torch.zeros_like(v) for k, v in sets[0].items()}
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        held.forward(*(buf[k] for k in INPUTS))
        held.backward(*(buf[k] for k in INPUTS), buf["dr"], buf["dv"])
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        fw = held.forward(*(buf[k] for k in INPUTS))
        out = dict(zip(NAMES, (*fw, *held.backward(*(buf[k] for k in INPUTS), buf["dr"], buf["dv"]))))
    for rep in range(4):
        s = sets[rep % 2]
        for k in buf:
            buf[k].copy_(s[k])
        gr.replay()
        ref = run(eager, s)
        for k in NAMES:
            assert torch.equal(out[k], ref[k]), (rep, k)
