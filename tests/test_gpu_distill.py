"""GPU parity of the distillation loss (mdl_distill) against the float64 oracle.

Tolerances, with u = 2^-24: an exponential of x = (z - max) / tau has the rounding of the difference, of 1 / tau and of
their product in its argument, 3 |x| u, the hardware exp2's 1 ulp and its correction, 4 u, and with bfloat16 logits the
rounded product with log2 e, |x| u more. A sum takes at most S = 160 additions in a row (128 elements a lane, 6 exchanges,
16 waves, 10 spare). With q-averages written <.>:
    ln L is off by <4 |x|> u + (S + 4) u + 4 u |ln L|,  ln T alike, and a class's term by 6 u of its magnitude;
    q is off by q (4 |x| + <4 |x|> + S + 12) u, p alike; the gradient adds both, and a half step of its type."""

import numpy as np
import pytest
import torch

from fp_bounds import U
from oracle import sequence as oseq

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
S = 160
TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": U, "bf16": 2.0 ** -8}

if torch.cuda.is_available():
    import directional_mdlstm_handwriting_amd as M
    from directional_mdlstm_handwriting_amd.layer import TopKDistill


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def make(seed, N, V, k, dtype, t_dtype="f32"):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(N, V, generator=g) * 3
    t, ids = torch.topk(z + torch.randn(N, V, generator=g), k, dim=1)
    w = torch.rand(N, generator=g) + 0.5
    return z.to(TDT[dtype]).to(DEV), ids.to(torch.int32).to(DEV), t.to(TDT[t_dtype]).to(DEV), w.to(DEV)


def check(z, ids, t, w, tau, loss, dz, dtype):
    Z, I, T = _np(z), ids.cpu().numpy(), _np(t)
    W = np.ones(len(Z)) if w is None else _np(w)
    ref_l, ref_d = oseq.distill(Z, I, T, W, tau)
    got_l = _np(loss)
    got_d = None if dz is None else _np(dz)
    for n in range(len(Z)):
        if np.isnan(ref_l[n]):
            assert np.isnan(got_l[n]), n
            assert got_d is None or not got_d[n].any() or np.isnan(ref_d[n]).any(), n
            continue
        keep = I[n] >= 0
        if not keep.any() or W[n] == 0:
            assert got_l[n] == 0 and (got_d is None or not got_d[n].any()), n
            continue
        if np.isinf(ref_l[n]):
            assert got_l[n] == ref_l[n], n
        x = np.abs(Z[n] - Z[n].max()) / tau
        q = np.exp(-x)
        L = q.sum()
        q = q / L
        finite = q > 0
        mq = 4 * (q[finite] * x[finite]).sum()
        d = np.abs(T[n][keep] - T[n][keep].max()) / tau
        e = np.exp(-d)
        Tt = e.sum()
        p = e / Tt
        live = p > 0
        mp = 4 * (p[live] * d[live]).sum()
        if np.isfinite(ref_l[n]):
            mag = (p[live] * (d[live] + x[I[n][keep][live]])).sum()
            tol = (6 * mag + mq + mp + 2 * S + 16 + 4 * abs(np.log(L)) + 4 * abs(np.log(Tt))) * U
            scale = abs(W[n]) * tau * tau
            assert abs(got_l[n] - ref_l[n]) <= scale * tol + 4 * U * abs(ref_l[n]), (n, got_l[n], ref_l[n])
        if got_d is None:
            continue
        xx = np.where(finite, x, 0)
        tol = q * (5 * xx + mq + S + 12) * U
        for j, i in enumerate(I[n]):
            if i >= 0 and np.isfinite(T[n][j]):
                pj = np.exp((T[n][j] - T[n][keep].max()) / tau) / Tt
                tol[i] += pj * (4 * abs(T[n][j] - T[n][keep].max()) / tau + mp + S + 12) * U
        tol = abs(W[n]) * tau * tol
        bad = ~(np.abs(got_d[n] - ref_d[n]) <= tol + HALF[dtype] * (np.abs(ref_d[n]) + tol) + 1e-36)
        assert not bad.any(), (n, int(bad.sum()), int(np.flatnonzero(bad)[0]))


def run(z, ids, t, w, tau, dtype):
    N, V = z.shape
    print(f"[gpu] distill N={N} V={V} k={ids.shape[1]} {dtype}", flush=True)
    td = TopKDistill(N, V, ids.shape[1], dtype, tau, device=DEV)
    td.loss.fill_(7.0)
    td.dz.fill_(float("nan"))
    loss, dz = td.run(z, ids, t, w)
    torch.cuda.synchronize()
    check(z, ids, t, w, tau, loss, dz, dtype)
    return td, loss, dz


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 3, 4, 5, 7, 8, 9, 15, 33, 64, 65, 80, 127, 128, 129, 256, 257, 300, 511, 512, 513, 1000,
                               1024, 1025, 2048, 2049, 4097, 8192, 8193, 16384, 16385, 32000, 32769, 40001, 65537, 70001,
                               131072, 140003])
def test_class_counts(V, dtype):
    N = 35 if V <= 600 else 3
    z, ids, t, w = make(V, N, V, min(V, 7), dtype)
    run(z, ids, t, w, 2.0, dtype)


@pytest.mark.parametrize("k", [1, 2, 63, 64, 65, 300, 1024])
def test_kept_counts(k):
    for V, dtype in ((1024, "f32"), (5003, "bf16")):
        z, ids, t, w = make(k, 6, V, k, dtype)
        run(z, ids, t, None, 0.7, dtype)
    z, ids, t, w = make(k, 40, max(k, 2), k, "f32", "bf16")     # every class kept, or all but one
    run(z, ids, t, w, 1.0, "f32")


@pytest.mark.parametrize("V,dtype", [(128, "bf16"), (256, "bf16"), (512, "bf16"), (1024, "bf16"), (128, "f32"), (512, "f32")])
def test_every_class_kept(V, dtype):
    """As many kept classes as there are: the most LDS that a workgroup's rows can ask for."""
    z, ids, t, w = make(V, 70, V, V, dtype)
    run(z, ids, t, w, 1.3, dtype)


def test_more_than_2_31_elements():
    """Rows past 2^31 elements: the last rows' results are those of a small call on them alone."""
    N, V, k = 36000, 60001, 4
    g = torch.Generator(device=DEV).manual_seed(3)
    print(f"[gpu] distill N={N} V={V}", flush=True)
    z = torch.empty(N, V, dtype=torch.bfloat16, device=DEV)
    for a in range(0, N, 4000):
        z[a:a + 4000] = torch.randn(4000, V, generator=g, device=DEV, dtype=torch.bfloat16)
    ids = torch.randint(0, V, (N, k), generator=g, device=DEV, dtype=torch.int32)
    t = torch.randn(N, k, generator=g, device=DEV)
    loss, dz = TopKDistill(N, V, k, "bf16", 1.5, device=DEV).run(z, ids, t)
    part = slice(N - 5, N)
    l2, d2 = TopKDistill(5, V, k, "bf16", 1.5, device=DEV).run(z[part], ids[part].contiguous(), t[part].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(loss[part], l2) and torch.equal(dz[part], d2)
    check(z[part], ids[part], t[part], None, 1.5, l2, d2, "bf16")


def test_more_rows_than_one_launch_takes():
    N = (1 << 28) + 3
    print(f"[gpu] distill N={N} V=2", flush=True)
    z = torch.randn(N, 2, device=DEV, dtype=torch.bfloat16)
    ids = torch.ones(N, 1, dtype=torch.int32, device=DEV)
    t = torch.zeros(N, 1, device=DEV)
    loss, dz = TopKDistill(N, 2, 1, "bf16", 1.0, device=DEV).run(z, ids, t)
    torch.cuda.synchronize()
    for s in (slice(0, 5), slice((1 << 28) - 4, N)):
        check(z[s], ids[s], t[s], None, 1.0, loss[s], dz[s], "bf16")


@pytest.mark.parametrize("V", [6, 100, 500, 3001, 90001])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_that_count_for_nothing_and_masked_classes(V, dtype):
    z, ids, t, w = make(11, 12, V, 5, dtype)
    ids[1, 2:] = -1                        # two of five slots kept
    ids[2] = -1                            # nothing kept
    w[3] = 0.0                             # a padded frame, holding NaN
    z[3] = float("nan")
    ids[4, 1] = V                          # no such class
    ids[5, 0] = -7
    t[6, 0] = float("-inf")                # a kept class of no weight
    ids[7, 3] = ids[7, 0]                  # a class named twice, and five times
    ids[8] = ids[8, 0]
    free = [c for c in range(V) if c not in ids[9].tolist()][:1]
    z[9, free] = float("-inf")             # masked classes of the student
    z[10, ids[10, 2].item()] = float("-inf")     # one that the teacher keeps: infinite loss, finite gradient
    t[11] = t[11, 0]                       # ties
    _, loss, dz = run(z, ids, t, w, 1.5, dtype)
    assert torch.isnan(loss[4:6]).all() and not dz[4:6].any() and not dz[2:4].any()
    assert loss[10] == float("inf") and torch.isfinite(dz[10].float()).all()
    assert torch.isfinite(loss[[0, 1, 2, 3, 6, 7, 8, 9, 11]]).all()


def test_nan_stays_in_its_row():
    for V, dtype in ((60, "f32"), (3000, "bf16"), (80000, "f32")):
        z, ids, t, w = make(12, 5, V, 4, dtype)
        _, l0, d0 = run(z, ids, t, w, 1.0, dtype)
        l0, d0 = l0.clone(), d0.clone()
        z[2, V - 1] = float("nan")
        td = TopKDistill(5, V, 4, dtype, 1.0, device=DEV)
        loss, dz = td.run(z, ids, t, w)
        rows = [0, 1, 3, 4]
        assert torch.equal(loss[rows], l0[rows]) and torch.equal(dz[rows], d0[rows])
        assert torch.isnan(loss[2]) and torch.isnan(dz[2].float()).all()


def test_large_logits_and_sharp_temperatures():
    for dtype in ("f32", "bf16"):
        z, ids, t, w = make(13, 6, 900, 6, dtype)
        run((z * 100).contiguous(), ids, (t * 100).contiguous(), w, 1.0, dtype)
        run(z, ids, t, w, 0.05, dtype)
        run(z, ids, t, w, 50.0, dtype)


@pytest.mark.parametrize("V", [5, 77, 1001, 20011, 90003])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_in_place_and_loss_alone(V, dtype):
    N, k = 9, 5
    z, ids, t, w = make(14, N, V, k, dtype)
    dt = 1 if dtype == "bf16" else 0
    td, loss, dz = run(z, ids, t, w, 2.0, dtype)
    wide = torch.full((N, V + 5), 3.0, dtype=TDT[dtype], device=DEV)
    mid = wide[:, 1:V + 1]
    mid.copy_(z)
    l2 = torch.empty_like(loss)
    M.mdl_distill(N, V, k, dt, mid, wide.stride(0), ids, t, 0, w, 2.0, l2, None, 0)
    assert torch.equal(l2, loss) and torch.equal(mid, z)
    l2.fill_(0)
    M.mdl_distill(N, V, k, dt, mid, wide.stride(0), ids, t, 0, w, 2.0, l2, mid, wide.stride(0))
    torch.cuda.synchronize()
    assert torch.equal(l2, loss) and torch.equal(mid, dz)
    assert (wide[:, 0] == 3).all() and (wide[:, V + 1:] == 3).all()
    l3, none = td.run(z, ids, t, w, want_dz=False)
    assert none is None and torch.equal(l3, l2)


def test_gradient_against_differences():
    """Loss differences in the direction of a few single logits, in steps that fp32 losses resolve."""
    N, V, k, h = 4, 50, 6, 0.05
    z, ids, t, w = make(15, N, V, k, "f32")
    td = TopKDistill(N, V, k, "f32", 2.0, device=DEV)
    _, dz = td.run(z, ids, t, w)
    dz = dz.clone()
    for c in (0, 7, 49, ids[0, 0].item()):
        hi, lo = z.clone(), z.clone()
        hi[:, c] += h
        lo[:, c] -= h
        up = td.run(hi, ids, t, w, want_dz=False)[0].clone()
        diff = (up - td.run(lo, ids, t, w, want_dz=False)[0]) / (2 * h)
        # third derivatives of the log-sum are below 1 / tau^3 times w tau^2 < 1.5 tau^2: h^2 / 6 times that, and the
        # losses' own roundings of about 400 u over 2 h
        assert ((diff - dz[:, c]).abs() <= h * h / 6 * 0.75 + 400 * U * 6 / h).all()


def test_captured_replays():
    N, V, k = 30, 3000, 16
    sets = [make(50 + i, N, V, k, "bf16") for i in range(2)]
    held, eager = (TopKDistill(N, V, k, "bf16", 2.0, device=DEV) for _ in range(2))
    buf = [x.clone() for x in sets[0]]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        held.run(*buf)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = held.run(*buf)
    for rep in range(4):
        for b, s in zip(buf, sets[rep % 2]):
            b.copy_(s)
        gr.replay()
        ref = eager.run(*sets[rep % 2])
        torch.cuda.synchronize()
        assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
