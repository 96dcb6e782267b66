"""GPU parity of the gated linear recurrence (mdl_scan_forward / _backward / _step) against the float64 oracle.

Tolerances are computed, not chosen: beside each value the same recurrence is run on magnitudes, and an error term
follows it that takes in c u times the magnitude at every token (u = 2^-24):

    H_t = f H_{t-1} + (1 - f) |g|,   E_t = f E_{t-1} + c u H_t
    L_t = o |dy| + f_{t+1} L_{t+1},  F_t = f_{t+1} F_{t+1} + c u L_t

c counts the roundings of u a token can add to its terms: the sigmoid of the gate 7 (exp2 and reciprocal of the
hardware 1 ulp = 2 u each, the argument's carried product 1, the sum 1, the product 1), the input product 1, the state's
multiply-add 1, and the map that joins tiles the same again (product of gates and multiply-add, 8 + 1): c = 18. With bfloat16 inputs the exp2
argument is the plain rounded product, wrong by up to |z| u more, where u |z| is below 2^-18: c = 18 + |z|max. A bfloat16
output adds its half step, 2^-8 of the value. The gradients' tolerances are the product rule over these.
"""

import numpy as np
import pytest
import torch

from oracle import sequence as oseq

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
TINY = 1e-36    # gates below the smallest normal fp32 number flush to zero

if torch.cuda.is_available():
    import directional_mdlstm_handwriting_amd as M
    from directional_mdlstm_handwriting_amd.layer import DeviceLayout, ScanState, SequenceScan

TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": U, "bf16": 2.0 ** -8}


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _inputs(seed, T, S, D, dtype, gate=True, h0=True, shift=1.0):
    """Values exactly representable in the tensors' type, on the device, as column blocks of one matrix."""
    g = torch.Generator().manual_seed(seed)
    p = (torch.randn(T, 3 * D, generator=g) * 1.5)
    p[:, :D] += shift
    p = p.to(TDT[dtype]).to(DEV)
    zf, gg, zo = p[:, :D], p[:, D:2 * D], (p[:, 2 * D:] if gate else None)
    dy = torch.randn(T, D, generator=g).to(TDT[dtype]).to(DEV)
    h = torch.randn(S, D, generator=g).to(DEV) if h0 else None
    dhT = torch.randn(S, D, generator=g).to(DEV)
    return zf, gg, zo, h, dy, dhT


def _close(name, got, ref, tol, half):
    err = np.abs(_np(got) - ref)
    bad = err > tol + half * (np.abs(ref) + tol) + TINY
    assert not bad.any(), f"{name}: {int(bad.sum())} of {err.size}, worst {np.nanmax(err / (tol + half * np.abs(ref) + TINY)):.3g} of the tolerance"
    assert np.isfinite(_np(got)).all(), name


def check(off, zf, g, zo, h0, dy, dhT, reverse, dtype, got):
    """got: (y, hT, dzf, dg, dzo, dh0) over the rows of the sequences."""
    Z, G, DY = _np(zf), _np(g), _np(dy)
    O = None if zo is None else _np(zo)
    H0 = None if h0 is None else _np(h0)
    DT = _np(dhT)
    lo, hi = off[0], off[-1]
    sl = slice(lo, hi)
    c = 18 + (max(np.abs(Z[sl]).max(initial=0), 0 if O is None else np.abs(O[sl]).max(initial=0)) if dtype == "bf16" else 0)
    y, hT, h = oseq.scan_forward(off, Z, G, O, H0, reverse)
    grads = oseq.scan_backward(off, Z, G, O, DY, H0, DT, reverse)
    f, fc = oseq.sigmoid(Z), oseq.sigmoid(-Z)
    o, oc = (np.ones_like(Z), np.zeros_like(Z)) if O is None else (oseq.sigmoid(O), oseq.sigmoid(-O))
    S, D = len(off) - 1, Z.shape[1]
    H, E, PH, PE, L, F, P = (np.zeros_like(Z) for _ in range(7))
    HT, ET, L0, F0 = np.zeros((S, D)), np.zeros((S, D)), np.zeros((S, D)), np.zeros((S, D))
    for s in range(S):
        toks = list(range(off[s], off[s + 1]))
        toks = toks[::-1] if reverse else toks
        a, e = (np.zeros(D) if H0 is None else np.abs(H0[s])), np.zeros(D)
        q = np.zeros(D) if H0 is None else H0[s]
        for t in toks:
            PH[t], PE[t], P[t] = a, e, q
            a = f[t] * a + fc[t] * np.abs(G[t])
            e = f[t] * e + c * U * a
            H[t], E[t], q = a, e, h[t]
        HT[s], ET[s] = a, e
        a, e = np.abs(DT[s]), np.zeros(D)
        for t in toks[::-1]:
            L[t] = o[t] * np.abs(DY[t]) + a
            F[t] = e + c * U * L[t]
            a, e = f[t] * L[t], f[t] * F[t]
        L0[s], F0[s] = a, e
    half = HALF[dtype]
    k = 4 * c * U    # the factors' own roundings: at most three sigmoids and four products
    _close("y", got[0][sl], y[sl], (o * E + k * o * H)[sl], half)
    _close("hT", got[1], hT, ET + k * HT, U)
    mid = np.abs(P - G)
    w = PH + np.abs(G)
    _close("dzf", got[2][sl], grads["dzf"][sl], (f * fc * (mid * F + (PE + k * w) * (L + F)))[sl], half)
    _close("dg", got[3][sl], grads["dg"][sl], (fc * (F + k * L))[sl], half)
    if zo is not None:
        _close("dzo", got[4][sl], grads["dzo"][sl], (np.abs(DY) * o * oc * (E + k * H))[sl], half)
    if got[5] is not None:
        _close("dh0", got[5], grads["dh0"], F0 + k * L0, U)


def run(off, T, D, dtype, reverse=False, gate=True, h0=True, seed=0, shift=1.0):
    S = len(off) - 1
    print(f"[gpu] scan T={T} S={S} D={D} {dtype} reverse={reverse} gate={gate} h0={h0}", flush=True)
    zf, g, zo, h, dy, dhT = _inputs(seed, T, S, D, dtype, gate, h0, shift)
    sc = SequenceScan(off, T, D, dtype, reverse=reverse, device=DEV)
    sc.ws.fill_(0xA5)
    sc.y.fill_(7.0)
    sc.hT.fill_(float("nan"))
    y, hT = sc.forward(zf, g, zo, h)
    sc.dzf, sc.dg = torch.full_like(sc.y, 7.0), torch.full_like(sc.y, 7.0)
    sc.dzo = torch.full_like(sc.y, 7.0)
    sc.dh0 = torch.full_like(sc.hT, float("nan"))
    out = (y, hT, *sc.backward(zf, g, zo, dy, h, dhT))
    torch.cuda.synchronize()
    check(off, zf, g, zo, h, dy, dhT, reverse, dtype, out)
    for t in (out[0], out[2], out[3]):      # rows in no sequence: as they were
        assert (t[:off[0]] == 7).all() and (t[off[-1]:] == 7).all()
    return sc, out


def _off(lens, first=0):
    return np.concatenate([[first], first + np.cumsum(lens)]).astype(np.int64)


LENGTHS = {
    "one": [1],
    "empty_between": [0, 1, 0, 0, 3, 0],
    "tile_edges": [64, 63, 65, 1, 128, 127, 0, 129],
    "longer_tiles": [255, 257, 1, 512],
    "singles": [1] * 150,
    "long": [3000, 2],
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("lens", sorted(LENGTHS))
def test_lengths(lens, reverse, dtype):
    off = _off(LENGTHS[lens])
    run(off, int(off[-1]), 32, dtype, reverse)
    run(off, int(off[-1]), 5, dtype, reverse)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 2, 3, 4, 7, 8, 9, 16, 17, 31, 33, 50, 64, 65, 100, 127, 129, 200, 300])
def test_channels(D, dtype):
    off = _off([40, 0, 17, 300])
    run(off, int(off[-1]), D, dtype, reverse=D % 2 == 1)


@pytest.mark.parametrize("gate,h0", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_gate_or_initial_state(gate, h0, dtype):
    off = _off([100, 1, 200])
    run(off, int(off[-1]), 24, dtype, gate=gate, h0=h0)


@pytest.mark.parametrize("reverse", [False, True])
def test_rows_in_no_sequence(reverse):
    """A gap before the first sequence and a padded end longer than a tile, filled with NaN: left as they were."""
    for D, dtype in ((16, "f32"), (40, "bf16")):
        off = _off([30, 0, 90], first=70)
        T = 600
        zf, g, zo, h, dy, dhT = _inputs(3, T, 3, D, dtype)
        for t in (zf, g, zo, dy):
            t[:70] = float("nan")
            t[off[-1]:] = float("nan")
        sc = SequenceScan(off, T, D, dtype, reverse=reverse, device=DEV)
        y, hT = sc.forward(zf, g, zo, h)
        out = (y, hT, *sc.backward(zf, g, zo, dy, h, dhT))
        torch.cuda.synchronize()
        for t in (zf, g, zo, dy):
            t[:70] = 0
            t[off[-1]:] = 0
        check(off, zf, g, zo, h, dy, dhT, reverse, dtype, out)
        for t in (out[0], out[2], out[3], out[4]):
            assert not t[:70].any() and not t[off[-1]:].any()


def test_slow_gates_over_a_long_sequence():
    """Gates near one: memories of thousands of tokens, across hundreds of tiles."""
    off = _off([20000])
    run(off, 20000, 3, "f32", shift=9.0)
    run(off, 20000, 40, "bf16", shift=9.0, reverse=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_sequence_with_nan_keeps_it_to_itself(dtype):
    lens = [100, 150, 1, 90]
    off = _off(lens)
    T, D = int(off[-1]), 16
    zf, g, zo, h, dy, dhT = _inputs(5, T, 4, D, dtype)
    sc = SequenceScan(off, T, D, dtype, device=DEV)
    clean = [t.clone() for t in (*sc.forward(zf, g, zo, h), *sc.backward(zf, g, zo, dy, h, dhT))]
    g2, dy2 = g.clone(), dy.clone()
    p = torch.cat([zf, g2, zo], 1)
    p[off[1] + 20, D:2 * D] = float("nan")
    p[off[1] + 30, D:2 * D] = float("inf")
    dy2[off[1] + 40] = float("nan")
    zf2, g2, zo2 = p[:, :D], p[:, D:2 * D], p[:, 2 * D:]
    got = [t.clone() for t in (*sc.forward(zf2, g2, zo2, h), *sc.backward(zf2, g2, zo2, dy2, h, dhT))]
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[off[1]:off[2]] = False
    rows = torch.tensor([True, False, True, True], device=DEV)
    for i in (0, 2, 3, 4):
        assert torch.equal(got[i][keep], clean[i][keep])
    for i in (1, 5):
        assert torch.equal(got[i][rows], clean[i][rows])
    assert torch.isnan(got[0][off[1] + 20:off[2]].float()).all()         # NaN stays until the sequence ends
    assert torch.equal(got[0][off[1]:off[1] + 20], clean[0][off[1]:off[1] + 20])
    assert torch.isnan(got[1][1]).all()


def test_nan_gates_stay_in_their_sequence():
    """NaN in the gates themselves, where whole tiles' maps become NaN: the sequences around keep their bits."""
    off = _off([300, 900, 300])
    T, D = int(off[-1]), 8
    for dtype in ("f32", "bf16"):
        zf, g, zo, h, dy, dhT = _inputs(14, T, 3, D, dtype)
        sc = SequenceScan(off, T, D, dtype, device=DEV)
        clean = [t.clone() for t in (*sc.forward(zf, g, zo, h), *sc.backward(zf, g, zo, dy, h, dhT))]
        p = torch.cat([zf, g, zo], 1)
        p[off[1] + 400, :D] = float("nan")
        p[off[1] + 500, 2 * D:] = -float("nan")
        a = (p[:, :D], p[:, D:2 * D], p[:, 2 * D:])
        got = (*sc.forward(*a, h), *sc.backward(*a, dy, h, dhT))
        torch.cuda.synchronize()
        keep = torch.ones(T, dtype=torch.bool, device=DEV)
        keep[off[1]:off[2]] = False
        for i in (0, 2, 3, 4):
            assert torch.equal(got[i][keep], clean[i][keep]), (dtype, i)
        for i in (1, 5):
            assert torch.equal(got[i][[0, 2]], clean[i][[0, 2]]), (dtype, i)
        assert torch.equal(got[0][:off[1] + 400], clean[0][:off[1] + 400])
        assert torch.isnan(got[0][off[1] + 400:off[2]].float()).all() and torch.isnan(got[5][1]).all()


def test_sequences_without_tokens_only():
    """Tokens in no sequence at all, and sequences that are all empty: at the front, at the end, in between."""
    T, D = 700, 12
    zf, g, zo, h, dy, dhT = _inputs(15, T, 5, D, "f32")
    for off in ([0] * 6, [T] * 6, [0, 0, 300, 300, T, T], [333] * 6):
        off = np.array(off)
        for reverse in (False, True):
            sc = SequenceScan(off, T, D, "f32", reverse=reverse, device=DEV)
            y, hT = sc.forward(zf, g, zo, h)
            dzf, dg, dzo, dh0 = sc.backward(zf, g, zo, dy, h, dhT)
            torch.cuda.synchronize()
            empty = torch.as_tensor(np.diff(off) == 0, device=DEV)
            assert torch.equal(hT[empty], h[empty]) and torch.equal(dh0[empty], dhT[empty])
            check(off.tolist(), zf, g, zo, h, dy, dhT, reverse, "f32", (y, hT, dzf, dg, dzo, dh0))
            sc.forward(zf, g, zo)
            assert not sc.hT[empty].any()


def test_outputs_that_are_left_out():
    """No last states, no gradient of them, no gradient of the first ones: the other outputs keep their bits."""
    off = _off([90, 200, 0, 41])
    T, D, S = int(off[-1]), 40, 4
    zf, g, zo, h, dy, _ = _inputs(16, T, S, D, "bf16")
    sc = SequenceScan(off, T, D, "bf16", device=DEV)
    zero = torch.zeros(S, D, device=DEV)
    ref = [t.clone() for t in (*sc.forward(zf, g, zo, zero), *sc.backward(zf, g, zo, dy, zero, zero))]
    ld = zf.stride(0)
    y, dzf, dg, dzo = (torch.empty(T, D, dtype=torch.bfloat16, device=DEV) for _ in range(4))
    M.mdl_scan_forward(sc.off, S, T, D, 1, 0, zf, g, zo, ld, None, y, D, None, sc.ws, sc.ws_bytes)
    M.mdl_scan_backward(sc.off, S, T, D, 1, 0, zf, g, zo, ld, None, dy, D, None, dzf, dg, dzo, D, None, sc.ws,
                        sc.ws_bytes)
    torch.cuda.synchronize()
    for a, b in zip((y, dzf, dg, dzo), (ref[0], *ref[2:5])):
        assert torch.equal(a, b)


def test_gates_at_infinity():
    """f = 1 holds the state, f = 0 takes the input; the gradients follow."""
    off = _off([6])
    T, D = 6, 8
    zf, g, zo, h, dy, dhT = _inputs(6, T, 1, D, "f32")
    zf, g, zo = zf.clone(), g.clone(), zo.clone()
    zf[1:3], zf[4] = float("inf"), float("-inf")
    zo[5] = float("-inf")
    sc = SequenceScan(off, T, D, "f32", device=DEV)
    y, hT = sc.forward(zf, g, zo, h)
    dzf, dg, dzo, dh0 = sc.backward(zf, g, zo, dy, h, dhT)
    torch.cuda.synchronize()
    check(off, zf, g, zo, h, dy, dhT, False, "f32", (y, hT, dzf, dg, dzo, dh0))
    assert not dzf[1:3].any() and not dzf[4].any() and not dg[1:3].any()
    assert not y[5].any() and not dzo[5].any()


def test_results_repeat_bit_for_bit_on_any_stream():
    lens = [700, 3, 0, 1500, 64]
    off = _off(lens)
    T, D = int(off[-1]), 72
    zf, g, zo, h, dy, dhT = _inputs(8, T, len(lens), D, "bf16")
    sc = SequenceScan(off, T, D, "bf16", device=DEV)
    first = [t.clone() for t in (*sc.forward(zf, g, zo, h), *sc.backward(zf, g, zo, dy, h, dhT))]
    torch.cuda.synchronize()
    for _ in range(5):
        st = torch.cuda.Stream()
        sc.ws.fill_(0x5A)
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            sc.forward(zf, g, zo, h)
            again = sc.backward(zf, g, zo, dy, h, dhT)
            again2 = sc.backward(zf, g, zo, dy, h, dhT)      # the forward's workspace serves several backwards
        st.synchronize()
        for a, b in zip((sc.y, sc.hT, *again), first):
            assert torch.equal(a, b)
        assert again2[0] is again[0]


def test_two_calls_at_once():
    """Two scans on two streams, each with a workspace of its own, while a third stream keeps the device busy."""
    lens = [4000, 9000, 1, 6000]
    off = _off(lens)
    T, D = int(off[-1]), 128
    sets = [_inputs(60 + i, T, 4, D, "bf16") for i in range(2)]
    scans = [SequenceScan(off, T, D, "bf16", reverse=bool(i), device=DEV) for i in range(2)]

    def both(sc, s):
        return (*sc.forward(*s[:4]), *sc.backward(s[0], s[1], s[2], s[4], s[3], s[5]))

    ref = [[t.clone() for t in both(sc, s)] for sc, s in zip(scans, sets)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    noise = torch.randn(2048, 2048, device=DEV)
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(streams[2]):
            for _ in range(3):
                noise @ noise
        out = []
        for st, sc, s in zip(streams, scans, sets):
            with torch.cuda.stream(st):
                out.append(both(sc, s))
        torch.cuda.synchronize()
        for a, b in zip(out, ref):
            for x, y in zip(a, b):
                assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("reverse", [False, True])
def test_tiles_that_wait_for_nothing(reverse, dtype):
    """With no time allowed for any wait, every tile forms the maps it needs from the inputs: the same bits."""
    lens = [500, 3, 0, 700, 64, 1]
    off = _off(lens, first=5)
    T = int(off[-1]) + 150
    for D, gate, h0 in ((72, True, True), (20, False, True), (5, True, False)):
        zf, g, zo, h, dy, dhT = _inputs(12, T, len(lens), D, dtype, gate, h0)
        sc = SequenceScan(off, T, D, dtype, reverse=reverse, device=DEV)
        ref = [t.clone() for t in (*sc.forward(zf, g, zo, h), *sc.backward(zf, g, zo, dy, h, dhT)) if t is not None]
        try:
            M.mdl_set_wgrad_overlap(2)
            got = [t for t in (*sc.forward(zf, g, zo, h), *sc.backward(zf, g, zo, dy, h, dhT)) if t is not None]
            torch.cuda.synchronize()
        finally:
            M.mdl_set_wgrad_overlap(1)
        for i, (a, b) in enumerate(zip(got, ref)):
            assert torch.equal(a, b), (D, i)


def test_row_strides_and_unaligned_rows():
    """Outputs through the C ABI at strides of their own, rows starting at odd elements."""
    off = _off([50, 210, 5])
    T, D, S = int(off[-1]), 37, 3
    for dtype in ("f32", "bf16"):
        zf, g, zo, h, dy, dhT = _inputs(9, T, S, D, dtype)
        dt = 1 if dtype == "bf16" else 0
        sc = SequenceScan(off, T, D, dtype, device=DEV)
        ref = [t.clone() for t in (*sc.forward(zf, g, zo, h), *sc.backward(zf, g, zo, dy, h, dhT))]
        wide = torch.full((T, 4 * D + 3), 5.0, dtype=TDT[dtype], device=DEV)
        ldw = wide.stride(0)
        y, dzf, dg, dzo = (wide[:, 1 + i * D:1 + (i + 1) * D] for i in range(4))
        M.mdl_scan_forward(sc.off, S, T, D, dt, 0, zf, g, zo, zf.stride(0), h, y, ldw, sc.hT, sc.ws, sc.ws_bytes)
        assert torch.equal(y, ref[0])
        y.copy_(dy)
        M.mdl_scan_backward(sc.off, S, T, D, dt, 0, zf, g, zo, zf.stride(0), h, y, ldw, dhT, dzf, dg, dzo, ldw, sc.dh0,
                            sc.ws, sc.ws_bytes)
        torch.cuda.synchronize()
        for a, b in zip((dzf, dg, dzo), ref[2:5]):
            assert torch.equal(a, b)
        assert (wide[:, 0] == 5).all() and (wide[:, 1 + 4 * D:] == 5).all()


def test_captured_forward_and_backward_replay():
    """Two graphs that share one workspace, replayed in turn with eager work between them."""
    off = _off([400, 0, 333, 90])
    T, D, S = int(off[-1]), 48, 4
    eager = SequenceScan(off, T, D, "f32", device=DEV)
    sets = [_inputs(20 + i, T, S, D, "f32") for i in range(2)]
    held = SequenceScan(off, T, D, "f32", device=DEV)
    buf = [tuple(torch.zeros_like(t) for t in s) for s in sets]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for b in buf:
            held.forward(b[0], b[1], b[2], b[3])
            held.backward(b[0], b[1], b[2], b[4], b[3], b[5])
    torch.cuda.synchronize()
    for b in buf:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            y, hT = held.forward(b[0], b[1], b[2], b[3])
            gs = held.backward(b[0], b[1], b[2], b[4], b[3], b[5])
            out = [t.clone() for t in (y, hT, *gs)]
        graphs.append(gr)
        outs.append(out)
    for rep in range(3):
        for i, s in enumerate(sets):
            src = sets[(i + rep) % 2]
            for t, v in zip(buf[i], src):
                t.copy_(v)
            graphs[i].replay()
            ref = (*eager.forward(*src[:4]), *eager.backward(src[0], src[1], src[2], src[4], src[3], src[5]))
            torch.cuda.synchronize()
            for a, b in zip(outs[i], ref):
                assert torch.equal(a, b), rep


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 5, 8, 50, 129])
def test_step(D, dtype):
    S, n = 9, 14
    print(f"[gpu] scan step D={D} {dtype}", flush=True)
    zf, g, zo, _, _, _ = _inputs(30, S, S, D, dtype)
    st = ScanState(n, D, dtype, device=DEV)
    st.state.copy_(torch.randn(n, D, generator=torch.Generator().manual_seed(1)))
    before = st.state.clone()
    slots = torch.tensor([3, 0, 13, -1, 7, 14, 2, 5, 9], dtype=torch.int32, device=DEV)
    live = [i for i, s in enumerate(slots.tolist()) if 0 <= s < n]
    new = torch.full_like(st.state, 4.0)
    y = st.step(zf, g, zo, slots=slots, out=new)
    torch.cuda.synchronize()
    idx = slots.long()[live]
    ref_y, ref_h = oseq.scan_step(_np(zf)[live], _np(g)[live], _np(zo)[live], _np(before)[idx.cpu()])
    c = 18 + (max(np.abs(_np(zf)).max(), np.abs(_np(zo)).max()) if dtype == "bf16" else 0)
    mag = np.abs(_np(before)[idx.cpu()]) + np.abs(_np(g)[live])
    _close("h", new[idx], ref_h, c * U * mag, U)
    _close("y", y[live], ref_y, 2 * c * U * mag, HALF[dtype])
    others = [s for s in range(n) if s not in idx.tolist()]
    assert (new[others] == 4).all() and torch.equal(st.state, before)
    assert not y[[i for i in range(S) if i not in live]].any()
    # in place, and without an output gate, over the first rows
    y2 = st.step(zf, g)
    torch.cuda.synchronize()
    ref_y, ref_h = oseq.scan_step(_np(zf), _np(g), None, _np(before)[:S])
    mag = np.abs(_np(before)[:S]) + np.abs(_np(g))
    _close("h in place", st.state[:S], ref_h, c * U * mag, U)
    _close("y = h", y2, ref_y, c * U * mag, HALF[dtype])
    assert torch.equal(st.state[S:], before[S:])


def test_step_captured_beside_other_batch_sizes():
    """A captured step keeps its output while eager steps of other numbers of rows come and go."""
    D, n = 40, 6
    zf, g, zo, _, _, _ = _inputs(33, n, n, D, "f32")
    st, eager = ScanState(n, D, "f32", device=DEV), ScanState(n, D, "f32", device=DEV)
    place = st.step(zf[:2], g[:2], zo[:2]).data_ptr()
    st.state.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.step(zf[:2], g[:2], zo[:2])
    for rep in range(3):
        st.step(zf, g, zo)
        eager.step(zf, g, zo)
        others = [torch.full((2, D), float(i), device=DEV) for i in range(8)]
        graph.replay()
        want = eager.step(zf[:2], g[:2], zo[:2])
        torch.cuda.synchronize()
        y = st.step(zf[:2], g[:2], zo[:2], out=torch.empty_like(st.state))
        assert y.data_ptr() == place
        graph.replay()
        want = eager.step(zf[:2], g[:2], zo[:2])
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(st.state, eager.state), rep
        assert all((o == i).all() for i, o in enumerate(others)), rep


def test_stepped_tokens_continue_a_scanned_prefix():
    off = _off([90, 90])
    D, S = 40, 2
    zf, g, zo, h, _, _ = _inputs(31, 180, S, D, "f32")
    whole = SequenceScan(off, 180, D, "f32", device=DEV)
    y, hT = whole.forward(zf, g, zo, h)
    pre = SequenceScan(_off([87, 87]), 174, D, "f32", device=DEV)
    rows = torch.cat([torch.arange(87), torch.arange(90, 177)]).to(DEV)
    p = torch.cat([zf, g, zo], 1)[rows]
    _, mid = pre.forward(p[:, :D], p[:, D:2 * D], p[:, 2 * D:], h)
    st = ScanState(S, D, "f32", device=DEV)
    st.state.copy_(mid)
    for t in (87, 88, 89):
        r = torch.tensor([t, 90 + t], device=DEV)
        q = torch.cat([zf, g, zo], 1)[r]
        out = st.step(q[:, :D], q[:, D:2 * D], q[:, 2 * D:])
        # both sides are within 18 u per token of a state that remembers at most 90 of them
        assert (out - y[r]).abs().max() < 2 * 18 * 90 * U * 8
    assert (st.state - hT).abs().max() < 2 * 18 * 90 * U * 8


def test_image_rows_of_a_packed_layout():
    """Every row of every image, right to left, on the flat tensors of a layout; and its frames."""
    h, w = [5, 3, 8], [40, 9, 77]
    dl = DeviceLayout(h, w, 64, 1, "packed", DEV)
    off = dl.row_offsets()
    assert off.tolist() == _off(np.repeat(w, h)).tolist()
    assert dl.frame_offsets().tolist() == _off(w).tolist()
    run(off, int(off[-1]), 16, "f32", reverse=True)


@pytest.mark.parametrize("reverse", [False, True])
def test_more_than_2_31_elements(reverse):
    """Tokens past 2^31 elements: a sequence there, cut out at tile borders, gives the same bits alone."""
    D, L = 2056, 512 * 3
    T = 512 * 2100
    print(f"[gpu] scan T={T} D={D} reverse={reverse}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(5)
    zf, gg, dy = (torch.randn(T, D, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(3))
    h0, dhT = torch.randn(2, D, generator=g, device=DEV), torch.randn(2, D, generator=g, device=DEV)
    sc = SequenceScan([0, T - L, T], T, D, "bf16", reverse=reverse, device=DEV)
    got = (*sc.forward(zf, gg, None, h0), *sc.backward(zf, gg, None, dy, h0, dhT))
    part = slice(T - L, T)
    one = SequenceScan([0, L], L, D, "bf16", reverse=reverse, device=DEV)
    a = (zf[part], gg[part], None)
    ref = (*one.forward(*a, h0[1:].contiguous()), *one.backward(*a, dy[part], h0[1:].contiguous(), dhT[1:].contiguous()))
    torch.cuda.synchronize()
    for i in (0, 2, 3):
        assert torch.equal(got[i][part], ref[i]), i
    assert torch.equal(got[1][1:], ref[1]) and torch.equal(got[5][1:], ref[5])


def test_no_tokens_at_all():
    h = torch.randn(3, 6, device=DEV)
    z = torch.empty(0, 6, device=DEV)
    sc = SequenceScan([0, 0, 0, 0], 0, 6, "f32", device=DEV)
    y, hT = sc.forward(z, z, z, h)
    assert y.shape == (0, 6) and torch.equal(hT, h)
    dhT = torch.randn(3, 6, device=DEV)
    assert torch.equal(sc.backward(z, z, z, z, h, dhT)[3], dhT)
    sc.forward(z, z, z)
    assert not sc.hT.any()
