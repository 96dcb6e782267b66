"""The gated recurrence where its range or its rules end: rows of nearly 2^31 channels, tiles that wait for nothing."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TDT = {"f32": torch.float32, "bf16": torch.bfloat16}

if torch.cuda.is_available():
    import directional_mdlstm_handwriting_amd as M
    from directional_mdlstm_handwriting_amd.layer import SequenceScan
    from test_gpu_scan import _inputs


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_of_as_many_channels_as_the_header_allows(dtype):
    """One token of 2^31 - 1 channels: pieces of it, at the front, inside and at the end, have the bits of a step of
    those channels alone."""
    D = 2 ** 31 - 1
    print(f"[gpu] scan step D={D} {dtype}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(6)
    dt = 1 if dtype == "bf16" else 0
    zf, gg = (torch.randn(1, D, generator=g, device=DEV, dtype=TDT[dtype]) for _ in range(2))
    h = torch.randn(1, D, generator=g, device=DEV)
    new, y = torch.full_like(h, 7.0), torch.full_like(zf, 7.0)
    M.mdl_scan_step(1, D, dt, zf, gg, None, D, None, 1, h, new, y, D)
    for a, n in ((0, 1001), (D // 2 + 3, 5000), (D - 4097, 4097)):
        part = slice(a, a + n)
        h1, y1 = torch.empty(1, n, device=DEV), torch.empty(1, n, device=DEV, dtype=TDT[dtype])
        M.mdl_scan_step(1, n, dt, zf[:, part], gg[:, part], None, n, None, 1, h[:, part], h1, y1, n)
        torch.cuda.synchronize()
        assert torch.equal(new[:, part], h1) and torch.equal(y[:, part], y1), a


def _both(sc, zf, g, zo, h, dy, dhT):
    return [t for t in (*sc.forward(zf, g, zo, h), *sc.backward(zf, g, zo, dy, h, dhT)) if t is not None]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("D,gate,h0", [(1, True, True), (3, False, True), (4, True, False), (5, True, True), (8, True, False),
                                       (9, False, False), (20, True, True), (72, False, True)])
def test_no_tile_waits(D, gate, h0, reverse, dtype):
    """Every shape of tile (1024 tokens for up to four channels, 512 for a vector of them, 256 and 128), over sequences
    within one tile and over many, with rows in no sequence: the bits of tiles that wait."""
    lens = [2500, 3, 0, 1700, 64, 1, 3000]
    off = np.concatenate([[5], 5 + np.cumsum(lens)]).astype(np.int64)
    T = int(off[-1]) + 1500
    print(f"[gpu] scan without waits D={D} {dtype} reverse={reverse}", flush=True)
    a = _inputs(12, T, len(lens), D, dtype, gate, h0)
    sc = SequenceScan(off, T, D, dtype, reverse=reverse, device=DEV)
    ref = [t.clone() for t in _both(sc, *a)]
    try:
        M.mdl_set_scan_wait(0)
        got = _both(sc, *a)
        torch.cuda.synchronize()
    finally:
        M.mdl_set_scan_wait(1)
    for i, (x, y) in enumerate(zip(got, ref)):
        assert torch.equal(x, y), i


def test_the_wavefronts_test_mode_leaves_the_scan_alone():
    """mdl_set_wgrad_overlap(2), which makes the MDLSTM's overlaps give up, costs a scan nothing (without waits these
    passes take twice as long: 193 us after 88)."""
    T, D = 40000, 64
    print("[gpu] scan under the overlap modes", flush=True)
    zf, g, zo, _, dy, _ = _inputs(13, T, 1, D, "f32", True, False)
    sc = SequenceScan([0, T], T, D, device=DEV)

    def best():
        out = []
        for _ in range(12):
            s, e = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            s.record()
            sc.forward(zf, g, zo)
            sc.backward(zf, g, zo, dy)
            e.record()
            torch.cuda.synchronize()
            out.append(s.elapsed_time(e))
        return min(out)

    plain = best()
    try:
        M.mdl_set_wgrad_overlap(2)
        other = best()
    finally:
        M.mdl_set_wgrad_overlap(1)
    assert other < 1.5 * plain, (plain, other)
