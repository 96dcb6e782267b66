"""Refusals of the sequence operators, without a GPU: every check runs before any launch, so a call with a wrong
argument returns its documented code. The addresses given are never followed."""

import pytest

import directional_mdlstm_handwriting_amd as M

P = 1 << 20        # an address no check may follow
BIG = 1 << 62


def _code(fn, *args, **kw):
    with pytest.raises(M.MdlError) as e:
        fn(*args, **kw)
    assert M.mdl_last_error()
    return e.value.code


def _with(base, **change):
    d = dict(base)
    d.update(change)
    return d


SCAN_F = dict(seq_off=P, S=2, T=1000, D=8, dtype=M.MDL_F32, reverse=0, zf=P, g=P, zo=P, ldz=8, h0=P, y=P, ldy=8, hT=P,
              ws=P, ws_bytes=BIG, stream=0)
SCAN_B = dict(seq_off=P, S=2, T=1000, D=8, dtype=M.MDL_F32, reverse=0, zf=P, g=P, zo=P, ldz=8, h0=P, dy=P, ldy=8,
              dhT=P, dzf=P, dg=P, dzo=P, ldd=8, dh0=P, ws=P, ws_bytes=BIG, stream=0)
STEP = dict(S=4, D=8, dtype=M.MDL_F32, zf=P, g=P, zo=P, ldz=8, slots=P, n_slots=9, h_in=P, h_out=P, y=P, ldy=8,
            stream=0)


@pytest.mark.parametrize("change,code", [
    (dict(seq_off=None), M.MDL_EINVAL), (dict(zf=None), M.MDL_EINVAL), (dict(g=None), M.MDL_EINVAL),
    (dict(y=None), M.MDL_EINVAL), (dict(ws=None), M.MDL_EINVAL), (dict(ws=P + 4), M.MDL_EINVAL),
    (dict(S=0), M.MDL_EINVAL), (dict(S=-1), M.MDL_EINVAL), (dict(T=-1), M.MDL_EINVAL), (dict(D=0), M.MDL_EINVAL),
    (dict(dtype=2), M.MDL_EINVAL), (dict(ldz=7), M.MDL_EINVAL), (dict(ldy=-8), M.MDL_EINVAL),
    (dict(ws_bytes=16), M.MDL_ESIZE), (dict(T=1 << 58), M.MDL_EOVERFLOW), (dict(T=1 << 40), M.MDL_EOVERFLOW),
    (dict(ldz=1 << 55), M.MDL_EOVERFLOW),
])
def test_scan_forward_refuses(change, code):
    assert _code(M.mdl_scan_forward, **_with(SCAN_F, **change)) == code


@pytest.mark.parametrize("change,code", [
    (dict(seq_off=None), M.MDL_EINVAL), (dict(dy=None), M.MDL_EINVAL), (dict(dzf=None), M.MDL_EINVAL),
    (dict(dg=None), M.MDL_EINVAL), (dict(zo=None), M.MDL_EINVAL), (dict(dzo=None), M.MDL_EINVAL),
    (dict(ldd=3), M.MDL_EINVAL), (dict(ws_bytes=0), M.MDL_ESIZE), (dict(dtype=-1), M.MDL_EINVAL),
])
def test_scan_backward_refuses(change, code):
    assert _code(M.mdl_scan_backward, **_with(SCAN_B, **change)) == code


@pytest.mark.parametrize("change,code", [
    (dict(S=0), M.MDL_EINVAL), (dict(D=0), M.MDL_EINVAL), (dict(n_slots=0), M.MDL_EINVAL), (dict(zf=None), M.MDL_EINVAL),
    (dict(h_in=None), M.MDL_EINVAL), (dict(h_out=None), M.MDL_EINVAL), (dict(y=None), M.MDL_EINVAL),
    (dict(slots=None, n_slots=3), M.MDL_EINVAL), (dict(ldz=7), M.MDL_EINVAL), (dict(ldy=7), M.MDL_EINVAL),
    (dict(dtype=9), M.MDL_EINVAL),
])
def test_scan_step_refuses(change, code):
    assert _code(M.mdl_scan_step, **_with(STEP, **change)) == code


def test_scan_workspace_sizes():
    assert M.mdl_scan_workspace_size(0, 8, M.MDL_F32) == 0
    assert M.mdl_scan_workspace_size(1, 8, M.MDL_F32) == 0
    assert M.mdl_scan_workspace_size(100000, 8, M.MDL_BF16) > 0
    assert _code(M.mdl_scan_workspace_size, 1 << 50, 8, M.MDL_F32) == M.MDL_EOVERFLOW
    assert _code(M.mdl_scan_workspace_size, 5, 0, M.MDL_F32) == M.MDL_EINVAL
    assert _code(M.mdl_scan_workspace_size, 5, 8, 3) == M.MDL_EINVAL
