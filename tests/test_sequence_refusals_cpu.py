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
    (dict(dtype=9), M.MDL_EINVAL), (dict(S=1 << 30, n_slots=1 << 30), M.MDL_EOVERFLOW),
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


NORM_F = dict(N=10, D=8, dtype=M.MDL_F32, x=P, ldx=8, z=P, ldz=8, u=P, ldu=8, w_post=P, scale=P, w_pre=P, eps=1e-6, r=P,
              v=P, ldr=8, stream=0)
NORM_B = dict(N=10, D=8, dtype=M.MDL_F32, x=P, ldx=8, z=P, ldz=8, u=P, ldu=8, w_post=P, scale=P, w_pre=P, eps=1e-6,
              dr=P, dv=P, ldr=8, dx=P, dz=P, du=P, ldd=8, dw_post=P, dscale=P, dw_pre=P, ws=P, ws_bytes=BIG, stream=0)
DISTILL = dict(N=10, V=80, k=8, dtype=M.MDL_F32, z=P, ldz=80, ids=P, t=P, t_dtype=M.MDL_F32, w=P, tau=2.0, loss=P, dz=P,
               ldd=80, stream=0)


@pytest.mark.parametrize("change,code", [
    (dict(x=None), M.MDL_EINVAL), (dict(z=None), M.MDL_EINVAL), (dict(r=None), M.MDL_EINVAL),
    (dict(v=None), M.MDL_EINVAL), (dict(w_pre=None), M.MDL_EINVAL), (dict(N=-1), M.MDL_EINVAL),
    (dict(D=0), M.MDL_EINVAL), (dict(dtype=5), M.MDL_EINVAL), (dict(ldx=7), M.MDL_EINVAL), (dict(ldz=0), M.MDL_EINVAL),
    (dict(ldu=7), M.MDL_EINVAL), (dict(ldr=7), M.MDL_EINVAL), (dict(eps=-1.0), M.MDL_EINVAL),
    (dict(eps=float("nan")), M.MDL_EINVAL), (dict(eps=float("inf")), M.MDL_EINVAL),
    (dict(z=None, u=None, w_post=None, scale=None, r=None, w_pre=None, v=None), M.MDL_EINVAL),
    (dict(D=16385, ldx=16385, ldz=16385, ldu=16385, ldr=16385), M.MDL_EUNSUPPORTED),
    (dict(N=1 << 40), M.MDL_EOVERFLOW), (dict(ldx=1 << 59), M.MDL_EOVERFLOW),
])
def test_blocknorm_forward_refuses(change, code):
    assert _code(M.mdl_blocknorm_forward, **_with(NORM_F, **change)) == code


@pytest.mark.parametrize("change,code", [
    (dict(dx=None), M.MDL_EINVAL), (dict(dz=None), M.MDL_EINVAL), (dict(du=None), M.MDL_EINVAL),
    (dict(dv=None), M.MDL_EINVAL), (dict(dw_post=None), M.MDL_EINVAL), (dict(dscale=None), M.MDL_EINVAL),
    (dict(dw_pre=None), M.MDL_EINVAL), (dict(scale=None), M.MDL_EINVAL), (dict(ldd=7), M.MDL_EINVAL),
    (dict(ws=None), M.MDL_EINVAL), (dict(ws=P + 8), M.MDL_EINVAL), (dict(ws_bytes=8), M.MDL_ESIZE),
    (dict(w_pre=None, dw_pre=None, dv=None, dr=None), M.MDL_EINVAL),
])
def test_blocknorm_backward_refuses(change, code):
    assert _code(M.mdl_blocknorm_backward, **_with(NORM_B, **change)) == code


def test_blocknorm_workspace_sizes():
    assert M.mdl_blocknorm_workspace_size(1000, 8, M.MDL_F32) > 0
    assert _code(M.mdl_blocknorm_workspace_size, 10, 20000, M.MDL_F32) == M.MDL_EUNSUPPORTED
    assert _code(M.mdl_blocknorm_workspace_size, -1, 8, M.MDL_F32) == M.MDL_EINVAL


@pytest.mark.parametrize("change,code", [
    (dict(z=None), M.MDL_EINVAL), (dict(ids=None), M.MDL_EINVAL), (dict(t=None), M.MDL_EINVAL),
    (dict(loss=None), M.MDL_EINVAL), (dict(N=-1), M.MDL_EINVAL), (dict(V=0), M.MDL_EINVAL), (dict(k=0), M.MDL_EINVAL),
    (dict(k=81), M.MDL_EINVAL), (dict(dtype=2), M.MDL_EINVAL), (dict(t_dtype=2), M.MDL_EINVAL),
    (dict(tau=0.0), M.MDL_EINVAL), (dict(tau=-1.0), M.MDL_EINVAL), (dict(tau=float("nan")), M.MDL_EINVAL),
    (dict(tau=float("inf")), M.MDL_EINVAL), (dict(ldz=79), M.MDL_EINVAL), (dict(ldd=79), M.MDL_EINVAL),
    (dict(V=5000, ldz=5000, ldd=5000, k=1025), M.MDL_EUNSUPPORTED), (dict(N=1 << 40), M.MDL_EOVERFLOW),
    (dict(tau=1e-31), M.MDL_EINVAL),
])
def test_distill_refuses(change, code):
    assert _code(M.mdl_distill, **_with(DISTILL, **change)) == code


@pytest.mark.parametrize("S", [(1 << 31) - 1, (1 << 31) - 64])
def test_scan_refuses_more_sequences_than_its_search_counts(S):
    """The search through the offsets probes 64 at a time: its counts stay inside 32 bits."""
    assert _code(M.mdl_scan_forward, **_with(SCAN_F, S=S)) == M.MDL_EOVERFLOW
    assert _code(M.mdl_scan_backward, **_with(SCAN_B, S=S)) == M.MDL_EOVERFLOW


APART = {k: P + 4096 * (i + 1) for i, k in enumerate(("seq_off", "zf", "g", "zo", "h0", "y", "hT", "dy", "dhT", "dzf", "dg",
                                                      "dzo", "dh0", "ws"))}


@pytest.mark.parametrize("out,others", [("y", ("zf", "g", "zo", "hT")), ("hT", ("h0",))])
def test_scan_forward_refuses_outputs_over_inputs(out, others):
    base = _with(SCAN_F, **{k: v for k, v in APART.items() if k in SCAN_F})
    for o in others:
        assert _code(M.mdl_scan_forward, **_with(base, **{out: base[o]})) == M.MDL_EINVAL, o
    if out == "hT":     # [S][D] float32, one element past the first and one before the last
        n = base["S"] * base["D"] * 4
        assert _code(M.mdl_scan_forward, **_with(base, hT=base["h0"] + n - 4)) == M.MDL_EINVAL
        assert _code(M.mdl_scan_forward, **_with(base, h0=base["hT"] + 4)) == M.MDL_EINVAL
        assert _code(M.mdl_scan_forward, **_with(base, T=0, ldz=8, hT=base["h0"])) == M.MDL_EINVAL


@pytest.mark.parametrize("out,others", [("dzf", ("zf", "g", "zo", "dy", "dg", "dzo")), ("dg", ("zf", "g", "zo", "dy", "dzo")),
                                        ("dzo", ("zf", "g", "zo", "dy")), ("dh0", ("h0", "dhT"))])
def test_scan_backward_refuses_outputs_over_inputs(out, others):
    base = _with(SCAN_B, **{k: v for k, v in APART.items() if k in SCAN_B})
    for o in others:
        assert _code(M.mdl_scan_backward, **_with(base, **{out: base[o]})) == M.MDL_EINVAL, o


def test_scan_wait_is_on_or_off():
    for bad in (-1, 2):
        assert _code(M.mdl_set_scan_wait, bad) == M.MDL_EINVAL
    for on in (0, 1):
        M.mdl_set_scan_wait(on)
