"""Refusals of linear attention, dropout and the vocabulary's cross entropy, without a GPU: every check runs before any
launch, so a call with a wrong argument returns its documented code. The addresses given are never followed."""

import numpy as np
import pytest

import directional_mdlstm_handwriting_amd as M

BIG = 1 << 62


def A(n):
    """Addresses that no check may follow, far from each other."""
    return (1 << 30) * (n + 1)


def _code(fn, *args, **kw):
    with pytest.raises(M.MdlError) as e:
        fn(*args, **kw)
    assert M.mdl_last_error()
    return e.value.code


def _with(base, **change):
    d = dict(base)
    d.update(change)
    return d


ATTN_F = dict(seq_off=A(0), S=2, T=1000, H=2, Dk=8, Dv=4, dtype=M.MDL_F32, reverse=0, decay=A(1), scale=1.0, q=A(2), ldq=16,
              k=A(3), ldk=16, v=A(4), ldv=8, h0=A(5), y=A(6), ldy=8, hT=A(7), ws=A(8), ws_bytes=BIG, stream=0)
ATTN_B = dict(seq_off=A(0), S=2, T=1000, H=2, Dk=8, Dv=4, dtype=M.MDL_F32, reverse=0, decay=A(1), scale=1.0, q=A(2), ldq=16,
              k=A(3), ldk=16, v=A(4), ldv=8, h0=A(5), dy=A(6), lddy=8, dhT=A(7), dq=A(8), lddq=16, dk=A(9), lddk=16,
              dv=A(10), lddv=8, dh0=A(11), ws=A(12), ws_bytes=BIG, stream=0)
ATTN_S = dict(S=4, H=2, Dk=8, Dv=4, dtype=M.MDL_F32, decay=A(1), scale=1.0, q=A(2), ldq=16, k=A(3), ldk=16, v=A(4), ldv=8,
              slots=A(5), n_slots=9, h_in=A(6), h_out=A(6), y=A(7), ldy=8, stream=0)
COMMON = [
    (dict(H=0), M.MDL_EINVAL), (dict(Dk=0), M.MDL_EINVAL), (dict(Dv=-1), M.MDL_EINVAL), (dict(dtype=2), M.MDL_EINVAL),
    (dict(decay=None), M.MDL_EINVAL), (dict(q=None), M.MDL_EINVAL), (dict(k=None), M.MDL_EINVAL),
    (dict(v=None), M.MDL_EINVAL), (dict(ldq=15), M.MDL_EINVAL), (dict(ldk=-1), M.MDL_EINVAL), (dict(ldv=7), M.MDL_EINVAL),
    (dict(S=0), M.MDL_EINVAL), (dict(Dk=129, ldq=300, ldk=300), M.MDL_EUNSUPPORTED),
    (dict(Dv=129, ldv=300), M.MDL_EUNSUPPORTED),
    (dict(H=65536, ldq=1 << 20, ldk=1 << 20, ldv=1 << 20), M.MDL_EUNSUPPORTED),
]


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(seq_off=None), M.MDL_EINVAL), (dict(y=None), M.MDL_EINVAL), (dict(T=-1), M.MDL_EINVAL),
    (dict(ldy=7), M.MDL_EINVAL), (dict(ws=None), M.MDL_EINVAL), (dict(ws=A(8) + 8), M.MDL_EINVAL),
    (dict(ws_bytes=16), M.MDL_ESIZE), (dict(T=1 << 36), M.MDL_EOVERFLOW), (dict(ldq=1 << 23), M.MDL_EOVERFLOW),
    (dict(ldy=1 << 40), M.MDL_EOVERFLOW), (dict(S=2 ** 31 - 1), M.MDL_EOVERFLOW), (dict(S=1 << 30), M.MDL_EOVERFLOW),
    (dict(y=A(2)), M.MDL_EINVAL), (dict(y=A(4)), M.MDL_EINVAL), (dict(hT=A(5)), M.MDL_EINVAL),
    (dict(hT=A(5) + 64), M.MDL_EINVAL), (dict(hT=A(3)), M.MDL_EINVAL),
])
def test_attention_forward_refuses(change, code):
    assert _code(M.mdl_linattn_forward, **_with(ATTN_F, **change)) == code


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(seq_off=None), M.MDL_EINVAL), (dict(dy=None), M.MDL_EINVAL), (dict(dq=None), M.MDL_EINVAL),
    (dict(dk=None), M.MDL_EINVAL), (dict(dv=None), M.MDL_EINVAL), (dict(lddy=7), M.MDL_EINVAL),
    (dict(lddq=15), M.MDL_EINVAL), (dict(lddk=0), M.MDL_EINVAL), (dict(lddv=7), M.MDL_EINVAL),
    (dict(lddv=1 << 23), M.MDL_EOVERFLOW), (dict(ws_bytes=0), M.MDL_ESIZE), (dict(dq=A(6)), M.MDL_EINVAL),
    (dict(dk=A(8)), M.MDL_EINVAL), (dict(dh0=A(5)), M.MDL_EINVAL), (dict(dh0=A(7) + 32), M.MDL_EINVAL),
])
def test_attention_backward_refuses(change, code):
    assert _code(M.mdl_linattn_backward, **_with(ATTN_B, **change)) == code


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(n_slots=0), M.MDL_EINVAL), (dict(h_in=None), M.MDL_EINVAL), (dict(h_out=None), M.MDL_EINVAL),
    (dict(y=None), M.MDL_EINVAL), (dict(ldy=7), M.MDL_EINVAL), (dict(slots=None, n_slots=3), M.MDL_EINVAL),
    (dict(S=1 << 23), M.MDL_EOVERFLOW), (dict(ldq=1 << 59), M.MDL_EOVERFLOW), (dict(y=A(4)), M.MDL_EINVAL),
])
def test_attention_step_refuses(change, code):
    assert _code(M.mdl_linattn_step, **_with(ATTN_S, **change)) == code


def test_attention_workspace_sizes():
    f = M.mdl_linattn_workspace_size
    assert f(1, 0, 2, 8, 8, M.MDL_F32) == 0
    assert f(3, 1, 2, 8, 8, M.MDL_BF16) == 0
    assert f(1, 100000, 2, 8, 8, M.MDL_BF16) > 0
    assert _code(f, 1, 5, 2, 8, 8, 3) == M.MDL_EINVAL
    assert _code(f, 0, 5, 2, 8, 8, M.MDL_F32) == M.MDL_EINVAL
    assert _code(f, 1, -1, 2, 8, 8, M.MDL_F32) == M.MDL_EINVAL
    assert _code(f, 1, 5, 2, 8, 200, M.MDL_F32) == M.MDL_EUNSUPPORTED
    assert _code(f, 1, 1 << 50, 2, 8, 8, M.MDL_F32) == M.MDL_EOVERFLOW


DROP = dict(N=10, D=8, dtype=M.MDL_F32, x=A(0), ldx=8, r=A(1), ldr=8, p=0.1, rng=A(2), y=A(3), ldy=8, stream=0)


@pytest.mark.parametrize("change,code", [
    (dict(N=-1), M.MDL_EINVAL), (dict(D=0), M.MDL_EINVAL), (dict(dtype=7), M.MDL_EINVAL), (dict(x=None), M.MDL_EINVAL),
    (dict(y=None), M.MDL_EINVAL), (dict(rng=None), M.MDL_EINVAL), (dict(rng=A(2) + 4), M.MDL_EINVAL),
    (dict(ldx=7), M.MDL_EINVAL), (dict(ldr=7), M.MDL_EINVAL), (dict(ldy=7), M.MDL_EINVAL), (dict(p=-0.1), M.MDL_EINVAL),
    (dict(p=1.0), M.MDL_EINVAL), (dict(p=0.999999), M.MDL_EINVAL), (dict(p=float("nan")), M.MDL_EINVAL),
    (dict(N=(1 << 33) + 1), M.MDL_EOVERFLOW), (dict(ldx=1 << 58), M.MDL_EOVERFLOW),
])
def test_dropout_refuses(change, code):
    assert _code(M.mdl_dropout, **_with(DROP, **change)) == code


VOCAB = dict(N=10, D=8, V=80, dtype=M.MDL_F32, h=A(0), ldh=8, W=A(1), ids=A(2), w=A(3), loss=A(4), dh=A(5), lddh=8, dW=A(6),
             ws=A(7), ws_bytes=BIG, stream=0)


@pytest.mark.parametrize("change,code", [
    (dict(N=-1), M.MDL_EINVAL), (dict(D=0), M.MDL_EINVAL), (dict(V=0), M.MDL_EINVAL), (dict(dtype=4), M.MDL_EINVAL),
    (dict(h=None), M.MDL_EINVAL), (dict(W=None), M.MDL_EINVAL), (dict(ids=None), M.MDL_EINVAL),
    (dict(loss=None), M.MDL_EINVAL), (dict(dh=None), M.MDL_EINVAL), (dict(dW=None), M.MDL_EINVAL),
    (dict(ldh=7), M.MDL_EINVAL), (dict(lddh=7), M.MDL_EINVAL), (dict(W=A(1) + 8), M.MDL_EINVAL),
    (dict(dW=A(1)), M.MDL_EINVAL), (dict(dW=A(0)), M.MDL_EINVAL), (dict(dW=A(5)), M.MDL_EINVAL),
    (dict(dh=A(1)), M.MDL_EINVAL), (dict(ws=None), M.MDL_EINVAL), (dict(ws=A(7) + 4), M.MDL_EINVAL),
    (dict(ws_bytes=64), M.MDL_ESIZE), (dict(D=65537, ldh=65537, lddh=65537), M.MDL_EUNSUPPORTED),
    (dict(V=(1 << 20) + 1), M.MDL_EUNSUPPORTED), (dict(N=1 << 31), M.MDL_EOVERFLOW),
    (dict(N=1 << 22, V=1 << 20), M.MDL_EOVERFLOW), (dict(ldh=1 << 59), M.MDL_EOVERFLOW),
])
def test_vocab_loss_refuses(change, code):
    assert _code(M.mdl_vocab_loss, **_with(VOCAB, **change)) == code


def test_vocab_workspace_sizes():
    f = M.mdl_vocab_loss_workspace_size
    alone, grads = f(4096, 2048, 32000, M.MDL_BF16, False), f(4096, 2048, 32000, M.MDL_BF16, True)
    # the statistics and the packed rows; with gradients a piece of G and dh's sums, far below the logits' 524 MB in fp32
    assert 0 < alone < grads < 4096 * 32000 * 4
    assert _code(f, 5, 8, 0, M.MDL_F32, True) == M.MDL_EINVAL
    assert _code(f, 5, 1 << 17, 8, M.MDL_F32, True) == M.MDL_EUNSUPPORTED


def test_layer_checks_before_any_device_is_touched():
    from directional_mdlstm_handwriting_amd import layer as L
    with pytest.raises(ValueError):
        L._decays([0.5, 1.5], 2, "cpu")
    with pytest.raises(ValueError):
        L._decays([0.5], 2, "cpu")
    with pytest.raises(ValueError):
        L._decays([float("nan")], 1, "cpu")
    assert L._decays(np.float64([0.0, 1.0]), 2, "cpu").dtype == L.torch.float32
    for off in ([0], [0, 5, 3], [-1, 2], [0, 11]):
        with pytest.raises(ValueError):
            L._sequences(off, 10, "cpu")
