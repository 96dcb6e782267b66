"""Outputs over inputs that linear attention, dropout and the vocabulary's cross entropy refuse, without a GPU, and sizes of
workspaces at a launch's limits. The addresses given are never followed."""

import pytest

import directional_mdlstm_handwriting_amd as M
from test_block_refusals_cpu import ATTN_B, ATTN_F, ATTN_S, DROP, VOCAB, A, _code, _with


@pytest.mark.parametrize("change", [
    dict(y=A(3), ldy=9), dict(y=A(3), ldx=9), dict(y=A(0), ldy=9), dict(y=A(0), ldx=9), dict(y=A(1), ldr=9),
    dict(y=A(1), ldy=10), dict(y=A(2)),
])
def test_dropout_over_its_inputs_at_another_stride(change):
    base = _with(DROP, ldx=8, ldr=8, ldy=8, **{k: v for k, v in change.items() if k == "y"})
    rest = {k: v for k, v in change.items() if k != "y"}
    if base["y"] == A(3):                    # apart: nothing to refuse but what is refused anyway
        assert _code(M.mdl_dropout, **_with(base, x=None, **rest)) == M.MDL_EINVAL
    else:
        assert _code(M.mdl_dropout, **_with(base, **rest)) == M.MDL_EINVAL
        assert "over" in M.mdl_last_error()


@pytest.mark.parametrize("change", [dict(loss=A(0)), dict(loss=A(1)), dict(loss=A(2)), dict(loss=A(3)), dict(loss=A(5)),
                                    dict(loss=A(6)), dict(dh=A(2)), dict(dh=A(3)), dict(dW=A(2)), dict(dW=A(3))])
def test_vocab_loss_over_its_tensors(change):
    assert _code(M.mdl_vocab_loss, **_with(VOCAB, **change)) == M.MDL_EINVAL
    assert "over" in M.mdl_last_error()


@pytest.mark.parametrize("change", [dict(y=A(5)), dict(y=A(1)), dict(y=A(0)), dict(hT=A(1)), dict(hT=A(0)), dict(hT=A(6))])
def test_attention_forward_over_states_and_decays(change):
    assert _code(M.mdl_linattn_forward, **_with(ATTN_F, **change)) == M.MDL_EINVAL
    assert "over" in M.mdl_last_error()


@pytest.mark.parametrize("change", [dict(dq=A(5)), dict(dk=A(7)), dict(dv=A(1)), dict(dv=A(0)), dict(dh0=A(2)), dict(dh0=A(6)),
                                    dict(dh0=A(8)), dict(dh0=A(10)), dict(dh0=A(1)), dict(dq=A(11))])
def test_attention_backward_over_states_and_decays(change):
    assert _code(M.mdl_linattn_backward, **_with(ATTN_B, **change)) == M.MDL_EINVAL
    assert "over" in M.mdl_last_error()


# nine slots of 2 x 8 x 4 floats
@pytest.mark.parametrize("change", [dict(h_out=A(6) + 4), dict(h_out=A(6) + 256), dict(h_out=A(6) - 9 * 256 + 4),
                                    dict(y=A(6)), dict(h_out=A(9), y=A(9)), dict(y=A(1)), dict(y=A(5)), dict(h_out=A(2)),
                                    dict(h_out=A(1))])
def test_attention_step_over_states(change):
    assert _code(M.mdl_linattn_step, **_with(ATTN_S, **change)) == M.MDL_EINVAL
    assert "over" in M.mdl_last_error()


def test_vocab_loss_alone_in_launches_of_a_legal_size():
    """The loss alone of 2^23 rows over 32768 classes: one launch would have 2^16 x 2^8 tiles of 256 threads, 2^32. It is made
    of several, whose statistics (8 bytes a row and tile of 128 classes) the workspace holds one of."""
    f = M.mdl_vocab_loss_workspace_size
    N, V = 1 << 23, 1 << 15
    rows = N * (16 + 4 * 4)                  # the hidden states of 8 channels and a row's numbers
    assert f(N, 8, V, M.MDL_BF16, False) < rows + N * 4 + (1 << 16) + (N // 2) * (V // 128) * 8
