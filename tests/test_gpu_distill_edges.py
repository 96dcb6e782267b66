"""mdl_distill where its range or its rules end: weight 0 beside classes that do not exist, temperatures whose square is
no fp32 number, rows longer than the registers hold, and rows near 2^31 classes. Tolerances are test_gpu_distill.py's."""

import os
import re

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import directional_mdlstm_handwriting_amd as M
    import test_gpu_distill as td
    from test_gpu_distill import DEV, U, make, run

VEC = {"f32": 4, "bf16": 8}


def _held_vectors():
    """The longest row, in vectors of 16 bytes, that a workgroup keeps in registers: from the kernel's own dispatch, so
    that these tests follow it. Longer rows are read twice."""
    src = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "directional_mdlstm_handwriting_amd",
                       "csrc", "k_distill.hip")
    bounds = re.findall(r"nv <= (\d+)\) return fn\(ty, DistillShape<V, \d+, (\d+)>", open(src).read())
    assert bounds and all(int(nv) > 0 for _, nv in bounds)
    return max(int(b) for b, _ in bounds)


# the last row that is held; and of those read twice: the first, one of whole vectors, one of several walks and a tail
LONG = [(d, more) for d in ("f32", "bf16") for more in (0, 1, 64, 40003)]


def _long(dtype, more):
    return _held_vectors() * VEC[dtype] + more


@pytest.mark.parametrize("dtype,more", LONG)
def test_rows_read_twice(dtype, more):
    V = _long(dtype, more)
    z, ids, t, w = make(V, 3, V, 7, dtype)
    run(z, ids, t, w, 2.0, dtype)


@pytest.mark.parametrize("dtype,more", LONG[1::2])
def test_rows_read_twice_that_count_for_nothing_and_masked_classes(dtype, more):
    td.test_rows_that_count_for_nothing_and_masked_classes(_long(dtype, more), dtype)


@pytest.mark.parametrize("dtype,more", LONG[1:])
def test_rows_read_twice_strides_in_place_and_loss_alone(dtype, more):
    td.test_strides_in_place_and_loss_alone(_long(dtype, more), dtype)


@pytest.mark.parametrize("dtype,more", LONG[1:])
def test_rows_read_twice_keep_nan_and_infinities_to_themselves(dtype, more):
    """NaN and -inf at the row's first element, inside and behind its last whole vector."""
    V = _long(dtype, more)
    z, ids, t, w = make(23, 5, V, 4, dtype)
    _, l0, d0 = run(z, ids, t, w, 1.0, dtype)
    l0, d0 = l0.clone(), d0.clone()
    for at in (0, V // 2, V - 1):
        bad = z.clone()
        bad[2, at] = float("nan")
        bad[3] = float("-inf")
        bad[3, at] = 1.0
        loss, dz = td.TopKDistill(5, V, 4, dtype, 1.0, device=DEV).run(bad, ids, t, w)
        torch.cuda.synchronize()
        assert torch.equal(loss[[0, 1, 4]], l0[[0, 1, 4]]) and torch.equal(dz[[0, 1, 4]], d0[[0, 1, 4]]), at
        assert torch.isnan(loss[2]) and torch.isnan(dz[2].float()).all(), at
        td.check(bad[3:4], ids[3:4], t[3:4], w[3:4], 1.0, loss[3:4], dz[3:4], dtype)


@pytest.mark.parametrize("V,dtype", [(7, "f32"), (300, "bf16"), (5003, "f32")])
def test_weight_zero_wins_over_a_class_that_does_not_exist(V, dtype):
    """A padded frame whose ids were never set: loss 0 and gradient 0, like any other of weight 0."""
    z, ids, t, w = make(21, 6, V, 4, dtype)
    ids[1], w[1] = V, 0.0
    ids[2, 0], ids[2, 1], w[2] = -1, -5, 0.0
    ids[3, 2] = V + 1                               # with a weight: NaN
    ids[4], w[4], z[4], t[4] = 2 ** 31 - 1, 0.0, float("nan"), float("nan")
    _, loss, dz = run(z, ids, t, w, 1.5, dtype)
    assert not loss[[1, 2, 4]].any() and torch.isnan(loss[3]) and not dz[1:5].any()
    assert torch.isfinite(loss[[0, 5]]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tau", [1e-30, 1e-25, 1e-20, 3e-19, 1e15, 1e17])
def test_temperatures_whose_square_is_no_fp32_number(tau, dtype):
    """Sharp ones: the loss is w tau times the difference of the largest logits' gaps. Flat ones keep few classes, so
    that the loss, about w tau^2 ln(V / k), is within fp32."""
    z, ids, t, w = make(22, 9, 900, 6, dtype)
    _, loss, _ = run(z, ids, t, w, tau, dtype)
    assert torch.isfinite(loss).all() and (loss > 0).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("counts", [True, False])
def test_as_many_classes_as_the_header_allows(counts, dtype):
    """One row of 2^31 - 1 classes, between guards. A lane adds at most n = 2^31 / (4 1024 V) sums one after another
    (V elements a vector, four of them at a time), each of at most 4 V terms; 1024 lanes are added in 6 + 16."""
    V, k, tau, lead = 2 ** 31 - 1, 3, 2.0, 4096
    print(f"[gpu] distill V={V} {dtype} counts={counts}", flush=True)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device=DEV).manual_seed(5)
    z = torch.empty(1, V, dtype=dt, device=DEV)
    step = 1 << 27
    for a in range(0, V, step):
        z[0, a:a + step] = torch.randn(min(step, V - a), generator=g, device=DEV)
    ids = torch.tensor([[V - 1, 0, V - 2]], dtype=torch.int32, device=DEV)
    t = torch.tensor([[1.0, 0.5, -1.0]], device=DEV)
    z[0, ids[0].long()] = torch.tensor([2.0, -1.0, 3.0], device=DEV, dtype=dt)
    w = torch.tensor([1.0 if counts else 0.0], device=DEV)
    wide = torch.full((lead + V + lead,), 7.0, dtype=dt, device=DEV)
    dz, loss = wide[lead:lead + V], torch.full((1,), 7.0, device=DEV)
    M.mdl_distill(1, V, k, 1 if dtype == "bf16" else 0, z, V, ids, t, 0, w, tau, loss, dz, V)
    torch.cuda.synchronize()
    assert (wide[:lead] == 7).all() and (wide[lead + V:] == 7).all()
    if not counts:
        assert loss.item() == 0
        assert not any(dz[a:a + step].any() for a in range(0, V, step))
        return
    m = max(z[0, a:a + step].max().double().item() for a in range(0, V, step))
    L = sum(torch.exp((z[0, a:a + step].double() - m) / tau).sum().item() for a in range(0, V, step))
    vec = 8 if dtype == "bf16" else 4
    n = 2 ** 31 // (4096 * vec) + 4 * vec + 6 + 16
    x = (t.double() / tau)[0]
    p = torch.softmax(x, 0)
    lq = (z[0, ids[0].long()].double() - m) / tau - np.log(L)
    ref = tau * tau * (p * (torch.log(p) - lq)).sum().item()
    # an exponential's argument, at most 12 / 2 here, is off by 4 u of it
    rel = (n + 4 * 6 + 12) * U
    assert abs(loss.item() - ref) <= tau * tau * (rel + 64 * U * abs(np.log(L)))
    half = U if dtype == "f32" else 2.0 ** -8
    for a in range(0, V, step):
        q = torch.exp((z[0, a:a + step].double() - m) / tau) / L
        for j, c in enumerate(ids[0].tolist()):
            if a <= c < a + step:
                q[c - a] -= p[j]
        q *= tau
        got = dz[a:a + step].double()
        # the kept classes' own: p within 20 u of its magnitude
        tol = (rel + half) * q.abs() + 20 * U * tau * (q < 0) + 1e-36
        assert bool(((got - q).abs() <= tol).all()), a
