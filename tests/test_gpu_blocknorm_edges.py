"""The norms' weight gradients against the bound of the sums as they are made: a lane adds the rows that its workgroup
takes in turn, a workgroup the rows it holds at once, then every 64th workgroup's sum one after another, and 64 of those
pairwise."""

import numpy as np
import pytest
import torch

from fp_bounds import U, Err, assert_within
from oracle import sequence as oseq

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from directional_mdlstm_handwriting_amd.layer import BlockNorm
    from test_gpu_blocknorm import DEV, INPUTS, _np, make, run


def _additions(N, rows):
    """rows: what a workgroup holds at once."""
    turns = -(-N // rows)
    blocks = max(1, min(turns, max(256, min(turns // 4, 1024))))
    return -(-turns // blocks) + rows + -(-blocks // 64) + 6


@pytest.mark.parametrize("N,D,dtype,rows", [(20011, 50, "f32", 16), (5000, 16, "bf16", 32), (3001, 300, "bf16", 4),
                                            (1500, 2048, "bf16", 1), (70001, 9, "f32", 32), (2, 700, "f32", 1)])
def test_weight_gradients(N, D, dtype, rows):
    print(f"[gpu] norm weight gradients N={N} D={D} {dtype}", flush=True)
    t = make(N + 1, N, D, dtype)
    got = run(BlockNorm(N, D, dtype, device=DEV), t)
    a = {k: _np(v) for k, v in t.items()}
    ref = oseq.blocknorm_backward(*(a[k] for k in INPUTS), a["dr"], a["dv"], 1e-6)
    row, col, plain = 64, _additions(N, rows), dtype == "bf16"
    z = Err(a["z"])
    zh = z * ((z * z).sum(1, row, True) * (1.0 / D) + 1e-6).rsqrt()
    g, _ = Err(a["u"]).sigmoid(plain)
    r = Err(a["scale"]) * a["w_post"] * g * zh + a["x"]
    rho = ((r * r).sum(1, row, True) * (1.0 / D) + 1e-6).rsqrt()
    rh, tv = r * rho, Err(a["dv"]) * a["w_pre"]
    d = rho * (tv - rh * ((tv * r).sum(1, row, True) * rho * (1.0 / D))) + a["dr"]
    q = (d * g * zh).sum(0, col)
    bound = {"dw_post": q * a["scale"], "dscale": q * a["w_post"], "dw_pre": (rh * a["dv"]).sum(0, col)}
    for k, b in bound.items():
        assert_within(k, _np(got[k]), Err(ref[k], b.e), U)
