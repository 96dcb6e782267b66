"""The gated recurrence where its range or its rules end: rows of nearly 2^31 channels."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TDT = {"f32": torch.float32, "bf16": torch.bfloat16}

if torch.cuda.is_available():
    import directional_mdlstm_handwriting_amd as M


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
