"""Linear attention, dropout and the vocabulary's cross entropy together with the norms, as they are used: a residual block
along the frames of packed examples, trained on word pieces; and the same block serving, a prefix read at once and then token
by token. Every gradient against torch's autograd in float64 on the CPU.

    v = norm(x);  (q, k, z) = v Wp;  y = attention forward + attention backward;  r = x + dropout(y Wo);  v2 = norm(r)
    loss = cross entropy of v2 over the classes of We

Tolerance: a gradient passes about ten stages, each with sums of at most 130 fp32 terms (u = 2^-24 each) and a growth of
relative errors below ten: 10 * 130 * 10 u = 7.8e-4 of the tensor's largest magnitude.
"""

import numpy as np
import pytest
import torch

from oracle import block as oblk

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TOL = 7.8e-4
EPS = 1e-6

if torch.cuda.is_available():
    from directional_mdlstm_handwriting_amd.layer import (AttentionState, BlockNorm, DeviceLayout, DeviceParams, Dropout,
                                                          LayerGrads, LinearAttention, PackedStack, VocabLoss)
    from directional_mdlstm_handwriting_amd import mdl_blockconv_backward, mdl_blockconv_forward


def _close(name, got, ref):
    err, top = (got.double().cpu() - ref).abs().max().item(), ref.abs().max().item()
    assert err <= TOL * top, f"{name}: {err:.3g} of {top:.3g}"


def _params(seed, T, D, H, V):
    g = torch.Generator().manual_seed(seed)

    def rn(*s, scale=1.0, shift=0.0):
        return torch.randn(*s, generator=g) * scale + shift

    P = dict(x=rn(T, D), Wp=rn(D, 3 * D, scale=D ** -0.5), Wo=rn(D, D, scale=D ** -0.5), We=rn(V, D, scale=D ** -0.5),
             wa=rn(D, scale=0.1, shift=1.0), wb=rn(D, scale=0.1, shift=1.0))
    ids = torch.randint(0, V, (T,), generator=g)
    w = (torch.rand(T, generator=g) > 0.1).float()
    return P, ids, w


def test_block_trained_on_word_pieces():
    widths, D, H, V, p_drop, seed = [23, 140, 9, 31], 48, 3, 130, 0.25, 99
    T = sum(widths)
    P, ids, w = _params(1, T, D, H, V)
    dec = np.float32([0.9, 0.97, 0.995])
    mask = torch.as_tensor(oblk.dropout_mask(T, D, p_drop, seed, 5))
    off = np.concatenate([[0], np.cumsum(widths)])
    # the reference
    a = {n: t.double().clone().requires_grad_() for n, t in P.items()}

    def norm(t, wt):
        return t * torch.rsqrt(t.square().mean(1, keepdim=True) + EPS) * wt

    q, k, z = ((norm(a["x"], a["wa"]) @ a["Wp"]).view(T, 3, H, D // H)[:, i] for i in range(3))
    y = 0
    d = torch.as_tensor(dec.astype(np.float64))[:, None, None]
    for rev in (False, True):
        out = [None] * T
        for s in range(len(widths)):
            st = torch.zeros(H, D // H, D // H, dtype=torch.float64)
            rows = range(off[s], off[s + 1])
            for t in (reversed(rows) if rev else rows):
                st = d * st + k[t][:, :, None] * z[t][:, None, :]
                out[t] = (D // H) ** -0.5 * (q[t][:, :, None] * st).sum(1).flatten()
        y = y + torch.stack(out)
    v2 = norm(a["x"] + (y @ a["Wo"]) * mask, a["wb"])
    loss_ref = w.double() * torch.nn.functional.cross_entropy(v2 @ a["We"].T, ids, reduction="none")
    loss_ref.sum().backward()

    p = {n: t.to(DEV) for n, t in P.items()}
    dl = DeviceLayout([1] * len(widths), widths, 64, 1, "packed", DEV)
    frames = dl.frame_offsets()
    before, after = BlockNorm(T, D, eps=EPS, device=DEV), BlockNorm(T, D, eps=EPS, device=DEV)
    att = [LinearAttention(frames, T, H, D // H, D // H, dec, reverse=r, device=DEV) for r in (False, True)]
    drop = Dropout(T, D, p_drop, seed=seed, call=4, device=DEV)
    drop.advance()
    vl = VocabLoss(T, D, V, device=DEV)
    print(f"[gpu] block T={T} D={D}", flush=True)
    _, v = before.forward(p["x"], w_pre=p["wa"])
    proj = v @ p["Wp"]
    qkv = [proj[:, i * D:(i + 1) * D] for i in range(3)]
    y = att[0].forward(*qkv)[0] + att[1].forward(*qkv)[0]
    r = drop.forward(y @ p["Wo"], p["x"])
    _, v2 = after.forward(r, w_pre=p["wb"])
    loss, dv2, dWe = vl.run(v2, p["We"], ids.to(torch.int32).to(DEV), w.to(DEV))
    grads = dict(We=dWe)
    dr, _, _, _, _, grads["wb"] = after.backward(r, None, None, None, None, p["wb"], None, dv2)
    do = drop.backward(dr)
    grads["Wo"] = y.T @ do
    dy = do @ p["Wo"].T
    dp = sum(torch.cat(x.backward(*qkv, dy)[:3], 1) for x in att)
    grads["Wp"] = v.T @ dp
    grads["x"], _, _, _, _, grads["wa"] = before.backward(p["x"], None, None, None, None, p["wa"], dr, dp @ p["Wp"].T)
    torch.cuda.synchronize()
    _close("loss", loss, loss_ref.detach())
    for n, t in a.items():
        _close("d" + n, grads[n], t.grad)


def test_block_served_as_it_is_read():
    """A prefix of each stream read at once, then its tokens one at a time through norm, projection, step and norm: the rows
    of the block read whole, to the tolerance above."""
    S, L, P0, D, H = 3, 80, 70, 48, 3
    P, _, _ = _params(2, S * L, D, H, 10)
    p = {n: t.to(DEV) for n, t in P.items()}
    dec = [0.9, 0.97, 0.995]

    def read(x, off):
        n = x.shape[0]
        _, v = BlockNorm(n, D, eps=EPS, device=DEV).forward(x, w_pre=p["wa"])
        pr = v @ p["Wp"]
        y, hT = LinearAttention(off, n, H, D // H, D // H, dec, device=DEV).forward(pr[:, :D], pr[:, D:2 * D], pr[:, 2 * D:])
        r = x + y @ p["Wo"]
        return BlockNorm(n, D, eps=EPS, device=DEV).forward(r, w_pre=p["wb"])[1], hT

    x = p["x"].view(S, L, D)
    whole, hT = read(p["x"], np.arange(S + 1) * L)
    whole = whole.view(S, L, D).clone()
    first, h = read(x[:, :P0].reshape(-1, D).contiguous(), np.arange(S + 1) * P0)
    st = AttentionState(6, H, D // H, D // H, dec, device=DEV)
    slots = torch.tensor([4, 0, 3], dtype=torch.int32, device=DEV)
    st.state[slots.long()] = h
    one = [BlockNorm(S, D, eps=EPS, device=DEV) for _ in range(2)]
    for i in range(P0, L):
        xi = x[:, i].contiguous()
        _, v = one[0].forward(xi, w_pre=p["wa"])
        pr = v @ p["Wp"]
        r = xi + st.step(pr[:, :D], pr[:, D:2 * D], pr[:, 2 * D:], slots=slots) @ p["Wo"]
        _, v2 = one[1].forward(r, w_pre=p["wb"])
        b = whole[:, i]
        assert (v2 - b).abs().max() <= TOL * b.abs().max()
    assert (first.view(S, P0, D) - whole[:, :P0]).abs().max() <= TOL * whole.abs().max()
    assert (st.state[slots.long()] - hT).abs().max() <= TOL * hT.abs().max()


def _stack(dropout, seed=5):
    heights, widths = [9, 14, 6, 12], [30, 17, 40, 9]
    g = torch.Generator().manual_seed(3)
    C, Hs, couts = 1, [4, 6, 8], [6, 10]
    st = PackedStack(heights, widths, C, Hs, couts, [64, 16, 8], device=DEV, dropout=dropout, seed=seed)
    cin = [C, *couts]
    P = []
    for c, h in zip(cin, Hs):
        t = [torch.randn(4, r, 5 * h, generator=g) * 0.4 for r in (c, h, h)] + [torch.randn(4, 5 * h, generator=g) * 0.2]
        P.append(DeviceParams(*(x.to(DEV) for x in t)))
    convs = [((torch.randn(o, 4, h, 2, 4, generator=g) * 0.2).to(DEV), (torch.randn(o, generator=g) * 0.1).to(DEV))
             for o, h in zip(couts, Hs)]
    x = torch.randn(sum(a * b for a, b in zip(heights, widths)) * C, generator=g).to(DEV)
    dy = torch.randn(st.levels[-1].y.shape, generator=g).to(DEV)
    return st, P, convs, x, dy


def _step(st, P, convs, x, dy, **kw):
    y = st.forward(x, P, convs, **kw).clone()
    lg = [LayerGrads.like(p) for p in P]
    cg = [(torch.empty_like(W), torch.empty_like(b)) for W, b in convs]
    dx = torch.empty_like(x)
    st.backward(P, convs, dy, lg, cg, dx_flat=dx)
    torch.cuda.synchronize()
    return [y, dx] + [t for g in lg for t in (g.dWx, g.dUl, g.dUu, g.db)] + [t for c in cg for t in c]


def test_stack_with_dropout_between_its_levels():
    """Against the same kernels called one by one with masks multiplied in torch; masks differ by level and step, nothing is
    dropped without training, and a stack without dropout is what it was."""
    drop, P, convs, x, dy = _stack(0.4)
    plain = _stack(0.0)[0]
    assert plain.drops == [] and len(drop.drops) == 2
    base = _step(plain, P, convs, x, dy)
    for a, b in zip(_step(drop, P, convs, x, dy, train=False), base):
        assert torch.equal(a, b)
    for step in range(2):
        got = _step(drop, P, convs, x, dy)
        masks = [torch.as_tensor(oblk.dropout_mask(d.N, d.D, 0.4, 5, 2 * step + i).astype(np.float32)).to(DEV)
                 for i, d in enumerate(drop.drops)]
        assert not torch.equal(got[0], base[0])
        st = plain
        st.levels[0].scatter(x)
        for i, lay in enumerate(st.levels):
            lay.forward(P[i])
            if i < 2:
                nxt = st.levels[i + 1]
                mdl_blockconv_forward(lay.dl.layout, lay.dl.desc, nxt.dl.layout, nxt.dl.desc, lay.h_dirs, lay.H, 2, 4,
                                      *convs[i], st.couts[i], nxt.x_canvas)
                nxt.x_canvas.mul_(masks[i].view(nxt.x_canvas.shape))
        st.levels[-1].dirsum()
        ref_y = st.levels[-1].y.clone()
        lg = [LayerGrads.like(p) for p in P]
        cg = [(torch.empty_like(W), torch.empty_like(b)) for W, b in convs]
        dx = torch.empty_like(x)
        for i in (2, 1, 0):
            lay = st.levels[i]
            kw = dict(dy_flat=dy) if i == 2 else dict(dh_dirs=st.dh_dirs[i])
            kw.update(dict(dx_canvas=st.dx_canvas[i - 1]) if i else dict(dx_flat=dx))
            lay.backward(P[i], lg[i], **kw)
            if i:
                prev = st.levels[i - 1]
                st.dx_canvas[i - 1].mul_(masks[i - 1].view(st.dx_canvas[i - 1].shape))
                mdl_blockconv_backward(prev.dl.layout, prev.dl.desc, lay.dl.layout, lay.dl.desc, prev.h_dirs, prev.H, 2, 4,
                                       convs[i - 1][0], st.couts[i - 1], st.dx_canvas[i - 1], st.dh_dirs[i - 1], *cg[i - 1],
                                       *st.conv_ws[i - 1])
        torch.cuda.synchronize()
        ref = [ref_y, dx] + [t for g in lg for t in (g.dWx, g.dUl, g.dUu, g.db)] + [t for c in cg for t in c]
        for a, b in zip(got, ref):
            assert torch.equal(a, b), step
        drop.advance_dropout()
