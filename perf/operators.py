"""The sequence operators' measured cases: the gated linear recurrence over packed sequences (forward, backward, one
token), the norms before and after a block with its gate and residual scale, and the distillation loss from a
teacher's top logits.

Each case runs in its plain form (elementary torch operations in 32 bits, rounded once at the end) or, with ``own``
set, through the framework's entry points. ``exact`` evaluates the definitions in 64 bits, written apart from the
plain form.

    f = sigmoid(zf), o = sigmoid(zo);  h_t = f_t h_{t-1} + (1 - f_t) g_t,  y_t = o_t h_t  (y = h without zo)
    n = z rsqrt(mean z^2 + eps) w_post,  r = x + scale sigmoid(u) n,  v = r rsqrt(mean r^2 + eps) w_pre
    p = softmax_k(t / tau), q = softmax_V(z / tau),  loss = w tau^2 sum_j p_j (ln p_j - ln q_{id_j})
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
ESZ = {"f32": 4, "bf16": 2}


# ---- cases ------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one writer's line, read as it is written: one token of one stream, its state among 16 slots
        dict(name="step_one_line", op="step", S=1, slots=16, D=512, dtype="bf16"),
        # a server's live lines, one token each
        dict(name="step_live_batch", op="step", S=1024, slots=1280, D=1024, dtype="bf16"),
        # one line's frames read at once before its tokens are stepped
        dict(name="scan_prefix_f32", op="scan", S=1, lo=1000, hi=1000, D=512, dtype="f32", gate=True, reverse=False,
             h0=False),
        # the frames of the line batch (32 lines, 256 to 1024 wide), a training step's recurrence both ways
        dict(name="scan_lines", op="scan_train", S=32, lo=256, hi=1024, D=512, dtype="bf16", gate=True, reverse=False,
             h0=True),
        # every pixel row of the line batch's images (32 images of 32 rows) at H = 32, right to left
        dict(name="scan_rows_f32", op="scan_train", S=1024, lo=256, hi=1024, D=32, dtype="f32", gate=False,
             reverse=True, h0=False),
        # whole documents as one sequence each
        dict(name="scan_documents", op="scan_train", S=4, lo=40000, hi=65536, D=1024, dtype="bf16", gate=True,
             reverse=False, h0=True),
        # the block's norms beside a few stepped tokens
        dict(name="norm_step", op="norm", N=8, D=512, dtype="bf16"),
        # the stack's last level (H = 50): rows that are no multiple of 16 bytes
        dict(name="norm_odd_f32", op="norm_train", N=81920, D=50, dtype="f32"),
        # a wide block over the line batch's frames
        dict(name="norm_wide", op="norm_train", N=20480, D=2048, dtype="bf16"),
        # character classes of the CTC head (K = 80), a word batch's frames
        dict(name="distill_frames_f32", op="distill", N=6000, V=80, k=8, dtype="f32"),
        # word pieces
        dict(name="distill_pieces", op="distill", N=4096, V=32000, k=64, dtype="bf16"),
        # a large odd dictionary in 32 bits
        dict(name="distill_dictionary_f32", op="distill", N=1000, V=100003, k=20, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _odd(rng, v, m):
    """v as drawn, or its nearest multiple of m: half of the sizes are round ones."""
    return v if rng.random() < 0.5 else max(m, v // m * m)


def draw(rng):
    op = rng.choice(["step", "scan", "scan_train", "scan_train", "norm", "norm_train", "distill", "distill"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "step":
        S = _log(rng, 1, 2048)
        return dict(op=op, S=S, slots=S + rng.randrange(0, 300), D=_odd(rng, _log(rng, 16, 2048), 64), dtype=dtype)
    if op in ("scan", "scan_train"):
        D = _odd(rng, _log(rng, 2, 2048), 32)
        T = _log(rng, 64, max(128, min(400000, 100000000 // D)))     # tokens in all, about
        hi = _log(rng, 16, min(T, 65536))
        S = max(1, min(4096, 2 * T // (hi + 1)))
        return dict(op=op, S=S, lo=rng.choice([0 if S > 3 else 1, 1, max(1, hi // 4)]), hi=hi, D=D, dtype=dtype,
                    gate=rng.random() < 0.6, reverse=rng.random() < 0.5, h0=rng.random() < 0.5)
    if op in ("norm", "norm_train"):
        D = _odd(rng, _log(rng, 16, 8192), 64)
        return dict(op=op, N=_log(rng, 1, max(2, min(200000, 60000000 // D))), D=D, dtype=dtype)
    V = _odd(rng, _log(rng, 40, 131072), 64)
    return dict(op=op, N=_log(rng, 8, max(9, min(50000, 130000000 // V))), V=V, k=min(V, _log(rng, 1, 128)),
                dtype=dtype)


def _offsets(case):
    """The sequences' offsets [S + 1]: lengths lo..hi, fixed by the case."""
    r = np.random.default_rng([case["S"], case["lo"], case["hi"], case["D"]])
    return np.concatenate([[0], np.cumsum(r.integers(case["lo"], case["hi"] + 1, case["S"]))]).astype(np.int64)


def work(case):
    op, e = case["op"], ESZ[case["dtype"]]
    if op == "step":
        n = case["S"] * case["D"]
        return {"bytes": n * (4 * e + 8) + 4 * case["S"], "flops": 12 * n}
    if op in ("scan", "scan_train"):
        S, D = case["S"], case["D"]
        n = int(_offsets(case)[-1]) * D
        gates = 3 if case["gate"] else 2
        st = S * D * 4
        if op == "scan":
            return {"bytes": n * e * (gates + 1) + st * (1 + case["h0"]) + 8 * (S + 1), "flops": 12 * n}
        return {"bytes": n * e * (2 * gates + 2) + st * (2 + 2 * case["h0"]) + 8 * (S + 1), "flops": 40 * n}
    if op in ("norm", "norm_train"):
        n, D = case["N"] * case["D"], case["D"]
        if op == "norm":
            return {"bytes": 5 * n * e + 12 * D, "flops": 16 * n}
        return {"bytes": 10 * n * e + 24 * D, "flops": 56 * n}
    n = case["N"] * case["V"]
    return {"bytes": 2 * n * e + case["N"] * (case["k"] * 8 + 8), "flops": 8 * n}


# ---- inputs -----------------------------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(1000003 * seed + 17)
    dt = TDT[case["dtype"]]

    def rn(*shape, scale=1.0, shift=0.0, dtype=dt):
        return torch.randn(*shape, generator=g, device=DEV).mul_(scale).add_(shift).to(dtype)

    f32 = torch.float32
    st = dict(case=case)
    op = case["op"]
    if op == "step":
        S, D = case["S"], case["D"]
        # the gates are column blocks of one projection, as a block's input product leaves them
        st["p"] = rn(S, 3 * D, scale=1.2, shift=0.5)
        st["state"] = rn(case["slots"], D, scale=0.5, dtype=f32)
        st["slots"] = torch.randperm(case["slots"], generator=g, device=DEV)[:S].to(torch.int32)
    elif op in ("scan", "scan_train"):
        S, D = case["S"], case["D"]
        off = _offsets(case)
        T = int(off[-1])
        st["off"], st["T"] = torch.as_tensor(off, device=DEV), T
        st["zf"] = rn(T, D, scale=1.5, shift=2.0)       # memories of a few to a few hundred tokens
        st["g"] = rn(T, D)
        st["zo"] = rn(T, D) if case["gate"] else None
        st["h0"] = rn(S, D, scale=0.5, dtype=f32) if case["h0"] else None
        if op == "scan_train":
            st["dy"] = rn(T, D)
            st["dhT"] = rn(S, D, dtype=f32)
    elif op in ("norm", "norm_train"):
        N, D = case["N"], case["D"]
        st["x"], st["z"], st["u"] = rn(N, D, scale=2.0), rn(N, D), rn(N, D)
        st["w_post"], st["w_pre"] = rn(D, scale=0.1, shift=1.0, dtype=f32), rn(D, scale=0.1, shift=1.0, dtype=f32)
        st["scale"] = rn(D, scale=0.05, shift=0.3, dtype=f32)
        if op == "norm_train":
            st["dr"], st["dv"] = rn(N, D), rn(N, D)
    else:
        N, V, k = case["N"], case["V"], case["k"]
        z = torch.randn(N, V, generator=g, device=DEV).mul_(2.5)
        # the teacher agrees with the student up to noise; its k largest logits are kept, in 32 bits
        teacher = torch.randn(N, V, generator=g, device=DEV).add_(z)
        t, ids = torch.topk(teacher, k, dim=1)
        st["z"], st["t"], st["ids"] = z.to(dt), t.contiguous(), ids.to(torch.int32).contiguous()
        st["w"] = (torch.rand(N, generator=g, device=DEV) > 0.05).to(f32)     # padded frames count for nothing
        st["tau"] = 2.0
    if own:
        _plan(case, st)
    return st


def _plan(case, st):
    from directional_mdlstm_handwriting_amd.layer import BlockNorm, ScanState, SequenceScan, TopKDistill
    op = case["op"]
    if op == "step":
        st["own"] = ScanState(case["slots"], case["D"], case["dtype"], device=DEV)
        st["own"].state.copy_(st["state"])
        st["new"] = st["own"].state.clone()
    elif op in ("scan", "scan_train"):
        st["own"] = SequenceScan(st["off"], st["T"], case["D"], case["dtype"], reverse=case["reverse"])
    elif op in ("norm", "norm_train"):
        st["own"] = BlockNorm(case["N"], case["D"], case["dtype"], eps=EPS, device=DEV)
    else:
        st["own"] = TopKDistill(case["N"], case["V"], case["k"], case["dtype"], tau=st["tau"], device=DEV)


# ---- one pass ---------------------------------------------------------------------------------------------------

def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        o = st["own"]
        if op == "step":
            D = case["D"]
            p = st["p"]
            return [o.step(p[:, :D], p[:, D:2 * D], p[:, 2 * D:], slots=st["slots"], out=st["new"]), st["new"]]
        if op == "scan":
            return list(o.forward(st["zf"], st["g"], st["zo"], st["h0"]))
        if op == "scan_train":
            y, hT = o.forward(st["zf"], st["g"], st["zo"], st["h0"])
            grads = o.backward(st["zf"], st["g"], st["zo"], st["dy"], st["h0"], st["dhT"])
            return [t for t in (y, hT, *grads) if t is not None]
        if op == "norm":
            return list(o.forward(st["x"], st["z"], st["u"], st["w_post"], st["scale"], st["w_pre"]))
        if op == "norm_train":
            out = o.forward(st["x"], st["z"], st["u"], st["w_post"], st["scale"], st["w_pre"])
            grads = o.backward(st["x"], st["z"], st["u"], st["w_post"], st["scale"], st["w_pre"], st["dr"], st["dv"])
            return [*out, *grads]
        return list(o.run(st["z"], st["ids"], st["t"], st["w"]))
    if op == "step":
        return _plain_step(st)
    if op in ("scan", "scan_train"):
        return _plain_scan(st, op == "scan_train")
    if op in ("norm", "norm_train"):
        return _plain_norm(st, op == "norm_train")
    return _plain_distill(st)


def _plain_step(st):
    D, dt = st["case"]["D"], TDT[st["case"]["dtype"]]
    p = st["p"].float()
    f, g, o = torch.sigmoid(p[:, :D]), p[:, D:2 * D], torch.sigmoid(p[:, 2 * D:])
    idx = st["slots"].long()
    h = f * st["state"][idx] + torch.sigmoid(-p[:, :D]) * g
    new = st["state"].clone()
    new[idx] = h
    return [(o * h).to(dt), new]


def _affine_scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis, by doubling."""
    n, k = a.shape[0], 1
    while k < n:
        b = torch.cat([b[:k], torch.addcmul(b[k:], a[k:], b[:-k])])
        a = torch.cat([a[:k], a[k:] * a[:-k]])
        k *= 2
    return b


def _plain_scan(st, train):
    case = st["case"]
    dt = TDT[case["dtype"]]
    T, S = st["T"], case["S"]
    off = st["off"]
    live = off[1:] > off[:-1]
    s = torch.nonzero(live).flatten()
    first, last = off[:-1][s], off[1:][s] - 1
    if case["reverse"]:
        first, last = last, first

    def fwd_scan(a, b):
        return _affine_scan(a.flip(0), b.flip(0)).flip(0) if case["reverse"] else _affine_scan(a, b)

    def bwd_scan(a, b):
        return _affine_scan(a, b) if case["reverse"] else _affine_scan(a.flip(0), b.flip(0)).flip(0)

    zf, g = st["zf"].float(), st["g"].float()
    f, fc = torch.sigmoid(zf), torch.sigmoid(-zf)
    o = torch.sigmoid(st["zo"].float()) if st["zo"] is not None else None
    h0 = st["h0"] if st["h0"] is not None else torch.zeros(S, case["D"], device=DEV)
    a, b = f.clone(), fc * g
    b[first] += f[first] * h0[s]
    a[first] = 0
    h = fwd_scan(a, b)
    hT = h0.clone()
    hT[s] = h[last]
    y = (h if o is None else o * h).to(dt)
    if not train:
        return [y, hT]
    dy = st["dy"].float()
    prev = torch.roll(h, -1 if case["reverse"] else 1, 0)
    prev[first] = h0[s]
    # the gradient of h_t gathers f of the next token times its own
    a = torch.roll(f, 1 if case["reverse"] else -1, 0)
    a[last] = 0
    b = dy.clone() if o is None else o * dy
    b[last] += st["dhT"][s]
    lam = bwd_scan(a, b)
    out = [y, hT, (f * fc * (prev - g) * lam).to(dt), (fc * lam).to(dt)]
    if o is not None:
        out.append((dy * h * o * (1 - o)).to(dt))
    if st["h0"] is not None:
        dh0 = st["dhT"].clone()
        dh0[s] = f[first] * lam[first]
        out.append(dh0)
    return out


def _plain_norm(st, train):
    dt = TDT[st["case"]["dtype"]]
    x, z, u = st["x"].float(), st["z"].float(), st["u"].float()
    wp, sc, wn = st["w_post"], st["scale"], st["w_pre"]
    sig = torch.rsqrt(z.square().mean(1, keepdim=True) + EPS)
    zh = z * sig
    s = torch.sigmoid(u)
    r = x + sc * s * (zh * wp)
    rho = torch.rsqrt(r.square().mean(1, keepdim=True) + EPS)
    rh = r * rho
    out = [r.to(dt), (rh * wn).to(dt)]
    if not train:
        return out
    dr, dv = st["dr"].float(), st["dv"].float()
    t = dv * wn
    d = dr + rho * (t - rh * (t * rh).mean(1, keepdim=True))
    ds = d * s
    q = (ds * zh).sum(0)
    t = ds * sc * wp
    dz = sig * (t - zh * (t * zh).mean(1, keepdim=True))
    du = d * sc * (zh * wp) * s * (1 - s)
    return out + [d.to(dt), dz.to(dt), du.to(dt), sc * q, wp * q, (dv * rh).sum(0)]


def _plain_distill(st):
    dt, tau = TDT[st["case"]["dtype"]], st["tau"]
    z = st["z"].float() / tau
    m = z.max(1, keepdim=True).values
    e = torch.exp(z - m)
    tot = e.sum(1, keepdim=True)
    t = st["t"] / tau
    t = t - t.max(1, keepdim=True).values
    lp = t - torch.log(torch.exp(t).sum(1, keepdim=True))
    p = torch.exp(lp)
    ids = st["ids"].long()
    lq = z.gather(1, ids) - m - torch.log(tot)
    w = st["w"]
    loss = w * tau * tau * (p * (lp - lq)).sum(1)
    dz = (e / tot).scatter_add(1, ids, -p)
    return [loss, (dz * (tau * w)[:, None]).to(dt)]


# ---- the definitions in 64 bits ---------------------------------------------------------------------------------

def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    op = case["op"]
    with torch.no_grad():
        if op == "step":
            return _exact_step(st)
        if op in ("scan", "scan_train"):
            return _exact_scan(st, op == "scan_train")
        if op in ("norm", "norm_train"):
            return _exact_norm(st, op == "norm_train")
        return _exact_distill(st)


def _exact_step(st):
    D = st["case"]["D"]
    p = st["p"].double()
    new = st["state"].double()
    outs = []
    for i, slot in enumerate(st["slots"].tolist()):
        f = 1 / (1 + torch.exp(-p[i, :D]))
        new[slot] = f * new[slot] + (1 - f) * p[i, D:2 * D]
        outs.append(new[slot] / (1 + torch.exp(-p[i, 2 * D:])))
    return [torch.stack(outs), new]


def _exact_scan(st, train):
    """Token by token, all sequences that are long enough side by side."""
    case = st["case"]
    D, S, T = case["D"], case["S"], st["T"]
    off = st["off"].cpu().numpy()
    lens = off[1:] - off[:-1]
    order = np.argsort(-lens, kind="stable")
    count = np.searchsorted(-lens[order], -np.arange(1, int(lens.max()) + 1), side="right") if T else []
    begin = np.where(case["reverse"], off[1:] - 1, off[:-1])[order]
    begin = torch.as_tensor(begin, device=DEV)
    order = torch.as_tensor(order, device=DEV)
    step = -1 if case["reverse"] else 1
    f = 1 / (1 + torch.exp(-st["zf"].double()))
    fin = st["g"].double() * (1 - f)
    h = torch.zeros(S, D, dtype=torch.float64, device=DEV) if st["h0"] is None else st["h0"].double()[order]
    h_init = h.clone()
    hs = torch.empty_like(f)
    for i, n in enumerate(count):
        t = begin[:n] + step * i
        h[:n] = torch.addcmul(fin[t], f[t], h[:n])
        hs[t] = h[:n]
    del fin
    hT = torch.empty_like(h)
    hT[order] = h
    o = 1 / (1 + torch.exp(-st["zo"].double())) if st["zo"] is not None else None
    y = hs if o is None else hs * o
    if not train:
        return [y, hT]
    dy = st["dy"].double()
    lam = dy if o is None else dy * o          # becomes dL/dh, token by token from the last
    carry = st["dhT"].double()[order]
    dzo = None if o is None else dy * hs * o * (1 - o)
    if o is None:
        lam = lam.clone()
    for i in range(len(count) - 1, -1, -1):
        n = count[i]
        t = begin[:n] + step * i
        l = lam[t] + carry[:n]
        lam[t] = l
        carry[:n] = l * f[t]
    prev = torch.empty_like(hs)
    for i, n in enumerate(count):
        t = begin[:n] + step * i
        prev[t] = h_init[:n] if i == 0 else hs[t - step]
    dg = lam * (1 - f)
    dzf = dg * f * (prev - st["g"].double())
    out = [y, hT, dzf, dg]
    if o is not None:
        out.append(dzo)
    if st["h0"] is not None:
        dh0 = torch.empty_like(carry)
        dh0[order] = carry
        out.append(dh0)
    return out


def _exact_norm(st, train):
    """The outputs from the definition; the gradients from the Jacobians' rows written out per norm."""
    x, z, u = st["x"].double(), st["z"].double(), st["u"].double()
    wp, sc, wn = st["w_post"].double(), st["scale"].double(), st["w_pre"].double()
    D = x.shape[1]
    gate = 1 / (1 + torch.exp(-u))
    nz = torch.sqrt((z * z).sum(1) / D + EPS)[:, None]
    n = z / nz * wp
    r = x + gate * n * sc
    nr = torch.sqrt((r * r).sum(1) / D + EPS)[:, None]
    out = [r, r / nr * wn]
    if not train:
        return out
    dr, dv = st["dr"].double(), st["dv"].double()
    # v_i = w_i r_i / |r|: dv_i/dr_j = w_i (delta_ij / |r| - r_i r_j / (D |r|^3))
    d = dr + dv * wn / nr - r * (dv * wn * r).sum(1, keepdim=True) / (D * nr ** 3)
    dn = d * gate * sc
    dz = dn * wp / nz - z * (dn * wp * z).sum(1, keepdim=True) / (D * nz ** 3)
    du = d * n * sc * gate * (1 - gate)
    return out + [d, dz, du, (dn * z / nz).sum(0), (d * gate * n).sum(0), (dv * r / nr).sum(0)]


def _exact_distill(st):
    tau, w = st["tau"], st["w"].double()
    loss = torch.empty(w.shape[0], dtype=torch.float64, device=DEV)
    dz = torch.empty(st["z"].shape, dtype=torch.float64, device=DEV)
    for a in range(0, w.shape[0], 512):
        zz = st["z"][a:a + 512].double() / tau
        lse = torch.logsumexp(zz, 1, keepdim=True)
        tt = st["t"][a:a + 512].double() / tau
        lp = tt - torch.logsumexp(tt, 1, keepdim=True)
        ids = st["ids"][a:a + 512].long()
        q = torch.exp(zz - lse)
        loss[a:a + 512] = w[a:a + 512] * tau ** 2 * (torch.exp(lp) * (lp - zz.gather(1, ids) + lse)).sum(1)
        dz[a:a + 512] = q.scatter_add(1, ids, -torch.exp(lp)) * (w[a:a + 512] * tau)[:, None]
    return [loss, dz]
