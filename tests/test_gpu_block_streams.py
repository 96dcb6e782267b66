"""Linear attention, its stepped states, dropout and the vocabulary's cross entropy on streams of the caller's choice: a
`stream` that is not torch's current one, on the first call of an object, while the current stream is busy; two objects on
two streams at once; calls that a graph capture is the first to make, replayed with eager work between; and what the classes
refuse. Every result has to be, bit for bit, what the same call gives on the current stream."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"

if torch.cuda.is_available():
    from directional_mdlstm_handwriting_amd.layer import AttentionState, Dropout, LinearAttention, VocabLoss

OFF = np.array([5, 405, 405, 700, 1400])     # rows in no sequence at both ends
T, H, DK, DV, S, N, D, V = 1450, 3, 40, 64, 4, 300, 48, 700
DEC = [0.9, 0.99, 0.999]


def _data(dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(3)

    def rn(*s, dt=dtype):
        return torch.randn(*s, generator=g, device=DEV).to(dt)

    d = dict(q=rn(T, H * DK), k=rn(T, H * DK), v=rn(T, H * DV), dy=rn(T, H * DV), h0=rn(S, H, DK, DV, dt=torch.float32),
             dhT=rn(S, H, DK, DV, dt=torch.float32), x=rn(N, D), r=rn(N, D), W=rn(V, D), w=torch.ones(N, device=DEV))
    d["ids"] = torch.randint(0, V, (N,), generator=g, device=DEV, dtype=torch.int32)
    torch.cuda.synchronize()
    return d


def make(op):
    return {"attn": lambda: LinearAttention(OFF, T, H, DK, DV, DEC, "bf16", device=DEV),
            "step": lambda: AttentionState(N, H, DK, DV, DEC, "bf16", device=DEV),
            "drop": lambda: Dropout(N, D, 0.3, "bf16", seed=11, device=DEV),
            "vocab": lambda: VocabLoss(N, D, V, "bf16", device=DEV)}[op]()


def call(op, o, d, stream=None):
    if op == "attn":
        a = (d["q"], d["k"], d["v"])
        return (*o.forward(*a, d["h0"], stream=stream), *o.backward(*a, d["dy"], d["h0"], d["dhT"], stream=stream))
    if op == "step":
        return (o.step(d["q"][:N], d["k"][:N], d["v"][:N], stream=stream), o.state)
    if op == "drop":
        return (o.forward(d["x"], d["r"], stream=stream), o.backward(d["x"], stream=stream))
    return (*o.run(d["x"], d["W"], d["ids"], d["w"], stream=stream),)


class Busy:
    """Some 30 ms of products on the current stream, and then writes into a freed block of every size in use."""

    def __init__(self):
        self.m = torch.randn(8192, 8192, device=DEV).to(torch.bfloat16)

    def __call__(self, blocks):
        torch.cuda.synchronize()
        held = [torch.empty(b, dtype=torch.uint8, device=DEV) for b in blocks for _ in range(8)]
        for _ in range(30):
            self.m @ self.m
        for b in held:
            b.fill_(0x7F)


def _same(got, ref):
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(got, ref)):
        assert torch.equal(a, b), i


OPS = ("attn", "step", "drop", "vocab")


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("how", ["object", "handle", "context"])
def test_first_call_on_another_stream(op, how):
    print(f"[gpu] {op} stream as {how}", flush=True)
    d = _data()
    ref = [t.clone() for t in call(op, make(op), d)]
    sizes = sorted({t.numel() * t.element_size() for t in ref})
    busy, side = Busy(), torch.cuda.Stream()
    for made_before in (True, False):
        o = make(op) if made_before else None
        busy(sizes)
        if o is None:
            o = make(op)            # made behind the current stream's work, used at once on another
        if how == "context":
            with torch.cuda.stream(side):
                got = call(op, o, d)
        else:
            got = call(op, o, d, side if how == "object" else side.cuda_stream)
        _same(got, ref)
    third = torch.cuda.Stream()
    for s in (third, None):
        if op == "step":
            o.state.zero_()
            torch.cuda.synchronize()
        _same(call(op, o, d, s), ref)


@pytest.mark.parametrize("op", OPS)
def test_two_objects_at_once(op):
    """Two objects on two streams, their calls in turn: each as alone."""
    print(f"[gpu] two {op} at once", flush=True)
    d = _data()
    e = {k: t.flip(0).contiguous() if k != "ids" else (V - 1 - t) for k, t in d.items()}
    ref = [[t.clone() for t in call(op, make(op), x)] for x in (d, e)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    objs = [make(op), make(op)]
    torch.cuda.synchronize()
    for _ in range(3):
        if op == "step":
            for o in objs:
                o.state.zero_()
            torch.cuda.synchronize()
        got = [call(op, o, x, s) for o, x, s in zip(objs, (d, e), streams)]
        for a, b in zip(got, ref):
            _same(a, b)


@pytest.mark.parametrize("op", OPS)
def test_a_capture_is_the_first_to_call(op):
    """The capture's outputs are the graph's own: eager calls of the same object neither find nor disturb them."""
    print(f"[gpu] {op} captured first", flush=True)
    d = _data()
    ref = [t.clone() for t in call(op, make(op), d)]
    o = make(op)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(op, o, d)
    for _ in range(4):
        if op == "step":
            o.state.zero_()
        _same(call(op, o, d), ref)
        junk = [torch.full((1 << 20,), float("nan"), device=DEV) for _ in range(4)]
        if op == "step":
            o.state.zero_()
        graph.replay()
        _same(out, ref)
        del junk


def test_two_graphs_of_one_vocabulary_loss():
    """Graphs of the loss alone and of the loss with gradients, captured after eager calls, replayed in turn on new inputs:
    each keeps its own workspace, whichever ran last."""
    d = _data()
    o, fresh = make("vocab"), make("vocab")
    o.run(d["x"], d["W"], d["ids"], d["w"], want_grads=False)
    x = d["x"].clone()
    alone, both = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(alone):
        loss_a = o.run(x, d["W"], d["ids"], d["w"], want_grads=False)[0]
    o.run(x, d["W"], d["ids"], d["w"])
    with torch.cuda.graph(both):
        out = o.run(x, d["W"], d["ids"], d["w"])
    for i in range(4):
        x.copy_(d["x"] * (1 + i))
        ref = [t.clone() for t in fresh.run(x, d["W"], d["ids"], d["w"])]
        junk = [torch.full((1 << 22,), float("nan"), device=DEV) for _ in range(2)]
        for g in ((alone, both) if i % 2 else (both, alone)):
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(loss_a, ref[0])
        _same(out, ref)
        del junk


def test_results_repeat_bit_for_bit():
    """Fixed orders of summation: the same call gives the same bits, 20 times over."""
    d = _data()
    for op in ("attn", "vocab", "drop"):
        o = make(op)
        ref = [t.clone() for t in call(op, o, d)]
        for _ in range(20):
            _same(call(op, o, d), ref)


def test_offsets_that_do_not_ascend_stay_inside():
    """Unchecked device offsets beyond the tensors, descending or negative: unspecified results, and nothing outside the
    outputs is written. The tensors lie inside larger ones whose borders must stand."""
    d = _data()
    rows = 64
    big = {n: torch.full((T + 2 * rows, t.shape[1]), 3.0, dtype=t.dtype, device=DEV) for n, t in d.items()
           if n in ("q", "k", "v", "dy")}
    for n, t in big.items():
        t[rows:-rows] = d[n]
    for bad in ([0, 2 * T, T + 7], [T, 10, 900], [-50, 30, T], [2 ** 40, 2 ** 41, 2 ** 42], [900, 800, 700], [-5, -4, -3]):
        off = torch.tensor(bad, dtype=torch.int64, device=DEV)
        o = LinearAttention(off, T, H, DK, DV, DEC, "bf16", device=DEV)
        outs = {}
        for n, c in (("y", H * DV), ("dq", H * DK), ("dk", H * DK), ("dv", H * DV)):
            outs[n] = torch.full((T + 2 * rows, c), 3.0, dtype=torch.bfloat16, device=DEV)
            setattr(o, n, outs[n][rows:-rows])
        h0 = torch.zeros(2, H, DK, DV, device=DEV)
        a = [big[n][rows:-rows] for n in ("q", "k", "v")]
        o.forward(*a, h0)
        o.backward(*a, big["dy"][rows:-rows], h0, h0)
        torch.cuda.synchronize()
        for n, t in outs.items():
            assert (t[:rows] == 3).all() and (t[-rows:] == 3).all(), (bad, n)


def test_classes_refuse():
    d = _data()
    at = make("attn")
    with pytest.raises(ValueError):
        at.forward(d["q"][:-1], d["k"], d["v"])
    with pytest.raises(ValueError):
        at.forward(d["q"].float(), d["k"], d["v"])
    with pytest.raises(ValueError):
        at.forward(d["q"], d["k"], d["v"].t().contiguous().t())
    with pytest.raises(ValueError):
        at.forward(d["q"], d["k"], d["v"], d["h0"][:1])
    with pytest.raises(ValueError):
        LinearAttention(OFF, T, H, DK, DV, [0.5, 0.5], device=DEV)
    with pytest.raises(ValueError):
        LinearAttention(OFF, T - 100, H, DK, DV, DEC, device=DEV)
    with pytest.raises(ValueError):
        LinearAttention(OFF, T, H, DK, DV, torch.ones(2, device=DEV), device=DEV)
    st = make("step")
    with pytest.raises(ValueError):
        st.step(d["q"][:4], d["k"][:3], d["v"][:4])
    with pytest.raises(ValueError):
        st.step(d["q"][:4], d["k"][:4], d["v"][:4], slots=torch.arange(4, device=DEV))
    for p in (1.0, -0.1, 0.9999999, float("nan")):
        with pytest.raises(ValueError):
            Dropout(N, D, p, device=DEV)
    dr = make("drop")
    with pytest.raises(ValueError):
        dr.forward(d["x"], d["r"][:-1])
    with pytest.raises(ValueError):
        dr.forward(d["x"], rng=torch.zeros(2, device=DEV))
    vl = make("vocab")
    with pytest.raises(ValueError):
        vl.run(d["x"], d["W"].t().contiguous().t(), d["ids"])
    with pytest.raises(ValueError):
        vl.run(d["x"], d["W"], d["ids"].long())


def test_stepped_outputs_of_other_sizes_stand():
    d = _data()
    st = make("step")
    keep = torch.empty_like(st.state)
    got = [st.step(d["q"][:s], d["k"][:s], d["v"][:s], out=keep) for s in range(1, 30)]
    whole = make("step").step(d["q"][:N], d["k"][:N], d["v"][:N]).clone()
    torch.cuda.synchronize()
    for s, y in enumerate(got, 1):
        assert torch.equal(y, whole[:s]), s


def test_tokens_past_two_to_the_31_elements():
    """Rows whose elements lie past 2^31 of a tensor's start, as late rows of a long cache do: the last sequence as alone."""
    rows, h, dk = 2200, 1, 128
    ld = 1 << 20
    base = torch.zeros(rows * ld + 3 * dk, dtype=torch.bfloat16, device=DEV)
    q, k, v = (base[i * dk:].as_strided((rows, dk), (ld, 1)) for i in range(3))
    g = torch.Generator(device=DEV).manual_seed(1)
    for t in (q, k, v):
        t.copy_(torch.randn(rows, dk, generator=g, device=DEV))
    off = np.array([0, 2100, rows])
    o = LinearAttention(off, rows, h, dk, dk, [0.99], "bf16", device=DEV)
    dy = torch.randn(rows, dk, generator=g, device=DEV).to(torch.bfloat16)
    got = [t for t in (*o.forward(q, k, v), *o.backward(q, k, v, dy)) if t is not None]
    alone = LinearAttention(np.array([0, 100]), 100, h, dk, dk, [0.99], "bf16", device=DEV)
    a = [t[2100:].contiguous() for t in (q, k, v)]
    ref = [t for t in (*alone.forward(*a), *alone.backward(*a, dy[2100:])) if t is not None]
    torch.cuda.synchronize()
    assert torch.equal(got[0][2100:], ref[0]) and torch.equal(got[1][1], ref[1][0])
    for x, y in zip(got[2:], ref[2:]):
        assert torch.equal(x[2100:], y)
