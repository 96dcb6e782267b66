"""The sequence operators' classes on streams of the caller's choice: a `stream` that is not torch's current one, on the
first call of an object, while the current stream is busy; and calls that a graph capture is the first to make. Every
result has to be, bit for bit, what the same call gives on the current stream."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"

if torch.cuda.is_available():
    from directional_mdlstm_handwriting_amd.layer import BlockNorm, ScanState, SequenceScan, TopKDistill

OFF = np.array([5, 405, 405, 700, 900])     # rows in no sequence at both ends
T, D, S, N, V, K = 950, 48, 4, 300, 500, 6


def _data():
    g = torch.Generator(device=DEV).manual_seed(3)

    def rn(*s):
        return torch.randn(*s, generator=g, device=DEV)

    d = dict(zf=rn(T, D), g=rn(T, D), zo=rn(T, D), h0=rn(S, D), dy=rn(T, D), dhT=rn(S, D), x=rn(N, D), z=rn(N, D),
             u=rn(N, D), wa=rn(D), wb=rn(D), wc=rn(D), dr=rn(N, D), dv=rn(N, D), logits=rn(N, V), t=rn(N, K),
             w=torch.ones(N, device=DEV))
    d["ids"] = torch.stack([torch.randperm(V, generator=g, device=DEV)[:K] for _ in range(N)]).to(torch.int32)
    torch.cuda.synchronize()
    return d


def make(op):
    return {"scan": lambda: SequenceScan(OFF, T, D, device=DEV), "step": lambda: ScanState(N, D, device=DEV),
            "norm": lambda: BlockNorm(N, D, device=DEV), "distill": lambda: TopKDistill(N, V, K, device=DEV)}[op]()


def call(op, o, d, stream=None):
    if op == "scan":
        a = (d["zf"], d["g"], d["zo"])
        return (*o.forward(*a, d["h0"], stream=stream), *o.backward(*a, d["dy"], d["h0"], d["dhT"], stream=stream))
    if op == "step":
        return (o.step(d["x"], d["z"], d["u"], stream=stream), o.state)
    if op == "norm":
        a = (d["x"], d["z"], d["u"], d["wa"], d["wb"], d["wc"])
        return (*o.forward(*a, stream=stream), *o.backward(*a, d["dr"], d["dv"], stream=stream))
    return o.run(d["logits"], d["ids"], d["t"], d["w"], stream=stream)


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


OPS = ("scan", "step", "norm", "distill")


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("how", ["object", "handle", "context"])
def test_first_call_on_another_stream(op, how):
    print(f"[gpu] {op} stream as {how}", flush=True)
    d = _data()
    ref = [t.clone() for t in call(op, make(op), d)]
    sizes = sorted({t.numel() * t.element_size() for t in ref} | {D * 4})
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
    # and again, on a third stream and on the current one
    third = torch.cuda.Stream()
    for s in (third, None):
        if op == "step":
            o.state.zero_()
            torch.cuda.synchronize()
        _same(call(op, o, d, s), ref)


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
    for _ in range(3):
        if op == "step":
            o.state.zero_()
        _same(call(op, o, d), ref)
        if op == "step":
            o.state.zero_()
        graph.replay()
        _same(out, ref)


def test_step_holds_a_bounded_number_of_outputs():
    """Every batch size from 1 to 64: results that are still referenced stand, what the object holds stays within the
    outputs of its last sizes."""
    n, d = 64, 256
    print("[gpu] step sizes", flush=True)
    g = torch.Generator(device=DEV).manual_seed(9)
    z = [torch.randn(n, d, generator=g, device=DEV) for _ in range(3)]
    st = ScanState(n, d, device=DEV)
    keep = torch.empty_like(st.state)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    got = [st.step(*(t[:s] for t in z), out=keep) for s in range(1, n + 1)]
    whole = ScanState(n, d, device=DEV).step(*z).clone()
    torch.cuda.synchronize()
    for s, y in enumerate(got, 1):
        assert torch.equal(y, whole[:s]), s
    del got, y, whole
    assert torch.cuda.memory_allocated() - before <= ScanState.KEPT * n * d * 4


def test_captured_step_outlives_other_sizes():
    """The output that a graph writes is neither dropped nor handed out, however many sizes come between."""
    n, d = 40, 64
    print("[gpu] step captured", flush=True)
    g = torch.Generator(device=DEV).manual_seed(10)
    z = [torch.randn(n, d, generator=g, device=DEV) for _ in range(3)]
    st, eager = ScanState(n, d, device=DEV), ScanState(n, d, device=DEV)
    two = [t[:2] for t in z]
    st.step(*two)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = st.step(*two)
    place = y.data_ptr()
    del y
    for rep in range(3):
        st.state.zero_()
        eager.state.zero_()
        for s in range(1, n + 1):
            st.step(*(t[:s] for t in z))
            eager.step(*(t[:s] for t in z))
        junk = [torch.full((2, d), float(i), device=DEV) for i in range(64)]
        graph.replay()
        want = eager.step(*two)
        torch.cuda.synchronize()
        y = st.step(*two, out=torch.empty_like(st.state))
        assert y.data_ptr() == place
        st.state.copy_(eager.state)
        graph.replay()
        want = eager.step(*two)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(st.state, eager.state), rep
        assert all((j == i).all() for i, j in enumerate(junk)), rep
        del y
