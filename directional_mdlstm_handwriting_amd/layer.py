"""Device-side orchestration of the C ABI with torch-allocated buffers.

torch supplies device memory and the stream; every computation is a libmdlstm
kernel. ``PackedLayer`` holds one layout's descriptor and a layer's workspace
and runs scatter -> forward -> direction sum/un-pack, and the backward.
``PackedStack`` chains three levels with block-strided convolutions, each
level re-packed from the previous level's output sizes ("No Padding Please",
§V-A: packing happens just before each MDLSTM layer). ``CTCHead`` runs the
model head (height collapse, shared fully-connected layer, CTC loss) on the
last level's output. ``SequenceScan`` and ``ScanState`` run the gated linear
recurrence along the rows or frames of the packed examples, whole sequences
at once or a token at a time; ``BlockNorm`` the norms around such a block with
its gate and residual; ``TopKDistill`` the distillation loss of its logits.
"""

from __future__ import annotations

import contextlib
import dataclasses
from typing import List, Optional, Sequence

import numpy as np
import torch

from . import (MDL_BF16, MDL_CELL_LEAKY_LP, MDL_CELL_MDLSTM, MDL_F32, MDL_PACK_ALG1, MDL_PACK_EXACT, MDL_PACK_PADDED, Layout, mdl_backward,
               mdl_blockconv_backward, mdl_blockconv_forward, mdl_blockconv_workspace_size, mdl_dirsum_unpack, mdl_forward, mdl_forward_dirsum,
               mdl_layout_device_size, mdl_layout_rects, mdl_layout_upload, mdl_pack, mdl_pack_level, mdl_scatter, mdl_workspace_size,
               mdl_ctc_head, mdl_ctc_workspace_size, mdl_scan_backward, mdl_scan_forward, mdl_scan_step, mdl_scan_workspace_size,
               mdl_blocknorm_backward, mdl_blocknorm_forward, mdl_blocknorm_workspace_size, mdl_distill, _stream)


def _dev(a, device, dtype=torch.float32):
    if isinstance(a, torch.Tensor):
        return a.to(device=device, dtype=dtype).contiguous()
    return torch.as_tensor(np.ascontiguousarray(a), dtype=dtype, device=device).contiguous()


@dataclasses.dataclass
class DeviceParams:
    """A layer's weights on the device; Vl, Vu (the memory-state projections) only for the Leaky LP cell."""
    Wx: torch.Tensor
    Ul: torch.Tensor
    Uu: torch.Tensor
    b: torch.Tensor
    Vl: Optional[torch.Tensor] = None
    Vu: Optional[torch.Tensor] = None

    @staticmethod
    def from_host(P, device) -> "DeviceParams":
        V = [_dev(getattr(P, n), device) if getattr(P, n, None) is not None else None for n in ("Vl", "Vu")]
        return DeviceParams(_dev(P.Wx, device), _dev(P.Ul, device), _dev(P.Uu, device), _dev(P.b, device), *V)

    @property
    def cell(self):
        return MDL_CELL_MDLSTM if self.Vl is None else MDL_CELL_LEAKY_LP

    @property
    def C(self):
        return int(self.Wx.shape[1])

    @property
    def H(self):
        return int(self.Ul.shape[1])


PACK_MODES = {"packed": MDL_PACK_ALG1, "padded": MDL_PACK_PADDED, "exact": MDL_PACK_EXACT}


class DeviceLayout:
    """A packed layout plus its uploaded device descriptor."""

    def __init__(self, heights, widths, canvas_w_min: int, sep: int = 1, mode: str = "packed",
                 device: str = "cuda", stream=None, layout: Optional[Layout] = None):
        """Packs (heights, widths), or takes an already built `layout` (heights and widths then unused)."""
        if layout is None:
            if mode not in PACK_MODES:
                raise ValueError(f"unknown packing mode {mode!r}; one of {sorted(PACK_MODES)}")
            layout = mdl_pack(heights, widths, canvas_w_min, sep, PACK_MODES[mode])
        self.layout: Layout = layout
        self.device = device
        nbytes, self.eid_off, self.border_off = mdl_layout_device_size(self.layout)
        self.desc = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.desc_bytes = nbytes
        mdl_layout_upload(self.layout, self.desc, nbytes, stream)

    @property
    def info(self):
        return self.layout.info

    def sizes(self):
        """(heights, widths) of the examples, input order."""
        _, real = mdl_layout_rects(self.layout)
        return real[:, 2].copy(), real[:, 3].copy()

    def row_offsets(self) -> np.ndarray:
        """Offsets (int64) of every image row of every example in the flat [h][w][K] tensors, as sequences of w
        tokens: what a SequenceScan along the rows takes."""
        h, w = self.sizes()
        return np.concatenate([[0], np.cumsum(np.repeat(w.astype(np.int64), h))])

    def frame_offsets(self) -> np.ndarray:
        """Offsets (int64) of the examples' frames, one sequence of w tokens per example: the sequences of a
        height-collapsed [sum w][K] tensor."""
        _, w = self.sizes()
        return np.concatenate([[0], np.cumsum(w.astype(np.int64))])

    def device_maps(self):
        Hc, Wc = self.layout.Hc, self.layout.Wc
        P = Hc * Wc
        eid = self.desc[self.eid_off:self.eid_off + 4 * P].view(torch.int32).reshape(Hc, Wc)
        border = self.desc[self.border_off:self.border_off + P].reshape(Hc, Wc)
        return eid, border


class PackedLayer:
    """One 4-direction MDLSTM layer on one device layout."""

    def __init__(self, dl: DeviceLayout, C: int, H: int, x_dtype: str = "f32"):
        self.dl, self.C, self.H = dl, C, H
        self.x_dtype = MDL_BF16 if x_dtype == "bf16" else MDL_F32
        info = dl.info
        dev = dl.device
        self.ws_bytes = mdl_workspace_size(dl.layout, C, H)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)
        tdt = torch.bfloat16 if self.x_dtype == MDL_BF16 else torch.float32
        self.x_canvas = torch.empty(info["canvas_h"], info["canvas_w"], C, dtype=tdt, device=dev)
        self.h_dirs = torch.empty(4, info["canvas_h"], info["canvas_w"], H, dtype=torch.float32, device=dev)
        self.y = torch.empty(info["real_pixels"] * H, dtype=torch.float32, device=dev)

    def scatter(self, x_flat: torch.Tensor, stream=None):
        mdl_scatter(self.dl.layout, self.dl.desc, x_flat, self.C, self.x_dtype, self.x_canvas, stream)

    def forward(self, P: DeviceParams, stream=None):
        """The cell follows the parameters: the Leaky LP cell when they carry Vl, Vu."""
        mdl_forward(self.dl.layout, self.dl.desc, self.x_canvas, self.x_dtype, self.C, self.H, P.cell, P.Wx, P.Ul,
                    P.Uu, P.b, P.Vl, P.Vu, self.h_dirs, self.ws, self.ws_bytes, stream)

    def dirsum(self, stream=None):
        mdl_dirsum_unpack(self.dl.layout, self.dl.desc, self.h_dirs, self.H, self.y, stream)

    def forward_dirsum(self, P: DeviceParams, stream=None):
        """forward() and dirsum() in one call, the direction sum overlapping the wavefront where it can."""
        mdl_forward_dirsum(self.dl.layout, self.dl.desc, self.x_canvas, self.x_dtype, self.C, self.H, P.cell, P.Wx,
                           P.Ul, P.Uu, P.b, P.Vl, P.Vu, self.h_dirs, self.y, self.ws, self.ws_bytes, stream)

    def backward(self, P: DeviceParams, grads: "LayerGrads", dy_flat=None, dh_dirs=None, dx_flat=None,
                 dx_canvas=None, stream=None):
        mdl_backward(self.dl.layout, self.dl.desc, self.x_canvas, self.x_dtype, self.C, self.H, P.cell, P.Wx, P.Ul,
                     P.Uu, P.Vl, P.Vu, self.h_dirs, dy_flat, dh_dirs, dx_flat, dx_canvas, grads.dWx, grads.dUl,
                     grads.dUu, grads.db, grads.dVl, grads.dVu, self.ws, self.ws_bytes, stream)


@dataclasses.dataclass
class LayerGrads:
    """Weight gradients; dVl, dVu for the Leaky LP cell only."""
    dWx: torch.Tensor
    dUl: torch.Tensor
    dUu: torch.Tensor
    db: torch.Tensor
    dVl: Optional[torch.Tensor] = None
    dVu: Optional[torch.Tensor] = None

    @staticmethod
    def like(P: DeviceParams) -> "LayerGrads":
        V = [torch.empty_like(t) if t is not None else None for t in (P.Vl, P.Vu)]
        return LayerGrads(torch.empty_like(P.Wx), torch.empty_like(P.Ul), torch.empty_like(P.Uu),
                          torch.empty_like(P.b), *V)


def flat_input(xs: Sequence[np.ndarray], x_dtype: str, device) -> torch.Tensor:
    """Concatenate per-example [h][w][C] tensors (bf16-exact values for 'bf16')."""
    flat = np.concatenate([np.asarray(x, np.float32).reshape(-1) for x in xs])
    t = torch.as_tensor(flat, device=device)
    return t.to(torch.bfloat16) if x_dtype == "bf16" else t


class PackedStack:
    """MDLSTM -> block conv -> MDLSTM -> block conv -> MDLSTM, re-packed per level."""

    def __init__(self, heights, widths, C: int, Hs: Sequence[int], couts: Sequence[int], canvas_w_min: Sequence[int],
                 sep: int = 1, kh: int = 2, kw: int = 4, device: str = "cuda"):
        self.kh, self.kw = kh, kw
        self.levels: List[PackedLayer] = []
        c_in = C
        dl = DeviceLayout(heights, widths, canvas_w_min[0], sep, "packed", device)
        for lvl, H in enumerate(Hs):
            self.levels.append(PackedLayer(dl, c_in, H))
            if lvl + 1 < len(Hs):
                # the next level's examples: the block conv's output sizes, packed again (the library's rule)
                nxt = mdl_pack_level(dl.layout, kh, kw, canvas_w_min[lvl + 1], sep, MDL_PACK_ALG1)
                dl = DeviceLayout(None, None, 0, device=device, layout=nxt)
                c_in = couts[lvl]
        self.couts = list(couts)
        self.conv_ws = []
        self.dx_canvas = []
        self.dh_dirs = []
        for lvl in range(len(Hs) - 1):
            lk, lk1 = self.levels[lvl], self.levels[lvl + 1]
            nb = mdl_blockconv_workspace_size(lk1.dl.layout, lk.H, kh, kw, self.couts[lvl])
            self.conv_ws.append((torch.empty(max(nb, 4), dtype=torch.uint8, device=device), nb))
            self.dx_canvas.append(torch.empty_like(lk1.x_canvas, dtype=torch.float32))
            self.dh_dirs.append(torch.empty_like(lk.h_dirs))

    @property
    def level_sizes(self):
        """Per level, the (heights, widths) of its examples."""
        return [lay.dl.sizes() for lay in self.levels]

    def forward(self, x_flat, params: Sequence[DeviceParams], convs, stream=None):
        L0 = self.levels[0]
        L0.scatter(x_flat, stream)
        for lvl, lay in enumerate(self.levels):
            lay.forward(params[lvl], stream)
            if lvl + 1 < len(self.levels):
                nxt = self.levels[lvl + 1]
                W, b = convs[lvl]
                mdl_blockconv_forward(lay.dl.layout, lay.dl.desc, nxt.dl.layout, nxt.dl.desc, lay.h_dirs, lay.H,
                                      self.kh, self.kw, W, b, self.couts[lvl], nxt.x_canvas, stream)
        self.levels[-1].dirsum(stream)
        return self.levels[-1].y

    def backward(self, params, convs, dy_flat, lgrads: Sequence[LayerGrads], cgrads, dx_flat=None, stream=None):
        n = len(self.levels)
        for lvl in range(n - 1, -1, -1):
            lay = self.levels[lvl]
            kwargs = {}
            if lvl == n - 1:
                kwargs["dy_flat"] = dy_flat
            else:
                kwargs["dh_dirs"] = self.dh_dirs[lvl]
            if lvl > 0:
                kwargs["dx_canvas"] = self.dx_canvas[lvl - 1]
            else:
                kwargs["dx_flat"] = dx_flat
            lay.backward(params[lvl], lgrads[lvl], stream=stream, **kwargs)
            if lvl > 0:
                prev = self.levels[lvl - 1]
                W, _ = convs[lvl - 1]
                dW, db = cgrads[lvl - 1]
                wsb, nb = self.conv_ws[lvl - 1]
                mdl_blockconv_backward(prev.dl.layout, prev.dl.desc, lay.dl.layout, lay.dl.desc, prev.h_dirs, prev.H,
                                       self.kh, self.kw, W, self.couts[lvl - 1], self.dx_canvas[lvl - 1],
                                       self.dh_dirs[lvl - 1], dW, db, wsb, nb, stream)


class CTCHead:
    """The model head on a layout's direction-summed output: rows summed into frames, one fully-connected layer
    to K classes (0 = blank), CTC loss per example and the gradients of their sum (mdl_ctc_head). Labels are
    fixed at construction: one sequence of classes 1..K-1 per example of the layout, in input order."""

    def __init__(self, dl: DeviceLayout, H: int, K: int, labels: Sequence[Sequence[int]],
                 max_label: Optional[int] = None):
        n = dl.info["n"]
        if len(labels) != n:
            raise ValueError(f"need one label per example ({n}), got {len(labels)}")
        self.dl, self.K, self.H = dl, K, H
        flat = np.array([c for lab in labels for c in lab], dtype=np.int32)
        off = np.zeros(n + 1, dtype=np.int32)
        off[1:] = np.cumsum([len(lab) for lab in labels])
        self.max_label = int(max(len(lab) for lab in labels)) if max_label is None else int(max_label)
        dev = dl.device
        self.n_labels = int(flat.size)
        self.labels = torch.as_tensor(flat if flat.size else np.zeros(1, np.int32), device=dev)
        self.label_off = torch.as_tensor(off, device=dev)
        self.ws_bytes = mdl_ctc_workspace_size(dl.layout, H, K, self.max_label)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)
        self.loss = torch.empty(n, dtype=torch.float32, device=dev)
        self.dy = torch.empty(dl.info["real_pixels"] * H, dtype=torch.float32, device=dev)

    def run(self, y_flat: torch.Tensor, Wfc: torch.Tensor, bfc: torch.Tensor, dWfc: Optional[torch.Tensor] = None,
            dbfc: Optional[torch.Tensor] = None, want_dy: bool = True, stream=None):
        """Loss per example into self.loss, the gradient of the summed loss with respect to y_flat into self.dy
        (if want_dy), dWfc / dbfc if given."""
        mdl_ctc_head(self.dl.layout, self.dl.desc, y_flat, self.H, Wfc, bfc, self.K, self.labels, self.label_off,
                     self.n_labels, self.max_label, self.loss, self.dy if want_dy else None, dWfc, dbfc, self.ws,
                     self.ws_bytes, stream)
        return self.loss


_DTYPES = {"f32": (MDL_F32, torch.float32), "bf16": (MDL_BF16, torch.bfloat16)}


def _x_dtype(name: str):
    if name not in _DTYPES:
        raise ValueError(f"unknown dtype {name!r}; one of {sorted(_DTYPES)}")
    return _DTYPES[name]


def _device(device) -> torch.device:
    d = torch.device(device)
    if d.type == "cuda" and d.index is None:
        d = torch.device("cuda", torch.cuda.current_device())
    return d


def _rows(name: str, t: torch.Tensor, shape, dtype, device) -> int:
    """Checks a tensor of rows (any row stride, elements of a row adjacent) and returns its row stride."""
    if t.dtype != dtype or t.shape != shape or t.device != device:
        raise ValueError(f"{name}: need {shape} {dtype} on {device}, got {tuple(t.shape)} {t.dtype} on {t.device}")
    ld, inner = t.stride()
    if inner == 1 or shape[1] <= 1:
        if ld >= shape[1]:
            return ld
        if shape[0] <= 1:
            return shape[1]
    raise ValueError(f"{name}: need adjacent elements within a row and rows that do not overlap")


def _same_rows(names, ts, shape, dtype, device) -> int:
    """_rows of several tensors that share one row stride (column blocks of one matrix, or separate ones); None is
    left out. With one row, or none, the strides do not matter."""
    ld = None
    for n, t in zip(names, ts):
        if t is None:
            continue
        s = _rows(n, t, shape, dtype, device)
        if ld is None or shape[0] <= 1:
            ld = s
        elif s != ld:
            raise ValueError(f"{', '.join(names)}: one row stride for all, got {ld} and {s}")
    return ld


def _full(name: str, t: Optional[torch.Tensor], shape, dtype, device):
    """Checks a contiguous tensor (None passes)."""
    if t is not None and (t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous()):
        raise ValueError(f"{name}: need contiguous {shape} {dtype} on {device}, got {tuple(t.shape)} {t.dtype} on "
                         f"{t.device}")


def _here(device: torch.device):
    if torch.cuda.current_device() != device.index:
        raise ValueError(f"buffers are on {device}, the current device is cuda:{torch.cuda.current_device()}")


def _on(handle: int, device: torch.device):
    """The context in which torch allocates and fills on the stream of this handle."""
    if handle == _stream(None):
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(handle, device=device))


class _Buffers:
    """Buffers that an operator keeps from call to call, ordered with the calls whatever their stream. Those of the
    constructor are allocated and filled on torch's current stream: the first call on any other stream waits for that.
    Those that only some calls need are allocated and filled on the stream of the first such call. From then on the
    buffers are as any tensor's: the caller orders calls of one object that run on different streams. In a graph capture
    nothing is waited for (torch.cuda.graph synchronizes before it), and a buffer that the capture is the first to need
    belongs to the graph: the object does not keep it."""

    def _made(self, device: torch.device):
        self.device = device
        home = torch.cuda.current_stream(device)
        self._ready = None
        with torch.cuda.device(device):
            if not torch.cuda.is_current_stream_capturing():
                self._ready = home.record_event()
        self._joined = {home.cuda_stream}

    def _launch(self, stream) -> int:
        """The handle of the stream that a call launches on, with the constructor's work before it."""
        _here(self.device)
        handle = _stream(stream)
        if handle not in self._joined and self._ready is not None:
            with _on(handle, self.device):
                if not torch.cuda.is_current_stream_capturing():
                    torch.cuda.current_stream().wait_event(self._ready)
                    self._joined.add(handle)
        return handle

    def _capturing(self, handle: int) -> bool:
        with _on(handle, self.device):
            return torch.cuda.is_current_stream_capturing()

    def _new(self, handle: int, shape, dtype, zero: bool):
        """(tensor, whether to keep it)"""
        with _on(handle, self.device):
            make = torch.zeros if zero else torch.empty
            return make(shape, dtype=dtype, device=self.device), not torch.cuda.is_current_stream_capturing()


class SequenceScan(_Buffers):
    """The gated linear recurrence (mdl_scan_forward / _backward) over the sequences given by `seq_off` among T rows
    of D channels. seq_off: S + 1 ascending offsets, from the host (checked) or an int64 device tensor (taken as it
    is). Holds the outputs, the gradients and the workspace: a forward's results stand until the next forward, and a
    backward belongs to the forward before it."""

    def __init__(self, seq_off, T: int, D: int, x_dtype: str = "f32", reverse: bool = False, device: str = "cuda"):
        on_device = isinstance(seq_off, torch.Tensor) and seq_off.is_cuda
        self.device = seq_off.device if on_device else _device(device)
        if on_device:
            if seq_off.dtype != torch.int64 or seq_off.dim() != 1 or seq_off.numel() < 2:
                raise ValueError("seq_off: need S + 1 int64 offsets")
            self.off = seq_off.contiguous()
        else:
            host = np.asarray(seq_off, dtype=np.int64).reshape(-1)
            if host.size < 2 or host[0] < 0 or host[-1] > T or (np.diff(host) < 0).any():
                raise ValueError("seq_off: need S + 1 offsets that ascend within [0, T]")
            self.off = torch.as_tensor(host, device=self.device)
        self.S, self.T, self.D, self.reverse = int(self.off.numel()) - 1, int(T), int(D), int(bool(reverse))
        self.x_dtype, self.tdt = _x_dtype(x_dtype)
        self.ws_bytes = mdl_scan_workspace_size(self.T, self.D, self.x_dtype)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        # zeros: rows in no sequence are never written
        self.y = torch.zeros(self.T, self.D, dtype=self.tdt, device=self.device)
        self.hT = torch.empty(self.S, self.D, dtype=torch.float32, device=self.device)
        self.dzf = self.dg = self.dzo = self.dh0 = None
        self._made(self.device)

    def _inputs(self, zf, g, zo, h0):
        ldz = _same_rows(("zf", "g", "zo"), (zf, g, zo), (self.T, self.D), self.tdt, self.device)
        _full("h0", h0, (self.S, self.D), torch.float32, self.device)
        return ldz

    def forward(self, zf, g, zo=None, h0=None, stream=None):
        """(y, hT): zf, g, zo [T][D] at one row stride, h0 [S][D] float32. Neither the object's own y nor its hT can be an
        input: the last states of one piece of a long sequence are copied, or another object takes the next piece."""
        stream = self._launch(stream)
        ldz = self._inputs(zf, g, zo, h0)
        mdl_scan_forward(self.off, self.S, self.T, self.D, self.x_dtype, self.reverse, zf, g, zo, ldz, h0, self.y,
                         self.D, self.hT, self.ws, self.ws_bytes, stream)
        return self.y, self.hT

    def backward(self, zf, g, zo, dy, h0=None, dhT=None, stream=None):
        """(dzf, dg, dzo, dh0), dzo None without zo and dh0 None without h0, of the forward() just run on the same
        inputs."""
        stream = self._launch(stream)
        ldz = self._inputs(zf, g, zo, h0)
        ldy = _rows("dy", dy, (self.T, self.D), self.tdt, self.device)
        _full("dhT", dhT, (self.S, self.D), torch.float32, self.device)
        dzf, dg = self._grad("dzf", self.y, stream), self._grad("dg", self.y, stream)
        dzo = None if zo is None else self._grad("dzo", self.y, stream)
        dh0 = None if h0 is None else self._grad("dh0", self.hT, stream)
        mdl_scan_backward(self.off, self.S, self.T, self.D, self.x_dtype, self.reverse, zf, g, zo, ldz, h0, dy, ldy,
                          dhT, dzf, dg, dzo, self.D, dh0, self.ws, self.ws_bytes, stream)
        return dzf, dg, dzo, dh0

    def _grad(self, name, like, stream):
        t = getattr(self, name)
        if t is None:
            # zeros: as y, rows in no sequence are never written
            t, keep = self._new(stream, like.shape, like.dtype, like is self.y)
            if keep:
                setattr(self, name, t)
        return t


class ScanState(_Buffers):
    """The recurrence's states of n_slots live streams, advanced a token at a time (mdl_scan_step). Holds an output for
    each of the last `KEPT` numbers of rows that it met, so that calls of other sizes leave a result alone: a result
    stands until the next call with as many rows. A captured step writes the output that is held for its size, which is
    then held as long as the object (a server captures few sizes), or else one of the graph's own."""

    KEPT = 8
    HELD = -1

    def __init__(self, n_slots: int, D: int, x_dtype: str = "f32", device: str = "cuda"):
        self.device = _device(device)
        self.n_slots, self.D = int(n_slots), int(D)
        self.x_dtype, self.tdt = _x_dtype(x_dtype)
        self.state = torch.zeros(self.n_slots, self.D, dtype=torch.float32, device=self.device)
        # rows: (output, handle of the stream it was made on; HELD where a graph writes it), the oldest first
        self._y = {}
        self._made(self.device)

    def _output(self, S: int, handle: int) -> torch.Tensor:
        y, home = self._y.get(S, (None, None))
        if home == self.HELD:
            return y
        if y is not None and self._capturing(handle):
            self._y[S] = y, self.HELD
        elif home != handle:
            # never used on a stream but its own, on which its memory may be handed out again once it is dropped
            y, keep = self._new(handle, (S, self.D), self.tdt, True)
            if keep:
                self._y.pop(S, None)
                self._y[S] = y, handle
                loose = [s for s, (_, h) in self._y.items() if h != self.HELD]
                if len(loose) > self.KEPT:
                    del self._y[loose[0]]
        return y

    def step(self, zf, g, zo=None, slots=None, out=None, stream=None):
        """y [S][D] of one token for each row's slot (slots int32 [S], all different; the first S rows if None). The
        states advance in place, or into the same rows of `out` ([n_slots][D]). A row whose slot is no slot (-1 in a
        padded batch) is left out, and its y means nothing."""
        current = stream is None
        stream = self._launch(stream)
        S = int(zf.shape[0])
        ldz = _same_rows(("zf", "g", "zo"), (zf, g, zo), (S, self.D), self.tdt, self.device)
        _full("slots", slots, (S,), torch.int32, self.device)
        _full("out", out, (self.n_slots, self.D), torch.float32, self.device)
        y, home = self._y.get(S, (None, None))
        if home != stream or not current or torch.cuda.is_current_stream_capturing():
            y = self._output(S, stream)
        mdl_scan_step(S, self.D, self.x_dtype, zf, g, zo, ldz, slots, self.n_slots, self.state,
                      self.state if out is None else out, y, self.D, stream)
        return y


class BlockNorm(_Buffers):
    """The norms before and after a block over N rows of D channels, with the block's gate and scaled residual
    (mdl_blocknorm_forward / _backward). Weights are the caller's, [D] float32. Holds outputs and gradients: a call's
    results stand until the next call of the same method."""

    def __init__(self, N: int, D: int, x_dtype: str = "f32", eps: float = 1e-6, device: str = "cuda"):
        self.device = _device(device)
        self.N, self.D, self.eps = int(N), int(D), float(eps)
        self.x_dtype, self.tdt = _x_dtype(x_dtype)
        self.ws_bytes = mdl_blocknorm_workspace_size(self.N, self.D, self.x_dtype)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        self._bufs = {}
        self._made(self.device)

    def _out(self, stream, name, wanted, weight=False):
        if not wanted:
            return None
        t = self._bufs.get(name)
        if t is None:
            shape, dt = ((self.D,), torch.float32) if weight else ((self.N, self.D), self.tdt)
            t, keep = self._new(stream, shape, dt, False)
            if keep:
                self._bufs[name] = t
        return t

    def _inputs(self, x, z, u, w_post, scale, w_pre):
        lds = [_rows(n, t, (self.N, self.D), self.tdt, self.device) if t is not None else 0
               for n, t in (("x", x), ("z", z), ("u", u))]
        for n, t in (("w_post", w_post), ("scale", scale), ("w_pre", w_pre)):
            _full(n, t, (self.D,), torch.float32, self.device)
        return lds

    def forward(self, x, z=None, u=None, w_post=None, scale=None, w_pre=None, stream=None):
        """(r, v): r is x itself without z, v None without w_pre."""
        stream = self._launch(stream)
        ldx, ldz, ldu = self._inputs(x, z, u, w_post, scale, w_pre)
        r, v = self._out(stream, "r", z is not None), self._out(stream, "v", w_pre is not None)
        mdl_blocknorm_forward(self.N, self.D, self.x_dtype, x, ldx, z, ldz, u, ldu, w_post, scale, w_pre, self.eps, r,
                              v, self.D, stream)
        return (x if z is None else r), v

    def backward(self, x, z, u, w_post, scale, w_pre, dr, dv, stream=None):
        """(dx, dz, du, dw_post, dscale, dw_pre), None where the input is."""
        stream = self._launch(stream)
        ldx, ldz, ldu = self._inputs(x, z, u, w_post, scale, w_pre)
        _full("dr", dr, (self.N, self.D), self.tdt, self.device)
        _full("dv", dv, (self.N, self.D), self.tdt, self.device)
        out = [self._out(stream, n, t is not None) for n, t in (("dx", x), ("dz", z), ("du", u))]
        out += [self._out(stream, n, t is not None, True)
                for n, t in (("dw_post", w_post), ("dscale", scale), ("dw_pre", w_pre))]
        mdl_blocknorm_backward(self.N, self.D, self.x_dtype, x, ldx, z, ldz, u, ldu, w_post, scale, w_pre, self.eps,
                               dr, dv, self.D, *out[:3], self.D, *out[3:], self.ws, self.ws_bytes, stream)
        return tuple(out)


class TopKDistill(_Buffers):
    """Distillation loss of N frames over V classes from a teacher's k kept logits (mdl_distill): the loss per frame
    and its gradient in one call. Holds both; they stand until the next call."""

    def __init__(self, N: int, V: int, k: int, x_dtype: str = "f32", tau: float = 1.0, device: str = "cuda"):
        self.device = _device(device)
        self.N, self.V, self.k, self.tau = int(N), int(V), int(k), float(tau)
        self.x_dtype, self.tdt = _x_dtype(x_dtype)
        self.loss = torch.empty(self.N, dtype=torch.float32, device=self.device)
        self.dz = torch.empty(self.N, self.V, dtype=self.tdt, device=self.device)
        self._made(self.device)

    def run(self, z, ids, t, w=None, want_dz: bool = True, stream=None):
        """(loss [N], dz [N][V] or None): z [N][V] at any row stride, ids int32 and t (float32 or bfloat16) [N][k],
        w [N] float32 or None."""
        stream = self._launch(stream)
        ldz = _rows("z", z, (self.N, self.V), self.tdt, self.device)
        _full("ids", ids, (self.N, self.k), torch.int32, self.device)
        t_dtype = "bf16" if t.dtype == torch.bfloat16 else "f32"
        _full("t", t, (self.N, self.k), _DTYPES[t_dtype][1], self.device)
        _full("w", w, (self.N,), torch.float32, self.device)
        dz = self.dz if want_dz else None
        mdl_distill(self.N, self.V, self.k, self.x_dtype, z, ldz, ids, t, _DTYPES[t_dtype][0], w, self.tau, self.loss,
                    dz, self.V, stream)
        return self.loss, dz
