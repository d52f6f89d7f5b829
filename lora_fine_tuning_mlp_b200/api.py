"""PyTorch-facing wrappers of the C ABI.

PyTorch provides device memory and the current stream; every step of the
LoRA SwiGLU MLP and of the LoRA linear runs in the library's sm_100a kernels.  There is no fallback:
if the CUDA library is missing or the device is not a B200 the call raises.

A call with a `stream` runs on that stream and allocates for it.  Its inputs
are the caller's: they are ready for the stream when the call is made, and stay
until the stream has read them (Tensor.record_stream).
"""
from __future__ import annotations

import functools
from dataclasses import dataclass

import torch
from torch.autograd.function import once_differentiable

from . import _lib

BF16 = torch.bfloat16


def _p(t):
    return None if t is None else t.data_ptr()


# A Stream object costs 3 us a call; torch has the address without one under names that are not public.
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    """The address of a stream, by default of the current device's current one."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None or _current_device is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(_current_device())


def _need(t, name, dtype, shape=None):
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.is_contiguous()
            and (shape is None or t.shape == shape)):
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


@dataclass
class MLPWeights:
    """Frozen SwiGLU weights and the three LoRA adapters (nn.Linear layout).

    bf16 weights: Wg, Wu [d_ff, d], Wd [d, d_ff].  int4 weights: Wg, Wu uint8
    [d_ff, d/2], Wd uint8 [d, d_ff/2] and fp16 scales Sg, Su [d_ff, d/64],
    Sd [d, d_ff/64].  FP8 weights: Wg, Wu float8_e4m3fn [d_ff, d], Wd
    float8_e4m3fn [d, d_ff] and fp32 scales of the int4 shapes.  Adapters (bf16): Ag, Au [r, d]; Bg, Bu [d_ff, r];
    Ad [r, d_ff]; Bd [d, r].
    """
    Wg: torch.Tensor
    Wu: torch.Tensor
    Wd: torch.Tensor
    Ag: torch.Tensor
    Bg: torch.Tensor
    Au: torch.Tensor
    Bu: torch.Tensor
    Ad: torch.Tensor
    Bd: torch.Tensor
    alpha: float
    Sg: torch.Tensor | None = None
    Su: torch.Tensor | None = None
    Sd: torch.Tensor | None = None

    @property
    def int4(self) -> bool:
        return self.Wg.dtype == torch.uint8

    @property
    def fp8(self) -> bool:
        return self.Wg.dtype == torch.float8_e4m3fn

    @property
    def fmt(self) -> int:
        return _lib.WEIGHTS_INT4_B64 if self.int4 else (_lib.WEIGHTS_FP8_B64 if self.fp8 else _lib.WEIGHTS_BF16)

    @property
    def r(self) -> int:
        return int(self.Ag.shape[0])

    @property
    def d(self) -> int:
        return int(self.Ag.shape[1])

    @property
    def d_ff(self) -> int:
        return int(self.Bg.shape[0])

    def shape(self, N: int) -> _lib.Shape:
        return _lib.make_shape(N, self.d, self.d_ff, self.r, self.alpha, self.fmt)

    def validate(self):
        d, d_ff, r = self.d, self.d_ff, self.r
        if self.int4:
            _need(self.Wg, "Wg", torch.uint8, (d_ff, d // 2))
            _need(self.Wu, "Wu", torch.uint8, (d_ff, d // 2))
            _need(self.Wd, "Wd", torch.uint8, (d, d_ff // 2))
            _need(self.Sg, "Sg", torch.float16, (d_ff, d // 64))
            _need(self.Su, "Su", torch.float16, (d_ff, d // 64))
            _need(self.Sd, "Sd", torch.float16, (d, d_ff // 64))
        elif self.fp8:
            _need(self.Wg, "Wg", torch.float8_e4m3fn, (d_ff, d))
            _need(self.Wu, "Wu", torch.float8_e4m3fn, (d_ff, d))
            _need(self.Wd, "Wd", torch.float8_e4m3fn, (d, d_ff))
            _need(self.Sg, "Sg", torch.float32, (d_ff, d // 64))
            _need(self.Su, "Su", torch.float32, (d_ff, d // 64))
            _need(self.Sd, "Sd", torch.float32, (d, d_ff // 64))
        else:
            _need(self.Wg, "Wg", BF16, (d_ff, d))
            _need(self.Wu, "Wu", BF16, (d_ff, d))
            _need(self.Wd, "Wd", BF16, (d, d_ff))
        _need(self.Ag, "Ag", BF16, (r, d))
        _need(self.Au, "Au", BF16, (r, d))
        _need(self.Bg, "Bg", BF16, (d_ff, r))
        _need(self.Bu, "Bu", BF16, (d_ff, r))
        _need(self.Ad, "Ad", BF16, (r, d_ff))
        _need(self.Bd, "Bd", BF16, (d, r))

    def c_struct(self) -> _lib.Weights:
        return _lib.Weights(*[None if getattr(self, n) is None else getattr(self, n).data_ptr()
                              for n in _lib.WEIGHT_FIELDS])


@dataclass
class Saved:
    """What forward keeps for backward: the bf16 pre-activations g, u and the
    library's opaque rank-r buffer."""
    g: torch.Tensor
    u: torch.Tensor
    lowrank: torch.Tensor


class Workspace:
    """A reusable device scratch buffer (grown on demand)."""

    def __init__(self):
        self.buf = None

    def get(self, nbytes: int, device) -> torch.Tensor:
        if self.buf is None or self.buf.numel() < nbytes or self.buf.device != device:
            self.buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        return self.buf


def _allocate(stream, make, *args, **kw):
    """make(*args, **kw), memory for a call that runs on `stream`.  It comes from that stream's part of the allocator:
    what the current stream's part hands out may still be in use by work queued there, which `stream` does not wait
    for.  The caller goes on with it on the current stream, which the allocator is told."""
    if stream is None:
        return make(*args, **kw)
    here = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        t = make(*args, **kw)
    t.record_stream(here)
    return t


def _scratch(workspace, nbytes: int, device, stream):
    """The workspace's buffer, or one for this call alone."""
    if workspace is None:
        if stream is None:
            return torch.empty(nbytes, dtype=torch.uint8, device=device)
        with torch.cuda.stream(stream):
            return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if stream is None:
        return workspace.get(nbytes, device)
    buf = _allocate(stream, workspace.get, nbytes, device)
    buf.record_stream(stream)  # it may come from an earlier call on another one
    return buf


def _tensors(x):
    """The tensors of a call's results."""
    if hasattr(x, "record_stream"):
        yield x
    elif x is not None:
        for y in x.values() if isinstance(x, dict) else x if isinstance(x, (tuple, list)) else vars(x).values():
            yield from _tensors(y)


def _allocates_for_its_stream(call):
    """A call with a `stream` allocates as in _allocate and _scratch."""
    @functools.wraps(call)
    def on_its_stream(*args, stream=None, **kw):
        if stream is None:
            return call(*args, **kw)
        here = torch.cuda.current_stream(stream.device)
        with torch.cuda.stream(stream):
            results = call(*args, stream=stream, **kw)
        for t in _tensors(results):
            t.record_stream(here)
        if kw.get("workspace") is not None:
            for s in (here, stream):
                kw["workspace"].buf.record_stream(s)
        return results
    return on_its_stream


def sizes(w: MLPWeights, N: int):
    """(forward workspace, backward workspace, saved) byte counts."""
    return _lib.sizes(w.shape(N))


@_allocates_for_its_stream
def forward(X: torch.Tensor, w: MLPWeights, *, out=None, workspace: Workspace | None = None, stream=None):
    """out = MLP(X).  Returns (out, Saved)."""
    N, d = X.shape
    _need(X, "X", BF16, (N, w.d))
    w.validate()
    shape = w.shape(N)
    fws, _, svs = _lib.sizes(shape)
    dev = X.device
    out = torch.empty((N, d), dtype=BF16, device=dev) if out is None else _need(out, "out", BF16, (N, d))
    g = torch.empty((N, w.d_ff), dtype=BF16, device=dev)
    u = torch.empty((N, w.d_ff), dtype=BF16, device=dev)
    lowrank = torch.empty(max(svs, 256), dtype=torch.uint8, device=dev)
    ws = (workspace or Workspace()).get(fws, dev)
    _lib.check(_lib.forward(shape, w.c_struct(), _p(X), _p(out), _p(g), _p(u), _p(lowrank), _p(ws),
                            ws.numel(), _stream(stream)), "lora_mlp_forward")
    return out, Saved(g, u, lowrank)


@_allocates_for_its_stream
def backward(X: torch.Tensor, w: MLPWeights, saved: Saved, dOut: torch.Tensor, *, dX=None, grads=None,
             workspace: Workspace | None = None, stream=None):
    """Returns (dX, {dAg, dBg, dAu, dBu, dAd, dBd})."""
    N, d = X.shape
    _need(X, "X", BF16, (N, w.d))
    _need(dOut, "dOut", BF16, (N, d))
    w.validate()
    shape = w.shape(N)
    _, bws, _ = _lib.sizes(shape)
    dev = X.device
    dX = torch.empty((N, d), dtype=BF16, device=dev) if dX is None else _need(dX, "dX", BF16, (N, d))
    if grads is None:
        grads = {("d" + k): torch.empty_like(getattr(w, k)) for k in ("Ag", "Bg", "Au", "Bu", "Ad", "Bd")}
    gs = _lib.Grads(*[grads[k].data_ptr() for k in _lib.GRAD_FIELDS])
    ws = (workspace or Workspace()).get(bws, dev)
    _lib.check(_lib.backward(shape, w.c_struct(), _p(X), _p(saved.g), _p(saved.u), _p(saved.lowrank), _p(dOut),
                             _p(dX), gs, _p(ws), ws.numel(), _stream(stream)), "lora_mlp_backward")
    return dX, grads


def dequant_int4(packed: torch.Tensor, scales: torch.Tensor, stream=None) -> torch.Tensor:
    rows, half = packed.shape
    _need(packed, "packed", torch.uint8)
    _need(scales, "scales", torch.float16, (rows, 2 * half // 64))
    w = _allocate(stream, torch.empty, (rows, 2 * half), dtype=BF16, device=packed.device)
    _lib.check(_lib.dequant_int4(_p(packed), _p(scales), rows, 2 * half, _p(w), _stream(stream)),
               "lora_mlp_dequant_int4")
    return w


def dequant_fp8(codes: torch.Tensor, scales: torch.Tensor, stream=None) -> torch.Tensor:
    """bf16 [rows, cols] from FP8 E4M3 codes [rows, cols] (float8_e4m3fn or
    uint8) and fp32 block scales [rows, cols/64], by the library's kernel."""
    rows, cols = codes.shape
    if codes.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise TypeError("codes must be float8_e4m3fn or uint8")
    _need(scales, "scales", torch.float32, (rows, cols // 64))
    w = _allocate(stream, torch.empty, (rows, cols), dtype=BF16, device=codes.device)
    _lib.check(_lib.dequant_fp8(_p(codes), _p(scales), rows, cols, _p(w), _stream(stream)), "lora_mlp_dequant_fp8")
    return w


class LoRAMLPFunction(torch.autograd.Function):
    """autograd wrapper: out = LoRA-SwiGLU-MLP(X); backward fills X.grad and the
    adapter grads.  Usage: LoRAMLPFunction.apply(X, w, Ag, Bg, Au, Bu, Ad, Bd)
    where w is an MLPWeights whose adapter tensors are the same objects."""

    @staticmethod
    def forward(ctx, X, w: MLPWeights, Ag, Bg, Au, Bu, Ad, Bd):
        out, saved = forward(X.contiguous(), w)
        ctx.w = w
        ctx.saved_lr = saved
        ctx.save_for_backward(X)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dOut):
        (X,) = ctx.saved_tensors
        dX, g = backward(X, ctx.w, ctx.saved_lr, dOut.contiguous())
        return dX, None, g["dAg"], g["dBg"], g["dAu"], g["dBu"], g["dAd"], g["dBd"]


def weights_from_host(inp: dict, alpha: float, device="cuda") -> MLPWeights:
    """Upload a host input dict (bf16 bits as uint16 numpy arrays, int4 as
    packed uint8 + fp16 scales) to the device."""
    def bf(a):
        return torch.from_numpy(a.view("int16")).view(BF16).to(device)

    kw = {}
    for k in ("Ag", "Bg", "Au", "Bu", "Ad", "Bd"):
        kw[k] = bf(inp[k])
    if "Wg_q" in inp:
        for k, s in (("Wg", "Sg"), ("Wu", "Su"), ("Wd", "Sd")):
            kw[k] = torch.from_numpy(inp[k + "_q"]).to(device)
            kw[s] = torch.from_numpy(inp[k + "_scale"]).to(device)
    elif "Wg_f8" in inp:
        for k, s in (("Wg", "Sg"), ("Wu", "Su"), ("Wd", "Sd")):
            kw[k] = torch.from_numpy(inp[k + "_f8"]).view(torch.float8_e4m3fn).to(device)
            kw[s] = torch.from_numpy(inp[k + "_f8scale"]).to(device)
    else:
        for k in ("Wg", "Wu", "Wd"):
            kw[k] = bf(inp[k])
    return MLPWeights(alpha=float(alpha), **kw)


def to_device_bf16(a, device="cuda") -> torch.Tensor:
    return torch.from_numpy(a.view("int16")).view(BF16).to(device)


class HostBatchTrainer:
    """Forward + backward over batches that live in (pinned) host memory.

    The host-to-device copy of the next batch runs on its own stream while the
    current batch computes, and each step's adapter gradients are copied back
    to pinned host memory on a third stream while the next step computes.
    Inputs and gradients are double-buffered on the device (and the
    gradients on the host), ordered by CUDA events: a device buffer is
    refilled only once the step that used it, or its copy back, is done.
    Every step still moves its own inputs and result across PCIe; only the
    overlap with compute is new.
    """

    def __init__(self, w: MLPWeights, N: int, device=None, gamma: torch.Tensor | None = None, eps: float = 1e-5):
        """With `gamma`, each step runs the pre-norm block MLP(RMSNorm(X))."""
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self.w, self.N, self.dev = w, N, dev
        self.gamma, self.eps = gamma, eps
        d = w.d
        self.X = [torch.empty((N, d), dtype=BF16, device=dev) for _ in range(2)]
        self.dOut = [torch.empty((N, d), dtype=BF16, device=dev) for _ in range(2)]
        self.out = torch.empty((N, d), dtype=BF16, device=dev)
        self.dX = torch.empty((N, d), dtype=BF16, device=dev)
        names = ("Ag", "Bg", "Au", "Bu", "Ad", "Bd")
        self.grads = [{("d" + k): torch.empty_like(getattr(w, k)) for k in names} for _ in range(2)]
        self.grads_host = [{k: torch.empty(v.shape, dtype=v.dtype, pin_memory=True) for k, v in g.items()}
                           for g in self.grads]
        self.wsf, self.wsb = Workspace(), Workspace()
        self.copy_stream = torch.cuda.Stream(device=dev)
        self.d2h_stream = torch.cuda.Stream(device=dev)
        self.ready = [torch.cuda.Event(), torch.cuda.Event()]
        self.free = [torch.cuda.Event(), torch.cuda.Event()]
        self.computed = [torch.cuda.Event(), torch.cuda.Event()]
        self.fetched = [torch.cuda.Event(), torch.cuda.Event()]
        self.fetch_pending = [False, False]
        self.slot = 0
        self.primed = False

    def _stage(self, slot, Xh, dOh):
        with torch.cuda.stream(self.copy_stream):
            self.copy_stream.wait_event(self.free[slot])
            self.X[slot].copy_(Xh, non_blocking=True)
            self.dOut[slot].copy_(dOh, non_blocking=True)
            self.ready[slot].record(self.copy_stream)

    def h2d_bytes(self) -> int:
        return 2 * self.N * self.w.d * 2

    def d2h_bytes(self) -> int:
        return sum(v.numel() * v.element_size() for v in self.grads[0].values())

    def step(self, Xh, dOh, next_Xh=None, next_dOh=None):
        """One training step on host batch (Xh, dOh); if the next batch is
        given, its copy is started so that it overlaps this step's compute.
        Returns the dict of pinned host adapter gradients of this step: valid
        after `finish()` and a synchronisation of the current stream (or the
        device), and until the step after next overwrites them."""
        cur = self.slot
        if not self.primed:
            self._stage(cur, Xh, dOh)
            self.primed = True
        nxt = cur ^ 1
        if next_Xh is not None:
            self._stage(nxt, next_Xh, next_dOh)
        stream = torch.cuda.current_stream(self.dev)
        stream.wait_event(self.ready[cur])
        if self.fetch_pending[cur]:
            stream.wait_event(self.fetched[cur])  # this slot's gradients from two steps ago are home
        grads = self.grads[cur]
        if self.gamma is None:
            o, saved = forward(self.X[cur], self.w, out=self.out, workspace=self.wsf)
            backward(self.X[cur], self.w, saved, self.dOut[cur], dX=self.dX, grads=grads, workspace=self.wsb)
        else:
            o, saved = block_forward(self.X[cur], self.w, self.gamma, self.eps, out=self.out, workspace=self.wsf)
            block_backward(self.X[cur], self.w, self.gamma, saved, self.dOut[cur], dX=self.dX, grads=grads,
                           workspace=self.wsb)
        self.free[cur].record(stream)
        self.computed[cur].record(stream)
        with torch.cuda.stream(self.d2h_stream):
            self.d2h_stream.wait_event(self.computed[cur])
            for k, v in grads.items():
                self.grads_host[cur][k].copy_(v, non_blocking=True)
            self.fetched[cur].record(self.d2h_stream)
        self.fetch_pending[cur] = True
        self.slot = nxt
        if next_Xh is None:
            self.primed = False
        return self.grads_host[cur]

    def finish(self):
        """Orders the current stream after every gradient copy issued so far."""
        stream = torch.cuda.current_stream(self.dev)
        for i in range(2):
            if self.fetch_pending[i]:
                stream.wait_event(self.fetched[i])


# ----------------------------------------------------------------------------- LoRA linear


@dataclass
class LinearWeights:
    """One frozen projection with a LoRA adapter (nn.Linear layout).

    bf16: W [d_out, d_in].  int4: W uint8 [d_out, d_in/2] and fp16 scales
    S [d_out, d_in/64].  FP8: W float8_e4m3fn [d_out, d_in] and fp32 scales
    S [d_out, d_in/64].  Adapter (bf16): A [r, d_in], B [d_out, r].
    """
    W: torch.Tensor
    A: torch.Tensor
    B: torch.Tensor
    alpha: float
    S: torch.Tensor | None = None

    @property
    def int4(self) -> bool:
        return self.W.dtype == torch.uint8

    @property
    def fp8(self) -> bool:
        return self.W.dtype == torch.float8_e4m3fn

    @property
    def r(self) -> int:
        return int(self.A.shape[0])

    @property
    def d_in(self) -> int:
        return int(self.A.shape[1])

    @property
    def d_out(self) -> int:
        return int(self.B.shape[0])

    def shape(self, N: int) -> _lib.LinShape:
        fmt = _lib.WEIGHTS_INT4_B64 if self.int4 else (_lib.WEIGHTS_FP8_B64 if self.fp8 else _lib.WEIGHTS_BF16)
        return _lib.make_lin_shape(N, self.d_in, self.d_out, self.r, self.alpha, fmt)

    def validate(self):
        di, do, r = self.d_in, self.d_out, self.r
        if self.int4:
            _need(self.W, "W", torch.uint8, (do, di // 2))
            _need(self.S, "S", torch.float16, (do, di // 64))
        elif self.fp8:
            _need(self.W, "W", torch.float8_e4m3fn, (do, di))
            _need(self.S, "S", torch.float32, (do, di // 64))
        else:
            _need(self.W, "W", BF16, (do, di))
        _need(self.A, "A", BF16, (r, di))
        _need(self.B, "B", BF16, (do, r))

    def c_struct(self) -> _lib.LinWeights:
        return _lib.LinWeights(self.W.data_ptr(), None if self.S is None else self.S.data_ptr(),
                               self.A.data_ptr(), self.B.data_ptr())


def linear_sizes(w: LinearWeights, N: int):
    """(forward workspace, backward workspace, saved) byte counts."""
    return _lib.lin_sizes(w.shape(N))


@_allocates_for_its_stream
def linear_forward(X: torch.Tensor, w: LinearWeights, *, Y=None, workspace: Workspace | None = None,
                   stream=None):
    """Y = X (W + s B A)^T.  Returns (Y, saved) where saved is the opaque
    rank-r buffer backward needs."""
    N = X.shape[0]
    _need(X, "X", BF16, (N, w.d_in))
    w.validate()
    shape = w.shape(N)
    fws, _, svs = _lib.lin_sizes(shape)
    dev = X.device
    Y = torch.empty((N, w.d_out), dtype=BF16, device=dev) if Y is None else _need(Y, "Y", BF16, (N, w.d_out))
    saved = torch.empty(max(svs, 256), dtype=torch.uint8, device=dev)
    ws = (workspace or Workspace()).get(fws, dev)
    _lib.check(_lib.lin_forward(shape, w.c_struct(), _p(X), _p(Y), _p(saved), _p(ws), ws.numel(),
                                _stream(stream)), "lora_linear_forward")
    return Y, saved


@_allocates_for_its_stream
def linear_backward(X: torch.Tensor, w: LinearWeights, saved: torch.Tensor, dY: torch.Tensor, *, dX=None,
                    dA=None, dB=None, workspace: Workspace | None = None, stream=None):
    """Returns (dX, dA, dB)."""
    N = X.shape[0]
    _need(X, "X", BF16, (N, w.d_in))
    _need(dY, "dY", BF16, (N, w.d_out))
    w.validate()
    shape = w.shape(N)
    _, bws, _ = _lib.lin_sizes(shape)
    dev = X.device
    dX = torch.empty((N, w.d_in), dtype=BF16, device=dev) if dX is None else _need(dX, "dX", BF16, (N, w.d_in))
    dA = torch.empty_like(w.A) if dA is None else _need(dA, "dA", BF16, tuple(w.A.shape))
    dB = torch.empty_like(w.B) if dB is None else _need(dB, "dB", BF16, tuple(w.B.shape))
    ws = (workspace or Workspace()).get(bws, dev)
    _lib.check(_lib.lin_backward(shape, w.c_struct(), _p(X), _p(saved), _p(dY), _p(dX), _p(dA), _p(dB), _p(ws),
                                 ws.numel(), _stream(stream)), "lora_linear_backward")
    return dX, dA, dB


class LoRALinearFunction(torch.autograd.Function):
    """autograd wrapper: Y = X (W + s B A)^T.  Usage:
    LoRALinearFunction.apply(X, w, A, B) where w is a LinearWeights whose A and
    B are the same tensors."""

    @staticmethod
    def forward(ctx, X, w: LinearWeights, A, B):
        Y, saved = linear_forward(X.contiguous(), w)
        ctx.w = w
        ctx.saved_lr = saved
        ctx.save_for_backward(X)
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        (X,) = ctx.saved_tensors
        dX, dA, dB = linear_backward(X, ctx.w, ctx.saved_lr, dY.contiguous())
        return dX, None, dA, dB


def linear_weights_from_host(inp: dict, alpha: float, device="cuda") -> LinearWeights:
    """Upload a host LoRA-linear input dict to the device."""
    if "W_q" in inp:
        return LinearWeights(W=torch.from_numpy(inp["W_q"]).to(device), A=to_device_bf16(inp["A"], device),
                             B=to_device_bf16(inp["B"], device), alpha=float(alpha),
                             S=torch.from_numpy(inp["W_scale"]).to(device))
    if "W_f8" in inp:
        return LinearWeights(W=torch.from_numpy(inp["W_f8"]).view(torch.float8_e4m3fn).to(device),
                             A=to_device_bf16(inp["A"], device), B=to_device_bf16(inp["B"], device),
                             alpha=float(alpha), S=torch.from_numpy(inp["W_f8scale"]).to(device))
    return LinearWeights(W=to_device_bf16(inp["W"], device), A=to_device_bf16(inp["A"], device),
                         B=to_device_bf16(inp["B"], device), alpha=float(alpha))


# ----------------------------------------------------------------------------- RMSNorm and the pre-norm block


@_allocates_for_its_stream
def rmsnorm_forward(x: torch.Tensor, gamma: torch.Tensor, eps: float, *, stream=None):
    """Returns (y, rstd): y = RMSNorm(x) * gamma (bf16), rstd fp32 [N]."""
    N, d = x.shape
    _need(x, "x", BF16)
    _need(gamma, "gamma", BF16, (d,))
    y = torch.empty_like(x)
    rstd = torch.empty((N,), dtype=torch.float32, device=x.device)
    _lib.check(_lib.rmsnorm_forward(N, d, eps, _p(x), _p(gamma), _p(y), _p(rstd), _stream(stream)),
               "lora_rmsnorm_forward")
    return y, rstd


@_allocates_for_its_stream
def rmsnorm_backward(x: torch.Tensor, gamma: torch.Tensor, rstd: torch.Tensor, dy: torch.Tensor, *, stream=None):
    N, d = x.shape
    _need(x, "x", BF16)
    _need(gamma, "gamma", BF16, (d,))
    _need(rstd, "rstd", torch.float32, (N,))
    _need(dy, "dy", BF16, (N, d))
    dx = torch.empty_like(x)
    _lib.check(_lib.rmsnorm_backward(N, d, _p(x), _p(gamma), _p(rstd), _p(dy), _p(dx), _stream(stream)),
               "lora_rmsnorm_backward")
    return dx


class RMSNormFunction(torch.autograd.Function):
    """autograd wrapper of the library's RMSNorm: y = x * rstd * gamma per row,
    with the frozen gain gamma (no gradient for it) and the forward's rstd
    reused by the backward.  Usage: RMSNormFunction.apply(x, gamma, eps)."""

    @staticmethod
    def forward(ctx, x, gamma, eps=1e-5):
        x = x.contiguous()
        y, rstd = rmsnorm_forward(x, gamma, eps)
        ctx.save_for_backward(x, gamma, rstd)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, gamma, rstd = ctx.saved_tensors
        return rmsnorm_backward(x, gamma, rstd, dy.contiguous()), None, None


def fold_gamma(w: MLPWeights, gamma: torch.Tensor, stream=None) -> MLPWeights:
    """The weights of the fused-norm block: Wg, Wu with gamma folded into
    their columns (bf16_rne(W * gamma), by the library's kernel); Wd and the
    adapters are the same tensors as w's.  bf16 frozen weights only.  Done
    once: W and gamma are frozen."""
    if w.int4 or w.fp8:
        raise ValueError("gamma folds into bf16 frozen weights only")
    w.validate()
    _need(gamma, "gamma", BF16, (w.d,))
    Wg, Wu = (_allocate(stream, torch.empty_like, t) for t in (w.Wg, w.Wu))
    _lib.check(_lib.block_fold_gamma(w.shape(1), w.c_struct(), _p(gamma), _p(Wg), _p(Wu), _stream(stream)),
               "lora_mlp_block_fold_gamma")
    return MLPWeights(Wg=Wg, Wu=Wu, Wd=w.Wd, Ag=w.Ag, Bg=w.Bg, Au=w.Au, Bu=w.Bu, Ad=w.Ad, Bd=w.Bd, alpha=w.alpha)


@_allocates_for_its_stream
def block_forward(X: torch.Tensor, w: MLPWeights, gamma: torch.Tensor, eps: float, *, out=None,
                  workspace: Workspace | None = None, stream=None, folded: bool = False):
    """out = MLP(RMSNorm(X) * gamma).  Returns (out, Saved); Saved.lowrank
    also holds the per-row rstd.  folded=True: w comes from fold_gamma and
    the norm runs fused into the gate/up GEMM (lora_mlp_block_forward_folded)."""
    N, d = X.shape
    _need(X, "X", BF16, (N, w.d))
    _need(gamma, "gamma", BF16, (w.d,))
    w.validate()
    shape = w.shape(N)
    fws, _, svs = _lib.block_sizes(shape)
    dev = X.device
    out = torch.empty((N, d), dtype=BF16, device=dev) if out is None else _need(out, "out", BF16, (N, d))
    g = torch.empty((N, w.d_ff), dtype=BF16, device=dev)
    u = torch.empty((N, w.d_ff), dtype=BF16, device=dev)
    saved = torch.empty(max(svs, 256), dtype=torch.uint8, device=dev)
    ws = (workspace or Workspace()).get(fws, dev)
    fn = _lib.block_forward_folded if folded else _lib.block_forward
    _lib.check(fn(shape, w.c_struct(), _p(gamma), eps, _p(X), _p(out), _p(g), _p(u), _p(saved), _p(ws), ws.numel(),
                  _stream(stream)), "lora_mlp_block_forward" + ("_folded" if folded else ""))
    return out, Saved(g, u, saved)


@_allocates_for_its_stream
def block_backward(X: torch.Tensor, w: MLPWeights, gamma: torch.Tensor, saved: Saved, dOut: torch.Tensor, *,
                   dX=None, grads=None, workspace: Workspace | None = None, stream=None, folded: bool = False):
    """Returns (dX, {dAg, dBg, dAu, dBu, dAd, dBd}) for the block input X.
    folded as in block_forward (and the same as the forward's)."""
    N, d = X.shape
    _need(X, "X", BF16, (N, w.d))
    _need(gamma, "gamma", BF16, (w.d,))
    _need(dOut, "dOut", BF16, (N, d))
    w.validate()
    shape = w.shape(N)
    _, bws, _ = _lib.block_sizes(shape)
    dev = X.device
    dX = torch.empty((N, d), dtype=BF16, device=dev) if dX is None else _need(dX, "dX", BF16, (N, d))
    if grads is None:
        grads = {("d" + k): torch.empty_like(getattr(w, k)) for k in ("Ag", "Bg", "Au", "Bu", "Ad", "Bd")}
    gs = _lib.Grads(*[grads[k].data_ptr() for k in _lib.GRAD_FIELDS])
    ws = (workspace or Workspace()).get(bws, dev)
    fn = _lib.block_backward_folded if folded else _lib.block_backward
    _lib.check(fn(shape, w.c_struct(), _p(gamma), _p(X), _p(saved.g), _p(saved.u), _p(saved.lowrank), _p(dOut),
                  _p(dX), gs, _p(ws), ws.numel(), _stream(stream)),
               "lora_mlp_block_backward" + ("_folded" if folded else ""))
    return dX, grads


class LoRAMLPBlockFunction(torch.autograd.Function):
    """autograd wrapper of the pre-norm block: out = MLP(RMSNorm(X) * gamma).
    Usage: LoRAMLPBlockFunction.apply(X, w, gamma, eps, Ag, Bg, Au, Bu, Ad, Bd)
    (gamma frozen: no gradient)."""

    @staticmethod
    def forward(ctx, X, w: MLPWeights, gamma, eps, Ag, Bg, Au, Bu, Ad, Bd):
        out, saved = block_forward(X.contiguous(), w, gamma, eps)
        ctx.w, ctx.gamma, ctx.saved_lr = w, gamma, saved
        ctx.save_for_backward(X)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dOut):
        (X,) = ctx.saved_tensors
        dX, g = block_backward(X, ctx.w, ctx.gamma, ctx.saved_lr, dOut.contiguous())
        return dX, None, None, None, g["dAg"], g["dBg"], g["dAu"], g["dBu"], g["dAd"], g["dBd"]


# ----------------------------------------------------------------------------- chunked cross-entropy


def _ce_shape(logits: torch.Tensor, logit_scale: float, softcap: float, ignore_index: int):
    if logits.dim() != 2:
        raise ValueError("logits must be [N, V]")
    if logits.dtype != BF16 or not logits.is_cuda:
        raise TypeError("logits must be a bf16 CUDA tensor")
    if logits.stride(1) != 1:
        raise ValueError("logits rows must be contiguous")
    N, V = logits.shape
    return _lib.make_ce_shape(N, V, logits.stride(0), logit_scale, softcap, ignore_index)


@_allocates_for_its_stream
def ce_forward(logits: torch.Tensor, labels: torch.Tensor, *, logit_scale: float = 1.0, softcap: float = 0.0,
               ignore_index: int = -100, workspace: Workspace | None = None, stream=None):
    """Per-row cross-entropy of bf16 logits [N, V] (row stride a multiple of
    8) against int64 labels [N]: returns (loss [N] fp32, lse [N] fp32), loss 0
    for rows labelled ignore_index."""
    shape = _ce_shape(logits, logit_scale, softcap, ignore_index)
    N = shape.N
    _need(labels, "labels", torch.int64, (N,))
    dev = logits.device
    loss = torch.empty((N,), dtype=torch.float32, device=dev)
    lse = torch.empty((N,), dtype=torch.float32, device=dev)
    ws = (workspace or Workspace()).get(_lib.ce_sizes(shape), dev)
    _lib.check(_lib.ce_forward(shape, _p(logits), _p(labels), _p(loss), _p(lse), _p(ws), ws.numel(),
                               _stream(stream)), "lora_ce_forward")
    return loss, lse


@_allocates_for_its_stream
def ce_backward(logits: torch.Tensor, labels: torch.Tensor, lse: torch.Tensor, dloss: torch.Tensor, *,
                logit_scale: float = 1.0, softcap: float = 0.0, ignore_index: int = -100, out=None,
                inplace: bool = False, stream=None):
    """dlogits [N, V] bf16 for the per-row upstream gradient dloss [N] (fp32).
    inplace=True writes the gradient over the logits."""
    shape = _ce_shape(logits, logit_scale, softcap, ignore_index)
    N = shape.N
    _need(labels, "labels", torch.int64, (N,))
    _need(lse, "lse", torch.float32, (N,))
    _need(dloss, "dloss", torch.float32, (N,))
    # The kernel writes the gradient with the logits' row stride, so the
    # output keeps the logits' strides (empty_like would not for a padded view).
    if inplace:
        out = logits
    elif out is None:
        out = torch.empty_strided(logits.size(), logits.stride(), dtype=BF16, device=logits.device)
    elif (out.shape != logits.shape or out.stride() != logits.stride() or out.dtype != BF16 or not out.is_cuda):
        raise ValueError("out must have the logits' shape, strides and dtype")
    _lib.check(_lib.ce_backward(shape, _p(logits), _p(labels), _p(lse), _p(dloss), _p(out), _stream(stream)),
               "lora_ce_backward")
    return out


@_allocates_for_its_stream
def ce_loss(logits: torch.Tensor, labels: torch.Tensor, *, reduction: str = "mean", logit_scale: float = 1.0,
            softcap: float = 0.0, ignore_index: int = -100, workspace: Workspace | None = None, stream=None):
    """The cross-entropy reduced over the rows, computed by the library:
    returns (out [2] fp32, lse [N] fp32), out[0] the summed or mean loss and
    out[1] its derivative with respect to each row's loss (1, or 1 / rows
    taking part), the factor ce_backward_reduced applies."""
    red = {"sum": _lib.CE_REDUCTION_SUM, "mean": _lib.CE_REDUCTION_MEAN}.get(reduction)
    if red is None:
        raise ValueError("reduction must be 'sum' or 'mean'")
    shape = _ce_shape(logits, logit_scale, softcap, ignore_index)
    N = shape.N
    _need(labels, "labels", torch.int64, (N,))
    dev = logits.device
    out = torch.empty((2,), dtype=torch.float32, device=dev)
    lse = torch.empty((N,), dtype=torch.float32, device=dev)
    ws = (workspace or Workspace()).get(_lib.ce_sizes(shape), dev)
    _lib.check(_lib.ce_forward_reduced(shape, _p(logits), _p(labels), red, _p(out), _p(lse), _p(ws), ws.numel(),
                                       _stream(stream)), "lora_ce_forward_reduced")
    return out, lse


@_allocates_for_its_stream
def ce_backward_reduced(logits: torch.Tensor, labels: torch.Tensor, lse: torch.Tensor, dout: torch.Tensor,
                        fwd_out: torch.Tensor, *, logit_scale: float = 1.0, softcap: float = 0.0,
                        ignore_index: int = -100, out=None, inplace: bool = False, stream=None):
    """dlogits [N, V] bf16 for the upstream gradient dout (fp32, one element)
    of the loss ce_loss returned in fwd_out.  inplace=True writes the
    gradient over the logits."""
    shape = _ce_shape(logits, logit_scale, softcap, ignore_index)
    N = shape.N
    _need(labels, "labels", torch.int64, (N,))
    _need(lse, "lse", torch.float32, (N,))
    _need(fwd_out, "fwd_out", torch.float32, (2,))
    if dout.numel() != 1 or dout.dtype != torch.float32 or not dout.is_cuda:
        raise TypeError("dout must be one fp32 CUDA element")
    if inplace:
        out = logits
    elif out is None:
        out = torch.empty_strided(logits.size(), logits.stride(), dtype=BF16, device=logits.device)
    elif (out.shape != logits.shape or out.stride() != logits.stride() or out.dtype != BF16 or not out.is_cuda):
        raise ValueError("out must have the logits' shape, strides and dtype")
    _lib.check(_lib.ce_backward_reduced(shape, _p(logits), _p(labels), _p(lse), _p(dout), _p(fwd_out), _p(out),
                                        _stream(stream)), "lora_ce_backward_reduced")
    return out


class CrossEntropyFunction(torch.autograd.Function):
    """Mean cross-entropy over the rows whose label is not ignore_index, with
    the library's chunked kernels; the mean and its gradient factor are
    computed in the library.  Usage:
    CrossEntropyFunction.apply(logits, labels, logit_scale, softcap, ignore_index, inplace).
    By default the backward writes the logits' gradient to a new buffer.
    inplace=True writes it over the logits instead, as the pages' kernel does
    to save memory; the logits' version counter is then bumped, so any other
    autograd node that saved them raises instead of reading the gradient."""

    @staticmethod
    def forward(ctx, logits, labels, logit_scale=1.0, softcap=0.0, ignore_index=-100, inplace=False):
        out, lse = ce_loss(logits, labels, reduction="mean", logit_scale=logit_scale, softcap=softcap,
                           ignore_index=ignore_index)
        ctx.save_for_backward(logits, labels, lse, out)
        ctx.cfg = (logit_scale, softcap, ignore_index, bool(inplace))
        return out[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        logits, labels, lse, out = ctx.saved_tensors
        s, c, ign, inplace = ctx.cfg
        if g.dtype != torch.float32 or not g.is_cuda:
            raise TypeError("the upstream gradient of the loss must be fp32 on the GPU")
        dz = ce_backward_reduced(logits, labels, lse, g.contiguous(), out, logit_scale=s, softcap=c,
                                 ignore_index=ign, inplace=inplace)
        if inplace:
            torch.autograd.graph.increment_version(logits)
        return dz, None, None, None, None, None


# ----------------------------------------------------------------------------- token embedding


def embedding_forward(ids: torch.Tensor, E: torch.Tensor, *, scale: float = 1.0, out=None, stream=None):
    """out [N, d] = scale * E[ids] (bf16, rounded once) for int64 ids [N] and a bf16 table E [V, d], d a multiple
    of 8.  The row of an id outside [0, V) is NaN, and step_device_status reports it."""
    _need(ids, "ids", torch.int64)
    _need(E, "E", BF16)
    if ids.dim() != 1 or E.dim() != 2:
        raise ValueError("ids must be [N] and E [V, d]")
    (N,), (V, d) = ids.shape, E.shape
    if out is None:
        out = E.new_empty((N, d)) if stream is None else _allocate(stream, E.new_empty, (N, d))
    else:
        _need(out, "out", BF16, (N, d))
    _lib.check(_lib.embedding_forward(N, V, d, scale, _p(ids), _p(E), _p(out), _stream(stream)),
               "lora_embedding_forward")
    return out


def _check_padding(padding_idx, V):
    if padding_idx is not None and not 0 <= padding_idx < V:
        raise ValueError(f"padding_idx must be in [0, {V})")


def embedding_backward(dOut: torch.Tensor, ids: torch.Tensor, V: int, *, scale: float = 1.0, padding_idx=None,
                       dtype=BF16, dE=None, workspace: Workspace | None = None, stream=None):
    """dE [V, d], the gradient of embedding_forward's table: each row the sum of its tokens' rows of dOut [N, d]
    (in fp32, in a fixed order), rounded once to `dtype` (bf16 or fp32); zeros for ids without a token and for
    padding_idx."""
    _need(dOut, "dOut", BF16)
    if dOut.dim() != 2:
        raise ValueError("dOut must be [N, d]")
    N, d = dOut.shape
    _need(ids, "ids", torch.int64, (N,))
    kind = {BF16: _lib.EMBEDDING_GRAD_BF16, torch.float32: _lib.EMBEDDING_GRAD_FP32}.get(dtype)
    if kind is None:
        raise TypeError("dtype must be torch.bfloat16 or torch.float32")
    _check_padding(padding_idx, V)
    dev = dOut.device
    if dE is None:
        dE = _allocate(stream, torch.empty, (V, d), dtype=dtype, device=dev)
    else:
        _need(dE, "dE", dtype, (V, d))
    ws = _scratch(workspace, _lib.embedding_sizes(N, V, d), dev, stream)
    _lib.check(_lib.embedding_backward(N, V, d, scale, -1 if padding_idx is None else padding_idx, kind, _p(ids),
                                       _p(dOut), _p(dE), _p(ws), ws.numel(), _stream(stream)),
               "lora_embedding_backward")
    return dE


class EmbeddingFunction(torch.autograd.Function):
    """autograd wrapper of the scaled lookup: out = scale * E[ids].  Usage:
    EmbeddingFunction.apply(ids, E, scale, padding_idx) (padding_idx None or an id whose row gets no gradient)."""

    @staticmethod
    def forward(ctx, ids, E, scale=1.0, padding_idx=None):
        _check_padding(padding_idx, E.shape[0])
        ids = ids.contiguous()
        ctx.save_for_backward(ids)
        ctx.cfg = (E.shape[0], scale, padding_idx)
        return embedding_forward(ids, E, scale=scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, dOut):
        (ids,) = ctx.saved_tensors
        V, scale, padding_idx = ctx.cfg
        return None, embedding_backward(dOut.contiguous(), ids, V, scale=scale, padding_idx=padding_idx), None, None


# ----------------------------------------------------------------------------- queries' and keys' norm and rotation


def rope_table(P: int, rot: int, *, base: float = 10000.0, device=None):
    """(cos, sin), fp32 [P, rot/2], of the plain rotation: pair i of position p turns by p * base^(-2i/rot).  The
    angles are formed in fp64, so that far positions keep theirs.  A program makes the table once; one with scaled
    frequencies fills its own."""
    if P < 1 or rot < 2 or rot % 2:
        raise ValueError("P must be at least 1 and rot even")
    freq = float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    angle = torch.arange(P, dtype=torch.float64, device=device)[:, None] * freq
    return angle.cos().float(), angle.sin().float()


def _heads(t, name, shape=None, written=False):
    """A [B, S, heads, D] (or [S, heads, D]) view for the library: the last axis contiguous, other strides multiples
    of 8."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != BF16:
        raise TypeError(f"{name} must be {BF16}, got {t.dtype}")
    n = t.shape
    if (len(n) != 4 and len(n) != 3) or (shape is not None and n != shape):
        raise ValueError(f"{name} has shape {tuple(n)}, expected " +
                         ("[B, S, heads, D] or [S, heads, D]" if shape is None else str(tuple(shape))))
    # the stride of an axis of one entry is never used, and may be anything
    if len(n) == 4:
        B, S, H, _ = n
        sb, ss, sh, se = t.stride()
    else:
        B, (S, H, _) = 1, n
        sb, (ss, sh, se) = 0, t.stride()
    if B == 1:
        sb = 0
    if S == 1:
        ss = 0
    if H == 1:
        sh = 0
    if se != 1:
        raise ValueError(f"the elements of a head of {name} must be contiguous")
    if (sb | ss | sh) & 7:
        raise ValueError(f"the strides of {name} must be multiples of 8")
    if written and ((sb == 0 and B > 1) or (ss == 0 and S > 1) or (sh == 0 and H > 1)):
        raise ValueError(f"{name} must not overlap itself")
    return _lib.QKView(t.data_ptr(), sb, ss, sh)


def _heads_out(t, name, like, stream):
    """(t or a new contiguous tensor of `like`'s shape, its view)."""
    if t is not None:
        return t, _heads(t, name, like.shape, True)
    dense = torch.contiguous_format
    t = (torch.empty_like(like, memory_format=dense) if stream is None
         else _allocate(stream, torch.empty_like, like, memory_format=dense))
    S, H, D = t.shape[-3:]
    return t, _lib.QKView(t.data_ptr(), S * H * D, H * D, D)


def _qk_call(q, k, cos, sin, positions, q_gain, k_gain, eps, interleaved):
    """Checked arguments of both passes: (shape, view of q, view of k, gains, cos, sin, positions as pointers)."""
    vq, vk = _heads(q, "q"), _heads(k, "k")
    *first, Hq, D = q.shape
    *others, Hk, Dk = k.shape
    if first != others or D != Dk:
        raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} differ in more than their heads")
    B, S = first if len(first) == 2 else (1, *first)
    _need(cos, "cos", torch.float32)
    if cos.dim() != 2:
        raise ValueError("cos must be [P, rot/2]")
    P, half = cos.shape
    _need(sin, "sin", torch.float32, (P, half))
    if (q_gain is None) != (k_gain is None):
        raise ValueError("q_gain and k_gain are given together or not at all")
    if q_gain is not None:
        _need(q_gain, "q_gain", BF16, (D,))
        _need(k_gain, "k_gain", BF16, (D,))
    stride = 0
    if positions is not None:
        _need(positions, "positions", torch.int64)
        if positions.shape == (B, S):
            stride = S
        elif positions.shape != (S,):
            raise ValueError(f"positions must be [{S}] or [{B}, {S}], got {list(positions.shape)}")
    shape = _lib.QKShape(B, S, Hq, Hk, D, 2 * half, P, stride, eps, 1 if interleaved else 0)
    return shape, vq, vk, (_p(q_gain), _p(k_gain), cos.data_ptr(), sin.data_ptr(), _p(positions))


def qk_norm_rope_forward(q: torch.Tensor, k: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor, *, positions=None,
                         q_gain=None, k_gain=None, eps: float = 1e-6, interleaved: bool = False, q_out=None,
                         k_out=None, stream=None):
    """(q_out, k_out): each head of q [B, S, Hq, D] and k [B, S, Hk, D] (or without B) normed (times q_gain, k_gain
    [D]; no norm without them) and turned by its position's angles, cos and sin fp32 [P, rot/2].  positions: int64
    [B, S] or [S], else 0 .. S-1.  Pairs are (i, i + rot/2), or (2i, 2i + 1) with interleaved; elements from rot on
    do not turn.  q, k and given outputs may be strided views; new outputs are contiguous.  q_out may be q itself, and
    k_out k (in place); outputs overlap nothing else."""
    shape, vq, vk, rest = _qk_call(q, k, cos, sin, positions, q_gain, k_gain, eps, interleaved)
    q_out, oq = _heads_out(q_out, "q_out", q, stream)
    k_out, ok = _heads_out(k_out, "k_out", k, stream)
    _lib.check(_lib.qk_rope_forward(shape, vq, vk, *rest, oq, ok, _stream(stream)), "lora_qk_rope_forward")
    return q_out, k_out


def qk_norm_rope_backward(q: torch.Tensor, k: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor,
                          dq_out: torch.Tensor, dk_out: torch.Tensor, *, positions=None, q_gain=None, k_gain=None,
                          eps: float = 1e-6, interleaved: bool = False, gain_grads: bool = True, dq=None, dk=None,
                          workspace: Workspace | None = None, stream=None):
    """(dq, dk, dq_gain, dk_gain) from the forward's arguments and the gradients of its results; the gains'
    gradients are fp32 [D], None without gains or with gain_grads=False (frozen gains).  dq may be dq_out itself or q,
    and dk likewise; given outputs overlap nothing else."""
    shape, vq, vk, rest = _qk_call(q, k, cos, sin, positions, q_gain, k_gain, eps, interleaved)
    vdq_out, vdk_out = _heads(dq_out, "dq_out", q.shape), _heads(dk_out, "dk_out", k.shape)
    dq, vdq = _heads_out(dq, "dq", q, stream)
    dk, vdk = _heads_out(dk, "dk", k, stream)
    dgq = dgk = ws = None
    if q_gain is not None and gain_grads:
        both = (2, shape.D)
        dgq, dgk = (q.new_empty(both, dtype=torch.float32) if stream is None
                    else _allocate(stream, q.new_empty, both, dtype=torch.float32)).unbind(0)
        ws = _scratch(workspace, _lib.qk_rope_sizes(shape), q.device, stream)
    _lib.check(_lib.qk_rope_backward(shape, vq, vk, *rest, vdq_out, vdk_out, vdq, vdk, _p(dgq), _p(dgk), _p(ws),
                                     0 if ws is None else ws.numel(), _stream(stream)), "lora_qk_rope_backward")
    return dq, dk, dgq, dgk


def _heads_or_copy(t):
    """t itself where the library takes its strides, else a contiguous copy (autograd hands over any)."""
    ok = t.stride(-1) == 1 and t.data_ptr() % 16 == 0 and all(s % 8 == 0 for s in t.stride()[:-1])
    return t if ok else t.contiguous()


class QKNormRopeFunction(torch.autograd.Function):
    """autograd wrapper of the norm and rotation of queries and keys.  Usage:
    QKNormRopeFunction.apply(q, k, cos, sin, positions, q_gain, k_gain, eps, interleaved) -> (q_out, k_out);
    the gains may be None, and get a gradient where they require one."""

    @staticmethod
    def forward(ctx, q, k, cos, sin, positions=None, q_gain=None, k_gain=None, eps=1e-6, interleaved=False):
        q, k = _heads_or_copy(q), _heads_or_copy(k)
        ctx.save_for_backward(q, k, cos, sin, positions, q_gain, k_gain)
        ctx.cfg = (eps, interleaved)
        return qk_norm_rope_forward(q, k, cos, sin, positions=positions, q_gain=q_gain, k_gain=k_gain, eps=eps,
                                    interleaved=interleaved)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, cos, sin, positions, q_gain, k_gain = ctx.saved_tensors
        eps, interleaved = ctx.cfg
        want = q_gain is not None and (ctx.needs_input_grad[5] or ctx.needs_input_grad[6])
        dq, dk, dgq, dgk = qk_norm_rope_backward(
            q, k, cos, sin, _heads_or_copy(dq_out), _heads_or_copy(dk_out), positions=positions, q_gain=q_gain,
            k_gain=k_gain, eps=eps, interleaved=interleaved, gain_grads=want)
        if want:
            dgq, dgk = dgq.to(q_gain.dtype), dgk.to(k_gain.dtype)
        return dq, dk, None, None, None, dgq, dgk, None, None


# ----------------------------------------------------------------------------- distillation


def _distill_call(logits, values, ids, labels, temperature, logit_scale, softcap, ignore_index):
    """Checked arguments of every pass: (shape, logits, values, ids, labels as pointers)."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits must be [N, V]")
    if logits.dtype != BF16 or not logits.is_cuda:
        raise TypeError("logits must be a bf16 CUDA tensor")
    if logits.stride(1) != 1 and logits.shape[1] > 1:
        raise ValueError("logits rows must be contiguous")
    N, V = logits.shape
    if not isinstance(values, torch.Tensor) or values.dim() != 2:
        raise ValueError("teacher_logits must be [N, K]")
    if values.dtype not in (BF16, torch.float32):
        raise TypeError("teacher_logits must be bf16 or fp32")
    K = values.shape[1]
    _need(values, "teacher_logits", values.dtype, (N, K))
    if not isinstance(ids, torch.Tensor) or ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("teacher_ids must be an int32 or int64 tensor")
    _need(ids, "teacher_ids", ids.dtype, (N, K))
    if labels is not None:
        _need(labels, "labels", torch.int64, (N,))
    ld = logits.stride(0) if N > 1 else (V + 7) // 8 * 8  # one row: its stride is never used
    shape = _lib.DistillShape(N, V, ld, K, temperature, logit_scale, softcap,
                              _lib.DISTILL_VALUES_BF16 if values.dtype == BF16 else _lib.DISTILL_VALUES_FP32,
                              _lib.DISTILL_IDS_INT32 if ids.dtype == torch.int32 else _lib.DISTILL_IDS_INT64,
                              ignore_index)
    return shape, (_p(logits), _p(values), _p(ids), _p(labels))


def _distill_out(logits, out, inplace, stream):
    # the gradient is written with the logits' row stride, as in ce_backward
    if inplace:
        return logits
    if out is None:
        n = logits.shape, logits.stride()
        return logits.new_empty_strided(*n) if stream is None else _allocate(stream, logits.new_empty_strided, *n)
    if out.shape != logits.shape or out.stride() != logits.stride() or out.dtype != BF16 or not out.is_cuda:
        raise ValueError("out must have the logits' shape, strides and dtype")
    return out


def distill_forward(logits: torch.Tensor, teacher_logits: torch.Tensor, teacher_ids: torch.Tensor, *, labels=None,
                    temperature: float = 1.0, logit_scale: float = 1.0, softcap: float = 0.0,
                    ignore_index: int = -100, stream=None):
    """loss [N] fp32: for each row of the student's bf16 logits [N, V] (row stride a multiple of 8), T^2 times the
    divergence of the student's softmax from the teacher's, taken over the teacher's K highest logits
    teacher_logits [N, K] (bf16 or fp32) at teacher_ids [N, K] (int32 or int64, -1: no entry).  0 for rows whose
    label (int64 [N], optional) is ignore_index and for rows without an entry."""
    shape, ptrs = _distill_call(logits, teacher_logits, teacher_ids, labels, temperature, logit_scale, softcap,
                                ignore_index)
    loss = _allocate(stream, logits.new_empty, (shape.N,), dtype=torch.float32)
    _lib.check(_lib.distill_forward(shape, *ptrs, _p(loss), _stream(stream)), "lora_distill_forward")
    return loss


def distill_backward(logits: torch.Tensor, teacher_logits: torch.Tensor, teacher_ids: torch.Tensor,
                     dloss: torch.Tensor, *, labels=None, temperature: float = 1.0, logit_scale: float = 1.0,
                     softcap: float = 0.0, ignore_index: int = -100, out=None, inplace: bool = False, stream=None):
    """dlogits [N, V] bf16 for the per-row upstream gradient dloss [N] (fp32).  inplace=True writes the gradient
    over the logits."""
    shape, ptrs = _distill_call(logits, teacher_logits, teacher_ids, labels, temperature, logit_scale, softcap,
                                ignore_index)
    _need(dloss, "dloss", torch.float32, (shape.N,))
    out = _distill_out(logits, out, inplace, stream)
    _lib.check(_lib.distill_backward(shape, *ptrs, _p(dloss), _p(out), _stream(stream)), "lora_distill_backward")
    return out


def distill_loss(logits: torch.Tensor, teacher_logits: torch.Tensor, teacher_ids: torch.Tensor, *, labels=None,
                 reduction: str = "mean", temperature: float = 1.0, logit_scale: float = 1.0, softcap: float = 0.0,
                 ignore_index: int = -100, with_grad: bool = True, grad_out=None, inplace: bool = False,
                 workspace: Workspace | None = None, stream=None):
    """The rows' losses reduced ("mean" over the rows whose label is not ignore_index, or "sum") and, with
    with_grad, the gradient in the same pass over the logits: returns (out [2] fp32, dlogits or None), out[0] the
    loss and out[1] its derivative with respect to a row's loss.  dlogits is the gradient of out[0]:
    logits.backward(dlogits) goes on from there.  inplace=True writes it over the logits."""
    red = {"sum": _lib.DISTILL_REDUCTION_SUM, "mean": _lib.DISTILL_REDUCTION_MEAN}.get(reduction)
    if red is None:
        raise ValueError("reduction must be 'sum' or 'mean'")
    shape, ptrs = _distill_call(logits, teacher_logits, teacher_ids, labels, temperature, logit_scale, softcap,
                                ignore_index)
    out = (logits.new_empty((2,), dtype=torch.float32) if stream is None
           else _allocate(stream, logits.new_empty, (2,), dtype=torch.float32))
    dlogits = _distill_out(logits, grad_out, inplace, stream) if with_grad else None
    ws = _scratch(workspace, _lib.distill_sizes(shape), logits.device, stream)
    _lib.check(_lib.distill_loss(shape, *ptrs, red, _p(out), _p(dlogits), _p(ws), ws.numel(), _stream(stream)),
               "lora_distill_loss")
    return out, dlogits


def distill_backward_reduced(logits: torch.Tensor, teacher_logits: torch.Tensor, teacher_ids: torch.Tensor,
                             dout: torch.Tensor, fwd_out: torch.Tensor, *, labels=None, temperature: float = 1.0,
                             logit_scale: float = 1.0, softcap: float = 0.0, ignore_index: int = -100, out=None,
                             inplace: bool = False, stream=None):
    """dlogits [N, V] bf16 for the upstream gradient dout (fp32, one element) of the loss distill_loss returned in
    fwd_out."""
    shape, ptrs = _distill_call(logits, teacher_logits, teacher_ids, labels, temperature, logit_scale, softcap,
                                ignore_index)
    _need(fwd_out, "fwd_out", torch.float32, (2,))
    if dout.numel() != 1 or dout.dtype != torch.float32 or not dout.is_cuda:
        raise TypeError("dout must be one fp32 CUDA element")
    out = _distill_out(logits, out, inplace, stream)
    _lib.check(_lib.distill_backward_reduced(shape, *ptrs, _p(dout), _p(fwd_out), _p(out), _stream(stream)),
               "lora_distill_backward_reduced")
    return out


class DistillFunction(torch.autograd.Function):
    """Mean distillation loss over the rows whose label is not ignore_index.  Usage:
    DistillFunction.apply(logits, teacher_logits, teacher_ids, labels, temperature, logit_scale, softcap,
    ignore_index, inplace) (labels may be None).  No gradient for the teacher.  The backward reads the logits again,
    so that it can apply any upstream gradient before it rounds; a loop whose loss is this one alone saves that
    reading with distill_loss.  inplace=True writes the gradient over the logits, whose version counter is then
    bumped, as in CrossEntropyFunction."""

    @staticmethod
    def forward(ctx, logits, teacher_logits, teacher_ids, labels=None, temperature=1.0, logit_scale=1.0, softcap=0.0,
                ignore_index=-100, inplace=False):
        kw = {"temperature": temperature, "logit_scale": logit_scale, "softcap": softcap,
              "ignore_index": ignore_index}
        out, _ = distill_loss(logits, teacher_logits, teacher_ids, labels=labels, with_grad=False, **kw)
        ctx.save_for_backward(logits, teacher_logits, teacher_ids, labels, out)
        ctx.cfg = (kw, bool(inplace))
        return out[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        logits, teacher_logits, teacher_ids, labels, out = ctx.saved_tensors
        kw, inplace = ctx.cfg
        if g.dtype != torch.float32 or not g.is_cuda:
            raise TypeError("the upstream gradient of the loss must be fp32 on the GPU")
        dz = distill_backward_reduced(logits, teacher_logits, teacher_ids, g.contiguous(), out, labels=labels,
                                      inplace=inplace, **kw)
        if inplace:
            torch.autograd.graph.increment_version(logits)
        return dz, None, None, None, None, None, None, None, None


# ----------------------------------------------------------------------------- status


def step_device_status(stream=None) -> int:
    """Reads and clears the device-side status of the operators around the dense layers (embedding, norm and rotation
    of queries and keys, distillation): 0, _lib.ERR_INVALID_ARG after an id or position outside its range, or
    _lib.ERR_DEVICE_TIMEOUT after a wait between blocks that ran out.  Synchronises the stream."""
    return _lib.step_device_status(_stream(stream))
