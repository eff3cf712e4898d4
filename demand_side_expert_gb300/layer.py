"""What stands around the expert passes in a training step, on one GPU.

``Router``      logits -> experts, weights, counts, balance loss and z-loss; and back
``AddRMSNorm``  residual addition, RMS norm, 8-bit rows with scales; and back
``AdamW``       one optimizer step over many tensors, moments in 32 bits or in 8

Each owns its output buffers and workspace (allocated once through PyTorch on
its current stream, some of them by the first call that writes them, whose own
stream then waits for the current one; reused every call: a call overwrites what
the one before it returned) and issues the C-ABI calls of liblrm on the stream
it is given, else on torch's current one; the current device has to be the one
of the buffers. Inputs are checked for type, shape, layout and device on the
host; a mismatch raises ValueError before anything is launched. A buffer that
another stream wrote or will read is the caller's to order, as for every call
here.
"""

from __future__ import annotations

import ctypes
from bisect import bisect_right

import torch

from . import lrm
from .pipeline import _TORCH_DTYPE, _after_current, _need, _stream, dtype_code

_route, _route_bwd = lrm.entry("lrm_route"), lrm.entry("lrm_route_bwd")
_norm, _norm_bwd = lrm.entry("lrm_add_rmsnorm"), lrm.entry("lrm_add_rmsnorm_bwd")


def _owned(name: str) -> property:
    """A buffer of the object's own. It cannot be replaced: its address is read once."""
    attr = "_" + name
    return property(lambda self: getattr(self, attr))


def _address(t):
    return None if t is None else t.data_ptr()


def _need_rows(t, name: str, shape: tuple, dtype: torch.dtype, device: torch.device) -> int:
    """A device matrix whose rows are contiguous; returns its row stride."""
    if t.dtype is dtype and t.shape == shape and t.device == device:
        rows, cols = shape
        stride, step = t.stride()
        if rows <= 1:  # the one row's stride means nothing
            stride = cols
        if (step == 1 or cols == 1) and stride >= cols:
            return stride
    raise ValueError(f"{name}: a {dtype} tensor {shape} with contiguous rows that do not overlap, "
                     f"on {device}, is needed, got {t.dtype} {tuple(t.shape)} strides "
                     f"{t.stride()} on {t.device}")


def _device(device) -> torch.device:
    dev = torch.device(device)
    if dev.type != "cuda":
        raise ValueError(f"a CUDA device is needed, got {dev}")
    here = torch.device("cuda", lrm.current_device())
    if dev.index is not None and dev != here:  # kernels launch on the current device
        raise ValueError(f"{dev} is not the current device, {here}")
    return here


class Router:
    """Top-K router of T tokens over E experts.

    After ``route``: ``topk_idx`` [T, K] int32 and ``alpha`` [T, K] float32 (what
    ``RecalibratedExpertBackward`` takes); with statistics also ``counts`` [E]
    int32, ``prob_sum`` [E] and ``loss`` [2] = (balance loss, z-loss). After
    ``backward``: ``dlogits`` [T, E] in the logits' type. See lrm_route and
    lrm_route_bwd in include/lrm.h for the definitions.
    """

    def __init__(self, T: int, E: int, K: int, dtype: str = "f32", renorm: bool = False,
                 balance_coef: float = 0.01, z_coef: float = 0.0,
                 device: str | torch.device = "cuda"):
        self.T, self.E, self.K = T, E, K
        self._shape = (T, E)
        self.tdtype = _TORCH_DTYPE[dtype_code(dtype)]
        self.desc = lrm.lrm_router(T, E, K, dtype_code(dtype), E, int(renorm), balance_coef,
                                   z_coef)
        self.ws_bytes = lrm.lrm_router_workspace_bytes(self.desc)
        if self.ws_bytes == 0:
            raise ValueError(f"unsupported router shape T={T} E={E} K={K}: 1 <= K <= min(E, 32), "
                             "E <= 1024 and T*K < 2^31 are needed")
        self.device = dev = _device(device)

        def empty(*shape, dtype=torch.float32):
            return torch.empty(*shape, dtype=dtype, device=dev)

        with torch.inference_mode(False):  # inference tensors do not count their writes
            self._ws = empty(self.ws_bytes, dtype=torch.uint8)
            self._topk_idx, self._alpha = empty(T, K, dtype=torch.int32), empty(T, K)
            self._counts, self._prob_sum = empty(E, dtype=torch.int32), empty(E)
            self._loss = empty(2)
        self._dlogits = None
        # what backward may read: ids and counts of a route, or written by the caller since
        self._routed = self._counted = T == 0  # no token, nothing to read
        self._idx_at, self._counts_at = self._topk_idx._version, self._counts._version
        self._ref = ctypes.byref(self.desc)
        self._at = tuple(t.data_ptr() for t in (self._topk_idx, self._alpha, self._counts,
                                                self._prob_sum, self._loss, self._ws))
        lrm.lrm_clear_device_error(self._ws, self.ws_bytes)

    topk_idx, alpha, counts = _owned("topk_idx"), _owned("alpha"), _owned("counts")
    prob_sum, loss, ws = _owned("prob_sum"), _owned("loss"), _owned("ws")

    @property
    def dlogits(self) -> torch.Tensor:
        if self._dlogits is None:  # a router that only serves has no gradient
            self._dlogits = torch.empty(self.T, self.E, dtype=self.tdtype, device=self.device)
        return self._dlogits

    def _inputs(self, logits, mask):
        self.desc.stride = _need_rows(logits, "logits", self._shape, self.tdtype, self.device)
        if mask is not None:
            if mask.dtype is torch.bool:
                mask = mask.view(torch.uint8)
            _need(mask, "mask", (self.T,), torch.uint8, self.device)
        return mask

    def route(self, logits, mask=None, stats: bool = True, stream=None):
        """Routes the tokens of ``logits`` [T, E] (rows may be strided). ``mask`` [T]
        bool or uint8: tokens that are 0 there get weight 0 and count nowhere.
        ``stats=False`` skips counts and losses (serving)."""
        mask = self._inputs(logits, mask)
        at = _stream(self.device, stream)
        topk_idx, alpha, counts, prob_sum, loss, ws = self._at
        if not stats:
            counts = prob_sum = loss = None
        _route(self._ref, logits.data_ptr(), _address(mask), topk_idx, alpha, counts, prob_sum,
               loss, ws, self.ws_bytes, at)
        self._routed, self._counted = True, stats or self.T == 0
        if not stats:
            self._counts_at = self._counts._version

    def backward(self, logits, dalpha=None, mask=None, dloss=None, stream=None):
        """The logits' gradient, from the choices and counts of the last ``route``
        (with statistics) on the same logits and mask. ``dalpha`` [T, K] float32
        (``RecalibratedExpertBackward.gate_grad``), ``dloss`` [2] float32: what the
        two losses weigh in the total (1 each by default). Choices and counts that the
        caller wrote into ``topk_idx`` and ``counts`` serve as well; without either
        the call is refused (counts are not needed where both coefficients are 0)."""
        mask = self._inputs(logits, mask)
        if not self._routed and self._topk_idx._version == self._idx_at:
            raise ValueError("no choices to take the gradient of: call route before")
        if not self._counted and self._counts._version == self._counts_at and \
                (self.desc.balance_coef != 0 or self.desc.z_coef != 0):
            raise ValueError("the last route had no statistics, and the losses' gradient needs "
                             "its counts")
        if dalpha is not None:
            _need(dalpha, "dalpha", (self.T, self.K), torch.float32, self.device)
        if dloss is not None:
            _need(dloss, "dloss", (2,), torch.float32, self.device)
        at = _stream(self.device, stream)
        topk_idx, _, counts, _, _, ws = self._at
        if self._dlogits is None:
            _after_current(stream)
        _route_bwd(self._ref, logits.data_ptr(), _address(mask), topk_idx, counts,
                   _address(dalpha), _address(dloss), self.dlogits.data_ptr(), ws, self.ws_bytes,
                   at)

    def device_error(self, stream=None) -> int:
        return lrm.lrm_get_device_error(self._ws, self.ws_bytes, stream)


class AddRMSNorm:
    """RMS norm of T rows of D columns, the residual's addition in front.

    After ``forward``: ``h`` [T, D] (the sum, with a residual), ``y`` [T, D],
    ``rstd`` [T] float32; with ``q_cols`` given also ``q`` [T, D] float8_e4m3fn
    and ``q_scale`` [T, ceil(D / q_cols)] float32, y ~ q * scale (q_cols = 0: one
    scale a row). ``store_y`` (default: without 8-bit rows only) says whether y
    is written too. After ``backward``: ``dx`` [T, D] in ``grad_dtype``, the
    gradient of x and of the residual alike, and ``dw`` [D] float32.
    """

    def __init__(self, T: int, D: int, dtype: str = "bf16", eps: float = 1e-6,
                 q_cols: int | None = None, store_y: bool | None = None,
                 grad_dtype: str = "f32", device: str | torch.device = "cuda"):
        self.T, self.D = T, D
        self._shape, self._columns = (T, D), (D,)
        self.tdtype = _TORCH_DTYPE[dtype_code(dtype)]
        self.gdtype = _TORCH_DTYPE[dtype_code(grad_dtype)]
        self.desc = lrm.lrm_norm(T, D, dtype_code(dtype), dtype_code(grad_dtype), q_cols or 0,
                                 eps, D, D)
        self.ws_bytes = lrm.lrm_norm_workspace_bytes(self.desc)
        if self.ws_bytes == 0:
            raise ValueError(f"unsupported norm T={T} D={D} q_cols={q_cols} eps={eps}: D a "
                             "multiple of 8 up to 16384, q_cols one of 0, 32, 64, 128, 256 and "
                             "eps >= 0 are needed")
        self.device = dev = _device(device)

        def empty(*shape, dtype=torch.float32):
            return torch.empty(*shape, dtype=dtype, device=dev)

        with torch.inference_mode(False):  # inference tensors do not count their writes
            self._rstd = empty(T)
        self._rstd_at = self._rstd._version  # another one: the caller wrote it
        store_y = q_cols is None if store_y is None else store_y
        if q_cols is None and not store_y:
            raise ValueError("store_y=False leaves no output without q_cols")
        self._y = empty(T, D, dtype=self.tdtype) if store_y else None
        self._q = self._q_scale = None
        if q_cols is not None:
            self._q = empty(T, D, dtype=torch.float8_e4m3fn)
            self._q_scale = empty(T, -(-D // q_cols) if q_cols else 1)
        self._h = self._dx = self._dw = self._ws = None
        self._normed = T == 0  # there is a 1/rms to take the gradient with
        self._summed = False  # the last forward had a residual: h is its sum
        self._ref = ctypes.byref(self.desc)
        self._at = tuple(_address(t) for t in (self._y, self._q, self._q_scale, self._rstd))

    y, q, q_scale, rstd = _owned("y"), _owned("q"), _owned("q_scale"), _owned("rstd")

    @property
    def h(self) -> torch.Tensor:
        if self._h is None:
            self._h = torch.empty(self.T, self.D, dtype=self.tdtype, device=self.device)
        return self._h

    def _backward_buffers(self):
        """Gradients and workspace, allocated on the first backward call only."""
        if self._dx is None:
            dev = self.device
            self._dx = torch.empty(self.T, self.D, dtype=self.gdtype, device=dev)
            self._dw = torch.empty(self.D, dtype=torch.float32, device=dev)
            self._ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)

    @property
    def dx(self) -> torch.Tensor:
        self._backward_buffers()
        return self._dx

    @property
    def dw(self) -> torch.Tensor:
        self._backward_buffers()
        return self._dw

    def forward(self, x, w, residual=None, stream=None):
        """x, residual [T, D] (rows may be strided by a multiple of 8 elements), w [D]."""
        dt, dev = self.tdtype, self.device
        x_stride = _need_rows(x, "x", self._shape, dt, dev)
        _need(w, "w", self._columns, dt, dev)
        res, h, res_stride = None, None, self.D
        if residual is not None:
            res_stride = _need_rows(residual, "residual", self._shape, dt, dev)
            res = residual.data_ptr()
        at = _stream(dev, stream)
        if residual is not None:
            if self._h is None:
                _after_current(stream)
            h = self.h.data_ptr()
        desc = self.desc
        desc.x_stride, desc.res_stride = x_stride, res_stride
        y, q, q_scale, rstd = self._at
        try:
            _norm(self._ref, x.data_ptr(), res, w.data_ptr(), h, y, q, q_scale, rstd, at)
        except lrm.LrmError:
            desc.x_stride = desc.res_stride = self.D  # backward is not refused for them
            raise
        self._normed, self._summed = True, residual is not None

    def backward(self, dy, w, dh=None, h=None, stream=None):
        """dy [T, D]: the cotangent of y; dh: of the stored sum (the residual
        stream), or None. ``h``: the normed rows, self.h by default (pass x where
        there was no residual). Uses ``rstd`` of the last forward, or what the caller
        wrote there."""
        dt, gt, dev, shape = self.tdtype, self.gdtype, self.device, self._shape
        if not self._normed and self._rstd._version == self._rstd_at:
            raise ValueError("no 1/rms to take the gradient with: call forward before")
        if h is not None:
            _need(h, "h", shape, dt, dev)
        elif self._summed:
            h = self._h
        else:
            raise ValueError("h: the last forward had no residual, so pass its x")
        _need(dy, "dy", shape, gt, dev)
        if dh is not None:
            _need(dh, "dh", shape, gt, dev)
        _need(w, "w", self._columns, dt, dev)
        at = _stream(dev, stream)
        if self._dx is None:
            _after_current(stream)
        self._backward_buffers()
        _norm_bwd(self._ref, dy.data_ptr(), _address(dh), h.data_ptr(), w.data_ptr(), self._at[3],
                  self._dx.data_ptr(), self._dw.data_ptr(), self._ws.data_ptr(), self.ws_bytes, at)


_STATE = {"f32": lrm.LRM_STATE_F32, "f8": lrm.LRM_STATE_F8}
_STATE_BLOCK = 256
_CODE = {torch.float32: lrm.LRM_F32, torch.bfloat16: lrm.LRM_BF16}


def _addresses(tensors) -> list:
    return list(map(torch.Tensor.data_ptr, tensors))


def _spans(tensors) -> list:
    """(first byte, one past the last, index) of the tensors that hold any, in order."""
    return sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), i)
                  for i, t in enumerate(tensors) if t.numel())


def _moved(name: str, tensors, at) -> str:
    which = [f"{name}[{i}]" for i, (t, a) in enumerate(zip(tensors, at)) if t.data_ptr() != a]
    return f"{', '.join(which) or name}: not the storage taken before; "


class AdamW:
    """AdamW over a list of tensors, all of them in one call of liblrm.

    ``params`` and ``grads``: contiguous float32 or bfloat16 device tensors, read
    and updated in place (the framework's dw_gate, dw_up, dw_down are such
    gradients). No parameter may overlap another, nor a gradient but its own. ``weight_decay``: one number, or one a tensor. ``state``: "f32",
    or "f8" for 8-bit moments (e4m3 codes of m and of sqrt(v), one float32 scale
    for 256 values each). ``master=True`` keeps float32 copies beside bfloat16
    parameters.

    The tensors' storage is taken at construction: ``step`` refuses one that was
    given other storage since (a new AdamW, or ``set_grads``, takes it). The state
    lives in flat buffers over all tensors, each tensor beginning on a whole block
    of 256: ``m``, ``v`` (float32, or float8_e4m3fn with v holding the root),
    ``m_scale``, ``v_scale``, ``master`` (or None); tensor i holds
    [starts[i], starts[i] + numel).
    """

    m, v, master = _owned("m"), _owned("v"), _owned("master")
    m_scale, v_scale = _owned("m_scale"), _owned("v_scale")

    def __init__(self, params, grads, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay=0.01, state: str = "f32", master: bool = False):
        self.params, self.grads = list(params), list(grads)
        if len(self.params) != len(self.grads) or not self.params:
            raise ValueError(f"{len(self.params)} parameters and {len(self.grads)} gradients")
        if state not in _STATE:
            raise ValueError(f"state: 'f32' or 'f8', got {state!r}")
        if not (0 <= betas[0] < 1 and 0 <= betas[1] < 1 and eps >= 0):
            raise ValueError(f"betas in [0, 1) and eps >= 0 are needed, got {betas}, {eps}")
        n = len(self.params)
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else \
            [weight_decay] * n
        if len(decay) != n:
            raise ValueError(f"{len(decay)} weight decays for {n} tensors")
        self.device = dev = _device(self.params[0].device)
        self.lr, self.t, self.state = lr, 0, state
        self.starts, total = [], 0
        for i, p in enumerate(self.params):
            if p.dtype not in _CODE:
                raise ValueError(f"params[{i}]: float32 or bfloat16 is needed, got {p.dtype}")
            _need(p, f"params[{i}]", tuple(p.shape), p.dtype, dev)
            self.starts.append(total)
            total += -(-p.numel() // _STATE_BLOCK) * _STATE_BLOCK
        self._spans = _spans(self.params)
        for (_, end, i), (begin, _, j) in zip(self._spans, self._spans[1:]):
            if begin < end:  # two CTAs would update that memory at once
                raise ValueError(f"params[{i}] and params[{j}] overlap")
        blocks = total // _STATE_BLOCK
        f8 = state == "f8"
        st = torch.float8_e4m3fn if f8 else torch.float32
        self._m = torch.zeros(total, dtype=torch.uint8 if f8 else st, device=dev).view(st)
        self._v = torch.zeros(total, dtype=torch.uint8 if f8 else st, device=dev).view(st)
        self._m_scale = torch.zeros(blocks, device=dev) if f8 else None
        self._v_scale = torch.zeros(blocks, device=dev) if f8 else None
        master = master and any(p.dtype is torch.bfloat16 for p in self.params)
        self._master = torch.zeros(total, device=dev) if master else None
        if master:
            for p, a in zip(self.params, self.starts):
                self.master[a:a + p.numel()].copy_(p.detach().reshape(-1))
        self._hyper = lrm.lrm_adamw(lr, betas[0], betas[1], eps, 1, None)
        self._table = (lrm.lrm_adamw_tensor * n)()
        for i, (p, a) in enumerate(zip(self.params, self.starts)):
            s = self._table[i]
            s.param, s.n, s.param_dtype = p.data_ptr(), p.numel(), _CODE[p.dtype]
            s.master = self.master.data_ptr() + 4 * a \
                if master and p.dtype is torch.bfloat16 else None
            s.m = self.m.data_ptr() + a * self.m.element_size()
            s.v = self.v.data_ptr() + a * self.v.element_size()
            if f8:
                s.m_scale = self.m_scale.data_ptr() + 4 * (a // _STATE_BLOCK)
                s.v_scale = self.v_scale.data_ptr() + 4 * (a // _STATE_BLOCK)
            s.state, s.weight_decay = _STATE[state], decay[i]
        self._params_at = _addresses(self.params)
        self.set_grads(self.grads)

    def set_grads(self, grads):
        """Other gradient tensors for the same parameters."""
        grads = list(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"{len(self.params)} parameters and {len(grads)} gradients")
        for i, (p, g) in enumerate(zip(self.params, grads)):
            if g.dtype not in _CODE:
                raise ValueError(f"grads[{i}]: float32 or bfloat16 is needed, got {g.dtype}")
            _need(g, f"grads[{i}]", tuple(p.shape), g.dtype, self.device)
        for begin, end, i in _spans(grads):
            k = bisect_right(self._spans, (begin, float("inf")))
            for lo, hi, j in self._spans[max(k - 1, 0):k + 1]:
                # a gradient that is its own parameter is read where it is written
                if begin < hi and lo < end and not (i == j and (begin, end) == (lo, hi)):
                    raise ValueError(f"grads[{i}] and params[{j}] overlap")
        # all of them checked: the table never points to a tensor that is not held
        self.grads = grads
        for s, g in zip(self._table, grads):
            s.grad, s.grad_dtype = g.data_ptr(), _CODE[g.dtype]
        self._grads_at = _addresses(grads)

    def step(self, lr: float | None = None, grad_scale=None, stream=None):
        """One update. ``lr`` for this step only; ``grad_scale``: a float32 device
        scalar that every gradient is multiplied by (clipping, loss scaling)."""
        if grad_scale is not None:
            if grad_scale.numel() != 1:
                raise ValueError("grad_scale: one float32 value is needed")
            _need(grad_scale, "grad_scale", tuple(grad_scale.shape), torch.float32, self.device)
        if _addresses(self.params) != self._params_at:
            raise ValueError(_moved("params", self.params, self._params_at) + "make a new AdamW")
        if _addresses(self.grads) != self._grads_at:
            raise ValueError(_moved("grads", self.grads, self._grads_at) + "call set_grads")
        at = _stream(self.device, stream)
        h = self._hyper
        h.lr = self.lr if lr is None else lr
        h.step = self.t + 1
        h.grad_scale = None if grad_scale is None else grad_scale.data_ptr()
        lrm.lrm_adamw_step(h, self._table, len(self._table), at)
        self.t += 1

    def state_dict(self) -> dict:
        """The state's own buffers (clone them to keep a copy)."""
        return {"step": self.t, "master": self.master, "m": self.m, "v": self.v,
                "m_scale": self.m_scale, "v_scale": self.v_scale}

    def load_state_dict(self, state: dict):
        """Copies a state of the same layout in; on torch's current stream. The
        parameters are left as they are."""
        t, pairs = int(state["step"]), []
        if t < 0:
            raise ValueError(f"step: {t}")
        for name in ("master", "m", "v", "m_scale", "v_scale"):
            mine, other = getattr(self, name), state.get(name)
            if (mine is None) != (other is None):
                raise ValueError(f"{name}: the two states are of different kinds")
            if mine is not None:
                if other.shape != mine.shape or other.dtype is not mine.dtype:
                    raise ValueError(f"{name}: {mine.dtype} {tuple(mine.shape)} is needed, got "
                                     f"{other.dtype} {tuple(other.shape)}")
                pairs.append((mine, other))
        for mine, other in pairs:  # all of them checked
            mine.copy_(other.detach())
        self.t = t
