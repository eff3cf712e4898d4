"""Host orchestration of the recalibrated expert backward on one GPU.

``RecalibratedExpertBackward`` owns the device buffers of one layer shape
(allocated once through PyTorch, reused every step) and issues the C-ABI
calls of liblrm in order on one CUDA stream:

  lrm_dispatch_permute -> lrm_quota_from_rate -> lrm_score ->
  lrm_select_quota -> lrm_compact -> lrm_expert_bwd_grouped

and, for the forward expert pass that produces the saved state,
lrm_dispatch_permute -> lrm_expert_fwd_grouped.

Every step of the path runs in liblrm's kernels; this class only allocates
and passes pointers.
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import lrm

_TORCH_DTYPE = {lrm.LRM_F32: torch.float32, lrm.LRM_BF16: torch.bfloat16}


def dtype_code(name: str) -> int:
    return {"f32": lrm.LRM_F32, "bf16": lrm.LRM_BF16}[name]


def _need(t, name: str, shape: tuple, dtype: torch.dtype, device: torch.device):
    """A contiguous device tensor of this shape and type."""
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor {shape} on {device} is needed, got "
                         f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")
    return t


# The current device and its current stream's address, by the functions that torch's own
# compiled kernels are launched with: 0.1 us each, where a Stream object takes 3.
_device_now = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_stream_now = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream(device: torch.device, stream) -> int:
    """Address of a call's stream. Kernels launch on the current device, so that has to be
    the one of the call's buffers."""
    here = _device_now()
    if here != device.index:
        raise ValueError(f"the buffers are on {device}, the current device is cuda:{here}")
    return _stream_now(here) if stream is None else lrm.stream_address(stream)


def _after_current(stream):
    """Makes ``stream`` wait for torch's current one, for a buffer that a call on it
    allocates: the memory comes from the current stream's pool, and what it held
    before may have work pending there."""
    if stream is None:
        return
    current = torch.cuda.current_stream()
    address = lrm.stream_address(stream)
    if address == current.cuda_stream:
        return
    # ExternalStream takes address 0 for a new stream
    other = torch.cuda.ExternalStream(address) if address else torch.cuda.default_stream()
    other.wait_stream(current)


_pack = lrm.entry("lrm_pack_state")


def _device(device) -> torch.device:
    dev = torch.device(device)
    if dev.type != "cuda":
        raise ValueError(f"a CUDA device is needed, got {dev}")
    here = torch.device("cuda", lrm.current_device())
    if dev.index is not None and dev != here:  # kernels launch on the current device
        raise ValueError(f"{dev} is not the current device, {here}")
    return here


class PackedState:
    """The saved state of T * K routed pairs in 8 bits, in the place of [a | b] and phi.

    After ``pack``: ``q`` [N, 2H] float8_e4m3fn, ``scale`` [N, 2 ceil(H / cols)]
    float32 (the groups of a, then those of b) and ``phi_sq`` [N] float32, |phi|^2 of the
    unquantised state. 2H + 8 ceil(H / cols) + 4 bytes a pair instead of 6H in bfloat16.
    ``RecalibratedExpertBackward.forward`` packs into one, ``.step`` takes it in the place
    of [a | b]. See lrm_pack_state in include/lrm.h for the definitions.
    """

    def __init__(self, T: int, K: int, H: int, dtype: str = "bf16", cols: int = 128,
                 device: str | torch.device = "cuda"):
        self.N, self.H, self.cols = T * K, H, cols
        self.dtype_code = dtype_code(dtype)
        self.tdtype = _TORCH_DTYPE[self.dtype_code]
        if T < 0 or K <= 0 or H <= 0 or H % 8 or cols not in (32, 64, 128) or \
                max(self.N, H) >= 1 << 31:
            raise ValueError(f"unsupported state T={T} K={K} H={H} cols={cols}: H a multiple of "
                             "8, cols one of 32, 64, 128, T*K and H below 2^31 are needed")
        self.device = dev = _device(device)
        with torch.inference_mode(False):  # inference tensors do not count their writes
            self._q = torch.empty(self.N, 2 * H, dtype=torch.uint8, device=dev).view(
                torch.float8_e4m3fn)
            self._scale = torch.empty(self.N, 2 * -(-H // cols), device=dev)
            self._phi_sq = torch.empty(self.N, device=dev)
        self._filled = self.N == 0
        self._q_at = self._q._version  # another one: the caller wrote it
        self.desc = lrm.lrm_packed(self._q.data_ptr(), self._scale.data_ptr(),
                                   self._phi_sq.data_ptr(), self.N, H, cols, self.dtype_code, 0)
        self._ref = ctypes.byref(self.desc)

    q = property(lambda self: self._q)
    scale = property(lambda self: self._scale)
    phi_sq = property(lambda self: self._phi_sq)

    @property
    def filled(self) -> bool:
        """Whether there is a state: of ``pack``, or written by the caller."""
        return self._filled or self._q._version != self._q_at

    def pack(self, ab, stream=None):
        """Quantises ab [N, 2H], in the layer's type."""
        _need(ab, "ab", (self.N, 2 * self.H), self.tdtype, self.device)
        _pack(self._ref, ab.data_ptr(), _stream(self.device, stream))
        self._filled = True


def _x_groups(D: int, groups: int) -> int:
    """Columns under one scale of 8-bit rows with ``groups`` scales (0: a scale a row)."""
    for cols in (0, 256, 128, 64, 32):
        if groups == (-(-D // cols) if cols else 1):
            return cols
    raise ValueError(f"x: {groups} scales for {D} columns")


def _weight_gradient(name: str) -> property:
    """A float32 output of the backward pass that the caller may give memory for."""
    attr = "_" + name

    def give(self, t):
        if t is None:
            raise ValueError(f"{name}: the backward pass writes it")
        shape = (self.E, self.H, self.D) if name == "dw_down" else (self.E, self.D, self.H)
        setattr(self, attr, self._own(t, name, shape, torch.float32))

    return property(lambda self: getattr(self, attr), give)


class RecalibratedExpertBackward:
    """Buffers + call sequence for one (T, D, H, E, K, dtype) layer shape."""

    def __init__(self, T: int, D: int, H: int, E: int, K: int, dtype: str = "bf16",
                 device: str | torch.device = "cuda"):
        self.T, self.D, self.H, self.E, self.K = T, D, H, E, K
        self.N = T * K
        self.dtype_code = dtype_code(dtype)
        self.tdtype = _TORCH_DTYPE[self.dtype_code]
        self.shape = lrm.make_shape(T, D, H, E, K, self.dtype_code)
        dev = torch.device(device)
        self.device = dev
        i32, f32, dt = torch.int32, torch.float32, self.tdtype
        rows = max(self.N, 1)

        def empty(*shape, dtype):
            return torch.empty(*shape, dtype=dtype, device=dev)

        self.ws_bytes = lrm.lrm_workspace_bytes(self.shape)
        if self.ws_bytes == 0:
            raise lrm.LrmError("lrm_workspace_bytes", lrm.LRM_ERR_INVALID_ARG)
        self.ws = empty(self.ws_bytes, dtype=torch.uint8)
        self.perm, self.inv = empty(rows, dtype=i32), empty(rows, dtype=i32)
        self.counts, self.off = empty(E, dtype=i32), empty(E + 1, dtype=i32)
        self.quota = empty(E, dtype=i32)
        self.score = empty(rows, dtype=f32)
        self.keep = empty(rows, dtype=torch.uint8)
        self.sel_off, self.sel_pos = empty(E + 1, dtype=i32), empty(rows, dtype=i32)
        self.dy_c, self.x_c = empty(rows, D, dtype=dt), empty(rows, D, dtype=dt)
        self.ab_c, self.phi_c = empty(rows, 2 * H, dtype=dt), empty(rows, H, dtype=dt)
        self.tok_c, self.row_of_pos = empty(rows, dtype=i32), empty(rows, dtype=i32)
        self.dab_c, self.dx_c = empty(rows, 2 * H, dtype=dt), empty(rows, D, dtype=f32)
        self._dw_gate, self._dw_up = empty(E, D, H, dtype=f32), empty(E, D, H, dtype=f32)
        self._dw_down = empty(E, H, D, dtype=f32)
        self.dx = empty(max(T, 1), D, dtype=f32)
        self._y = self._out = None
        lrm.lrm_clear_device_error(self.ws, self.ws_bytes)

    dw_gate, dw_up = _weight_gradient("dw_gate"), _weight_gradient("dw_up")
    dw_down = _weight_gradient("dw_down")

    # -- forward side -------------------------------------------------------
    def dispatch(self, topk_idx, stream=None):
        lrm.lrm_dispatch_permute(self.shape, topk_idx, self.perm, self.inv, self.counts,
                                 self.off, self.ws, self.ws_bytes, stream)

    def _forward_buffers(self, stream):
        """Forward outputs, allocated on the first forward call only."""
        if getattr(self, "x_disp", None) is None:
            _after_current(stream)
            rows, dt, dev = max(self.N, 1), self.tdtype, self.device
            self.x_disp = torch.empty(rows, self.D, dtype=dt, device=dev)
            self.ab = torch.empty(rows, 2 * self.H, dtype=dt, device=dev)
            self.phi = torch.empty(rows, self.H, dtype=dt, device=dev)
        if self._out is None:
            _after_current(stream)
            self._out = torch.empty(max(self.T, 1), self.D, dtype=torch.float32,
                                    device=self.device)

    def _expert_outputs(self, stream):
        if self._y is None:
            _after_current(stream)
            self._y = torch.empty(max(self.N, 1), self.D, dtype=self.tdtype, device=self.device)
        return self._y

    @property
    def y(self) -> torch.Tensor:
        """Expert outputs [N, D] in dispatch order. Allocated by the first forward product
        that writes it, or for a caller who asks for it: until then there is nothing
        for ``gate_grad`` to read."""
        return self._expert_outputs(None)

    @y.setter
    def y(self, rows):
        self._y = self._own(rows, "y", (self.N, self.D), self.tdtype)

    @property
    def out(self) -> torch.Tensor:
        """The layer output [T, D], float32. Allocated by the first forward call."""
        if self._out is None:
            raise AttributeError("out: there was no forward call")
        return self._out

    @out.setter
    def out(self, rows):
        self._out = self._own(rows, "out", (self.T, self.D), torch.float32)

    def _own(self, t, name: str, shape: tuple, dtype: torch.dtype):
        """Memory of the caller's for an output of this shape (None: none)."""
        if t is not None and (t.dtype is not dtype or t.device != self.ws.device or
                              not t.is_contiguous() or t.numel() < math.prod(shape)):
            raise ValueError(f"{name}: a contiguous {dtype} tensor {shape} on {self.ws.device} is "
                             f"needed, got {t.dtype} {tuple(t.shape)} strides {t.stride()} on "
                             f"{t.device}")
        return t

    def forward(self, topk_idx, alpha, x, w_gate, w_up, w_down, stream=None,
                packed: PackedState | None = None):
        """Forward expert pass: dispatch, gather, gate/up + SwiGLU, down,
        combine. Leaves the saved state in ``ab`` / ``phi`` (dispatch order)
        and the layer output in ``out`` (float32 [T, D]). ``packed`` gets the
        state in 8 bits: ``ab`` and ``phi`` may then serve the next layer.

        One object can so serve several layers of its shape, forward one after
        the other and back again. What stays a layer's own until its backward
        pass, beside x, the choices and ``packed``: ``y`` where ``gate_grad`` is
        to be called, ``out`` where something reads it, and ``dw_gate``,
        ``dw_up``, ``dw_down``. Assign the layer's own rows to these before the
        call that writes or reads them; ``gate_grad`` says what else it needs."""
        if packed is not None:
            self._check_packed(packed)
        self._forward_buffers(stream)
        self._expert_outputs(stream)
        self.dispatch(topk_idx, stream)
        lrm.lrm_expert_fwd_grouped(self.shape, self.perm, self.inv, self.off, alpha, x, w_gate,
                                   w_up, w_down, self.x_disp, self.ab, self.phi, self.y,
                                   self.out, self.ws, self.ws_bytes, stream)
        if packed is not None:
            packed.pack(self.ab[:self.N], stream)

    def _check_packed(self, packed: PackedState, filled: bool = False):
        if packed.N != self.N or packed.H != self.H or packed.tdtype is not self.tdtype:
            raise ValueError(f"packed: a state of {self.N} pairs, H={self.H}, {self.tdtype} is "
                             f"needed, got {packed.N}, {packed.H}, {packed.tdtype}")
        if packed.device != self.ws.device:
            raise ValueError(f"packed: on {packed.device}, the buffers are on {self.ws.device}")
        if filled and not packed.filled:
            raise ValueError("packed: nothing has been packed into it")

    def gather_tokens(self, x, stream=None):
        self._forward_buffers(stream)
        lrm.lrm_gather_tokens(self.shape, self.perm, x, self.x_disp, self.ws, self.ws_bytes,
                              stream)

    def fc1_fwd(self, w_gate, w_up, stream=None):
        lrm.lrm_expert_fc1_fwd(self.shape, self.off, self.x_disp, w_gate, w_up, self.ab,
                               self.phi, self.ws, self.ws_bytes, stream)

    def fc2_fwd(self, w_down, stream=None):
        self._expert_outputs(stream)
        lrm.lrm_expert_fc2_fwd(self.shape, self.off, self.phi, w_down, self.y, self.ws,
                               self.ws_bytes, stream)

    def combine(self, alpha, stream=None):
        lrm.lrm_combine(self.shape, self.y, alpha, self.inv, self.out, self.ws, self.ws_bytes,
                        stream)

    def gate_grad(self, g, stream=None) -> torch.Tensor:
        """Gradient of the routing weights [T, K] (float32) from the cotangent g
        [T, D] of the layer output, in the layer's type, and the rows ``y`` of the
        last forward, in the order of the last dispatch. Where other layers have
        used the object since: assign this layer's rows to ``y``, and call it after
        its ``step``, or ``dispatch``, with its choices."""
        if self._y is None:
            raise RuntimeError("gate_grad needs the expert outputs of a forward call")
        device = self.ws.device
        _need(g, "g", (self.T, self.D), self.tdtype, device)
        at = _stream(device, stream)
        if getattr(self, "dalpha", None) is None:
            _after_current(stream)
            self.dalpha = torch.empty(max(self.T, 1), self.K, dtype=torch.float32,
                                      device=self.device)[: self.T]
        lrm.lrm_gate_grad(self.shape, g, self._y, self.inv, self.dalpha, self.ws, self.ws_bytes,
                          at)
        return self.dalpha

    def to_dispatch_order(self, rows_by_pair: torch.Tensor, stream=None) -> torch.Tensor:
        """Lay per-pair rows out in dispatch order with the current perm."""
        out = torch.empty_like(rows_by_pair)
        row_bytes = rows_by_pair[0].numel() * rows_by_pair.element_size()
        lrm.lrm_permute_rows(self.perm, self.N, rows_by_pair, out, row_bytes, stream)
        return out

    # -- backward -----------------------------------------------------------
    def quota_from_rate(self, num: int, den: int, cap: int = 0, stream=None):
        lrm.lrm_quota_from_rate(self.counts, self.E, num, den, cap, self.quota, stream)

    def score_pairs(self, alpha, g, phi, stream=None, metric: int = 0, seed: int = 0):
        """LRM scores (metric 0) or one of the ablation criteria (lrm.LRM_METRIC_*).
        phi may be a PackedState, which holds its rows' squares."""
        if isinstance(phi, PackedState):
            self._check_packed(phi, filled=True)
            if metric == lrm.LRM_METRIC_LRM:
                lrm.lrm_score_packed(self.shape, phi.desc, g, alpha, self.inv, self.score, self.ws,
                                     self.ws_bytes, _stream(phi.device, stream))
                return
            phi = None  # the other criteria do not read it
        if metric == lrm.LRM_METRIC_LRM:
            lrm.lrm_score(self.shape, g, phi, alpha, self.inv, self.score, self.ws,
                          self.ws_bytes, stream)
        else:
            lrm.lrm_score_variant(self.shape, metric, seed, g, phi, alpha, self.inv, self.score,
                                  self.ws, self.ws_bytes, stream)

    def select_rate(self, num: int, den: int, cap: int = 0, stream=None):
        """Quotas from the rate and the selection in one launch."""
        lrm.lrm_select_rate(self.shape, self.score, self.off, num, den, cap, self.quota,
                            self.keep, self.sel_off, self.sel_pos, self.ws, self.ws_bytes, stream)

    def select(self, stream=None):
        lrm.lrm_select_quota(self.shape, self.score, self.off, self.quota, self.keep,
                             self.sel_off, self.sel_pos, self.ws, self.ws_bytes, stream)

    def compact(self, alpha, x, g, ab, phi, stream=None, gathered: bool = False):
        """Gather the retained rows; ab=None copies no [a | b] (recompute);
        gathered=True writes only the gradient rows (the products then read
        x, ab and phi in place). With a PackedState as ab, [a | b] and phi are
        rebuilt from it, gathered is about x alone, and x may be 8-bit rows with
        their scales (see ``step``)."""
        if isinstance(ab, PackedState):
            self._compact_packed(alpha, x, g, ab, stream, gathered)
            return
        x_c = None if gathered else self.x_c
        ab_c = None if (gathered or ab is None) else self.ab_c
        phi_c = None if gathered else self.phi_c
        lrm.lrm_compact(self.shape, self.perm, self.keep, self.sel_off, self.sel_pos, alpha, x,
                        g, ab, phi, self.dy_c, x_c, ab_c, phi_c, self.tok_c, self.row_of_pos,
                        self.ws, self.ws_bytes, stream)

    def _packed_rows(self, alpha, x, g, packed, gathered):
        """Checks what a packed state is compacted with: x, its scales or None, and the
        columns under one of them."""
        self._check_packed(packed, filled=True)
        dev, x_scale, cols = self.ws.device, None, 0
        if isinstance(x, (tuple, list)):
            if gathered:
                raise ValueError("8-bit x is not read in place: gathered=False")
            x, x_scale = x
            _need(x, "x", (self.T, self.D), torch.float8_e4m3fn, dev)
            cols = _x_groups(self.D, x_scale.shape[-1])
            _need(x_scale, "x's scales", (self.T, x_scale.shape[-1]), torch.float32, dev)
        else:
            _need(x, "x", (self.T, self.D), self.tdtype, dev)
        _need(g, "g", (self.T, self.D), self.tdtype, dev)
        _need(alpha, "alpha", (self.T, self.K), torch.float32, dev)
        return x, x_scale, cols

    def _compact_packed(self, alpha, x, g, packed, stream, gathered):
        x, x_scale, cols = self._packed_rows(alpha, x, g, packed, gathered)
        lrm.lrm_compact_packed(self.shape, packed.desc, self.perm, self.keep, self.sel_off,
                               self.sel_pos, alpha, x, x_scale, cols, g, self.dy_c,
                               None if gathered else self.x_c, self.ab_c, self.phi_c, self.tok_c,
                               self.row_of_pos, self.ws, self.ws_bytes,
                               _stream(self.ws.device, stream))

    def expert_bwd_compacted(self, x, w_gate, w_up, w_down, stream=None):
        """The expert backward over compacted [a | b] and phi, reading x rows in place
        (after a gathered compaction of a PackedState)."""
        lrm.lrm_expert_bwd_compacted(
            self.shape, self.sel_off, self.tok_c, w_gate, w_up, w_down, self.dy_c, x, self.ab_c,
            self.phi_c, self.inv, self.row_of_pos, self.dab_c, self.dx_c, self.dw_gate,
            self.dw_up, self.dw_down, self.dx, self.ws, self.ws_bytes, stream)

    def fc1_recompute(self, w_gate, w_up, stream=None):
        """[a | b] of the retained rows rebuilt from x_c (no saved [a | b])."""
        lrm.lrm_expert_fc1_recompute(self.shape, self.sel_off, self.x_c, w_gate, w_up,
                                     self.ab_c, self.ws, self.ws_bytes, stream)

    def score_select_compact(self, alpha, x, g, ab, phi, stream=None, metric: int = 0,
                             seed: int = 0, gathered: bool = False):
        self.score_pairs(alpha, g, phi, stream, metric, seed)
        self.select(stream)
        self.compact(alpha, x, g, ab, phi, stream, gathered)

    def expert_bwd_gathered(self, x, ab, phi, w_gate, w_up, w_down, parts: int | None = None,
                            stream=None):
        """The expert backward reading x, ab and phi rows in place (after a
        gathered compaction); `parts` selects sub-steps (lrm.LRM_BWD_*)."""
        lrm.lrm_expert_bwd_gathered(
            self.shape, lrm.LRM_BWD_ALL if parts is None else parts, self.sel_off, self.sel_pos,
            self.tok_c, w_gate, w_up, w_down, self.dy_c, x, ab, phi, self.inv, self.row_of_pos,
            self.dab_c, self.dx_c, self.dw_gate, self.dw_up, self.dw_down, self.dx, self.ws,
            self.ws_bytes, stream)

    def expert_bwd(self, w_gate, w_up, w_down, stream=None):
        lrm.lrm_expert_bwd_grouped(
            self.shape, self.sel_off, w_gate, w_up, w_down, self.dy_c, self.x_c, self.ab_c,
            self.phi_c, self.inv, self.row_of_pos, self.dab_c, self.dx_c, self.dw_gate,
            self.dw_up, self.dw_down, self.dx, self.ws, self.ws_bytes, stream)

    # the same backward as five separate calls (one kernel each), so that a
    # caller can time or overlap the sub-steps
    def fc2_dgrad(self, w_down, stream=None):
        lrm.lrm_expert_fc2_dgrad(self.shape, self.sel_off, w_down, self.dy_c, self.ab_c,
                                 self.dab_c, self.ws, self.ws_bytes, stream)

    def fc2_wgrad(self, stream=None):
        lrm.lrm_expert_fc2_wgrad(self.shape, self.sel_off, self.phi_c, self.dy_c, self.dw_down,
                                 self.ws, self.ws_bytes, stream)

    def fc1_wgrad(self, stream=None):
        lrm.lrm_expert_fc1_wgrad(self.shape, self.sel_off, self.x_c, self.dab_c, self.dw_gate,
                                 self.dw_up, self.ws, self.ws_bytes, stream)

    def fc1_dgrad(self, w_gate, w_up, stream=None):
        lrm.lrm_expert_fc1_dgrad(self.shape, self.sel_off, w_gate, w_up, self.dab_c, self.dx_c,
                                 self.ws, self.ws_bytes, stream)

    def scatter_dx(self, stream=None):
        lrm.lrm_scatter_dx(self.shape, self.dx_c, self.inv, self.row_of_pos, self.dx, self.ws,
                           self.ws_bytes, stream)

    def step(self, topk_idx, alpha, x, g, ab, phi, w_gate, w_up, w_down, rate=(1, 1),
             cap: int = 0, quota: torch.Tensor | None = None, stream=None, metric: int = 0,
             seed: int = 0, gathered: bool = False):
        """One pass of the whole path. ab / phi are in dispatch order; `metric`
        picks the selection criterion (LRM by default). ab=None recomputes
        [a | b] of the retained rows instead of reading saved state;
        gathered=True lets the products read x, ab and phi rows in place.
        ab a PackedState (phi is then not needed): [a | b] and phi of the
        retained rows come from its 8 bits; x may then be (q, q_scale), 8-bit
        rows as AddRMSNorm and BlockNorm write them; gathered lets the product
        read a 16- or 32-bit x in place."""
        if gathered and ab is None:
            raise ValueError("the gathered backward reads saved [a | b]")
        packed = isinstance(ab, PackedState)
        if packed:
            self._packed_rows(alpha, x, g, ab, gathered)  # all of it, before anything runs
            phi = ab
        elif isinstance(x, (tuple, list)):
            raise ValueError("8-bit x goes with a PackedState")
        self.dispatch(topk_idx, stream)
        self.score_pairs(alpha, g, phi, stream, metric, seed)
        if quota is None:
            self.select_rate(rate[0], rate[1], cap, stream)
        else:
            self.quota.copy_(quota)
            self.select(stream)
        self.compact(alpha, x, g, ab, phi, stream, gathered)
        if packed and gathered:
            self.expert_bwd_compacted(x, w_gate, w_up, w_down, stream)
            return
        if gathered:
            self.expert_bwd_gathered(x, ab, phi, w_gate, w_up, w_down, stream=stream)
            return
        if ab is None:
            self.fc1_recompute(w_gate, w_up, stream)
        self.expert_bwd(w_gate, w_up, w_down, stream)

    def device_error(self, stream=None) -> int:
        return lrm.lrm_get_device_error(self.ws, self.ws_bytes, stream)

    def clear_device_error(self, stream=None):
        lrm.lrm_clear_device_error(self.ws, self.ws_bytes, stream)

    @property
    def retained_rows(self) -> int:
        return int(self.sel_off[self.E].item())
