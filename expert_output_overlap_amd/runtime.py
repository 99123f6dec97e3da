"""Device buffers and calls of one MoE expert-compute-plus-return problem (torch allocates, the library computes).

``MoePath`` owns every buffer the C-ABI needs for one shape and calls the entry points in order:
route -> layout -> expert FFN with return -> combine.  Nothing here computes anything itself.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import binding as B

NAME_SIZES = ("counts", "padded_off", "recv_off", "tile_owner", "tile_expert", "tile_valid", "tile_order", "seg_desc",
              "row_src", "combine_plan", "scalars", "status", "mtile_desc", "seg_mtiles")


class MoePath:
    def __init__(self, R, T_o, G, E_l, k, d, f, M, mgb=1, dtype="bf16", self_rank=0, device="cuda"):
        self.R, self.T_o, self.G, self.E_l, self.k, self.d, self.f, self.M = R, T_o, G, E_l, k, d, f, M
        self.T = R * T_o
        self.dtype = dtype
        self.device = torch.device(device)
        self.shape = B.moe_shape(R, T_o, G, E_l, k, self_rank, d, f, M, mgb, B.MOE_BF16 if dtype == "bf16" else B.MOE_F32)
        nbytes = B.moe_layout_workspace_bytes(self.shape)
        if nbytes < 0:
            raise B.MoeError("moe_layout_workspace_bytes", -1, "invalid shape")
        self.ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=self.device)
        base = (self.ws.data_ptr() + 255) // 256 * 256
        self.ws_aligned = self.ws[base - self.ws.data_ptr():]
        self.L = B.moe_layout()
        B.moe_layout_bind(self.shape, self.ws_aligned, self.L)
        cap = self.L.cap_rows
        self.tdtype = torch.bfloat16 if dtype == "bf16" else torch.float32
        z = dict(device=self.device)
        self.x_pad = torch.empty(cap, d, dtype=self.tdtype, **z)
        self.h = torch.empty(cap, f, dtype=self.tdtype, **z)
        self.y_pad = torch.empty(cap, d, dtype=self.tdtype, **z)
        self.recv_cap = T_o * min(k, E_l)
        self.recv = [torch.empty(max(self.recv_cap, 1), d, dtype=self.tdtype, **z) for _ in range(R)]
        self.flags = torch.zeros(B.moe_ffn_flags_count(self.shape), dtype=torch.int32, **z)
        self.topk_idx = torch.empty(max(self.T, 1), k, dtype=torch.int32, **z)
        self.topk_w = torch.empty(max(self.T, 1), k, dtype=torch.float32, **z)
        self.out = torch.empty(max(self.T, 1), d, dtype=self.tdtype, **z)
        self.timestamps = torch.zeros(2 + 2 * self.L.cap_tiles, dtype=torch.int64, **z)
        self.epoch = 0

    @classmethod
    def from_spec(cls, s, device="cuda"):
        return cls(s.R, s.T_o, s.G, s.E_l, s.k, s.d, s.f, s.M, s.mgb, s.dtype, 0, device)

    # ---- views of the layout arrays (int32 tensors in the workspace) ----------------------------------------
    def array(self, name: str) -> torch.Tensor:
        L = self.L
        sizes = {
            "counts": self.E_l * self.R, "padded_off": self.E_l * self.R, "recv_off": self.E_l * self.R,
            "tile_owner": L.cap_tiles, "tile_expert": L.cap_tiles, "tile_valid": L.cap_tiles,
            "tile_order": L.cap_tiles, "seg_desc": L.cap_tiles * B.MOE_SEG_FIELDS, "row_src": L.cap_rows,
            "combine_plan": self.T * self.k, "scalars": 5 + self.R, "status": 1,
            "mtile_desc": L.cap_mtiles * B.MT_FIELDS, "seg_mtiles": L.cap_tiles * 2, "seg_sched": L.cap_tiles,
            "mt_order": L.cap_mtiles,
        }
        off = (getattr(L, name) - self.ws_aligned.data_ptr()) // 4
        return self.ws_aligned.view(torch.int32)[off: off + sizes[name]]

    # ---- calls ---------------------------------------------------------------------------------------------------
    def route(self, logits: torch.Tensor, stream=None):
        B.moe_route(self.shape, logits, self.topk_idx, self.topk_w, stream)

    def layout(self, x: torch.Tensor | None, topk_idx: torch.Tensor | None = None, stream=None):
        """x None: no gather into x_pad (the FFN call lands the rows, ``ffn(x_tokens=...)``)."""
        B.moe_layout_build(self.shape, self.topk_idx if topk_idx is None else topk_idx, x, self.L, self.x_pad, stream)

    def ffn(self, w_gate_up, w_down, mode=0, consumer_cus=0, band_window=0, timestamps=False, watchdog_ticks=0,
            epoch=None, tile_order=0, x_tokens: torch.Tensor | None = None, gu_out: torch.Tensor | None = None,
            stream=None):
        """gu_out: None, or [cap_rows, 2f] fp32 (gu_buffer()) for the first GEMM's pre-activations g | u, which a
        backward call can take instead of recomputing them."""
        if epoch is None:
            self.epoch += 1
            epoch = self.epoch
        cfg = B.moe_overlap_cfg(consumer_cus, mode, epoch, band_window, watchdog_ticks,
                                self.timestamps.data_ptr() if timestamps else None, tile_order,
                                None if x_tokens is None else x_tokens.data_ptr(),
                                None if gu_out is None else gu_out.data_ptr())
        B.moe_expert_ffn_overlap(self.shape, self.L, self.x_pad, w_gate_up, w_down, self.h, self.y_pad, self.recv,
                                 self.flags, cfg, stream)
        return epoch

    # ---- backward ---------------------------------------------------------------------------------------------
    def bwd_buffers(self):
        """The backward call's workspaces and outputs, allocated on first use (bf16 only)."""
        if getattr(self, "_bwd", None) is None:
            cap, d, f, z = self.L.cap_rows, self.d, self.f, dict(device=self.device)
            n = B.moe_bwd_flags_count(self.shape)
            if n < 0:
                raise B.MoeError("moe_bwd_flags_count", -1, "shape has no backward pass")
            self._bwd = {
                "dy_pad": torch.empty(cap, d, dtype=torch.bfloat16, **z),
                "dh_ws": torch.empty(cap, f, dtype=torch.float32, **z),
                "dgu_ws": torch.empty(cap, 2 * f, dtype=torch.bfloat16, **z),
                "dx_pad": torch.empty(cap, d, dtype=torch.bfloat16, **z),
                "dx_recv": [torch.empty(max(self.recv_cap, 1), d, dtype=torch.bfloat16, **z) for _ in range(self.R)],
                "dw_gate_up": torch.empty(self.E_l, 2 * f, d, dtype=torch.float32, **z),
                "dw_down": torch.empty(self.E_l, d, f, dtype=torch.float32, **z),
                "flags": torch.zeros(n, dtype=torch.int32, **z),
                "dx": torch.empty(max(self.T, 1), d, dtype=torch.bfloat16, **z),
                "dw_route": torch.empty(max(self.T, 1), self.k, dtype=torch.float32, **z),
            }
            self.bwd_epoch = 0
        return self._bwd

    def gu_buffer(self):
        """[cap_rows, 2f] fp32 for the forward's g | u (ffn(gu_out=...), backward(gu=...)), allocated on first use."""
        if getattr(self, "_gu", None) is None:
            self._gu = torch.empty(self.L.cap_rows, 2 * self.f, dtype=torch.float32, device=self.device)
        return self._gu

    def backward(self, d_out: torch.Tensor, w_gate_up, w_down, mode=0, consumer_cus=0, watchdog_ticks=0, epoch=None,
                 gu: torch.Tensor | None = None, stream=None):
        """The expert FFN's backward with the dX return (moe_expert_ffn_backward), for the routing, layout and x_pad
        of the last forward; the forward's h workspace receives the recomputed h.  gu: None, or the g | u that forward
        stored (ffn(gu_out=...)), which the h / dG / dU items then read instead of recomputing the first GEMM."""
        b = self.bwd_buffers()
        if epoch is None:
            self.bwd_epoch += 1
            epoch = self.bwd_epoch
        cfg = B.moe_overlap_cfg(consumer_cus, mode, epoch, 0, watchdog_ticks, None, 0, None)
        t = {"topk_idx": self.topk_idx, "topk_w": self.topk_w, "x_pad": self.x_pad, "w_gate_up": w_gate_up,
             "w_down": w_down, "d_out": d_out, "h_ws": self.h, "gu": gu,
             **{k: b[k] for k in ("dy_pad", "dh_ws", "dgu_ws", "dx_pad", "dw_gate_up", "dw_down")}}
        B.moe_expert_ffn_backward(self.shape, self.L, t, b["dx_recv"], b["flags"], cfg, stream)
        return epoch

    def combine_backward(self, d_out: torch.Tensor, stream=None):
        """dx and the routing weights' gradient (moe_combine_backward) from the delivered dX rows and the forward's
        delivered y rows."""
        b = self.bwd_buffers()
        B.moe_combine_backward(self.shape, self.L, d_out, self.recv, b["dx_recv"], b["dx"], b["dw_route"], stream)

    def combine(self, topk_w: torch.Tensor | None = None, stream=None):
        B.moe_combine(self.shape, self.L, self.topk_w if topk_w is None else topk_w, self.recv, self.out, stream)

    def partition_record(self):
        """The launch's consumer-partition record (bf16): (consumer CUs of the last overlapped call, observed producer
        flops per CU-tick, observed consumer bytes per CU-tick, whether both rates hold observations)."""
        import struct

        w = self.flags[-B.MOE_OBS_WORDS:].cpu().numpy().astype("<i4").view("<u4")
        f = lambda v: struct.unpack("<f", struct.pack("<I", int(v)))[0]
        return int(w[12]), f(w[10]), f(w[11]), int(w[13]) == 3

    def status(self, stream=None) -> int:
        return B.moe_read_status(self.L, stream)

    def scalars(self):
        sc = self.array("scalars").cpu().tolist()
        return {"M_pad": sc[0], "n_tiles": sc[1], "n_segs": sc[2], "N_r": sc[3:3 + self.R], "n_mtiles": sc[3 + self.R],
                "n_remote_mtiles": sc[4 + self.R]}


# ---- the operators around the routed experts ---------------------------------------------------------------------

TORCH_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
MOE_DTYPES = {"bf16": B.MOE_BF16, "f32": B.MOE_F32, torch.bfloat16: B.MOE_BF16, torch.float32: B.MOE_F32}


def _need(t: torch.Tensor, name: str, shape: tuple, dtype, device, strided=False):
    """A tensor that a kernel reads or writes through its address alone: anything else than what it takes is an error."""
    if t.dtype is not dtype or t.device != device or t.shape != shape:
        raise ValueError("%s: %s %s on %s, wanted %s %s on %s" % (name, t.dtype, tuple(t.shape), t.device, dtype, tuple(shape),
                                                                  device))
    if strided:
        if t.stride(1) != 1 and t.shape[1] > 1 or t.stride(0) < t.shape[1] and t.shape[0] > 1:
            raise ValueError("%s: rows must hold their elements side by side and not overlap" % name)
    elif not t.is_contiguous():
        raise ValueError("%s: not contiguous" % name)


def _first(t: torch.Tensor, n: int) -> torch.Tensor:
    """The first n rows (a view costs a microsecond, so none of all of them)."""
    return t if n == t.shape[0] else t[:n]


def _device(device) -> torch.device:
    device = torch.device(device)
    return torch.device(device.type, torch.cuda.current_device()) if device.type == "cuda" and device.index is None else device


def _on_own_device(f):
    """The method with its object's device as the current one (a launch goes to a stream of that device)."""

    @functools.wraps(f)
    def g(self, *args, **kw):
        if torch._C._cuda_getDevice() == self.device.index:
            return f(self, *args, **kw)
        with torch.cuda.device(self.device):
            return f(self, *args, **kw)

    return g


def _workspace(nbytes: int, fn: str, device):
    if nbytes < 0:
        raise B.MoeError(fn, B.MOE_EINVAL, "invalid shape")
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


class LayerNorm:
    """Layer norm over up to ``rows`` rows of ``d`` elements (moe_layer_norm, moe_layer_norm_backward), with the buffers of
    its results: y, and for training dx, dweight, dbias and what the backward call needs.  Rows may lie apart (a slice of
    a wider tensor).  A call's results stay until the next call of the same kind."""

    def __init__(self, rows, d, dtype="bf16", param_dtype="f32", eps=1e-5, train=True, device="cuda"):
        self.device = _device(device)
        self.rows, self.d, self.train = rows, d, train
        self.dtype, self.param_dtype = TORCH_DTYPES[dtype], TORCH_DTYPES[param_dtype]
        self.shape = B.moe_norm_shape(rows, d, MOE_DTYPES[dtype], MOE_DTYPES[param_dtype], eps, 0, 0, 0)
        z = dict(device=self.device)
        ws = _workspace(B.moe_layer_norm_workspace_bytes(self.shape), "moe_layer_norm_workspace_bytes", self.device)
        self.y = torch.empty(rows, d, dtype=self.dtype, **z)
        self.mean = self.rstd = None
        if train:
            self.workspace = ws
            self.mean, self.rstd = (torch.empty(rows, dtype=torch.float32, **z) for _ in range(2))
            self.dx = torch.empty(rows, d, dtype=self.dtype, **z)
            self.dweight, self.dbias = (torch.empty(d, dtype=self.param_dtype, **z) for _ in range(2))

    def _rows(self, x):
        if x.shape[0] > self.rows:
            raise ValueError("%d rows, made for up to %d" % (x.shape[0], self.rows))
        return x.shape[0]

    def _stride(self, t):
        return t.stride(0) if t.shape[0] > 1 else 0

    def _param(self, t, name):
        if t is not None:
            _need(t, name, (self.d,), self.param_dtype, self.device)

    @_on_own_device
    def forward(self, x, weight=None, bias=None, y=None, stream=None):
        n = self._rows(x)
        y = _first(self.y, n) if y is None else y
        _need(x, "x", (n, self.d), self.dtype, self.device, strided=True)
        _need(y, "y", (n, self.d), self.dtype, self.device, strided=True)
        self._param(weight, "weight")
        self._param(bias, "bias")
        s = self.shape
        s.rows, s.x_stride, s.y_stride = n, self._stride(x), self._stride(y)
        B.moe_layer_norm(s, x, weight, bias, y, self.mean, self.rstd, stream)
        return y

    @_on_own_device
    def backward(self, dy, x, weight=None, residual=None, dx=None, stream=None):
        """dx (added to ``residual`` where given), and dweight and dbias in their buffers, for the rows x of the last
        forward call."""
        if not self.train:
            raise RuntimeError("made without train=True")
        n = self._rows(x)
        dx = _first(self.dx, n) if dx is None else dx
        for name, t in (("x", x), ("dy", dy), ("dx", dx)):
            _need(t, name, (n, self.d), self.dtype, self.device, strided=True)
        if residual is not None:
            _need(residual, "residual", (n, self.d), self.dtype, self.device, strided=True)
            if self._stride(residual) != self._stride(dx):
                raise ValueError("residual and dx: their rows must lie equally far apart")
        self._param(weight, "weight")
        s = self.shape
        s.rows, s.x_stride, s.y_stride, s.dx_stride = n, self._stride(x), self._stride(dy), self._stride(dx)
        B.moe_layer_norm_backward(s, dy, x, weight, self.mean, self.rstd, residual, dx, self.dweight, self.dbias,
                                  self.workspace, stream)
        return dx


class SharedFFN:
    """The shared expert's gated feed-forward block over up to ``tokens`` tokens (moe_shared_ffn, moe_shared_ffn_backward),
    with the buffers of its results and workspaces.  A call's results stay until the next call of the same kind."""

    def __init__(self, tokens, d, f, dtype="bf16", train=True, device="cuda"):
        self.device = _device(device)
        self.tokens, self.d, self.f, self.train = tokens, d, f, train
        self.dtype = TORCH_DTYPES[dtype]
        self.shape = B.moe_shared_shape(tokens, d, f, MOE_DTYPES[dtype])
        row = B.moe_shared_ffn_row(self.shape)
        if row < 0:
            raise B.MoeError("moe_shared_ffn_row", B.MOE_EINVAL, "invalid shape")
        need = max(B.moe_shared_ffn_workspace_bytes(self.shape, b) for b in ((False, True) if train else (False,)))
        self.workspace = _workspace(need, "moe_shared_ffn_workspace_bytes", self.device)
        z = dict(dtype=self.dtype, device=self.device)
        self.y, self.h = torch.empty(tokens, d, **z), torch.empty(tokens, row, **z)
        self.gu = None
        if train:
            self.gu = torch.empty(tokens, 2 * row, dtype=torch.float32, device=self.device)
            self.dgu = torch.empty(tokens, 2 * row, **z)
            self.dx = torch.empty(tokens, d, **z)
            self.dw_gate_up, self.dw_down = torch.empty(2 * f, d, **z), torch.empty(d, f, **z)

    def _check(self, x, w_gate_up, w_down, **rows):
        n = x.shape[0]
        if n > self.tokens:
            raise ValueError("%d tokens, made for up to %d" % (n, self.tokens))
        for name, t in (("x", x), *rows.items()):
            if t is not None:
                _need(t, name, (n, self.d), self.dtype, self.device)
        _need(w_gate_up, "w_gate_up", (2 * self.f, self.d), self.dtype, self.device)
        _need(w_down, "w_down", (self.d, self.f), self.dtype, self.device)
        self.shape.tokens = n
        return n

    @_on_own_device
    def forward(self, x, w_gate_up, w_down, residual=None, y=None, stream=None):
        y = _first(self.y, x.shape[0]) if y is None else y
        self._check(x, w_gate_up, w_down, residual=residual, y=y)
        B.moe_shared_ffn(self.shape, x, w_gate_up, w_down, residual, self.h, self.gu, y, self.workspace, stream)
        return y

    @_on_own_device
    def backward(self, dy, x, w_gate_up, w_down, residual=None, dx=None, stream=None):
        """dx (added to ``residual`` where given), and dw_gate_up and dw_down in their buffers, for the x and the weights of
        the last forward call."""
        if not self.train:
            raise RuntimeError("made without train=True")
        dx = _first(self.dx, x.shape[0]) if dx is None else dx
        self._check(x, w_gate_up, w_down, dy=dy, residual=residual, dx=dx)
        t = {"x": x, "w_gate_up": w_gate_up, "w_down": w_down, "h": self.h, "gu": self.gu, "dy": dy, "residual": residual,
             "dgu_ws": self.dgu, "dx": dx, "dw_gate_up": self.dw_gate_up, "dw_down": self.dw_down}
        B.moe_shared_ffn_backward(self.shape, t, self.workspace, stream)
        return dx


class AdamW:
    """AdamW over many tensors in one launch (moe_adamw_*).  tensors: dicts of device tensors with equal numbers of elements,
    "p" (bf16 or fp32), "g", "m" and "v" (fp32, or uint8 codes with "m_scale" and "v_scale", see ``states``), optionally
    "copy" (bf16, the new p), "m_values" and "root_values" (bf16, what ``read_states`` fills), and numbers "weight_decay" and
    "lr_scale".  The tensors' addresses are bound: their contents may change between steps, not they themselves."""

    FIELDS = dict(param="p", copy="copy", grad="g", m="m", v="v", m_scale="m_scale", v_scale="v_scale", m_values="m_values",
                  root_values="root_values")

    def __init__(self, tensors, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.0, stream=None):
        self.tensors = [dict(t) for t in tensors]
        self.device = self.tensors[0]["p"].device if self.tensors else _device("cuda")
        self.betas, self.eps = betas, eps
        table = (B.moe_adamw_tensor * len(self.tensors))()
        for i, (q, t) in enumerate(zip(table, self.tensors)):
            n, bits = t["p"].numel(), 8 if t["m"].dtype is torch.uint8 else 32
            state = torch.uint8 if bits == 8 else torch.float32
            blocks = -(-n // B.MOE_ADAMW_BLOCK)
            wanted = dict(copy=(torch.bfloat16, n), m=(state, n), v=(state, n), m_scale=(torch.uint8, blocks),
                          v_scale=(torch.uint8, blocks), m_values=(torch.bfloat16, n), root_values=(torch.bfloat16, n))
            for field, key in self.FIELDS.items():
                x = t.get(key)
                if x is None:
                    continue
                dtype, k = wanted.get(key, (x.dtype, n))
                if x.dtype is not dtype or x.numel() != k or not x.is_contiguous() or x.device != self.device:
                    raise ValueError("tensor %d, %s: %d %s on %s, wanted %d contiguous %s on %s" % (
                        i, key, x.numel(), x.dtype, x.device, k, dtype, self.device))
                setattr(q, field, x.data_ptr())
            if t["p"].dtype not in MOE_DTYPES or t["g"].dtype not in MOE_DTYPES:
                raise ValueError("tensor %d: p and g must be bf16 or fp32" % i)
            q.n, q.param_dtype, q.grad_dtype, q.state_bits = n, MOE_DTYPES[t["p"].dtype], MOE_DTYPES[t["g"].dtype], bits
            q.weight_decay, q.lr_scale = t.get("weight_decay", weight_decay), t.get("lr_scale", 1.0)
        self.workspace = _workspace(B.moe_adamw_workspace_bytes(table), "moe_adamw_workspace_bytes", self.device)
        self.plan = B.moe_adamw_plan()
        with torch.cuda.device(self.device):
            B.moe_adamw_bind(table, self.workspace, self.plan, stream)

    @staticmethod
    def states(p: torch.Tensor, bits: int = 32) -> dict:
        """The states of a tensor before its first step: zeros."""
        if bits not in (8, 32):
            raise ValueError("states in 8 or 32 bits, not %r" % (bits,))
        n, z = p.numel(), dict(device=p.device)
        if bits == 32:
            return {k: torch.zeros(n, dtype=torch.float32, **z) for k in ("m", "v")}
        blocks = -(-n // B.MOE_ADAMW_BLOCK)
        return {k: torch.zeros(k.endswith("scale") and blocks or n, dtype=torch.uint8, **z)
                for k in ("m", "v", "m_scale", "v_scale")}

    @_on_own_device
    def step(self, step, lr, grad_scale=None, stream=None):
        """step: 1, 2, ..., or an int64 tensor on the device; lr: a number, or an fp32 tensor on the device (both: what a
        captured step reads anew at each replay); grad_scale: None, or an fp32 tensor on the device."""
        cfg = B.moe_adamw_cfg(0.0, *self.betas, self.eps, 1, None, None, None)
        for field, value, dtype in (("step", step, torch.int64), ("lr", lr, torch.float32),
                                    ("grad_scale", grad_scale, torch.float32)):
            if isinstance(value, torch.Tensor):
                if value.dtype is not dtype or value.numel() != 1 or value.device != self.device:
                    raise ValueError("%s: one %s on %s wanted" % (field, dtype, self.device))
                setattr(cfg, "grad_scale" if field == "grad_scale" else field + "_dev", value.data_ptr())
            elif field != "grad_scale":
                setattr(cfg, field, value)
            elif value is not None:  # its field is an address: a number there would be read through
                raise ValueError("grad_scale: one %s on %s wanted, not %r" % (dtype, self.device, value))
        B.moe_adamw_step(self.plan, cfg, stream)

    @_on_own_device
    def read_states(self, stream=None):
        """The 8-bit states' values into the tensors' "m_values" and "root_values", where given."""
        B.moe_adamw_read_states(self.plan, stream)


class MoeBlock:
    """A pre-norm MoE block of one rank: n = norm(x); out = combine(routed experts(n)) + shared expert(n), and its backward.
    The router's product is the caller's: ``norm`` gives the rows its logits come from, ``experts`` takes the logits;
    ``experts_backward`` gives the gradient of n (and path.bwd_buffers()["dw_route"] that of the routing weights), to which
    the caller adds the router's part before ``norm_backward``.  Every call takes all of the path's T rows; logits are fp32
    [T, G].  w: norm_weight, norm_bias, w_gate_up, w_down (the routed experts' [E_l, ...]), shared_gate_up, shared_down."""

    def __init__(self, path: MoePath, shared_f: int, eps=1e-5, train=True):
        self.path, self.train = path, train
        self.norm_op = LayerNorm(path.T, path.d, path.dtype, "f32", eps, train, path.device)
        self.shared = SharedFFN(path.T, path.d, shared_f, path.dtype, train, path.device)
        self.device = self.norm_op.device

    def _experts_weights(self, w):
        """The routed path takes addresses: what it reads has to be there."""
        p = self.path
        _need(w["w_gate_up"], "w_gate_up", (p.E_l, 2 * p.f, p.d), p.tdtype, self.device)
        _need(w["w_down"], "w_down", (p.E_l, p.d, p.f), p.tdtype, self.device)

    @_on_own_device
    def norm(self, x, w, stream=None):
        _need(x, "x", (self.path.T, self.path.d), self.path.tdtype, self.device, strided=True)
        self.n = self.norm_op.forward(x, w["norm_weight"], w["norm_bias"], stream=stream)
        return self.n

    @_on_own_device
    def experts(self, logits, w, stream=None):
        p, out = self.path, self.path.out[: self.path.T]
        _need(logits, "logits", (p.T, p.G), torch.float32, self.device)
        self._experts_weights(w)
        p.route(logits, stream)
        p.layout(self.n, stream=stream)
        p.ffn(w["w_gate_up"], w["w_down"], gu_out=p.gu_buffer() if self.train else None, stream=stream)
        p.combine(stream=stream)
        return self.shared.forward(self.n, w["shared_gate_up"], w["shared_down"], residual=out, y=out, stream=stream)

    @_on_own_device
    def experts_backward(self, d_out, w, stream=None):
        if not self.train:
            raise RuntimeError("made without train=True")
        p = self.path
        _need(d_out, "d_out", (p.T, p.d), p.tdtype, self.device)
        self._experts_weights(w)
        p.backward(d_out, w["w_gate_up"], w["w_down"], gu=p.gu_buffer(), stream=stream)
        p.combine_backward(d_out, stream=stream)
        dn = p.bwd_buffers()["dx"][: p.T]
        return self.shared.backward(d_out, self.n, w["shared_gate_up"], w["shared_down"], residual=dn, dx=dn, stream=stream)

    @_on_own_device
    def norm_backward(self, dn, x, w, residual=None, stream=None):
        """dx; residual: the gradient that reaches x past the block."""
        return self.norm_op.backward(dn, x, w["norm_weight"], residual=residual, stream=stream)


def to_device(a, dtype: str, device="cuda") -> torch.Tensor:
    """Host array from moe_inputs (bf16 bits as uint16, or fp32/int32) to a device tensor of the right type."""
    import numpy as np

    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).to(device)
    return torch.from_numpy(a).to(device)
