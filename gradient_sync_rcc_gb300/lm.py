"""Binding of the language-model operators of librcc (include/rcc.h): token
embedding and its gradient, the RMS norm that keeps its input in 8 bits, alone
and with the residual's addition, rotary positions, the output layer with
softmax cross entropy, and AdamW over many tensors.  Reached as attributes of
`rcc`, like the rest of the binding.

The work of a call -- checks of what the C entry points cannot see (a type, a
device, a shape that does not fit: ValueError), outputs and workspaces that
the caller left out, the C call itself -- is done by the compiled module _lm.
New tensors are allocated on the inputs' device for `stream` (the current one
by default), as under torch.cuda.stream; tensors passed in must be safe to use
there.  The inputs' device must be the current one.
"""
import ctypes as C

import torch

from gradient_sync_rcc_gb300 import rcc as _rcc
try:
    from gradient_sync_rcc_gb300 import _lm
except ImportError as e:
    raise ImportError("the language-model operators' binding _lm.so does not load (%s); build it "
                      "with gradient_sync_rcc_gb300.build.build()" % e) from e


def _fail(status):
    raise _rcc.RccError(status, _rcc.last_error())


_lib = _rcc.lib()
_lm.bind(_fail, *(C.cast(getattr(_lib, name), C.c_void_p).value for name in (
    "rcc_embedding_forward", "rcc_embedding_backward", "rcc_embedding_backward_workspace",
    "rcc_rmsnorm_forward", "rcc_rmsnorm_backward", "rcc_rmsnorm_backward_workspace",
    "rcc_linear_ce_forward", "rcc_linear_ce_backward", "rcc_linear_ce_workspace",
    "rcc_add_rmsnorm_forward", "rcc_add_rmsnorm_backward", "rcc_rotary_forward",
    "rcc_rotary_backward", "rcc_adamw_step")))


# ------------------------------------------------------------- embedding

def embedding_forward(table, ids, scale=1.0, out=None, out_dtype=None, stream=None):
    """rcc_embedding_forward: scale * table[ids], a row of zeros for an id
    outside the table.  Returns out [tokens, dim] of out_dtype (the table's)."""
    return _lm.embedding_forward(table, ids, scale, out, out_dtype, stream)


def embedding_backward_workspace(tokens, vocab, dim):
    return _lib.rcc_embedding_backward_workspace(tokens, vocab, dim)


def embedding_backward(dout, ids, dtable, scale=1.0, accumulate=False, workspace=None,
                       stream=None):
    """rcc_embedding_backward: the gradient of embedding_forward's table, into
    dtable [vocab, dim] (added to it with accumulate).  Returns dtable."""
    return _lm.embedding_backward(dout, ids, dtable, scale, accumulate, workspace, stream)


# ------------------------------------------------------------- RMS norm

KEEP_GROUP = 128   # columns that share one scale of the 8-bit form


class Kept:
    """A norm's input in 8 bits: values [tokens, 128 G] int8 and scales
    [tokens, G] float32 of its `dim` columns, G = ceil(dim / 128), one after
    the other in one buffer."""

    __slots__ = ("data", "tokens", "dim")

    def __init__(self, tokens, dim, device=None, data=None):
        self.tokens, self.dim = tokens, dim
        self.data = torch.empty(tokens * self.groups * (KEEP_GROUP + 4), dtype=torch.uint8,
                                device=device) if data is None else data

    @property
    def groups(self):
        return -(-self.dim // KEEP_GROUP)

    @property
    def values(self):
        n = self.groups * KEEP_GROUP
        return self.data[:self.tokens * n].view(torch.int8).view(self.tokens, n)

    @property
    def scales(self):
        at = self.tokens * self.groups * KEEP_GROUP
        n = self.tokens * self.groups * 4
        return self.data[at:at + n].view(torch.float32).view(self.tokens, self.groups)

    def dequantize(self):
        """What it stands for, [tokens, dim] float32."""
        t, g = self.tokens, self.groups
        v = self.values.view(t, g, KEEP_GROUP) * self.scales[:, :, None]
        return v.view(t, g * KEEP_GROUP)[:, :self.dim]


def rmsnorm_forward(x, weight, eps=1e-6, keep=False, out=None, stream=None):
    """rcc_rmsnorm_forward.  Returns y, or (y, kept) with keep: True, or a Kept
    of these sizes to be written."""
    if keep is True:
        y, data = _lm.rmsnorm_forward(x, weight, eps, True, 0, 0, out, stream)
        return y, Kept(x.shape[0], x.shape[1], data=data)
    if not keep:
        return _lm.rmsnorm_forward(x, weight, eps, None, 0, 0, out, stream)
    return _lm.rmsnorm_forward(x, weight, eps, keep.data, keep.tokens, keep.dim, out, stream), keep


def rmsnorm_backward_workspace(tokens, dim):
    return _lib.rcc_rmsnorm_backward_workspace(tokens, dim)


def rmsnorm_backward(dy, kept, weight, eps=1e-6, dx=None, dweight=None, accumulate=False,
                     workspace=None, stream=None):
    """rcc_rmsnorm_backward from a Kept.  Returns (dx, dweight); with accumulate
    dweight is passed and added to."""
    return _lm.rmsnorm_backward(dy, kept.data, kept.tokens, kept.dim, weight, eps, dx, dweight,
                                accumulate, workspace, stream)


# ------------------------------------------------------------- RMS norm with the residual's addition

class Scaled:
    """A matrix in 8 bits: values [tokens, dim] float8_e4m3fn and scales
    [tokens, ceil(dim / 128)] float32."""

    __slots__ = ("values", "scales")

    def __init__(self, values, scales):
        self.values, self.scales = values, scales

    def dequantize(self):
        """What it stands for, [tokens, dim] float32."""
        dim = self.values.shape[1]
        return self.values.float() * self.scales.repeat_interleave(KEEP_GROUP, 1)[:, :dim]


def add_rmsnorm_forward(x, residual, weight, eps=1e-6, out_dtype=None, keep=False, h=None,
                        out=None, stream=None):
    """rcc_add_rmsnorm_forward: h = x + residual and y = RMS norm of h.  Returns
    (y, h), or (y, h, kept) with keep: True, or a Kept of these sizes to be
    written.

    y is of x's type; with out_dtype=torch.float8_e4m3fn, or a Scaled as `out`,
    it is a Scaled.  h may be x or residual itself.  A residual of None (8-bit
    y) adds nothing and gives an h of None."""
    eight, values, scales = False, None, None
    if out_dtype is not None or out is not None:
        eight = isinstance(out, Scaled) if out_dtype is None else out_dtype == torch.float8_e4m3fn
        if out_dtype not in (None, x.dtype, torch.float8_e4m3fn) or \
                (out is not None and isinstance(out, Scaled) != eight):
            raise ValueError("out_dtype must be x's type or torch.float8_e4m3fn, and out fit it")
        values, scales = (out.values, out.scales) if isinstance(out, Scaled) else (out, None)
    if not keep:
        y, scales, h, _ = _lm.add_rmsnorm_forward(x, residual, weight, eps, eight, None, 0, 0, h,
                                                  values, scales, stream)
        return (out or Scaled(y, scales)) if eight else y, h
    buffer, tokens, dim = (True, 0, 0) if keep is True else (keep.data, keep.tokens, keep.dim)
    y, scales, h, data = _lm.add_rmsnorm_forward(x, residual, weight, eps, eight, buffer, tokens,
                                                 dim, h, values, scales, stream)
    return (out or Scaled(y, scales)) if eight else y, h, \
        Kept(x.shape[0], x.shape[1], data=data) if keep is True else keep


def add_rmsnorm_backward(dy, dh, kept, weight, eps=1e-6, dx=None, dweight=None, accumulate=False,
                         workspace=None, stream=None):
    """rcc_add_rmsnorm_backward from a Kept of h: the gradient of x, which is also
    residual's, for dy of y and dh of h (None: h has no other use).  Returns
    (dx, dweight); dx may be dh itself, and with accumulate dweight is passed
    and added to.  Workspace: rmsnorm_backward_workspace."""
    return _lm.add_rmsnorm_backward(dy, dh, kept.data, kept.tokens, kept.dim, weight, eps, dx,
                                    dweight, accumulate, workspace, stream)


# ------------------------------------------------------------- rotary positions

_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {"linear": 1, "base": 2, "parts": 3}


def rotary_turns(turned, base=10000.0, scaling=None, device="cuda"):
    """rcc_rotary_turns for the first `turned` elements of a head: int64
    [turned / 2] on `device`, once for a model.

    scaling: None, ("linear", factor), ("base", factor) or ("parts", factor,
    length trained on, low, high)."""
    if turned < 2 or turned % 2:
        raise ValueError("an even number of elements is turned, got %r" % (turned,))
    arg = None
    if scaling is not None:
        kind, *numbers = scaling
        if kind not in _SCALINGS or len(numbers) != (4 if kind == "parts" else 1):
            raise ValueError("scaling %r is not one of linear, base and parts with its numbers"
                             % (scaling,))
        arg = _rcc.RotaryScaling(_SCALINGS[kind], *numbers)
    turns = torch.empty(turned // 2, dtype=torch.int64)
    _rcc._check(_lib.rcc_rotary_turns(turned // 2, base, None if arg is None else C.byref(arg),
                                      turns.data_ptr()))
    return turns.to(device)


def _layout(name):
    if name not in _LAYOUTS:
        raise ValueError("layout must be one of %s" % ", ".join(_LAYOUTS))
    return _LAYOUTS[name]


def rotary_forward(q, k, turns, positions=None, offset=0, layout="half", scale=1.0, q_out=None,
                   k_out=None, stream=None):
    """rcc_rotary_forward: q and k [tokens, heads, head_dim] (k may be None),
    turned by their tokens' positions: positions + offset, or 0, 1, ... + offset.
    Returns (q, k) turned.  Any strides that keep the heads apart; a head's
    elements lie side by side.  q_out may be q itself."""
    return _lm.rotary(False, q, k, turns, positions, offset, _layout(layout), scale, q_out, k_out,
                      stream)


def rotary_backward(dq, dk, turns, positions=None, offset=0, layout="half", scale=1.0, q_out=None,
                    k_out=None, stream=None):
    """rcc_rotary_backward: the gradients of rotary_forward's q and k, for dq and
    dk of its results; the other arguments as there."""
    return _lm.rotary(True, dq, dk, turns, positions, offset, _layout(layout), scale, q_out, k_out,
                      stream)


# ------------------------------------------------------------- AdamW over many tensors

class AdamWPlan:
    """The tensors of rcc_adamw_step, with their states and the workspace.

    tensors: dicts with param (float32), grad (float32 or bfloat16), and if
    wanted copy (bfloat16, receives the new parameters), all contiguous and of
    one size.  States that are left out are made, as zeros of `states`
    (torch.float32 or torch.float8_e4m3fn): exp_avg, exp_avg_sq and, for 8 bits,
    exp_avg_scale and exp_avg_sq_scale [ceil(n / 128)].  `.tensors` has them all;
    saved with the report's step, and given again with that step, they resume.

    The tensors' addresses are kept: a step reads the gradients where they were.
    The plan and the states it makes belong to `stream`; steps on another one have
    to wait for it, and that one, if it is not torch's, has to live as long as the
    plan.  A plan may be dropped while its steps run, but graphs need it to live.
    One step after the other: a plan's steps, and graphs of them, share its
    workspace."""

    def __init__(self, tensors, states=torch.float32, seed=0, step=0, betas=(0.9, 0.999),
                 stream=None):
        self.handle = None
        if states not in (torch.float32, torch.float8_e4m3fn):
            raise ValueError("states must be torch.float32 or torch.float8_e4m3fn")
        tensors = [self._checked(i, t, states) for i, t in enumerate(tensors)]
        if not tensors:
            raise ValueError("no tensors")
        dev = tensors[0]["param"].device
        if any(v.device != dev for t in tensors for v in t.values()):
            raise ValueError("every buffer must be on one device")
        if dev.type != "cuda":
            raise ValueError("the operators take tensors on a CUDA device")
        _lm.check_device(dev.index, torch.cuda.current_device())
        self.device = dev.index
        given = {id(v) for t in tensors for v in t.values()}
        with _lm_stream(stream, dev):
            self.last = torch.cuda.current_stream().cuda_stream   # stream of the last step
            self.streams = {self.last}                            # that its memory is known to
            self.tensors = [self._with_states(t, states) for t in tensors]
            arr = (_rcc.AdamWTensor * len(self.tensors))(*map(self._entry, self.tensors))
            need = _lib.rcc_adamw_workspace(arr, len(arr))
            self.workspace = torch.empty(need, dtype=torch.uint8, device=dev)
            handle = C.c_void_p()
            _rcc._check(_lib.rcc_adamw_create(
                arr, len(arr), seed & 0xFFFFFFFF, step, betas[0], betas[1],
                self.workspace.data_ptr(), need, torch.cuda.current_stream().cuda_stream,
                C.byref(handle)))
        self.handle = handle.value
        self._own = [self.workspace] + [v for t in self.tensors for v in t.values()
                                        if id(v) not in given]
        # the last step's gradient norm: float64, on the device, written by each step
        self.grad_norm = self.workspace[8:16].view(torch.float64)[0]

    @staticmethod
    def _checked(i, given, states):
        t = {k: v for k, v in given.items() if v is not None}
        if "param" not in t or "grad" not in t:
            raise ValueError("tensor %d lacks a param or grad" % i)
        n = t["param"].numel()
        kind = t["exp_avg"].dtype if "exp_avg" in t else states
        f32, scales = (torch.float32,), -(-n // 128)
        want = {"param": (n, f32), "grad": (n, (torch.float32, torch.bfloat16)),
                "copy": (n, (torch.bfloat16,)),
                "exp_avg": (n, (torch.float32, torch.float8_e4m3fn)), "exp_avg_sq": (n, (kind,))}
        if kind == torch.float8_e4m3fn:
            want |= {"exp_avg_scale": (scales, f32), "exp_avg_sq_scale": (scales, f32)}
            # values without the scales that they were held with mean nothing
            if any((k in t) != (k + "_scale" in t) for k in ("exp_avg", "exp_avg_sq")):
                raise ValueError("tensor %d: 8-bit states come with their scales" % i)
        for k, v in t.items():
            if k not in want:
                raise ValueError("tensor %d: %r is not a buffer of AdamW, or not of its states"
                                 % (i, k))
            count, types = want[k]
            if v.numel() != count or v.dtype not in types or not v.is_contiguous():
                raise ValueError("tensor %d: %s must be %d contiguous elements of %s"
                                 % (i, k, count, " or ".join(map(str, types))))
        return t

    @staticmethod
    def _with_states(t, states):
        param = t["param"].detach()
        kind = t["exp_avg"].dtype if "exp_avg" in t else states
        for k in ("exp_avg", "exp_avg_sq"):
            if k in t:
                continue
            if kind == torch.float32:
                t[k] = torch.zeros_like(param)
            else:
                t[k] = torch.zeros_like(param, dtype=torch.uint8).view(kind)
                t[k + "_scale"] = torch.zeros(-(-param.numel() // 128), device=param.device)
        return t

    @staticmethod
    def _entry(t):
        p = {k: v.data_ptr() for k, v in t.items()}
        return _rcc.AdamWTensor(
            t["param"].numel(), p["grad"],
            _rcc.BF16 if t["grad"].dtype == torch.bfloat16 else _rcc.F32, p["param"],
            p["exp_avg"], p["exp_avg_sq"], p.get("exp_avg_scale"), p.get("exp_avg_sq_scale"),
            p.get("copy"))

    def _used_on(self, stream):
        """Memory that a step on another stream may still be using is not given out
        again before that step is through."""
        self.streams.add(stream)
        for v in self._own:
            v.record_stream(_stream_of(stream, self.workspace.device))

    def __del__(self):
        if self.handle is not None and _lib is not None:   # None: the interpreter ends
            _lib.rcc_adamw_destroy(self.handle)
            self.handle = None


def _stream_of(handle, dev):
    return torch.cuda.default_stream(dev) if handle in (0, 1) else \
        torch.cuda.ExternalStream(handle, device=dev)


def _lm_stream(stream, dev):
    """The given stream as the current one, as the compiled calls have it."""
    return torch.cuda.stream(_stream_of(stream, dev) if isinstance(stream, int) else stream)


def adamw_step(plan, cfg, scale=1.0, stream=None):
    """rcc_adamw_step: one step over a plan's tensors, their gradients carrying
    the loss scale `scale` (1 / scale a normal fp32 number).  cfg: adamw_cfg.
    Nothing is read back."""
    if not isinstance(cfg, _rcc.AdamWCfg):
        raise ValueError("cfg must be one of adamw_cfg's")
    used = _lm.adamw_step(plan.handle, C.addressof(cfg), scale, plan.device, stream)
    plan.last = used
    if used not in plan.streams:
        plan._used_on(used)


def adamw_report(plan, stream=None):
    """What the plan's last step did, an AdamWStatus: waits for it, on whichever
    stream adamw_step ran it, and for what is on `stream` (replays of a graph)."""
    dev = plan.workspace.device
    with _lm_stream(stream, dev):
        torch.cuda.current_stream(dev).wait_stream(_stream_of(plan.last, dev))
        return _rcc.AdamWStatus.from_buffer_copy(
            plan.workspace[:C.sizeof(_rcc.AdamWStatus)].cpu().numpy().tobytes())


# ------------------------------------------------------------- output layer + cross entropy

def linear_ce_workspace(tokens, vocab, dim, backward=False, grad_dtype=torch.bfloat16):
    return _lib.rcc_linear_ce_workspace(tokens, vocab, dim, 1 if backward else 0,
                                        _rcc.F32 if grad_dtype == torch.float32 else _rcc.BF16)


def linear_ce_forward(x, w, labels, loss=None, lse=None, workspace=None, stream=None):
    """rcc_linear_ce_forward: softmax cross entropy of the logits x w^T.
    Returns (loss, lse), [tokens] float32 each."""
    return _lm.linear_ce_forward(x, w, labels, loss, lse, workspace, stream)


def linear_ce_backward(x, w, labels, lse, dloss, grad_dtype=None, dx=None, dw=None,
                       accumulate=False, workspace=None, need_dx=True, need_dw=True,
                       stream=None):
    """rcc_linear_ce_backward: gradients of sum(dloss * loss).  Returns (dx, dw)
    of grad_dtype (a passed output's, else bfloat16); None for one that is not
    needed.  With accumulate dw is passed and added to.

    The type also decides how exact the gradients are: for bfloat16 dz is
    rounded to bfloat16 too (0.0020 off 64 bits in all, where the rounding of
    the results alone is 0.0017); for float32 it keeps 24 bits (7e-7 off) at
    three times the gradients' products."""
    return _lm.linear_ce_backward(x, w, labels, lse, dloss, grad_dtype, dx, dw, accumulate,
                                  workspace, need_dx, need_dw, stream)
