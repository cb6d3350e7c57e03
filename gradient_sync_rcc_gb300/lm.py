"""Python binding of the language-model operators of librcc (include/rcc.h):
token embedding and its gradient, the RMS norm that keeps its input in 8 bits,
and the output layer with softmax cross entropy.  Reached as attributes of
`rcc`, like the rest of the binding.

The C calls receive bare pointers, sizes and strides; what they cannot see (a
type, a device, a shape that does not fit) is checked here.  An output or a
workspace that is not passed is allocated on the inputs' device, to be used on
`stream` (the current one by default; tensors passed in must be safe to use
there).  The checks read each attribute once: on small inputs the call's own
time is what a user waits for.
"""
import torch

from gradient_sync_rcc_gb300.rcc import BF16, F32, I32, I64, OK, RccError, last_error, lib

_lib = lib()

_TYPES = {torch.float32: F32, torch.bfloat16: BF16}
_INDEX = {torch.int32: I32, torch.int64: I64}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, dev):
    """The caller's stream, or the device's current one."""
    if stream is None:
        if dev < 0:
            raise ValueError("the operators take tensors on a CUDA device")
        if _raw_stream is not None:
            return _raw_stream(dev)
        return torch.cuda.current_stream(dev).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _check(status):
    if status != OK:
        raise RccError(status, last_error())


def _type(t, what):
    kind = _TYPES.get(t.dtype)
    if kind is None:
        raise ValueError("%s must be float32 or bfloat16, not %s" % (what, t.dtype))
    return kind


def _matrix(t, what, dev):
    """Rows, columns and row stride of a matrix whose rows are contiguous."""
    shape = t.shape
    if len(shape) != 2 or t.get_device() != dev:
        raise ValueError("%s must be a matrix on the inputs' device" % what)
    n, d = shape
    if t.is_contiguous():
        return n, d, d
    ld, step = t.stride()
    if step != 1 and d != 1:
        raise ValueError("the rows of %s must be contiguous" % what)
    if n < 2:
        return n, d, d
    if ld < d:
        raise ValueError("the rows of %s overlap" % what)
    return n, d, ld


def _index(t, what, dev, n):
    """The index type of a contiguous vector of n ids."""
    kind = _INDEX.get(t.dtype)
    if kind is None or t.dim() != 1 or t.get_device() != dev or t.numel() != n or \
            not t.is_contiguous():
        raise ValueError("%s must be a contiguous vector of %d int32 or int64 on the inputs' device"
                         % (what, n))
    return kind


def _floats(t, what, dev, n):
    """The address of a contiguous vector of n float32."""
    if t.dtype != torch.float32 or t.dim() != 1 or t.get_device() != dev or t.numel() != n or \
            not t.is_contiguous():
        raise ValueError("%s must be a contiguous vector of %d float32 on the inputs' device"
                         % (what, n))
    return t.data_ptr()


def _output(t, what, like, shape, dtype):
    """The caller's output, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    if t.shape != shape or t.dtype != dtype or t.get_device() != like.get_device() or \
            not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on the inputs' device"
                         % (what, dtype, tuple(shape)))
    return t


def _workspace(t, like, need):
    """The workspace, its address and its bytes."""
    if t is None:
        t = torch.empty(need, dtype=torch.uint8, device=like.device)
        return t, t.data_ptr(), need
    if t.get_device() != like.get_device() or not t.is_contiguous():
        raise ValueError("the workspace must be a contiguous tensor on the inputs' device")
    return t, t.data_ptr(), t.numel() * t.element_size()


# ------------------------------------------------------------- embedding

def embedding_forward(table, ids, scale=1.0, out=None, out_dtype=None, stream=None):
    """rcc_embedding_forward: scale * table[ids], a row of zeros for an id
    outside the table.  Returns out [tokens, dim] of out_dtype (the table's)."""
    dev = table.get_device()
    vocab, dim, ld = _matrix(table, "table", dev)
    tokens = ids.numel()
    index = _index(ids, "ids", dev, tokens)
    kind = _type(table, "table")
    if out is None:
        if out_dtype is None:
            out_dtype = table.dtype
        out_kind = _TYPES.get(out_dtype)
        if out_kind is None:
            raise ValueError("out_dtype must be float32 or bfloat16, not %s" % out_dtype)
        out = torch.empty((tokens, dim), dtype=out_dtype, device=table.device)
    else:
        _output(out, "out", table, (tokens, dim), out_dtype or out.dtype)
        out_kind = _type(out, "out")
    st = _lib.rcc_embedding_forward(
        table.data_ptr(), kind, ld, ids.data_ptr(), index, tokens, vocab, dim, scale,
        out.data_ptr(), out_kind, _stream(stream, dev))
    if st:
        _check(st)
    return out


def embedding_backward_workspace(tokens, vocab, dim):
    return _lib.rcc_embedding_backward_workspace(tokens, vocab, dim)


def embedding_backward(dout, ids, dtable, scale=1.0, accumulate=False, workspace=None,
                       stream=None):
    """rcc_embedding_backward: the gradient of embedding_forward's table, into
    dtable [vocab, dim] (added to it with accumulate).  Returns dtable."""
    dev = dout.get_device()
    tokens, dim, ld = _matrix(dout, "dout", dev)
    if dtable.dim() != 2 or dtable.shape[1] != dim:
        raise ValueError("dtable must have dout's %d columns" % dim)
    vocab = dtable.shape[0]
    index = _index(ids, "ids", dev, tokens)
    _output(dtable, "dtable", dout, (vocab, dim), dtable.dtype)
    kinds = _type(dout, "dout"), _type(dtable, "dtable")
    ws, at, have = _workspace(workspace, dout, embedding_backward_workspace(tokens, vocab, dim))
    _check(_lib.rcc_embedding_backward(
        dout.data_ptr(), kinds[0], ld, ids.data_ptr(), index, tokens, vocab, dim, scale,
        dtable.data_ptr(), kinds[1], 1 if accumulate else 0, at, have, _stream(stream, dev)))
    return dtable


# ------------------------------------------------------------- RMS norm

KEEP_GROUP = 128   # columns that share one scale of the 8-bit form


class Kept:
    """A norm's input in 8 bits: values [tokens, 128 G] int8 and scales
    [tokens, G] float32 of its `dim` columns, G = ceil(dim / 128), one after
    the other in one buffer."""

    __slots__ = ("data", "tokens", "dim", "groups", "_scales_at")

    def __init__(self, tokens, dim, device):
        self.tokens, self.dim, self.groups = tokens, dim, -(-dim // KEEP_GROUP)
        self._scales_at = tokens * self.groups * KEEP_GROUP
        self.data = torch.empty(self._scales_at + tokens * self.groups * 4, dtype=torch.uint8,
                                device=device)

    @property
    def values(self):
        return self.data[:self._scales_at].view(torch.int8).view(self.tokens,
                                                                 self.groups * KEEP_GROUP)

    @property
    def scales(self):
        return self.data[self._scales_at:].view(torch.float32).view(self.tokens, self.groups)

    def dequantize(self):
        """What it stands for, [tokens, dim] float32."""
        t, g = self.tokens, self.groups
        v = self.values.view(t, g, KEEP_GROUP) * self.scales[:, :, None]
        return v.view(t, g * KEEP_GROUP)[:, :self.dim]

    def _checked(self, tokens, dim, dev):
        """The addresses of the values and the scales."""
        if self.dim != dim or self.tokens != tokens or self.data.get_device() != dev:
            raise ValueError("kept holds %d x %d on %s where %d x %d on the inputs' device is needed"
                             % (self.tokens, self.dim, self.data.device, tokens, dim))
        at = self.data.data_ptr()
        return at, at + self._scales_at


def rmsnorm_forward(x, weight, eps=1e-6, keep=False, out=None, stream=None):
    """rcc_rmsnorm_forward.  Returns y, or (y, kept) with keep: True, or a Kept
    of these sizes to be written."""
    dev = x.get_device()
    tokens, dim, ld = _matrix(x, "x", dev)
    kind = _type(x, "x")
    w = _floats(weight, "weight", dev, dim)
    y = torch.empty_like(x) if out is None and ld == dim else \
        _output(out, "out", x, (tokens, dim), x.dtype)
    kept = q = s = None
    if keep:
        kept = Kept(tokens, dim, x.device) if keep is True else keep
        q, s = kept._checked(tokens, dim, dev)
    st = _lib.rcc_rmsnorm_forward(x.data_ptr(), kind, ld, w, eps, tokens, dim, y.data_ptr(), q, s,
                                  _stream(stream, dev))
    if st:
        _check(st)
    return y if kept is None else (y, kept)


def rmsnorm_backward_workspace(tokens, dim):
    return _lib.rcc_rmsnorm_backward_workspace(tokens, dim)


def rmsnorm_backward(dy, kept, weight, eps=1e-6, dx=None, dweight=None, accumulate=False,
                     workspace=None, stream=None):
    """rcc_rmsnorm_backward from a Kept.  Returns (dx, dweight); with accumulate
    dweight is passed and added to."""
    dev = dy.get_device()
    tokens, dim, ld = _matrix(dy, "dy", dev)
    kind = _type(dy, "dy")
    q, s = kept._checked(tokens, dim, dev)
    w = _floats(weight, "weight", dev, dim)
    if accumulate and dweight is None:
        raise ValueError("accumulate needs the dweight to add to")
    dx = torch.empty_like(dy) if dx is None and ld == dim else \
        _output(dx, "dx", dy, (tokens, dim), dy.dtype)
    dweight = _output(dweight, "dweight", dy, (dim,), torch.float32)
    ws, at, have = _workspace(workspace, dy, rmsnorm_backward_workspace(tokens, dim))
    _check(_lib.rcc_rmsnorm_backward(
        dy.data_ptr(), kind, ld, q, s, w, eps, tokens, dim, dx.data_ptr(), dweight.data_ptr(),
        1 if accumulate else 0, at, have, _stream(stream, dev)))
    return dx, dweight


# ------------------------------------------------------------- output layer + cross entropy

def linear_ce_workspace(tokens, vocab, dim, backward=False, grad_dtype=torch.bfloat16):
    return _lib.rcc_linear_ce_workspace(tokens, vocab, dim, 1 if backward else 0,
                                         _TYPES[grad_dtype])


def _ce_inputs(x, w, labels):
    dev = x.get_device()
    if x.dtype != torch.bfloat16 or w.dtype != torch.bfloat16:
        raise ValueError("x and w must be bfloat16")
    tokens, dim, ld_x = _matrix(x, "x", dev)
    vocab, wide, ld_w = _matrix(w, "w", dev)
    if wide != dim:
        raise ValueError("x has %d columns, w %d" % (dim, wide))
    return dev, tokens, vocab, dim, ld_x, ld_w, _index(labels, "labels", dev, tokens)


def linear_ce_forward(x, w, labels, loss=None, lse=None, workspace=None, stream=None):
    """rcc_linear_ce_forward: softmax cross entropy of the logits x w^T.
    Returns (loss, lse), [tokens] float32 each."""
    dev, tokens, vocab, dim, ld_x, ld_w, index = _ce_inputs(x, w, labels)
    loss = _output(loss, "loss", x, (tokens,), torch.float32)
    lse = _output(lse, "lse", x, (tokens,), torch.float32)
    ws, at, have = _workspace(workspace, x, _lib.rcc_linear_ce_workspace(tokens, vocab, dim, 0, F32))
    _check(_lib.rcc_linear_ce_forward(
        x.data_ptr(), ld_x, w.data_ptr(), ld_w, labels.data_ptr(), index, tokens, vocab, dim,
        loss.data_ptr(), lse.data_ptr(), at, have, _stream(stream, dev)))
    return loss, lse


def linear_ce_backward(x, w, labels, lse, dloss, grad_dtype=None, dx=None, dw=None,
                       accumulate=False, workspace=None, need_dx=True, need_dw=True,
                       stream=None):
    """rcc_linear_ce_backward: gradients of sum(dloss * loss).  Returns (dx, dw)
    of grad_dtype (a passed output's, else bfloat16); None for one that is not
    needed.  With accumulate dw is passed and added to."""
    dev, tokens, vocab, dim, ld_x, ld_w, index = _ce_inputs(x, w, labels)
    at_lse, at_dloss = _floats(lse, "lse", dev, tokens), _floats(dloss, "dloss", dev, tokens)
    if accumulate and dw is None:
        raise ValueError("accumulate needs the dw to add to")
    if grad_dtype is None:
        given = dx if dx is not None else dw
        grad_dtype = torch.bfloat16 if given is None else given.dtype
    grad = _TYPES.get(grad_dtype)
    if grad is None:
        raise ValueError("grad_dtype must be float32 or bfloat16, not %s" % grad_dtype)
    dx = _output(dx, "dx", x, (tokens, dim), grad_dtype) if need_dx else None
    dw = _output(dw, "dw", x, (vocab, dim), grad_dtype) if need_dw else None
    ws, at, have = _workspace(workspace, x,
                              _lib.rcc_linear_ce_workspace(tokens, vocab, dim, 1, grad))
    _check(_lib.rcc_linear_ce_backward(
        x.data_ptr(), ld_x, w.data_ptr(), ld_w, labels.data_ptr(), index, at_lse, at_dloss,
        tokens, vocab, dim, None if dx is None else dx.data_ptr(),
        None if dw is None else dw.data_ptr(), grad, 1 if accumulate else 0, at, have,
        _stream(stream, dev)))
    return dx, dw
