"""Binding of the language-model operators of librcc (include/rcc.h): token
embedding and its gradient, the RMS norm that keeps its input in 8 bits, and
the output layer with softmax cross entropy.  Reached as attributes of `rcc`,
like the rest of the binding.

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
    "rcc_linear_ce_forward", "rcc_linear_ce_backward", "rcc_linear_ce_workspace")))


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
