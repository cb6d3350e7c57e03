"""Refusals of the language-model operators' C ABI and binding (no GPU needed).

Every malformed call returns its status before any CUDA call, so the fake
addresses below are never dereferenced.
"""
import pytest
import torch

BASE = 0x7F0000000000   # fake device addresses, 256-byte aligned


def at(i):
    return BASE + (i << 32)


@pytest.fixture
def L(rcc_lib):
    return rcc_lib


def changed(good, **by):
    args = dict(good, **by)
    return list(args.values())


def refused(L, name, good, status, **by):
    st = L.raw(name, *changed(good, **by))
    assert st == status, (by, st, L.last_error())
    assert L.last_error()


EMBED = dict(table=at(0), table_type=1, ld=64, ids=at(1), index=1, tokens=10, vocab=100, dim=64,
             scale=1.0, out=at(2), out_type=1, stream=None)


def test_embedding_forward_refusals(L):
    bad = L.ERR_INVALID_ARGUMENT
    for by in (dict(table=None), dict(ids=None), dict(out=None), dict(table_type=2),
               dict(out_type=-1), dict(index=2), dict(vocab=0), dict(dim=0), dict(dim=1 << 21),
               dict(tokens=1 << 31), dict(ld=1 << 31), dict(table=at(0) + 1), dict(ids=at(1) + 4),
               dict(out=at(0) + 64), dict(out=at(1) + 32, tokens=100),
               dict(tokens=(1 << 31) - 1000, dim=1 << 20, ld=1 << 20)):
        refused(L, "rcc_embedding_forward", EMBED, bad, **by)
    refused(L, "rcc_embedding_forward", EMBED, L.ERR_SHAPE_MISMATCH, ld=63)
    assert L.raw("rcc_embedding_forward", *changed(EMBED, tokens=0, table=None)) == L.OK


def test_embedding_backward_refusals(L):
    need = L.embedding_backward_workspace(10, 100, 64)
    good = dict(dout=at(0), dout_type=1, ld=64, ids=at(1), index=0, tokens=10, vocab=100, dim=64,
                scale=1.0, dtable=at(2), dtable_type=0, accumulate=0, ws=at(3), bytes=need,
                stream=None)
    for by in (dict(dout=None), dict(ids=None), dict(dtable=None), dict(ws=None),
               dict(dout_type=3), dict(dtable_type=9), dict(index=-1), dict(vocab=0), dict(dim=0),
               dict(ws=at(3) + 128), dict(dtable=at(2) + 2), dict(dtable=at(3) - 256),
               dict(dtable=at(0))):
        refused(L, "rcc_embedding_backward", good, L.ERR_INVALID_ARGUMENT, **by)
    for by in (dict(bytes=need - 1), dict(ld=1)):
        refused(L, "rcc_embedding_backward", good, L.ERR_SHAPE_MISMATCH, **by)
    assert L.raw("rcc_embedding_backward", *changed(good, tokens=0, accumulate=1)) == L.OK


def test_rmsnorm_refusals(L):
    good = dict(x=at(0), type=0, ld=256, weight=at(1), eps=1e-6, tokens=4, dim=256, y=at(2),
                kept=at(3), scales=at(4), stream=None)
    for by in (dict(x=None), dict(weight=None), dict(y=None), dict(kept=None), dict(scales=None),
               dict(type=2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(dim=0), dict(dim=32769, ld=32769), dict(x=at(0) + 2), dict(kept=at(3) + 8),
               dict(y=at(0)), dict(scales=at(3) + 16)):
        refused(L, "rcc_rmsnorm_forward", good, L.ERR_INVALID_ARGUMENT, **by)
    refused(L, "rcc_rmsnorm_forward", good, L.ERR_SHAPE_MISMATCH, ld=255)
    assert L.raw("rcc_rmsnorm_forward", *changed(good, tokens=0)) == L.OK
    need = L.rmsnorm_backward_workspace(4, 256)
    good = dict(dy=at(0), type=1, ld=256, kept=at(1), scales=at(2), weight=at(3), eps=0.0,
                tokens=4, dim=256, dx=at(4), dweight=at(5), accumulate=0, ws=at(6), bytes=need,
                stream=None)
    for by in (dict(dy=None), dict(kept=None), dict(scales=None), dict(weight=None),
               dict(dx=None), dict(dweight=None), dict(ws=None), dict(type=5), dict(eps=-0.5),
               dict(dim=1 << 16, ld=1 << 16), dict(kept=at(1) + 4), dict(dx=at(0)),
               dict(dweight=at(3) + 4), dict(ws=at(6) + 16)):
        refused(L, "rcc_rmsnorm_backward", good, L.ERR_INVALID_ARGUMENT, **by)
    for by in (dict(bytes=0), dict(ld=8)):
        refused(L, "rcc_rmsnorm_backward", good, L.ERR_SHAPE_MISMATCH, **by)


def test_linear_ce_refusals(L):
    need = L.linear_ce_workspace(4, 100, 64)
    good = dict(x=at(0), ld_x=64, w=at(1), ld_w=64, labels=at(2), index=1, tokens=4, vocab=100,
                dim=64, loss=at(3), lse=at(4), ws=at(5), bytes=need, stream=None)
    for by in (dict(x=None), dict(w=None), dict(labels=None), dict(loss=None), dict(lse=None),
               dict(ws=None), dict(index=7), dict(vocab=0), dict(dim=60), dict(ld_x=68),
               dict(ld_w=65), dict(x=at(0) + 8), dict(w=at(1) + 2), dict(loss=at(4) + 12),
               dict(ws=at(5) + 64), dict(vocab=1 << 31)):
        refused(L, "rcc_linear_ce_forward", good, L.ERR_INVALID_ARGUMENT, **by)
    for by in (dict(bytes=need - 1), dict(ld_x=56), dict(ld_w=0)):
        refused(L, "rcc_linear_ce_forward", good, L.ERR_SHAPE_MISMATCH, **by)
    assert L.raw("rcc_linear_ce_forward", *changed(good, tokens=0, x=None)) == L.OK
    for kind, dtype in ((0, torch.float32), (1, torch.bfloat16)):
        need = L.linear_ce_workspace(4, 100, 64, True, dtype)
        good = dict(x=at(0), ld_x=64, w=at(1), ld_w=64, labels=at(2), index=1, lse=at(3),
                    dloss=at(4), tokens=4, vocab=100, dim=64, dx=at(5), dw=at(6), kind=kind,
                    accumulate=0, ws=at(7), bytes=need, stream=None)
        for by in (dict(lse=None), dict(dloss=None), dict(dx=None, dw=None), dict(kind=2),
                   dict(dx=at(5) + 8), dict(dw=at(6) + 4), dict(dw=at(5)), dict(dx=at(0)),
                   dict(dim=4), dict(ws=None)):
            refused(L, "rcc_linear_ce_backward", good, L.ERR_INVALID_ARGUMENT, **by)
        for by in (dict(bytes=need // 2), dict(ld_w=8)):
            refused(L, "rcc_linear_ce_backward", good, L.ERR_SHAPE_MISMATCH, **by)


def test_workspaces_of_sizes_that_no_call_takes(L):
    assert L.embedding_backward_workspace(1 << 40, 10, 10) == 0
    assert L.rmsnorm_backward_workspace(10, 0) == 0
    assert L.rmsnorm_backward_workspace(10, 1 << 20) == 0
    assert L.linear_ce_workspace(0, 10, 8) == 0


def test_binding_refuses_what_the_pointers_hide(L):
    f, b = torch.float32, torch.bfloat16
    table, ids = torch.zeros(10, 16), torch.zeros(4, dtype=torch.int64)
    for args in ((table.half(), ids), (table, ids.float()), (table, ids.view(2, 2)),
                 (table.t(), ids), (table, ids.repeat(2)[::2])):
        with pytest.raises(ValueError):
            L.embedding_forward(*args)
    with pytest.raises(ValueError, match="CUDA device"):
        L.embedding_forward(table, ids)
    with pytest.raises(ValueError):
        L.embedding_forward(table, ids, out=torch.zeros(4, 8))
    with pytest.raises(ValueError):
        L.embedding_backward(torch.zeros(4, 8), ids, table)
    with pytest.raises(ValueError):
        L.embedding_backward(torch.zeros(4, 16), ids[:3], table)
    x, weight = torch.zeros(4, 256), torch.ones(256)
    for args in ((x, weight.to(b)), (x, weight[:8]), (x.double(), weight), (x.expand(4, 256)[0], weight)):
        with pytest.raises(ValueError):
            L.rmsnorm_forward(*args)
    with pytest.raises(ValueError, match="CUDA device"):
        L.rmsnorm_forward(x, weight, keep=True)
    kept = L.Kept(4, 255, "cpu")
    with pytest.raises(ValueError):
        L.rmsnorm_backward(x, kept, weight)
    with pytest.raises(ValueError):
        L.rmsnorm_backward(x, L.Kept(4, 256, "cpu"), weight, accumulate=True)
    x, w = torch.zeros(4, 64, dtype=b), torch.zeros(100, 64, dtype=b)
    lab, v = torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    for args in ((x.to(f), w, lab), (x, w.to(f), lab), (x, w[:, :32], lab), (x, w, lab[:2])):
        with pytest.raises(ValueError):
            L.linear_ce_forward(*args)
    with pytest.raises(ValueError, match="CUDA device"):
        L.linear_ce_forward(x, w, lab)
    with pytest.raises(ValueError, match="CUDA device"):
        L.linear_ce_backward(x, w, lab, v, v)
    for args, more in (((x, w, lab, v[:1], v), {}), ((x, w, lab, v, v.to(b)), {}),
                       ((x, w, lab, v, v), dict(dx=torch.zeros(4, 64), dw=torch.zeros(100, 64, dtype=b))),
                       ((x, w, lab, v, v), dict(accumulate=True)),
                       ((x, w, lab, v, v), dict(grad_dtype=torch.float16))):
        with pytest.raises(ValueError):
            L.linear_ce_backward(*args, **more)
