"""Refusals of the training-step operators that need no GPU: sizes, types,
pointers, alignment, workspaces, and the shape checks of the binding."""
import ctypes

import pytest
import torch

from matrix_optimizers_gb300 import _binding as B

P = ctypes.c_void_p
A, ODD = P(1 << 20), P((1 << 20) + 1)            # never dereferenced: every call below is refused or a no-op


def test_struct_size_matches_header():
    assert ctypes.sizeof(B.mo_distill) == 80


def lookup(lib, W=A, wd=0, vocab=8, dim=8, ldw=8, ids=A, idd=B.MO_I32, n=4, out=A, od=0, ldo=8):
    return lib.embedding_lookup(W, wd, vocab, dim, ldw, ids, idd, n, 1.0, out, od, ldo, None)


def test_embedding_lookup_refusals(lib):
    inv, al, un = B.MO_ERR_INVALID_ARG, B.MO_ERR_ALIGNMENT, B.MO_ERR_UNSUPPORTED
    for kw in (dict(wd=2), dict(od=7), dict(idd=0), dict(vocab=-1), dict(dim=-1), dict(n=-1), dict(W=None),
               dict(ids=None), dict(out=None), dict(ldw=7), dict(ldo=7)):
        assert lookup(lib, **kw) == inv, kw
    for kw in (dict(W=ODD), dict(out=ODD), dict(ids=ODD)):
        assert lookup(lib, **kw) == al, kw
    assert lookup(lib, vocab=1 << 31) == un and lookup(lib, n=1 << 31) == un
    assert lookup(lib, n=0, W=None, ids=None, out=None) == B.MO_OK and lookup(lib, dim=0, out=None) == B.MO_OK


def egrad(lib, dY=A, yd=0, n=4, dim=8, ldy=8, ids=A, idd=B.MO_I64, vocab=8, dW=A, wd=0, ldw=8, acc=0, ws=A,
          wsb=1 << 30):
    return lib.embedding_grad(dY, yd, n, dim, ldy, ids, idd, vocab, 1.0, dW, wd, ldw, acc, ws, wsb, None)


def test_embedding_grad_refusals(lib):
    inv, al = B.MO_ERR_INVALID_ARG, B.MO_ERR_ALIGNMENT
    for kw in (dict(yd=3), dict(wd=-1), dict(idd=1), dict(n=-1), dict(dim=-2), dict(vocab=-1), dict(acc=2),
               dict(dY=None), dict(ids=None), dict(dW=None), dict(ldy=7), dict(ldw=7)):
        assert egrad(lib, **kw) == inv, kw
    for kw in (dict(dY=ODD), dict(dW=ODD), dict(ids=P((1 << 20) + 4))):
        assert egrad(lib, **kw) == al, kw
    for kw in (dict(ws=None), dict(ws=P((1 << 20) + 64)), dict(wsb=16)):
        assert egrad(lib, **kw) == B.MO_ERR_WORKSPACE, kw
    assert egrad(lib, n=1 << 31) == B.MO_ERR_UNSUPPORTED
    assert egrad(lib, vocab=0, dW=None) == B.MO_OK and egrad(lib, dim=0, dW=None) == B.MO_OK
    out = ctypes.c_size_t(0)
    assert lib.embedding_grad_workspace_bytes(4, 8, 8, None) == inv
    assert lib.embedding_grad_workspace_bytes(0, 8, 8, ctypes.byref(out)) == B.MO_OK and out.value >= 256
    assert B.embedding_grad_workspace_bytes(32768, 128000, 2048) < 32768 * 2048 * 2


def fwd(lib, X=A, ldx=16, W=A, ldw=16, sw=128, off=A, R=4, n=8, k=16, E=2, Y=A, yd=1, ldy=8, ws=A, wsb=1 << 30):
    return lib.expert_linear(X, ldx, W, ldw, sw, off, R, n, k, E, Y, yd, ldy, ws, wsb, None)


def dgrad(lib, dY=A, ldy=8, W=A, ldw=16, sw=128, off=A, R=4, n=8, k=16, E=2, dX=A, xd=1, ldx=16, ws=A, wsb=1 << 30):
    return lib.expert_linear_dgrad(dY, ldy, W, ldw, sw, off, R, n, k, E, dX, xd, ldx, ws, wsb, None)


def wgrad(lib, dY=A, ldy=8, X=A, ldx=16, off=A, R=4, n=8, k=16, E=2, dW=A, wd=0, ldw=16, sw=128, acc=0, ws=A,
          wsb=1 << 30):
    return lib.expert_linear_wgrad(dY, ldy, X, ldx, off, R, n, k, E, dW, wd, ldw, sw, acc, ws, wsb, None)


@pytest.mark.parametrize("f,ptrs,lds", [(fwd, ("X", "W", "Y"), ("ldx", "ldw", "ldy")),
                                        (dgrad, ("dY", "W", "dX"), ("ldy", "ldw", "ldx")),
                                        (wgrad, ("dY", "X", "dW"), ("ldy", "ldx", "ldw"))])
def test_expert_refusals(lib, f, ptrs, lds):
    inv, al, un = B.MO_ERR_INVALID_ARG, B.MO_ERR_ALIGNMENT, B.MO_ERR_UNSUPPORTED
    for kw in [{p: None} for p in ptrs] + [{l: 1} for l in lds] + [dict(R=-1), dict(n=-1), dict(k=-1), dict(E=0),
                                                                  dict(off=None), dict(sw=120)]:
        assert f(lib, **kw) == inv, kw
    for kw in [{p: P((1 << 20) + 8)} for p in ptrs] + [{l: 17} for l in lds] + [dict(off=ODD), dict(sw=1000 + 1)]:
        assert f(lib, **kw) == al, kw
    for kw in (dict(E=1025), dict(R=(1 << 31) - 1), dict(n=(1 << 20) + 8), dict(k=(1 << 20) + 8)):
        assert f(lib, **kw) == un, kw
    for kw in (dict(ws=None), dict(ws=P((1 << 20) + 16)), dict(wsb=8)):
        assert f(lib, **kw) == B.MO_ERR_WORKSPACE, kw


def test_expert_no_ops(lib):
    assert fwd(lib, R=0, X=None, Y=None) == B.MO_OK and fwd(lib, n=0, W=None, Y=None) == B.MO_OK
    assert dgrad(lib, R=0, dY=None, dX=None) == B.MO_OK and dgrad(lib, k=0, W=None, dX=None) == B.MO_OK
    assert wgrad(lib, n=0, dW=None) == B.MO_OK and wgrad(lib, k=0, dW=None) == B.MO_OK
    assert wgrad(lib, acc=3) == B.MO_ERR_INVALID_ARG and fwd(lib, yd=4) == B.MO_ERR_INVALID_ARG
    assert lib.expert_linear_workspace_bytes(4, 8, 16, 2, None) == B.MO_ERR_INVALID_ARG


def dist(lib, which="both", n=2, vocab=16, ldl=16, top=4, ld_=0, idd=B.MO_I32, td=0, T=1.0, logits=A, idx=A, t=A, w=None,
         loss=A, stats=A, grad=P(1 << 21), gd=0, ldg=16):
    d = B.mo_distill(n, vocab, ldl, top, ld_, idd, td, T, 1.0, logits, idx, t, w)
    r = ctypes.byref(d)
    if which == "loss":
        return lib.distill_topk_loss(r, loss, stats, None)
    if which == "grad":
        return lib.distill_topk_grad(r, stats, grad, gd, ldg, None)
    return lib.distill_topk_loss_grad(r, loss, grad, gd, ldg, None)


@pytest.mark.parametrize("which", ["loss", "grad", "both"])
def test_distill_refusals(lib, which):
    inv, al, un = B.MO_ERR_INVALID_ARG, B.MO_ERR_ALIGNMENT, B.MO_ERR_UNSUPPORTED
    for kw in (dict(n=-1), dict(vocab=-1), dict(ldl=15), dict(top=0), dict(ld_=2), dict(idd=0), dict(td=5), dict(T=0.0),
               dict(T=-1.0), dict(T=float("nan")), dict(T=float("inf")), dict(logits=None), dict(idx=None),
               dict(t=None)):
        assert dist(lib, which, **kw) == inv, kw
    for kw in (dict(logits=ODD), dict(idx=ODD), dict(t=ODD), dict(w=ODD)):
        assert dist(lib, which, **kw) == al, kw
    for kw in (dict(top=1025), dict(vocab=1 << 31, ldl=1 << 31, ldg=1 << 31)):
        assert dist(lib, which, **kw) == un, kw
    if which != "grad":
        assert dist(lib, which, loss=None) == inv and dist(lib, which, loss=ODD) == al
    if which != "both":
        assert dist(lib, which, stats=None) == inv and dist(lib, which, stats=ODD) == al
    if which != "loss":
        assert dist(lib, which, grad=None) == inv and dist(lib, which, gd=9) == inv and dist(lib, which, ldg=9) == inv
        assert dist(lib, which, grad=ODD) == al
        assert dist(lib, which, grad=A, gd=1) == inv and dist(lib, which, grad=A, ldg=24) == inv    # in place
    assert dist(lib, which, n=0, logits=None, idx=None, t=None, loss=None, stats=None, grad=None) == B.MO_OK
    assert lib.distill_topk_loss(None, A, A, None) == inv


def test_binding_refuses_host_tensors_and_wrong_shapes():
    f, i = torch.zeros((4, 8)), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: B.embedding_lookup(f, i, f), lambda: B.embedding_grad(f, i, f, f),
                 lambda: B.expert_linear(f, f, i, f, f), lambda: B.distill_topk_loss(f, i, f, f, f)):
        with pytest.raises(B.MoError) as e:
            call()
        assert e.value.status == B.MO_ERR_INVALID_ARG


@pytest.mark.parametrize("which", ["loss", "grad", "both"])
def test_distill_refuses_what_its_arithmetic_cannot_hold(lib, which):
    # a thread's column index, one stride of 256 past the last column, must fit 31 bits
    for vocab in ((1 << 31) - 1, (1 << 31) - 256):
        assert dist(lib, which, vocab=vocab, ldl=vocab, ldg=vocab) == B.MO_ERR_UNSUPPORTED, vocab
    # log2(e) / T must be finite
    for T in (1e-45, 1e-39):
        assert dist(lib, which, T=T) == B.MO_ERR_INVALID_ARG, T


class _On:
    """What _op_stream asks of a tensor or a stream."""

    def __init__(self, device, handle=0):
        self.device, self.cuda_stream = torch.device("cuda", device), handle

    def get_device(self):
        return self.device.index


def test_tensors_and_streams_of_another_device_are_refused(monkeypatch):
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    monkeypatch.setattr(B, "_current_raw_stream", lambda device: 100 + device)
    assert B._op_stream(None, (_On(0), _On(0))) == 100
    assert B._op_stream(_On(0, 7), (_On(0),)) == 7
    for stream, tensors in ((None, (_On(1), _On(1))), (_On(1, 7), (_On(1),)), (_On(1, 7), (_On(0),)), (None, (_On(0), _On(1)))):
        with pytest.raises(B.MoError) as e:
            B._op_stream(stream, tensors)
        assert e.value.status == B.MO_ERR_INVALID_ARG


def test_pitches_of_single_rows_do_not_depend_on_their_strides():
    t = torch.zeros((3, 2, 100))
    assert B._matrix(t[:, 0][:1], "") == B._matrix(t[0, 0][None], "")          # the same row
    for dtype, k in ((torch.float32, 12), (torch.bfloat16, 24)):
        for stack in (torch.zeros((2, 1, k), dtype=dtype), torch.zeros((1, 2, k), dtype=dtype).transpose(0, 1)):
            *_, experts, rows, cols, ld, stride = B._stack(stack, "")
            assert (experts, rows, cols, stride) == (2, 1, k, k) and cols <= ld and rows * ld <= stride
            assert ld * stack.element_size() % 16 == 0
    *_, ld, stride = B._stack(torch.zeros((1, 1, 13)), "")
    assert ld >= 13 and ld % 4 == 0 and stride % 4 == 0
