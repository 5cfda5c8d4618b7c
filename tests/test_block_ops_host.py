"""Refusals of the block operators (routing, rows to the experts and back, norms,
AdamW over many tensors) that need no GPU: sizes, types, pointers, alignment,
workspaces, and the shape checks of the binding."""
import ctypes

import pytest
import torch

from matrix_optimizers_gb300 import _binding as B

P = ctypes.c_void_p
A, ODD = P(1 << 20), P((1 << 20) + 1)            # never dereferenced: every call below is refused or a no-op
INV, AL, UN, WS = B.MO_ERR_INVALID_ARG, B.MO_ERR_ALIGNMENT, B.MO_ERR_UNSUPPORTED, B.MO_ERR_WORKSPACE


def test_struct_sizes_match_header():
    assert ctypes.sizeof(B.mo_route) == 48
    assert ctypes.sizeof(B.mo_block_norm) == 112
    assert ctypes.sizeof(B.mo_adamw_tensor) == 80
    assert ctypes.sizeof(B.mo_adamw_cfg) == 48


def route(lib, n=4, ldl=8, E=8, top=2, dt=0, re=0, logits=A, mask=None, idx=A, gates=A, pos=A, order=None, offsets=A,
          counts=A, loss=None, ws=A, wsb=1 << 30):
    r = B.mo_route(n, ldl, E, top, dt, re, logits, mask)
    return lib.expert_route(ctypes.byref(r), idx, gates, pos, order, offsets, counts, loss, ws, wsb, None)


def route_grad(lib, n=4, ldl=8, E=8, top=2, dt=0, re=0, logits=A, mask=None, idx=A, counts=A, dgates=A,
               out=P(1 << 21), gd=0, ldg=8):
    r = B.mo_route(n, ldl, E, top, dt, re, logits, mask)
    return lib.expert_route_grad(ctypes.byref(r), idx, counts, dgates, 0.0, 0.0, out, gd, ldg, None)


@pytest.mark.parametrize("f", [route, route_grad])
def test_route_refusals(lib, f):
    for kw in (dict(n=-1), dict(E=0), dict(top=0), dict(top=9), dict(ldl=7), dict(dt=2), dict(re=2), dict(logits=None),
               dict(idx=None), dict(counts=None)):
        assert f(lib, **kw) == INV, kw
    for kw in (dict(logits=ODD), dict(idx=ODD), dict(counts=ODD)):
        assert f(lib, **kw) == AL, kw
    for kw in (dict(E=1025, ldl=1025, ldg=1025), dict(top=33, E=64, ldl=64, ldg=64), dict(n=(1 << 30) - 256), dict(n=1 << 62)):
        if f is route:
            kw.pop("ldg", None)
        assert f(lib, **kw) == UN, kw


def test_route_outputs_and_workspace(lib):
    for kw in (dict(gates=None), dict(pos=None), dict(offsets=None)):
        assert route(lib, **kw) == INV, kw
    for kw in (dict(gates=ODD), dict(pos=ODD), dict(offsets=ODD), dict(order=ODD), dict(loss=ODD)):
        assert route(lib, **kw) == AL, kw
    for kw in (dict(ws=None), dict(ws=P((1 << 20) + 64)), dict(wsb=16)):
        assert route(lib, **kw) == WS, kw
    assert lib.expert_route(None, A, A, A, None, A, A, None, A, 1 << 30, None) == INV
    assert lib.expert_route_workspace_bytes(4, 8, 2, None) == INV
    out = ctypes.c_size_t(0)
    for bad in ((-1, 8, 2), (4, 0, 1), (4, 8, 9)):
        assert lib.expert_route_workspace_bytes(*bad, ctypes.byref(out)) == INV
    assert lib.expert_route_workspace_bytes(4, 2000, 2, ctypes.byref(out)) == UN
    assert 0 < B.expert_route_workspace_bytes(0, 8, 2) <= B.expert_route_workspace_bytes(1 << 20, 1024, 32) < 1 << 27
    assert route_grad(lib, n=0, logits=None, idx=None, counts=None, out=None) == B.MO_OK
    for kw in (dict(out=None), dict(gd=5), dict(ldg=7), dict(out=A, gd=1), dict(out=A, ldg=16)):
        assert route_grad(lib, **kw) == INV, kw
    assert route_grad(lib, out=ODD) == AL and route_grad(lib, dgates=ODD) == AL


def scat(lib, X=A, xd=0, n=4, dim=8, ldx=8, pos=A, top=2, Xs=A, sd=0, slots=8, lds=8):
    return lib.expert_scatter(X, xd, n, dim, ldx, pos, top, Xs, sd, slots, lds, None)


def comb(lib, Ys=A, sd=0, slots=8, lds=8, pos=A, gates=None, n=4, top=2, dim=8, Y=A, yd=0, ldy=8, acc=0):
    return lib.expert_combine(Ys, sd, slots, lds, pos, gates, n, top, dim, Y, yd, ldy, acc, None)


def cgrad(lib, dY=A, yd=0, ldy=8, Ys=A, sd=0, slots=8, lds=8, pos=A, gates=None, n=4, top=2, dim=8, dYs=P(1 << 21),
          ldd=8, dgates=A):
    return lib.expert_combine_grad(dY, yd, ldy, Ys, sd, slots, lds, pos, gates, n, top, dim, dYs, ldd, dgates, None)


@pytest.mark.parametrize("f,ptrs,lds", [(scat, ("X", "Xs"), ("ldx", "lds")), (comb, ("Ys", "Y"), ("lds", "ldy")),
                                        (cgrad, ("dY", "Ys", "dYs"), ("ldy", "lds", "ldd"))])
def test_exchange_refusals(lib, f, ptrs, lds):
    for kw in [{p: None} for p in ptrs] + [{v: 7} for v in lds] + [dict(n=-1), dict(dim=-1), dict(slots=-1), dict(top=0),
                                                                  dict(sd=2), dict(pos=None)]:
        assert f(lib, **kw) == INV, kw
    for kw in [{p: ODD} for p in ptrs] + [dict(pos=ODD)]:
        assert f(lib, **kw) == AL, kw
    for kw in (dict(top=33), dict(n=1 << 31), dict(n=1 << 30), dict(slots=1 << 31), dict(dim=(1 << 24) + 1)):
        assert f(lib, **kw) == UN, kw
    assert f(lib, n=0, **{p: None for p in ptrs}) == B.MO_OK


def test_exchange_options(lib):
    assert comb(lib, acc=2) == INV and comb(lib, gates=ODD) == AL and cgrad(lib, gates=ODD) == AL
    assert cgrad(lib, dgates=ODD) == AL and cgrad(lib, dYs=A, ldd=16) == INV
    assert scat(lib, dim=0, X=None, Xs=None) == B.MO_OK and comb(lib, dim=0, Ys=None, Y=None) == B.MO_OK


def norm(lib, n=4, dim=8, ldx=8, ldr=8, rpg=4, ldgate=8, xd=0, sd=0, pd=0, eps=1e-6, x=A, res=None, post=None,
         gate=None, pre=None, y=P(1 << 21), ldy=8, h=None, ldh=8):
    p = B.mo_block_norm(n, dim, ldx, ldr, rpg, ldgate, xd, sd, pd, eps, 1.0, 1.0, x, res, post, gate, pre)
    return lib.block_norm(ctypes.byref(p), y, ldy, h, ldh, None)


def norm_grad(lib, n=4, dim=8, ldx=8, rpg=4, ldgate=8, xd=0, sd=0, pd=0, eps=1e-6, x=A, post=None, gate=None,
              pre=None, y=P(1 << 21), ldy=8, dy=None, lddy=8, dh=None, lddh=8, dx=P(1 << 22), lddx=8, dr=None, lddr=8,
              dpost=None, dgate=None, dpre=None, acc=0, ws=A, wsb=1 << 30):
    p = B.mo_block_norm(n, dim, ldx, 0, rpg, ldgate, xd, sd, pd, eps, 1.0, 1.0, x, None, post, gate, pre)
    return lib.block_norm_grad(ctypes.byref(p), y, ldy, dy, lddy, dh, lddh, dx, lddx, dr, lddr, dpost, dgate, dpre, acc,
                               ws, wsb, None)


@pytest.mark.parametrize("f", [norm, norm_grad])
def test_norm_refusals(lib, f):
    for kw in (dict(n=-1), dict(dim=-1), dict(xd=2), dict(sd=3), dict(pd=-1), dict(eps=-1.0),
               dict(eps=float("nan")), dict(x=None), dict(ldx=7), dict(gate=A, rpg=0), dict(gate=A, ldgate=7)):
        assert f(lib, **kw) == INV, kw
    for kw in (dict(x=ODD), dict(post=ODD), dict(gate=ODD), dict(y=ODD)):
        assert f(lib, **kw) == AL, kw
    for kw in (dict(dim=8193, ldx=1 << 15), dict(n=1 << 31)):
        assert f(lib, **kw) == UN, kw


def test_norm_outputs(lib):
    for kw in (dict(pre=A), dict(h=A), dict(y=None), dict(ldy=7), dict(pre=A, h=P(1 << 22), ldh=7), dict(res=A, ldr=7),
               dict(res=P(1 << 21), ldr=16), dict(pre=A, h=A, ldh=16)):
        assert norm(lib, **kw) == INV, kw
    assert norm(lib, res=ODD) == AL and norm(lib, pre=A, h=ODD) == AL
    assert norm(lib, n=0, x=None, y=None) == B.MO_OK and norm(lib, dim=0, x=None, y=None) == B.MO_OK
    for kw in (dict(acc=2), dict(pre=A), dict(dh=A), dict(dpre=A), dict(dpost=A), dict(dgate=A), dict(dx=None),
               dict(lddx=7), dict(dy=A, lddy=7), dict(pre=A, dh=A, y=None), dict(pre=A, dh=A, ldy=7),
               dict(pre=A, dh=A, lddh=7), dict(dr=A, lddr=7), dict(dy=A, dr=A, lddr=16), dict(dx=A, lddx=16),
               dict(pre=A, dh=P(1 << 22), lddh=16)):
        assert norm_grad(lib, **kw) == INV, kw
    for kw in (dict(dx=ODD), dict(dy=ODD), dict(dr=ODD), dict(pre=A, dh=ODD), dict(post=A, dpost=ODD)):
        assert norm_grad(lib, **kw) == AL, kw
    for kw in (dict(ws=None), dict(ws=P((1 << 20) + 64)), dict(wsb=8)):
        assert norm_grad(lib, **kw) == WS, kw
    assert norm_grad(lib, dim=0, x=None, dx=None) == B.MO_OK
    assert lib.block_norm_grad_workspace_bytes(4, 8, 0, None) == INV
    out = ctypes.c_size_t(0)
    assert lib.block_norm_grad_workspace_bytes(4, 8193, 0, ctypes.byref(out)) == UN
    assert lib.block_norm_grad_workspace_bytes(-4, 8, 0, ctypes.byref(out)) == INV
    assert B.block_norm_grad_workspace_bytes(0, 8, 0) >= 256


def adam(lib, cfg=None, count=1, arr=True, **kw):
    t = dict(numel=8, W=A, g=A, m=A, v=A, ms=None, vs=None, wd=0, gd=0, sd=0)
    t.update(kw)
    d = (B.mo_adamw_tensor * 1)(B.mo_adamw_tensor(t["numel"], t["W"], t["g"], t["m"], t["v"], t["ms"], t["vs"], t["wd"],
                                                  t["gd"], t["sd"], 1e-3, 0.0, 0))
    c = dict(b1=0.9, b2=0.95, eps=1e-8, step=1, ptr=None, mul=None, dither=0)
    c.update(cfg or {})
    cfg_ = B.mo_adamw_cfg(c["b1"], c["b2"], c["eps"], 1.0, c["step"], c["ptr"], c["mul"], 0, c["dither"])
    return lib.adamw_step_batched(d if arr else None, count, ctypes.byref(cfg_), None)


def test_adamw_batch_refusals(lib):
    for kw in (dict(numel=-1), dict(wd=2), dict(gd=4), dict(sd=1), dict(W=None), dict(g=None), dict(m=None),
               dict(v=None), dict(sd=4), dict(sd=4, ms=A), dict(count=-1), dict(arr=False)):
        assert adam(lib, **kw) == INV, kw
    for kw in (dict(W=ODD), dict(g=ODD), dict(m=ODD), dict(v=ODD), dict(sd=4, ms=ODD, vs=A)):
        assert adam(lib, **kw) == AL, kw
    assert adam(lib, numel=1 << 40) == UN
    for c in (dict(step=0), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0), dict(b2=float("nan")), dict(eps=-1.0),
              dict(dither=2)):
        assert adam(lib, cfg=c) == INV, c
    assert adam(lib, cfg=dict(ptr=P((1 << 20) + 4), step=0)) == AL and adam(lib, cfg=dict(mul=ODD)) == AL
    assert lib.adamw_step_batched(None, 0, None, None) == INV
    assert adam(lib, count=0, arr=False) == B.MO_OK and adam(lib, numel=0, W=None, g=None, m=None, v=None) == B.MO_OK


def refused(call):
    with pytest.raises(B.MoError) as e:
        call()
    assert e.value.status == INV


def test_binding_refuses_host_tensors():
    f, i, b = torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    o = torch.zeros(9, dtype=torch.int32)
    refused(lambda: B.expert_route(f, i, f, i, o, o, None, b))
    refused(lambda: B.expert_route_grad(f, i, o, None, f))
    refused(lambda: B.expert_scatter(f, i, f))
    refused(lambda: B.expert_combine(f, i, f))
    refused(lambda: B.expert_combine_grad(f, f, i, None, f, None))
    refused(lambda: B.block_norm(f, f, None))
    refused(lambda: B.block_norm_grad(f, f, None, None, f, b))
    refused(lambda: B.adamw_step_batched([B.make_adamw_tensor(f, f, f, f)], 1))


class _Cuda(torch.Tensor):
    """A host tensor that says it is on cuda:0, for the checks that come after that one."""

    def get_device(self):
        return 0


@pytest.fixture
def on_cuda(monkeypatch):
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    monkeypatch.setattr(B, "_current_raw_stream", lambda device: 0)
    monkeypatch.setattr(B, "_call", lambda name: lambda *a: pytest.fail(f"{name} was called"))
    return lambda *shape, dtype=torch.float32: torch.zeros(shape, dtype=dtype).as_subclass(_Cuda)


def test_binding_refuses_wrong_shapes_and_types(on_cuda):
    z = on_cuda
    f, i, b = z(4, 8), z(4, 2, dtype=torch.int32), z(256, dtype=torch.uint8)
    g, o = z(4, 2), z(9, dtype=torch.int32)
    ok = dict(logits=f, idx=i, gates=g, pos=i, offsets=o, counts=o, loss=None, ws=b)
    for kw in (dict(idx=z(4, dtype=torch.int32)), dict(idx=z(3, 2, dtype=torch.int32)), dict(idx=g), dict(gates=i),
               dict(gates=z(4, 3)), dict(pos=z(4, 3, dtype=torch.int32)), dict(offsets=z(8, dtype=torch.int32)),
               dict(counts=z(8, dtype=torch.int32)), dict(loss=z(3)), dict(order=z(7, dtype=torch.int32)),
               dict(mask=z(4)), dict(mask=z(5, dtype=torch.bool)), dict(logits=f.half()), dict(logits=z(8, 4).t())):
        refused(lambda: B.expert_route(**{**ok, **kw}))
    for kw in (dict(dgates=z(4, 3)), dict(dlogits=z(4, 7)), dict(counts=o[:4]), dict(idx=z(3, 2, dtype=torch.int32))):
        refused(lambda: B.expert_route_grad(**{**dict(logits=f, idx=i, counts=o, dgates=g, dlogits=f), **kw}))
    for kw in (dict(Xs=z(8, 7)), dict(pos=i.long()), dict(pos=i[:3]), dict(X=z(4, 8, 1))):
        refused(lambda: B.expert_scatter(**{**dict(X=f, pos=i, Xs=z(8, 8)), **kw}))
    refused(lambda: B.expert_combine(z(8, 7), i, f))
    refused(lambda: B.expert_combine(z(8, 8), i, f, gates=z(4, 3)))
    for kw in (dict(dYs=z(7, 8)), dict(dYs=z(8, 8, dtype=torch.bfloat16)), dict(dgates=z(4, 1)), dict(dY=z(4, 7))):
        ok2 = dict(dY=f, Ys=z(8, 8), pos=i, gates=g, dYs=z(8, 8), dgates=g)
        refused(lambda: B.expert_combine_grad(**{**ok2, **kw}))
    v = z(8)
    for kw in (dict(post=z(7)), dict(pre=z(9)), dict(post=v, pre=z(8, dtype=torch.bfloat16)), dict(gate=z(3, 8)),
               dict(gate=z(2, 8), rows_per_gate=4), dict(gate=z(2, 7)), dict(gate=z(2, 8), rows_per_gate=0),
               dict(residual=z(4, 7)), dict(residual=z(4, 8, dtype=torch.bfloat16)), dict(y=z(5, 8)), dict(h=z(4, 9)),
               dict(pre=v, h=z(4, 8, dtype=torch.bfloat16))):
        refused(lambda: B.block_norm(**{**dict(x=f, y=z(4, 8), h=None), **kw}))
    ok3 = dict(x=f, y=f, dy=f, dh=None, dx=z(4, 8), ws=b)
    for kw in (dict(dx=z(4, 8, dtype=torch.bfloat16)), dict(dy=z(4, 8, dtype=torch.bfloat16)), dict(post=v, dpost=z(7)),
               dict(gate=z(2, 8), dgate=z(8)), dict(dresidual=z(3, 8))):
        refused(lambda: B.block_norm_grad(**{**ok3, **kw}))
    e = z(8, dtype=torch.float8_e4m3fn)
    for args, kw in (((v, v, v, z(7)), {}), ((v, v.half(), v, v), {}), ((v, v, e, v), {}), ((v, v, e, e), {}),
                     ((v, v, e, e), dict(m_scale=z(1), v_scale=z(2))), ((v, v, v, v), dict(m_scale=z(1))),
                     ((z(4, 4)[:, :2], v, v, v), {})):
        refused(lambda: B.make_adamw_tensor(*args, **kw))
    one = [B.make_adamw_tensor(v, v, v, v)]
    refused(lambda: B.adamw_step_batched(one, z(1)))
    refused(lambda: B.adamw_step_batched(one, z(2, dtype=torch.int64)))
    refused(lambda: B.adamw_step_batched(one, 1, grad_mul=z(2)))
    B.adamw_step_batched([], 1)


def test_adamw_list_refuses_tensors_that_overlap(on_cuda):
    z = on_cuda
    mine = lambda n=512: [z(n) for _ in range(4)]  # noqa: E731
    a, b = B.make_adamw_tensor(*mine()), B.make_adamw_tensor(*mine())
    assert B.adamw_tensors([a, b]).count == 2
    refused(lambda: B.adamw_tensors([a, b, a]))
    whole, (W, g, m, v) = z(1000), mine()
    B.adamw_tensors([B.make_adamw_tensor(whole[:512], g, m, v), B.make_adamw_tensor(whole[512:], *[z(488) for _ in range(3)])])
    refused(lambda: B.adamw_tensors([B.make_adamw_tensor(whole[:512], g, m, v),
                                     B.make_adamw_tensor(whole[511:], *[z(489) for _ in range(3)])]))
    refused(lambda: B.adamw_tensors([B.make_adamw_tensor(W, g, m, m)]))
    e, f = z(512, dtype=torch.float8_e4m3fn), z(512, dtype=torch.float8_e4m3fn)
    s = z(2)
    refused(lambda: B.adamw_tensors([B.make_adamw_tensor(W, g, e, f, s, s)]))
    B.adamw_tensors([B.make_adamw_tensor(W, g, e, f, s, z(2)), B.make_adamw_tensor(z(0), g[:0], m[:0], v[:0])])
    B.adamw_tensors([B.make_adamw_tensor(W, g, m, v), B.make_adamw_tensor(z(512), g, z(512), z(512))])   # a gradient may be shared
    for kw in (dict(step=z(1)), dict(step=z(2, dtype=torch.int64)), dict(step=1, grad_mul=z(2))):
        refused(lambda: B.adamw_step_batched([a], **kw))


@pytest.fixture
def no_launch(monkeypatch, on_cuda):
    """Calls end where the library's would begin, with success; their arguments are kept."""
    made = []
    monkeypatch.setattr(B, "_call", lambda name: lambda *a: made.append((name, a)) or B.MO_OK)
    return on_cuda, made


@pytest.mark.parametrize("gate_shape,rows_per_gate", [((8,), None), ((1, 8), None), ((8,), 4), ((3, 8), 4), ((0, 8), 4)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_without_rows_the_gradient_of_a_gate_is_zero(no_launch, gate_shape, rows_per_gate, accumulate):
    z, made = no_launch
    x, gate, dgate = z(0, 8), z(*gate_shape), z(*gate_shape) + 3
    B.block_norm_grad(x, x, x, None, z(0, 8), z(256, dtype=torch.uint8), gate=gate, dgate=dgate, rows_per_gate=rows_per_gate,
                      accumulate=accumulate)
    assert len(made) == 1 and bool((dgate == (3 if accumulate else 0)).all())


def test_an_empty_batch_may_have_a_gate_of_no_rows(no_launch):
    """One gate for each sequence, and no sequences."""
    z, made = no_launch
    x, gate = z(0, 8), z(0, 8)
    B.block_norm(x, x, None, gate=gate)
    B.block_norm_grad(x, x, x, None, z(0, 8), z(256, dtype=torch.uint8), gate=gate, dgate=z(0, 8))
    assert [name for name, _ in made] == ["block_norm", "block_norm_grad"]
    refused(lambda: B.block_norm(z(4, 8), z(4, 8), None, gate=gate))
    assert len(made) == 2


def test_adamw_list_refuses_a_gradient_that_another_tensor_s_step_writes(on_cuda):
    z = on_cuda
    mine = lambda: [z(512) for _ in range(4)]  # noqa: E731
    (W, g, m, v), (W2, g2, m2, v2) = mine(), mine()
    make = B.make_adamw_tensor
    for k in (W, m, v):
        refused(lambda: B.adamw_tensors([make(W, g, m, v), make(W2, k, m2, v2)]))
        refused(lambda: B.adamw_tensors([make(W2, k, m2, v2), make(W, g, m, v)]))
    refused(lambda: B.adamw_tensors([make(W, W, m, v)]))
    whole = z(2000)
    for at in (0, 1, 511, 1000, 1022):                   # of the gradient's 512; W has 511 .. 1022
        t = [make(whole[511:1023], g, m, v), make(W2, whole[at: at + 512], m2, v2)]
        refused(lambda: B.adamw_tensors(t)) if at else B.adamw_tensors([make(whole[512:1024], g, m, v), t[1]])
    B.adamw_tensors([make(whole[511:1023], g, m, v), make(W2, whole[1023:1535], m2, v2)])
    s = z(4)
    e, f = (z(512, dtype=torch.float8_e4m3fn) for _ in range(2))
    refused(lambda: B.adamw_tensors([make(W, g, e, f, s[:2], s[2:]), make(z(2), s[1:3], z(2), z(2))]))
    # gradients that share memory among themselves, a long one over short ones
    B.adamw_tensors([make(W, whole[:512], m, v), make(W2, whole[100:612], m2, v2), make(z(2000), whole, z(2000), z(2000))])
    refused(lambda: B.adamw_tensors([make(z(2000), whole, z(2000), z(2000)), make(W, whole[:5].new_zeros(512), m, v),
                                     make(whole[1990:], z(10), z(10), z(10))]))


def test_adamw_batch_refuses_an_eps_beyond_its_division(lib):
    for eps in (2.0 ** 125 * 1.0001, 2e38, float("inf"), float("nan")):
        assert adam(lib, cfg=dict(eps=eps)) == INV, eps
    assert adam(lib, cfg=dict(eps=2.0 ** 125), numel=0, W=None, g=None, m=None, v=None) == B.MO_OK
