"""AdamW over many tensors.  The states (float32, or e4m3 codes and scales) equal the
oracle's float32 operations bit for bit, dithered ones too.  The weights: with u =
2^-24, the move carries under 16 roundings (bias corrections, root, division, products), W
two and the subtraction one, and the rounding to W's type."""
import numpy as np
import pytest
import torch

import matrix_optimizers_gb300 as mo
from oracle import adamw as oa
from oracle import blocks as ob
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
U = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
u = 2.0 ** -24


def _np(t):
    return t.detach().float().cpu().numpy()


class Param:
    """One tensor with its states, at an offset from an aligned address."""

    def __init__(self, rng, n, w=F32, g=F32, state=F32, shift=0, lr=1e-3, decay=0.1, zero=False):
        def put(a, dtype):
            buf = torch.zeros(n + shift + 8, dtype=dtype, device=dev())
            buf[shift: shift + n].copy_(torch.from_numpy(a.astype(np.float32)).to(dtype))
            return buf[shift: shift + n]

        self.n, self.state, self.lr, self.decay = n, state, lr, decay
        self.W, self.g = put(rng.standard_normal(n), w), put(0.01 * rng.standard_normal(n), g)
        m = 0.003 * rng.standard_normal(n) * (not zero)
        r = 0.01 * np.abs(rng.standard_normal(n)) * (not zero)
        if state == F32:
            self.m, self.v, self.scales = put(m, F32), put(r * r, F32), {}
        else:
            self.scales, codes = {}, {}
            for name, x in (("m", m), ("v", r)):
                c, sc = ob.quantise(x.astype(np.float32))
                buf = torch.zeros(n + shift + 8, dtype=torch.uint8, device=dev())
                buf[shift: shift + n].copy_(torch.from_numpy(c))
                codes[name] = buf[shift: shift + n].view(E4M3)
                self.scales[name + "_scale"] = torch.from_numpy(sc).to(dev())
            self.m, self.v = codes["m"], codes["v"]

    def make(self):
        return mo.make_adamw_tensor(self.W, self.g, self.m, self.v, lr=self.lr, weight_decay=self.decay, **self.scales)

    def copy(self):
        c = {"W": _np(self.W).copy(), "g": _np(self.g).copy()}
        if self.state == F32:
            c["m"], c["v"] = _np(self.m).copy(), _np(self.v).copy()
        else:
            for k in "mv":
                t = getattr(self, k).view(torch.uint8).cpu().numpy()
                c[k] = ob.dequantise(t, self.scales[k + "_scale"].cpu().numpy())
            c["v"] = (c["v"] * c["v"]).astype(np.float32)
        return c


def _check(p, before, index, step, grad_scale=1.0, seed=None, b1=0.9, b2=0.95, eps=1e-8):
    m, v = ob.adamw_states(before["g"], before["m"], before["v"], b1, b2, grad_scale)
    W, move = ob.adamw_weights(before["W"], m, v, step, p.lr, b1, b2, eps, p.decay)
    got = _np(p.W).astype(np.float64)
    tol = 16 * u * move + 4 * u * np.abs(before["W"])
    assert np.all(np.abs(got - W) <= tol + U[p.W.dtype] * 1.01 * (np.abs(W) + tol))
    if p.state == F32:
        assert np.array_equal(_np(p.m), m, equal_nan=True) and np.array_equal(_np(p.v), v, equal_nan=True)
        return
    bits = (None, None) if seed is None else ob.dither_bits(seed, step, index, p.n)
    for name, x, b, least in (("m", m, bits[0], False), ("v", np.sqrt(v), bits[1], True)):
        codes, scale = ob.quantise(x, b, least)
        assert np.array_equal(p.scales[name + "_scale"].cpu().numpy(), scale, equal_nan=True), name
        assert np.array_equal(getattr(p, name).view(torch.uint8).cpu().numpy(), codes), name


SIZES = [1, 7, 8, 255, 256, 257, 2047, 2048, 2049, 5000, 40000]


@pytest.mark.parametrize("w,g", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("state,seed", [(F32, None), (E4M3, None), (E4M3, 12345)])
@pytest.mark.parametrize("shift", [0, 3])
def test_sizes_and_types(w, g, state, seed, shift):
    rng = np.random.default_rng(len(SIZES))
    ps = [Param(rng, n, w, g, state, shift, lr=1e-3 * (1 + i), decay=0.1 * (i % 3)) for i, n in enumerate(SIZES)]
    tensors = mo.adamw_tensors([p.make() for p in ps])
    for step in (1, 2, 3):
        before = [p.copy() for p in ps]
        mo.adamw_step_batched(tensors, step, grad_scale=0.7, seed=seed)
        for i, p in enumerate(ps):
            _check(p, before[i], i, step, np.float32(0.7), seed)


@pytest.mark.parametrize("count", [1, 8, 9, 64, 65, 320, 321, 700])
def test_many_tensors_of_mixed_kinds(count):
    rng = np.random.default_rng(count)
    ps = [Param(rng, int(rng.integers(1, 900)), (F32, BF16)[i % 2], (F32, BF16)[i // 2 % 2], (F32, E4M3)[i % 3 == 0],
                i % 5 if i % 7 == 0 else 0, lr=1e-3, decay=0.0) for i in range(count)]
    empty = mo.make_adamw_tensor(*[torch.zeros(0, device=dev())] * 4)
    tensors = [empty] + [p.make() for p in ps] + [empty]
    before = [p.copy() for p in ps]
    mo.adamw_step_batched(tensors, 5, beta1=0.8, beta2=0.99, eps=1e-6, seed=3)
    for i, p in enumerate(ps):
        _check(p, before[i], i + 1, 5, seed=3, b1=0.8, b2=0.99, eps=1e-6)


def test_neighbours_are_left_alone():
    for state in (F32, E4M3):
        buf = {k: torch.full((600,), 3.0, device=dev()).to(F32 if k in "Wg" else state) for k in ("W", "g", "m", "v")}
        scales = [torch.full((5,), 9.0, device=dev()) for _ in range(2)]
        kw = dict(m_scale=scales[0][1:3], v_scale=scales[1][1:3]) if state == E4M3 else {}
        mo.adamw_step_batched([mo.make_adamw_tensor(*[buf[k][100:401] for k in ("W", "g", "m", "v")], **kw)], 1)
        for k in ("W", "m", "v"):
            t = buf[k].float()
            assert bool((t[:100] == 3).all()) and bool((t[401:] == 3).all())
            assert k == "m" or bool((t[100:401] != 3).all())         # (0.9 * 3 + 0.1 * 3 stays 3)
        if state == E4M3:
            for t in scales:
                assert bool((t[[0, 3, 4]] == 9).all()) and bool((t[1:3] != 9).all())


def test_blocks_of_zeros_tiny_values_and_values_that_are_not_finite():
    rng = np.random.default_rng(1)
    p = Param(rng, 256 * 6, state=E4M3, zero=True)
    g = np.zeros(256 * 6, np.float32)
    g[256:512] = 1e-38 * rng.standard_normal(256)               # m below the smallest scale, sqrt(v) not
    g[512], g[1024 + 7], g[1280:1536] = np.inf, np.nan, 1e-30
    p.g.copy_(torch.from_numpy(g))
    before = p.copy()
    mo.adamw_step_batched([p.make()], 1)
    m, v = ob.adamw_states(before["g"], before["m"], before["v"], 0.9, 0.95, 1.0)
    for name, x, least in (("m", m, False), ("v", np.sqrt(v), True)):
        codes, scale = ob.quantise(x, None, least)
        assert np.array_equal(p.scales[name + "_scale"].cpu().numpy(), scale, equal_nan=True)
        assert np.array_equal(getattr(p, name).view(torch.uint8).cpu().numpy(), codes)
    nan = np.isnan(p.scales["m_scale"].cpu().numpy())
    assert nan.tolist() == [False, False, True, False, True, False]
    W = _np(p.W)
    assert np.isnan(W[[512, 1031]]).all() and np.isfinite(np.delete(W, [512, 1031])).all()


def test_float32_states_agree_with_the_tail_s_oracle_over_steps():
    """20 steps in float32 against float64: each step adds at most 4 roundings to a state,
    which decays by beta, and 16 to the move: 20 * 24 u of the moves' sum."""
    rng = np.random.default_rng(2)
    p = Param(rng, 3000, zero=True)
    W, m, v = _np(p.W).astype(np.float64), np.zeros(3000), np.zeros(3000)
    W0 = W.copy()
    f = lambda x: float(np.float32(x))  # noqa: E731
    for step in range(1, 21):
        p.g.copy_(torch.from_numpy(0.01 * rng.standard_normal(3000)).float())
        mo.adamw_step_batched([p.make()], step)
        W, m, v = oa.adamw_step(W, _np(p.g), m, v, step, f(1e-3), f(0.9), f(0.95), f(1e-8), f(0.1))
    assert np.abs(_np(p.W) - W).max() <= 480 * u * np.abs(W - W0).max() + 40 * u * np.abs(W).max()


def test_step_and_gradient_factor_from_the_device_also_in_a_replayed_graph():
    rng = np.random.default_rng(3)
    for state, seed in ((F32, None), (E4M3, 8)):
        a, b = Param(np.random.default_rng(4), 3000, state=state), Param(np.random.default_rng(4), 3000, state=state)
        step, mul = torch.zeros((), dtype=torch.int64, device=dev()), torch.full((), 0.5, device=dev())
        ta, tb = mo.adamw_tensors([a.make()]), mo.adamw_tensors([b.make()])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step.add_(1)
            mo.adamw_step_batched(ta, step, grad_scale=0.5, grad_mul=mul, seed=seed)
        for k in range(1, 4):
            mul.fill_(0.5 / k)
            graph.replay()
            mo.adamw_step_batched(tb, k, grad_scale=float(np.float32(0.5) * np.float32(0.5 / k)), seed=seed)
        torch.cuda.synchronize()
        for x, y in ((a.m, b.m), (a.v, b.v), *zip(a.scales.values(), b.scales.values())):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        # the bias corrections come from two implementations of pow: one rounding to float32 apart at most
        assert float((a.W - b.W).abs().max()) <= 4 * u * float(b.W.abs().max())
    del rng


def test_a_list_and_another_stream_give_the_same():
    a, b = (Param(np.random.default_rng(5), 70000, state=E4M3) for _ in range(2))
    mo.adamw_step_batched([a.make()], 4, seed=1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    mo.adamw_step_batched(mo.adamw_tensors([b.make()]), 4, seed=1, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a.W, b.W) and torch.equal(a.m.view(torch.uint8), b.m.view(torch.uint8))


@pytest.mark.parametrize("w", [F32, BF16])
@pytest.mark.parametrize("eps", [1e-30, 1e-38, 1e-40, 1e-44, 1e32, 2.0 ** 125])
def test_an_eps_of_any_size(eps, w):
    """Gradients of 1e-25 leave float32 roots of v of 0, so that eps alone divides their m of 1e-26; beside
    them gradients that hide the smallest eps, and with the largest the moves are small ones."""
    for state in (F32, E4M3):
        p = Param(np.random.default_rng(6), 3 * 256, w=w, state=state, lr=1e-10 if eps < 1 else 1e32, decay=0.0, zero=True)
        g = 0.01 * np.random.default_rng(7).standard_normal(3 * 256).astype(np.float32)
        g[:256] *= 1e-23
        p.g.copy_(torch.from_numpy(g))
        before = p.copy()
        mo.adamw_step_batched([p.make()], 3, eps=eps)
        _check(p, before, 0, 3, eps=eps)


def test_a_rate_and_a_decay_changed_in_the_list_count_from_the_next_step():
    rng = np.random.default_rng(9)
    ps = [Param(rng, 700, state=s) for s in (F32, E4M3)]
    tensors = mo.adamw_tensors([p.make() for p in ps])
    for step, (lr, decay) in enumerate(((1e-3, 0.1), (4e-3, 0.0), (0.0, 0.2)), 1):
        for i, p in enumerate(ps):
            p.lr, p.decay = lr, decay
            tensors.array[i].lr, tensors.array[i].weight_decay = lr, decay
        before = [p.copy() for p in ps]
        mo.adamw_step_batched(tensors, step)
        for i, p in enumerate(ps):
            _check(p, before[i], i, step)
