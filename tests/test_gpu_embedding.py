"""Embedding lookup and gradient against the float64 oracle.

Tolerances, per element: u = 2^-24 for a float32 result's rounding and 2^-8 for
bf16's (to nearest).  The lookup rounds once in float32 (the product) and once
to the output.  A gradient sums c terms in float32: its error is at most
(c + 2) 2^-24 times the sum of the terms' magnitudes, plus the output's rounding."""
import numpy as np
import pytest
import torch

import matrix_optimizers_gb300 as mo
from oracle import training as ot
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def _f64(t):
    return t.detach().double().cpu().numpy()


def _rand(rng, shape, dtype, ld=None, shift=0):
    """A device tensor; with ld a column slice of a wider buffer, with shift
    starting that many elements after an aligned address (NaN around it)."""
    rows, cols = shape
    ld = ld or cols
    buf = torch.full((rows * ld + shift + 8,), float("nan"), dtype=dtype, device=dev())
    view = buf[shift: shift + rows * ld].view(rows, ld)[:, :cols]
    view.copy_(torch.from_numpy(rng.standard_normal(shape)).to(dtype))
    return view


@pytest.mark.parametrize("w_dtype", [F32, BF16])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("n,vocab,dim,ld,shift,id_dtype", [
    (1, 1, 1, None, 0, torch.int64), (1, 50, 768, None, 0, torch.int32), (37, 100, 64, None, 0, torch.int64),
    (130, 33, 515, None, 0, torch.int32), (64, 40, 96, 104, 0, torch.int64), (65, 40, 95, 99, 3, torch.int64),
    (2000, 500, 1024, None, 0, torch.int32)])
def test_lookup(n, vocab, dim, ld, shift, id_dtype, w_dtype, out_dtype):
    rng = np.random.default_rng(n + dim)
    W = _rand(rng, (vocab, dim), w_dtype, ld, shift)
    ids = rng.integers(-2, vocab + 2, n)
    ids[0] = vocab - 1
    out = _rand(rng, (n, dim), out_dtype, ld, shift)
    mo.embedding_lookup(W, torch.from_numpy(ids).to(id_dtype).to(dev()), out, scale=1.37)
    want = ot.embedding_lookup(_f64(W), ids, np.float32(1.37))
    got = _f64(out)
    assert np.all(np.abs(got - want) <= (2.0 ** -23 + U[out_dtype]) * 1.01 * np.abs(want))
    assert np.all(got[(ids < 0) | (ids >= vocab)] == 0)


def test_lookup_leaves_the_rest_of_a_strided_output_alone_and_pads_with_plus_zero():
    buf = torch.full((3, 40), 7.0, device=dev())
    W = torch.full((4, 33), float("inf"), device=dev())
    mo.embedding_lookup(W, torch.tensor([-1, 9, 2**40], device=dev()), buf[:, :33], scale=-1.0)
    assert torch.all(buf[:, :33].view(torch.int32) == 0) and torch.all(buf[:, 33:] == 7.0)


def _check_grad(dY, ids, vocab, dW, scale, start=None):
    x = _f64(dY)
    want = ot.embedding_grad(x, ids, vocab, np.float32(scale), start)
    mag = ot.embedding_grad(np.abs(x), ids, vocab, scale, None if start is None else np.abs(start))
    count = np.bincount(np.asarray(ids)[(ids >= 0) & (ids < vocab)], minlength=vocab)[:, None]
    got = _f64(dW)
    tol = (count + 2) * 2.0 ** -24 * mag + U[dW.dtype] * 1.01 * np.abs(want)
    if dW.dtype == BF16:
        tol += 2.0 ** -8 * (count + 2) * 2.0 ** -24 * mag
    assert np.all(np.abs(got - want) <= tol)


GRAD_CASES = [
    (1, 1, 1, None, 0, "one"), (5, 3, 8, None, 0, "uniform"), (64, 1000, 64, None, 0, "uniform"),
    (777, 503, 515, None, 0, "zipf"), (129, 40, 95, 99, 3, "uniform"), (300, 700, 128, 136, 0, "zipf"),
    (3000, 257, 72, None, 0, "one"), (5000, 2000, 1032, None, 0, "zipf"), (1025, 512, 16, None, 0, "sorted"),
    (700, 511, 24, None, 0, "dropped"), (20000, 300000, 8, None, 0, "uniform"),
    (65536, 1023, 4, None, 0, "zipf"), (70001, 1500, 4, None, 0, "zipf"), (140001, 1500, 4, None, 0, "zipf"), (8193, 600, 12, None, 0, "one")]


def _ids(rng, n, vocab, how):
    if how == "one":
        return np.full(n, vocab - 1)
    if how == "sorted":
        return np.sort(rng.integers(0, vocab, n))
    if how == "dropped":
        return np.where(rng.random(n) < 0.9, -1, rng.integers(0, vocab + 3, n))
    if how == "zipf":
        return np.minimum((np.exp(rng.random(n) * np.log(vocab + 1.0)) - 1).astype(np.int64), vocab - 1)
    return rng.integers(0, vocab, n)


@pytest.mark.parametrize("dy_dtype,dw_dtype", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("n,vocab,dim,ld,shift,how", GRAD_CASES)
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient(n, vocab, dim, ld, shift, how, dy_dtype, dw_dtype, accumulate):
    rng = np.random.default_rng(n + vocab)
    ids = _ids(rng, n, vocab, how)
    dY = _rand(rng, (n, dim), dy_dtype, ld, shift)
    dW = _rand(rng, (vocab, dim), dw_dtype, ld, shift)
    start = _f64(dW) if accumulate else None
    if not accumulate:
        dW.fill_(float("nan"))
    ws = torch.full((mo.embedding_grad_workspace_bytes(n, vocab, dim),), 255, dtype=torch.uint8, device=dev())
    t = torch.from_numpy(ids).to(dev())
    mo.embedding_grad(dY, t if n % 2 else t.int(), dW, ws, scale=0.75, accumulate=accumulate)
    _check_grad(dY, ids, vocab, dW, 0.75, start)


def test_gradient_is_the_same_bit_for_bit_and_ignores_dropped_rows():
    rng = np.random.default_rng(3)
    n, vocab, dim = 4096, 300, 264
    ids = _ids(rng, n, vocab, "zipf")
    ids[::5] = -1
    dY = _rand(rng, (n, dim), BF16)
    dY[::5] = float("nan")
    t = torch.from_numpy(ids).to(dev())
    ws = torch.empty(mo.embedding_grad_workspace_bytes(n, vocab, dim), dtype=torch.uint8, device=dev())
    out = [torch.empty((vocab, dim), device=dev()) for _ in range(3)]
    for o in out:
        mo.embedding_grad(dY, t, o, ws)
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2]) and bool(torch.isfinite(out[0]).all())


@pytest.mark.parametrize("n", [31, 32, 33, 511, 513, 2049, 4095, 4096, 4097])
def test_gradient_at_the_ends_of_the_sorts(n):
    rng = np.random.default_rng(n)
    ids = _ids(rng, n, 90, "zipf")
    ids[rng.random(n) < 0.1] = -1
    dY = _rand(rng, (n, 12), F32)
    dW = torch.full((90, 12), float("nan"), device=dev())
    ws = torch.full((mo.embedding_grad_workspace_bytes(n, 90, 12),), 255, dtype=torch.uint8, device=dev())
    mo.embedding_grad(dY, torch.from_numpy(ids).to(dev()), dW, ws)
    _check_grad(dY, ids, 90, dW, 1.0)


@pytest.mark.parametrize("vocab", [60, 300000])           # sorted in one launch, in passes
@pytest.mark.parametrize("dim,dtype", [(20, F32), (1100, BF16), (1031, F32)])
def test_gradient_of_runs_that_end_at_and_around_chunks(vocab, dim, dtype):
    """Runs of 1 to 70 chunks whose ends fall on, before and after a chunk's, twice with one workspace."""
    rng = np.random.default_rng(dim)
    lengths = [3, 8, 8, 16, 5, 1, 2, 64, 63, 65, 128, 256, 264, 255, 31 * 64, 33 * 64 + 1, 7, 9, 560, 1, 1, 70]
    ws = None
    for order in (lengths, lengths[::-1]):
        ids = np.repeat(np.arange(len(order)), order)
        rng.shuffle(ids)
        n = len(ids)
        dY = _rand(rng, (n, dim), dtype)
        dW = _rand(rng, (vocab, dim), F32)
        start = _f64(dW[:64])
        if ws is None:
            ws = torch.full((mo.embedding_grad_workspace_bytes(n, vocab, dim),), 255, dtype=torch.uint8, device=dev())
        mo.embedding_grad(dY, torch.from_numpy(ids).to(dev()), dW, ws, scale=0.5, accumulate=True)
        _check_grad(dY, ids, min(vocab, 64), dW[:64], 0.5, start)


def test_gradient_of_no_positions_is_zero_and_runs_on_another_stream():
    dW = torch.ones((70, 33), device=dev())
    ws = torch.empty(mo.embedding_grad_workspace_bytes(0, 70, 33), dtype=torch.uint8, device=dev())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mo.embedding_grad(torch.empty((0, 33), device=dev()), torch.empty(0, dtype=torch.int64, device=dev()), dW, ws,
                      stream=s)
    s.synchronize()
    assert torch.all(dW == 0)
    dW.fill_(2.0)
    mo.embedding_grad(torch.empty((0, 33), device=dev()), torch.empty(0, dtype=torch.int64, device=dev()), dW, ws,
                      accumulate=True)
    assert torch.all(dW == 2.0)


def test_gradient_matches_differences_of_the_lookup():
    """<lookup(W + hD) - lookup(W - hD), dY> / 2h = <gradient, D>; the map is linear,
    so h = 1/2 has only rounding error: 4096 x 2 float32 products."""
    rng = np.random.default_rng(5)
    W, D, dY = (_rand(rng, s, F32) for s in ((50, 64), (50, 64), (64, 64)))
    ids = torch.from_numpy(rng.integers(0, 50, 64)).to(dev())
    up, down, g = torch.empty_like(dY), torch.empty_like(dY), torch.empty_like(W)
    mo.embedding_lookup(W + 0.5 * D, ids, up, scale=3.0)
    mo.embedding_lookup(W - 0.5 * D, ids, down, scale=3.0)
    ws = torch.empty(mo.embedding_grad_workspace_bytes(64, 50, 64), dtype=torch.uint8, device=dev())
    mo.embedding_grad(dY, ids, g, ws, scale=3.0)
    diff = float(((up.double() - down.double()) * dY.double()).sum())
    terms = float((up.double().abs() * dY.double().abs()).sum() + (down.double().abs() * dY.double().abs()).sum())
    assert abs(diff - float((g.double() * D.double()).sum())) <= 16 * 2.0 ** -24 * terms


def test_gradient_feeds_the_adamw_tail():
    rng = np.random.default_rng(6)
    vocab, dim = 40, 24
    W, dY = _rand(rng, (vocab, dim), F32).contiguous(), _rand(rng, (100, dim), BF16)
    ids = torch.from_numpy(rng.integers(0, vocab, 100)).to(dev())
    g, m, v = (torch.zeros_like(W) for _ in range(3))
    ws = torch.empty(mo.embedding_grad_workspace_bytes(100, vocab, dim), dtype=torch.uint8, device=dev())
    mo.embedding_grad(dY, ids, g, ws)
    want = W.double() - 1e-2 * g.double() / (g.double().abs() + 1e-8)      # AdamW's first step
    mo.muon_step_batched([], mo.make_cfg(), None, tail=mo.make_tail(W, g, m, v, 1, lr=1e-2))
    assert torch.allclose(W.double(), want, atol=1e-6)


def test_single_rows_and_refused_layouts():
    W, out = torch.randn((1, 13), device=dev()), torch.empty((1, 13), device=dev())
    mo.embedding_lookup(W, torch.zeros(1, dtype=torch.int64, device=dev()), out, scale=2.0)
    assert torch.equal(out, 2 * W)
    ids = torch.zeros(4, dtype=torch.int64, device=dev())
    ws = torch.empty(mo.embedding_grad_workspace_bytes(4, 1, 13), dtype=torch.uint8, device=dev())
    for bad in (out.expand(4, 13), torch.zeros((13, 4), device=dev()).T):
        with pytest.raises(mo.MoError):
            mo.embedding_lookup(W, ids, bad)
        with pytest.raises(mo.MoError):
            mo.embedding_grad(bad, ids, W, ws)
    with pytest.raises(mo.MoError):
        mo.embedding_lookup(W, ids[::2], torch.empty((2, 13), device=dev()))
