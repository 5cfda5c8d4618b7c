"""Matrix products grouped by expert against the float64 oracle.

Tolerances, per element: bf16 products are exact in float32 and a float32 sum
of d terms is off by at most d 2^-23 times the sum of their magnitudes (a
truncating accumulator loses up to one unit in the last place per addition);
the output's rounding adds 2^-8 (bf16) or 2^-24 of the result."""
import numpy as np
import pytest
import torch

import matrix_optimizers_gb300 as mo
from matrix_optimizers_gb300 import _binding as B
from oracle import training as ot
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[-1, 0, 1, 2], ids=["auto", "single", "pair", "few"], autouse=True)
def geometry(request):
    """Every test runs with the size-chosen tile geometry and with each of the others."""
    prev = B.mo_debug_set_expert_shape(request.param)
    yield request.param
    B.mo_debug_set_expert_shape(prev)

F32, BF16 = torch.float32, torch.bfloat16
U = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def _f64(t):
    return t.detach().double().cpu().numpy()


def _pad8(c):
    return (c + 7) // 8 * 8


def _mat(rng, rows, cols, ld=None, scale=1.0):
    ld = ld or _pad8(cols)
    buf = torch.full((max(rows, 1), ld), float("nan"), dtype=BF16, device=dev())
    buf[:rows, :cols] = torch.from_numpy(scale * rng.standard_normal((rows, cols))).to(BF16).to(dev())
    return buf[:rows, :cols]


def _stack(rng, E, rows, cols, dtype=BF16, extra=0, fill=None):
    ld = _pad8(cols) + extra
    buf = torch.full((E, rows + (1 if extra else 0), ld), float("nan"), dtype=dtype, device=dev())
    v = buf[:, :rows, :cols]
    v.copy_(torch.from_numpy(rng.standard_normal((E, rows, cols))).to(dtype) if fill is None
            else torch.full((E, rows, cols), fill, dtype=dtype))
    return v


def _ws(rows, n, k, E):
    return torch.zeros(mo.expert_linear_workspace_bytes(rows, n, k, E), dtype=torch.uint8, device=dev())


def _offsets(sizes, first=0):
    return np.concatenate([[first], first + np.cumsum(sizes)]).astype(np.int32)


def _assert_close(got_t, want, mag, depth):
    got = _f64(got_t)
    u = U[got_t.dtype]
    tol = (depth + 2) * 2.0 ** -23 * mag * (1 + u) + u * 1.01 * np.abs(want)
    assert np.all(np.isfinite(got))
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


CASES = [
    # sizes, rows before the first / after the last expert, n, k, extra columns of the leading dimensions
    ([1], 0, 0, 1, 1, 0), ([1], 0, 0, 64, 64, 0), ([5], 0, 0, 24, 40, 0), ([0, 1, 0], 0, 0, 136, 72, 0),
    ([3, 0, 130, 1, 17, 0], 0, 0, 200, 136, 8), ([128, 256, 64], 0, 0, 256, 128, 0),
    ([300], 0, 0, 520, 264, 0), ([257, 255, 1, 513], 3, 5, 384, 200, 16), ([0, 0, 0], 0, 7, 72, 40, 0),
    ([40] * 20, 0, 0, 104, 296, 0), ([33, 90], 2, 0, 77, 129, 0), ([1000, 3], 0, 0, 129, 513, 8),
    ([0] * 70 + [9], 0, 0, 264, 64, 0)]


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("sizes,before,after,n,k,extra", CASES)
def test_forward_and_gradients(sizes, before, after, n, k, extra, out_dtype):
    rng = np.random.default_rng(n + k)
    E, off = len(sizes), _offsets(sizes, before)
    R = int(off[-1]) + after
    X, dY = _mat(rng, R, k, _pad8(k) + extra), _mat(rng, R, n, _pad8(n) + extra)
    W = _stack(rng, E, n, k, extra=extra)
    o = torch.from_numpy(off).to(dev())
    ws = _ws(R, n, k, E)
    pad = 8
    Y = torch.full((R, _pad8(n) + pad), 3.0, dtype=out_dtype, device=dev())
    dX = torch.full((R, _pad8(k) + pad), 3.0, dtype=out_dtype, device=dev())
    mo.expert_linear(X, W, o, Y[:, :n], ws)
    mo.expert_linear_dgrad(dY, W, o, dX[:, :k], ws)
    dW = _stack(rng, E, n, k, dtype=out_dtype, extra=extra, fill=7.0)
    mo.expert_linear_wgrad(dY, X, o, dW, ws)
    x, dy, w = _f64(X), _f64(dY), _f64(W)
    _assert_close(Y[:, :n], ot.expert_linear(x, w, off), ot.expert_linear(np.abs(x), np.abs(w), off), k)
    _assert_close(dX[:, :k], ot.expert_linear_dgrad(dy, w, off),
                  ot.expert_linear_dgrad(np.abs(dy), np.abs(w), off), n)
    _assert_close(dW, ot.expert_linear_wgrad(dy, x, off), ot.expert_linear_wgrad(np.abs(dy), np.abs(x), off),
                  max(sizes))
    assert torch.all(Y[:, n:] == 3.0) and torch.all(dX[:, k:] == 3.0)
    out = np.ones(R, bool)
    out[off[0]:off[-1]] = False
    assert np.all(_f64(Y[:, :n])[out] == 0) and np.all(_f64(dX[:, :k])[out] == 0)
    assert mo.mo_check_device_status(ws) == 0


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("sizes", [[7, 0, 100], [600, 1]])
def test_weight_gradient_accumulates(sizes, out_dtype):
    rng = np.random.default_rng(4)
    E, off, n, k = len(sizes), _offsets(sizes), 72, 136
    R = int(off[-1])
    X, dY = _mat(rng, R, k), _mat(rng, R, n)
    dW = _stack(rng, E, n, k, dtype=out_dtype)
    start = _f64(dW)
    o, ws = torch.from_numpy(off).to(dev()), _ws(R, n, k, E)
    mo.expert_linear_wgrad(dY, X, o, dW, ws, accumulate=True)
    x, dy = _f64(X), _f64(dY)
    _assert_close(dW, ot.expert_linear_wgrad(dy, x, off, start),
                  ot.expert_linear_wgrad(np.abs(dy), np.abs(x), off, np.abs(start)), max(sizes))
    assert np.array_equal(_f64(dW)[np.array(sizes) == 0], start[np.array(sizes) == 0])


def test_values_of_one_expert_do_not_reach_another():
    """Infinities and NaN in the rows (or weights) of one expert stay in its outputs,
    also where a tile's end holds the next expert's rows."""
    rng = np.random.default_rng(8)
    sizes, n, k = [37, 20, 75], 136, 72
    E, off = 3, _offsets(sizes)
    R = int(off[-1])
    X, dY, W = _mat(rng, R, k), _mat(rng, R, n), _stack(rng, E, n, k)
    X[37:57] = float("nan")
    dY[37:57] = float("inf")
    W[1] = float("nan")
    o, ws = torch.from_numpy(off).to(dev()), _ws(R, n, k, E)
    Y, dX = torch.empty((R, n), dtype=BF16, device=dev()), torch.empty((R, k), dtype=BF16, device=dev())
    dW = torch.empty((E, n, k), device=dev())
    mo.expert_linear(X, W, o, Y, ws)
    mo.expert_linear_dgrad(dY, W, o, dX, ws)
    mo.expert_linear_wgrad(dY, X, o, dW, ws)
    clean = np.r_[0:37, 57:132]
    x, dy, w = _f64(X), _f64(dY), _f64(W)
    x[37:57], dy[37:57], w[1] = 0, 0, 0
    _assert_close(Y[clean], ot.expert_linear(x, w, off)[clean], ot.expert_linear(np.abs(x), np.abs(w), off)[clean], k)
    _assert_close(dX[clean], ot.expert_linear_dgrad(dy, w, off)[clean],
                  ot.expert_linear_dgrad(np.abs(dy), np.abs(w), off)[clean], n)
    _assert_close(dW[[0, 2]], ot.expert_linear_wgrad(dy, x, off)[[0, 2]],
                  ot.expert_linear_wgrad(np.abs(dy), np.abs(x), off)[[0, 2]], 75)
    assert bool(torch.isnan(Y[37:57]).all()) and bool(torch.isnan(dW[1]).all())


def test_results_repeat_bit_for_bit_and_on_another_stream():
    rng = np.random.default_rng(9)
    sizes, n, k = [700, 0, 301, 64, 1500], 392, 264
    off = _offsets(sizes)
    R, E = int(off[-1]), len(sizes)
    X, dY, W = _mat(rng, R, k), _mat(rng, R, n), _stack(rng, E, n, k)
    o, ws = torch.from_numpy(off).to(dev()), _ws(R, n, k, E)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    runs = []
    for _ in range(3):
        Y, dX, dW = (torch.empty(s, device=dev()) for s in ((R, n), (R, k), (E, n, k)))
        torch.cuda.synchronize()
        mo.expert_linear(X, W, o, Y, ws, stream=st)
        mo.expert_linear_dgrad(dY, W, o, dX, ws, stream=st)
        mo.expert_linear_wgrad(dY, X, o, dW, ws, stream=st)
        st.synchronize()
        runs.append((Y, dX, dW))
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(r, runs[0]))


def test_offsets_outside_the_rows_stay_in_range():
    """Wrong offsets give wrong numbers, not an access out of range (rows are held to [0, rows])."""
    rng = np.random.default_rng(10)
    R, n, k = 50, 72, 40
    X, dY, W = _mat(rng, R, k), _mat(rng, R, n), _stack(rng, 3, n, k)
    ws = _ws(R, n, k, 3)
    Y, dX = torch.zeros((R, n), device=dev()), torch.zeros((R, k), device=dev())
    dW = torch.zeros((3, n, k), device=dev())
    for off in ([-5, 10, 60, 2**31 - 1], [40, 10, 30, 50], [50, 50, 50, 0]):
        o = torch.tensor(off, dtype=torch.int32, device=dev())
        mo.expert_linear(X, W, o, Y, ws)
        mo.expert_linear_dgrad(dY, W, o, dX, ws)
        mo.expert_linear_wgrad(dY, X, o, dW, ws)
        assert mo.mo_check_device_status(ws) == 0


def test_gradients_match_differences():
    """The product is linear in X and in W: <Y(X + D) - Y(X - D), dY> / 2 = <dX, D>, and
    the same for W, up to the rounding of X +- D (exact here: small integers)."""
    rng = np.random.default_rng(11)
    sizes, n, k = [20, 45], 48, 56
    off = _offsets(sizes)
    R = 65
    ints = lambda *s: torch.from_numpy(rng.integers(-4, 5, s)).to(BF16).to(dev())
    X, DX, W, DW, dY = ints(R, k), ints(R, k), ints(2, n, k), ints(2, n, k), ints(R, n)
    o, ws = torch.from_numpy(off).to(dev()), _ws(R, n, k, 2)
    Y = [torch.empty((R, n), device=dev()) for _ in range(2)]
    dX, dW = torch.empty((R, k), device=dev()), torch.empty((2, n, k), device=dev())
    mo.expert_linear_dgrad(dY, W, o, dX, ws)
    mo.expert_linear_wgrad(dY, X, o, dW, ws)
    for a, b, want in ((X + DX, W, (dX.double() * DX.double()).sum()), (X, W + DW, (dW.double() * DW.double()).sum())):
        c, d = (X - DX, W) if b is W else (X, W - DW)
        mo.expert_linear(a, b, o, Y[0], ws)
        mo.expert_linear(c, d, o, Y[1], ws)
        assert float(((Y[0].double() - Y[1].double()) * dY.double()).sum()) / 2 == float(want)   # integers below 2^24


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("sizes,before,after,n,k", [
    ([4100], 0, 0, 264, 200), ([3], 2, 1, 136, 8200), ([3], 0, 2, 8200, 72), ([5000, 0], 1, 4, 129, 77),
    ([2051, 1], 0, 0, 257, 2056)])
def test_long_sums_with_few_tiles_are_split_and_joined(sizes, before, after, n, k, out_dtype, geometry):
    rng = np.random.default_rng(n * 3 + k)
    E, off = len(sizes), _offsets(sizes, before)
    R = int(off[-1]) + after
    X, dY, W = _mat(rng, R, k), _mat(rng, R, n), _stack(rng, E, n, k)
    o, ws = torch.from_numpy(off).to(dev()), _ws(R, n, k, E)
    if max(n, k, max(sizes)) > 4000:
        assert ws.numel() > 4096                       # room for the parts: some call is split
    Y = torch.full((R, _pad8(n) + 8), 3.0, dtype=out_dtype, device=dev())
    dX = torch.full((R, _pad8(k) + 8), 3.0, dtype=out_dtype, device=dev())
    dW = _stack(rng, E, n, k, dtype=out_dtype, extra=8)
    start = _f64(dW)
    x, dy, w = _f64(X), _f64(dY), _f64(W)
    for _ in range(2):                                 # a second call finds the first one's parts in the workspace
        mo.expert_linear(X, W, o, Y[:, :n], ws)
        mo.expert_linear_dgrad(dY, W, o, dX[:, :k], ws)
    mo.expert_linear_wgrad(dY, X, o, dW, ws, accumulate=True)
    _assert_close(Y[:, :n], ot.expert_linear(x, w, off), ot.expert_linear(np.abs(x), np.abs(w), off), k)
    _assert_close(dX[:, :k], ot.expert_linear_dgrad(dy, w, off),
                  ot.expert_linear_dgrad(np.abs(dy), np.abs(w), off), n)
    _assert_close(dW, ot.expert_linear_wgrad(dy, x, off, start),
                  ot.expert_linear_wgrad(np.abs(dy), np.abs(x), off, np.abs(start)), max(sizes))
    assert torch.all(Y[:, n:] == 3.0) and torch.all(dX[:, k:] == 3.0)
    out = np.ones(R, bool)
    out[off[0]:off[-1]] = False
    assert np.all(_f64(Y[:, :n])[out] == 0) and np.all(_f64(dX[:, :k])[out] == 0)
    assert mo.mo_check_device_status(ws) == 0


def test_a_single_row_of_any_width_and_refused_layouts():
    """One row needs no aligned pitch; a broadcast or misaligned matrix is refused, not misread."""
    rng = np.random.default_rng(12)
    W = _stack(rng, 1, 77, 201)
    X, Y = torch.randn((1, 201), device=dev()).to(BF16), torch.empty((1, 77), device=dev())
    o, ws = torch.tensor([0, 1], dtype=torch.int32, device=dev()), _ws(1, 77, 201, 1)
    mo.expert_linear(X, W, o, Y, ws)
    _assert_close(Y, ot.expert_linear(_f64(X), _f64(W), [0, 1]),
                  ot.expert_linear(np.abs(_f64(X)), np.abs(_f64(W)), [0, 1]), 201)
    o4, Y4 = torch.tensor([0, 4], dtype=torch.int32, device=dev()), torch.empty((4, 80), device=dev())[:, :77]
    for bad, status in ((X.expand(4, 201), B.MO_ERR_INVALID_ARG), (torch.zeros((4, 201), device=dev(), dtype=BF16),
                                                                   B.MO_ERR_ALIGNMENT),
                        (torch.zeros((4, 208), device=dev(), dtype=BF16)[:, 1:202], B.MO_ERR_ALIGNMENT),
                        (torch.zeros((201, 4), device=dev(), dtype=BF16).T, B.MO_ERR_INVALID_ARG),
                        (torch.zeros((4, 208), device=dev())[:, :201], B.MO_ERR_INVALID_ARG)):
        with pytest.raises(B.MoError) as e:
            mo.expert_linear(bad, W, o4, Y4, ws)
        assert e.value.status == status


@pytest.mark.slow
def test_large_sizes_against_float64_on_the_device():
    """Long groups, many tiles: sampled rows and columns."""
    g = torch.Generator(device=dev()).manual_seed(1)
    sizes, n, k = [5000, 0, 1, 2047, 3001], 1544, 2056
    off = _offsets(sizes)
    R, E = int(off[-1]), len(sizes)
    mk = lambda *s: torch.randn(s, generator=g, device=dev()).to(BF16)
    X, dY, W = mk(R, k), mk(R, n), mk(E, n, k)
    o, ws = torch.from_numpy(off).to(dev()), _ws(R, n, k, E)
    Y, dX, dW = (torch.empty(s, device=dev()) for s in ((R, n), (R, k), (E, n, k)))
    mo.expert_linear(X, W, o, Y, ws)
    mo.expert_linear_dgrad(dY, W, o, dX, ws)
    mo.expert_linear_wgrad(dY, X, o, dW, ws)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        x, d, w = X[a:b].double(), dY[a:b].double(), W[e].double()
        for got, want, mag, depth in ((Y[a:b], x @ w.T, x.abs() @ w.abs().T, k), (dX[a:b], d @ w, d.abs() @ w.abs(), n),
                                      (dW[e], d.T @ x, d.abs().T @ x.abs(), max(b - a, 1))):
            tol = (depth + 2) * 2.0 ** -23 * mag + 2.0 ** -24 * want.abs()
            assert bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("k", [12, 8, 100])
@pytest.mark.parametrize("permuted", [False, True])
def test_stacks_of_one_row_matrices(k, permuted):
    """Several experts of one output feature each: a matrix of one row needs no pitch of its own, only
    a stack stride of whole 16 bytes."""
    rng = np.random.default_rng(k)
    off = _offsets([20, 0, 31])
    dY, X = _mat(rng, 51, 1), _mat(rng, 51, k)
    buf = torch.full((3, 1, _pad8(k)) if not permuted else (1, 3, _pad8(k)), 3.0, device=dev())
    if k == 12 and not permuted:
        buf = torch.full((3, 1, 12), 3.0, device=dev())                 # 48 bytes
    dW = (buf.transpose(0, 1) if permuted else buf)[:, :, :k]
    o, ws = torch.from_numpy(off).to(dev()), _ws(51, 1, k, 3)
    mo.expert_linear_wgrad(dY, X, o, dW, ws)
    x, dy = _f64(X), _f64(dY)
    _assert_close(dW, ot.expert_linear_wgrad(dy, x, off), ot.expert_linear_wgrad(np.abs(dy), np.abs(x), off), 31)
    W = torch.from_numpy(rng.standard_normal((1, 3, _pad8(k)))).to(BF16).to(dev()).transpose(0, 1)[:, :, :k]
    Y = torch.empty((51, 8), device=dev())[:, :1]
    mo.expert_linear(X, W, o, Y, ws)
    w = _f64(W)
    _assert_close(Y, ot.expert_linear(x, w, off), ot.expert_linear(np.abs(x), np.abs(w), off), k)
    assert mo.mo_check_device_status(ws) == 0


def test_a_product_over_no_features_is_zero():
    """n == 0: the input's gradient is an empty sum, whatever the empty stack's strides."""
    dX = torch.full((5, 16), 3.0, device=dev())[:, :13]
    o, ws = torch.tensor([0, 2, 5], dtype=torch.int32, device=dev()), _ws(5, 0, 13, 2)
    mo.expert_linear_dgrad(torch.empty((5, 0), dtype=BF16, device=dev()), torch.empty((2, 0, 13), dtype=BF16, device=dev()),
                           o, dX, ws)
    assert torch.all(dX == 0)


@pytest.mark.slow
@pytest.mark.parametrize("mode", ["forward", "dgrad", "wgrad"])
def test_long_bf16_sums_do_not_drift(mode, geometry):
    """The tensor core's accumulator drops bits always towards zero: each 16-term step may
    lose 2^-23 of a sum of positive terms.  Over at most 4096 terms that is 256 x 2^-23, and
    the float32 additions of the pieces (depth / 4096 of them) lose at most 2^-24 each; both
    together bound the mean relative error.  The bf16 roundings, each up to 2^-8 and uniform
    over the results' spread, average out to 2^-8 / sqrt(3 count); five times that is allowed.
    Rows and columns are so many that no geometry splits the sums."""
    g = torch.Generator(device=dev()).manual_seed(3)
    depth, rows, cols, some = 1 << 20, 1024, 2560, 16
    # factors that spread the results evenly over a binade
    fr = torch.exp2(torch.linspace(0, 1, rows + 1, device=dev())[:rows])
    fc = torch.exp2(torch.linspace(0, 1, cols + 1, device=dev())[:cols])

    def pos(f, *shape):
        return torch.rand(shape, generator=g, device=dev()).add_(0.5).mul_(f).to(BF16)

    if mode == "wgrad":                                # dW [rows, cols] = dY^T X
        a, b = pos(fr, depth, rows), pos(fc, depth, cols)
        o, ws = torch.tensor([0, depth], dtype=torch.int32, device=dev()), _ws(depth, rows, cols, 1)
        out = torch.empty((1, rows, cols), dtype=BF16, device=dev())
        mo.expert_linear_wgrad(a, b, o, out, ws)
        got, terms = out[0, :some], lambda i, j: (a[i:j, :some].double(), b[i:j].double())
    else:                                              # cols tokens, rows features: out [cols, rows]
        a, o = pos(fc[:, None], cols, depth), torch.tensor([0, cols], dtype=torch.int32, device=dev())
        out = torch.empty((cols, rows), dtype=BF16, device=dev())
        if mode == "forward":
            w, ws = pos(fr[:, None], 1, rows, depth), _ws(cols, rows, depth, 1)
            mo.expert_linear(a, w, o, out, ws)
            terms = lambda i, j: (w[0, :some, i:j].double().T, a[:, i:j].double().T)
        else:
            w, ws = pos(fr, 1, depth, rows), _ws(cols, depth, rows, 1)
            mo.expert_linear_dgrad(a, w, o, out, ws)
            terms = lambda i, j: (w[0, i:j, :some].double(), a[:, i:j].double().T)
        got = out[:, :some].T
    want = torch.zeros((some, cols), dtype=torch.float64, device=dev())
    for i in range(0, depth, 1 << 16):
        l, r = terms(i, i + (1 << 16))
        want += l.T @ r
    assert mo.mo_check_device_status(ws) == 0
    drift = float(((got.double() - want) / want).mean().abs())
    assert drift <= 256 * 2.0 ** -23 + depth / 4096 * 2.0 ** -24 + 5 * 2.0 ** -8 / (3 * some * cols) ** 0.5, drift


def _ints(rng, rows, cols, most=3):
    buf = torch.full((max(rows, 1), _pad8(cols)), float("nan"), dtype=BF16, device=dev())
    buf[:rows, :cols] = torch.from_numpy(rng.integers(-most, most + 1, (rows, cols))).to(BF16).to(dev())
    return buf[:rows, :cols]


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("sizes,before,after,n,k", [
    ([4100], 0, 0, 264, 200), ([3, 70], 2, 1, 136, 8200), ([3, 40], 0, 2, 8200, 72), ([5000, 0, 1], 1, 4, 129, 77),
    ([2051, 1, 767, 769], 0, 0, 257, 2056), ([300, 16, 33, 257], 0, 0, 776, 1032), ([9001, 4097], 0, 3, 72, 136)])
def test_long_sums_of_integers_are_exact(sizes, before, after, n, k, out_dtype, geometry):
    """Every product and partial sum is an integer below 2^24 (9001 x 9), which float32
    holds exactly in any order: a lost, repeated or misplaced term shows."""
    rng = np.random.default_rng(n + 5 * k)
    E, off = len(sizes), _offsets(sizes, before)
    R = int(off[-1]) + after
    X, dY = _ints(rng, R, k), _ints(rng, R, n)
    W = _stack(rng, E, n, k)
    W.copy_(torch.from_numpy(rng.integers(-3, 4, (E, n, k))).to(BF16))
    o, ws = torch.from_numpy(off).to(dev()), _ws(R, n, k, E)
    Y = torch.full((R, _pad8(n)), 3.0, dtype=out_dtype, device=dev())[:, :n]
    dX = torch.full((R, _pad8(k)), 3.0, dtype=out_dtype, device=dev())[:, :k]
    dW, dA = _stack(rng, E, n, k, dtype=out_dtype, fill=7.0), _stack(rng, E, n, k, dtype=out_dtype, fill=5.0)
    mo.expert_linear(X, W, o, Y, ws)
    mo.expert_linear_dgrad(dY, W, o, dX, ws)
    mo.expert_linear_wgrad(dY, X, o, dW, ws)
    mo.expert_linear_wgrad(dY, X, o, dA, ws, accumulate=True)
    y, dx, dw = torch.zeros(R, n, dtype=torch.float64), torch.zeros(R, k, dtype=torch.float64), []
    x, d, w = X.double().cpu(), dY.double().cpu(), W.double().cpu()
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        y[a:b], dx[a:b] = x[a:b] @ w[e].T, d[a:b] @ w[e]
        dw.append(d[a:b].T @ x[a:b])
    dw = torch.stack(dw)
    for got, want in ((Y, y), (dX, dx), (dW, dw), (dA, dw + 5)):
        assert torch.equal(got.cpu(), want.to(out_dtype))
    assert mo.mo_check_device_status(ws) == 0


@pytest.mark.parametrize("rows", [4099, 65536])
def test_long_float32_sums_keep_float32_accuracy(rows, geometry):
    """The relative 2-norm error of a float32 weight gradient stays below 1.5e-6, twice what
    is documented for sums that leave the accumulator every 768 terms (7.5e-7).  Left there
    for the whole of a part, 65536 rows fail; the shorter sum is split in parts of few terms."""
    g = torch.Generator(device=dev()).manual_seed(rows)
    n, k = 256, 264
    dY, X = (torch.randn((rows, c), generator=g, device=dev()).to(BF16) for c in (n, k))
    o, ws = torch.tensor([0, rows], dtype=torch.int32, device=dev()), _ws(rows, n, k, 1)
    dW = torch.empty((1, n, k), device=dev())
    mo.expert_linear_wgrad(dY, X, o, dW, ws)
    want = dY.double().T @ X.double()
    assert float((dW[0].double() - want).norm() / want.norm()) < 1.5e-6
