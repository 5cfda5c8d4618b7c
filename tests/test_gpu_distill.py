"""Distillation from a teacher's top logits against the float64 oracle.

Tolerances, derived from the float32 arithmetic.  exp's argument z = (s - m)/T
carries a relative error of 3 roundings and the exp 2 ulp more: q is off by at
most (4 + 4 |z|) 2^-24 + e_z, e_z = (V / 128 + 64) 2^-24 bounding the sum's error
(at least 128 partial sums).  p has the same form over the teacher's entries.
The gradient adds the two and rounds to the output type.  A loss term
p (log p - log q) is off by p's error times its size plus the logs' own
(|log p| + |log q| + |z|) 2^-22 + e_z."""
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


def _buf(shape, dtype, ld=None, shift=0):
    rows, cols = shape
    ld = ld or cols
    buf = torch.full((rows * ld + shift + 8,), float("nan"), dtype=dtype, device=dev())
    return buf[shift: shift + rows * ld].view(rows, ld)[:, :cols]


def _inputs(seed, n, V, top, dtype, t_dtype=F32, idx_dtype=torch.int32, ld=None, shift=0):
    rng = np.random.default_rng(seed)
    s = _buf((n, V), dtype, ld, shift)
    s.copy_(torch.from_numpy(2 * rng.standard_normal((n, V))).to(dtype))
    idx = np.stack([rng.permutation(max(V, top))[:top] for _ in range(n)])
    t = torch.from_numpy(2 * rng.standard_normal((n, top))).to(t_dtype).to(dev())
    return s, torch.from_numpy(idx).to(idx_dtype).to(dev()), t


def _check(s, idx, t, T, w, gs, loss, grad):
    want_l, want_g, q, z = ot.distill_topk(_f64(s), idx.cpu().numpy(), _f64(t), np.float32(T),
                                           None if w is None else _f64(w), np.float32(gs))
    n, V = q.shape
    e_z = (V / 128 + 64) * 2.0 ** -24
    with np.errstate(all="ignore"):
        span = (np.nanmax(np.where(np.isfinite(_f64(t)), _f64(t), np.nan), 1) -
                np.nanmin(np.where(np.isfinite(_f64(t)), _f64(t), np.nan), 1)) / T
    span = np.nan_to_num(span)[:, None]
    e_p = (8 + 4 * span) * 2.0 ** -24 + (t.size(1) / 32 + 16) * 2.0 ** -24
    ww = np.ones(n) if w is None else np.abs(_f64(w))
    if grad is not None:
        got = _f64(grad)
        zz = np.where(np.isfinite(z), np.abs(z), 0)
        tol = gs * T * ww[:, None] * (q * ((4 + 4 * zz) * 2.0 ** -24 + e_z) + 1.0 * e_p * (np.abs(want_g) > 0) *
                                      _teacher_mass(idx, t, T, V)) * 1.01
        tol += (U[grad.dtype] + 4 * 2.0 ** -24) * 1.01 * np.abs(want_g) + 1e-37
        assert np.array_equal(np.isfinite(got), np.isfinite(want_g))
        assert np.all((np.abs(got - want_g) <= tol) | ~np.isfinite(want_g)), np.max(np.abs(got - want_g) - tol)
    if loss is not None:
        got = _f64(loss)
        p = _teacher_mass(idx, t, T, V)
        with np.errstate(all="ignore"):
            logq = z - np.log(np.exp(z).sum(1, keepdims=True))      # q itself underflows for a masked logit
            size = np.where(p > 0, p * (np.abs(np.log(np.where(p > 0, p, 1))) + np.abs(logq) + np.abs(z)), 0).sum(1)
            size = np.where(np.isfinite(size), size, 0)
        k = np.log(t.size(1) + 1)
        tol = ww * T * T * ((size + k) * (e_p[:, 0] + 2.0 ** -21) + e_z) * 1.01
        assert np.array_equal(got[~np.isfinite(want_l)], want_l[~np.isfinite(want_l)])
        fin = np.isfinite(want_l)
        assert np.all(np.abs(got - want_l)[fin] <= tol[fin]), np.max((np.abs(got - want_l) - tol)[fin])


def _teacher_mass(idx, t, T, V):
    """The teacher's probability at each place, summed over repeated places."""
    tt, ii = _f64(t), idx.cpu().numpy()
    out = np.zeros((len(tt), V))
    for r in range(len(tt)):
        on = (ii[r] >= 0) & (ii[r] < V) & (tt[r] != -np.inf)
        if not on.any():
            continue
        x = (tt[r][on] - tt[r][on].max()) / T
        np.add.at(out[r], ii[r][on], np.exp(x) / np.exp(x).sum())
    return out


def _run(s, idx, t, T=1.0, w=None, gs=1.0, g_dtype=None, ld=None, shift=0):
    """Both orders; they must agree with each other and are returned."""
    n, V = s.shape
    g_dtype = g_dtype or s.dtype
    loss, loss2 = (torch.full((n,), float("nan"), device=dev()) for _ in range(2))
    stats = torch.full((n, 2), float("nan"), device=dev())
    g1, g2 = _buf((n, V), g_dtype, ld, shift), _buf((n, V), g_dtype, ld, shift)
    mo.distill_topk_loss_grad(s, idx, t, loss, g1, temperature=T, row_weight=w, grad_scale=gs)
    mo.distill_topk_loss(s, idx, t, loss2, stats, temperature=T, row_weight=w)
    mo.distill_topk_grad(s, idx, t, stats, g2, temperature=T, row_weight=w, grad_scale=gs)
    return (loss, g1), (loss2, g2)


CASES = [
    # n, V, top, ld, shift: one-row and one-place rows, odd vocabularies, strides, offsets, rows split in parts
    (1, 1, 1, None, 0), (1, 7, 3, None, 0), (3, 100, 100, None, 0), (5, 1000, 16, 1008, 0), (4, 999, 33, 1003, 1),
    (2, 5003, 1024, None, 3), (7, 32000, 64, None, 0), (2, 50021, 100, None, 0), (3, 130001, 20, 130008, 5),
    (2, 300000, 8, None, 0), (1, 900001, 50, None, 0), (300, 515, 5, None, 0)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,V,top,ld,shift", CASES)
def test_loss_and_gradient(n, V, top, ld, shift, dtype):
    s, idx, t = _inputs(n + V, n, V, top, dtype, t_dtype=BF16 if n % 2 else F32,
                        idx_dtype=torch.int64 if n % 2 else torch.int32, ld=ld, shift=shift)
    w = torch.from_numpy(np.random.default_rng(V).uniform(0.1, 2.0, n).astype(np.float32)).to(dev())
    for loss, grad in _run(s, idx, t, T=1.5, w=w, gs=0.7, ld=ld, shift=shift):
        _check(s, idx, t, 1.5, w, 0.7, loss, grad)


@pytest.mark.parametrize("dtype,g_dtype", [(F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("T", [0.25, 1.0, 8.0])
@pytest.mark.parametrize("shift,gshift", [(0, 0), (1, 2), (0, 3)])
def test_other_gradient_type_and_alignment(dtype, g_dtype, T, shift, gshift):
    s, idx, t = _inputs(9, 6, 2049, 12, dtype, shift=shift)
    for loss, grad in _run(s, idx, t, T=T, g_dtype=g_dtype, shift=gshift):
        _check(s, idx, t, T, None, 1.0, loss, grad)


@pytest.mark.parametrize("V", [64, 4097, 140000])
def test_repeated_absent_and_masked_entries(V):
    s, idx, t = _inputs(11, 6, V, 9, F32)
    idx[0, 4:7] = idx[0, 1]                      # one place named four times
    idx[1, ::2] = -1                             # absent entries, also past the vocabulary
    idx[1, 1] = V
    idx[2] = -1                                  # a row without a teacher
    t[3] = float("-inf")                         # a row whose entries are all masked
    t[4, 2:] = float("-inf")
    s[5, 1::3] = float("-inf")                   # masked logits away from ...
    idx[5] = torch.arange(9, device=dev()) * 3   # ... and at none of the teacher's places
    for loss, grad in _run(s, idx, t):
        _check(s, idx, t, 1.0, None, 1.0, loss, grad)
        assert loss[2] == 0 and loss[3] == 0 and torch.all(grad[2:4] == 0)
        assert torch.all(grad[5, 1::3] == 0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [50, 20000])
def test_lowest_values_infinities_and_nan(dtype, V):
    s, idx, t = _inputs(12, 8, V, 6, dtype)
    low = torch.finfo(dtype).min
    s[0, 10:40] = low                            # masks of the type's lowest value
    s[1] = low                                   # everywhere: q is uniform
    s[2] = float("-inf")                         # everywhere: q = 0, the loss infinite
    s[3, idx[3, 0].item()] = float("-inf")       # the teacher wants a masked logit: infinite loss
    t[4] = torch.finfo(t.dtype).min              # uniform teacher at the lowest value
    w = torch.ones(8, device=dev())
    s[5] = float("nan")
    w[5] = 0                                     # a row without weight is not read
    s[6, 3] = float("nan")                       # NaN spreads within its row only
    s[7] = 3e38 if dtype == F32 else 3e38
    for loss, grad in _run(s, idx, t, T=0.5, w=w):
        ok = torch.tensor([0, 1, 2, 3, 4, 5, 7], device=dev())
        _check(s[ok], idx[ok], t[ok], 0.5, w[ok], 1.0, loss[ok], grad[ok])
        assert loss[2] == float("inf") and loss[3] == float("inf") and bool(torch.isfinite(grad[2:4]).all())
        assert loss[5] == 0 and torch.all(grad[5] == 0)
        assert bool(torch.isnan(loss[6])) and bool(torch.isnan(grad[6]).all())


@pytest.mark.parametrize("V", [777, 70000, 1200000])
def test_gradient_in_place(V):
    s, idx, t = _inputs(13, 3, V, 10, BF16)
    idx[1, 3] = idx[1, 4]
    (loss, want), (_, want2) = _run(s, idx, t, T=2.0)
    a, b, l2, st = s.clone(), s.clone(), torch.empty_like(loss), torch.empty((3, 2), device=dev())
    mo.distill_topk_loss_grad(a, idx, t, l2, a, temperature=2.0)
    assert torch.equal(a, want) and torch.equal(l2, loss)
    mo.distill_topk_loss(b, idx, t, l2, st, temperature=2.0)
    mo.distill_topk_grad(b, idx, t, st, b, temperature=2.0)
    assert torch.equal(b, want2)


def test_results_repeat_bit_for_bit_and_neighbours_stay_untouched():
    s, idx, t = _inputs(14, 40, 33003, 25, F32, ld=33011)
    buf = torch.full((40, 33011), 5.0, device=dev())
    runs = []
    for _ in range(3):
        loss = torch.empty(40, device=dev())
        mo.distill_topk_loss_grad(s, idx, t, loss, buf[:, :33003])
        runs.append((loss, buf[:, :33003].clone()))
    assert all(torch.equal(r[0], runs[0][0]) and torch.equal(r[1], runs[0][1]) for r in runs)
    assert torch.all(buf[:, 33003:] == 5.0)


def test_gradient_matches_differences_of_the_loss():
    """A directional difference of the float32 loss, h = 2^-4: the loss's third
    derivative term is below h^2 |D|_max^3 / 6 of its size (about 1e-3 of the sum),
    its rounding 2^-21 of the loss over h."""
    s, idx, t = _inputs(15, 8, 300, 7, F32)
    D = torch.from_numpy(np.sign(np.random.default_rng(1).standard_normal((8, 300))).astype(np.float32)).to(dev())
    h = 2.0 ** -4
    l1, l2, st = torch.empty(8, device=dev()), torch.empty(8, device=dev()), torch.empty((8, 2), device=dev())
    mo.distill_topk_loss(s + h * D, idx, t, l1, st, temperature=2.0)
    mo.distill_topk_loss(s - h * D, idx, t, l2, st, temperature=2.0)
    (_, grad), _ = _run(s, idx, t, T=2.0)
    diff = (l1.double() - l2.double()) / (2 * h)
    dot = (grad.double() * D.double()).sum(1)
    assert torch.all((diff - dot).abs() <= 2e-3 * (1 + grad.double().abs().sum(1)) + 2.0 ** -21 * l1.double().abs() / h)


def test_other_stream():
    s, idx, t = _inputs(16, 4, 5000, 8, BF16)
    loss, g = torch.empty(4, device=dev()), torch.empty_like(s)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    mo.distill_topk_loss_grad(s, idx, t, loss, g, stream=st)
    st.synchronize()
    _check(s, idx, t, 1.0, None, 1.0, loss, g)


def _wide_range_rows(s, idx, far):
    """Rows whose largest or smallest logits are `far` away from the ordinary ones, and
    rows on either side of where float32 logits get sparse."""
    V = s.size(1)
    low, high = -far, far
    s[0, : 3 * V // 4] = low                     # a masked run: threads that see nothing else at first
    s[1] = low                                   # the whole row: q is uniform
    s[2, :9] = low                               # what lies before the first, after the last 16-byte boundary
    s[2, -9:] = low
    s[3] = low                                   # all but one
    s[3, V // 2] = 1.0
    s[4, idx[4, :2].long()] = low                # where the teacher wants them
    s[5, V // 3] = high                          # one logit far above the others
    s[6] = high
    at = torch.arange(V, device=s.device) * 7 % 11
    s[7] = (3e7 + 2 * at).to(s.dtype)            # neighbouring float32 values
    s[8] = (-2.4e7 - 2 * at).to(s.dtype)
    s[8, ::3] = low


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [0.3, 1.0, 2.0, 4.0])
@pytest.mark.parametrize("far", [1e9, 1e10, 1e12, 1e20])
@pytest.mark.parametrize("n,V,ld,shift", [(9, 61, 67, 1), (9, 20001, 20010, 3), (320, 2050, None, 0)])
def test_logits_of_any_size(n, V, ld, shift, far, T, dtype):
    s, idx, t = _inputs(17, n, V, 6, dtype, ld=ld, shift=shift)
    _wide_range_rows(s, idx, far)
    for loss, grad in _run(s, idx, t, T=T, ld=ld, shift=shift):
        _check(s, idx, t, T, None, 1.0, loss, grad)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1e-5, 1e-9, 1e-20, 1e-30])
@pytest.mark.parametrize("n,V,shift", [(64, 50, 1), (8, 20001, 0)])
def test_low_temperatures(n, V, shift, T, dtype):
    """The largest logit alone counts, whatever its product with 1/T rounds to.  (Half of
    the teachers are uniform: their probabilities do not depend on T.)"""
    s, idx, t = _inputs(18, n, V, 6, dtype, shift=shift)
    s += 10
    s[1] = s[1, 0].clone()
    t[::2] = 1.0
    for loss, grad in _run(s, idx, t, T=T, shift=shift):
        _check(s, idx, t, T, None, 1.0, loss, grad)


@pytest.mark.parametrize("n", [1, 3])
def test_statistics_hold_the_maximum_and_the_sum(n):
    """stats = {max s, sum exp((s - max) / T)} also for a maximum whose product with 1/T rounds coarsely."""
    s, idx, t = _inputs(19, n, 4000, 5, F32)
    s[0] = 1e9
    s[0, :100] = 1e9 - 64
    for T in (1.0, 64.0, 1e-9):
        loss, stats = torch.empty(n, device=dev()), torch.empty((n, 2), device=dev())
        mo.distill_topk_loss(s, idx, t, loss, stats, temperature=T)
        x = s.double()
        z = torch.exp((x - x.amax(1, keepdim=True)) / float(np.float32(T))).sum(1)
        assert torch.equal(stats[:, 0], s.amax(1))
        assert torch.all((stats[:, 1].double() - z).abs() <= (4000 / 128 + 68) * 2.0 ** -24 * z)
