"""A teacher's top logits, the divergence of a student's logits from them and its gradient,
against the fp64 reference.

Tolerances.  With d the bound of the relative error of a row's sum of exponentials over the tokens not
listed (oracle.distill.exp_error: fp32 exponentials, fp32 sums per thread, fp64 across) and everything else
in fp64, and EPS32 half a step of fp32:
  logp = z / tau - lse: lse is off by q_rest d, and logp is rounded once;
  rest: off by (1 + q_rest) d, rounded once;
  loss: w (P q_rest d + r (1 + q_rest) d) and one rounding;
  a listed token's gradient: w / tau (total q q_rest d + 4 EPS32 sum p) (the probabilities are fp32
  exponentials: two units and one rounding of their sum) and the rounding to the gradient's type;
  one not listed: its exponential (3 |x - max x| + 4 roundings), times a coefficient (2 more) whose two parts
  are off by q_rest d and by d, and the rounding to the gradient's type."""
import ctypes

import numpy as np
import pytest
import torch

import synth
from oracle import distill as D

nq = pytest.importorskip("sub_bit_weight_amd")

DEV = "cuda:0"
DUMMY = 0x100000
EPS = D.EPS32
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # half a step, relative to the value (bf16: to the binade's lower end)
THREADS = 256  # the fewest threads that share a row
gpu = pytest.mark.gpu


def _rows(tag, T, V, dtype):
    z = 2.0 * synth.normal_f32(f"distill/{tag}/z", (T, V))
    g = synth.rng(f"distill/{tag}/likely")
    for t in range(T):
        z[t, g.integers(0, V, min(V, 6))] += np.float32(7.0)
    return synth.round_bf16(z) if dtype == "bf16" else z


def _record(tag, T, V, k, tau, rest=True):
    """A record as fp32 arrays, of a teacher of its own."""
    ids, logp, left = D.logits_top_ref(_rows(tag + "/teacher", T, V, "f32"), k, tau)
    return ids, logp.astype(np.float32), left.astype(np.float32) if rest else None


# ---------------------------------------------------------------- the reference


@pytest.mark.parametrize("rest", [True, False])
def test_reference_gradient_matches_differences(rest):
    T, V, tau = 3, 9, 1.7
    ids, logp, left = _record("diff", T, V, 4, tau, rest)
    ids[1, 2] = ids[1, 0]  # a token twice
    ids[2, 1:] = -1
    w = np.array([1.0, 0.3, 2.0])
    s = _rows("diff/s", T, V, "f32").astype(np.float64)
    grad = D.distill_ref(ids, logp, left, tau, s, w)[1]
    for i in np.ndindex(s.shape):
        up, down = s.copy(), s.copy()
        up[i] += 1e-4
        down[i] -= 1e-4
        num = (D.distill_ref(ids, logp, left, tau, up, w)[0] - D.distill_ref(ids, logp, left, tau, down, w)[0]).sum() / 2e-4
        assert abs(num - grad[i]) <= 1e-7 + 1e-6 * abs(grad[i])


def test_reference_of_a_whole_row_is_the_divergence():
    T, V, tau = 4, 11, 0.8
    z, s = _rows("whole/z", T, V, "f32"), _rows("whole/s", T, V, "f32")
    ids, logp, rest = D.logits_top_ref(z, V, tau)
    assert np.isneginf(rest).all()
    lp = z / tau - np.log(np.exp(z / tau).sum(1, keepdims=True))
    lq = s / tau - np.log(np.exp(s / tau).sum(1, keepdims=True))
    want = (np.exp(lp) * (lp - lq)).sum(1)
    for left in (rest, None):
        loss, grad = D.distill_ref(ids, logp, left, tau, s)
        assert np.allclose(loss, want, rtol=1e-5)
        assert np.allclose(grad, (np.exp(lq) - np.exp(lp)) / tau, atol=1e-6)


# ---------------------------------------------------------------- refusals (no GPU)


def _top(x=DUMMY, dt=nq.NQ_BF16, T=3, V=100, ld=100, k=4, tau=1.0, ids=DUMMY, logp=DUMMY, rest=DUMMY):
    return nq.lib().nq_logits_top(x, dt, T, V, ld, k, tau, ids, logp, rest, None)


def _teacher(**kw):
    d = dict(k=4, ids=DUMMY, logp=DUMMY, rest=DUMMY, temperature=1.0)
    d.update(kw)
    return nq.nq_teacher(**d)


def _loss(p, x=DUMMY, dt=nq.NQ_BF16, T=3, V=100, ld=100, weight=DUMMY, loss=DUMMY):
    return nq.lib().nq_distill_loss(None if p is None else ctypes.byref(p), x, dt, T, V, ld, weight, loss, None)


def _grads(p, x=DUMMY, dt=nq.NQ_BF16, T=3, V=100, ld=100, weight=DUMMY, loss=DUMMY, dl=2 * DUMMY, dd=nq.NQ_BF16, ldd=100):
    return nq.lib().nq_distill_grads(None if p is None else ctypes.byref(p), x, dt, T, V, ld, weight, loss, dl, dd, ldd,
                                     None)


LOGITS = [(dict(x=None), 1), (dict(x=DUMMY + 1), 1), (dict(dt=nq.NQ_F32, x=DUMMY + 2), 1), (dict(dt=7), 1), (dict(T=0), 1),
          (dict(V=0), 1), (dict(ld=99), 1), (dict(T=(1 << 21) + 1), 2), (dict(V=(1 << 20) + 1, ld=1 << 21), 2)]
SCALARS = [(dict(k=0), 1), (dict(k=-3), 1), (dict(k=1025), 2), (dict(temperature=0.0), 1), (dict(temperature=-1.0), 1),
           (dict(temperature=float("nan")), 1), (dict(temperature=float("inf")), 1), (dict(temperature=2.0 ** -21), 1)]


@pytest.mark.parametrize("kw,status", LOGITS)
def test_rejects_bad_logits(kw, status):
    for st in (_top(**kw), _loss(_teacher(), **kw), _grads(_teacher(), **{"ldd": 1 << 21, **kw})):
        assert st == status and nq.last_error() != ""


@pytest.mark.parametrize("kw,status", SCALARS)
def test_rejects_bad_sizes(kw, status):
    assert _loss(_teacher(**kw)) == status and nq.last_error() != ""
    assert _grads(_teacher(**kw)) == status
    kw = {"tau" if n == "temperature" else n: v for n, v in kw.items()}
    assert _top(**kw) == status


def test_rejects_bad_pointers():
    for kw in (dict(ids=None), dict(logp=None), dict(ids=DUMMY + 2), dict(logp=DUMMY + 1), dict(rest=DUMMY + 2)):
        assert _top(**kw) == nq.NQ_ERR_ARG, kw
        assert _loss(_teacher(**kw)) == nq.NQ_ERR_ARG, kw
        assert _grads(_teacher(**kw)) == nq.NQ_ERR_ARG, kw
    p = _teacher()
    assert _loss(None) == nq.NQ_ERR_ARG and _grads(None) == nq.NQ_ERR_ARG
    assert _loss(p, loss=None) == nq.NQ_ERR_ARG
    for call in (_loss, _grads):
        assert call(p, weight=DUMMY + 2) == nq.NQ_ERR_ARG
        assert call(p, loss=DUMMY + 1) == nq.NQ_ERR_ARG
    for kw in (dict(dl=None), dict(dl=DUMMY + 1), dict(dd=9), dict(ldd=99), dict(dd=nq.NQ_F32, dl=DUMMY + 2),
               dict(dl=DUMMY, dd=nq.NQ_F32), dict(dl=DUMMY, ldd=104)):
        assert _grads(p, **kw) == nq.NQ_ERR_ARG, kw


# ---------------------------------------------------------------- GPU


def _dev(a, dtype=None):
    t = torch.from_numpy(np.array(a)).to(DEV)  # a copy: a view's rows are laid out anew
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def _host(t):
    return t.float().cpu().numpy().astype(np.float64)


def _round_err(v, dtype):
    return HALF[dtype] * np.abs(v) + 1e-37


def _check_top(z, k, tau, got):
    ids, logp, rest = D.logits_top_ref(z, k, tau)
    assert np.array_equal(got.ids.cpu().numpy(), ids)
    glp, grest = _host(got.logp), _host(got.rest)
    for t in range(z.shape[0]):
        listed = np.zeros(z.shape[1], bool)
        listed[ids[t][ids[t] >= 0]] = True
        d = D.exp_error(z[t] / tau, listed, THREADS)
        q = np.exp(rest[t])
        fine = np.isfinite(logp[t])
        assert np.array_equal(glp[t][~fine], logp[t][~fine], equal_nan=True)
        assert (np.abs(glp[t] - logp[t])[fine] <= q * d + 2 * EPS * np.abs(logp[t][fine]) + 1e-9).all(), t
        if np.isfinite(rest[t]):
            assert abs(grest[t] - rest[t]) <= (1 + q) * d + 2 * EPS * abs(rest[t]) + 1e-9, t
        else:
            assert np.array_equal(grest[t], rest[t], equal_nan=True), t


TOP = [(1, 1, 1, "f32", 1.0), (3, 2, 1, "bf16", 1.0), (2, 7, 9, "f32", 1.0), (5, 33, 4, "f32", 0.5), (4, 1000, 64, "bf16", 2.0),
       (3, 1027, 1024, "f32", 1.0), (2, 4097, 300, "bf16", 1.0), (3, 8200, 16, "f32", 1.0), (2, 32000, 64, "bf16", 1.0),
       (2, 50021, 37, "f32", 1.3), (2, 70001, 100, "f32", 1.0), (2, 131072, 128, "bf16", 1.0), (1, 131079, 7, "bf16", 1.0),
       (1, 1 << 20, 1024, "bf16", 1.0)]


@gpu
@pytest.mark.parametrize("T,V,k,dtype,tau", TOP)
def test_top(T, V, k, dtype, tau):
    z = _rows(f"top/{V}/{k}", T, V, dtype)
    _check_top(z, k, tau, nq.logits_top(_dev(z, dtype), k, temperature=tau))


def _orders(V):
    g = synth.rng(f"distill/orders/{V}")
    up = np.linspace(-8, 8, V).astype(np.float32)
    few = g.choice(np.float32([1.0, 1.5, -2.0]), V)
    zeros = np.where(g.random(V) < 0.5, np.float32(0.0), np.float32(-0.0))
    run = np.full(V, -5.0, np.float32)
    run[V // 3:V // 3 + V // 4] = up[V // 3:V // 3 + V // 4]
    lanes = np.full(V, -3.0, np.float32)
    lanes[::512] = 4.0 + g.random(len(lanes[::512])).astype(np.float32)  # the largest in few threads' elements
    return np.stack([up, up[::-1], np.full(V, 1.25, np.float32), few, zeros, run, lanes])


@gpu
@pytest.mark.parametrize("V,k", [(40, 13), (3000, 64), (3000, 1024), (33001, 50), (140000, 200)])
def test_top_of_equal_and_sorted_logits(V, k):
    for dtype in ("f32", "bf16"):
        z = _orders(V)
        z = synth.round_bf16(z) if dtype == "bf16" else z
        _check_top(z, k, 1.0, nq.logits_top(_dev(z, dtype), k))


def _odd_rows(tag, V):
    """Rows with masked tokens, infinities and NaN."""
    z = _rows(tag, 9, V, "bf16")
    z[0] = -np.inf
    z[1, 3:] = -np.inf
    z[2, V // 2] = np.nan
    z[3, 1] = np.inf
    z[4, ::2] = -np.inf
    z[5] = np.float32(-3.3895313892515355e38)  # masks of bf16's lowest value
    z[5, :4] = [0.5, -1.0, 2.0, 0.25]
    z[6] = synth.round_bf16(np.full(V, 3e38, np.float32))
    z[7, -1] = 40.0
    return synth.round_bf16(z)


@gpu
@pytest.mark.parametrize("V,k", [(50, 6), (50, 60), (4100, 70), (40001, 9)])
def test_top_of_masked_and_non_finite_rows(V, k):
    z = _odd_rows(f"odd/{V}", V)
    for dtype in ("f32", "bf16"):
        _check_top(z, k, 1.0, nq.logits_top(_dev(z, dtype), k))


def _check_distill(ids, logp, rest, tau, s, weight, loss, grad=None, gtype="f32"):
    want, wgrad = D.distill_ref(ids, logp, rest, tau, s, weight)
    loss, grad = _host(loss), None if grad is None else _host(grad)
    for t in range(s.shape[0]):
        if not np.isfinite(want[t]) or not np.isfinite(wgrad[t]).all():
            assert np.array_equal(loss[t], want[t], equal_nan=True), t
            if grad is not None and np.isnan(wgrad[t]).all():
                assert np.isnan(grad[t]).all(), t
            if not np.isfinite(wgrad[t]).all():
                continue
        w = 1.0 if weight is None else float(weight[t])
        v = ids[t][ids[t] >= 0]
        listed = np.zeros(s.shape[1], bool)
        listed[v] = True
        x = s[t].astype(np.float64) / tau
        d = D.exp_error(x, listed, THREADS)
        p = np.exp(logp[t].astype(np.float64))[ids[t] >= 0]
        P, r = p.sum(), 0.0 if rest is None else np.exp(float(rest[t]))
        if P + r == 0.0 or w == 0.0:
            assert loss[t] == 0.0 and (grad is None or (grad[t] == 0.0).all()), t
            continue
        if rest is None:
            p, P = p / P, 1.0
        m = x.max()
        e = np.exp(x - m)
        q, away = e / e.sum(), e[~listed].sum() / e.sum()
        if np.isfinite(want[t]):
            tol = abs(w) * (P * away * d + r * (1 + away) * d) + EPS * abs(want[t]) + 1e-12 * abs(w)
            assert abs(loss[t] - want[t]) <= tol, (t, loss[t], want[t], tol)
        if grad is None:
            continue
        c, total = abs(w) / tau, P + r
        sums = np.zeros(s.shape[1])
        np.add.at(sums, v, p)
        tol = c * (total * q * away * d + 4 * EPS * sums)
        if np.isfinite(x[~listed]).any():
            top = x[~listed].max()
            share = np.exp(np.minimum(x - top, 0.0))
            own = (3 * np.minimum(np.abs(x - top), 200.0) + 6) * EPS  # beyond 200 the value is 0
            part = total * q * away * d + r * share / share[~listed].sum() * d
            tol = np.where(listed, tol, c * part + np.abs(wgrad[t]) * own)
        tol = tol + _round_err(wgrad[t], gtype) + 1e-12 * c * (total * q + sums)
        bad = np.abs(grad[t] - wgrad[t]) > tol
        assert not bad.any(), (t, np.argwhere(bad)[:4], grad[t][bad][:4], wgrad[t][bad][:4], tol[bad][:4])


CASES = [(1, 1, 1, "f32", 1.0, True), (3, 2, 1, "bf16", 1.0, True), (2, 7, 7, "f32", 1.0, True), (2, 7, 7, "f32", 1.0, False),
         (5, 33, 4, "f32", 0.5, True), (4, 1000, 64, "bf16", 2.0, False), (3, 1025, 1024, "f32", 1.0, True),
         (2, 2048, 3, "bf16", 1.0, True), (3, 4099, 20, "f32", 1.0, False), (2, 8200, 300, "bf16", 1.0, True),
         (2, 16400, 16, "f32", 0.7, True), (2, 32000, 64, "bf16", 1.0, True), (2, 33000, 64, "bf16", 1.0, True),
         (2, 50021, 37, "f32", 2.0, False), (1, 65540, 5, "f32", 1.0, True), (2, 70001, 100, "f32", 1.0, True),
         (2, 131072, 128, "bf16", 1.0, True), (1, 131079, 9, "bf16", 1.0, False), (1, 1 << 20, 1024, "bf16", 1.0, True)]


@gpu
@pytest.mark.parametrize("T,V,k,dtype,tau,rest", CASES)
def test_loss_and_gradient(T, V, k, dtype, tau, rest):
    ids, logp, left = _record(f"grad/{V}/{k}", T, V, k, tau, rest)
    s = _rows(f"grad/{V}/s", T, V, dtype)
    w = (0.25 + synth.rng(f"distill/{V}/w").random(T)).astype(np.float32)
    P = nq.Teacher(_dev(ids), _dev(logp), None if left is None else _dev(left), tau)
    x = _dev(s, dtype)
    loss = nq.distill_loss(P, x, _dev(w))
    _check_distill(ids, logp, left, tau, s, w, loss)
    loss2, grad = nq.distill_grads(P, x, _dev(w))
    assert grad.dtype == x.dtype and torch.equal(nq.distill_loss(P, x, _dev(w)), loss)
    _check_distill(ids, logp, left, tau, s, w, loss2, grad, dtype)
    other = torch.float32 if dtype == "bf16" else torch.bfloat16
    grad2 = torch.empty(T, V, dtype=other, device=DEV)
    loss3, _ = nq.distill_grads(P, x, None, dlogits=grad2)
    _check_distill(ids, logp, left, tau, s, None, loss3, grad2, "f32" if dtype == "bf16" else "bf16")
    assert all(torch.equal(a, b) for a, b in zip(nq.distill_grads(P, x, _dev(w)), (loss2, grad)))  # run to run


@gpu
@pytest.mark.parametrize("rest", [True, False])
def test_gradient_matches_differences_of_the_loss(rest):
    """The kernel's gradient against differences of the reference loss (central, fp64)."""
    T, V, tau = 2, 23, 1.5
    ids, logp, left = _record("gdiff", T, V, 5, tau, rest)
    s = _rows("gdiff/s", T, V, "f32")
    P = nq.Teacher(_dev(ids), _dev(logp), None if left is None else _dev(left), tau)
    grad = _host(nq.distill_grads(P, _dev(s))[1])
    for i in np.ndindex(s.shape):
        up, down = s.astype(np.float64), s.astype(np.float64)
        up[i] += 1e-4
        down[i] -= 1e-4
        num = (D.distill_ref(ids, logp, left, tau, up)[0] - D.distill_ref(ids, logp, left, tau, down)[0]).sum() / 2e-4
        assert abs(num - grad[i]) <= 2e-6


@gpu
@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("V", [60, 5003, 40001])
def test_entries_missing_repeated_and_out_of_range(V, rest):
    T, k, tau = 8, 7, 1.0
    ids, logp, left = _record(f"entries/{V}", T, V, k, tau)
    ids[0, 3:] = -1
    ids[1] = -1                       # nothing listed
    ids[2, 4] = ids[2, 1]             # once more
    ids[3] = ids[3, 0]                # one token only
    ids[4, 2] = V                     # out of range
    logp[5, 1:3] = -np.inf            # listed, of probability 0
    ids[6], left[6] = -1, -np.inf     # an empty record
    ids[7, 1:] = -5
    left = left if rest else None
    s = _rows(f"entries/{V}/s", T, V, "bf16")
    P = nq.Teacher(_dev(ids), _dev(logp), None if left is None else _dev(left), tau)
    loss, grad = nq.distill_grads(P, _dev(s, "bf16"))
    _check_distill(ids, logp, left, tau, s, None, loss, grad, "bf16")
    assert torch.isnan(loss[4]) and torch.isnan(grad[4]).all()


@gpu
@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("V", [50, 5000, 40001])
def test_masked_and_non_finite_logits(V, rest):
    s = _odd_rows(f"oddgrad/{V}", V)
    T, k = s.shape[0], 5
    ids, logp, left = _record(f"oddgrad/{V}", T, V, k, 1.0, rest)
    ids[1] = [0, 1, 2, 3, 4]   # two of them masked in the student: an infinite loss, a finite gradient
    ids[4] = [1, 3, 5, 7, 9]   # none of them masked
    ids[7, 0] = V - 1
    P = nq.Teacher(_dev(ids), _dev(logp), None if left is None else _dev(left))
    for dtype in ("f32", "bf16"):
        loss, grad = nq.distill_grads(P, _dev(s, dtype))
        _check_distill(ids, logp, left, 1.0, s, None, loss, grad, dtype)
        _check_distill(ids, logp, left, 1.0, s, None, nq.distill_loss(P, _dev(s, dtype)))


@gpu
@pytest.mark.parametrize("V", [300, 20000, 140001])
def test_rows_of_weight_zero_are_not_read(V):
    ids, logp, left = _record(f"zero/{V}", 3, V, 4, 1.0)
    s = _rows(f"zero/{V}/s", 3, V, "bf16")
    s[1] = np.nan
    ids[1, 0] = V
    w = np.float32([1.0, 0.0, -2.0])
    P = nq.Teacher(_dev(ids), _dev(logp), _dev(left))
    loss, grad = nq.distill_grads(P, _dev(s, "bf16"), _dev(w))
    assert loss[1] == 0 and (grad[1] == 0).all() and nq.distill_loss(P, _dev(s, "bf16"), _dev(w))[1] == 0
    s[1] = 0.0
    ids[1, 0] = 0
    _check_distill(ids, logp, left, 1.0, s, w, loss, grad, "bf16")


@gpu
@pytest.mark.parametrize("V,ld,shift", [(100, 100, 1), (1001, 1001, 0), (999, 1009, 3), (4096, 4104, 0), (32001, 32003, 5),
                                        (70001, 70003, 1), (131071, 131073, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_and_misaligned_rows(V, ld, shift, dtype):
    """Rows at any alignment: the same results as contiguous ones, and nothing behind or between the rows is written."""
    T, k = 3, 6
    ids, logp, left = _record(f"ld/{V}", T, V, k, 1.0)
    s = _rows(f"ld/{V}/s", T, V, dtype)
    x = _dev(s, dtype)
    P = nq.Teacher(_dev(ids), _dev(logp), _dev(left))
    loss, grad = nq.distill_grads(P, x)

    def view(fill):
        flat = torch.full((shift + T * ld + 64,), fill, dtype=x.dtype, device=DEV)
        return flat, flat[shift:shift + T * ld].view(T, ld)[:, :V]
    flat, xs = view(float("nan"))
    xs.copy_(x)
    gflat, gs = view(7.0)
    loss2, out = nq.distill_grads(P, xs, dlogits=gs)
    assert out is gs and torch.equal(loss2, loss) and torch.equal(gs, grad)
    gs.fill_(7.0)
    assert (gflat == 7.0).all()
    assert torch.equal(nq.distill_loss(P, xs), nq.distill_loss(P, x))
    a, b = nq.logits_top(x, k), nq.logits_top(xs, k)
    assert torch.equal(a.ids, b.ids) and torch.equal(a.logp, b.logp) and torch.equal(a.rest, b.rest)
    before = xs.clone()
    loss3, out = nq.distill_grads(P, xs, dlogits=xs)  # in place
    assert out is xs and torch.equal(loss3, loss) and torch.equal(xs, grad)
    xs.copy_(before)
    xs.fill_(float("nan"))
    assert torch.isnan(flat).all()


@gpu
@pytest.mark.parametrize("T,V,dtype", [(1, 256, "f32"), (300, 1500, "bf16"), (700, 9000, "bf16")])
def test_a_student_that_is_the_teacher(T, V, dtype):
    """Record and student of the same logits: a divergence of zero, to the roundings of the record and the sums."""
    z = _dev(_rows(f"same/{V}", T, V, dtype), dtype)
    P = nq.logits_top(z, 50, temperature=1.5)
    loss, grad = nq.distill_grads(P, z.float())
    # the record's logarithms (up to 16 in size, one rounding each) and both sums' errors (|x| up to 20)
    tol = 16 * EPS + 2 * (3 * 20 + 4 + 48) * EPS
    assert loss.abs().max() <= tol and grad.abs().max() <= tol


@gpu
def test_other_stream_and_captured_calls():
    T, V, k = 5, 3001, 17
    ids, logp, left = _record("graph", T, V, k, 1.0)
    P = nq.Teacher(_dev(ids), _dev(logp), _dev(left))
    xs = [_dev(_rows(f"graph/{i}", T, V, "bf16"), "bf16") for i in range(3)]
    want = [(nq.logits_top(x, k), nq.distill_grads(P, x), nq.distill_loss(P, x)) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = nq.distill_grads(P, xs[0], stream=side)
    top = nq.logits_top(xs[0], k, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[1], want[0][1][1]) and torch.equal(got[0], want[0][1][0])
    assert torch.equal(top.ids, want[0][0].ids) and torch.equal(top.logp, want[0][0].logp)
    x = xs[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rec = nq.logits_top(x, k)
        loss = nq.distill_loss(P, x)
        loss2, grad = nq.distill_grads(P, x)
    for i in (0, 1, 2, 1):
        x.copy_(xs[i])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(rec.ids, want[i][0].ids) and torch.equal(rec.rest, want[i][0].rest)
        assert torch.equal(loss, want[i][2]) and torch.equal(loss2, want[i][1][0]) and torch.equal(grad, want[i][1][1])
        nq.distill_grads(P, xs[(i + 1) % 3])  # eager work between the replays


@gpu
def test_binding_refuses_wrong_tensors():
    ids, logp, left = _record("refuse", 4, 30, 3, 1.0)
    ids, logp, left = _dev(ids), _dev(logp), _dev(left)
    x = torch.zeros(4, 30, device=DEV)
    P = nq.Teacher(ids, logp, left)
    for kw in (dict(ids=ids.long()), dict(ids=ids[:, :0]), dict(ids=ids.cpu()), dict(logp=logp[:, :2]),
               dict(logp=logp.bfloat16()), dict(rest=left[:3]), dict(ids=ids.t())):
        with pytest.raises(ValueError):
            nq.Teacher(**{**dict(ids=ids, logp=logp, rest=left), **kw}).struct()
    for bad in (x[:3], x.half(), x.cpu(), x.t().contiguous().t(), x[0], x[:, :0], x[:1].expand(4, 30)):
        with pytest.raises(ValueError):
            nq.distill_loss(P, bad)
        with pytest.raises(ValueError):
            nq.distill_grads(P, bad)
    for bad in (x.half(), x.cpu(), x[0], x[:0], x[:1].expand(4, 30)):
        with pytest.raises(ValueError):
            nq.logits_top(bad, 3)
    for kw in (dict(weight=torch.ones(3, device=DEV)), dict(weight=torch.ones(4, device=DEV).double())):
        with pytest.raises(ValueError):
            nq.distill_loss(P, x, **kw)
    with pytest.raises(ValueError):
        nq.distill_loss(P, x, loss=torch.zeros(3, device=DEV))
    for g in (torch.zeros(4, 29, device=DEV), torch.zeros(4, 30, device=DEV).half(), torch.zeros(4, 30)):
        with pytest.raises(ValueError):
            nq.distill_grads(P, x, dlogits=g)
    with pytest.raises(ValueError):
        nq.logits_top(x, 0)
    for call in (lambda: nq.logits_top(x, 2000), lambda: nq.logits_top(x, 3, temperature=0.0),
                 lambda: nq.distill_loss(nq.Teacher(ids, logp, left, -1.0), x)):
        with pytest.raises(nq.NqError):
            call()


# ---------------------------------------------------------------- every kernel that a rule chooses


def _many_rows(tag, V):
    """Distinct rows of every kind (spread, sorted, in runs, equal, masked, not finite), and which of them each of 1030
    rows is: more rows than 1024 choose fewer threads per row."""
    rows = np.concatenate([_rows(f"{tag}/{V}", 12, V, "bf16"), synth.round_bf16(_orders(V)), _odd_rows(f"{tag}/odd", V)])
    order = synth.rng(f"distill/{tag}/{V}/order").permutation(1030) % len(rows)
    first = np.array([np.flatnonzero(order == i)[0] for i in range(len(rows))])
    return rows, order, first


def _pick(teacher, at):
    at = torch.from_numpy(at).to(DEV)
    return nq.Teacher(teacher.ids[at].contiguous(), teacher.logp[at].contiguous(), teacher.rest[at].contiguous(),
                      teacher.temperature)


@gpu
@pytest.mark.parametrize("V,k", [(32003, 64), (20011, 200), (9000, 128), (40001, 300)])
def test_top_of_many_rows(V, k):
    """256 threads a row over several steps (512 for k to 256, 1024 beyond): bounds taken anew, candidates pruned and
    more than a wave has room for."""
    rows, order, first = _many_rows("many", V)
    for dtype in ("bf16", "f32"):
        z = _dev(rows, dtype)[torch.from_numpy(order).to(DEV)]
        got = nq.logits_top(z, k)
        _check_top(rows, k, 1.0, _pick(got, first))
        again = torch.from_numpy(first[order]).to(DEV)  # rows of the same logits have the same record
        assert torch.equal(got.ids[again], got.ids)
        assert torch.equal(got.logp[again].nan_to_num(3.0), got.logp.nan_to_num(3.0))
        assert torch.equal(got.rest[again].nan_to_num(3.0), got.rest.nan_to_num(3.0))


@gpu
@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("V,k", [(32003, 64), (20011, 700)])
def test_loss_of_many_rows(V, k, rest):
    """A loss of more than 1024 rows takes 256 threads a row over several steps."""
    rows, order, first = _many_rows("manyloss", V)
    ids, logp, left = _record(f"manyloss/{V}", len(rows), V, k, 1.0, rest)
    ids[2, 3], ids[3, 5:9], ids[4, 1] = ids[2, 0], -1, V
    w = (0.25 + synth.rng(f"distill/{V}/w").random(len(rows))).astype(np.float32)
    w[5] = 0.0
    P = nq.Teacher(_dev(ids[order]), _dev(logp[order]), None if left is None else _dev(left[order]))
    at = torch.from_numpy(first).to(DEV)
    for dtype in ("bf16", "f32"):
        x = _dev(rows, dtype)[torch.from_numpy(order).to(DEV)]
        loss = nq.distill_loss(P, x, _dev(w[order]))
        _check_distill(ids, logp, left, 1.0, rows, w, loss[at])
        assert torch.equal(loss[at][torch.from_numpy(order).to(DEV)].nan_to_num(-7.0), loss.nan_to_num(-7.0))
        loss2, grad = nq.distill_grads(P, x, _dev(w[order]))
        _check_distill(ids, logp, left, 1.0, rows, w, loss2[at], grad[at], dtype)


@gpu
@pytest.mark.parametrize("tau", [2.0 ** -20, 2.0 ** 20])
@pytest.mark.parametrize("V,k", [(300, 8), (9001, 40)])
def test_temperatures_at_both_limits(V, k, tau):
    """The coldest softmax is one token's (or none's beside it), the hottest even; a weight of the temperature keeps
    the gradient's scale."""
    T = 4
    w = np.full(T, min(tau, 1.0), np.float32)
    for dtype in ("f32", "bf16"):
        z, s = _rows(f"limits/{V}/z", T, V, dtype), _rows(f"limits/{V}/s", T, V, dtype)
        s[1] = z[1]
        s[2, :5] = s[2].max() + 1.0  # several that share the largest value
        _check_top(z, k, tau, nq.logits_top(_dev(z, dtype), k, temperature=tau))
        for rest in (True, False):
            ids, logp, left = _record(f"limits/{V}", T, V, k, tau, rest)
            P = nq.Teacher(_dev(ids), _dev(logp), None if left is None else _dev(left), tau)
            loss, grad = nq.distill_grads(P, _dev(s, dtype), _dev(w))
            _check_distill(ids, logp, left, tau, s, w, loss, grad, dtype)
            _check_distill(ids, logp, left, tau, s, w, nq.distill_loss(P, _dev(s, dtype), _dev(w)))


@gpu
@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("V,k", [(500, 7), (5003, 60), (40001, 300)])
def test_listed_gradients_are_those_of_exact_probabilities(V, k, rest):
    """The listed probabilities and their sums are formed in fp64, so a listed token's gradient is off by the rest's sum
    alone, w / tau * total q q_rest d, and by the rounding of the result."""
    T, tau = 3, 1.3
    ids, logp, left = _record(f"listed/{V}", T, V, k, tau, rest)
    ids[0, 4] = ids[0, 2]
    s = _rows(f"listed/{V}/s", T, V, "f32")
    P = nq.Teacher(_dev(ids), _dev(logp), None if left is None else _dev(left), tau)
    grad = _host(nq.distill_grads(P, _dev(s))[1])
    # the call's temperature is an fp32 number, 3.7e-8 below 1.3, and every gradient is in proportion to 1 / temperature:
    # 0.6 of the rounding that the bound leaves the result
    tau = float(np.float32(tau))
    want = D.distill_ref(ids, logp, left, tau, s)[1]
    for t in range(T):
        x = s[t].astype(np.float64) / tau
        listed = np.zeros(V, bool)
        listed[ids[t]] = True
        d = D.exp_error(x, listed, THREADS)
        e = np.exp(x - x.max())
        q, away = e / e.sum(), e[~listed].sum() / e.sum()
        total = 1.0 if left is None else np.exp(logp[t].astype(np.float64)).sum() + np.exp(float(left[t]))
        tol = (total * q * away * d + 1e-14) / tau + EPS * np.abs(want[t])
        assert (np.abs(grad[t] - want[t]) <= tol)[listed].all(), t


@gpu
def test_logits_of_more_than_2_to_31_elements():
    """Rows far behind, at offsets that 32 bits do not hold: eight rows repeated give their results again."""
    V, n, k = 131072, 2100, 9
    T = 8 * n
    assert T * V > 2 ** 31
    rows = _rows("far", 8, V, "bf16")
    x = _dev(rows, "bf16").repeat(n, 1)
    top = nq.logits_top(x, k)
    _check_top(rows, k, 1.0, nq.Teacher(top.ids[-8:].contiguous(), top.logp[-8:].contiguous(), top.rest[-8:].contiguous()))
    ids, logp, left = _record("far", 8, V, k, 1.0)
    P = nq.Teacher(_dev(np.tile(ids, (n, 1))), _dev(np.tile(logp, (n, 1))), _dev(np.tile(left, n)))
    _check_distill(ids, logp, left, 1.0, rows, None, nq.distill_loss(P, x)[-8:])
    loss, grad = nq.distill_grads(P, x, dlogits=x)
    _check_distill(ids, logp, left, 1.0, rows, None, loss[-8:], grad[-8:], "bf16")
    for t in (T // 2 // 8 * 8, T - 16):
        assert torch.equal(top.ids[t:t + 8], top.ids[-8:]) and torch.equal(grad[t:t + 8], grad[-8:])
