"""Newton-Schulz orthogonalisation against the fp64 reference.

Tolerances.  A shorter side up to 64 is fp64 throughout: one rounding of the
result, 2^-24 (fp32) or 2^-8 (bf16) of each value, beside fp64 errors.  Those
start at 2^-53 n and grow by at most a^2 = 11.9 a step on the Gram matrix:
11.9^5 * 1e-15 < 1e-8 of the largest value.
A longer shorter side rounds four operands a step (x in G, G, B and x again) to
u = 2^-11 (one fp16 term) or 2^-21 (two).  A rounding error E of B adds E X, of
size u |B|_F |X|_2 <= u * 2.8 sqrt(p) * 1.25, beside a result of 0.7 sqrt(p) or
more once singular values are near one: at most 5 u; the same holds for the
other three.  Independent over steps * 4 roundings: 5 u sqrt(4 steps).  fp32
sums of up to n products add 4 sqrt(n) 2^-24 each, likewise, and the result's
own rounding comes last."""
import ctypes

import numpy as np
import pytest
import torch

import synth
from oracle import adapters as A

nq = pytest.importorskip("sub_bit_weight_amd")

DEV = "cuda:0"
DUMMY = 0x100000
NS = nq.NEWTON_SCHULZ
gpu = pytest.mark.gpu


def _gradient(tag, batch, rows, cols):
    """A few strong directions over a floor, rows and columns of uneven size."""
    k = max(1, min(rows, cols) // 8)
    out = np.empty((batch, rows, cols), dtype=np.float32)
    for i in range(batch):
        t = f"ortho/{tag}/{i}"
        u = synth.normal_f32(t + "/u", (rows, k)) * np.exp(-4.0 * np.arange(k) / k)
        out[i] = u @ synth.normal_f32(t + "/v", (k, cols)) / np.sqrt(k) + 0.5 * synth.normal_f32(t + "/n", (rows, cols))
        out[i] *= 1e-3 * np.exp(0.5 * synth.normal_f32(t + "/r", (rows, 1))) * np.exp(0.5 * synth.normal_f32(t + "/c", (1, cols)))
    return out


def _check(got, want, steps, out, shape):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    p, q = min(shape), max(shape)
    last = 2.0 ** -24 if out == torch.float32 else 2.0 ** -8
    d, norm = np.abs(got - want), np.linalg.norm(want)
    if p <= 64:
        assert (d <= last * np.abs(want) + 1e-8 * np.abs(want).max()).all(), d.max()
    else:
        u = 2.0 ** -11 if out == torch.bfloat16 else 2.0 ** -21
        tol = (5 * u + 4 * np.sqrt(3 * q) * 2.0 ** -24) * np.sqrt(4 * steps) + last
        err = np.linalg.norm(got - want) / norm
        assert err <= tol, (err, tol)
        # no single value is off by more than 40 such errors of the average value
        assert (d <= 40 * tol * np.maximum(norm / np.sqrt(want.size), np.abs(want))).all(), d.max()


# ---------------------------------------------------------------- without a GPU


def test_reference_maps_singular_values():
    x = _gradient("sv", 1, 12, 20)[0]
    u, s, vt = np.linalg.svd(x.astype(np.float64), full_matrices=False)
    s /= np.sqrt((s * s).sum())
    for _ in range(3):
        s = NS[0] * s + NS[1] * s ** 3 + NS[2] * s ** 5
    assert np.allclose(A.orthogonalize_ref(x, 3, NS), (u * s) @ vt, atol=1e-12)
    assert np.allclose(A.orthogonalize_ref(x.T, 3, NS), A.orthogonalize_ref(x, 3, NS).T, atol=1e-12)


def _call(x=DUMMY, xd=nq.NQ_F32, batch=2, rows=8, cols=12, ldx=12, stride=96, steps=5, co=NS, y=DUMMY, yd=nq.NQ_F32,
          ws=DUMMY, wsb=1 << 40):
    return nq.lib().nq_orthogonalize(x, xd, batch, rows, cols, ldx, stride, steps, *co, y, yd, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), nq.NQ_ERR_ARG), (dict(rows=0), nq.NQ_ERR_ARG), (dict(cols=-1), nq.NQ_ERR_ARG),
    (dict(batch=65536), nq.NQ_ERR_UNSUPPORTED), (dict(rows=65537, cols=65, ldx=65), nq.NQ_ERR_UNSUPPORTED),
    (dict(rows=4, cols=(1 << 24) + 1, ldx=1 << 25), nq.NQ_ERR_UNSUPPORTED),
    (dict(xd=7), nq.NQ_ERR_ARG), (dict(yd=2), nq.NQ_ERR_ARG), (dict(x=None), nq.NQ_ERR_ARG), (dict(y=None), nq.NQ_ERR_ARG),
    (dict(x=DUMMY + 2), nq.NQ_ERR_ARG), (dict(y=DUMMY + 2), nq.NQ_ERR_ARG), (dict(yd=nq.NQ_BF16, y=DUMMY + 1), nq.NQ_ERR_ARG),
    (dict(ldx=11), nq.NQ_ERR_ARG), (dict(stride=-96), nq.NQ_ERR_ARG), (dict(steps=0), nq.NQ_ERR_ARG),
    (dict(steps=65), nq.NQ_ERR_ARG), (dict(co=(4.0, -4.775, 2.0315)), nq.NQ_ERR_ARG),
    (dict(co=(float("nan"), 0.0, 0.0)), nq.NQ_ERR_ARG), (dict(co=(2.0, 0.0, 0.0)), nq.NQ_ERR_ARG),
    (dict(co=(-3.0, 2.0, 0.0)), nq.NQ_ERR_ARG), (dict(co=(1.5625 * 2.0 ** 600, -2.0 ** 600, 2.0 ** -10), ws=None), nq.NQ_ERR_ARG), (dict(ws=None), nq.NQ_ERR_WORKSPACE), (dict(wsb=64), nq.NQ_ERR_WORKSPACE),
    (dict(ws=DUMMY + 4), nq.NQ_ERR_ARG),
])
def test_rejects_bad_args(kw, status):
    assert _call(**kw) == status
    assert nq.last_error() != ""


@pytest.mark.parametrize("co", [NS, (1.5, -0.5, 0.0), (1.875, -1.25, 0.375), (0.5, 0.0, 0.0), (-1.5, 0.5, 0.0)])
def test_usual_coefficients_pass_the_range_check(co):
    assert _call(co=co, ws=None) == nq.NQ_ERR_WORKSPACE  # the next check


@pytest.mark.parametrize("cc", [0.0, 1e-16, -1e-17, 1e-20, -1e-300, 5e-324])
@pytest.mark.parametrize("ca,cb", [(15.625, -10.0), (4.0, -3.2), (-4.0, 3.2)])
def test_rejects_an_interior_maximum_beside_a_tiny_quintic_term(ca, cb, cc):
    """All three leave 1.25 inside (at s = 0.72 or 0.65) although their ends do not."""
    assert _call(co=(ca, cb, cc), ws=None) == nq.NQ_ERR_ARG
    assert _call(co=(1.5, -0.5, cc), ws=None) == nq.NQ_ERR_WORKSPACE  # the next check


FORMS = [dict(rows=60, cols=100, ldx=100), dict(rows=100, cols=200, ldx=200), dict(rows=600, cols=700, ldx=700),
         dict(rows=600, cols=700, ldx=700, yd=nq.NQ_BF16)]  # fp64, two terms twice, one or two


def _chebyshev(f):
    """f * 1.25 * T5(s / 1.25): touches +-1.25 f five times, with a slope of 25 f at 1.25."""
    return (5.0 * f, -12.8 * f, 6.5536 * f)


@pytest.mark.parametrize("form", FORMS, ids=str)
def test_coefficients_leave_room_for_roundings(form):
    def call(co, steps=64):
        return _call(co=co, steps=steps, ws=None, **form)
    for co in (NS, (1.5, -0.5, 0.0), (1.875, -1.25, 0.375), (1.0, 0.0, 0.0), (3.7418, -5.5913, 2.3037), _chebyshev(0.9)):
        assert call(co) == nq.NQ_ERR_WORKSPACE, co  # the next check
    # 1.25 (1 - 1e-15) in exact arithmetic; roundings leave it, and grow 25 times a step from there
    assert call(_chebyshev(1 - 1e-15)) == nq.NQ_ERR_ARG and "roundings" in nq.last_error()
    for steps in (1, 2, 64):
        assert call(_chebyshev(0.999), steps=steps) == nq.NQ_ERR_WORKSPACE


def test_workspace_query():
    lib = nq.lib()
    assert lib.nq_orthogonalize_workspace_bytes(1, 16, 4096, nq.NQ_F32) > 0
    assert lib.nq_orthogonalize_workspace_bytes(1, 0, 4096, nq.NQ_F32) == 0
    assert lib.nq_orthogonalize_workspace_bytes(1, 16, 16, 9) == 0
    one, two = (lib.nq_orthogonalize_workspace_bytes(1, 512, 1024, d) for d in (nq.NQ_BF16, nq.NQ_F32))
    assert two > one >= 512 * 1024 * 4


def test_binding_refuses_host_tensors_and_shapes():
    with pytest.raises(ValueError):
        nq.orthogonalize(torch.zeros(4, 4))
    with pytest.raises(ValueError):
        nq.orthogonalize(torch.zeros(4))


# ---------------------------------------------------------------- GPU


SMALL = [(1, 1), (1, 9), (5, 3), (16, 256), (17, 300), (33, 1025), (64, 64), (64, 129), (500, 33), (2050, 48), (130, 2), (63, 640)]
LARGE = [(65, 65), (65, 200), (130, 100), (257, 300), (300, 257), (128, 1030), (700, 400), (65, 9000), (4100, 190)]


@gpu
@pytest.mark.parametrize("shape", SMALL + LARGE, ids=str)
@pytest.mark.parametrize("xd,out", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                    (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
def test_orthogonalize(shape, xd, out):
    x = torch.from_numpy(_gradient(f"{shape}", 2, *shape)).to(DEV).to(xd)
    y = nq.orthogonalize(x, out_dtype=out)
    assert y.shape == x.shape and y.dtype == out
    for i in range(2):
        _check(y[i], A.orthogonalize_ref(x[i].double().cpu().numpy(), 5, NS), 5, out, shape)


@gpu
@pytest.mark.parametrize("steps,co", [(1, NS), (3, NS), (8, (1.5, -0.5, 0.0)), (4, (1.875, -1.25, 0.375))])
@pytest.mark.parametrize("shape", [(24, 200), (90, 150)], ids=str)
def test_steps_and_coefficients(shape, steps, co):
    # near-orthogonal rows, so that every step's singular values are of the size of the largest
    x = np.linalg.qr(synth.normal_f32("ortho/steps", (shape[1], shape[1])).astype(np.float64))[0][:shape[0]]
    x = torch.from_numpy((x + 0.01 * synth.normal_f32("ortho/steps/n", shape)).astype(np.float32)).to(DEV)
    y = nq.orthogonalize(x, steps=steps, coeffs=co)
    _check(y, A.orthogonalize_ref(x.double().cpu().numpy(), steps, co), steps, torch.float32, shape)


@gpu
@pytest.mark.parametrize("batch,rows,cols,out", [(4, 2048, 2100, torch.bfloat16), (8, 1300, 1411, torch.bfloat16),
                                                 (4, 1900, 2048, torch.float32)])
def test_large_matrices(batch, rows, cols, out):
    """Enough 256 x 256 tiles to fill the chip, also where the symmetric products skip half of theirs."""
    x = torch.randn(batch, rows, cols, device=DEV, generator=torch.Generator(device=DEV).manual_seed(7))
    x = x * torch.exp(0.5 * torch.randn(batch, rows, 1, device=DEV))
    y = nq.orthogonalize(x, out_dtype=out)
    for i in range(batch):
        w = x[i].double()
        w = w / torch.linalg.vector_norm(w)
        for _ in range(5):
            g = w @ w.T
            w = NS[0] * w + NS[1] * (g @ w) + NS[2] * (g @ (g @ w))
        _check(y[i], w.cpu().numpy(), 5, out, (rows, cols))


@gpu
@pytest.mark.parametrize("shape", [(16, 100), (100, 120)], ids=str)
def test_zero_and_non_finite_matrices_stay_apart(shape):
    x = _gradient(f"nan/{shape}", 5, *shape)
    clean = nq.orthogonalize(torch.from_numpy(x).to(DEV))
    x[1] = 0
    x[2, 3, 5] = np.inf
    x[3, 0, 0] = np.nan
    y = nq.orthogonalize(torch.from_numpy(x).to(DEV))
    assert torch.equal(y[0], clean[0]) and torch.equal(y[4], clean[4])
    assert not y[1].any() and torch.isnan(y[2]).all() and torch.isnan(y[3]).all()


@gpu
@pytest.mark.parametrize("shape", [(16, 100), (100, 120)], ids=str)
@pytest.mark.parametrize("power", [-126, -70, 70, 110])
def test_any_magnitude(shape, power):
    """A power of two times the matrix gives the same result: no square leaves its range."""
    x = _gradient(f"mag/{shape}", 1, *shape)[0]
    x = np.ldexp(np.sign(x), np.clip(np.round(np.log2(np.abs(x) + 1e-9)), -16, 8).astype(int)).astype(np.float32)
    a = nq.orthogonalize(torch.from_numpy(x).to(DEV))
    b = nq.orthogonalize(torch.from_numpy(np.ldexp(x, power).astype(np.float32)).to(DEV))
    if power > -126:  # the smallest entries are subnormal there and lose bits
        assert torch.equal(a, b)
    assert torch.isfinite(b).all() and float((a - b).norm() / a.norm()) <= 2.0 ** -7


@gpu
@pytest.mark.parametrize("shape", [(20, 90), (150, 70)], ids=str)
def test_views_workspace_and_streams(shape):
    rows, cols = shape
    x = torch.from_numpy(_gradient(f"view/{shape}", 3, rows, cols)).to(DEV)
    want = nq.orthogonalize(x)
    big = torch.full((rows, 3, cols + 7), float("nan"), device=DEV)
    view = big.permute(1, 0, 2)[:, :, 2:2 + cols]
    view.copy_(x)
    ws = torch.full((nq.orthogonalize_workspace_bytes(3, rows, cols),), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(nq.orthogonalize(view, workspace=ws), want)
    assert torch.equal(nq.orthogonalize(view[1]), want[1])
    torch.cuda.synchronize()
    outs = [nq.orthogonalize(x, stream=torch.cuda.Stream()) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    with pytest.raises(nq.NqError):
        nq.orthogonalize(x, workspace=ws[:128])
    with pytest.raises(ValueError):
        nq.orthogonalize(x, workspace=ws.cpu())
    with pytest.raises(ValueError):
        nq.orthogonalize(x.transpose(1, 2))
    with pytest.raises(ValueError):
        nq.orthogonalize(x, out_dtype=torch.float16)


@gpu
def test_captured_training_step_of_adapters():
    """Forward, gradients and update as they are used together: eager against fp64, and a captured
    step replayed beside eager ones."""
    T, n, r, d_in, d_out = 150, 3, 8, 96, 130
    g = torch.Generator(device=DEV).manual_seed(3)
    a0 = torch.randn(n, r, d_in, device=DEV, generator=g) / d_in ** 0.5
    b0 = torch.randn(n, d_out, r, device=DEV, generator=g) / r ** 0.5
    scale = torch.ones(n, device=DEV)
    x = torch.randn(T, d_in, device=DEV, generator=g)
    target = torch.randn(T, d_out, device=DEV, generator=g)
    ids = torch.randint(-1, n, (T,), device=DEV, generator=g, dtype=torch.int32)
    pool = nq.Lora(a0.clone(), b0.clone(), scale)

    def step():
        y = nq.lora_linear(pool, x, ids)
        _, da, db = nq.lora_grads(pool, x, y - target, ids)
        pool.a.sub_(nq.orthogonalize(da), alpha=0.02)
        pool.b.sub_(nq.orthogonalize(db), alpha=0.02)
        return y
    y = step()
    w = lambda t: t.double().cpu().numpy()  # noqa: E731
    yw = A.lora_linear_ref(w(a0), w(b0), w(scale), w(x), ids.cpu().numpy())
    _, da, db = A.lora_grads_ref(w(a0), w(b0), w(scale), w(x), yw - w(target), ids.cpu().numpy())
    # fp32 sums of at most 3 T + d terms on the way: sqrt(n) 2^-24 of each value, times 4; a gradient that is off by
    # e changes its orthogonalisation by at most 3.5^5 e (the slope of the quintic at zero, five times)
    tol = 4 * np.sqrt(3 * T + d_out) * 2.0 ** -24
    assert np.linalg.norm(w(y) - yw) <= tol * np.linalg.norm(yw)
    for got, start, grad in ((pool.a, a0, da), (pool.b, b0, db)):
        want = np.stack([w(start)[i] - 0.02 * A.orthogonalize_ref(grad[i], 5, NS) for i in range(n)])
        assert np.linalg.norm(w(got) - want) <= 3.5 ** 5 * tol * 0.02 * np.sqrt(n * r) + 2.0 ** -24 * np.linalg.norm(want)

    eager = []
    pool.a.copy_(a0), pool.b.copy_(b0)
    for _ in range(4):
        eager.append((step(), pool.a.clone(), pool.b.clone()))
    pool.a.copy_(a0), pool.b.copy_(b0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = step()
    pool.a.copy_(a0), pool.b.copy_(b0)
    for yw, aw, bw in eager:
        torch.cuda.synchronize()
        graph.replay()
        nq.orthogonalize(x)  # eager work of the program's own between replays
        torch.cuda.synchronize()
        assert torch.equal(y, yw) and torch.equal(pool.a, aw) and torch.equal(pool.b, bw)


# ---------------------------------------------------------------- many steps, short sides


def _definition(x, steps, co):
    """The iteration as written, in 80 bits."""
    x = x.astype(np.longdouble)
    x = x.T if x.shape[0] > x.shape[1] else x
    x = x / np.sqrt((x * x).sum())
    for _ in range(steps):
        g = x @ x.T
        gx = g @ x
        x = co[0] * x + co[1] * gx + co[2] * (g @ gx)
    return x


def _deficient(kind, p, q):
    """p x q of a known rank or spectrum, exact in bf16 (but for the spectrum)."""
    g = synth.rng(f"ortho/deficient/{kind}/{p}/{q}")
    if kind == "six decades":
        u, v = np.linalg.qr(g.standard_normal((p, p)))[0], np.linalg.qr(g.standard_normal((q, p)))[0]
        return ((u * 10.0 ** (-6.0 * np.arange(p) / (p - 1))) @ v.T).astype(np.float32)
    if kind == "duplicated row":
        x = g.integers(-8, 9, (p, q))
        x[p - 1] = x[p // 2]
    else:
        r = {"rank 1": 1, "a quarter": max(1, p // 4), "three quarters": 3 * p // 4}[kind]
        u = np.zeros((p, r), dtype=int)
        u[np.arange(p), g.integers(0, r, p)] = 1  # each row one of r, times a sign: small integers
        x = (u * g.choice([-1, 1], (p, 1))) @ g.integers(-8, 9, (r, q))
    return x.astype(np.float32)


KINDS = ["rank 1", "a quarter", "three quarters", "duplicated row", "six decades"]


@gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", [(5, 40), (16, 600), (200, 16), (33, 500), (130, 48), (64, 300)], ids=str)
@pytest.mark.parametrize("steps,co", [(s, NS) for s in (5, 6, 8, 10, 12, 20)] + [(17, (1.5, -0.5, 0.0)), (40, (1.5, -0.5, 0.0))])
def test_many_steps_of_deficient_matrices(kind, shape, steps, co):
    """Gradients of fewer tokens than rows.  An fp64 evaluation of the definition rounds values of size one
    to 2^-53, in sums of p products (4 sqrt(p) of them); a direction without a singular value of its own
    multiplies what it gets of that by ca a step, a geometric sum of ca^steps * ca / (ca - 1) at most, while
    the result's norm is 0.7 or more.  1e-8 and the last rounding as at five steps."""
    p, q = min(shape), max(shape)
    x = _deficient(kind, p, q)
    x = x.T.copy() if shape[0] > shape[1] else x
    y = nq.orthogonalize(torch.from_numpy(x).to(DEV), steps=steps, coeffs=co).double().cpu().numpy()
    want = _definition(x, steps, co)
    want = np.asarray(want.T if shape[0] > shape[1] else want, dtype=np.float64)
    noise = 4 * np.sqrt(p) * 2.0 ** -53 * co[0] ** steps * co[0] / (co[0] - 1) / 0.7
    assert np.linalg.norm(y - want) <= (2.0 ** -24 + 1e-8 + noise) * np.linalg.norm(want)


@gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", [(16, 600), (200, 16), (64, 300)], ids=str)
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_the_most_steps_stay_in_range(kind, shape, out):
    """64 steps: no singular value leaves [0, 1.25], which the coefficients promise, beyond the result's rounding."""
    p, q = min(shape), max(shape)
    x = _deficient(kind, p, q)
    x = x.T.copy() if shape[0] > shape[1] else x
    y = nq.orthogonalize(torch.from_numpy(x).to(DEV), steps=64, out_dtype=out).double().cpu().numpy()
    last = 2.0 ** -24 if out == torch.float32 else 2.0 ** -8
    assert np.isfinite(y).all()
    assert np.linalg.norm(y, 2) <= 1.25 * (1 + last * np.sqrt(p))
    if kind == "six decades":  # no direction without a singular value: rounding errors grow by 1e6 at most, then stay
        want = _definition(x, 64, NS)
        want = np.asarray(want.T if shape[0] > shape[1] else want, dtype=np.float64)
        assert np.linalg.norm(y - want) <= (last + 1e-8) * np.linalg.norm(want)


@gpu
@pytest.mark.parametrize("shape", [(16, 100), (90, 40)], ids=str)
def test_many_steps_of_a_batch(shape):
    """Zero and non-finite matrices, views, a dirty workspace, bf16 and a captured call at more steps than one Gram matrix serves."""
    rows, cols = shape
    x = _gradient(f"batch/{shape}", 5, rows, cols)
    steps = 13
    want = nq.orthogonalize(torch.from_numpy(x).to(DEV), steps=steps)
    for i in range(5):
        w = _definition(x[i], steps, NS)
        w = np.asarray(w.T if rows > cols else w, dtype=np.float64)
        # the smallest singular value is 1e-2 or more of the largest
        assert np.linalg.norm(want[i].double().cpu().numpy() - w) <= (2.0 ** -24 + 1e-8) * np.linalg.norm(w)
    x[1] = 0
    x[2, 3, 5] = np.inf
    x[3, 0, 0] = np.nan
    big = torch.full((rows, 5, cols + 7), float("nan"), device=DEV)
    view = big.permute(1, 0, 2)[:, :, 2:2 + cols]
    view.copy_(torch.from_numpy(x))
    ws = torch.full((nq.orthogonalize_workspace_bytes(5, rows, cols),), 255, dtype=torch.uint8, device=DEV)
    y = nq.orthogonalize(view, steps=steps, workspace=ws)
    assert torch.equal(y[0], want[0]) and torch.equal(y[4], want[4])
    assert not y[1].any() and torch.isnan(y[2]).all() and torch.isnan(y[3]).all()
    half = torch.from_numpy(x[4]).to(DEV).to(torch.bfloat16)
    assert torch.equal(nq.orthogonalize(half, steps=steps), nq.orthogonalize(half.float(), steps=steps).to(torch.bfloat16))
    src = torch.from_numpy(x[0]).to(DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = nq.orthogonalize(src, steps=steps)
    for i in (0, 4, 0):
        src.copy_(torch.from_numpy(x[i]))
        eager = nq.orthogonalize(src, steps=steps)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager) and torch.equal(y, want[i])


# ---------------------------------------------------------------- bf16 results


@gpu
@pytest.mark.parametrize("steps", [5, 12])
@pytest.mark.parametrize("shape", [(65, 300), (66, 4096), (300, 130), (256, 600), (900, 511)], ids=str)
def test_bf16_results_of_smaller_matrices_lose_their_rounding_alone(shape, steps):
    """A result z rounded to bf16 is off by at most half a step of it and |z - z*|.  So what is left of each
    value's error beyond half a step of z* is at most |z - z*| and the step's growth, whose norm is that
    of an fp32 result: two-term products as above (twice, for values that cross a power of two)."""
    p, q = min(shape), max(shape)
    x = synth.normal_f32(f"ortho/bf16/{shape}", shape) * np.exp(0.3 * synth.normal_f32(f"ortho/bf16r/{shape}", (shape[0], 1)))
    y = nq.orthogonalize(torch.from_numpy(x.astype(np.float32)).to(DEV), steps=steps, out_dtype=torch.bfloat16)
    want = A.orthogonalize_ref(x.astype(np.float32), steps, NS)
    tol = (5 * 2.0 ** -21 + 4 * np.sqrt(3 * q) * 2.0 ** -24) * np.sqrt(4 * steps)
    half = 2.0 ** (np.floor(np.log2(np.abs(want) + 1e-30)) - 8)
    beyond = np.maximum(np.abs(y.double().cpu().numpy() - want) - half, 0)
    assert np.linalg.norm(beyond) <= 2 * tol * np.linalg.norm(want)


@gpu
@pytest.mark.parametrize("shape,out,f", [((48, 200), torch.float32, 0.999999), ((130, 200), torch.float32, 0.999),
                                         ((300, 200), torch.bfloat16, 0.999), ((520, 600), torch.bfloat16, 0.999)])
def test_coefficients_near_the_edge_stay_in_range(shape, out, f):
    """The steepest polynomials that are accepted, for the most steps."""
    x = torch.from_numpy(synth.normal_f32(f"ortho/edge/{shape}", shape)).to(DEV)
    y = nq.orthogonalize(x, steps=64, coeffs=_chebyshev(f), out_dtype=out).double().cpu().numpy()
    assert np.isfinite(y).all() and np.linalg.norm(y, 2) <= 1.3125


@gpu
@pytest.mark.parametrize("steps,co", [(6, NS), (12, NS), (20, NS), (40, (1.875, -1.25, 0.375))])
@pytest.mark.parametrize("shape", [(512, 600), (700, 520)], ids=str)
def test_bf16_results_after_many_steps_lose_their_rounding_alone(shape, steps, co):
    """As above, from 512 rows on, where only few steps take one-term operands."""
    p, q = min(shape), max(shape)
    x = synth.normal_f32(f"ortho/bf16/{shape}", shape).astype(np.float32)
    y = nq.orthogonalize(torch.from_numpy(x).to(DEV), steps=steps, coeffs=co, out_dtype=torch.bfloat16)
    want = A.orthogonalize_ref(x, steps, co)
    tol = (5 * 2.0 ** -21 + 4 * np.sqrt(3 * q) * 2.0 ** -24) * np.sqrt(4 * steps)
    half = 2.0 ** (np.floor(np.log2(np.abs(want) + 1e-30)) - 8)
    beyond = np.maximum(np.abs(y.double().cpu().numpy() - want) - half, 0)
    assert np.linalg.norm(beyond) <= 2 * tol * np.linalg.norm(want)


@gpu
def test_many_steps_of_large_bf16_batches():
    """The form with one transposed copy: a dirty workspace, zero and NaN matrices beside others, tall and wide, captured."""
    x = synth.normal_f32("ortho/copies", (3, 513, 580)).astype(np.float32)
    xd = torch.from_numpy(x).to(DEV)
    want = nq.orthogonalize(xd, steps=9, out_dtype=torch.bfloat16)
    both = nq.orthogonalize(xd, steps=9).to(torch.bfloat16)  # two copies
    # the same operands and products in the same order: the last rounding alone differs
    assert torch.equal(want, both)
    xd[1] = 0
    xd[2, 1, 2] = float("nan")
    ws = torch.full((nq.orthogonalize_workspace_bytes(3, 580, 513, torch.bfloat16),), 255, dtype=torch.uint8, device=DEV)
    y = nq.orthogonalize(xd.transpose(1, 2).contiguous(), steps=9, out_dtype=torch.bfloat16, workspace=ws).transpose(1, 2)
    assert torch.equal(y[0], want[0]) and not y[1].any() and torch.isnan(y[2]).all()
    src = torch.from_numpy(x[0]).to(DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = nq.orthogonalize(src, steps=9, out_dtype=torch.bfloat16)
    for i in (0, 1, 2, 0):
        src.copy_(torch.from_numpy(x[i]))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, nq.orthogonalize(src, steps=9, out_dtype=torch.bfloat16))
