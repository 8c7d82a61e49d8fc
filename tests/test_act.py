"""The packed linear's epilogue and its gradients, against the fp64 reference.

The epilogue's tolerance takes the layer's own output as given (nq_lrb_linear's, fp32: the same products and sums)
and counts the epilogue's roundings (oracle.distill.epilogue_ref, act_grads_ref) and that of the result, half a step
of its type.  Against the layer's fp64 oracle the bars are the layer's own (tests/gpu_cases.py), plus the rounding of
the result and the roundings of the epilogue."""
import ctypes

import numpy as np
import pytest
import torch

import synth
from oracle import distill as D
from oracle import nq_oracle as O
from tests import gpu_cases as G

nq = pytest.importorskip("sub_bit_weight_amd")

DEV = "cuda:0"
DUMMY = 0x100000
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
gpu = pytest.mark.gpu


# ---------------------------------------------------------------- the reference


@pytest.mark.parametrize("act", ACTS)
def test_reference_derivative_matches_differences(act):
    z = np.linspace(-6, 6, 241) + 0.013
    num = (D.act_ref(act, z + 1e-5)[0] - D.act_ref(act, z - 1e-5)[0]) / 2e-5
    assert np.allclose(D.act_ref(act, z)[1], num, atol=1e-9)


def test_reference_activations_are_torchs():
    z = torch.linspace(-7, 7, 301, dtype=torch.float64)
    f = torch.nn.functional
    for act, want in (("relu", f.relu(z)), ("gelu", f.gelu(z)), ("gelu_tanh", f.gelu(z, approximate="tanh")),
                      ("silu", f.silu(z))):
        assert np.allclose(D.act_ref(act, z.numpy())[0], want.numpy(), rtol=1e-12, atol=1e-14), act


# ---------------------------------------------------------------- refusals (no GPU)


def _layer(**kw):
    d = dict(d_out=64, d_in=64, r=32, u_bits=DUMMY, ldu=64, vt_bits=DUMMY, ldv=32, s1=DUMMY, s2=DUMMY)
    d.update(kw)
    return nq.nq_lrb(**d)


def _linear(L=None, x=DUMMY, xd=nq.NQ_BF16, T=20, y=2 * DUMMY, yd=nq.NQ_BF16, ws=DUMMY, wsb=1 << 40, null=False, **kw):
    e = nq.nq_epilogue(**{**dict(act=0), **kw})
    L = L or _layer()
    return nq.lib().nq_lrb_linear_act(ctypes.byref(L), x, xd, T, None if null else ctypes.byref(e), y, yd, ws, wsb, None)


def _grads(act=4, z=DUMMY, zd=1, mul=3 * DUMMY, md=1, dy=5 * DUMMY, dyd=1, T=300, d=64, dz=7 * DUMMY, dzd=1, dmul=9 * DUMMY,
           dmd=1, db=DUMMY, ws=DUMMY, wsb=1 << 30):
    return nq.lib().nq_act_grads(act, z, zd, mul, md, dy, dyd, T, d, dz, dzd, dmul, dmd, db, ws, wsb, None)


@pytest.mark.parametrize("kw", [
    dict(null=True), dict(act=-1), dict(act=5), dict(T=0), dict(x=None), dict(xd=4), dict(y=None), dict(yd=2),
    dict(y=DUMMY + 1), dict(yd=0, y=DUMMY + 2), dict(bias=DUMMY + 2), dict(mul=DUMMY + 1, mul_dtype=1),
    dict(mul=DUMMY, mul_dtype=3), dict(residual=DUMMY + 2, residual_dtype=0), dict(residual=DUMMY, residual_dtype=-1),
    dict(z=DUMMY, z_dtype=9), dict(z=DUMMY + 1, z_dtype=1), dict(z=2 * DUMMY, z_dtype=1),
    dict(z=DUMMY, z_dtype=1, mul=DUMMY, mul_dtype=1), dict(mul=2 * DUMMY, mul_dtype=0),
    dict(residual=2 * DUMMY, residual_dtype=0), dict(y=DUMMY), dict(y=DUMMY, residual=DUMMY, residual_dtype=1),
    dict(z=DUMMY, z_dtype=1), dict(ws=DUMMY + 4), dict(L=_layer(d_in=0)), dict(L=_layer(ldu=1))])
def test_linear_rejects(kw):
    assert _linear(**kw) == nq.NQ_ERR_ARG and nq.last_error() != ""


def test_linear_rejects_workspace_and_sizes():
    assert _linear(ws=None) == nq.NQ_ERR_WORKSPACE
    assert _linear(wsb=4) == nq.NQ_ERR_WORKSPACE
    assert _linear(T=(1 << 24) + 1) == nq.NQ_ERR_UNSUPPORTED
    q = nq.lib().nq_lrb_act_workspace_bytes
    assert q(ctypes.byref(_layer(r=0)), 3) == 0 and q(ctypes.byref(_layer()), 0) == 0
    assert q(ctypes.byref(_layer()), 8) == 0  # one workgroup needs none
    for T in (1, 8, 9, 1000):
        L = _layer(d_out=2000, ldu=2000)
        assert q(ctypes.byref(L), T) >= nq.lib().nq_lrb_workspace_bytes(ctypes.byref(L), T) > 0


@pytest.mark.parametrize("kw,status", [
    (dict(act=9), 1), (dict(T=0), 1), (dict(d=0), 1), (dict(T=(1 << 24) + 1), 2), (dict(d=(1 << 24) + 1), 2),
    (dict(dy=None), 1), (dict(dz=None), 1), (dict(z=None), 1), (dict(act=0, z=None), 1), (dict(mul=None), 1),
    (dict(zd=2), 1), (dict(md=-1), 1), (dict(dyd=7), 1), (dict(dzd=5), 1), (dict(dmd=3), 1), (dict(db=DUMMY + 2), 1),
    (dict(dy=DUMMY + 1), 1), (dict(dzd=0, dz=DUMMY + 2), 1), (dict(dmul=7 * DUMMY), 1), (dict(dz=5 * DUMMY, dzd=0), 1),
    (dict(dmul=3 * DUMMY, dmd=0), 1), (dict(dz=DUMMY, dzd=0), 1), (dict(ws=None), 3), (dict(wsb=1), 3), (dict(ws=DUMMY + 8), 1)])
def test_grads_reject(kw, status):
    assert _grads(**kw) == status and nq.last_error() != ""


def test_grads_workspace_query():
    q = nq.lib().nq_act_grads_workspace_bytes
    assert q(0, 4) == 0 and q(4, 0) == 0 and q(1 << 25, 1) == 0 and q(256, 9) == 0 and q(4096, 1000) >= 4000


# ---------------------------------------------------------------- GPU


def _act_layer(d_out, d_in, r):
    """A layer whose outputs are around one, and its oracle."""
    dev, ref, _ = G.latent_layer(G.tiny_config(f"act/{d_out}/{d_in}/{r}"), synth.LayerShape("act", d_out, d_in, r))
    for t, a, n in ((dev.s1, ref.s1, r), (dev.s2, ref.s2, d_in)):
        t.mul_(50.0 / np.sqrt(n))
        a[:] = t.cpu().numpy()
    return dev, ref


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _rand(tag, shape, dtype):
    return torch.from_numpy(synth.normal_f32(f"act/{tag}", shape)).to(DEV).to(dtype)


def _close(got, want, err, what):
    got, tol = _np(got), err + HALF[got.dtype] * np.abs(want)
    with np.errstate(invalid="ignore"):
        bad = ~((np.abs(got - want) <= tol) | (got == want) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], tol[bad][:4])


SHAPES = [(1, 1, 1), (200, 130, 70), (256, 256, 64), (1100, 130, 70), (1111, 1030, 517), (3000, 700, 520)]


@gpu
@pytest.mark.parametrize("T", [1, 3, 8, 9, 40, 200])
@pytest.mark.parametrize("d_out,d_in,r", SHAPES)
def test_linear_act(d_out, d_in, r, T):
    layer, ref = _act_layer(d_out, d_in, r)
    bias = _rand("bias", (d_out,), torch.float32)
    for i, act in enumerate(ACTS):
        for xd in ("bf16", "f32"):
            dt = TYPES[xd]
            x = _rand(f"x/{d_in}", (T, d_in), dt)
            mul, res = _rand("mul", (T, d_out), dt), _rand("res", (T, d_out), TYPES["f32" if i % 2 else xd])
            z = torch.empty(T, d_out, dtype=dt, device=DEV)
            v = nq.lrb_linear(layer, x)
            for kw in (dict(), dict(bias=bias, mul=mul, residual=res), dict(bias=bias, z=z), dict(mul=mul, z=z),
                       dict(residual=res, out_dtype=torch.bfloat16), dict(bias=bias, mul=mul, out_dtype=torch.float32)):
                y = nq.lrb_linear_act(layer, x, act=act, **kw)
                assert y.dtype == kw.get("out_dtype", dt)
                want, wz, err = D.epilogue_ref(_np(v), act, *[None if kw.get(n) is None else _np(kw[n])
                                                              for n in ("bias", "mul", "residual")])
                _close(y, want, err, (act, xd, list(kw)))
                if "z" in kw:
                    _close(z, wz, np.abs(wz) * D.EPS32, (act, "z"))
            # against the oracle of the whole layer: the layer's bar, a gated activation being at most 1.13-Lipschitz
            if T <= 40 or d_out < 300:
                y0 = O.linear_ref(ref, _np(x).astype(np.float32))
                want, _, err = D.epilogue_ref(y0, act, _np(bias), None, _np(res))
                y = nq.lrb_linear_act(layer, x, act=act, bias=bias, residual=res, out_dtype=torch.float32)
                bar = 1.2 * G.tol_for(T, xd) * np.linalg.norm(y0) + np.linalg.norm(err + D.EPS32 * np.abs(want))
                assert np.linalg.norm(_np(y) - want) <= bar, (act, xd)


@gpu
@pytest.mark.parametrize("T", [2, 30, 130])
def test_linear_act_in_place_and_given_outputs(T):
    layer, _ = _act_layer(1100, 600, 530)
    for dt in (torch.float32, torch.bfloat16):
        x, mul, res = _rand("ip/x", (T, 600), dt), _rand("ip/mul", (T, 1100), dt), _rand("ip/res", (T, 1100), dt)
        want = nq.lrb_linear_act(layer, x, "silu", mul=mul, residual=res)
        a, b = mul.clone(), res.clone()
        assert nq.lrb_linear_act(layer, x, "silu", mul=a, residual=res, y=a) is a and torch.equal(a, want)
        assert torch.equal(nq.lrb_linear_act(layer, x, "silu", mul=mul, residual=b, y=b), want)
        ws = torch.full((nq.lrb_act_workspace_bytes(layer, T) + 512,), 0x5A, dtype=torch.uint8, device=DEV)
        y = torch.full((T + 2, 1100), 3.0, dtype=dt, device=DEV)
        nq.lrb_linear_act(layer, x, "silu", mul=mul, residual=res, y=y[1:T + 1], workspace=ws[:-512])
        assert torch.equal(y[1:T + 1], want) and (y[0] == 3).all() and (y[T + 1] == 3).all() and (ws[-512:] == 0x5A).all()


@gpu
@pytest.mark.parametrize("T", [1, 5, 20])
def test_linear_act_of_infinite_and_extreme_values(T):
    """Large arguments of either sign reach the activations' limits; NaN in an operand stays at its element."""
    layer, _ = _act_layer(300, 40, 33)
    x = _rand("inf/x", (T, 40), torch.float32)
    bias = torch.zeros(300, device=DEV)
    bias[:12] = torch.tensor([1e4, -1e4, 1e30, -1e30, float("inf"), float("-inf"), float("nan"), 88.0, -88.0, -104.0, 30.0,
                              -30.0], device=DEV)
    mul, res = _rand("inf/mul", (T, 300), torch.float32), _rand("inf/res", (T, 300), torch.float32)
    mul[0, 20], res[T - 1, 30] = float("nan"), float("inf")
    v = _np(nq.lrb_linear(layer, x))
    for act in ACTS:
        got = _np(nq.lrb_linear_act(layer, x, act, bias=bias, mul=mul, residual=res))
        with np.errstate(all="ignore"):
            want, _, err = D.epilogue_ref(v, act, _np(bias), _np(mul), _np(res))
        ok = np.isfinite(want) & np.isfinite(err)
        assert (np.abs(got - want)[ok] <= (err + D.EPS32 * np.abs(want))[ok]).all(), act
        assert np.array_equal(np.isnan(got), np.isnan(want)), act


GRADS = [(1, 1), (3, 7), (17, 15), (130, 23), (5, 64), (64, 300), (65, 1117), (200, 257), (777, 1000), (2100, 96), (300, 4104)]


@gpu
@pytest.mark.parametrize("T,d", GRADS)
def test_act_grads(T, d):
    for act in ACTS:
        for dt in (torch.float32, torch.bfloat16):
            z, dy = 2 * _rand("g/z", (T, d), dt), _rand("g/dy", (T, d), dt)
            for mul in (None, _rand("g/mul", (T, d), dt)):
                dz, dmul, dbias = nq.act_grads(act, z, dy, mul=mul)
                wz, wm, wb, (ez, em, eb) = D.act_grads_ref(act, _np(z), _np(dy), None if mul is None else _np(mul))
                _close(dz, wz, ez, (act, "dz"))
                _close(dbias, wb, eb, (act, "dbias"))
                assert (dmul is None) == (mul is None)
                if mul is not None:
                    _close(dmul, wm, em, (act, "dmul"))
                again = nq.act_grads(act, z, dy, mul=mul)
                assert torch.equal(again[2], dbias) and torch.equal(again[0], dz)
                assert nq.act_grads(act, z, dy, mul=mul, bias=False)[2] is None


@gpu
def test_act_grads_mixed_types_in_place_and_strange_operands():
    T, d = 90, 513
    z, dy, mul = _rand("m/z", (T, d), torch.float32), _rand("m/dy", (T, d), torch.bfloat16), _rand("m/mul", (T, d), torch.float32)
    dz = torch.empty(T, d, device=DEV)
    dmul = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
    got = nq.act_grads("gelu", z, dy, mul=mul, dz=dz, dmul=dmul)
    wz, wm, wb, (ez, em, eb) = D.act_grads_ref("gelu", _np(z), _np(dy), _np(mul))
    assert got[0] is dz and got[1] is dmul
    _close(dz, wz, ez, "dz"), _close(dmul, wm, em, "dmul"), _close(got[2], wb, eb, "dbias")
    a, b = dy.float(), mul.clone()
    dz2, dmul2, _ = nq.act_grads("gelu", z, a, mul=b, dz=a, dmul=b)
    assert dz2 is a and dmul2 is b and torch.equal(a, dz)
    _close(b, wm, em, "dmul")
    c = z.clone()
    assert torch.equal(nq.act_grads("gelu", c, dy.float(), mul=mul, dz=c)[0], dz)
    # without z: act none and no gate
    dz3, none, db3 = nq.act_grads("none", None, dy)
    assert none is None and torch.equal(dz3, dy)
    _close(db3, _np(dy).sum(0), T * D.EPS32 * np.abs(_np(dy)).sum(0), "dbias")
    # a misaligned view, rows of padding that hold nothing
    flat = torch.zeros(T * d + 3, dtype=torch.bfloat16, device=DEV)
    flat[1:1 + T * d].copy_(dy.flatten())
    assert torch.equal(nq.act_grads("relu", z, flat[1:1 + T * d].view(T, d))[0], nq.act_grads("relu", z, dy)[0])
    z[3], dy[5] = float("nan"), 0.0
    dz4, _, db4 = nq.act_grads("silu", z, dy)
    assert torch.isnan(dz4[3]).all() and torch.isnan(db4).all() and (dz4[5] == 0).all() and torch.isfinite(dz4[6]).all()


@gpu
def test_act_grads_of_extreme_values():
    """Where a square or a cube of z leaves fp32, the derivatives have reached their limits."""
    z = torch.tensor([0.0, 30.0, 104.0, 1e4, 1e13, 1e19, 1.9e19, 1e20, 3e38], device=DEV)
    z = torch.cat((z, -z))[None].repeat(2, 1)
    for act in ACTS:
        for dt in (torch.float32, torch.bfloat16):
            zt, dy = z.to(dt), _rand("x/dy", tuple(z.shape), dt)
            dz, _, dbias = nq.act_grads(act, zt, dy)
            wz, _, wb, (ez, _, _) = D.act_grads_ref(act, _np(zt), _np(dy))
            # the lost parts' bound grows with z^2; the derivatives themselves are within 8 roundings of 0 or 1 there
            ez = np.minimum(ez, np.abs(_np(dy)) * 512 * D.EPS32)
            _close(dz, wz, ez, (act, dt))
            _close(dbias, wb, ez.sum(0) + 2 * D.EPS32 * np.abs(wz).sum(0), (act, dt))
    # x is the residual: a result of its own
    layer, _ = _act_layer(96, 96, 40)
    for T in (3, 20):
        x = _rand("x/res", (T, 96), torch.float32)
        want = nq.lrb_linear(layer, x) + x
        assert torch.equal(nq.lrb_linear_act(layer, x, residual=x), want)
        with pytest.raises(nq.NqError):
            nq.lrb_linear_act(layer, x, residual=x, y=x)


@gpu
def test_streams_and_captured_calls():
    layer, _ = _act_layer(1100, 600, 530)
    ws = {}
    side = torch.cuda.Stream()
    for T in (4, 50):
        xs = [_rand(f"cap/{T}/{i}", (T, 600), torch.bfloat16) for i in range(3)]
        dys = [_rand(f"cap/{T}/dy/{i}", (T, 1100), torch.bfloat16) for i in range(3)]
        mul = _rand(f"cap/{T}/mul", (T, 1100), torch.bfloat16)
        z = torch.empty(T, 1100, dtype=torch.bfloat16, device=DEV)

        def run(x, dy, z, **kw):
            y = nq.lrb_linear_act(layer, x, "silu", mul=mul, z=z, **kw)
            return (y, *nq.act_grads("silu", z, dy, mul=mul, **({"stream": kw["stream"]} if "stream" in kw else {})))
        want = [[t.clone() for t in run(x, dy, z)] for x, dy in zip(xs, dys)]
        side.wait_stream(torch.cuda.current_stream())
        got = run(xs[0], dys[0], z, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
        x, dy, z2 = xs[0].clone(), dys[0].clone(), torch.empty_like(z)
        ws[T] = torch.empty(nq.lrb_act_workspace_bytes(layer, T), dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run(x, dy, z2, workspace=ws[T])
        for i in (0, 1, 2, 1):
            x.copy_(xs[i]), dy.copy_(dys[i])
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want[i])), (T, i)
            run(xs[0], dys[0], z)  # eager work between the replays


@gpu
def test_binding_refuses_wrong_tensors():
    layer, _ = _act_layer(200, 130, 70)
    x = torch.zeros(4, 130, device=DEV)
    row = torch.zeros(4, 200, device=DEV)
    for kw in (dict(x=x[:, :60].contiguous()), dict(x=x.half()), dict(x=x.cpu()), dict(act="tanh"), dict(bias=row[0].bfloat16()),
               dict(bias=row[0, :5]), dict(mul=row[:3]), dict(mul=row.half()), dict(residual=row.cpu()),
               dict(residual=torch.zeros(4, 400, device=DEV)[:, ::2]), dict(z=row.double()), dict(y=row[:2]),
               dict(y=row, out_dtype=torch.bfloat16), dict(out_dtype=torch.float16),
               dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            nq.lrb_linear_act(**{**dict(layer=layer, x=x), **kw})
    with pytest.raises(nq.NqError):
        nq.lrb_linear_act(layer, x, y=row, z=row)
    with pytest.raises(nq.NqError):
        nq.lrb_linear_act(layer, torch.zeros(20, 130, device=DEV), workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(nq.NqError):
        nq.act_grads("none", None, torch.zeros(300, 7, device=DEV), workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    for kw in (dict(z=None), dict(z=row[:2]), dict(dy=row.half()), dict(mul=row[:, :9]), dict(dmul=row), dict(dz=row[:1]),
               dict(act="x"), dict(dy=row[0]), dict(dz=row.cpu())):
        with pytest.raises(ValueError):
            nq.act_grads(**{**dict(act="silu", z=row, dy=row), **kw})


# ---------------------------------------------------------------- a step of scale-only reconstruction




@gpu
@pytest.mark.parametrize("T", [6, 40])
def test_a_step_of_scale_only_reconstruction(T):
    """A packed gated block (up, gate with silu and the up's output, down with a residual) and a packed head, its
    logits against a teacher's record: the loss and every gradient of the scales against fp64 automatic
    differentiation of the same formulas.  Bars: every product of the chain is within the layer's own bar of
    its exact value (G.tol_for, fp32 activations), and a gradient passes through at most eight of them."""
    d, f, V, k = 96, 260, 1000, 30
    names = dict(up=(f, d, 60), gate=(f, d, 60), down=(d, f, 60), head=(V, d, 70))
    layers = {n: _act_layer(*shape) for n, shape in names.items()}
    dev = {n: v[0] for n, v in layers.items()}
    adj = {n: nq.Adjoint.of(v) for n, v in dev.items()}
    x = _rand(f"step/{T}/x", (T, d), torch.float32)
    bias = 0.1 * _rand("step/bias", (f,), torch.float32)
    teacher = nq.logits_top(3 * _rand(f"step/{T}/teacher", (T, V), torch.float32), k)
    w = torch.full((T,), 1.0 / T, device=DEV)

    up = nq.lrb_linear_act(dev["up"], x)
    z = torch.empty(T, f, device=DEV)
    h = nq.lrb_linear_act(dev["gate"], x, "silu", bias=bias, mul=up, z=z)
    hidden = nq.lrb_linear_act(dev["down"], h, residual=x)
    logits = nq.lrb_linear_act(dev["head"], hidden)
    loss, dlogits = nq.distill_grads(teacher, logits, weight=w)
    dhidden, *head = nq.lrb_scale_grads(dev["head"], adj["head"], hidden, dlogits)
    dh, *down = nq.lrb_scale_grads(dev["down"], adj["down"], h, dhidden)
    dz, dup, dbias = nq.act_grads("silu", z, dh, mul=up)
    dx_gate, *gate = nq.lrb_scale_grads(dev["gate"], adj["gate"], x, dz)
    dx_up, *ups = nq.lrb_scale_grads(dev["up"], adj["up"], x, dup)
    dx = dx_gate + dx_up + dhidden

    p64 = {n: [torch.tensor(v[1].s1, dtype=torch.float64, requires_grad=True),
               torch.tensor(v[1].s2, dtype=torch.float64, requires_grad=True),
               torch.from_numpy(np.array(v[1].U(), dtype=np.float64)), torch.from_numpy(np.array(v[1].Vt().T, dtype=np.float64))]
           for n, v in layers.items()}

    def lin(n, a):
        s1, s2, u, v = p64[n]
        return ((a * s2) @ v @ u.T) * s1
    x64 = x.double().cpu().requires_grad_()
    b64 = bias.double().cpu().requires_grad_()
    hid = lin("down", torch.nn.functional.silu(lin("gate", x64) + b64) * lin("up", x64)) + x64
    logq = torch.log_softmax(lin("head", hid), 1)
    ids, lp, rest = teacher.ids.long().cpu(), teacher.logp.double().cpu(), teacher.rest.double().cpu()
    away = torch.logsumexp(logq.scatter(1, ids, -float("inf")), 1)
    loss64 = (lp.exp() * (lp - logq.gather(1, ids))).sum(1) + rest.exp() * (rest - away)
    (loss64 / T).sum().backward()
    assert np.linalg.norm(_np(loss) - loss64.detach().numpy() / T) <= 8e-5 * np.linalg.norm(loss64.detach().numpy() / T)
    got = dict(head=head, down=down, gate=gate, up=ups)
    for n, g in got.items():
        for a, b in zip(g, p64[n][:2]):
            assert np.linalg.norm(_np(a) - b.grad.numpy()) <= 8e-5 * np.linalg.norm(b.grad.numpy()), n
    for a, b in ((dx, x64), (dbias, b64)):
        assert np.linalg.norm(_np(a) - b.grad.numpy()) <= 8e-5 * np.linalg.norm(b.grad.numpy())


# ---------------------------------------------------------------- tails


def _tail_bounds(act, z):
    """(act(z), act'(z), bounds of their errors before the result's own rounding), relative in the tails.  A function of
    the hardware is within one unit, two roundings; erfc within 16 units (OpenCL's bound).  The logistic q = E r or r,
    p = r or E r, r = 1 / (1 + E), E = exp(-|u|): exp2 2, its argument (in [-1/2, 1/2]) 1, the sum 1, the reciprocal 2,
    the products 2, so 8; u of gelu_tanh is off by 7 roundings of its own size (four products, two constants, a sum).
    A value below 2^-126 is off by at most 2^-149 besides."""
    z = np.asarray(z, dtype=np.float64)
    a, da, _ = D.act_ref(act, z)
    lost = (np.abs(z) + 2) * 2.0 ** -148
    if act == "gelu":
        cdf, pdf = np.where(z == 0, 0.5, a / np.where(z == 0, 1.0, z)), np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
        c = cdf * (34 + 2 * z * z)  # the argument's two roundings, felt z^2 times at most
        return a, da, (np.abs(z) * c + np.abs(a)) * D.EPS32 + lost, (
            c + np.abs(z) * pdf * (12 + z * z) + np.abs(da)) * D.EPS32 + lost
    if act == "silu":
        u, du, own = z, np.ones_like(z), 0.0
    else:
        k, b = np.sqrt(2 / np.pi), 0.044715
        u, du, own = 2 * k * (z + b * z ** 3), 2 * k * (1 + 3 * b * z * z), 7.0
    q, p = 1 / (1 + np.exp(-u)), 1 / (1 + np.exp(u))
    e_q, e_p = q * (8 + own * np.abs(u) * p), p * (8 + own * np.abs(u) * q)
    e_da = e_q + np.abs(z * du) * (e_q * p + q * e_p + 8 * p * q) + np.abs(da)
    return a, da, (np.abs(z) * e_q + np.abs(a)) * D.EPS32 + lost, e_da * D.EPS32 + lost * np.abs(du)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_tail_bounds_are_relative(act):
    """Far out on the left the bounds are a small part of the value: a result of 0 there does not pass."""
    z = np.array([-3.0, -5.0, -7.0])
    a, da, ea, eda = _tail_bounds(act, z)
    assert (ea < 1e-4 * np.abs(a)).all() and (eda < 1e-4 * np.abs(da)).all()


@gpu
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations_in_the_tails(act):
    """Values and derivatives keep their bits where they are small: the layer's input is zero, so z is the bias."""
    far = 91.0 if act == "silu" else 12.9  # to where the results leave fp32's normal numbers
    for d_out, d_in, r in ((256, 256, 64), (1100, 130, 70)):  # one workgroup; decode and the matrix-core regime
        layer, _ = _act_layer(d_out, d_in, r)
        bias = torch.linspace(-far, far, d_out, device=DEV)
        a, _, err, _ = _tail_bounds(act, _np(bias))
        for T in (1, 3, 20):
            x = torch.zeros(T, d_in, device=DEV)
            _close(nq.lrb_linear_act(layer, x, act, bias=bias), np.tile(a, (T, 1)), np.tile(err, (T, 1)), (act, T))
    z = torch.linspace(-far, far, 4099, device=DEV)[None].repeat(3, 1)
    a, da, err, derr = _tail_bounds(act, _np(z))
    dz, dmul, _ = nq.act_grads(act, z, torch.ones_like(z), mul=torch.ones_like(z))
    _close(dz, da, derr, (act, "dz"))
    _close(dmul, a, err, (act, "dmul"))


@gpu
@pytest.mark.parametrize("act", ACTS)
def test_activations_of_infinities(act):
    """Infinite values are the formulas' (and products of infinity and zero NaN), as the derivatives' are."""
    layer, _ = _act_layer(300, 40, 33)
    inf = float("inf")
    bias = torch.zeros(300, device=DEV)
    bias[:4] = torch.tensor([inf, -inf, float("nan"), 3e38], device=DEV)
    for T in (1, 5, 20):
        x = torch.zeros(T, 40, device=DEV)
        res = torch.zeros(T, 300, device=DEV)
        res[:, 7], res[:, 8], res[:, 0] = inf, -inf, 5.0
        got = _np(nq.lrb_linear_act(layer, x, act, bias=bias, residual=res))
        with np.errstate(all="ignore"):
            want = D.epilogue_ref(np.zeros((T, 300)), act, _np(bias), None, _np(res))[0]
        odd = ~np.isfinite(want)
        assert odd[:, [0, 2, 7, 8]].all() and np.array_equal(got[odd], want[odd], equal_nan=True), act
        assert np.isfinite(got[~odd]).all()
    z = torch.tensor([inf, -inf, float("nan"), 1.0], device=DEV)[None]
    with np.errstate(all="ignore"):
        want = D.act_ref(act, _np(z))[1]
    dz = _np(nq.act_grads(act, z, torch.ones_like(z))[0])
    assert np.array_equal(np.isnan(dz), np.isnan(want)) and np.array_equal(dz[0, :2], want[0, :2], equal_nan=True)


# ---------------------------------------------------------------- every kernel that a rule chooses


@gpu
@pytest.mark.parametrize("T,d", [(1037, 8195), (5000, 2051), (300, 28677)])
def test_act_grads_of_many_workgroups(T, d):
    """Sizes that fill the chip with 16 rows of threads (512 workgroups and more), each walking several tokens in
    several chunks, with ragged tokens and columns.  Columns are independent, so some are compared: the ends, those
    around a workgroup's (64 and 128 wide) and the ragged ones."""
    cols = sorted({0, 1, 7, 63, 64, 127, 128, 129, d // 2, d - 9, d - 8, d - 5, d - 4, d - 3, d - 2, d - 1})
    for i, act in enumerate(ACTS):
        for dt in (torch.float32, torch.bfloat16):
            z, dy = 2 * _rand("w/z", (T, d), dt), _rand("w/dy", (T, d), dt)
            mul = _rand("w/mul", (T, d), dt) if i % 2 else None
            dz, dmul, dbias = nq.act_grads(act, z, dy, mul=mul)
            wz, wm, wb, (ez, em, eb) = D.act_grads_ref(act, _np(z[:, cols]), _np(dy[:, cols]),
                                                       None if mul is None else _np(mul[:, cols]))
            _close(dz[:, cols], wz, ez, (act, "dz"))
            _close(dbias[cols], wb, eb, (act, "dbias"))
            if mul is not None:
                _close(dmul[:, cols], wm, em, (act, "dmul"))
            a, b = dy.clone(), None if mul is None else mul.clone()
            got = nq.act_grads(act, z, a, mul=b, dz=a, dmul=b)  # in place
            assert got[0] is a and torch.equal(a, dz) and torch.equal(got[2], dbias)
            assert mul is None or torch.equal(b, dmul)


@gpu
@pytest.mark.parametrize("T", [9, 40, 200])
@pytest.mark.parametrize("d_out,d_in,r", [(1100, 1030, 70), (1111, 2050, 130)])
def test_linear_act_of_a_split_first_stage(d_out, d_in, r, T):
    """A long input dimension before a small rank: the first product's reduction is split, the second's is not and
    takes the prepared t and the epilogue in one kernel."""
    test_linear_act(d_out, d_in, r, T)


UNSPLIT = [(1100, 130, 70), (1111, 130, 70), (1111, 1030, 70)]  # the second product whole: its tiles apply the epilogue


@gpu
@pytest.mark.parametrize("d_out,d_in,r", UNSPLIT)
@pytest.mark.parametrize("T", [30, 130])
def test_linear_act_in_place_by_tiles(d_out, d_in, r, T):
    layer, _ = _act_layer(d_out, d_in, r)
    for dt in (torch.float32, torch.bfloat16):
        x, mul, res = _rand("it/x", (T, d_in), dt), _rand("it/mul", (T, d_out), dt), _rand("it/res", (T, d_out), dt)
        z = torch.empty(T, d_out, dtype=dt, device=DEV)
        want = nq.lrb_linear_act(layer, x, "silu", mul=mul, residual=res, z=z)
        a, b, z2 = mul.clone(), res.clone(), torch.empty_like(z)
        assert nq.lrb_linear_act(layer, x, "silu", mul=a, residual=res, y=a, z=z2) is a
        assert torch.equal(a, want) and torch.equal(z2, z)
        assert torch.equal(nq.lrb_linear_act(layer, x, "silu", mul=mul, residual=b, y=b), want)
        both = mul.clone()
        want2 = nq.lrb_linear_act(layer, x, "gelu", mul=mul, residual=mul)
        assert torch.equal(nq.lrb_linear_act(layer, x, "gelu", mul=both, residual=both, y=both), want2)
        y = torch.full((T + 2, d_out), 3.0, dtype=dt, device=DEV)  # rows at any alignment, nothing beside them written
        nq.lrb_linear_act(layer, x, "silu", mul=mul, residual=res, y=y[1:T + 1])
        assert torch.equal(y[1:T + 1], want) and (y[0] == 3).all() and (y[T + 1] == 3).all()


@gpu
@pytest.mark.parametrize("d_out,d_in,r", UNSPLIT)
def test_captured_calls_by_tiles(d_out, d_in, r):
    layer, _ = _act_layer(d_out, d_in, r)
    T = 50
    for dt in (torch.float32, torch.bfloat16):
        xs = [_rand(f"ct/{i}", (T, d_in), dt) for i in range(3)]
        mul, res = _rand("ct/mul", (T, d_out), dt), _rand("ct/res", (T, d_out), dt)

        def run(x, z):
            return nq.lrb_linear_act(layer, x, "gelu_tanh", mul=mul, residual=res, z=z), z
        want = [run(x, torch.empty(T, d_out, dtype=dt, device=DEV)) for x in xs]
        x, z = xs[0].clone(), torch.empty(T, d_out, dtype=dt, device=DEV)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run(x, z)
        for i in (0, 1, 2, 1):
            x.copy_(xs[i])
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want[i])), i
            run(xs[0], torch.empty_like(z))  # eager work between the replays


@gpu
@pytest.mark.parametrize("T", [6, 40])
def test_a_captured_step_of_scale_only_reconstruction(T):
    """The step of test_a_step_of_scale_only_reconstruction in one graph, replayed on new inputs and records with
    eager work between: every result is the eager step's."""
    d, f, V, k = 96, 260, 1000, 30
    names = dict(up=(f, d, 60), gate=(f, d, 60), down=(d, f, 60), head=(V, d, 70))
    dev = {n: _act_layer(*shape)[0] for n, shape in names.items()}
    adj = {n: nq.Adjoint.of(v) for n, v in dev.items()}
    bias = 0.1 * _rand("step/bias", (f,), torch.float32)
    w = torch.full((T,), 1.0 / T, device=DEV)

    def step(x, teacher_logits):
        teacher = nq.logits_top(teacher_logits, k)
        up = nq.lrb_linear_act(dev["up"], x)
        z = torch.empty(T, f, device=DEV)
        h = nq.lrb_linear_act(dev["gate"], x, "silu", bias=bias, mul=up, z=z)
        hidden = nq.lrb_linear_act(dev["down"], h, residual=x)
        logits = nq.lrb_linear_act(dev["head"], hidden)
        loss, dlogits = nq.distill_grads(teacher, logits, weight=w)
        dhidden, *head = nq.lrb_scale_grads(dev["head"], adj["head"], hidden, dlogits)
        dh, *down = nq.lrb_scale_grads(dev["down"], adj["down"], h, dhidden)
        dz, dup, dbias = nq.act_grads("silu", z, dh, mul=up)
        dx, *gate = nq.lrb_scale_grads(dev["gate"], adj["gate"], x, dz)
        dx_up, *ups = nq.lrb_scale_grads(dev["up"], adj["up"], x, dup)
        return [teacher.ids, teacher.logp, teacher.rest, loss, dlogits, dz, dup, dbias, dx, dx_up, *head, *down, *gate, *ups]

    xs = [_rand(f"step/{T}/x/{i}", (T, d), torch.float32) for i in range(3)]
    ts = [3 * _rand(f"step/{T}/teacher/{i}", (T, V), torch.float32) for i in range(3)]
    want = [[t.clone() for t in step(a, b)] for a, b in zip(xs, ts)]
    assert not torch.equal(want[0][3], want[1][3])
    x, t = xs[0].clone(), ts[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, t)
    for i in (0, 1, 2, 1):
        x.copy_(xs[i]), t.copy_(ts[i])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i])), (i, [torch.equal(a, b) for a, b in zip(out, want[i])])
        step(xs[2], ts[0])  # eager work between the replays


@gpu
@pytest.mark.parametrize("T,d", [(16, 1117), (64, 1117), (64, 300)])
def test_bias_gradients_add_across_threads_in_fp64(T, d):
    """With one token to a thread (16 rows of threads, or 64) nothing is added in fp32: the sum is rounded once."""
    for dt in (torch.float32, torch.bfloat16):
        dy = (1 + _rand("once/dy", (T, d), torch.float32).abs()).to(dt)
        want = _np(dy).sum(0)
        dbias = _np(nq.act_grads("none", None, dy)[2])
        assert (np.abs(dbias - want) <= D.EPS32 * (1 + 2.0 ** -20) * want).all()


@gpu
def test_operands_of_more_than_2_to_31_elements():
    """Rows far behind, at offsets that 32 bits do not hold: 128 rows repeated give their results again."""
    n, d = 600, 28672
    T = 128 * n
    assert T * d > 2 ** 31
    layer, _ = _act_layer(d, 64, 40)
    x, mul = _rand("far/x", (128, 64), torch.bfloat16), _rand("far/mul", (128, d), torch.bfloat16)
    xs, muls = x.repeat(n, 1), mul.repeat(n, 1)
    z = torch.empty_like(muls)
    y = nq.lrb_linear_act(layer, xs, "silu", mul=muls, z=z)
    want, _, err = D.epilogue_ref(_np(nq.lrb_linear(layer, xs[:128].contiguous())), "silu", None, _np(mul))
    # another number of tokens, another split of the reduction: fp16 operands either way
    assert np.linalg.norm(_np(y[:128]) - want) <= 2 * G.prefill_tol("bf16") * np.linalg.norm(want) + np.linalg.norm(
        HALF[torch.bfloat16] * np.abs(want))
    for at in (T // 2, T - 128 * 21, T - 256, T - 128):
        assert torch.equal(y[at:at + 128], y[:128]) and torch.equal(z[at:at + 128], z[:128]), at
    dz, dmul, dbias = nq.act_grads("silu", z, y, mul=muls, dz=y, dmul=muls)
    for at in (T // 2, T - 128 * 21, T - 256, T - 128):
        assert torch.equal(dz[at:at + 128], dz[:128]) and torch.equal(dmul[at:at + 128], dmul[:128]), at
    assert not torch.equal(dz[:128], dmul[:128]) and torch.isfinite(dbias).all()


@gpu
@pytest.mark.parametrize("T", [4, 50])
def test_calls_on_two_streams_at_once(T):
    """Linears with an epilogue, plain ones and gradients on two streams, workspaces of each call's own."""
    layers = [_act_layer(1100, 600, 530)[0], _act_layer(1111, 1030, 70)[0]]
    xs = [_rand(f"two/x/{L.d_in}", (T, L.d_in), torch.bfloat16) for L in layers]
    muls = [_rand(f"two/mul/{L.d_out}", (T, L.d_out), torch.bfloat16) for L in layers]

    def run(i):
        L, x, m = layers[i], xs[i], muls[i]
        z = torch.empty_like(m)
        y = nq.lrb_linear_act(L, x, "silu", mul=m, z=z)
        return [y, z, nq.lrb_linear(L, x), *nq.act_grads("gelu", z, y, mul=m)]
    want = [run(i) for i in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(run(i))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
