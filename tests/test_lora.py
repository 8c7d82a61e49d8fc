"""Low-rank adapters beside a shared projection and their gradients, against
the fp64 reference.

Tolerances.  Every product of two inputs is exact in the arithmetic used (bf16
times bf16, or three bf16 terms that add up to the fp32 value), and sums are
fp32, so a result differs from the exact one by at most one rounding, 2^-24 of
the absolute sums, per addition or product:
  deterministic, every element: |y - y*| <= n * 2^-24 * (the sum of absolute
  terms), n the additions on a result's path: the reduction of the hidden
  vector (d), three terms per rank (3r), for factor gradients three per token
  (3T) and one for each join, scale and base (16);
  normwise: the roundings of one result are independent, so their sum grows as
  sqrt(n); 4 sqrt(n) 2^-24.
fp32 factors or activations round each product once, as one more addition
each: n doubles."""
import ctypes

import numpy as np
import pytest
import torch

import synth
from oracle import adapters as A

nq = pytest.importorskip("sub_bit_weight_amd")

DEV = "cuda:0"
U = 2.0 ** -24
DUMMY = 0x100000
gpu = pytest.mark.gpu


# ---------------------------------------------------------------- the reference


def _case(tag, T, n, r, d_in, d_out, xd="bf16", wd="bf16", ids=None):
    rnd = {"bf16": synth.round_bf16, "f32": lambda v: v}
    g = synth.rng(f"lora/{tag}")
    if ids is None:
        ids = g.integers(-1, n, T)
    return dict(a=rnd[wd](synth.normal_f32(f"lora/{tag}/a", (n, r, d_in)) / np.float32(np.sqrt(d_in))),
                b=rnd[wd](synth.normal_f32(f"lora/{tag}/b", (n, d_out, r))),
                scale=np.exp(0.3 * g.standard_normal(n)).astype(np.float32),
                x=rnd[xd](synth.normal_f32(f"lora/{tag}/x", (T, d_in))), ids=np.asarray(ids, dtype=np.int32),
                base=synth.normal_f32(f"lora/{tag}/base", (T, d_out)),
                g=rnd[xd](synth.normal_f32(f"lora/{tag}/g", (T, d_out))),
                dx_base=synth.normal_f32(f"lora/{tag}/dxb", (T, d_in)), xd=xd, wd=wd)


def test_reference_gradients_match_differences():
    c = _case("diff", 6, 3, 2, 5, 4, "f32", "f32", [0, 2, -1, 0, 2, 2])
    w = c["g"].astype(np.float64)

    def loss(a, b, x):
        return float((A.lora_linear_ref(a, b, c["scale"], x, c["ids"]) * w).sum())
    dx, da, db = A.lora_grads_ref(c["a"], c["b"], c["scale"], c["x"], w, c["ids"])
    args = [c["a"].astype(np.float64), c["b"].astype(np.float64), c["x"].astype(np.float64)]
    for which, grad in ((0, da), (1, db), (2, dx)):
        num = np.zeros_like(grad)
        for i in np.ndindex(grad.shape):
            at = [v.copy() for v in args]
            at[which][i] += 1e-3
            up = loss(*at)
            at[which][i] -= 2e-3
            num[i] = (up - loss(*at)) / 2e-3
        assert np.allclose(grad, num, rtol=1e-6, atol=1e-7), which


# ---------------------------------------------------------------- refusals (no GPU)


def _pool(**kw):
    d = dict(n=4, d_out=64, d_in=32, r=8, dtype=nq.NQ_BF16, a=DUMMY, lda=32, stride_a=256, b=DUMMY, ldb=8, stride_b=512,
             scale=DUMMY)
    d.update(kw)
    return nq.nq_lora(**d)


def _linear(p, x=DUMMY, xd=nq.NQ_BF16, ids=DUMMY, T=3, base=None, y=DUMMY, ws=DUMMY, wsb=1 << 40):
    return nq.lib().nq_lora_linear(None if p is None else ctypes.byref(p), x, xd, ids, T, base, y, ws, wsb, None)


def _grads(p, x=DUMMY, xd=nq.NQ_BF16, g=DUMMY, gd=nq.NQ_F32, ids=DUMMY, T=3, base=None, dx=DUMMY, da=DUMMY, db=DUMMY,
           ws=DUMMY, wsb=1 << 40):
    return nq.lib().nq_lora_grads(ctypes.byref(p), x, xd, g, gd, ids, T, base, dx, da, db, ws, wsb, None)


BAD_POOLS = [
    (dict(n=0), nq.NQ_ERR_ARG), (dict(r=0), nq.NQ_ERR_ARG), (dict(d_out=-1), nq.NQ_ERR_ARG), (dict(d_in=0), nq.NQ_ERR_ARG),
    (dict(n=8193), nq.NQ_ERR_UNSUPPORTED), (dict(r=1025, ldb=1025), nq.NQ_ERR_UNSUPPORTED),
    (dict(d_in=(1 << 24) + 1, lda=(1 << 24) + 1), nq.NQ_ERR_UNSUPPORTED),
    (dict(dtype=5), nq.NQ_ERR_ARG), (dict(a=None), nq.NQ_ERR_ARG), (dict(b=None), nq.NQ_ERR_ARG),
    (dict(scale=None), nq.NQ_ERR_ARG), (dict(a=DUMMY + 1), nq.NQ_ERR_ARG), (dict(scale=DUMMY + 2), nq.NQ_ERR_ARG),
    (dict(dtype=nq.NQ_F32, b=DUMMY + 2), nq.NQ_ERR_ARG), (dict(lda=31), nq.NQ_ERR_ARG), (dict(ldb=7), nq.NQ_ERR_ARG),
    (dict(stride_a=-1), nq.NQ_ERR_ARG), (dict(stride_b=-8), nq.NQ_ERR_ARG),
]


@pytest.mark.parametrize("kw,status", BAD_POOLS)
def test_rejects_bad_pool(kw, status):
    p = _pool(**kw)
    assert _linear(p) == status and nq.last_error() != ""
    assert _grads(p) == status
    assert nq.lib().nq_lora_workspace_bytes(ctypes.byref(p), 3) == 0
    assert nq.lib().nq_lora_grads_workspace_bytes(ctypes.byref(p), 3) == 0


def test_rejects_bad_io():
    p = _pool()
    assert _linear(None) == nq.NQ_ERR_ARG
    for call in (_linear, _grads):
        assert call(p, T=0) == nq.NQ_ERR_ARG
        assert call(p, T=(1 << 24) + 1) == nq.NQ_ERR_UNSUPPORTED
        assert call(p, xd=9) == nq.NQ_ERR_ARG
        assert call(p, x=None) == nq.NQ_ERR_ARG
        assert call(p, ids=None) == nq.NQ_ERR_ARG
        assert call(p, ids=DUMMY + 2) == nq.NQ_ERR_ARG
        assert call(p, base=DUMMY + 2) == nq.NQ_ERR_ARG
        assert call(p, ws=None) == nq.NQ_ERR_WORKSPACE
        assert call(p, wsb=8) == nq.NQ_ERR_WORKSPACE
        assert call(p, ws=DUMMY + 64) == nq.NQ_ERR_ARG
    assert _linear(p, y=None) == nq.NQ_ERR_ARG
    assert _grads(p, g=None) == nq.NQ_ERR_ARG
    assert _grads(p, gd=3) == nq.NQ_ERR_ARG
    assert _grads(p, dx=None) == nq.NQ_ERR_ARG
    assert _grads(p, da=None) == nq.NQ_ERR_ARG
    assert _grads(p, db=DUMMY + 1) == nq.NQ_ERR_ARG


def test_layer_with_adapters_rejects_other_sizes():
    L = nq.nq_lrb(d_out=64, d_in=64, r=32, u_bits=DUMMY, ldu=64, vt_bits=DUMMY, ldv=32, s1=DUMMY, s2=DUMMY)

    def call(p, ids=DUMMY, wsb=1 << 40):
        return nq.lib().nq_lrb_lora_linear(ctypes.byref(L), ctypes.byref(p), DUMMY, nq.NQ_BF16, ids, 3, DUMMY, DUMMY, wsb, None)
    assert call(_pool()) == nq.NQ_ERR_ARG and "beside" in nq.last_error()
    ok = _pool(d_in=64, lda=64)
    assert call(ok, ids=None) == nq.NQ_ERR_ARG
    assert call(ok, wsb=100) == nq.NQ_ERR_WORKSPACE
    lib = nq.lib()
    both = lib.nq_lrb_lora_workspace_bytes(ctypes.byref(L), ctypes.byref(ok), 3)
    assert both >= lib.nq_lrb_workspace_bytes(ctypes.byref(L), 3) + lib.nq_lora_workspace_bytes(ctypes.byref(ok), 3)


def test_binding_refuses_what_the_library_cannot_see():
    a, b, s = torch.zeros(2, 4, 8), torch.zeros(2, 6, 4), torch.ones(2)
    with pytest.raises(ValueError):
        nq.Lora(a, b, s).struct()  # host tensors
    with pytest.raises(ValueError):
        nq.Lora(a, torch.zeros(2, 6, 5), s).struct()
    with pytest.raises(ValueError):
        nq.Lora(a.half(), b.half(), s).struct()
    with pytest.raises(ValueError):
        nq.Lora(a, b.bfloat16(), s).struct()
    with pytest.raises(ValueError):
        nq.Lora(a[:0], b[:0], s[:0]).struct()


def test_a_pool_keeps_a_bounded_number_of_workspace_sizes():
    pool = nq.Lora(torch.zeros(2, 4, 8), torch.zeros(2, 6, 4), torch.ones(2))
    st = _pool(n=2, d_in=8, d_out=6, r=4)
    object.__setattr__(pool, "_struct", st)
    for T in range(1, 5000):
        want = nq.lib().nq_lora_workspace_bytes(ctypes.byref(st), T)
        assert pool._workspace_bytes("nq_lora_workspace_bytes", T) == want
        assert pool._workspace_bytes("nq_lora_workspace_bytes", T) == want
        assert len(pool._bytes) <= 256


# ---------------------------------------------------------------- GPU


def _dev(v, kind="f32"):
    t = torch.from_numpy(np.ascontiguousarray(v)).to(DEV)
    return t.to(torch.bfloat16) if kind == "bf16" else t


def _gpu_pool(c):
    return nq.Lora(_dev(c["a"], c["wd"]), _dev(c["b"], c["wd"]), _dev(c["scale"]))


def _check(got, want, absolute, n, wide):
    got = got.cpu().numpy().astype(np.float64)
    n = n * (2 if wide else 1)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    d = np.abs(np.where(nan, 0, got - want))
    bad = d > n * U * np.where(nan, 0, absolute) + 1e-37
    assert not bad.any(), (np.argwhere(bad)[:4], d[bad][:4], absolute[bad][:4])
    norm = np.linalg.norm(np.where(nan, 0, want))
    assert np.linalg.norm(d) <= 4 * np.sqrt(n) * U * norm + 1e-37, np.linalg.norm(d) / norm


def _run_linear(c, base=True, **kw):
    y = nq.lora_linear(_gpu_pool(c), _dev(c["x"], c["xd"]), _dev(c["ids"]), _dev(c["base"]) if base else None, **kw)
    T, d_in = c["x"].shape
    args = (c["a"], c["b"], c["scale"], c["x"], c["ids"], c["base"] if base else None)
    _check(y, A.lora_linear_ref(*args), A.lora_abs(*args), d_in + 3 * c["a"].shape[1] + 16, "f32" in (c["xd"], c["wd"]))
    return y


SHAPES = [  # T, n, r, d_in, d_out
    (1, 1, 1, 1, 1), (1, 3, 16, 256, 128), (2, 1, 8, 64, 64), (5, 4, 17, 100, 33), (17, 1, 4, 37, 129),
    (64, 5, 16, 520, 260), (64, 64, 7, 65, 513), (65, 3, 16, 256, 256), (33, 2, 64, 130, 1030), (100, 7, 33, 1031, 77),
    (130, 40, 65, 300, 520), (200, 2, 130, 64, 100), (257, 1, 48, 2100, 640), (96, 300, 2, 16, 9),
    (90, 3, 12, 512, 300), (150, 2, 20, 768, 264), (70, 40, 41, 1032, 520),  # ranks that are no multiple of 8
    (4, 2, 16, 2048, 600), (3, 3, 5, 2047, 1030), (4, 1, 16, 2049, 70), (4, 2, 17, 300, 70), (5, 5, 16, 256, 64),
]


@gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("xd,wd", [("bf16", "bf16"), ("f32", "f32")])
def test_linear(shape, xd, wd):
    _run_linear(_case(f"lin/{shape}", *shape, xd, wd))


@gpu
@pytest.mark.parametrize("T", [6, 150])
@pytest.mark.parametrize("xd,wd", [("bf16", "f32"), ("f32", "bf16")])
def test_linear_mixed_types_without_base(T, xd, wd):
    _run_linear(_case(f"mix/{T}", T, 3, 20, 270, 140, xd, wd), base=False)


@gpu
@pytest.mark.parametrize("T,n", [(40, 3), (300, 5)])
def test_linear_ids_without_an_adapter_and_out_of_range(T, n):
    ids = synth.rng(f"lora/ids/{T}").integers(-3, n, T)
    ids[[0, T // 2, T - 1]] = [n, 2 ** 31 - 1, -2 ** 31]
    y = _run_linear(_case(f"ids/{T}", T, n, 16, 128, 192, ids=ids))
    assert torch.isnan(y[0]).all() and torch.isnan(y[T // 2]).all() and not torch.isnan(y[T - 1]).any()
    c = _case(f"none/{T}", T, n, 16, 128, 192, ids=np.full(T, -1))
    assert torch.equal(_run_linear(c).cpu(), torch.from_numpy(c["base"]))


@gpu
@pytest.mark.parametrize("T", [20, 90])
def test_linear_keeps_non_finite_values_in_their_rows(T):
    """NaN and infinities in one adapter, one token and unused adapters reach no other token's row."""
    n = 4
    ids = np.arange(T) % 3  # adapter 3 has no token
    c = _case(f"nan/{T}", T, n, 12, 70, 150, ids=ids)
    clean = nq.lora_linear(_gpu_pool(c), _dev(c["x"], "bf16"), _dev(ids.astype(np.int32)), _dev(c["base"]))
    c["a"][3] = np.nan
    c["b"][3] = np.inf
    c["a"][1, 2, 5] = np.nan
    c["b"][1, 7] = np.inf
    c["x"][3, 4] = np.inf  # adapter 0
    c["base"][8, 1] = np.nan  # adapter 2
    y = nq.lora_linear(_gpu_pool(c), _dev(c["x"], "bf16"), _dev(ids.astype(np.int32)), _dev(c["base"]))
    for t in range(T):
        if t == 8:
            assert torch.isnan(y[t, 1]) and torch.equal(y[t, 2:], clean[t, 2:])
        elif ids[t] == 1 or t == 3:
            assert not torch.isfinite(y[t]).all()
        else:
            assert torch.equal(y[t], clean[t]), t


@gpu
@pytest.mark.parametrize("T", [9, 77])
def test_linear_in_place_strided_and_dirty_workspace(T):
    c = _case(f"view/{T}", T, 3, 20, 96, 200)
    pool, x, ids, base = _gpu_pool(c), _dev(c["x"], "bf16"), _dev(c["ids"]), _dev(c["base"])
    want = nq.lora_linear(pool, x, ids, base)
    ws = torch.full((nq.lora_workspace_bytes(pool, T),), 255, dtype=torch.uint8, device=DEV)  # NaN bit patterns
    y = base.clone()
    assert nq.lora_linear(pool, x, ids, y, y=y, workspace=ws).data_ptr() == y.data_ptr()
    assert torch.equal(y, want)
    # factors inside larger buffers: padded rows, adapters in reverse rank order of their strides
    a = torch.full((25, 3, 101), float("nan"), dtype=torch.bfloat16, device=DEV)
    b = torch.full((3, 203, 27), float("nan"), dtype=torch.bfloat16, device=DEV)
    av, bv = a[:20, :, 3:99].permute(1, 0, 2), b[:, 1:201, 5:25]
    av.copy_(pool.a)
    bv.copy_(pool.b)
    assert torch.equal(nq.lora_linear(nq.Lora(av, bv, pool.scale), x, ids, base), want)


def _run_grads(c, base=True):
    T, d_in = c["x"].shape
    n, d_out, r = c["b"].shape
    got = nq.lora_grads(_gpu_pool(c), _dev(c["x"], c["xd"]), _dev(c["g"], c["xd"]), _dev(c["ids"]),
                        _dev(c["dx_base"]) if base else None)
    args = (c["a"], c["b"], c["scale"], c["x"], c["g"], c["ids"], c["dx_base"] if base else None)
    want, absolute = A.lora_grads_ref(*args), A.lora_grads_abs(*args)
    wide = "f32" in (c["xd"], c["wd"])
    for v, w, s, n_add in zip(got, want, absolute, (d_out + 3 * r + 16, d_out + 3 * T + 16, d_in + 3 * T + 16)):
        _check(v, w, s, n_add, wide)
    return got


@gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("xd,wd", [("bf16", "bf16"), ("f32", "f32")])
def test_grads(shape, xd, wd):
    _run_grads(_case(f"grads/{shape}", *shape, xd, wd))


@gpu
@pytest.mark.parametrize("xd,wd", [("bf16", "f32"), ("f32", "bf16")])
def test_grads_mixed_types_without_base(xd, wd):
    _run_grads(_case("gmix", 150, 3, 20, 270, 140, xd, wd), base=False)


@gpu
@pytest.mark.parametrize("T,n,d_in,d_out", [(33, 2, 130, 1030), (70, 9, 1500, 1100), (500, 30, 1100, 2100)])
def test_grads_with_a_dirty_workspace(T, n, d_in, d_out):
    """Reductions cut into spans, tiles fewer than the most there could be, and a workspace full of ones."""
    c = _case(f"dirty/{T}", T, n, 20, d_in, d_out, ids=synth.rng(f"lora/dirty/{T}").integers(0, (n + 1) // 2, T))
    pool, x, g, ids = _gpu_pool(c), _dev(c["x"], "bf16"), _dev(c["g"], "bf16"), _dev(c["ids"])
    ws = torch.full((nq.lora_grads_workspace_bytes(pool, T),), 255, dtype=torch.uint8, device=DEV)
    wl = torch.full((nq.lora_workspace_bytes(pool, T),), 255, dtype=torch.uint8, device=DEV)
    got = nq.lora_grads(pool, x, g, ids, _dev(c["dx_base"]), workspace=ws)
    args = (c["a"], c["b"], c["scale"], c["x"], c["g"], c["ids"], c["dx_base"])
    for v, w, s, n_add in zip(got, A.lora_grads_ref(*args), A.lora_grads_abs(*args),
                              (d_out + 3 * 20 + 16, d_out + 3 * T + 16, d_in + 3 * T + 16)):
        _check(v, w, s, n_add, False)
    y = nq.lora_linear(pool, x, ids, _dev(c["base"]), workspace=wl)
    args = (c["a"], c["b"], c["scale"], c["x"], c["ids"], c["base"])
    _check(y, A.lora_linear_ref(*args), A.lora_abs(*args), d_in + 3 * 20 + 16, False)


@gpu
def test_grads_of_few_adapters_with_many_tokens():
    """One adapter's tokens cut into chunks whose sums are joined."""
    _run_grads(_case("chunks", 2100, 1, 16, 40, 24))
    _run_grads(_case("chunks2", 1500, 2, 24, 200, 130, "f32", "f32"))


@gpu
@pytest.mark.parametrize("T,n,r,d_in,d_out,kind", [
    (1 << 24, 3, 2, 3, 5, "f32"),        # the largest call: offsets past 32 bits, a grid at its limit
    (4200, 3, 20, 8192, 8200, "bf16"),   # several 16-slot groups a workgroup
    (1 << 16, 8192, 33, 40, 24, "f32"),  # the most adapters
])
def test_exact_on_integers_at_large_sizes(T, n, r, d_in, d_out, kind):
    """Small integers and scales of 1/2: every sum is exact, so results are equal bit for bit."""
    gen = torch.Generator(DEV).manual_seed(T + n)

    def ints(shape, top, t=torch.float32):
        return torch.randint(-top, top + 1, shape, generator=gen, device=DEV).to(t)
    t = torch.bfloat16 if kind == "bf16" else torch.float32
    a, b, x, g = ints((n, r, d_in), 1, t), ints((n, d_out, r), 1, t), ints((T, d_in), 1, t), ints((T, d_out), 1, t)
    base, dxb = ints((T, d_out), 9), ints((T, d_in), 9)
    ids = torch.randint(-1, n + 1, (T,), generator=gen, device=DEV, dtype=torch.int32)
    scale = torch.full((n,), 0.5, device=DEV)
    pool = nq.Lora(a, b, scale)
    y = nq.lora_linear(pool, x, ids, base)
    dx, da, db = nq.lora_grads(pool, x, g, ids, dxb)
    none, bad = ids < 0, ids >= n
    assert torch.equal(y[none], base[none]) and torch.equal(dx[none], dxb[none])
    assert torch.isnan(y[bad]).all() and torch.isnan(dx[bad]).all()
    for i in range(n) if n < 10 else (0, 1, 4095, n - 2, n - 1):
        rows = (ids == i).nonzero()[:, 0]
        xi, gi, ai, bi = x[rows].double(), g[rows].double(), a[i].double(), b[i].double()
        h, dh = xi @ ai.T, 0.5 * (gi @ bi)
        assert torch.equal(y[rows].double(), base[rows] + 0.5 * (h @ bi.T)), i
        assert torch.equal(dx[rows].double(), dxb[rows] + dh @ ai), i
        assert torch.equal(da[i].double(), dh.T @ xi) and torch.equal(db[i].double(), 0.5 * (gi.T @ h)), i


@gpu
def test_grads_leave_out_tokens_without_an_adapter():
    T, n = 120, 4
    ids = np.arange(T) % 2  # adapters 2 and 3 without tokens
    ids[[1, 50]] = [-1, -7]
    ids[[2, 60]] = [n, n + 5]
    c = _case("gids", T, n, 16, 100, 60, ids=ids)
    c["x"][[1, 2]] = np.nan  # rows of no adapter: in nobody's sums
    c["g"][[50, 60]] = np.inf
    c["a"][3] = np.nan
    got = nq.lora_grads(_gpu_pool(c), _dev(c["x"], "bf16"), _dev(c["g"], "bf16"), _dev(c["ids"]), _dev(c["dx_base"]))
    c["x"][[1, 2]], c["g"][[50, 60]], c["a"][3] = 0, 0, 0
    want = A.lora_grads_ref(c["a"], c["b"], c["scale"], c["x"], c["g"], c["ids"], c["dx_base"])
    absolute = A.lora_grads_abs(c["a"], c["b"], c["scale"], c["x"], c["g"], c["ids"], c["dx_base"])
    for v, w, s in zip(got, want, absolute):
        _check(v, w, s, 100 + 3 * T + 16, False)
    assert torch.equal(got[0][1].cpu(), torch.from_numpy(c["dx_base"][1])) and torch.isnan(got[0][2]).all()
    assert not got[1][2:].any() and not got[2][2:].any()


@gpu
def test_grads_match_differences_of_the_forward_call():
    c = _case("fwd-diff", 90, 3, 8, 60, 50, "f32", "f32")
    pool, x, ids, g = _gpu_pool(c), _dev(c["x"]), _dev(c["ids"]), _dev(c["g"])
    dx, da, db = nq.lora_grads(pool, x, g, ids)

    def loss(p, v):
        return float((nq.lora_linear(p, v, ids).double() * g.double()).sum())
    eps = 2.0 ** -4  # y is linear in each of a, b and x, so a difference has no truncation error
    for which, grad in (("a", da), ("b", db), ("x", dx)):
        step = torch.from_numpy(synth.normal_f32(f"lora/step/{which}", tuple(grad.shape))).to(DEV)

        def at(sign):
            if which == "x":
                return loss(pool, x + sign * eps * step)
            f = {"a": pool.a, "b": pool.b}
            f[which] = f[which] + sign * eps * step
            return loss(nq.Lora(f["a"], f["b"], pool.scale), x)
        num, want = (at(1) - at(-1)) / (2 * eps), float((grad.double() * step.double()).sum())
        # a loss sums T * d_out values, each off by at most n roundings of its absolute terms
        size = float(np.abs(A.lora_abs(c["a"], c["b"], c["scale"], c["x"], c["ids"]) * c["g"]).sum())
        assert abs(num - want) <= 2 * (60 + 24 + 16) * 2 * U * size / (2 * eps) * 2, (which, num, want)


@gpu
def test_results_repeat_and_streams_do_not_mix():
    c = _case("streams", 300, 5, 16, 512, 700)
    pool, x, ids, base = _gpu_pool(c), _dev(c["x"], "bf16"), _dev(c["ids"]), _dev(c["base"])
    g, dxb = _dev(c["g"], "bf16"), _dev(c["dx_base"])
    want, wantg = nq.lora_linear(pool, x, ids, base), nq.lora_grads(pool, x, g, ids, dxb)
    small = nq.lora_linear(pool, x[:40], ids[:40], base[:40])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(3):
        outs = [(nq.lora_linear(pool, x, ids, base, stream=s), nq.lora_grads(pool, x, g, ids, dxb, stream=s),
                 nq.lora_linear(pool, x[:40], ids[:40], base[:40], stream=s)) for s in streams]
        torch.cuda.synchronize()
        for y, gr, ys in outs:
            assert torch.equal(y, want) and torch.equal(ys, small)
            assert all(torch.equal(p, q) for p, q in zip(gr, wantg))


@gpu
@pytest.mark.parametrize("T", [12, 200])
def test_captured_calls_follow_their_inputs(T):
    """A captured run of forward and gradients, replayed on new tokens and new ids, gives what eager calls give."""
    cs = [_case(f"graph/{T}/{i}", T, 4, 16, 256, 320) for i in range(3)]
    pool = _gpu_pool(cs[0])
    x, ids, base = _dev(cs[0]["x"], "bf16"), _dev(cs[0]["ids"]), _dev(cs[0]["base"])
    g, dxb = _dev(cs[0]["g"], "bf16"), _dev(cs[0]["dx_base"])
    wsl = torch.empty(nq.lora_workspace_bytes(pool, T), dtype=torch.uint8, device=DEV)
    wsg = torch.empty(nq.lora_grads_workspace_bytes(pool, T), dtype=torch.uint8, device=DEV)
    nq.lora_linear(pool, x, ids, base, workspace=wsl)
    nq.lora_grads(pool, x, g, ids, dxb, workspace=wsg)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = nq.lora_linear(pool, x, ids, base, workspace=wsl)
        gr = nq.lora_grads(pool, x, g, ids, dxb, workspace=wsg)
    for i in (0, 1, 2, 1):
        c = cs[i]
        for dst, name in ((x, "x"), (g, "g"), (ids, "ids"), (base, "base"), (dxb, "dx_base")):
            dst.copy_(torch.from_numpy(c[name]))
        want, wantg = nq.lora_linear(pool, x, ids, base), nq.lora_grads(pool, x, g, ids, dxb)  # eager, beside the graph
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and all(torch.equal(p, q) for p, q in zip(gr, wantg))


@gpu
@pytest.mark.parametrize("T", [3, 8, 70])
def test_layer_with_adapters_is_the_two_calls(T):
    shape = synth.LayerShape("w", 300, 200, 64)
    inp = synth.lrb_inputs(synth.Config("lora", "lora", [], (1,), "bf16"), shape)
    layer = nq.Lrb(300, 200, 64, nq.pack_u(_dev(inp["U_latent"])), nq.pack_v(_dev(inp["V_latent"])), _dev(inp["s1"]),
                   _dev(inp["s2"]))
    c = _case(f"both/{T}", T, 3, 16, 200, 300)
    pool, x, ids = _gpu_pool(c), _dev(c["x"], "bf16"), _dev(c["ids"])
    want = nq.lora_linear(pool, x, ids, nq.lrb_linear(layer, x))
    assert torch.equal(nq.lrb_lora_linear(layer, pool, x, ids), want)


@gpu
def test_binding_refuses_wrong_tensors():
    c = _case("refuse", 5, 2, 4, 16, 8)
    pool, x, ids = _gpu_pool(c), _dev(c["x"], "bf16"), _dev(c["ids"])
    bad = [dict(x=x[:, :8].contiguous()), dict(ids=ids.long()), dict(ids=ids[:4].contiguous()), dict(ids=ids.cpu()),
           dict(base=torch.zeros(5, 9, device=DEV)), dict(base=torch.zeros(5, 8, device=DEV, dtype=torch.bfloat16)),
           dict(y=torch.zeros(4, 8, device=DEV)), dict(x=x.half()), dict(x=x.t().contiguous().t()),
           dict(workspace=torch.empty(1 << 20, dtype=torch.uint8)),
           dict(workspace=torch.empty(1 << 20, 2, dtype=torch.uint8, device=DEV)[:, 0])]
    for kw in bad:
        with pytest.raises(ValueError):
            nq.lora_linear(**{**dict(pool=pool, x=x, ids=ids), **kw})
    with pytest.raises(ValueError):
        nq.lora_grads(pool, x, torch.zeros(5, 9, device=DEV), ids)
    with pytest.raises(ValueError):
        nq.lora_grads(pool, x, torch.zeros(5, 8, device=DEV), ids, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError):
        nq.lora_grads(pool, x, torch.zeros(5, 8, device=DEV), ids, dx_base=torch.zeros(5, 15, device=DEV))
    with pytest.raises(nq.NqError):
        nq.lora_linear(pool, x, ids, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


def _non_finite(tag, T, n, r, d_in, d_out, xd, wd):
    """Small integers (hidden values of few bits) with infinities and NaN in factors, activations, g and base."""
    g = synth.rng(f"lora/inf/{tag}")
    ids = np.arange(T) % n
    few = [-2, -1, 1, 2]  # no zeros, beside which an infinity is NaN
    c = dict(a=g.integers(-2, 3, (n, r, d_in)), b=g.choice(few, (n, d_out, r)), scale=np.full(n, 0.5),
             x=g.choice(few, (T, d_in)), base=g.integers(-9, 10, (T, d_out)), g=g.choice(few, (T, d_out)),
             dx_base=g.integers(-9, 10, (T, d_in)))
    c = {k: v.astype(np.float32) for k, v in c.items()}
    c.update(ids=ids.astype(np.int32), xd=xd, wd=wd)
    c["b"][1, 7, 2] = np.inf          # one column of adapter 1's rows
    c["b"][2, :3, 0] = [-np.inf, np.nan, np.inf]
    c["a"][3, r - 1, 5] = -np.inf     # one hidden value of adapter 3's tokens
    c["x"][0, 4] = np.inf             # adapter 0
    c["g"][0, 3] = -np.inf
    c["g"][T // 2, 1] = np.nan
    c["base"][T - 1, 1] = c["dx_base"][T - 1, 2] = np.inf
    return c


def _same_class(got, want):
    got = got.cpu().numpy().astype(np.float64)
    for f in (np.isnan, np.isposinf, np.isneginf):
        assert np.array_equal(f(got), f(want)), (f.__name__, np.argwhere(f(got) != f(want))[:5])
    fine = np.isfinite(want)
    assert np.array_equal(got[fine], want[fine])  # integers and halves: exact


@gpu
@pytest.mark.parametrize("xd,wd", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("T,d_in", [(4, 90), (20, 90), (96, 90), (96, 520)])
def test_non_finite_values_are_those_of_the_formula(T, d_in, xd, wd):
    """Element by element: infinite where the formula's products and sums are, NaN where they are not a number,
    the same at any number of tokens."""
    c = _non_finite(f"{T}/{d_in}", T, 4, 12, d_in, 60, xd, wd)
    with np.errstate(invalid="ignore"):
        want = A.lora_linear_ref(c["a"], c["b"], c["scale"], c["x"], c["ids"], c["base"])
    _same_class(nq.lora_linear(_gpu_pool(c), _dev(c["x"], xd), _dev(c["ids"]), _dev(c["base"])), want)


@gpu
@pytest.mark.parametrize("xd,wd", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("T,d_in,d_out", [(20, 90, 60), (96, 520, 600)])
def test_non_finite_gradients_are_those_of_the_formula(T, d_in, d_out, xd, wd):
    c = _non_finite(f"g/{T}/{d_in}", T, 4, 12, d_in, d_out, xd, wd)
    with np.errstate(invalid="ignore"):
        want = A.lora_grads_ref(c["a"], c["b"], c["scale"], c["x"], c["g"], c["ids"], c["dx_base"])
    got = nq.lora_grads(_gpu_pool(c), _dev(c["x"], xd), _dev(c["g"], xd), _dev(c["ids"]), _dev(c["dx_base"]))
    for v, w in zip(got, want):
        _same_class(v, w)
