"""Timed cases of distillation from a teacher's top logits and of the packed linear's epilogue.

Five operators of a step of scale-only reconstruction: `top` (a teacher's top
logits and the mass of the rest), `loss` and `grads` (the divergence of a
student's logits from them, and its gradient), `linear` (a packed low-rank
binary linear with bias, activation, gate and residual) and `act_grads` (the
gradients of that epilogue).  `run` computes them from elementary torch
operations in 32 bits, or, with `own`, through sub_bit_weight_amd.  `exact` is
their definition in 64 bits.

Layer sizes and ranks are those of this repository's configurations (256, 4096,
8192, 11008, 28672) or generic; vocabulary sizes are generic.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def listed():
    def top(name, **k):
        return {"name": name, "op": "top", **k}

    def loss(name, **k):
        return {"name": name, "op": "loss", **k}

    def grads(name, **k):
        return {"name": name, "op": "grads", **k}

    def linear(name, **k):
        return {"name": name, "op": "linear", **k}

    def act_grads(name, **k):
        return {"name": name, "op": "act_grads", **k}

    return [
        # one position's record of a teacher that answers: latency
        top("top one row", T=1, V=32000, k=64, dtype="bf16", tau=1.0),
        # recording a teacher over a calibration sequence of 2048 tokens
        top("top calibration sequence", T=2048, V=32000, k=64, dtype="bf16", tau=1.0),
        # watching the divergence of a few positions of a small vocabulary: latency
        loss("loss few rows", T=8, V=4096, k=16, dtype="f32", tau=1.0, rest=True),
        # evaluating a calibration set against a recorded teacher with a large vocabulary
        loss("loss evaluation", T=2048, V=131072, k=128, dtype="bf16", tau=1.0, rest=True),
        # a step on a short sequence in full precision, odd sizes throughout, a softened teacher made to sum to one
        grads("grads odd f32", T=301, V=50021, k=37, dtype="f32", tau=2.0, rest=False),
        # a step on a calibration sequence of 2048 tokens
        grads("grads calibration sequence", T=2048, V=32000, k=64, dtype="bf16", tau=1.0, rest=True),
        # the largest: two long sequences with a large vocabulary
        grads("grads large vocabulary", T=4096, V=131072, k=128, dtype="bf16", tau=1.0, rest=True),
        # the smallest layer, one token in full precision: latency
        linear("linear one token", T=1, d_out=256, d_in=256, r=64, dtype="f32", act="gelu", bias=True, mul=False,
               residual=False, z=False),
        # a decode step of eight requests through a gate projection: silu times the up projection's output
        linear("linear decode gate", T=8, d_out=11008, d_in=4096, r=2368, dtype="bf16", act="silu", bias=False,
               mul=True, residual=False, z=False),
        # a calibration sequence through the widest gate projection, z kept for the backward pass
        linear("linear sequence gate", T=2048, d_out=28672, d_in=8192, r=6336, dtype="bf16", act="silu", bias=False,
               mul=True, residual=False, z=True),
        # a short sequence in full precision through odd sizes
        act_grads("act_grads odd f32", T=77, d=1117, dtype="f32", act="gelu", mul=False),
        # the backward pass of the widest gate projection over a calibration sequence
        act_grads("act_grads sequence gate", T=2048, d=28672, dtype="bf16", act="silu", mul=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(rng, v):
    """Half of the sizes as they are drawn, the others a multiple of 16."""
    return v if rng.random() < 0.5 or v < 32 else v // 16 * 16


def draw(rng):
    op = rng.choice(["top", "loss", "grads", "grads", "linear", "linear", "act_grads"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("top", "loss", "grads"):
        V = _odd(rng, _log(rng, 200, 131072))
        T = min(_log(rng, 1, 8192), (1 << 28) // V)
        case = {"op": op, "T": T, "V": V, "k": _log(rng, 1, min(256, V // 2)), "dtype": dtype,
                "tau": rng.choice([1.0, 1.0, 2.0, 0.7])}
        return case if op == "top" else {**case, "rest": rng.random() < 0.6}
    act, mul = rng.choice(ACTS), rng.random() < 0.5
    if op == "act_grads":
        d = _odd(rng, _log(rng, 64, 28672))
        return {"op": op, "T": min(_log(rng, 1, 8192), (1 << 26) // d), "d": d, "dtype": dtype, "act": act, "mul": mul}
    d_in, d_out = _odd(rng, _log(rng, 64, 11008)), _odd(rng, _log(rng, 64, 28672))
    r = _odd(rng, max(8, int(d_in * d_out / (d_in + d_out) * rng.uniform(0.25, 1.0))))
    return {"op": op, "T": _log(rng, 1, 8) if rng.random() < 0.5 else _log(rng, 9, 2048), "d_out": d_out, "d_in": d_in,
            "r": r, "dtype": dtype, "act": act, "bias": rng.random() < 0.5, "mul": mul, "residual": rng.random() < 0.5,
            "z": rng.random() < 0.25}


# ---------------------------------------------------------------- inputs


def _words(gen, n_red, n_out):
    """Random sign words [ceil(n_red/32)][n_out]; bits past the reduction are 0."""
    nw = (n_red + 31) // 32
    w = torch.randint(-(1 << 31), 1 << 31, (nw, n_out), device=DEV, generator=gen, dtype=torch.int64)
    if n_red % 32:
        w[-1] &= (1 << (n_red % 32)) - 1
    return w.to(torch.int32)


def _padding(case):
    """Padding rows at a batch's end (weight zero): one in sixteen."""
    return case["T"] // 16


def _inputs(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, device=DEV, generator=gen)

    T = case["T"]
    if case["op"] == "linear":
        d_out, d_in, r = case["d_out"], case["d_in"], case["r"]
        s = {"u_bits": _words(gen, r, d_out), "vt_bits": _words(gen, d_in, r), "s1": normal(d_out).abs() / math.sqrt(r),
             "s2": normal(d_in).abs() / math.sqrt(d_in), "x": normal(T, d_in).to(dt)}
        s["bias"] = 0.5 * normal(d_out) if case["bias"] else None
        s["mul"] = normal(T, d_out).to(dt) if case["mul"] else None
        s["residual"] = normal(T, d_out).to(dt) if case["residual"] else None
        return s
    if case["op"] == "act_grads":
        d = case["d"]
        return {"zin": normal(T, d).to(dt), "dy": (0.01 * normal(T, d)).to(dt),
                "mul": normal(T, d).to(dt) if case["mul"] else None}
    # a teacher: a broad floor and a few likely tokens in each row; a student that has most of it
    V, k = case["V"], case["k"]
    z = normal(T, V)
    likely = torch.randint(0, V, (T, 12), device=DEV, generator=gen)
    z.scatter_add_(1, likely, 4.0 + 6.0 * torch.rand(T, 12, device=DEV, generator=gen))
    if case["op"] == "top":
        return {"logits": z.to(dt)}
    values, ids = torch.topk(z, k, dim=1)
    lse = torch.logsumexp(z.double() / case["tau"], 1, keepdim=True) if T * V <= 1 << 24 else torch.logsumexp(
        z / case["tau"], 1, keepdim=True).double()
    logp = (values.double() / case["tau"] - lse).float()
    rest = torch.log1p(-torch.exp(logp.double()).sum(1).clamp(max=1 - 1e-6)).float()
    weight = (0.5 + torch.rand(T, device=DEV, generator=gen)) / T
    weight[T - _padding(case):] = 0.0
    logits = z.add_(normal(T, V), alpha=0.7).to(dt)
    return {"logits": logits, "ids": ids.to(torch.int32), "logp": logp, "rest": rest if case["rest"] else None,
            "weight": weight}


def prepare(case, seed):
    s = {**{k: case.get(k) for k in ("op", "k", "tau", "act", "r", "d_in", "d_out")}, "keep_z": case.get("z", False),
         **_inputs(case, seed)}
    if own:  # what a program makes once: the layer's handle, the teacher's record
        import sub_bit_weight_amd as nq
        if case["op"] == "linear":
            s["layer"] = nq.Lrb(s["d_out"], s["d_in"], s["r"], s["u_bits"], s["vt_bits"], s["s1"], s["s2"])
        if case["op"] in ("loss", "grads"):
            s["teacher"] = nq.Teacher(s["ids"], s["logp"], s["rest"], s["tau"])
    return s


# ---------------------------------------------------------------- the operators


def _top(s):
    z = s["logits"].float()
    values, order = torch.sort(z, dim=1, descending=True, stable=True)
    e = torch.exp((values - values[:, :1]) / s["tau"])
    lse = values[:, :1] / s["tau"] + torch.log(e.sum(1, keepdim=True))
    k = s["k"]
    ids, values, tail, below = order[:, :k], values[:, :k], e[:, k:], values[:, :1]
    return {"ids": ids.to(torch.int32), "logp": values / s["tau"] - lse,
            "rest": below[:, 0] / s["tau"] + torch.log(tail.sum(1)) - lse[:, 0]}


def _lse(x):
    """In 64 bits: the divergence is a small difference of such numbers."""
    m = x.amax(1, keepdim=True)
    return m.double() + torch.log(torch.exp(x - m).sum(1, keepdim=True, dtype=torch.float64))


def _teacher(s):
    """Listed probabilities and their logarithms, and those of the rest (0 and -inf where the list sums to one)."""
    logp = s["logp"].double()
    if s["rest"] is None:
        logp = logp - torch.log(torch.exp(logp).sum(1, keepdim=True))
        rest = torch.full_like(logp[:, :1], -math.inf)
    else:
        rest = s["rest"].double()[:, None]
    return torch.exp(logp), logp, torch.exp(rest), rest


def _distill(s, grads):
    x = s["logits"].float() / s["tau"]
    ids = s["ids"].long()
    p, logp, r, rest = _teacher(s)
    lse = _lse(x)
    away = x.scatter(1, ids, -math.inf)
    away_lse = _lse(away)
    loss = (p * (logp - (torch.gather(x, 1, ids) - lse))).sum(1)
    if s["rest"] is not None:
        loss = loss + (r * (rest - (away_lse - lse)))[:, 0]
    loss = (s["weight"] * loss).float()
    if not grads:
        return loss
    c = s["weight"][:, None] / s["tau"]
    mass = (p.sum(1, keepdim=True) + r).float()
    d = mass * torch.exp(x - lse.float()) - r.float() * torch.exp(away - away_lse.float())
    d = c * d.scatter_add(1, ids, -p.float())
    return {"loss": loss, "dlogits": d.to(s["logits"].dtype)}


def _signs(words, n_red):
    """[n_red][n_out] of +-1 from sign words [ceil(n_red/32)][n_out]."""
    bits = (words[:, None, :] >> torch.arange(32, device=DEV, dtype=torch.int32)[None, :, None]) & 1
    return (1 - 2 * bits).reshape(-1, words.shape[1])[:n_red].float()


def _act(name, z):
    """act(z) and its derivative."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z * (z > 0), (z > 0).to(z.dtype)
    if name == "silu":
        q = 1 / (1 + torch.exp(-z))
        return z * q, q * (1 + z * (1 - q))
    if name == "gelu":
        cdf = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    a = math.sqrt(2 / math.pi)
    t = torch.tanh(a * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)


def _linear(s):
    dt = s["x"].dtype
    t = torch.matmul(s["x"].float() * s["s2"], _signs(s["vt_bits"], s["d_in"]))
    z = torch.matmul(t, _signs(s["u_bits"], s["r"])) * s["s1"]
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(s["act"], z)[0]
    if s["mul"] is not None:
        y = y * s["mul"].float()
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(dt), "z": z.to(dt)} if s["keep_z"] else {"y": y.to(dt)}


def _act_grads(s):
    dt = s["dy"].dtype
    a, da = _act(s["act"], s["zin"].float())
    dy = s["dy"].float()
    dz = dy * da
    if s["mul"] is None:
        return {"dz": dz.to(dt), "dbias": dz.sum(0)}
    dz = dz * s["mul"].float()
    return {"dz": dz.to(dt), "dbias": dz.sum(0), "dmul": (dy * a).to(dt)}


def run(s):
    op = s["op"]
    if own:
        import sub_bit_weight_amd as nq
        if op == "top":
            t = nq.logits_top(s["logits"], s["k"], temperature=s["tau"])
            return {"ids": t.ids, "logp": t.logp, "rest": t.rest}
        if op == "loss":
            return nq.distill_loss(s["teacher"], s["logits"], weight=s["weight"])
        if op == "grads":
            loss, dlogits = nq.distill_grads(s["teacher"], s["logits"], weight=s["weight"])
            return {"loss": loss, "dlogits": dlogits}
        if op == "linear":
            z = torch.empty(s["x"].shape[0], s["d_out"], dtype=s["x"].dtype, device=DEV) if s["keep_z"] else None
            y = nq.lrb_linear_act(s["layer"], s["x"], act=s["act"], bias=s["bias"], mul=s["mul"],
                                  residual=s["residual"], z=z)
            return {"y": y, "z": z} if s["keep_z"] else {"y": y}
        dz, dmul, dbias = nq.act_grads(s["act"], s["zin"], s["dy"], mul=s["mul"])
        return {"dz": dz, "dbias": dbias} if dmul is None else {"dz": dz, "dbias": dbias, "dmul": dmul}
    if op == "top":
        return _top(s)
    if op in ("loss", "grads"):
        return _distill(s, op == "grads")
    return _linear(s) if op == "linear" else _act_grads(s)


# ---------------------------------------------------------------- the definition in 64 bits


def _exact_distill(case, s):
    """Rows in blocks, as the sums over probabilities that define the divergence."""
    losses, grads = [], []
    T, V = s["logits"].shape
    step = max(1, (1 << 27) // V)
    for t0 in range(0, T, step):
        x, ids, logp, w = (s[k][t0:t0 + step] for k in ("logits", "ids", "logp", "weight"))
        ids = ids.long()
        logq = torch.log_softmax(x.double() / case["tau"], 1)
        p = torch.exp(logp)
        if s["rest"] is None:
            p = p / p.sum(1, keepdim=True)
        listed = torch.zeros(x.shape, dtype=torch.bool, device=DEV).scatter_(1, ids, True)
        q = torch.exp(logq)
        away = torch.where(listed, torch.zeros_like(q), q)
        loss = (p * (torch.log(p) - torch.gather(logq, 1, ids))).sum(1)
        d = -torch.zeros_like(q).scatter_add_(1, ids, p)
        mass = p.sum(1, keepdim=True)
        if s["rest"] is not None:
            r, m = torch.exp(s["rest"][t0:t0 + step]), away.sum(1)
            loss = loss + r * (torch.log(r) - torch.log(m))
            d -= away * (r / m)[:, None]
            mass = mass + r[:, None]
        losses.append(w * loss)
        if case["op"] == "grads":
            d += q * mass
            d *= w[:, None] / case["tau"]
            grads.append(d)
    loss = torch.cat(losses)
    return {"loss": loss, "dlogits": torch.cat(grads)} if case["op"] == "grads" else loss


def _exact_signs(words, n_red):
    """[n_out][n_red] of +-1 by a table of the bytes' bits."""
    table = torch.tensor([[-1.0 if b >> i & 1 else 1.0 for i in range(8)] for b in range(256)], dtype=torch.float64,
                         device=DEV)
    n = words.shape[1]
    octets = words.T.contiguous().view(torch.uint8).reshape(n, -1)  # little-endian: element 8j + i in bit i of byte j
    return table[octets.long()].reshape(n, -1)[:, :n_red]


def _exact_act(name, z):
    if name == "silu":
        q = torch.sigmoid(z)
        return z * q, q + z * q * (1 - q)
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        a, b = math.sqrt(2 / math.pi), 0.044715
        q = torch.sigmoid(2 * a * (z + b * z ** 3))
        return z * q, q + z * q * (1 - q) * 2 * a * (1 + 3 * b * z ** 2)
    return (torch.clamp(z, min=0.0), (z > 0).double()) if name == "relu" else (z, torch.ones_like(z))


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] in ("loss", "grads"):
        keep = s["logits"]
        s = {k: v.double() if v is not None and v.is_floating_point() and v is not keep else v for k, v in s.items()}
        return _exact_distill(case, s)
    s = {k: v.double() if v is not None and v.is_floating_point() else v for k, v in s.items()}
    if case["op"] == "top":
        z, k = s["logits"], case["k"]
        order = torch.argsort(z, dim=1, descending=True, stable=True)
        logp = torch.log_softmax(z / case["tau"], 1)
        ids = order[:, :k]
        return {"ids": ids.to(torch.int32), "logp": torch.gather(logp, 1, ids),
                "rest": torch.logsumexp(torch.gather(logp, 1, order[:, k:]), 1)}
    if case["op"] == "linear":
        u, vt = _exact_signs(s["u_bits"], case["r"]), _exact_signs(s["vt_bits"], case["d_in"])
        z = s["s1"] * ((s["s2"] * s["x"]) @ vt.T @ u.T) + (0 if s["bias"] is None else s["bias"])
        y = _exact_act(case["act"], z)[0] * (1 if s["mul"] is None else s["mul"]) + (
            0 if s["residual"] is None else s["residual"])
        return {"y": y, "z": z} if case["z"] else {"y": y}
    a, da = _exact_act(case["act"], s["zin"])
    dz = s["dy"] * da * (1 if s["mul"] is None else s["mul"])
    return {"dz": dz, "dbias": dz.sum(0)} if s["mul"] is None else {"dz": dz, "dbias": dz.sum(0), "dmul": s["dy"] * a}


# ---------------------------------------------------------------- the least work


def work(case):
    op, T, e = case["op"], case["T"], SIZE[case["dtype"]]
    if op == "linear":
        d_out, d_in, r = case["d_out"], case["d_in"], case["r"]
        signs = 4 * (d_out * ((r + 31) // 32) + r * ((d_in + 31) // 32))
        rows = 1 + case["mul"] + case["residual"] + case["z"]
        return {"bytes": signs + 4 * (d_out + d_in + d_out * case["bias"]) + e * T * (d_in + rows * d_out),
                "flops": 2.0 * T * r * (d_in + d_out)}
    if op == "act_grads":
        n = T * case["d"]
        return {"bytes": n * e * (5 if case["mul"] else 3 - (case["act"] == "none")) + 4 * case["d"], "flops": 10.0 * n}
    V, k = case["V"], case["k"]
    if op == "top":
        return {"bytes": T * V * e + T * (8 * k + 4), "flops": 4.0 * T * V}
    rows = T - _padding(case)
    return {"bytes": rows * (V * e + 8 * k) + T * (8 + 4 * case["rest"]) + (T * V * e if op == "grads" else 0),
            "flops": (8.0 if op == "grads" else 4.0) * rows * V}
