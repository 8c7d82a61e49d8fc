"""Timed cases of the low-rank adapter operators and of the orthogonalised update.

Three operators: `linear` (adapters of many requests beside a shared
projection), `grads` (the gradients of the adapters and of the input) and
`orthogonalize` (the Newton-Schulz iteration that makes an update of a factor's
gradient).  `run` computes them from elementary torch operations in 32 bits, or,
with `own`, through sub_bit_weight_amd.  `exact` is their definition in 64 bits.

Layer sizes are those of this repository's configurations (256, 4096, 8192,
11008, 28672) or generic; ranks and request counts are those of adapter serving
and training in general.
"""
import math

import torch

own = False

DEV = "cuda"
NS = (3.4445, -4.7750, 2.0315)  # quintic Newton-Schulz coefficients
STEPS = 5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    def linear(name, **k):
        return {"name": name, "op": "linear", **k}

    def grads(name, **k):
        return {"name": name, "op": "grads", **k}

    def ortho(name, **k):
        return {"name": name, "op": "orthogonalize", **k}

    return [
        # one request decoding one token through the smallest layer: latency
        linear("linear one token", T=1, n=8, r=16, d_in=256, d_out=256, dtype="bf16", mixed=True),
        # a decode step of 48 requests, nearly each with an adapter of its own, on a wide up-projection
        linear("linear decode step", T=48, n=64, r=16, d_in=8192, d_out=28672, dtype="bf16", mixed=True),
        # prompts of a few requests, one after another, on a square projection
        linear("linear prompts", T=2048, n=8, r=16, d_in=8192, d_out=8192, dtype="bf16", mixed=False),
        # adapters still in training precision, odd sizes throughout
        linear("linear odd f32", T=777, n=5, r=41, d_in=4099, d_out=1117, dtype="f32", mixed=False),
        # the largest: long prompts of many requests with wide adapters on a wide projection
        linear("linear long prompts", T=8192, n=32, r=64, d_in=8192, d_out=28672, dtype="bf16", mixed=False),
        # a few short sequences of a small layer in full precision: latency
        grads("grads small f32", T=16, n=4, r=8, d_in=256, d_out=256, dtype="f32", mixed=False),
        # fine-tuning a handful of adapters of an up-projection at once
        grads("grads up-projection", T=2048, n=4, r=16, d_in=4096, d_out=11008, dtype="bf16", mixed=False),
        # odd sizes, tokens of all adapters mixed
        grads("grads odd f32", T=1501, n=7, r=24, d_in=1001, d_out=1703, dtype="f32", mixed=True),
        # the largest: a full batch with wide adapters on a square projection
        grads("grads full batch", T=8192, n=16, r=64, d_in=8192, d_out=8192, dtype="bf16", mixed=False),
        # the gradients of 64 adapters' A factors, updated together
        ortho("orthogonalize adapters", batch=64, rows=16, cols=4096, dtype="f32", out="f32"),
        # two odd tall factors kept in full precision
        ortho("orthogonalize odd f32", batch=2, rows=2203, cols=1371, dtype="f32", out="f32"),
        # the latent factor of an up-projection, its update applied in bf16
        ortho("orthogonalize latent", batch=1, rows=11008, cols=4096, dtype="f32", out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(rng, v):
    """Half of the sizes as they are drawn, the others a multiple of 16."""
    return v if rng.random() < 0.5 or v < 32 else v // 16 * 16


def draw(rng):
    op = rng.choice(["linear", "linear", "grads", "grads", "orthogonalize"])
    if op == "orthogonalize":
        rows, cols = _odd(rng, _log(rng, 4, 4096)), _odd(rng, _log(rng, 16, 8192))
        if rng.random() < 0.5:
            rows, cols = cols, rows
        batch = max(1, min(_log(rng, 1, 64), (1 << 24) // (rows * cols)))
        return {"op": op, "batch": batch, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "f32"]),
                "out": rng.choice(["bf16", "f32"])}
    d_in, d_out = _odd(rng, _log(rng, 64, 8192)), _odd(rng, _log(rng, 64, 8192 if op == "grads" else 16384))
    n, r = _log(rng, 1, 48), _odd(rng, _log(rng, 2, 64))
    T = min(_log(rng, 1, 8192), (8192 * 16 * 64) // (n * r) + 1)
    return {"op": op, "T": T, "n": n, "r": r, "d_in": d_in, "d_out": d_out, "dtype": rng.choice(["bf16", "bf16", "f32"]),
            "mixed": T <= 64 or rng.random() < 0.3}


# ---------------------------------------------------------------- inputs


def _ids(case, gen):
    """Adapter of each token; about one request in eight has none.  mixed: every
    token is a request of its own; otherwise requests of uneven lengths follow
    one another."""
    T, n = case["T"], case["n"]
    if case["mixed"]:
        request = torch.arange(T, device=DEV)
    else:
        new = torch.rand(T, device=DEV, generator=gen) < 2.0 * n / T
        request = torch.cumsum(new, 0)
    adapter = torch.randint(0, n, (T + 1,), device=DEV, generator=gen, dtype=torch.int32)
    none = torch.rand(T + 1, device=DEV, generator=gen) < 0.125
    none[0] = False
    return torch.where(none, torch.full_like(adapter, -1), adapter)[request].contiguous()


def _inputs(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, device=DEV, generator=gen)

    if case["op"] == "orthogonalize":
        b, m, n = case["batch"], case["rows"], case["cols"]
        # a gradient: a few strong directions over a flat floor, rows and columns of uneven size
        k = max(1, min(m, n) // 8)
        u, v = normal(b, m, k), normal(b, k, n)
        x = torch.matmul(u * torch.exp(-4.0 * torch.arange(k, device=DEV) / k), v) / math.sqrt(k) + 0.5 * normal(b, m, n)
        x = x * torch.exp(0.5 * normal(b, m, 1)) * (1e-3 * torch.exp(0.5 * normal(b, 1, n)))
        return {"x": x.to(dt)}
    T, n, r, d_in, d_out = (case[k] for k in ("T", "n", "r", "d_in", "d_out"))
    s = {"ids": _ids(case, gen), "x": normal(T, d_in).to(dt),
         "a": (normal(n, r, d_in) / math.sqrt(d_in)).to(dt), "b": (0.3 * normal(n, d_out, r) / math.sqrt(r)).to(dt),
         "scale": torch.exp(0.25 * normal(n))}
    if case["op"] == "linear":
        s["base"] = normal(T, d_out)
    else:
        s["g"] = (0.01 * normal(T, d_out)).to(dt)
        s["dx_base"] = 0.01 * normal(T, d_in)
    return s


def prepare(case, seed):
    s = {"op": case["op"], "out": TYPES[case.get("out", "f32")], **_inputs(case, seed)}
    if own and case["op"] != "orthogonalize":  # the pool of adapters that a program loads once
        import sub_bit_weight_amd as nq
        s["pool"] = nq.Lora(s["a"], s["b"], s["scale"])
    return s


# ---------------------------------------------------------------- the operators


def _hidden(x, w, ids):
    """Tokens [T][d] times every adapter's [r][d] rows: [T][n*r], zero but at the token's own adapter."""
    n, r, d = w.shape
    keep = ids.long()[:, None] == torch.arange(n, device=DEV).repeat_interleave(r)
    return torch.matmul(x, w.reshape(n * r, d).T) * keep


def _linear(s):
    x, a, b, ids = s["x"].float(), s["a"].float(), s["b"].float(), s["ids"].long()
    n, d_out, r = b.shape
    if x.shape[0] <= 64:  # few tokens: each one's own factors
        i = ids.clamp(min=0)
        h = torch.bmm(a[i], x[:, :, None]) * (s["scale"][i] * (ids >= 0))[:, None, None]
        return s["base"] + torch.bmm(b[i], h)[:, :, 0]
    h = _hidden(x, a, ids) * s["scale"].repeat_interleave(r)
    return s["base"] + torch.matmul(h, b.permute(0, 2, 1).reshape(n * r, d_out))


def _grads(s):
    x, g, a, b, ids = s["x"].float(), s["g"].float(), s["a"].float(), s["b"].float(), s["ids"]
    n, d_out, r = b.shape
    d_in = a.shape[2]
    scale = s["scale"].repeat_interleave(r)
    h = _hidden(x, a, ids) * scale
    dh = _hidden(g, b.permute(0, 2, 1).contiguous(), ids) * scale
    dx = s["dx_base"] + torch.matmul(dh, a.reshape(n * r, d_in))
    da = torch.matmul(dh.T, x).reshape(n, r, d_in)
    db = torch.matmul(h.T, g).reshape(n, r, d_out).permute(0, 2, 1).contiguous()
    return {"dx": dx, "da": da, "db": db}


def _orthogonalize(s):
    x = s["x"].float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    x = x / torch.sqrt((x * x).sum((1, 2), keepdim=True))
    for _ in range(STEPS):
        gram = torch.matmul(x, x.transpose(1, 2).contiguous())
        x = NS[0] * x + torch.matmul(NS[1] * gram + NS[2] * torch.matmul(gram, gram), x)
    return (x.transpose(1, 2) if tall else x).to(s["out"]).contiguous()


def run(s):
    if own:
        import sub_bit_weight_amd as nq
        if s["op"] == "linear":
            return nq.lora_linear(s["pool"], s["x"], s["ids"], base=s["base"])
        if s["op"] == "grads":
            dx, da, db = nq.lora_grads(s["pool"], s["x"], s["g"], s["ids"], dx_base=s["dx_base"])
            return {"dx": dx, "da": da, "db": db}
        return nq.orthogonalize(s["x"], steps=STEPS, coeffs=NS, out_dtype=s["out"])
    return {"linear": _linear, "grads": _grads, "orthogonalize": _orthogonalize}[s["op"]](s)


# ---------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    s = {k: v.double() if v.is_floating_point() else v for k, v in _inputs(case, seed).items()}
    if case["op"] == "orthogonalize":
        out = []
        for x in s["x"]:
            x = x / torch.linalg.vector_norm(x)
            for _ in range(STEPS):  # from whichever side is the shorter: the same polynomial of x
                if x.shape[0] <= x.shape[1]:
                    p = x @ x.T
                    x = NS[0] * x + NS[1] * (p @ x) + NS[2] * (p @ (p @ x))
                else:
                    p = x.T @ x
                    x = NS[0] * x + NS[1] * (x @ p) + NS[2] * ((x @ p) @ p)
            out.append(x)
        return torch.stack(out)
    y = s["base"].clone() if case["op"] == "linear" else None
    dx = None if y is not None else s["dx_base"].clone()
    da, db = torch.zeros_like(s["a"]), torch.zeros_like(s["b"])
    for i in range(case["n"]):
        t = (s["ids"] == i).nonzero()[:, 0]
        x, a, b, c = s["x"][t], s["a"][i], s["b"][i], s["scale"][i]
        if y is not None:
            y[t] += c * ((x @ a.T) @ b.T)
        else:
            g = s["g"][t]
            dx[t] += c * ((g @ b) @ a)
            da[i] = c * ((g @ b).T @ x)
            db[i] = c * (g.T @ (x @ a.T))
    return y if y is not None else {"dx": dx, "da": da, "db": db}


# ---------------------------------------------------------------- the least work


def work(case):
    if case["op"] == "orthogonalize":
        b, m, n = case["batch"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
        # symmetric products by one half; the iteration on x itself, or on the m x m product with x applied at the end
        direct = STEPS * (3.0 * m * m * n + m ** 3)
        gram = 3.0 * m * m * n + STEPS * 4.0 * m ** 3
        return {"bytes": b * m * n * (SIZE[case["dtype"]] + SIZE[case["out"]]), "flops": b * min(direct, gram)}
    T, n, r, d_in, d_out, e = (case[k] for k in ("T", "n", "r", "d_in", "d_out", "dtype"))
    used = n * (1.0 - (1.0 - 1.0 / n) ** min(T, 2 * n if not case["mixed"] else T)) if n > 1 else 1.0
    weights = used * r * (d_in + d_out) * SIZE[e]
    if case["op"] == "linear":
        return {"bytes": T * d_in * SIZE[e] + weights + 8 * T * d_out + 4 * T, "flops": 2.0 * T * r * (d_in + d_out)}
    return {"bytes": T * (d_in + d_out) * SIZE[e] + weights + 8 * T * d_in + 4 * n * r * (d_in + d_out) + 4 * T,
            "flops": 2.0 * T * r * (3 * d_in + 2 * d_out)}
