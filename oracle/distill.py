"""fp64 references of distillation from a teacher's top logits and of the packed
linear's epilogue (test infrastructure; numpy only, nothing here reads the GPU
library)."""
from __future__ import annotations

import math

import numpy as np

EPS32 = 2.0 ** -24  # half a step of fp32, relative


def _lse(x):
    m = np.max(x) if x.size else -np.inf
    if np.isnan(x).any():
        return np.nan
    return m if not np.isfinite(m) else m + math.log(np.exp(x - m).sum())


def _scaled(row, tau):
    """row / tau less a constant that no probability depends on, the largest finite logit's: at 3e38 a logarithm of a
    count would not change even an fp64 number."""
    fine = row[np.isfinite(row)]
    return (row - (fine.max() if fine.size else 0.0)) / tau


def logits_top_ref(z, k, tau):
    """(ids [T][k], logp [T][k], rest [T]): the k largest of each row, equal ones by index (NaN above all), -inf
    never listed."""
    z = np.asarray(z, dtype=np.float64)
    T, V = z.shape
    ids, logp, rest = np.full((T, k), -1, np.int32), np.full((T, k), -np.inf), np.full(T, -np.inf)
    for t in range(T):
        row = z[t]
        order = np.lexsort((np.arange(V), -np.where(np.isnan(row), 0.0, row), ~np.isnan(row)))
        order = order[~np.isneginf(row[order])][:k]
        with np.errstate(invalid="ignore"):
            x = _scaled(row, tau)
            lse = _lse(x) if not np.isposinf(row).any() else np.nan
            ids[t, :len(order)] = order
            logp[t, :len(order)] = x[order] - lse
            away = np.delete(x, order)
            rest[t] = np.nan if np.isnan(lse) else _lse(away) - lse if np.isfinite(away).any() else -np.inf
    return ids, logp, rest


def distill_ref(ids, logp, rest, tau, s, weight=None):
    """(loss [T], gradient [T][V]) of the divergence of softmax(s / tau) from the record."""
    s, logp = np.asarray(s, dtype=np.float64), np.asarray(logp, dtype=np.float64)
    T, V = s.shape
    loss, grad = np.zeros(T), np.zeros((T, V))
    for t in range(T):
        w = 1.0 if weight is None else float(weight[t])
        if w == 0.0:
            continue
        if (ids[t] >= V).any():
            loss[t], grad[t] = np.nan, np.nan
            continue
        e = ids[t] >= 0
        v, lp = ids[t][e], logp[t][e]
        p = np.exp(lp)
        r = 0.0 if rest is None else math.exp(rest[t])
        if p.sum() + r == 0.0:
            continue
        if rest is None:
            lp = lp - math.log(p.sum())
            p = np.exp(lp)
        x = _scaled(s[t], tau)
        with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
            lse = _lse(x) if not np.isposinf(x).any() and not np.isneginf(x).all() else np.nan
            logq = x - lse
            q = np.exp(logq)
            listed = np.zeros(V, bool)
            listed[v] = True
            away = _lse(x[~listed])
            on = p > 0
            loss[t] = w * ((p[on] * (lp[on] - logq[v[on]])).sum() + (r * (rest[t] - (away - lse)) if r > 0 else 0.0))
            g = (p.sum() + r) * q
            np.subtract.at(g, v, p)
            if r > 0 and np.isfinite(away):
                g[~listed] -= r * np.exp(x[~listed] - away)
        grad[t] = w / tau * g
    return loss, grad


def exp_error(x, listed, threads):
    """Bound of the relative error of the sum over the tokens not listed of exp(x - max x), x = logits / tau, from fp32
    exponentials added in fp32 by `threads` threads: each exponent y = (x - max) log2(e) carries three
    roundings of its size (the difference, the product, the sum of its parts; ln 2 of them each reach the value),
    exp2 two units in the last place, and a thread adds ceil(V / threads) terms."""
    away = np.asarray(x, dtype=np.float64)[~listed]
    away = away[np.isfinite(away)]
    if not away.size:
        return 0.0
    d = away - away.max()
    e = np.exp(d)
    each = (3 * np.abs(d) + 4) * EPS32
    return float((e * each).sum() / e.sum()) + (math.ceil(len(x) / threads) + 8) * EPS32


def act_ref(name, z):
    """(act(z), act'(z), how many roundings of each are felt: the condition of the formula's exponent)."""
    z = np.asarray(z, dtype=np.float64)
    one = np.ones_like(z)
    erfc = np.vectorize(math.erfc, otypes=[float])
    with np.errstate(over="ignore", invalid="ignore"):
        if name == "none":
            return z, one, 0 * one
        if name == "relu":
            return np.where(z < 0, 0.0, z), np.where(np.isnan(z), z, (z > 0).astype(float)), 0 * one
        if name == "silu":
            q = 1 / (1 + np.exp(-z))
            return z * q, q + z * q * (1 / (1 + np.exp(z))), np.abs(z)
        if name == "gelu":
            c = 0.5 * erfc(-z / math.sqrt(2))
            return z * c, c + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi), z * z
        a, b = math.sqrt(2 / math.pi), 0.044715
        u = 2 * a * (z + b * z ** 3)
        q = 1 / (1 + np.exp(-u))
        return z * q, q + z * q * (1 / (1 + np.exp(u))) * 2 * a * (1 + 3 * b * z ** 2), np.abs(u)


def epilogue_ref(v, act="none", bias=None, mul=None, residual=None):
    """(y, z, bound of the rounding errors of y before its own rounding): act(v + bias) * mul + residual.

    z = v + bias is off by one rounding, which reaches act by its derivative.  An activation's own arithmetic is within
    8 roundings of its value (two or three functions of at most two units each, a product, a quotient) and within 4
    for each unit of its exponent; its derivative adds at most two such values.  mul and residual round once each.
    Parts below 2^-125, of z of it and of the derivative, are not held to the value."""
    v = np.asarray(v, dtype=np.float64)
    z = v if bias is None else v + np.asarray(bias, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        a, da, cond = act_ref(act, z)
        err = np.abs(da) * np.abs(z) * EPS32 * (bias is not None) + np.abs(a) * (8 + 4 * cond) * EPS32 * (act != "none")
        y = a
        if mul is not None:
            m = np.asarray(mul, dtype=np.float64)
            y, err = a * m, err * np.abs(m) + np.abs(a * m) * EPS32
        if residual is not None:
            y = y + np.asarray(residual, dtype=np.float64)
            err = err + np.abs(y) * EPS32
        tiny = (np.abs(z) + 1) * 2.0 ** -125 * (1 if mul is None else np.abs(np.asarray(mul, dtype=np.float64)))
    return y, z, err + np.where(np.isfinite(tiny), tiny, 0.0)


def act_grads_ref(act, z, dy, mul=None):
    """(dz, dmul, dbias, bounds of their errors before their own rounding).  The derivative is a sum of at most two
    terms of the size of its parts, |q| + |z q (1 - q) u'|, each within the roundings of act_ref."""
    dy = np.asarray(dy, dtype=np.float64)
    m = np.ones_like(dy) if mul is None else np.asarray(mul, dtype=np.float64)
    z = np.zeros_like(dy) if z is None else np.asarray(z, dtype=np.float64)
    a, da, cond = act_ref(act, z)
    own = act not in ("none", "relu")
    parts = (np.abs(da) + 2 * np.minimum(np.abs(z), 4.0) + 1.0) if own else np.abs(da)
    # the derivative's parts are at most 1 + max |z q (1 - q) u'|, and fall off as the exponent grows
    e_da = parts * (8 + 4 * np.minimum(cond, 64.0)) * EPS32 * own
    dz, dmul = dy * m * da, dy * a
    tiny = (z * z + 2) * 2.0 ** -125
    e_dz = np.abs(dy * m) * (e_da + tiny) + 2 * np.abs(dz) * EPS32
    e_dmul = np.abs(dy * a) * (1 + own * (8 + 4 * cond)) * EPS32 + np.abs(dy) * tiny
    n = dz.shape[0]
    e_dbias = e_dz.sum(0) + n * EPS32 * np.abs(dz).sum(0)
    return dz, dmul, dz.sum(0), (e_dz, e_dmul, e_dbias)
