"""fp64 references of the low-rank adapter operators (test infrastructure; numpy
only, nothing here reads the GPU library).

Token t with adapter a = ids[t] >= 0 adds scale[a] * B_a (A_a x_t) to its row;
tokens with a negative id add nothing.  An id >= n is an error the operators
answer with a NaN row."""
from __future__ import annotations

import numpy as np


def _f64(*arrays):
    return [np.asarray(v, dtype=np.float64) for v in arrays]


def lora_linear_ref(a, b, scale, x, ids, base=None):
    """y [T][d_out]."""
    a, b, scale, x = _f64(a, b, scale, x)
    y = np.zeros((x.shape[0], b.shape[1])) if base is None else np.array(base, dtype=np.float64)
    for t, i in enumerate(np.asarray(ids)):
        if i >= a.shape[0]:
            y[t] = np.nan
        elif i >= 0:
            y[t] += scale[i] * (b[i] @ (a[i] @ x[t]))
    return y


def lora_grads_ref(a, b, scale, x, g, ids, dx_base=None):
    """(dx [T][d_in], da [n][r][d_in], db [n][d_out][r]) of the loss whose gradient at y is g."""
    a, b, scale, x, g = _f64(a, b, scale, x, g)
    dx = np.zeros_like(x) if dx_base is None else np.array(dx_base, dtype=np.float64)
    da, db = np.zeros_like(a), np.zeros_like(b)
    for t, i in enumerate(np.asarray(ids)):
        if i >= a.shape[0]:
            dx[t] = np.nan
        elif i >= 0:
            dh = scale[i] * (b[i].T @ g[t])
            dx[t] += a[i].T @ dh
            da[i] += np.outer(dh, x[t])
            db[i] += scale[i] * np.outer(g[t], a[i] @ x[t])
    return dx, da, db


def lora_abs(a, b, scale, x, ids, base=None):
    """The same sums with every term's absolute value: what rounding errors of y are relative to."""
    return lora_linear_ref(np.abs(a), np.abs(b), np.abs(scale), np.abs(x), ids,
                           None if base is None else np.abs(base))


def lora_grads_abs(a, b, scale, x, g, ids, dx_base=None):
    return lora_grads_ref(np.abs(a), np.abs(b), np.abs(scale), np.abs(x), np.abs(g), ids,
                          None if dx_base is None else np.abs(dx_base))


def orthogonalize_ref(x, steps, coeffs):
    """`steps` times X <- a X + (b G + c G^2) X, G = X X^T, from X / ||X||_F; a zero matrix stays zero."""
    x = np.asarray(x, dtype=np.float64)
    norm = np.linalg.norm(x)
    x = x / norm if norm != 0 else x
    a, b, c = coeffs
    for _ in range(steps):
        if x.shape[0] <= x.shape[1]:
            g = x @ x.T
            x = a * x + b * (g @ x) + c * (g @ (g @ x))
        else:  # the same polynomial from the other side
            g = x.T @ x
            x = a * x + b * (x @ g) + c * ((x @ g) @ g)
    return x
