"""fp64 definitions of the operators around the attention (numpy; test infrastructure only).

Written from the formulas alone; shares no code with the package.  Every function returns the
value and, where a kernel works in fp32, a bound on what fp32 sums and products may add to it
(the caller adds the rounding to the output's type).
"""
import math

import numpy as np

U32 = 2.0 ** -24          # half a unit in the last place of fp32, relative


def angles(pos, dims, thetas):
    """[N][R/2] angles of positions [N][axes]."""
    cols = []
    for a, d in enumerate(dims):
        f = np.array([float(thetas[a]) ** (-2.0 * i / d) for i in range(d // 2)])
        cols.append(np.outer(np.asarray(pos, np.float64)[:, a], f))
    return np.concatenate(cols, axis=1)


def rms_norm(x, weight, eps):
    """x [..., D] times weight (broadcast) over its root mean square."""
    r = 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    return x * r * weight


def rotate(x, cs, halves):
    """x [..., N, D] with its first R columns turned by cs [..., N, R/2, 2] (cos, sin)."""
    P = cs.shape[-2]
    j = np.arange(P)
    ia, ib = (j, j + P) if halves else (2 * j, 2 * j + 1)
    c, s = cs[..., 0], cs[..., 1]
    out = x.copy()
    out[..., ia] = x[..., ia] * c - x[..., ib] * s
    out[..., ib] = x[..., ia] * s + x[..., ib] * c
    return out


def pair_sum(x, P, halves):
    """|x| with the two columns of every rotated pair replaced by the sum of both: what bounds
    each of them after a rotation."""
    x = np.abs(x)
    out = x.copy()
    j = np.arange(P)
    ia, ib = (j, j + P) if halves else (2 * j, 2 * j + 1)
    out[..., ia] = out[..., ib] = x[..., ia] + x[..., ib]
    return out


def norm_rope(x, weight, eps, norm, cs, halves, x_err=None):
    """Value and fp32 bound of the norm (norm=True) and the rotation (cs not None).

    x_err: bound on the error x itself carries (a projection's accumulators)."""
    x_err = np.zeros_like(x) if x_err is None else x_err
    D = x.shape[-1]
    if norm:
        r = 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
        u = x * r * weight
        # the sum of squares is D fp32 terms (its relative error halves under the root); an
        # error of x moves the root by at most |x_err|_2 / |x|_2, relative
        nx = np.sqrt((x * x).sum(axis=-1, keepdims=True)) + 1e-300
        ne = np.sqrt((x_err * x_err).sum(axis=-1, keepdims=True))
        bound = np.abs(r * weight) * (x_err + np.abs(x) * np.minimum(1.0, ne / nx))
        bound += (D / 2 + 4) * U32 * np.abs(u)
    else:
        u, bound = x, x_err
    if cs is not None:
        P = cs.shape[-2]
        # two products and a sum, each rounded once
        bound = pair_sum(bound, P, halves) + 3 * U32 * pair_sum(u, P, halves)
        u = rotate(u, cs, halves)
    return u, bound


def _gelu(v):
    return 0.5 * v * (1.0 + np.vectorize(math.erf)(v / math.sqrt(2.0)))


def _gelu_tanh(v):
    return 0.5 * v * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))


def _silu(v):
    return v / (1.0 + np.exp(-v))


ACTS = {"none": lambda v: v, "gelu": _gelu, "gelu_tanh": _gelu_tanh, "silu": _silu}


def activation(v, act):
    """Value of an activation in a form that keeps its relative accuracy far below zero, and the
    relative error of an fp32 evaluation of it that does the same (its scale is |act(v)|).

    Counted in units of 2^-24: two dozen for exponential, reciprocal and the products around them
    (and a polynomial of ten terms, erf form).  Below zero the result is proportional to exp(-y),
    and each rounding of y is worth |y| units of it (silu: y = |v|, tanh form: y = 2|u|, erf form:
    y = v^2/2); y beyond 100 is left out, where exp(-y) is no normal fp32 number.  Above zero
    the exponential is added to 1, and y exp(-y) < 0.4."""
    with np.errstate(over="ignore", invalid="ignore"):
        if act == "silu":
            y, value, per_y, units = v, v / (1.0 + np.exp(-v)), 2, 24
        elif act == "gelu_tanh":
            y = 2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)
            value, per_y, units = v / (1.0 + np.exp(-y)), 6, 24
        else:
            y, per_y, units = v * v / 2.0, 4, 48
            value = 0.5 * v * np.vectorize(math.erfc)(-v / math.sqrt(2.0))
        return value, U32 * (units + per_y * np.where(v < 0, np.minimum(np.abs(y), 100.0), 1.0))


def product(x, w, bias):
    """x [M][K] w [C][K]^T + bias and its fp32 bound: K products summed in any order, with the
    truncating adds of a tensor core (one unit, not half, per add)."""
    v = x @ w.T + (0.0 if bias is None else bias)
    K = x.shape[1]
    return v, 2 * K * U32 * (np.abs(x) @ np.abs(w).T) + 2 * U32 * np.abs(v)


def linear(x, w, bias=None, act="none", gate=None, residual=None):
    """Value and fp32 bound of residual + gate * act(x w^T + bias); gate broadcast to rows."""
    v, bound = product(x, w, bias)
    y = ACTS[act](v)
    if act != "none":
        # |act'| <= 1.13; the activation itself: exp, erf and a division of a few units each
        # (u of the tanh form grows with |v|, its exponential with |u| units)
        bound = 1.13 * bound + U32 * np.abs(v) * (16 + 4 * np.minimum(np.abs(v), 30.0))
    if gate is not None:
        y, bound = y * gate, np.abs(gate) * bound + U32 * np.abs(y * gate)
    if residual is not None:
        y = y + residual
        bound = bound + U32 * np.abs(y)
    return y, bound
