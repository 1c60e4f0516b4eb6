"""Reference of the transformer-layer operators in float64 (numpy), with error bounds.

Product with an epilogue: Z = row_scale·col_scale·(A·B) + bias, D = act(Z) + residual, and its
gradients; RMS norm and layer norm with the residual's addition, 8-bit results with row or block
scales, and their gradients; quantised rows.  Inputs are float64 arrays holding the values the device buffers stand for.
"""

import math

import numpy as np

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24, "e4m3": 2.0 ** -4, "e5m2": 2.0 ** -3}
# half the spacing of the smallest numbers: what rounding costs however small the value is
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150, "e4m3": 2.0 ** -10, "e5m2": 2.0 ** -17}
QMAX = {"e4m3": 448.0, "e5m2": 57344.0, "i8": 127.0}
AMAX_FLOOR = 2.0 ** -100
U32 = 2.0 ** -24

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _phi(z):
    return 0.5 * _erfc(z * -math.sqrt(0.5)) if np.size(z) else np.asarray(z, np.float64)


def _sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def act(z, kind):
    if kind == "relu":
        return np.where(z > 0, z, np.where(np.isnan(z), z, 0.0))
    if kind == "gelu":
        return z * _phi(z)
    if kind == "gelu_tanh":
        return z * _sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if kind == "silu":
        return z * _sigmoid(z)
    return np.array(z, np.float64)


def act_grad(z, kind):
    if kind == "relu":
        return np.where(z > 0, 1.0, 0.0)
    if kind == "gelu":
        return _phi(z) + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        zc = np.clip(z, -100, 100)
        s = _sigmoid(2 * c * (zc + 0.044715 * zc ** 3))
        return s + zc * s * (1 - s) * 2 * c * (1 + 3 * 0.044715 * zc ** 2)
    if kind == "silu":
        zc = np.clip(z, -700, 700)
        s = _sigmoid(zc)
        return s * (1 + zc * (1 - s))
    return np.ones_like(z)


def product_bound(A, B, eight):
    """Error of the sum over K: fp32 accumulation of K products in any order is within K·2^-23 of
    the sum of magnitudes; fp8 operands are summed in groups of 8 whose members lose at most 2^-13 of
    the group's largest product each, 8·2^-13 of the sum of magnitudes at most."""
    K = A.shape[1]
    mag = np.abs(A) @ np.abs(B)
    return ((K + 8) * 2 * U32 + (2.0 ** -10 if eight else 0.0)) * mag


def product(A, B, kind="none", bias=None, residual=None, row_scale=None, col_scale=None, out="bf16",
            eight=False, ints=False):
    """(D, Z, bound of D, bound of Z) for A [M][K], B [K][N].  ints: operands of 8-bit integers, whose sums
    are exact and rounded to fp32 once."""
    P = A @ B
    err = U32 * np.abs(P) if ints else product_bound(A, B, eight)
    scale = np.ones((A.shape[0], B.shape[1]))
    if row_scale is not None:
        scale = scale * row_scale[:, None]
    if col_scale is not None:
        scale = scale * col_scale[None, :]
    Z = P * scale
    err = err * np.abs(scale) + 3 * U32 * np.abs(Z)
    if bias is not None:
        Z = Z + bias[None, :]
        err = err + U32 * (np.abs(Z) + err)
    D = act(Z, kind)
    # the activations' slope is at most 1.13; their fp32 evaluation is good to 16 units of |z|
    # (exp of an argument of magnitude up to ~90 carries its rounding as a relative error, where the
    # result is then tiny: counted as 2^-20 of the result)
    derr = err if kind == "none" else 1.13 * err + 16 * U32 * np.abs(Z) + 2.0 ** -20 * np.abs(D)
    if residual is not None:
        D = D + residual
        derr = derr + U32 * (np.abs(D) + derr)
    h, t = HALF_STEP[out], TINY[out]
    return D, Z, derr * (1 + h) + h * np.abs(D) + t, err * (1 + h) + h * np.abs(Z) + t


def act_backward(dY, Z, kind, out):
    """(dZ, its bound, dbias, its bound): dbias sums dZ before the rounding, in fp32."""
    g = act_grad(Z, kind)
    dZ = dY * g
    err = np.abs(dY) * ((0.0 if kind == "none" else 32 * U32 * (1 + np.abs(Z)) * (np.abs(g) + 2.0 ** -20)) + U32)
    M = dY.shape[0]
    s = dZ.sum(axis=0)
    serr = err.sum(axis=0) + (M + 8) * 2 * U32 * np.abs(dZ).sum(axis=0) + 2.0 ** -140
    h = HALF_STEP[out]
    return dZ, err * (1 + h) + h * np.abs(dZ) + TINY[out], s, serr


def matmul_bound(A, B, out):
    """(A·B, bound) of a plain product of the given operands rounded to `out`."""
    P = A @ B
    err = product_bound(A, B, False)
    h = HALF_STEP[out]
    return P, err * (1 + h) + h * np.abs(P) + TINY[out]


def norm(H, w, eps):
    """(Y, rstd) of the rows of H."""
    rstd = 1.0 / np.sqrt(np.mean(H * H, axis=1) + eps)
    return H * rstd[:, None] * w[None, :], rstd


def norm_rel(cols):
    """Relative error of rstd in fp32: half that of the mean of squares (cols additions of positive
    numbers) plus the division and the root."""
    return (0.5 * (cols + 8) * 2 + 6) * U32


def row_scale(Y, fmt):
    return np.maximum(np.abs(Y).max(axis=1), AMAX_FLOOR) / QMAX[fmt]


def block_scale(Y, fmt):
    """Exponents e with 2^e the smallest power of two that brings each 32 columns' maximum to qmax."""
    top = np.maximum(np.abs(Y).reshape(Y.shape[0], -1, 32).max(axis=2), AMAX_FLOOR)
    return np.ceil(np.log2(top / QMAX[fmt])).astype(np.int64)


def norm_backward(dY, H, w, rstd, dH, out):
    """(dX, bound, dw, bound)."""
    cols = H.shape[1]
    xh = H * rstd[:, None]
    g = dY * w[None, :]
    c = np.mean(g * xh, axis=1)
    dX = rstd[:, None] * (g - xh * c[:, None])
    cerr = (cols + 8) * 2 * U32 * np.mean(np.abs(g * xh), axis=1)
    err = np.abs(rstd[:, None]) * (6 * U32 * (np.abs(g) + np.abs(xh * c[:, None])) + np.abs(xh) * cerr[:, None])
    if dH is not None:
        dX = dX + dH
        err = err + U32 * np.abs(dX)
    h = HALF_STEP[out]
    dw = (dY * xh).sum(axis=0)
    dwerr = (H.shape[0] + 8) * 2 * U32 * np.abs(dY * xh).sum(axis=0) + 2.0 ** -140
    return dX, err * (1 + h) + h * np.abs(dX) + TINY[out], dw, dwerr


def layer_norm(H, w, b, eps):
    """(Y, mean, rstd, bound of Y, bound of mean, relative bound of rstd) of the rows of H, in fp32.

    The mean carries its sum's rounding: e = (cols+8)·2^-23 of the mean magnitude at most.  The deviations
    carry e and their own rounding; their mean square, to first order, 2·(rounding) relative, the additions'
    (cols+8)·2^-23 and e² (a shift of the centre adds its square), rstd half of it all and a root's and a
    division's rounding."""
    cols = H.shape[1]
    mean = H.mean(axis=1)
    d = H - mean[:, None]
    var = np.mean(d * d, axis=1)
    rstd = 1.0 / np.sqrt(var + eps)
    merr = (cols + 8) * 2 * U32 * np.mean(np.abs(H), axis=1) + U32 * np.abs(mean)
    # rounding of a deviation is relative to it; its root mean square bounds the mean's effect
    rel = 0.5 * ((cols + 8) * 2 * U32 + 4 * U32) + 0.5 * (merr * rstd) ** 2 + U32 * merr * rstd + 6 * U32
    xh = d * rstd[:, None]
    Y = xh * w[None, :]
    err = (merr * rstd)[:, None] * np.abs(w)[None, :] + (rel[:, None] + 4 * U32) * np.abs(Y)
    if b is not None:
        Y = Y + b[None, :]
        err = err + U32 * (np.abs(Y) + err)
    return Y, mean, rstd, err, merr, rel


def layer_norm_backward(dY, H, w, mean, rstd, dH, out):
    """(dX, bound, dw, bound, db, bound)."""
    cols = H.shape[1]
    d = H - mean[:, None]
    xh = d * rstd[:, None]
    xerr = 3 * U32 * np.abs(xh)
    g = dY * w[None, :]
    gm, c = np.mean(g, axis=1), np.mean(g * xh, axis=1)
    s = (cols + 8) * 2 * U32
    gmerr = s * np.mean(np.abs(g), axis=1)
    cerr = (s + 4 * U32) * np.mean(np.abs(g * xh), axis=1)
    dX = rstd[:, None] * (g - gm[:, None] - xh * c[:, None])
    err = np.abs(rstd[:, None]) * (6 * U32 * (np.abs(g) + np.abs(gm[:, None]) + np.abs(xh * c[:, None])) + gmerr[:, None]
                                   + np.abs(xh) * cerr[:, None] + xerr * np.abs(c[:, None]))
    if dH is not None:
        dX = dX + dH
        err = err + U32 * (np.abs(dX) + err)
    h = HALF_STEP[out]
    rows = (H.shape[0] + 8) * 2 * U32
    dw, db = (dY * xh).sum(axis=0), dY.sum(axis=0)
    return (dX, err * (1 + h) + h * np.abs(dX) + TINY[out], dw, (rows + 4 * U32) * np.abs(dY * xh).sum(axis=0) + 2.0 ** -140,
            db, rows * np.abs(dY).sum(axis=0) + 2.0 ** -140)


def quantised_rows(X, fmt):
    """(codes before their rounding, scales): the scale is an fp32 quotient, for integers the fp32 product
    with the fp32 value of 1/127, and the codes are X by it."""
    top = np.maximum(np.abs(X).max(axis=1), AMAX_FLOOR).astype(np.float32)
    s = (top * (np.float32(1) / np.float32(127)) if fmt == "i8" else top / np.float32(QMAX[fmt])).astype(np.float64)
    return X / s[:, None], s


def gated(A, B, kind="silu", bias=None, row_scale=None, col_scale=None, out="bf16", eight=False, ints=False):
    """(D, Z, bound of D, bound of Z) for A [M][K], B [K][2N]: Z = [G | U] = scales·A·B + bias, D = act(G)·U."""
    N = B.shape[1] // 2
    P = A @ B
    scale = np.ones(P.shape)
    if row_scale is not None:
        scale = scale * row_scale[:, None]
    if col_scale is not None:
        scale = scale * col_scale[None, :]
    Z = P * scale
    err = (U32 * np.abs(P) if ints else product_bound(A, B, eight)) * np.abs(scale) + 3 * U32 * np.abs(Z)
    if bias is not None:
        Z = Z + bias[None, :]
        err = err + U32 * (np.abs(Z) + err)
    G, U, ge, ue = Z[:, :N], Z[:, N:], err[:, :N], err[:, N:]
    a = act(G, kind)
    # the activation's error as in product()
    ae = ge if kind == "none" else 1.13 * ge + 16 * U32 * np.abs(G) + 2.0 ** -20 * np.abs(a)
    D = a * U
    derr = ae * np.abs(U) + np.abs(a) * ue + ae * ue + U32 * np.abs(D)
    h, t = HALF_STEP[out], TINY[out]
    return D, Z, derr * (1 + h) + h * np.abs(D) + t, err * (1 + h) + h * np.abs(Z) + t


def act_grad_size(z, kind):
    """What the fp32 evaluation of act_grad is accurate relative to.  The derivative is a sum of two terms,
    gelu: Phi + z·phi, gelu_tanh and silu: s + (a multiple of) z·s·(1 - s), which cancel where it crosses zero
    (z = -0.7518, -0.7524, -1.2785): each term is good to some units of fp32 relative to itself, so the sum is to
    as many units of the terms' magnitudes, here |Phi| + |z·phi| and so on, however small it is."""
    if kind == "gelu":
        return _phi(z) + np.abs(z) * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if kind in ("gelu_tanh", "silu"):
        zc = np.clip(z, -100, 100) if kind == "gelu_tanh" else np.clip(z, -700, 700)
        c = 2 * math.sqrt(2 / math.pi) if kind == "gelu_tanh" else 1.0
        q = 0.044715 if kind == "gelu_tanh" else 0.0
        s = _sigmoid(c * (zc + q * zc ** 3))
        return s + np.abs(zc) * s * (1 - s) * c * (1 + 3 * q * zc ** 2)
    return np.abs(act_grad(z, kind))


def gated_backward(dY, Z, kind, out, row_scale=None, col_scale=None):
    """(dZ, its bound, dbias, its bound) of D = act(G)·U: dbias sums before the scales and the rounding, in fp32."""
    M, N = dY.shape
    G, U = Z[:, :N], Z[:, N:]
    g, a = act_grad(G, kind), act(G, kind)
    exact = 0.0 if kind == "none" else 1.0
    dG, dU = dY * U * g, dY * a
    ge = np.abs(dY * U) * (exact * 32 * U32 * (1 + np.abs(G)) * (act_grad_size(G, kind) + 2.0 ** -20) + 2 * U32 * np.abs(g))
    ue = np.abs(dY) * (exact * (16 * U32 * np.abs(G) + 2.0 ** -20 * np.abs(a)) + U32 * np.abs(a))
    d, err = np.concatenate([dG, dU], axis=1), np.concatenate([ge, ue], axis=1)
    s = d.sum(axis=0)
    serr = err.sum(axis=0) + (M + 8) * 2 * U32 * np.abs(d).sum(axis=0) + 2.0 ** -140
    if row_scale is not None or col_scale is not None:
        scale = np.ones_like(d)
        if row_scale is not None:
            scale = scale * row_scale[:, None]
        if col_scale is not None:
            scale = scale * col_scale[None, :]
        d, err = d * scale, err * np.abs(scale) + 3 * U32 * np.abs(d * scale)
    h = HALF_STEP[out]
    return d, err * (1 + h) + h * np.abs(d) + TINY[out], s, serr
