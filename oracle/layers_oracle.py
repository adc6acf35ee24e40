"""Plain fp64 definitions of the layer norm and the linear layer over
[P][C][N] tensors, with bounds on what an fp32 evaluation may be off by.

Each function returns {name: (value, err)}: `err` bounds the error of an
evaluation that reads the same inputs, forms products exactly or in fp32 and
sums in fp32, before the result is rounded to its stored type.  With u =
2^-24 (half a step of fp32), a sum of terms t_i through at most D additions
per term is off by at most D·u·sum |t_i| to first order; a function of fp32
library quality (erf, exp) by 4u of its magnitude.  `rounding` adds half a
step of the stored type."""
from __future__ import annotations

import math

import numpy as np
import torch

U = 2.0 ** -24


def rounding(value: np.ndarray, err: np.ndarray, stored: str) -> np.ndarray:
    """The bound for a value stored in "f32" or "bf16": half a step of the
    type relative to the computed value, at most |value| + err, and half the
    smallest subnormal step."""
    half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}[stored]
    tiny = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134}[stored]
    return err + half * (np.abs(value) + err) + tiny


def _erf(x):
    return torch.erf(torch.from_numpy(np.ascontiguousarray(x))).numpy()


def _sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1, e) / (1 + e)


def act_value(z: np.ndarray, act: str) -> np.ndarray:
    if act == "relu":
        return np.where(z < 0, 0.0, z)
    if act == "gelu":
        return 0.5 * z * (1 + _erf(z / math.sqrt(2)))
    if act == "silu":
        return z * _sigmoid(z)
    return z.copy()


def act_slope(z: np.ndarray, act: str) -> np.ndarray:
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "gelu":
        return 0.5 * (1 + _erf(z / math.sqrt(2))) + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "silu":
        s = _sigmoid(z)
        return s * (1 + z * (1 - s))
    return np.ones_like(z)


def channel_adds(C: int, N: int) -> int:
    """Roundings per term of a mean over the C channels of a [P][C][N] tensor,
    1/C's own and the product with it (2) among them.
    Rows (N = 1): 16 values in a thread, 5 additions across a warp, 5 across
    the warps: 15 + 5 + 5 + 2 < 32.
    Tiles: up to 16 values in a thread; then, where the tile's lanes divide no
    warp, halvings of up to 1024 rows, 15 + 10 + 2 < 32.  Where they do, 5 at
    most across the warp, and the warps' sums one after another: a thread
    holds 8 channels at 4 batch items of a tile of 64 at most (16 lanes), or
    16 channels at one of 32 lanes at most, so there are C / 16 warps and a
    part of one at most, and no more than 32: 15 + 5 + min(32, C / 16 + 1) + 2."""
    return 32 if N == 1 else max(32, 22 + min(32, C // 16 + 1))


def ln_fwd(x, gamma, beta, eps):
    x = np.asarray(x, np.float64)
    C = x.shape[1]
    g = np.ones(C) if gamma is None else np.asarray(gamma, np.float64)
    b = np.zeros(C) if beta is None else np.asarray(beta, np.float64)
    g, b = g[None, :, None], b[None, :, None]
    mean = x.mean(1, keepdims=True)
    xc = x - mean
    var = (xc * xc).mean(1, keepdims=True)
    rstd = (var + eps) ** -0.5
    y = xc * rstd * g + b
    adds = channel_adds(C, x.shape[2])
    e_mean = adds * U * np.abs(x).mean(1, keepdims=True)
    e_xc = e_mean + U * np.abs(xc)
    # d var: the sum's own error, and 2|xc|·e_xc per term; rstd = (var + eps)^-1/2
    e_var = (adds + 2) * U * var + (2 * np.abs(xc) * e_xc + e_xc * e_xc).mean(1, keepdims=True)
    e_rstd = rstd * (0.5 * e_var / (var + eps) + 4 * U)
    e_y = np.abs(g) * (e_xc * (rstd + e_rstd) + np.abs(xc) * e_rstd) + 3 * U * (np.abs(y) + np.abs(b))
    return {"y": (y, e_y), "mean": (mean[:, 0], e_mean[:, 0]), "rstd": (rstd[:, 0], e_rstd[:, 0])}


def column_adds(units: int) -> int:
    """Additions per term of a parameter gradient, at most.
    Layer norm: 148 blocks or all `units` share the rows or tiles, and one of
    them takes a thread's sum through 4 additions at most (4 batch items);
    then the block's groups and, where no shuffles add them (5), the lanes of
    each in turn, 256 together, since a block that has several groups has 256
    threads; then up to 296 blocks' rows in 32 parts, 10 and 5:
    4·ceil(units / 148) + 256 + 15.
    Activation gradient, up to 8192 channels: a thread adds its positions,
    P·N / 18 at most (1184 blocks or four positions a block; a block has 256
    threads along N, or 8 rows of tokens), then 8 elements, 256 threads, and
    up to 1184 rows and their batch tiles in 32 parts, 37 and 5.
    Both are below the sum here."""
    return 8 * (-(-units // 148) + 1) + 64 + 148 * 32 // 8 + 8


def ln_bwd(gy, x, mean, rstd, gamma):
    gy, x = np.asarray(gy, np.float64), np.asarray(x, np.float64)
    P, C, N = x.shape
    mean, rstd = (np.asarray(t, np.float64).reshape(P, 1, N) for t in (mean, rstd))
    gam = (np.ones(C) if gamma is None else np.asarray(gamma, np.float64))[None, :, None]
    xh = (x - mean) * rstd
    e_xh = 2 * U * np.abs(x - mean) * rstd
    g = gam * gy
    m1, m2 = g.mean(1, keepdims=True), (g * xh).mean(1, keepdims=True)
    a1, a2 = np.abs(g).mean(1, keepdims=True), np.abs(g * xh).mean(1, keepdims=True)
    gx = rstd * (g - m1 - xh * m2)
    adds = channel_adds(C, N)
    e1 = (adds + 2) * U * a1
    e2 = (adds + 4) * U * a2
    e_gx = rstd * (e1 + np.abs(xh) * e2 + e_xh * (np.abs(m2) + e2)
                   + 4 * U * (np.abs(g) + np.abs(m1) + np.abs(xh * m2))) + 2 * U * np.abs(gx)
    D = column_adds(P * N)
    return {"gx": (gx, e_gx),
            "ggamma": ((gy * xh).sum((0, 2)), (D + 4) * U * np.abs(gy * xh).sum((0, 2))),
            "gbeta": (gy.sum((0, 2)), D * U * np.abs(gy).sum((0, 2)))}


def _product_err(K: int, S: np.ndarray) -> np.ndarray:
    """A sum of K exact products: K additions, each off by at most a whole
    step (2u, in case the sum truncates) of the running sum, at most S."""
    return 2 * U * (K + 1) * S


def lin_fwd(w, x, bias, residual, act):
    w, x = np.asarray(w, np.float64), np.asarray(x, np.float64)
    z = np.einsum("oi,pin->pon", w, x, optimize=True)
    S = np.einsum("oi,pin->pon", np.abs(w), np.abs(x), optimize=True)
    e_z = _product_err(w.shape[1], S)
    if bias is not None:
        z = z + np.asarray(bias, np.float64)[None, :, None]
        e_z = e_z + U * (np.abs(z) + e_z)
    y = act_value(z, act)
    if act == "none":
        e_y = e_z
    else:
        # |act'| <= 1.13; erf and exp are off by 4u of at most 1, times |z|
        e_y = 1.13 * e_z + 12 * U * (np.abs(z) + e_z)
    if residual is not None:
        y = y + np.asarray(residual, np.float64)
        e_y = e_y + U * (np.abs(y) + e_y)
    return {"y": (y, e_y), "z": (z, e_z)}


def lin_act_grad(gy, z, act):
    gy = np.asarray(gy, np.float64)
    P, _, N = gy.shape
    if act == "none":
        slope, e_s = np.ones_like(gy), np.zeros_like(gy)
    else:
        z = np.asarray(z, np.float64)
        slope = act_slope(z, act)
        # relu's slope is exact; the others are sums of terms of magnitude at
        # most 1.5, each through at most 12 roundings, and |z|·exp(-z^2/2)
        # carries z^2/2 roundings of the exponent into a term below 1
        e_s = np.zeros_like(gy) if act == "relu" else np.full_like(gy, 16 * U)
    # relu selects: an infinite gy where it is off is dropped
    gz = np.where(slope > 0, gy, 0.0) if act == "relu" else gy * slope
    e_gz = np.abs(gy) * e_s + U * np.abs(gz)
    return {"gz": (gz, e_gz),
            "gbias": (gz.sum((0, 2)), (column_adds(P * N) * U * np.abs(gz) + e_gz).sum((0, 2)))}


def lin_dgrad(w, gz):
    w, gz = np.asarray(w, np.float64), np.asarray(gz, np.float64)
    gx = np.einsum("oi,pon->pin", w, gz, optimize=True)
    S = np.einsum("oi,pon->pin", np.abs(w), np.abs(gz), optimize=True)
    return {"gx": (gx, _product_err(w.shape[0], S))}


def lin_wgrad(gz, x):
    gz, x = np.asarray(gz, np.float64), np.asarray(x, np.float64)
    gw = np.einsum("pon,pin->oi", gz, x, optimize=True)
    S = np.einsum("pon,pin->oi", np.abs(gz), np.abs(x), optimize=True)
    return {"gw": (gw, _product_err(x.shape[0] * x.shape[2], S))}
