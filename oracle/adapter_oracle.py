"""Plain float64 restatement of the adapter operators, the 8-bit checkpoints and the packed layer's input
gradient, each with a bound on what float32 sums and the stated roundings may cost.

Rounding facts used by the bounds (relative to the value rounded):

* to bfloat16: 2^-8;  to float32: 2^-24
* a float32 value as the sum of two bfloat16 values (rounded value and rounded rest): 2^-16
* a float32 sum on the tensor cores or in lanes: every accumulation step off by at most one unit of the
  partial sum, 2^-23; a sum of n products takes at most n / 16 + 16 steps one after the other.  With
  partial sums bounded by the sum of magnitudes S, the error is at most (n / 16 + 16) 2^-23 S.
"""

from __future__ import annotations

from typing import Optional, Tuple

import numpy as np

from .convrot_oracle import regular_hadamard, unpack_int4

BF16 = 2.0 ** -8
PAIR = 2.0 ** -16


def steps(n: int) -> float:
    return (n / 16 + 16) * 2.0 ** -23


def row_masks(adapter: Optional[np.ndarray], M: int, L: int):
    """(adapter, boolean rows) for every adapter of the pool."""
    for a in range(L):
        yield a, (np.ones(M, bool) if adapter is None else np.asarray(adapter) == a)


def rotate64(y: np.ndarray, group: int = 256) -> np.ndarray:
    h = np.asarray(regular_hadamard(group), np.float64)
    return (y.reshape(y.shape[0], -1, group) @ h).reshape(y.shape)


def lora_forward(x, down, up, scale, adapter=None, base=None) -> Tuple[np.ndarray, ...]:
    """(Y, V, bound on Y, bound on the bfloat16 V), all float64."""
    L, r, K = down.shape
    N, M = up.shape[2], x.shape[0]
    y = np.zeros((M, N)) if base is None else np.array(base, np.float64)
    v, ev, ey = np.zeros((M, r)), np.zeros((M, r)), np.zeros((M, N))
    for a, rows in row_masks(adapter, M, L):
        if not rows.any():
            continue
        xs, s = x[rows], float(scale[a])
        v[rows] = xs @ down[a].T
        ev[rows] = steps(K) * (np.abs(xs) @ np.abs(down[a]).T)
        y[rows] += s * (v[rows] @ up[a])
        # V from float32 sums, times the scale (rounded), as a bfloat16 pair, and the sum over the rank
        per = ev[rows] + (PAIR + 2.0 ** -23 + steps(2 * r)) * np.abs(v[rows])
        ey[rows] = abs(s) * (per @ np.abs(up[a]))
    return y, v, ey * (1 + BF16) + (BF16 + 2.0 ** -23) * np.abs(y), ev * (1 + BF16) + BF16 * np.abs(v)


def lora_backward(dy, x, v, down, up, scale, adapter=None, base=None, x_abs=None):
    """(dX, d_down, d_up) and their bounds.  ``x_abs``: magnitudes entering the sums over rows (those of
    the rotated codes for a checkpoint, whose product is taken in the rotated basis)."""
    L, r, K = down.shape
    M, N = dy.shape
    x_abs = np.abs(x) if x_abs is None else x_abs
    dx = np.zeros((M, K)) if base is None else np.array(base, np.float64)
    ex = np.zeros((M, K))
    dd, ed = np.zeros((L, r, K)), np.zeros((L, r, K))
    du, eu = np.zeros((L, r, N)), np.zeros((L, r, N))
    for a, rows in row_masks(adapter, M, L):
        if not rows.any():
            continue
        s, dys, n = float(scale[a]), dy[rows], int(rows.sum())
        dv = s * (dys @ up[a].T)
        ev = abs(s) * steps(N) * (np.abs(dys) @ np.abs(up[a]).T) + 2.0 ** -23 * np.abs(dv)
        per = ev + (PAIR + 2.0 ** -23) * np.abs(dv)
        dx[rows] += dv @ down[a]
        ex[rows] = (per + steps(2 * r) * np.abs(dv)) @ np.abs(down[a])
        dd[a] = dv.T @ x[rows]
        # a further 16 float32 steps: partial sums joined, the rotation of the result
        ed[a] = (per + (steps(2 * M) + 2.0 ** -19) * np.abs(dv)).T @ x_abs[rows]
        du[a] = s * (v[rows].T @ dys)
        eu[a] = abs(s) * (PAIR + steps(2 * M) + 2.0 ** -19) * (np.abs(v[rows]).T @ np.abs(dys))
    fin = lambda t, e: e * (1 + BF16) + (BF16 + 2.0 ** -23) * np.abs(t)  # noqa: E731
    return (dx, dd, du), (fin(dx, ex), fin(dd, ed), fin(du, eu))


def ckpt_save(x):
    """(codes, float32 scales, y / s before rounding) of finite rows."""
    M, K = x.shape
    y = rotate64(np.asarray(x, np.float64)).reshape(M, K // 256, 256)
    s = np.maximum((np.abs(y).max(-1) / 127), 2.0 ** -100).astype(np.float32)
    t = y / s.astype(np.float64)[..., None]
    return np.rint(t).astype(np.int8).reshape(M, K), s, t.reshape(M, K)


def ckpt_values(codes, scales):
    """(x^, magnitudes that entered its sums): codes times scales, rotated back."""
    M, K = codes.shape
    c = (codes.astype(np.float64).reshape(M, -1, 256) * scales.astype(np.float64)[..., None]).reshape(M, K)
    mags = np.repeat(np.abs(c).reshape(M, -1, 256).sum(-1) / 16, 256, axis=1).reshape(M, K)
    return rotate64(c), mags


def grad_input(dy, wq_packed, w_scale, group: int = 256):
    """(dX, bound): one operand of each product rounded to bfloat16 once, float32 sums, one rounding.

    Either the weight is rounded, or w_scale[n] dY[m, n], whose relative error all columns k share, so that the
    rotation of the sums carries it to |dY[m, n]| |W^[n, k]|, too.  The float32 sums are taken of the weights, or
    of the codes and rotated then (at most 16 roundings one after the other): errors of theirs spread over the
    group by the rotation's magnitudes, which are at least those of the weights.
    """
    q = unpack_int4(wq_packed).astype(np.float64)
    s = np.asarray(w_scale, np.float64)
    w = rotate64(q, group) * s[:, None]
    dx = dy @ w
    mags = np.abs(dy) @ np.abs(w)
    p = np.abs(dy) @ (np.abs(q) * s[:, None])
    h = np.abs(np.asarray(regular_hadamard(group), np.float64))
    spread = (p.reshape(p.shape[0], -1, group) @ h).reshape(p.shape)
    e = (BF16 + 2.0 ** -22) * mags + (steps(dy.shape[1]) + 2.0 ** -20) * spread
    return dx, e * (1 + BF16) + BF16 * np.abs(dx)
