"""Plain fp64 forms of the standalone operators (test infrastructure only): what include/flint_ops.h
states, written from the formulas with numpy, no rounding but the caller's own."""

import numpy as np

from . import flint_moe_ref as R


def q4_weight(fmt, codes, scales, tscale=None):
    """fp64 [N][K] of the stored matrix (rotated storage stays rotated). codes u8 [N][K/2]; scales: bf16 bits
    (uint16) for int4, E4M3 bytes (uint8) for nvfp4."""
    if fmt == "int4":
        return R.dequant_int4(codes, scales, tscale)
    return R.dequant_nvfp4(codes, scales, 1.0 if tscale is None else tscale)


def q4_linear(x, fmt, codes, scales, tscale=None, rotated=False):
    x = np.asarray(x, dtype=np.float64)
    return (R.rotate_segments(x) if rotated else x) @ q4_weight(fmt, codes, scales, tscale).T


def group_rows(offsets, P):
    """Group of every row, -1 for rows of none; offsets clamped to [0, P]."""
    off = np.clip(np.asarray(offsets, dtype=np.int64), 0, P)
    g = np.full(P, -1)
    for e in range(len(off) - 1):
        if off[e + 1] > off[e]:
            g[off[e]:off[e + 1]] = e
    return g


def grouped_linear(x, w, offsets, rows=None, row_div=1, swiglu=False):
    """(y [P][N_out], mask [P] of the rows that belong to a group)."""
    x, w = np.asarray(x, dtype=np.float64), np.asarray(w, dtype=np.float64)
    P = x.shape[0] if rows is None else len(rows)
    g = group_rows(offsets, P)
    src = np.arange(P) if rows is None else np.clip(np.asarray(rows) // row_div, 0, x.shape[0] - 1)
    n_out = w.shape[1] // 2 if swiglu else w.shape[1]
    y = np.zeros((P, n_out))
    for e in np.unique(g[g >= 0]):
        p = np.nonzero(g == e)[0]
        v = x[src[p]] @ w[e].T
        y[p] = R.silu(v[:, :n_out]) * v[:, n_out:] if swiglu else v
    return y, g >= 0


def expert_permute(ids, E):
    """(offsets [E+1], perm [P], inv [T][top_k]); ids outside [0, E) dropped."""
    flat = np.asarray(ids).reshape(-1)
    perm = np.full(flat.size, -1, dtype=np.int32)
    inv = np.full(flat.size, -1, dtype=np.int32)
    offsets = np.zeros(E + 1, dtype=np.int32)
    n = 0
    for e in range(E):
        for i in np.nonzero(flat == e)[0]:
            perm[n], inv[i] = i, n
            n += 1
        offsets[e + 1] = n
    return offsets, perm, inv.reshape(np.asarray(ids).shape)


def expert_combine(o, inv, w, addend=None, scale=1.0):
    o, w = np.asarray(o, dtype=np.float64), np.asarray(w, dtype=np.float64)
    y = np.zeros((inv.shape[0], o.shape[1]))
    for t in range(inv.shape[0]):
        for k in range(inv.shape[1]):
            if 0 <= inv[t, k] < o.shape[0]:
                y[t] += w[t, k] * o[inv[t, k]]
    return scale * y + (0.0 if addend is None else np.asarray(addend, dtype=np.float64))


def block_norm(x, y=None, *, post_norm=False, post_weight=None, gate=None, sigmoid=False, res_scale=1.0,
               branch_scale=1.0, pre_weight=None, eps=1e-6):
    x = np.asarray(x, dtype=np.float64) * res_scale
    if y is not None:
        b = np.asarray(y, dtype=np.float64)
        if post_norm:
            b = b / np.sqrt((b * b).mean(1, keepdims=True) + eps) * (1.0 if post_weight is None else post_weight)
        if gate is not None:
            g = np.asarray(gate, dtype=np.float64)
            b = b * (1.0 / (1.0 + np.exp(-g)) if sigmoid else g)
        x = x + branch_scale * b
    z = x / np.sqrt((x * x).mean(1, keepdims=True) + eps) * (1.0 if pre_weight is None else pre_weight)
    return x, z
