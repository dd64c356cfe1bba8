"""Plain CPU oracle for the norms around a block, forward and backward.

TEST INFRASTRUCTURE ONLY.  Nothing in the product path may import, call or execute
this module; it shares no code with the HIP path.

    N(v; g)  = g v / sqrt(mean(v^2) + eps)
    n[t]     = N(y[t]; post_gain), or y[t]
    out[t]   = rs x[t] + bs a(gate[t // gate_rows]) n[t]
    h[t]     = N(out[t]; next_gain)

and, given the gradients of out and h, the chain rule in reverse.  The Jacobian of
v / q with q = sqrt(mean(v^2) + eps) is (1 - v v^T / (d q^2)) / q.  Every step runs in
float64 with numpy.

Each function also returns the size of what it adds up: the same sums with every
term's magnitude.  A float32 evaluation whose terms are each off by a relative e is off
by at most e times that size, which is what the GPU tests bound their errors with.
"""
from __future__ import annotations

import numpy as np


def act(z, kind):
    """(a(z), a'(z))"""
    if kind == "sigmoid":
        a = 1.0 / (1.0 + np.exp(-z))
        return a, a * (1.0 - a)
    if kind == "tanh":
        a = np.tanh(z)
        return a, 1.0 - a * a
    return z, np.ones_like(z)


def combine(y_perm, slot_row, topk_w):
    """y[t] = sum_j w[t,j] y_perm[slot_row[t,j]], slots outside the rows skipped."""
    y_perm, w = np.asarray(y_perm, np.float64), np.asarray(topk_w, np.float64)
    rows = np.asarray(slot_row, np.int64)
    y, size = np.zeros((2, rows.shape[0], y_perm.shape[1]))
    for j in range(rows.shape[1]):
        ok = (rows[:, j] >= 0) & (rows[:, j] < y_perm.shape[0])
        term = w[ok, j][:, None] * y_perm[rows[ok, j]]
        y[ok] += term
        size[ok] += np.abs(term)
    return y, size


def norm_scale(v, eps):
    """1 / sqrt(mean(v^2) + eps) of each row"""
    return 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)


def forward(x, y, post_gain, gate, gate_rows, kind, rs, bs, eps, next_gain, y_size=None):
    """(out, h, size of out, size of h); y None: out is x.  y_size: the size of a y that is itself a sum."""
    out = x
    size = np.abs(x)
    if y is not None:
        a = 1.0
        if gate is not None:
            a = act(gate, kind)[0][np.arange(x.shape[0]) // gate_rows]
        f = bs * a * (norm_scale(y, eps) * post_gain if post_gain is not None else 1.0)
        out = rs * x + f * y
        size = np.abs(rs * x) + np.abs(f) * (np.abs(y) if y_size is None else y_size)
    h = h_size = None
    if next_gain is not None:
        r = norm_scale(out, eps)
        h = out * r * next_gain
        # an error of out also moves its norm: at most the norm of the errors, relative to out's
        moved = np.sqrt((size * size).mean(1, keepdims=True)) * r
        h_size = (size + np.abs(out) * moved) * r * np.abs(next_gain)
    return out, h, size, h_size


def norm_backward(v, up, up_size, eps):
    """Gradient of v / q through the norm's Jacobian, and its size."""
    r = norm_scale(v, eps)
    u = v * r
    grad = r * (up - u * (u * up).mean(1, keepdims=True))
    size = r * (up_size + np.abs(u) * (np.abs(u) * up_size).mean(1, keepdims=True))
    return grad, size


def backward(out, y, post_gain, gate, gate_rows, kind, rs, bs, eps, next_gain, d_out, dh):
    """{name: (value, size)} for dx, dy, d_post_gain, dgate, d_next_gain (those that there are)."""
    r = {}
    like = d_out if d_out is not None else dh
    D = np.zeros_like(like) if d_out is None else d_out
    size = np.abs(D)
    if dh is not None:
        u = out * norm_scale(out, eps)
        r["d_next_gain"] = ((dh * u).sum(0), np.abs(dh * u).sum(0))
        more, more_size = norm_backward(out, dh * next_gain, np.abs(dh * next_gain), eps)
        D, size = D + more, size + more_size
    r["dx"] = (rs * D, np.abs(rs) * size)
    if y is None:
        return r
    unit = y * norm_scale(y, eps) if post_gain is not None else y
    n = unit * post_gain if post_gain is not None else unit
    dn, dn_size = bs * D, np.abs(bs) * size
    if gate is not None:
        rows = np.arange(y.shape[0]) // gate_rows
        a, p = (v[rows] for v in act(gate, kind))
        # the slope is computed from a: for 1 - a^2 and a (1 - a) an error of a counts in full
        each, each_size = dn * p * n, dn_size * np.abs(n) * (np.abs(p) + (2.0 if kind != "none" else 0.0))
        dgate, dgate_size = np.zeros((2,) + gate.shape)
        np.add.at(dgate, rows, each)
        np.add.at(dgate_size, rows, each_size)
        r["dgate"] = (dgate, dgate_size)
        dn, dn_size = dn * a, dn_size * np.abs(a)
    if post_gain is not None:
        r["d_post_gain"] = ((dn * unit).sum(0), (dn_size * np.abs(unit)).sum(0))
        dn, dn_size = norm_backward(y, dn * post_gain, dn_size * np.abs(post_gain), eps)
    r["dy"] = (dn, dn_size)
    return r
