"""Plain CPU oracle for 4-bit weights with group scales and the products over them.

TEST INFRASTRUCTURE ONLY.  Nothing in the product path may import, call or execute
this module; it shares no code with the HIP path.

    W[r, c] = s[r, c // group] (q[r, c] - 8),  q in 0..15
    s = bf16(max over the group |w| * (1/7 in float32)),  q = 8 + round(w / s) clamped to 0..15

Every product runs in float64 with numpy; the scale's rounding to bf16 is done on its
bits.  products() also returns sum |s x| and sum |s (q - 8) x| of each result, which
bound the float32 errors of an evaluation.
"""
from __future__ import annotations

import numpy as np


def round_bf16(a) -> np.ndarray:
    """float32 -> the nearest bf16, halves to even, as float32 (finite values)."""
    b = np.asarray(a, np.float32).view(np.uint32)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & np.uint32(0xFFFF0000)
    return b.view(np.float32)


def groups_of(w, group):
    """w [.., C] padded with zeros to whole groups: [.., ceil(C/group), group]"""
    pad = -w.shape[-1] % group
    w = np.concatenate([w, np.zeros(w.shape[:-1] + (pad,))], -1)
    return w.reshape(w.shape[:-1] + (-1, group))


def quantize(w, group):
    """(codes [.., C], scales [.., ceil(C/group)]) of w, both float64."""
    w = np.asarray(w, np.float64)
    g = groups_of(w, group)
    s = round_bf16(np.abs(g).max(-1).astype(np.float32) * (np.float32(1) / np.float32(7))).astype(np.float64)
    q = np.rint(g / np.where(s > 0, s, 1.0)[..., None])
    q = np.where(s[..., None] > 0, np.clip(q, -8, 7), 0) + 8
    return q.reshape(w.shape[:-1] + (-1,))[..., :w.shape[-1]], s


def values(q, s, group):
    """s (q - 8) for codes [.., C] and scales [.., ceil(C/group)]"""
    C = q.shape[-1]
    return (np.asarray(q, np.float64) - 8) * np.asarray(s, np.float64)[..., np.arange(C) // group]


def products(x, q, s, group):
    """(x W^T, sum |s x|, sum |s (q - 8) x|) for x [T, C], codes [R, C]"""
    x = np.asarray(x, np.float64)
    each = np.asarray(s, np.float64)[..., np.arange(q.shape[-1]) // group]
    W = values(q, s, group)
    return x @ W.T, np.abs(x) @ np.abs(each).T, np.abs(x) @ np.abs(W).T


def silu(z):
    return z / (1.0 + np.exp(-z))
