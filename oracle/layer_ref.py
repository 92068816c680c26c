"""CPU reference of what a decoder layer runs around its products (numpy): the
residual's addition with an RMS norm to int8, the gated activation to int8, and
attention with a sliding window and visible first tokens.  Written from the
definitions in include/sherry.h; shares no code with the library.

Readings: L1 h = x + r is one fp32 addition, the residual kept is h rounded to
its type, and the norm is of h itself; L2 the sum of squares, mean, eps, root and
reciprocal are fp64, rounded once to fp32, to its largest number where they
pass it; L3 (h a) w are two fp32 products; L4
the codes are act_ref's (A1-A3); L5 the token at position p sees j <= p with
j > p - window or j < sinks.
"""
import numpy as np

from . import act_ref


def rms_norm(x, r, w, eps):
    """x, r (or None) [m, k] of fp32-exact values -> y fp32, h fp32"""
    h = np.asarray(x, np.float32)
    if r is not None:
        h = h + np.asarray(r, np.float32)
    ss = np.array([sum_of_squares(row) for row in h])
    a = 1.0 / np.sqrt(ss / h.shape[1] + np.float64(np.float32(eps)))
    a = np.minimum(a, np.finfo(np.float32).max).astype(np.float32)
    return ((h * a[:, None]).astype(np.float32) * np.asarray(w, np.float32)).astype(np.float32), h


def sum_of_squares(row):
    import math

    d = row.astype(np.float64)
    return math.fsum(d * d)  # squares of fp32 are exact, and fsum rounds once


def rms_norm_quant(x, r, w, eps):
    """-> codes int8 [m, k], scales fp32 [m], h fp32 (to be rounded to the residual's type)"""
    y, h = rms_norm(x, r, w, eps)
    q, s = act_ref.quantize(y)
    return q, s, h


def gate(g, act):
    """fp64"""
    g = np.asarray(g, np.float64)
    if act == "silu":
        z = g
    elif act == "gelu_tanh":
        z = 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    else:
        raise ValueError(act)
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-z))


def gated(g, u, act):
    """fp64 act(g) u"""
    return gate(g, act) * np.asarray(u, np.float64)


def visible(n, length, window, sinks):
    """[n, length] truth values: what each of the n new tokens of a sequence with
    `length` cached ones sees"""
    p = np.arange(n)[:, None] + (length - n)
    j = np.arange(length)[None, :]
    return (j <= p) & ((j > p - window) | (j < sinks))


def window_attention(q, k, v, scale, window, sinks, vmag=None):
    """attn_ref.attention with a window: out fp64 [n, hq, d], lse [n, hq], and
    sum_j w_j vmag_j"""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    vmag = np.abs(v) if vmag is None else vmag
    n, hq, d = q.shape
    length, hkv = k.shape[:2]
    out, mag = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    lse = np.full((n, hq), -np.inf)
    see = visible(n, length, window, sinks)
    for h in range(hq):
        kh = h // (hq // hkv)
        for i in range(n):
            at = np.flatnonzero(see[i])
            if at.size == 0:
                continue
            s = scale * (k[at, kh] @ q[i, h])
            m = s.max()
            e = np.exp(s - m)
            lse[i, h] = m + np.log(e.sum())
            out[i, h] = e @ v[at, kh] / e.sum()
            mag[i, h] = e @ vmag[at, kh] / e.sum()
    return out, lse, mag
