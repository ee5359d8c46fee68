"""The operators on 4-bit weights by their definitions, in fp64 on the CPU
(test infrastructure: shares no code with the CUDA path).

A layer's weight is W[r, i] = scales[g, r] * n[r, i], n = u - (z + 1), g = i // 128,
from GPTQ v1 tensors with act-order off; a table's row v is scale * (u - 8) from
the selection's scales and code words.
"""
from __future__ import annotations

import math

import numpy as np

from . import gptq

GROUP = gptq.GROUP
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def layer(qweight, qzeros, scales):
    """(n float64 [R, K], s float64 [R, K/128]) of a layer's v1 tensors."""
    K, R = qweight.shape[0] * 8, qweight.shape[1]
    ones = np.full(np.asarray(scales).shape, np.float16(1).view(np.uint16))
    n = gptq.dequantize_v1(qweight, qzeros, ones, np.arange(K) // GROUP)
    return n, np.asarray(scales, dtype=np.uint16).view(np.float16).astype(np.float64).T.copy()


def weight(n, s):
    return n * np.repeat(s, GROUP, axis=1)


def activation(z, act):
    z = np.asarray(z, dtype=np.float64)
    if act == "none":
        return z
    if act == "relu":
        return np.where(z < 0, 0.0, z)
    if act == "gelu":
        return 0.5 * z * _erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z / (1 + np.exp(-z))


def slope(z, act):
    z = np.asarray(z, dtype=np.float64)
    if act == "none":
        return np.ones_like(z)
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "gelu":
        return 0.5 * _erfc(-z / math.sqrt(2)) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    p = 1 / (1 + np.exp(-z))
    return p * (1 + z * (1 - p))


def linear(x, n, s, bias=None, act="none", residual=None):
    """(y, pre) of y = act(x W^T + bias) + residual."""
    z = x @ weight(n, s).T
    if bias is not None:
        z = z + bias
    y = activation(z, act)
    return (y if residual is None else y + residual), z


def linear_backward(dz, x, n, s):
    """(dx, dscales [K/128, R])."""
    R, K = n.shape
    dw = dz.T @ x
    return dz @ weight(n, s), (dw * n).reshape(R, K // GROUP, GROUP).sum(axis=2).T.copy()


def activation_backward(dy, pre, act):
    dz = dy * slope(pre, act)
    return dz, dz.sum(axis=0)


def table(scales, codes, K):
    """(q float64 [V, K], s float64 [V, K/128]) of a quantised table."""
    q = gptq.unpack_group_codes(codes).astype(np.float64) - gptq.ZERO
    s = np.asarray(scales, dtype=np.uint16).view(np.float16).astype(np.float64)
    return q.reshape(-1, K), s.reshape(-1, K // GROUP)


def embedding(ids, q, s, multiplier=1.0):
    out = np.zeros((len(ids), q.shape[1]))
    for t, v in enumerate(ids):
        if 0 <= v < q.shape[0]:
            out[t] = multiplier * np.repeat(s[v], GROUP) * q[v]
    return out


def embedding_backward(dout, ids, q, multiplier=1.0):
    out = np.zeros((q.shape[0], q.shape[1] // GROUP))
    for t, v in enumerate(ids):
        if 0 <= v < q.shape[0]:
            out[v] += multiplier * (dout[t] * q[v]).reshape(-1, GROUP).sum(axis=1)
    return out
