"""Activations of the products' epilogues and their derivatives in 64 bits."""

import math

import numpy as np

NONE, RELU, GELU, GELU_TANH, SILU = range(5)
_ERFC = np.vectorize(math.erfc, otypes=[np.float64])


def _sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


def value(z, act):
    z = np.asarray(z, np.float64)
    if act == RELU:
        return np.maximum(z, 0)
    if act == GELU:
        return 0.5 * z * _ERFC(-z / math.sqrt(2))
    if act == GELU_TANH:
        return z * _sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if act == SILU:
        return z * _sigmoid(z)
    return z


def slope(z, act):
    z = np.asarray(z, np.float64)
    if act == RELU:
        return (z > 0).astype(np.float64)
    if act == GELU:
        return 0.5 * _ERFC(-z / math.sqrt(2)) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == GELU_TANH:
        c = 2 * math.sqrt(2 / math.pi)
        s = _sigmoid(c * (z + 0.044715 * z ** 3))
        return s + z * s * (1 - s) * c * (1 + 3 * 0.044715 * z * z)
    if act == SILU:
        s = _sigmoid(z)
        return s * (1 + z * (1 - s))
    return np.ones_like(z)
