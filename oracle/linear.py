"""Linear layers in fp64 NumPy, from their formulas.  Test infrastructure only."""
import numpy as np


def product(x, w, bias=None):
    """x w^T + bias, and a bound of an fp32 sum of its K products: 16 at a time, each add off
    by at most 2^-23 of the absolute sum, and 32 adds more for what follows."""
    z = x @ w.T
    size = (w.shape[1] / 16 + 32) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
    if bias is not None:
        z, size = z + bias, size + 2.0 ** -22 * np.abs(bias)
    return z, size


def gelu_tanh(z):
    return 0.5 * z * (1 + np.tanh(np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)))


def gelu_tanh_slope(z):
    k = np.sqrt(2 / np.pi)
    t = np.tanh(k * (z + 0.044715 * z ** 3))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
