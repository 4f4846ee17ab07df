"""The steps around the attention in fp64 NumPy, written from their definitions: the
rotary positions over several axes and the block selection.  Test infrastructure only."""
import numpy as np


def coordinates(grid):
    """Row-major positions [N, axes] of a grid."""
    return np.stack([x.ravel() for x in np.meshgrid(*[np.arange(g) for g in grid], indexing="ij")], 1)


def rotate(x, pos, dims, theta=1e4, halves=False, inverse=False):
    """x [..., N, d] turned by pos [N, axes], and the sum |a| + |b| of each element's pair
    (0 for channels past the axes)."""
    y, size, at = x.copy(), np.zeros_like(x), 0
    for ax, D in enumerate(dims):
        for j in range(D // 2):
            i, k = (at + j, at + D // 2 + j) if halves else (at + 2 * j, at + 2 * j + 1)
            ang = pos[:, ax] * theta ** (-2.0 * j / D) * (-1 if inverse else 1)
            a, b = x[..., i], x[..., k]
            y[..., i], y[..., k] = a * np.cos(ang) - b * np.sin(ang), a * np.sin(ang) + b * np.cos(ang)
            size[..., i] = size[..., k] = np.abs(a) + np.abs(b)
        at += D
    return y, size


def rotation_bound(want, size, half_step):
    """The error of a rotated value: half a step of its type, and 1e-6 of the pair for
    the angle as one float (2^-24 pi), sincospi (2 ulp) and three fp32 roundings."""
    return half_step * np.abs(want) + 1e-6 * size


def select(q, k, keep, bq, bk, first=0, diagonal=False):
    """Block mask [B, H, nq, nk] of the highest products of block means."""
    N = q.shape[2]
    mean = lambda x, b: np.stack([x[:, :, i:i + b].mean(2) for i in range(0, N, b)], 2)
    s = np.einsum("bhid,bhjd->bhij", mean(q, bq), mean(k, bk))
    i, j = np.arange(s.shape[2])[:, None], np.arange(s.shape[3])[None]
    forced = (j < first) | (diagonal & (j * bk < np.minimum((i + 1) * bq, N)) & (np.minimum((j + 1) * bk, N) > i * bq))
    order = np.argsort(np.where(forced, -np.inf, -s), axis=-1, kind="stable")     # the forced ones first
    kept = np.arange(s.shape[3]) < np.maximum(keep, forced.sum(1))[:, None]
    out = np.zeros(s.shape, np.uint8)
    np.put_along_axis(out, order, np.broadcast_to(kept, s.shape).astype(np.uint8), -1)
    return out
