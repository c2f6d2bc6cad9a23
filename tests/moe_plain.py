"""The mixture-of-experts operators from their definitions, in 64 bits (numpy),
and the inputs of their tests.  Each expert's weights come from the oracle."""
import numpy as np

import oracle

U16 = 2.0 ** -11  # half a step of FP16, relative
U16_TINY = 2.0 ** -25  # half a step of its smallest values
U32 = 2.0 ** -24


def sort(ids, E):
    """(offsets [E + 1], dest [M, topk]) of expert ids [M, topk]."""
    M, topk = ids.shape
    dest = np.full(M * topk, -1, dtype=np.int32)
    offsets = [0]
    flat = ids.reshape(-1)
    row = 0
    for e in range(E):
        for p in np.flatnonzero(flat == e):
            dest[p] = row
            row += 1
        offsets.append(row)
    return np.array(offsets, dtype=np.int32), dest.reshape(M, topk)


def sorted_rows(x, dest, out):
    """`out` with the tokens' rows at their places."""
    out = out.copy()
    for m in range(dest.shape[0]):
        for d in dest[m]:
            if d >= 0:
                out[d] = x[m]
    return out


def combine(y, dest, weights):
    """(sums in 64 bits [M, H], sums of the terms' magnitudes)."""
    M, topk = dest.shape
    out = np.zeros((M, y.shape[1]))
    size = np.zeros_like(out)
    for m in range(M):
        for j, d in enumerate(dest[m]):
            if d >= 0:
                w = 1.0 if weights is None else np.float64(weights[m, j])
                out[m] += w * y[d].astype(np.float64)
                size[m] += abs(w) * np.abs(y[d].astype(np.float64))
    return out, size


def combine_tol(ref, size, topk):
    # topk FP32 multiply-adds, then one rounding to FP16
    return topk * U32 * size * (1 + U16) + U16 * np.abs(ref) + U16_TINY


def dweights(dout, y, dest):
    """(dot products in 64 bits [M, topk], sums of magnitudes)."""
    out = np.zeros(dest.shape)
    size = np.zeros(dest.shape)
    g = dout.astype(np.float64)
    for m in range(dest.shape[0]):
        for j, d in enumerate(dest[m]):
            if d >= 0:
                t = g[m] * y[d].astype(np.float64)
                out[m, j], size[m, j] = t.sum(), np.abs(t).sum()
    return out, size


def expert_weights(qweight, scales, group):
    """[E, K, N] FP16, each expert's from the oracle."""
    return np.stack([oracle.dequant(np.ascontiguousarray(q), np.ascontiguousarray(s), group)
                     for q, s in zip(qweight, scales)])


def product(rows, w, offsets, gradient=False):
    """(products in 64 bits [R, width], sums of magnitudes); NaN in the rows
    that belong to no expert."""
    w64 = w.astype(np.float64)
    width = w.shape[1] if gradient else w.shape[2]
    out = np.full((rows.shape[0], width), np.nan)
    size = np.full_like(out, np.nan)
    r64 = rows.astype(np.float64)
    for e in range(w.shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            we = w64[e].T if gradient else w64[e]
            out[lo:hi] = r64[lo:hi] @ we
            size[lo:hi] = np.abs(r64[lo:hi]) @ np.abs(we)
    return out, size


def product_tol(ref, size, length):
    """FP32 sums of `length` exact products in any order; the tensor cores may
    truncate instead of rounding, hence twice U32 each; then one rounding."""
    return 2 * U32 * length * size * (1 + U16) + U16 * np.abs(ref) + U16_TINY


def make_rows(rng, rows, width):
    return rng.standard_normal((rows, width)).astype(np.float16)


def make_weights(rng, E, K, N, group):
    n_groups = 1 if group == -1 or group >= K else -(-K // group)
    q = rng.integers(-2 ** 31, 2 ** 31, size=(E, K // 8, N), dtype=np.int64).astype(np.int32)
    s = rng.uniform(1e-3, 2e-2, size=(E, n_groups, N)).astype(np.float16)
    return q, s


def make_ids(rng, M, E, topk, drop=0.0, skew=1.0):
    """Distinct experts per token (random scores with a bias per expert), some
    choices dropped."""
    scores = rng.standard_normal((M, E)) + skew * rng.standard_normal(E)
    ids = np.argsort(-scores, axis=1)[:, :topk].astype(np.int32)
    ids[rng.random(ids.shape) < drop] = -1
    return ids


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
