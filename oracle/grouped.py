"""Float64 references of the expert-grouped and 8-bit integer products (test infrastructure).

Plain loops over groups in float64 (integers in int64) on values already
decoded; no code shared with the CUDA library.  Each product also returns its
error scale D: the sum of absolute values that went into each output, the
denominator of the normalised error.
"""
from __future__ import annotations

import numpy as np

from . import EPI_BIAS_GELU, EPI_BIAS_GELU_TANH, EPI_BIAS_RELU, EPI_BIAS_SILU, EPI_NONE, gelu, gelu_tanh, relu, silu

_ACT = {EPI_BIAS_GELU: gelu, EPI_BIAS_GELU_TANH: gelu_tanh, EPI_BIAS_SILU: silu, EPI_BIAS_RELU: relu}


def grouped_reference(offsets, A, B, epilogue=EPI_NONE, alpha=1.0, beta=0.0, C=None, bias=None, row_scale=None,
                      col_scale=None):
    """Y, D for A (M x K), B (G x K x N), bias / col_scale (G x N), row_scale (M); rows in no group keep C
    (NaN without one) and D = 0.  alpha == 0 or K == 0 leaves A, B and the scales out."""
    M, N = A.shape[0], B.shape[2]
    Y = np.full((M, N), np.nan) if C is None else np.array(C, dtype=np.float64)
    D = np.zeros((M, N))
    for g in range(B.shape[0]):
        r0, r1 = int(offsets[g]), int(offsets[g + 1])
        z = np.zeros((r1 - r0, N))
        d = np.zeros((r1 - r0, N))
        if alpha != 0.0 and A.shape[1] > 0:
            s = np.full((r1 - r0, N), float(alpha))
            if row_scale is not None:
                s = s * np.asarray(row_scale[r0:r1], dtype=np.float64)[:, None]
            if col_scale is not None:
                s = s * np.asarray(col_scale[g], dtype=np.float64)
            z = s * (A[r0:r1] @ B[g])
            d = np.abs(s) * (np.abs(A[r0:r1]) @ np.abs(B[g]))
        if beta != 0.0:
            z = z + beta * C[r0:r1]
            d = d + np.abs(beta * C[r0:r1])
        if epilogue != EPI_NONE:
            z = z + bias[g]
            d = d + np.abs(bias[g])
            z = _ACT.get(epilogue, lambda v: v)(z)
        Y[r0:r1] = z
        D[r0:r1] = d
    return Y, D


def wgrad_reference(offsets, A, Dy, alpha=1.0, beta=0.0, C=None, a_sum=None):
    """(C[g], D, a_sum[g], D of a_sum) for A (T x M) and Dy (T x N)."""
    G, M, N = len(offsets) - 1, A.shape[1], Dy.shape[1]
    Y, D = np.zeros((G, M, N)), np.zeros((G, M, N))
    S, SD = np.zeros((G, M)), np.zeros((G, M))
    for g in range(G):
        r0, r1 = int(offsets[g]), int(offsets[g + 1])
        if alpha != 0.0:
            Y[g] = alpha * (A[r0:r1].T @ Dy[r0:r1])
            D[g] = abs(alpha) * (np.abs(A[r0:r1]).T @ np.abs(Dy[r0:r1]))
            S[g] = alpha * A[r0:r1].sum(0)
            SD[g] = abs(alpha) * np.abs(A[r0:r1]).sum(0)
        if beta != 0.0:
            Y[g] += beta * C[g]
            D[g] += np.abs(beta * C[g])
            if a_sum is not None:
                S[g] += beta * a_sum[g]
                SD[g] += np.abs(beta * a_sum[g])
    return Y, D, S, SD


def quantize_reference(X):
    """Codes (int8) and scales (float64) of the rows of X: round half to even of 127 x / max|x|, max|x| / 127;
    0 for a row of zeros, NaN scale and codes 0 for a row that is not finite."""
    q = np.zeros(X.shape, dtype=np.int8)
    scale = np.zeros(X.shape[0])
    for i, x in enumerate(X):
        if x.size and not np.isfinite(x).all():
            scale[i] = np.nan
            continue
        peak = np.abs(x).max() if x.size else 0.0
        scale[i] = peak / 127.0
        if peak > 0:
            q[i] = np.rint(127.0 * x / peak).astype(np.int8)
    return q, scale
