"""64-bit references and inputs of the operators beside the routed-MoE call
(router, MXFP4 linear layer, few-token MoE layer), on the CPU in numpy, from
the definitions in oracle.formats."""

from __future__ import annotations

import numpy as np

from oracle import formats as F

U32 = 2.0 ** -24  # half a step of binary32, relative


def half_step(dtype: str) -> float:
    return {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}[dtype]


def weights(codes, scales):
    """MXFP4 bytes [..., n/2] and E8M0 bytes [..., n/32] -> float64 [..., n]."""
    return F.mx_fp4_decode(F.unpack_fp4(codes), scales)


def random_weights(rng, *shape, lo=118, hi=123):
    """Random MXFP4 codes [..., n/2] (all 16 of them) and scales [..., n/32]."""
    n = shape[-1]
    codes = rng.integers(0, 256, shape[:-1] + (n // 2,), dtype=np.uint8)
    scales = rng.integers(lo, hi, shape[:-1] + (n // 32,), dtype=np.uint8)
    return codes, scales


def sum_error(n):
    """Relative to the sum of magnitudes, the most a binary32 sum of n exact
    products may be off: an MFMA adds 32 products and its accumulator in an
    unknown order (at most 32 roundings, taken as a whole step 2^-23 each, of
    at most the magnitudes' sum), at most n/32 of them are chained, and at
    most 16 partial sums are joined (epilogue additions among them)."""
    return (32 + -(-n // 32) + 16) * 2.0 ** -23


def linear(x, codes, scales, bias=None, residual=None):
    """(exact y, sum of magnitudes) of a linear layer, float64."""
    W = weights(codes, scales)
    y, mag = x @ W.T, np.abs(x) @ np.abs(W).T
    for t in (bias, residual):
        if t is not None:
            y, mag = y + t, mag + np.abs(t)
    return y, mag


def route(logits, k, scaling):
    """Top-k ids (ties to the lower id) and weights of fp32 logits."""
    ids = np.argsort(-logits.astype(np.float64), axis=1, kind="stable")[:, :k]
    sig = 1.0 / (1.0 + np.exp(-np.take_along_axis(logits.astype(np.float64), ids, 1)))
    return ids.astype(np.int32), sig / sig.sum(1, keepdims=True) * scaling


def layer(x, rw, w13, s13, w2, s2, k, scaling):
    """The few-token layer: (out, bound on |binary32 result - out| before the
    final rounding, ids, weights), float64."""
    M, H = x.shape
    I = w13.shape[1] // 2
    logits = (x @ rw.T).astype(np.float32)
    ids, wt = route(logits, k, scaling)
    out, err = np.zeros((M, H)), np.zeros((M, H))
    W13 = {e: weights(w13[e], s13[e]) for e in np.unique(ids)}
    W2 = {e: weights(w2[e], s2[e]) for e in np.unique(ids)}
    for t in range(M):
        for j in range(k):
            A, B = W13[ids[t, j]], W2[ids[t, j]]
            gu, mag = A @ x[t], np.abs(A) @ np.abs(x[t])
            G, U = gu[:I], gu[I:]
            eG, eU = sum_error(H) * mag[:I], sum_error(H) * mag[I:]
            sig = 1.0 / (1.0 + np.exp(-G))
            h = G * sig * U
            # |SiLU'| <= 1.1; SiLU, the products with U and the weight and the
            # weight itself in binary32: under 32 half steps (exp's argument
            # error is |G| half steps, |G| SiLU' small where |G| is large);
            # the two-bf16 split: 2^-17
            eh = 1.1 * eG * (np.abs(U) + eU) + np.abs(G * sig) * eU + np.abs(h) * (32 * U32 + 2.0 ** -17)
            aB = np.abs(B)
            out[t] += wt[t, j] * (B @ h)
            err[t] += wt[t, j] * (aB @ eh + sum_error(2 * I * min(M * k, 256)) * (aB @ np.abs(h)))
    return out, err, ids, wt
