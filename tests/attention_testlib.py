"""Attention in 64 bits and what rounding allows a kernel to be off by, for the tests of the serving operators."""
import math

import torch

D = 128


def attend(q, K, V, sees):
    """64-bit attention of rows q [n][D] over K, V [m][D] with sees [n][m]: values, sum p |v|, and the largest
    sum |q k| scale of a row (what logit errors scale with).  Rows that see nothing are zeros."""
    scale = 1 / math.sqrt(D)
    K, V = K.double().nan_to_num(0, 0, 0), V.double().nan_to_num(0, 0, 0)
    q = q.double()
    x = (q @ K.T * scale).masked_fill(~sees, -math.inf)
    dead = ~sees.any(-1, keepdim=True)
    p = torch.softmax(x.masked_fill(dead, 0), -1).masked_fill(dead, 0)
    return p @ V, p @ V.abs(), (q.abs() @ K.abs().T * scale).amax(-1, keepdim=True)


def close(got, want, absv, qk, n, dtype):
    """What rounding allows.  fp32: a logit is a sum of 128 products, off by at most 130 half steps of sum |q k|, which
    moves p by twice that (itself and its row sum); n products and sums of P.V, and a few more per merge (64); bf16
    adds the rounding of p to bf16 in P.V (half a step of bf16 each) and that of the result."""
    u = 2.0 ** -24
    tol = absv * (2 * 130 * u * qk + (2 * n + 64) * u)
    if dtype == torch.bfloat16:
        half = torch.finfo(dtype).eps / 2
        tol = tol + absv * half * 1.01 + want.abs() * half * 1.01
    else:
        tol = tol + want.abs() * u
    err = (got.double() - want).abs()
    assert bool((err <= tol + 1e-30).all()), float((err - tol).max())
