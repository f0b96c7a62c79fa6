"""Attention of rows that see given counts of positions, in 64 bits, and what its kernels may be off by.

The bounds are of kernels that hold queries as they are given, weights to 2^-16 and every sum in fp32, whatever else is
in the call (U is half a step of fp32)."""
import torch

from tests.layer_reference import U


def attention(q, k, v, sees, scale):
    """q [t, Hq, d], k, v [heads, n, d] in 64 bits; token j sees the first sees[j] positions.  Returns o, lse, sum w|v| and
    the largest sum |scale q k| of each row."""
    t, Hq, d = q.shape
    heads, n = k.shape[:2]
    o, m = torch.zeros(t, Hq, d, dtype=torch.float64), torch.zeros(t, Hq, d, dtype=torch.float64)
    lse, top = torch.full((t, Hq), -torch.inf, dtype=torch.float64), torch.zeros(t, Hq, dtype=torch.float64)
    sees = torch.as_tensor(sees)
    hidden = torch.arange(n) >= sees[:, None]
    some = sees > 0
    for h in range(Hq):
        kk, vv = k[h * heads // Hq], v[h * heads // Hq]
        s = (q[:, h] @ kk.T.contiguous() * scale).masked_fill(hidden, -torch.inf)
        w = torch.softmax(s, -1)[some]
        o[some, h], m[some, h] = w @ vv, w @ vv.abs()
        lse[some, h] = torch.logsumexp(s, -1)[some]
        top[:, h] = (q[:, h].abs() @ kk.abs().T.contiguous()).masked_fill(hidden, 0).amax(-1) * abs(scale)
    return o, lse, m, top


def bounds(d, length, top, out_dtype):
    """Errors of o relative to sum w|v| (as [.., 1]), and of lse.

    A score has d products summed and is scaled (d + 2 roundings of its terms' sum) and moves by three more where the maximum
    is taken off; the exponential 2, and 1.3 per unit of an argument that the score's own bound counts.  Each moves weight and
    sum.  A weight as two bf16 values is off by 2^-16, as three by U.  Sums: 16 positions a product at the least, for each
    piece (length / 8 steps of two pieces), 32 within a step, and 600 for what is joined after."""
    score = (d + 5) * U * top + 4 * U
    pieces = 2.0 ** -16 if out_dtype == torch.bfloat16 else U
    return (2 * score + pieces + (32 + length / 8 + 600) * U)[..., None], score + (length / 16 + 600) * U
