"""The full-attention layers' operators in 64 bits, from their definitions, and
the error bounds their tests use (U is half a step of fp32)."""
import torch

from tests.layer_reference import U

BLOCK = 32
MAGNITUDES = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def pair_channels(rot, interleaved):
    """(first, second) channels of the rotated pairs."""
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def angles(inv_freq, axis, positions):
    """[n, pairs] in 64 bits: positions [axes, n]."""
    ax = torch.zeros(len(inv_freq), dtype=torch.long) if axis is None else axis.long().cpu().clamp(0, len(positions) - 1)
    return positions.double().cpu()[ax].T * inv_freq.double().cpu()


def rotate(x, angle, rot, interleaved):
    """x [n, heads, d], angle [n, pairs]."""
    a, b = pair_channels(rot, interleaved)
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    y = x.clone()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y


def pair_magnitude(x, rot, interleaved):
    """|a| + |b| over the rotated pairs, |x| elsewhere."""
    a, b = pair_channels(rot, interleaved)
    m = x.abs()
    y = m.clone()
    y[..., a] = y[..., b] = m[..., a] + m[..., b]
    return y


def normed(x, weight, eps):
    x = x.double().cpu()
    return x if weight is None else x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double().cpu()


# The sum of squares: 16 in a lane, 4 steps over its lanes, the mean and eps, halved by the root (11); the root 2 with its
# step, the weight and the row 2; a product and a sum or difference in the rotation 2; sine and cosine: the hardware's
# 1.2e-7 (2), the angle in turns rounded to fp32 (pi / 2 of a turn's rounding at half a turn, 4 with both).
ROPE_REL = (11 + 2 + 2 + 2 + 2 + 4 + 1) * U


def qk_backward(x, weight, dy, angle, rot, interleaved, eps):
    """(dx, dw, magnitudes of the terms of each)."""
    x, g = x.double().cpu(), dy.double().cpu()
    gm = g.abs()
    if rot:
        g, gm = rotate(g, -angle, rot, interleaved), pair_magnitude(g, rot, interleaved)
    if weight is None:
        return g, None, gm, None
    w = weight.double().cpu()
    inv = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n, u, um = x * inv, g * w, gm * w.abs()
    dx = inv * (u - n * (u * n).mean(-1, keepdim=True))
    return (dx, (g * n).sum((0, 1)), inv * (um + n.abs() * (um * n.abs()).mean(-1, keepdim=True)),
            (gm * n.abs()).sum((0, 1)))


def quantised(x):
    """[..., d] -> (codes uint8 [..., d], scale bytes uint8 [..., d / 32]) of the nearest values, in 64 bits."""
    x = x.double()
    b = x.unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1)
    e = torch.full(top.shape, 1, dtype=torch.long, device=x.device)
    m, p = torch.frexp(torch.where(top.isfinite(), top, torch.ones_like(top)))
    e = torch.where(m <= 0.75, p - 3, p - 2).long() + 127      # 6 = 0.75 * 2^3
    bad = ~(top < 2.0 ** 127)                                  # NaN, infinite, too large
    e = torch.where(bad, 255, e.clamp(min=1))
    v = b / torch.exp2((e - 127).double())[..., None]
    size = torch.tensor(MAGNITUDES, dtype=torch.float64, device=x.device)
    middle = (size[1:] + size[:-1]) / 2
    a = v.abs()[..., None]
    odd = torch.arange(1, 8, device=x.device) % 2 == 1
    code = torch.where(odd, a > middle, a >= middle).sum(-1)   # a tie goes to the even code
    code = torch.where(bad[..., None], 0, code + 8 * torch.signbit(v).long())
    return code.flatten(-2).to(torch.uint8), e.to(torch.uint8)


def values(code, scale):
    """What codes [..., d] and scale bytes [..., d / 32] stand for, in 64 bits."""
    size = torch.tensor(MAGNITUDES, dtype=torch.float64, device=code.device)
    v = size[(code & 7).long()] * torch.where(code >= 8, -1.0, 1.0)
    s = torch.where(scale == 255, torch.nan, torch.exp2(scale.double() - 127))
    return (v.unflatten(-1, (-1, BLOCK)) * s[..., None]).flatten(-2)


def stored(pages, table, length):
    """The codes and scales of a sequence's first `length` positions, [heads, length, ...]: pages (values, scales)."""
    byte, scale = pages
    size = byte.shape[2]
    at = torch.arange(length, device=byte.device)
    page = table.long()[at // size]
    b = byte[page, :, at % size].transpose(0, 1)
    s = scale[page, :, :, at % size].transpose(0, 1)
    return torch.stack((b & 15, b >> 4), -1).flatten(-2), s


def attention(q, k, v, length, scale):
    """q [t, Hq, d], k, v [heads, length, d] in 64 bits, the last t of `length` positions being q's own.
    Returns (o, lse, sum w|v|, (the largest sum |scale q k| of each row, the largest sum over blocks of 32 channels of
    max|q| sum|k| times scale))."""
    t, Hq, d = q.shape
    heads = k.shape[0]
    o, m = torch.zeros(t, Hq, d, dtype=torch.float64), torch.zeros(t, Hq, d, dtype=torch.float64)
    lse, top = torch.full((t, Hq), -torch.inf, dtype=torch.float64), torch.zeros(2, t, Hq, dtype=torch.float64)
    block = k.abs().unflatten(-1, (-1, BLOCK)).sum(-1)
    for j in range(t):
        sees = min(length, length - t + j + 1)
        if sees <= 0:
            continue
        for h in range(Hq):
            g = h * heads // Hq
            kk, vv = k[g, :sees], v[g, :sees]
            s = kk @ q[j, h] * scale
            w = torch.softmax(s, 0)
            o[j, h], m[j, h], lse[j, h] = w @ vv, w @ vv.abs(), torch.logsumexp(s, 0)
            top[0, j, h] = (kk.abs() @ q[j, h].abs()).max() * abs(scale)
            top[1, j, h] = (block[g, :sees] @ q[j, h].abs().unflatten(-1, (-1, BLOCK)).amax(-1)).max() * abs(scale)
    return o, lse, m, top


def attention_rel(d, length, top, q_dtype, out_dtype, rows):
    """Error of o relative to sum w|v| (as [.., 1]), and of lse, for a key head's `rows` rows of one sequence (0: not known).

    A score has d products summed and is scaled (d + 2 roundings of its terms' sum), and moves by as much again when the
    maximum is taken off; the exponential 2.  Each moves weight and sum.  For bf16 outputs a query's three 6-bit pieces
    leave half a step of the last, 2^-12 of the first's unit, which is less than its block's largest / 3.75; the pieces'
    products are exact.  The weights' pieces: two bf16 leave 2^-16, one 2^-8 (in the sum that divides too; the most for
    rows above 16), three 2^-24.  A step sums 32 products, a row at most length / 32 steps and their joins."""
    score = (d + 2 + 3) * U * top[0] + 4 * U
    if out_dtype == torch.bfloat16:
        score = score + 2.0 ** -12 / 3.75 * top[1]
        pieces = 2.0 ** -16 if 0 < rows <= 16 else 2 * 2.0 ** -8
    else:
        pieces = U
    lse = 0.0 if pieces < 2.0 ** -15 else 2.0 ** -8
    return (2 * score + pieces + (32 + length / 32 + 600) * U)[..., None], score + lse + (length / 8 + 600) * U
