"""The operators around the core in 64 bits, from their definitions (torch
doubles on the CPU or the GPU), and the error bounds their tests use.

U is half a step of fp32.  A bound counts roundings: every fp32 operation on a
value is off by at most U of it (the fast exponential and reciprocal by 2 U
each, plus 1.3 U per unit of the exponent's argument), and a sum of terms by
at most U per addition along its longest chain, relative to the sum of the
terms' magnitudes.
"""
import torch

U = 2.0 ** -24
BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 1e-30


def half_step(dtype):
    """Half a step of a type, relative to the value; 0 for a result kept in fp32 (its roundings are in U)."""
    return 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2


def norm_chain(hidden):
    """Additions along the longest chain of a row's sum, and the roundings of 1 / sqrt(mean + eps) and of the products
    after it.  A lane adds at most 32 squares, its wave 6 steps, the row 16 waves; the sum's error halves in the root."""
    return 0.5 * (32 + 6 + 16 + 2) + 8


def rms_inv(v, eps):
    return 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)


def sum_h(x, residual):
    """x + residual as stored: one fp32 sum, rounded to the io type."""
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


def rmsnorm(h, weight, eps):
    h = h.double()
    return h * rms_inv(h, eps) * weight.double()


def rmsnorm_backward(h, weight, dy, d_h, eps):
    """(dx, dw, magnitude of dx's terms, magnitude of dw's terms)."""
    h, dy, w = h.double(), dy.double(), weight.double()
    inv = rms_inv(h, eps)
    n, g = h * inv, dy * w
    d = torch.zeros_like(h) if d_h is None else d_h.double()
    dx = inv * (g - n * (g * n).mean(-1, keepdim=True)) + d
    lead = tuple(range(h.dim() - 1))
    return (dx, (dy * n).sum(lead), inv * (g.abs() + n.abs() * (g * n).abs().mean(-1, keepdim=True)) + d.abs(),
            (dy * n).abs().sum(lead))


def output_gate(o, gate, weight, eps):
    o = o.double()
    return o * rms_inv(o, eps) * weight.double() * torch.sigmoid(gate.double())


def output_gate_backward(o, gate, weight, dy, eps):
    """(d_o, dgate, dw, and the magnitudes of the terms of each)."""
    o, dy, w, s = o.double(), dy.double(), weight.double(), torch.sigmoid(gate.double())
    inv = rms_inv(o, eps)
    n, g = o * inv, dy * w * s
    lead = tuple(range(o.dim() - 1))
    return (inv * (g - n * (g * n).mean(-1, keepdim=True)), dy * w * n * s * (1 - s), (dy * n * s).sum(lead),
            inv * (g.abs() + n.abs() * (g * n).abs().mean(-1, keepdim=True)), (dy * w * n * s * (1 - s)).abs(),
            (dy * n * s).abs().sum(lead))


def blocks_of(v, fill=0.0):
    """The last axis in blocks of 128, the last one filled up."""
    short = -v.shape[-1] % BLOCK
    return torch.nn.functional.pad(v, (0, short), value=fill).unflatten(-1, (-1, BLOCK))


def block_scale(y):
    return blocks_of(y).abs().amax(-1).clamp(min=AMAX_FLOOR) / E4M3_MAX


def e4m3_half_step(v):
    """Half the step of e4m3 at |v|: steps of 2^(e - 3) from 2^-6 up, 2^-9 below."""
    _, e = torch.frexp(v)
    return torch.exp2((e - 5).clamp(min=-10).double())


def check_rows_fp8(q, scale, y, rel, note=""):
    """An e4m3 row against its values y in 64 bits, which the kernel's own fp32 values are off by at most rel of."""
    ref = block_scale(y)
    assert torch.isfinite(scale).all(), note
    off = (scale.double() - ref).abs() / ref
    assert off.max() <= rel + 2 * U, f"{note} scale off by {off.max():.2e}"
    v = y / scale.double().repeat_interleave(BLOCK, -1)[..., :y.shape[-1]]
    excess = (q.double() - v).abs() - e4m3_half_step(v) - (rel + 4 * U) * v.abs()
    assert excess.max() <= 0, f"{note} e4m3 off by {excess.max():.2e} beyond half a step"


def check(got, ref, magnitude, rel, note=""):
    """|got - ref| <= rel * magnitude + half a step of got's type."""
    assert torch.isfinite(got).all(), note
    lim = rel * magnitude + half_step(got.dtype) * (ref.abs() + rel * magnitude) + 1e-37
    ratio = ((got.double() - ref).abs() / lim).max().item() if got.numel() else 0.0
    assert ratio <= 1, f"{note} {ratio:.2f} of the bound"


def dequantised(q, scale, rows_per_scale=1):
    s = scale.double()
    if rows_per_scale > 1:
        s = s.repeat_interleave(rows_per_scale, 0)[:q.shape[0]]
    return q.double() * s.repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]


def quantise_weight(w):
    """[N, K] in e4m3 with a scale per 128 x 128 block, as a user's program makes them once."""
    n, k = w.shape
    p = torch.nn.functional.pad(w.float(), (0, -k % BLOCK, 0, -n % BLOCK))
    p = p.view(p.shape[0] // BLOCK, BLOCK, p.shape[1] // BLOCK, BLOCK)
    scale = p.abs().amax((1, 3)).clamp(min=AMAX_FLOOR) / E4M3_MAX
    q = (p / scale[:, None, :, None]).reshape(p.shape[0] * BLOCK, -1)[:n, :k]
    return q.to(torch.float8_e4m3fn).contiguous(), scale


def check_matmul(y, a, a_scale, w, w_scale, rows=slice(None), cols=slice(None), note=""):
    """y against the product in 64 bits.

    An fp32 y: up to 128 additions in a scale block, then a scaled one per block, 16 joined sums and three products, each
    off by at most U.  A bf16 y: the matrix cores cut each product of an e4m3 step at 2^-13 of the step's largest one, so
    a block adds at most 128 * 2^-13 * max|a| max|w| to that, scaled; and since the cuts are small against bf16's own
    rounding (at most 2^-8, on average over a binade's positions 2^-8 / sqrt(3) or less in the 2-norm), the whole
    result's 2-norm error stays under 2^-8 / sqrt(3) + 1e-4 wherever it has 1000 values or more."""
    k = a.shape[-1]
    x, z = dequantised(a, a_scale)[rows], dequantised(w, w_scale, BLOCK)[cols]
    e, m = x @ z.T.contiguous(), x.abs() @ z.abs().T.contiguous()
    lim = (min(k, BLOCK) + (k + BLOCK - 1) // BLOCK + 16 + 3) * U * m
    if y.dtype == torch.bfloat16:
        lim = lim + BLOCK * 2.0 ** -13 * (blocks_of(x).abs().amax(-1) @ blocks_of(z).abs().amax(-1).T.contiguous())
        if e.numel() >= 1000:
            rel = (y.double()[rows][:, cols] - e).norm() / e.norm()
            assert rel <= 2.0 ** -8 / 3 ** 0.5 + 1e-4, f"{note} 2-norm off by {rel:.2e}"
    check(y[rows][:, cols], e, lim, 1.0, note)
