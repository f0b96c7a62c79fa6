"""The steps of the full-attention layers that stand between KDA layers in a hybrid decoder, as a user calls them, and their plain forms.

  rope       RMS norm of each query and key head and the rotation by position, one or several position axes
  rope_bwd   its gradients, of q, k and both weights
  append     new keys (normed and rotated on the way) and values into a paged cache of 4 bits, and those rows read back
  attend     attention of each sequence's newest tokens over that cache: one token, a few drafts, or a long chunk

The cache holds e2m1 values (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign), two to a byte, with one power of two (e8m0) for
each 32 channels: the least 2^e with max|v| <= 6 * 2^e.

Sizes are those of the library's own workloads (256 decoding sequences, prefills of 32768 tokens, 32 heads of 128, the
page's 16 query and 2 key heads with a quarter of the channels rotated, drafts of a few tokens) and generic odd ones.
"""
import torch

own = False

EPS = 1e-6
THETA = 1e6
BLOCK = 32
T = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


def listed():
    return [
        # one sequence decoding: latency alone
        {"name": "rope_decode", "op": "rope", "n": 1, "hq": 16, "hkv": 2, "d": 256, "rot": 64, "axes": 1, "inter": False, "io": "bf16"},
        # a prefill of images and text: three position axes
        {"name": "rope_prefill_axes", "op": "rope", "n": 32768, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "axes": 3, "inter": False, "io": "bf16"},
        # an all-fp32 model, odd counts, neighbouring channels paired
        {"name": "rope_fp32_odd", "op": "rope", "n": 1021, "hq": 7, "hkv": 1, "d": 64, "rot": 48, "axes": 1, "inter": True, "io": "fp32"},
        # a training step over one 32768-token sequence
        {"name": "rope_bwd_train", "op": "rope_bwd", "n": 32768, "hq": 16, "hkv": 2, "d": 256, "rot": 64, "axes": 1, "inter": False, "io": "bf16"},
        # a small ragged fp32 training batch with two axes
        {"name": "rope_bwd_fp32_odd", "op": "rope_bwd", "n": 777, "hq": 6, "hkv": 3, "d": 128, "rot": 64, "axes": 2, "inter": True, "io": "fp32"},
        # a decode step of 256 sequences: one key and value each, at the end of ragged contexts
        {"name": "append_decode", "op": "append", "seqs": 256, "q": 1, "ctx": 8192, "hq": 16, "hkv": 2, "d": 256, "rot": 64, "axes": 1, "inter": False, "page": 64, "io": "bf16"},
        # the prefill of 4 x 32768 tokens
        {"name": "append_prefill", "op": "append", "seqs": 4, "q": 32768, "ctx": 32768, "hq": 16, "hkv": 2, "d": 256, "rot": 64, "axes": 1, "inter": False, "page": 64, "io": "bf16"},
        # ragged chunks of an fp32 model behind contexts of their own, three axes
        {"name": "append_fp32_odd", "op": "append", "seqs": 13, "q": 301, "ctx": 4001, "hq": 6, "hkv": 3, "d": 64, "rot": 64, "axes": 3, "inter": True, "page": 32, "io": "fp32"},
        # one sequence at the start of its answer, fp32: latency alone
        {"name": "attend_one_fp32", "op": "attend", "seqs": 1, "q": 1, "ctx": 777, "hq": 6, "hkv": 3, "d": 64, "page": 32, "io": "fp32"},
        # a decode step of 256 sequences of ragged lengths up to 8192: the cache's bytes
        {"name": "attend_decode", "op": "attend", "seqs": 256, "q": 1, "ctx": 8192, "hq": 16, "hkv": 2, "d": 256, "page": 64, "io": "bf16"},
        # three draft tokens and the last accepted one, 32 heads in groups of 4
        {"name": "attend_drafts", "op": "attend", "seqs": 37, "q": 4, "ctx": 16384, "hq": 32, "hkv": 8, "d": 128, "page": 128, "io": "bf16"},
        # chunks of two long prompts behind what is cached already: the matrix cores' rate
        {"name": "attend_prefill", "op": "attend", "seqs": 2, "q": 2048, "ctx": 16384, "hq": 16, "hkv": 2, "d": 256, "page": 64, "io": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, its logarithm spread evenly."""
    return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "append", "attend", "attend"])
    io = rng.choice(["bf16", "bf16", "fp32"])
    d, hkv, group = rng.choice([64, 128, 256]), _spread(rng, 1, 8), _spread(rng, 1, 16)
    c = {"op": op, "hq": hkv * group, "hkv": hkv, "d": d}
    if op != "attend":
        rot = rng.choice([r for r in (16, 32, 48, 64, 96, 128, 192, 256) if r <= d])
        c.update(rot=rot, axes=rng.choice([1, 1, 2, 3]), inter=rng.random() < 0.3)
    if op in ("rope", "rope_bwd"):
        most = 32768 * 18 * 256 * 2 // SIZE[io] // ((hkv + c["hq"]) * d)
        return {**c, "n": _spread(rng, 1, max(1, min(32768, most))), "io": io}
    c["page"] = rng.choice([32, 64, 128, 256])
    if op == "append":
        most = 110000 * 2 * 256 * 2 // SIZE[io] // (hkv * d)   # tokens, a little under the largest listed case
        seqs = _spread(rng, 1, min(256, most))
        q = _spread(rng, 1, min(32768, most // seqs))
        return {**c, "seqs": seqs, "q": q, "ctx": min(32768, q + _spread(rng, 1, 8192)), "io": io}
    if rng.random() < 0.3:     # a chunk of prompts
        most = (240 if io == "bf16" else 60) * 10**9 // (c["hq"] * d)   # sequences x new tokens x tokens held
        q = _spread(rng, 16, min(2048, int(most ** 0.5)))
        seqs = _spread(rng, 1, min(4, most // q**2))
        ctx = min(16384, _spread(rng, q, max(q, most // (seqs * q))))
    else:
        q = rng.choice([1, 1, 1, 2, 3, 5, 8])
        seqs = _spread(rng, 1, 256)
        ctx = _spread(rng, 16, max(16, min(65536, 256 * 8192 * 2 * 256 // (seqs * hkv * d))))
    return {**c, "seqs": seqs, "q": min(q, ctx), "ctx": ctx, "io": io}


def _fill(i, step):
    return (i * step) % 1.0


def _lengths(case):
    """(new tokens, tokens held with them) of each sequence: ragged, the same for every seed."""
    some = [(case["q"] if case["q"] < 16 or case["seqs"] < 3 else max(1, round(case["q"] * (0.2 + 0.8 * _fill(i + 1, 0.7548776662)))),
             round(case["ctx"] * (0.1 + 0.9 * _fill(i + 1, 0.6180339887))) if case["seqs"] > 2 else case["ctx"])
            for i in range(case["seqs"])]
    return [(q, max(q, n)) for q, n in some]


def _codes(g, shape):
    """Bytes of e2m1 values of normal data, and scales as they leave blocks of it, some channels far larger."""
    x = torch.randn((*shape[:-1], shape[-1] // BLOCK, BLOCK), generator=g, device="cuda")
    values, e = _quantised(x * 0.2)
    e = e + (torch.rand(e.shape, generator=g, device="cuda") < 0.05).to(torch.int32) * 2
    return _packed(values.flatten(-2)), (e + 127).to(torch.uint8).transpose(-1, -2).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def ints(hi, *shape):
        return torch.randint(0, hi, shape, generator=g, device="cuda", dtype=torch.int32)

    s = {"case": dict(case)}
    op, io, d, hq, hkv = case["op"], T[case["io"]], case["d"], case["hq"], case["hkv"]
    if op != "attend":
        half = case["rot"] // 2
        s["inv_freq"] = (THETA ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
        s["axis"] = (torch.arange(half, device="cuda") * case["axes"] // half).int()
        s["k_weight"] = 1 + 0.1 * randn(d)
    if op in ("rope", "rope_bwd"):
        n = case["n"]
        row = 10.0 ** (2 * torch.rand((n, 1, 1), generator=g, device="cuda") - 1)
        s["q"], s["k"] = (randn(n, hq, d) * row).to(io), (randn(n, hkv, d) * row).to(io)
        s["q_weight"] = 1 + 0.1 * randn(d)
        # text runs on from a far place; images have places of their own on each axis
        s["positions"] = (ints(262144, 1) + torch.arange(n, device="cuda", dtype=torch.int32))[None] if case["axes"] == 1 else ints(65536, case["axes"], n)
        if op == "rope_bwd":
            s["dq_out"], s["dk_out"] = randn(n, hq, d).to(io), randn(n, hkv, d).to(io)
    else:
        lens, P = _lengths(case), case["page"]
        n = sum(q for q, _ in lens)
        s["lengths"] = torch.tensor([m for _, m in lens], dtype=torch.int32, device="cuda")
        s["cu"] = torch.tensor([0] + [q for q, _ in lens], device="cuda").cumsum(0).int()
        s["max_q"] = max(q for q, _ in lens)
        held = [(m + P - 1) // P for _, m in lens]
        pages, wide = sum(held), max(held)
        order = torch.randperm(pages, generator=g, device="cuda").int()
        # places of the table behind a sequence's last page hold -1
        at = torch.tensor(held, device="cuda")[:, None] > torch.arange(wide, device="cuda")
        s["table"] = torch.full((len(lens), wide), -1, dtype=torch.int32, device="cuda").masked_scatter(at, order)
        if op == "append":
            s["k_new"], s["v_new"] = (randn(n, hkv, d) * 3).to(io), randn(n, hkv, d).to(io)
            s["positions"] = ints(65536, case["axes"], n) if case["axes"] > 1 else None
            b = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device="cuda")   # noqa: E731
            s["cache"] = [t for _ in "kv" for t in (b(pages, hkv, P, d // 2), b(pages, hkv, d // BLOCK, P))]
        else:
            s["cache"] = [t for _ in "kv" for t in _codes(g, (pages, hkv, P, d))]
            s["q"] = (randn(n, hq, d) * 3).to(io)
    if own:
        import gated_delta_rule_03_amd as kda
        s["cfg"] = kda.Config(A_log=None, dt_bias=None, conv_w_q=None, conv_w_k=None, conv_w_v=None, num_heads=hq,
                              head_k_dim=d, head_v_dim=d, io_dtype=io, out_dtype=io)
        if op != "attend":
            s["rope"] = kda.Rope(s["inv_freq"], axis=s["axis"], num_axes=case["axes"], interleaved=case["inter"])
        if "cache" in s:
            s["kv"] = kda.KvCache(*s["cache"])
    return s


# ---- the plain forms -------------------------------------------------------

def _cos_sin(s, positions):
    """cos and sin of every frequency, [n, 1, rot / 2]; the angles of far positions need 64 bits."""
    a = (positions.double()[s["axis"].long()] * s["inv_freq"].double()[:, None]).t()[:, None]
    return torch.cos(a), torch.sin(a)


def _pairs(x, case):
    """The two members of each pair of the rotated channels, and the others."""
    r = x[..., :case["rot"]]
    a, b = (r[..., 0::2], r[..., 1::2]) if case["inter"] else r.chunk(2, -1)
    return a, b, x[..., case["rot"]:]


def _whole(a, b, rest, case):
    r = torch.stack((a, b), -1).flatten(-2) if case["inter"] else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1)


def _rotated(x, cos, sin, case):
    a, b, rest = _pairs(x, case)
    return _whole(a * cos - b * sin, a * sin + b * cos, rest, case)


def _normed(x, weight):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight


def _norm_rope_bwd(x, weight, dy, cos, sin, case):
    x, g = x.float(), _rotated(dy.float(), cos, -sin, case)
    inv = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    n, gw = x * inv, g * weight
    return inv * (gw - n * (gw * n).mean(-1, keepdim=True)), (g * n).sum((0, 1))


def _quantised(x):
    """[..., blocks, 32] as the nearest e2m1 values (ties to the even code) and the exponent of each block."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m <= 0.75, e - 3, e - 2).clamp(min=-126)     # 6 = 0.75 * 2^3
    v = torch.ldexp(x, -e[..., None])
    size = v.abs()
    step = torch.where(size < 2, 0.5, torch.where(size < 4, 1.0, 2.0))
    return torch.round(v / step) * step, e


def _packed(values):
    """e2m1 values as bytes, the even channel in the low half."""
    size = values.abs()
    code = torch.where(size < 2, size * 2, torch.where(size < 4, size + 2, size / 2 + 4)).to(torch.uint8)
    code = code | (torch.signbit(values).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _rows(codes, scale, table, at):
    """The values that a cache stands for at positions `at` of sequences, [..., heads, d] in fp32: table [..., pages]."""
    P = codes.shape[2]
    page, off = torch.gather(table.long(), -1, (at // P).long()).clamp(min=0), (at % P).long()
    e = scale[page, :, :, off].int()
    byte = codes[page, :, off]
    byte = torch.stack((byte & 15, byte >> 4), -1).flatten(-2)
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    value = torch.cat((value, -value))[byte.int()]
    return torch.ldexp(value.unflatten(-1, (-1, BLOCK)), (e - 127)[..., None]).flatten(-2)


def _append(s):
    case = s["case"]
    cu, lengths, hkv, d, io = s["cu"], s["lengths"], case["hkv"], case["d"], T[case["io"]]
    k_codes, k_scale, v_codes, v_scale = s["cache"]
    n, P = s["k_new"].shape[0], case["page"]
    token = torch.arange(n, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(cu, token, right=True) - 1
    at = lengths[seq] - cu[seq + 1] + token
    cos, sin = _cos_sin(s, at[None].expand(case["axes"], n) if s["positions"] is None else s["positions"])
    # values next to a border between two codes: 64 bits
    k = _rotated(_normed(s["k_new"].double(), s["k_weight"].double()), cos, sin, case)
    page, off = s["table"][seq, at // P].long(), (at % P).long()
    k_value, k_e = _quantised(k.unflatten(-1, (-1, BLOCK)))
    v_value, v_e = _quantised(s["v_new"].float().unflatten(-1, (-1, BLOCK)))
    k_codes[page, :, off], v_codes[page, :, off] = _packed(k_value.flatten(-2)), _packed(v_value.flatten(-2))
    k_scale[page, :, :, off], v_scale[page, :, :, off] = (k_e + 127).to(torch.uint8), (v_e + 127).to(torch.uint8)
    table = s["table"][seq]
    return (_rows(k_codes, k_scale, table, at[:, None])[:, 0].to(io), _rows(v_codes, v_scale, table, at[:, None])[:, 0].to(io))


def _attend(s):
    case = s["case"]
    cu, lengths, hkv, d = s["cu"].long(), s["lengths"].long(), case["hkv"], case["d"]
    k_codes, k_scale, v_codes, v_scale = s["cache"]
    N, Q, L = len(lengths), s["max_q"], s["table"].shape[1] * case["page"]
    at = torch.arange(L, device="cuda").expand(N, L)
    # queries with a place for each of the longest chunk's tokens
    i = torch.arange(Q, device="cuda")
    have = i < (cu[1:] - cu[:-1])[:, None]
    row = torch.where(have, cu[:-1, None] + i, 0)
    q = s["q"].float()[row].view(N, Q, hkv, -1, d).permute(0, 2, 3, 1, 4).flatten(2, 3)   # [N, hkv, group * Q, d]
    last = lengths[:, None] - (cu[1:] - cu[:-1])[:, None] + i                              # what token i sees
    k = _rows(k_codes, k_scale, s["table"], at).permute(0, 2, 3, 1)
    w = torch.matmul(q, k) * d ** -0.5
    del k
    hidden = (at[:, None] > last[..., None])[:, None, None]                                # [N, 1, 1, Q, L]
    w = w.view(N, hkv, -1, Q, L).masked_fill(hidden, -torch.inf)
    w = torch.exp(w - w.amax(-1, keepdim=True)).view(N, hkv, -1, L)
    v = _rows(v_codes, v_scale, s["table"], at).permute(0, 2, 1, 3)
    o = torch.matmul(w, v) / w.sum(-1, keepdim=True)
    return o.view(N, hkv, -1, Q, d).permute(0, 3, 1, 2, 4).flatten(2, 3)[have].to(s["q"].dtype)


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import gated_delta_rule_03_amd as kda
        cfg = s["cfg"]
        if op == "rope":
            return kda.kda_qk_norm_rope(cfg, s["rope"], s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], EPS)
        if op == "rope_bwd":
            return kda.kda_qk_norm_rope_backward(cfg, s["rope"], s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"],
                                                 s["dq_out"], s["dk_out"], EPS)
        if op == "append":
            kda.kda_append_kv(cfg, s["kv"], s["cu"], s["table"], s["lengths"], s["k_new"], s["v_new"], s["k_weight"], EPS,
                              rope=s["rope"], positions=s["positions"])
            return kda.kda_read_kv(cfg, s["kv"], s["cu"], s["table"], s["lengths"], s["k_new"].shape[0])
        return kda.kda_paged_attention(cfg, s["kv"], s["q"], s["cu"], s["table"], s["lengths"], case["d"] ** -0.5, max_q=s["max_q"])
    if op == "append":
        return _append(s)
    if op == "attend":
        return _attend(s)
    cos, sin = (t.float() for t in _cos_sin(s, s["positions"]))
    if op == "rope":
        return tuple(_rotated(_normed(x.float(), w), cos, sin, case).to(x.dtype)
                     for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])))
    dq, dqw = _norm_rope_bwd(s["q"], s["q_weight"], s["dq_out"], cos, sin, case)
    dk, dkw = _norm_rope_bwd(s["k"], s["k_weight"], s["dk_out"], cos, sin, case)
    return dq, dk, dqw, dkw


def work(case):
    op, e, d, hq, hkv = case["op"], SIZE[case["io"]], case["d"], case["hq"], case["hkv"]
    if op in ("rope", "rope_bwd"):
        values = case["n"] * (hq + hkv) * d
        small = 4 * case["n"] * case["axes"] + 8 * d
        if op == "rope":
            return {"bytes": values * 2 * e + small, "flops": 10 * values}
        return {"bytes": values * (2 * e + 4) + small + 8 * d, "flops": 20 * values}
    lens = _lengths(case)
    new = sum(q for q, _ in lens)
    held = 17 * d // 32 * hkv * 2    # bytes of a token's key and value
    if op == "append":
        return {"bytes": new * (4 * e * hkv * d + 2 * held), "flops": 30 * new * hkv * d}
    seen = sum(q * n - q * (q - 1) // 2 for q, n in lens)
    return {"bytes": sum(n for _, n in lens) * held + 2 * new * hq * d * e, "flops": 4 * seen * hq * d}


# ---- from the definitions, in 64 bits --------------------------------------

def _turned(x, angle, case):
    """Pairs as complex numbers times e^(i angle)."""
    rot, half = case["rot"], case["rot"] // 2
    first = torch.arange(half, device=x.device) * (2 if case["inter"] else 1)
    second = first + (1 if case["inter"] else half)
    z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(angle), angle)[:, None, :]
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    assert 2 * half == rot
    return y


def _angle(s, positions):
    return torch.stack([positions[a].double() * f for a, f in zip(s["axis"].tolist(), s["inv_freq"].double())], -1)


def _nearest(x):
    """The values that blocks of 32 are held as: the nearest of the 15, between two the one with the even code."""
    x = x.unflatten(-1, (-1, BLOCK))
    most = x.abs().max(-1, keepdim=True).values
    scale = torch.full_like(most, 2.0 ** -126)
    for e in range(-125, 126):
        scale = torch.where(most > 6 * scale, torch.full_like(most, 2.0 ** e), scale)
    sizes = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    v = x.abs() / scale
    got = torch.zeros_like(v)
    for code in range(1, 8):
        middle = (sizes[code - 1] + sizes[code]) / 2
        up = (v > middle) if code % 2 else (v >= middle)    # a tie goes up to an even code only
        got = torch.where(up, torch.full_like(v, sizes[code]), got)
    return (got * scale * torch.sign(x)).flatten(-2)


def _held(codes, scale, pages, n):
    """The first n rows of a sequence, [heads, n, d]."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=codes.device)
    c = codes[pages].transpose(0, 1).flatten(1, 2)[:, :n].long()                            # [heads, n, d / 2]
    x = torch.empty((*c.shape[:2], c.shape[2] * 2), dtype=torch.float64, device=codes.device)
    x[..., 0::2], x[..., 1::2] = table[c % 16], table[c // 16]
    e = scale[pages].permute(1, 0, 3, 2).flatten(1, 2)[:, :n].double()                      # [heads, n, d / 32]
    return x * torch.exp2(e - 127).repeat_interleave(BLOCK, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op, d, hkv = case["op"], case["d"], case["hkv"]
    if op == "attend":
        cu, lens = s["cu"].tolist(), s["lengths"].tolist()
        o = torch.zeros((cu[-1], case["hq"], d), dtype=torch.float64, device="cuda")
        for i, n in enumerate(lens):
            pages = s["table"][i, :(n + case["page"] - 1) // case["page"]].long()
            k, v = _held(*s["cache"][:2], pages, n), _held(*s["cache"][2:], pages, n)
            q = s["q"][cu[i]:cu[i + 1]].double()
            future = torch.arange(n, device="cuda") > n - len(q) + torch.arange(len(q), device="cuda")[:, None]
            for h in range(case["hq"]):
                g = h * hkv // case["hq"]
                a = (q[:, h] @ k[g].T.contiguous()) / d ** 0.5
                a[future] = -torch.inf
                o[cu[i]:cu[i + 1], h] = torch.softmax(a, -1) @ v[g]
        return o

    def normed(x, w):
        x = x.double()
        return x / torch.sqrt(torch.sum(x * x, -1, keepdim=True) / d + EPS) * w.double()

    if op == "append":
        at = torch.cat([torch.arange(n - q, n, device="cuda") for q, n in _lengths(case)])
        pos = at.expand(case["axes"], -1) if s["positions"] is None else s["positions"]
        k = _turned(normed(s["k_new"], s["k_weight"]), _angle(s, pos), case)
        return _nearest(k), _nearest(s["v_new"].double())
    angle = _angle(s, s["positions"])
    if op == "rope":
        return tuple(_turned(normed(s[x], s[x + "_weight"]), angle, case) for x in "qk")
    dx, dw = [], []
    for x in "qk":
        v, g = s[x].double(), _turned(s["d" + x + "_out"].double(), -angle, case)
        r2 = torch.sum(v * v, -1, keepdim=True) / d + EPS
        gw = g * s[x + "_weight"].double()
        dx.append(gw * r2 ** -0.5 - v * torch.sum(gw * v, -1, keepdim=True) * r2 ** -1.5 / d)
        dw.append(torch.sum(g * v * r2 ** -0.5, (0, 1)))
    return (*dx, *dw)
