"""Attention over the paged 4-bit cache against its definition in 64 bits."""
import pytest
import torch

from tests import attention_reference as ref
from tests.layer_reference import check
from tests.test_gpu_kv_cache import Batch
from tests.test_gpu_layer import BF, F32, Rand, guarded
from tests.test_gpu_rope import EPS, expected, kda, make_cfg, make_rope  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def check_attention(o, lse, b, q, scale, max_q=0, note=""):
    """Every sequence against 64 bits; max_q as the call had it (0: not known)."""
    cu, total = b.cu.tolist(), [0.0, 0.0, 0]
    rows = max_q * q.shape[1] // b.heads
    for i, (t, n) in enumerate(b.seqs):
        if t == 0:
            continue
        k, v = b.held(i)
        x = q[cu[i]:cu[i + 1]].double().cpu()
        e, el, m, top = ref.attention(x, k, v, n, scale)
        rel, rl = ref.attention_rel(q.shape[2], n, top, q.dtype, o.dtype, rows)
        got = o[cu[i]:cu[i + 1]].cpu()
        check(got, e, m, rel, f"{note} sequence {i}")
        total = [total[0] + (got.double() - e).square().sum(), total[1] + e.square().sum(), total[2] + e.numel()]
        if lse is not None:
            g = lse[cu[i]:cu[i + 1]].double().cpu()
            none = el.isinf()
            assert torch.equal(g.isinf(), none) and (g[none] < 0).all()
            off = (g - el)[~none].abs()
            lim = (rl + 4 * 2.0 ** -24 * el.abs().nan_to_num(posinf=0))[~none]
            assert (off <= lim).all(), f"{note} lse of sequence {i}: {float((off / lim).max())} of the bound"
    if o.dtype == torch.bfloat16 and total[2] >= 1000:
        # in the 2-norm: the output's rounding, and the weights' where they are one bf16 value, which moves an output by
        # as much where the values are independent of each other, as here; and what else there is by a tenth of that
        assert (total[0] / total[1]) ** 0.5 <= (2.0 ** 0.5 + 0.1) * 2.0 ** -8 / 3 ** 0.5, note


SEQS = {
    "one": [(1, 1)],
    "edges": [(1, n) for n in (1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 0, 500)],
    "drafts": [(4, 4), (4, 37), (4, 300), (4, 2), (4, 0), (0, 50), (4, 1025)],
    "ragged": [(3, 700), (1, 90), (17, 17), (9, 130), (2, 33)],
    "chunk": [(70, 200), (33, 33)],
    "long": [(1, 9000), (2, 20001)],
}


@pytest.mark.parametrize("seqs", list(SEQS))
@pytest.mark.parametrize("d,heads,group,page", [(64, 3, 2, 32), (128, 2, 4, 64), (256, 2, 8, 128), (128, 1, 16, 256), (64, 1, 1, 64),
                                                (256, 1, 3, 32), (128, 1, 20, 32)])
@pytest.mark.parametrize("io,out", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
def test_attention(kda, seqs, d, heads, group, page, io, out):  # noqa: F811
    b = Batch(kda, SEQS[seqs], heads, d, page, seed=d + group, extra=2)
    b.fill()
    r = Rand(3)
    q = r(b.n, heads * group, d, dtype=io, scale=2)
    o, ok = guarded(q.shape, out)
    lse, ok2 = guarded(q.shape[:2], F32)
    scale = d ** -0.5
    max_q = max(t for t, _ in b.seqs)
    kda.kda_paged_attention(make_cfg(kda, heads * group, d, io, out), b.cache, q, *b.where, max_q=max_q, o=o, lse=lse)
    assert ok() and ok2()
    check_attention(o, lse, b, q, scale, max_q)
    # the largest count not known: another kernel may take it
    o2 = kda.kda_paged_attention(make_cfg(kda, heads * group, d, io, out), b.cache, q, *b.where, scale)
    check_attention(o2, None, b, q, scale, note="max_q 0")


@pytest.mark.parametrize("io,out", [(BF, BF), (F32, F32)])
@pytest.mark.parametrize("drafts", [1, 3, 40])
def test_what_is_not_seen_has_no_effect(kda, io, out, drafts):  # noqa: F811
    """Bytes behind the length, in other pages, and in later drafts' positions: NaN scales in all of them."""
    d, heads, group = 128, 2, 4
    b = Batch(kda, [(drafts, 150), (drafts, 64)], heads, d, 64, seed=2)
    b.fill()
    q = Rand(7)(b.n, heads * group, d, dtype=io)
    cfg = make_cfg(kda, heads * group, d, io, out)
    o = kda.kda_paged_attention(cfg, b.cache, q, *b.where, max_q=drafts)
    mine = torch.zeros(b.cache.k.shape[0], 64, dtype=torch.bool)
    for i, (_, n) in enumerate(b.seqs):
        for p in range(n):
            mine[int(b.table[i, p // 64]), p % 64] = True
    other = (~mine)[:, None, None].cuda()
    for s in (b.cache.k_scale, b.cache.v_scale):
        s.masked_fill_(other.expand_as(s), 255)
    assert torch.equal(kda.kda_paged_attention(cfg, b.cache, q, *b.where, max_q=drafts), o)
    # a NaN in the last token's own key or value reaches the last token alone
    for s in (b.cache.k_scale, b.cache.v_scale):
        keep = s.clone()
        s[int(b.table[0, 149 // 64]), 1, 2, 149 % 64] = 255
        p = kda.kda_paged_attention(cfg, b.cache, q, *b.where, max_q=drafts)
        last = drafts - 1
        assert torch.equal(p[:last], o[:last]) and torch.equal(p[drafts:], o[drafts:])
        assert torch.equal(p[last, :group], o[last, :group])
        bad = p[last, group:].isnan()
        assert bad.all() if s is b.cache.k_scale else (bad[:, 64:96].all() and not bad[:, :64].any() and not bad[:, 96:].any())
        s.copy_(keep)


def test_nan_inside_reaches_every_row_that_sees_it(kda):  # noqa: F811
    d = 64
    b = Batch(kda, [(1, 300)], 1, d, 32)
    b.fill()
    cfg = make_cfg(kda, 2, d, BF, F32)
    q = Rand(7)(1, 2, d, dtype=BF)
    b.cache.v_scale[int(b.table[0, 2]), 0, 1, 5] = 255
    o = kda.kda_paged_attention(cfg, b.cache, q, *b.where)
    assert o[..., 32:].isnan().all() and not o[..., :32].isnan().any()
    b.cache.k_scale[int(b.table[0, 3]), 0, 0, 5] = 255
    assert kda.kda_paged_attention(cfg, b.cache, q, *b.where).isnan().all()


@pytest.mark.parametrize("io,out", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("tokens", [1, 9, 90])
def test_queries_with_nan_and_infinity(kda, io, out, tokens):  # noqa: F811
    """They make their own row NaN, and no other; so does a NaN in the only key that a row sees."""
    d, group = 128, 2
    b = Batch(kda, [(tokens, tokens + 50), (1, 1)], 2, d, 32)
    b.fill()
    q = Rand(7)(b.n, 2 * group, d, dtype=io)
    cfg = make_cfg(kda, 2 * group, d, io, out)
    o = kda.kda_paged_attention(cfg, b.cache, q, *b.where, max_q=tokens)
    q[0, 1, 5], q[tokens - 1, 2, 100] = float("nan"), float("inf")
    b.cache.k_scale[int(b.table[1, 0]), 1, 3, 0] = 255
    lse = torch.zeros(b.n, 2 * group, device="cuda")
    p = kda.kda_paged_attention(cfg, b.cache, q, *b.where, max_q=tokens, lse=lse)
    bad = torch.zeros(b.n, 2 * group, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[tokens - 1, 2] = bad[tokens, group:] = True
    assert p[bad].isnan().all() and lse[bad].isnan().all()
    assert torch.equal(p[~bad], o[~bad]) and lse[~bad].isfinite().all()


def test_far_scores(kda):  # noqa: F811
    """Scores of hundreds that rise and fall along the positions: the running maximum moves many times."""
    d = 64
    b = Batch(kda, [(1, 1500), (3, 1500)], 1, d, 32)
    b.fill()
    ramp = (b.cache.k_scale.float().mean().item(), 0)
    for i in range(2):
        for p in range(0, 1500):
            pg = int(b.table[i, p // 32])
            up = (p // 100) % 8
            b.cache.k_scale[pg, :, :, p % 32] = 118 + up
    del ramp
    for io, out in ((BF, BF), (F32, F32)):
        q = Rand(3)(b.n, 2, d, dtype=io, scale=60)
        lse = torch.empty(b.n, 2, device="cuda")
        o = kda.kda_paged_attention(make_cfg(kda, 2, d, io, out), b.cache, q, *b.where, 1.0, lse=lse)
        check_attention(o, lse, b, q, 1.0)
    # a negative scale, and a scale of 0 (the mean of the values)
    for scale in (-0.5, 0.0):
        o = kda.kda_paged_attention(make_cfg(kda, 2, d, F32, F32), b.cache, q, *b.where, scale)
        check_attention(o, None, b, q, scale)


def test_pages_that_are_not_held(kda):  # noqa: F811
    """A page number out of range leaves its positions out; a length beyond the table counts to its end; a sequence whose
    pages are all missing gives zeros."""
    d = 128
    b = Batch(kda, [(1, 200), (2, 128), (1, 100)], 2, d, 64)
    b.fill()
    q = Rand(3)(b.n, 4, d)
    cfg = make_cfg(kda, 4, d, F32, F32)
    k, v = b.held(0)
    b.table[0, 1] = 10**9
    b.table[2] = -1
    b.lengths[1] = 2**31 - 1
    lse = torch.zeros(b.n, 4, device="cuda")
    o = kda.kda_paged_attention(cfg, b.cache, q, *b.where, lse=lse)
    keep = torch.tensor([p for p in range(200) if p // 64 != 1])
    e, _, m, top = ref.attention(q[:1].double().cpu(), k[:, keep], v[:, keep], len(keep), d ** -0.5)
    check(o[:1].cpu(), e, m, ref.attention_rel(d, 200, top, F32, F32, 0)[0])
    assert (o[3] == 0).all() and (lse[3] == -torch.inf).all()
    # the table holds 4 pages: positions 128 .. 255 of sequence 1 are pages of -1; both its tokens see all of them
    k, v = b.held(1)
    b.seqs[1] = (2, 128)
    for j in range(2):
        e, _, m, top = ref.attention(q[1 + j:2 + j].double().cpu(), k, v, 128, d ** -0.5)
        check(o[1 + j:2 + j].cpu(), e, m, ref.attention_rel(d, 128, top, F32, F32, 0)[0])


def test_padded_batch_streams_and_graph(kda):  # noqa: F811
    """Rows behind the last sequence stay as they were; another stream; two captured steps that share a workspace run one
    after the other, with lengths that grow on the device between replays."""
    d, heads, group = 128, 2, 4
    b = Batch(kda, [(1, n) for n in (300, 1, 700, 64)], heads, d, 64)
    b.fill()
    cfg = make_cfg(kda, heads * group, d)
    r = Rand(5)
    q = r(9, heads * group, d, dtype=BF)
    o = torch.full_like(q, 7.0)
    kda.kda_paged_attention(cfg, b.cache, q, *b.where, max_q=1, o=o)   # (one kernel for all of these: the same bits)
    assert (o[4:] == 7).all()
    check_attention(o, None, b, q, d ** -0.5, 1)
    assert torch.equal(kda.kda_paged_attention(cfg, b.cache, q[:4], None, b.table, b.lengths), o[:4])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s = kda.kda_paged_attention(cfg, b.cache, q[:4], *b.where, max_q=1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(s, o[:4])
    ws = torch.empty(kda.kda_paged_attention_workspace_bytes(cfg, heads, 4, 4, 1), dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(kda.kda_paged_attention(cfg, b.cache, q[:4], None, b.table, b.lengths, workspace=ws))
        graphs.append(g)
    full = b.lengths.clone()
    for i in range(4):
        b.lengths.copy_((full - 3 + i).clamp(min=0))
        e = kda.kda_paged_attention(cfg, b.cache, q[:4], None, b.table, b.lengths)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, e) for x in outs), i


def test_many_sequences(kda):  # noqa: F811
    """The most sequences of a call, most of them empty."""
    d, N = 64, 4096
    b = Batch(kda, [(1, 40) if i % 500 == 0 else (1, 0) if i % 2 else (0, 0) for i in range(N)], 1, d, 32)
    b.fill()
    q = Rand(5)(b.n, 1, d, dtype=BF)
    o = kda.kda_paged_attention(make_cfg(kda, 1, d), b.cache, q, *b.where, max_q=1)
    check_attention(o, None, b, q, d ** -0.5)


def test_a_step_of_a_full_attention_layer(kda):  # noqa: F811
    """Norm and rotation, append and attention together, as a layer calls them: a prompt in two chunks, then drafts."""
    hq, heads, d, page = 8, 2, 128, 64
    r = Rand(21)
    cfg, rope, wq, wk = make_cfg(kda, hq, d), make_rope(kda, 32), r.weight(d), r.weight(d)
    b = Batch(kda, [(0, 400), (0, 150)], heads, d, page)
    sizes = [(0, 0)] * 2
    for new in ((100, 37), (180, 64), (1, 1), (4, 4), (1, 1)):
        sizes = [(t, n + t) for t, (_, n) in zip(new, sizes)]
        b.seqs = sizes
        b.n = sum(new)
        b.cu = torch.tensor([0, new[0], b.n], dtype=torch.int32, device="cuda")
        b.lengths = torch.tensor([n for _, n in sizes], dtype=torch.int32, device="cuda")
        qkv = r(b.n, (hq + 2 * heads) * d, dtype=BF, scale=2)
        q, k, v = (t.unflatten(1, (-1, d)) for t in qkv.split([hq * d, heads * d, heads * d], 1))
        pos = torch.cat([torch.arange(n - t, n) for t, n in sizes]).int()
        x, _ = kda.kda_qk_norm_rope(cfg, rope, q, None, wq, None, pos.cuda())
        kda.kda_append_kv(cfg, b.cache, *b.where, k, v, wk, rope=rope)
        o = kda.kda_paged_attention(cfg, b.cache, x, *b.where, max_q=max(new))
        check(x.cpu(), *expected(q.contiguous(), wq, rope, pos[None]), ref.ROPE_REL)
        check_attention(o, None, b, x, d ** -0.5)
