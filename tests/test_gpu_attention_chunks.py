"""Attention of chunks of new tokens, at the sizes where the work is split in another way, and what lies far in a cache."""
import pytest
import torch

from tests import attention_reference as ref
from tests.layer_reference import check
from tests.test_gpu_attention import check_attention
from tests.test_gpu_kv_cache import Batch
from tests.test_gpu_layer import BF, F32, Rand, guarded
from tests.test_gpu_rope import kda, make_cfg, make_rope  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


class Some:
    """Some sequences and key heads of a batch, for a check."""

    def __init__(self, b, every=1, heads=None):
        self.b, self.cu = b, b.cu
        self.seqs = [(t, n) if i % every == 0 else (0, n) for i, (t, n) in enumerate(b.seqs)]
        self.of = range(b.heads) if heads is None else [h for h in heads if h < b.heads]
        self.heads = len(self.of)

    def held(self, i):
        return [x[list(self.of)] for x in self.b.held(i)]

    def check(self, o, lse, q, scale, max_q=0):
        group = q.shape[1] // self.b.heads
        rows = [h * group + x for h in self.of for x in range(group)]
        check_attention(o[:, rows], None if lse is None else lse[:, rows], self, q[:, rows], scale, max_q)


def attend(kda, b, group, io=BF, out=BF, scale=None, every=1, heads=None, **args):  # noqa: F811
    """The call, every'th sequence and the heads given of it checked."""
    b.fill()
    q = Rand(3)(b.n, b.heads * group, b.d, dtype=io, scale=2)
    o, ok = guarded(q.shape, out)
    lse, ok2 = guarded(q.shape[:2], F32)
    cfg = make_cfg(kda, b.heads * group, b.d, io, out)
    kda.kda_paged_attention(cfg, b.cache, q, *b.where, scale, o=o, lse=lse, **args)
    assert ok() and ok2()
    Some(b, every, heads).check(o, lse, q, b.d ** -0.5 if scale is None else scale, args.get("max_q", 0))


@pytest.mark.parametrize("d,tokens", [(64, 100), (128, 170), (256, 140)])
@pytest.mark.parametrize("io", [BF, F32])
def test_more_tiles_than_units_of_the_card(kda, d, tokens, io):  # noqa: F811
    """So many that none is split, of ragged lengths, empty ones among them."""
    seqs = [(tokens - i % 3, tokens + i) if i % 5 else (i % 2, 0) for i in range(40)]
    attend(kda, Batch(kda, seqs, 8, d, 64), 1, io, every=6, heads=(0, 3, 7), max_q=tokens)


@pytest.mark.parametrize("d,heads,group", [(64, 1, 4), (128, 5, 24), (256, 1, 16)])
def test_a_table_with_room_for_more(kda, d, heads, group):  # noqa: F811
    """The split goes by the table's room; sequences far shorter than it have fewer parts, or one; rows that see nothing."""
    seqs = [(90, 1500), (70, 71), (33, 0), (80, 50), (20, 300)]
    attend(kda, Batch(kda, seqs, heads, d, 32, extra=600), group, heads=(0, 4), max_q=90)


@pytest.mark.parametrize("d,heads", [(64, 1), (128, 129), (256, 17)])
@pytest.mark.parametrize("rows", [255, 256, 257, 300, 513])
def test_rows_around_a_tile(kda, d, heads, rows):  # noqa: F811
    attend(kda, Batch(kda, [(rows, rows + 190)], heads, d, 64), 1, heads=(0, 5, 128), max_q=rows)
    attend(kda, Batch(kda, [(rows, rows)], heads, d, 256), 1, heads=(0, 16), max_q=0)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 0.5])
def test_scales(kda, scale):  # noqa: F811
    attend(kda, Batch(kda, [(90, 400)], 128, 128, 64), 4, scale=scale, heads=(0, 127))
    attend(kda, Batch(kda, [(90, 400)], 2, 64, 64), 4, scale=scale)


@pytest.mark.parametrize("d,heads", [(64, 2), (128, 5), (256, 2)])
def test_pages_that_are_not_held(kda, d, heads):  # noqa: F811
    """As for single tokens: their positions are left out, a length beyond the table counts to its end."""
    tokens = 160
    b = Batch(kda, [(tokens, 700), (tokens, 700), (tokens, 512)], heads, d, 64)
    b.fill()
    q = Rand(3)(b.n, 16 * heads, d, dtype=BF)
    k, v = b.held(0)
    b.table[0, 2], b.table[0, 5] = -7, 2**31 - 1
    b.table[1] = -1
    b.lengths[2] = 2**31 - 1
    o, ok = guarded(q.shape, BF)
    lse = torch.zeros(b.n, 16 * heads, device="cuda")
    kda.kda_paged_attention(make_cfg(kda, 16 * heads, d), b.cache, q, *b.where, o=o, lse=lse, max_q=tokens)
    assert ok()
    assert (o[tokens:2 * tokens] == 0).all() and (lse[tokens:2 * tokens] == -torch.inf).all()
    for j in (0, 57, tokens - 1):
        sees = 700 - tokens + j + 1
        keep = torch.tensor([p for p in range(sees) if p // 64 not in (2, 5)])
        e, _, m, top = ref.attention(q[j:j + 1].double().cpu(), k[:, keep], v[:, keep], len(keep), d ** -0.5)
        check(o[j:j + 1].cpu(), e, m, ref.attention_rel(d, 700, top, BF, BF, 0)[0])
        e, _, m, top = ref.attention(q[2 * tokens + j][None].double().cpu(), *b.held(2), 512, d ** -0.5)
        check(o[2 * tokens + j][None].cpu(), e, m, ref.attention_rel(d, 512, top, BF, BF, 0)[0])


@pytest.mark.parametrize("d,heads", [(64, 2), (128, 8), (256, 2)])
def test_what_is_not_seen_has_no_effect(kda, d, heads):  # noqa: F811
    """NaN behind the lengths, in pages of no one and at later tokens; and one that is seen reaches those that see it."""
    tokens, group = 140, 16
    b = Batch(kda, [(tokens, 450), (tokens, 140)], heads, d, 64, seed=2)
    b.fill()
    q = Rand(7)(b.n, heads * group, d, dtype=BF)
    cfg = make_cfg(kda, heads * group, d)
    run = lambda: kda.kda_paged_attention(cfg, b.cache, q, *b.where, max_q=tokens)
    o = run()
    mine = torch.zeros(b.cache.k.shape[0], 64, dtype=torch.bool)
    for i, (_, n) in enumerate(b.seqs):
        for p in range(n):
            mine[int(b.table[i, p // 64]), p % 64] = True
    other = (~mine)[:, None, None].cuda()
    for s in (b.cache.k_scale, b.cache.v_scale):
        s.masked_fill_(other.expand_as(s), 255)
    assert torch.equal(run(), o)
    for at in (450 - tokens + 33, 449):
        for s in (b.cache.k_scale, b.cache.v_scale):
            keep = s.clone()
            s[int(b.table[0, at // 64]), 1, 1, at % 64] = 255
            p, first = run(), at - (450 - tokens)
            assert torch.equal(p[:first], o[:first]) and torch.equal(p[tokens:], o[tokens:])
            assert torch.equal(p[first:tokens, :group], o[first:tokens, :group])
            assert torch.equal(p[first:tokens, 2 * group:], o[first:tokens, 2 * group:])
            bad = p[first:tokens, group:2 * group].isnan()
            assert bad.all() if s is b.cache.k_scale else (bad[..., 32:64].all() and not bad[..., :32].any()
                                                           and not bad[..., 64:].any())
            s.copy_(keep)


@pytest.mark.parametrize("io,out,max_q", [(BF, BF, 0), (BF, BF, 130), (F32, F32, 0)])
def test_the_most_sequences(kda, io, out, max_q):  # noqa: F811
    d, N = 256, 4096
    seqs = [(1, 40) if i % 500 == 0 else (0, 9 * (i % 2)) for i in range(N)]
    seqs[77] = (130, 200)
    attend(kda, Batch(kda, seqs, 1, d, 32), 32, io, out, max_q=max_q)


def test_max_q_that_was_too_small(kda):  # noqa: F811
    """Only the choice of the kernel goes by it."""
    attend(kda, Batch(kda, [(70, 200), (1, 300), (5, 5)], 2, 128, 64), 2, max_q=1)
    b = Batch(kda, [(250, 300), (250, 400), (250, 250)], 2, 64, 64)
    attend(kda, b, 1, max_q=100)


def test_streams_and_graphs(kda):  # noqa: F811
    """The same bits on another stream and with rows behind the last sequence; two captured calls that share a workspace,
    one of them split and one not, replayed in turn while the lengths grow."""
    d, heads, group = 128, 8, 24
    b = Batch(kda, [(80, 700), (100, 2000)], heads, d, 64, extra=200)
    b.fill()
    cfg = make_cfg(kda, heads * group, d)
    q = Rand(5)(b.n + 7, heads * group, d, dtype=BF)
    o = torch.full_like(q, 7.0)
    kda.kda_paged_attention(cfg, b.cache, q, *b.where, max_q=100, o=o)
    assert (o[b.n:] == 7).all()
    Some(b, 2, (0,)).check(o, None, q, d ** -0.5, 100)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s = kda.kda_paged_attention(cfg, b.cache, q, *b.where, max_q=100, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(s[:b.n], o[:b.n])
    short = b.table[:, :1].contiguous()
    ws = torch.empty(kda.kda_paged_attention_workspace_bytes(cfg, heads, 2, b.n, 100), dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for table in (b.table, short):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(kda.kda_paged_attention(cfg, b.cache, q[:b.n], b.cu, table, b.lengths, max_q=100, workspace=ws))
        graphs.append(g)
    full = b.lengths.clone()
    for i in range(4):
        b.lengths.copy_(full - 600 + 200 * i)
        want = [kda.kda_paged_attention(cfg, b.cache, q[:b.n], b.cu, t, b.lengths, max_q=100) for t in (b.table, short)]
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, want)), i


def test_far_in_a_large_cache(kda):  # noqa: F811
    """Pages beyond 32 bits of bytes: the same codes and results as in a small cache."""
    d, heads, page, tokens = 256, 2, 64, 150
    seqs = [(tokens, 300), (1, 130)]
    b = Batch(kda, seqs, heads, d, page)
    pages = (1 << 32) // (heads * page * d // 2) + 5000
    far = kda.KvCache.empty(pages, heads, d, page)
    table = torch.where(b.table >= 0, pages - 1 - 500 * b.table, b.table)
    cfg = make_cfg(kda, 16 * heads, d)
    r, lengths = Rand(6), b.lengths - torch.tensor([tokens, 1], dtype=torch.int32, device="cuda")
    first = torch.tensor([0, 150, 279], dtype=torch.int32, device="cuda")
    rope, w = make_rope(kda, 64), r.weight(d)
    for cu, n, many in ((first, lengths, 279), (b.cu, b.lengths, b.n)):
        k, v = r(many, heads, d, dtype=BF), r(many, heads, d, dtype=BF)
        for cache, t in ((b.cache, b.table), (far, table)):
            kda.kda_append_kv(cfg, cache, cu, t, n, k, v, w, rope=rope)
    whole = torch.tensor([0, 300, 430], dtype=torch.int32, device="cuda")
    for x, y in zip(kda.kda_read_kv(cfg, b.cache, whole, b.table, b.lengths, 430),
                    kda.kda_read_kv(cfg, far, whole, table, b.lengths, 430)):
        assert torch.equal(x, y) and (x != 0).any()
    q = r(b.n, 16 * heads, d, dtype=BF)
    for c in (cfg, make_cfg(kda, 16 * heads, d, BF, F32)):
        for max_q in (0, 1):
            x = kda.kda_paged_attention(c, b.cache, q, b.cu, b.table, b.lengths, max_q=max_q)
            assert torch.equal(kda.kda_paged_attention(c, far, q, b.cu, table, b.lengths, max_q=max_q), x)
    check_attention(kda.kda_paged_attention(cfg, far, q, b.cu, table, b.lengths), None, b, q, d ** -0.5)


@pytest.mark.parametrize("tokens", [1, 110])
def test_sequences_that_share_pages(kda, tokens):  # noqa: F811
    """A prefix held once, and one page twice in a sequence."""
    b = Batch(kda, [(tokens, 400), (tokens, 333), (tokens, 400)], 2, 64, 32)
    b.fill()
    b.table[1, :7], b.table[2, 5] = b.table[0, :7], b.table[2, 1]
    q = Rand(3)(b.n, 4, 64, dtype=BF)
    o = kda.kda_paged_attention(make_cfg(kda, 4, 64), b.cache, q, *b.where, max_q=tokens)
    check_attention(o, None, b, q, 64 ** -0.5, tokens)


@pytest.mark.parametrize("d,heads", [(64, 2), (128, 16), (256, 2)])
def test_missing_pages_beside_held_ones(kda, d, heads):  # noqa: F811
    """Every third page of 32 positions is missing; NaN in all pages of no one, the first among them, has no effect."""
    tokens = 160
    b = next(b for b in (Batch(kda, [(tokens, 900)], heads, d, 32, seed=s) for s in range(50)) if not (b.table == 0).any())
    b.fill()
    q = Rand(3)(b.n, 16 * heads, d, dtype=BF)
    k, v = b.held(0)
    b.table[0, 1::3] = -1
    others = [p for p in range(b.cache.k.shape[0]) if p not in b.table[0].tolist()]
    assert 0 in others
    b.cache.k_scale[others], b.cache.v_scale[others] = 255, 255
    o, ok = guarded(q.shape, BF)
    kda.kda_paged_attention(make_cfg(kda, 16 * heads, d), b.cache, q, *b.where, o=o, max_q=tokens)
    assert ok()
    for j in (0, 31, tokens - 1):
        keep = torch.tensor([p for p in range(900 - tokens + j + 1) if p // 32 % 3 != 1])
        e, _, m, top = ref.attention(q[j:j + 1].double().cpu(), k[:, keep], v[:, keep], len(keep), d ** -0.5)
        check(o[j:j + 1].cpu(), e, m, ref.attention_rel(d, 900, top, BF, BF, 0)[0])
