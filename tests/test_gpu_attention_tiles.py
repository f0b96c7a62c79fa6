"""Attention of chunks at the sizes that the kernel of 256-row tiles takes (bf16; rows of a key head above 128, 192 at 128
channels, and 65536 of all heads, at 256 channels 8192): tiles, parts, missing pages, NaN, scales, graphs, what lies far in a cache."""
import pytest
import torch

from tests import test_gpu_attention_chunks as chunks
from tests.test_gpu_attention import check_attention
from tests.test_gpu_kv_cache import Batch
from tests.test_gpu_layer import BF, F32, Rand
from tests.test_gpu_rope import kda, make_cfg, make_rope  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,heads", [(64, 260), (128, 260), (256, 40)])
@pytest.mark.parametrize("rows", [255, 256, 257, 300, 513])
def test_rows_around_a_tile(kda, d, heads, rows):  # noqa: F811
    chunks.attend(kda, Batch(kda, [(rows, rows + 190)], heads, d, 64), 1, heads=(0, 5, heads - 1), max_q=rows)
    chunks.attend(kda, Batch(kda, [(rows, rows)], heads, d, 256), 1, heads=(0, 16), max_q=0)


@pytest.mark.parametrize("d,tokens", [(64, 230), (128, 230), (256, 140)])
def test_more_tiles_than_units_of_the_card(kda, d, tokens):  # noqa: F811
    """So many that none is split, of ragged lengths, empty ones among them."""
    seqs = [(tokens - i % 3, tokens + i) if i % 5 else (i % 2, 0) for i in range(50)]
    chunks.attend(kda, Batch(kda, seqs, 8, d, 64), 1, every=8, heads=(0, 3, 7), max_q=tokens)


@pytest.mark.parametrize("d,heads,group", [(64, 64, 4), (128, 32, 8), (256, 4, 16)])
def test_a_table_with_room_for_more(kda, d, heads, group):  # noqa: F811
    """The split goes by the table's room; sequences far shorter than it have fewer parts, or one; rows that see nothing."""
    seqs = [(90, 1500), (70, 71), (33, 0), (80, 50), (20, 300)]
    chunks.attend(kda, Batch(kda, seqs, heads, d, 32, extra=600), group, heads=(0, heads - 1), max_q=90)


@pytest.mark.parametrize("d,heads", [(64, 16), (128, 16), (256, 2)])
def test_pages_and_what_is_not_seen(kda, d, heads):  # noqa: F811
    chunks.test_pages_that_are_not_held(kda, d, heads)
    chunks.test_what_is_not_seen_has_no_effect(kda, d, heads)


@pytest.mark.parametrize("d,heads", [(64, 32), (128, 32), (256, 4)])
def test_missing_pages_beside_held_ones(kda, d, heads):  # noqa: F811
    chunks.test_missing_pages_beside_held_ones(kda, d, heads)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 0.5])
@pytest.mark.parametrize("d,heads", [(64, 128), (128, 128), (256, 16)])
def test_scales(kda, d, heads, scale):  # noqa: F811
    chunks.attend(kda, Batch(kda, [(100, 400)], heads, d, 64), 8, scale=scale, heads=(0, heads - 1))


def test_the_most_sequences(kda):  # noqa: F811
    N = 4096
    seqs = [(1, 40) if i % 500 == 0 else (0, 9 * (i % 2)) for i in range(N)]
    seqs[77] = (130, 200)
    chunks.attend(kda, Batch(kda, seqs, 2, 256, 32), 32, max_q=130)


@pytest.mark.parametrize("d,heads", [(64, 16), (128, 16), (256, 4)])
def test_nan_in_queries(kda, d, heads):  # noqa: F811
    """They make their own row NaN, and no other."""
    tokens, group = 150, 32
    b = Batch(kda, [(tokens, tokens + 50)], heads, d, 32)
    b.fill()
    q = Rand(7)(b.n, heads * group, d, dtype=BF)
    cfg = make_cfg(kda, heads * group, d)
    o = kda.kda_paged_attention(cfg, b.cache, q, *b.where, max_q=tokens)
    q[0, 1, 5], q[tokens - 1, 2, d - 3] = float("nan"), float("inf")
    lse = torch.zeros(b.n, heads * group, device="cuda")
    p = kda.kda_paged_attention(cfg, b.cache, q, *b.where, max_q=tokens, lse=lse)
    bad = torch.zeros(b.n, heads * group, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[tokens - 1, 2] = True
    assert p[bad].isnan().all() and lse[bad].isnan().all()
    assert torch.equal(p[~bad], o[~bad]) and lse[~bad].isfinite().all()


def test_streams_and_graphs(kda):  # noqa: F811
    """The same bits on another stream and with rows behind the last sequence; two captured calls that share a workspace,
    one of them split and one not, replayed in turn while the lengths grow, with eager calls in between."""
    d, heads, group = 128, 16, 24
    b = Batch(kda, [(80, 700), (100, 2000)], heads, d, 64, extra=200)
    b.fill()
    cfg = make_cfg(kda, heads * group, d)
    q = Rand(5)(b.n + 7, heads * group, d, dtype=BF)
    o = torch.full_like(q, 7.0)
    kda.kda_paged_attention(cfg, b.cache, q, *b.where, max_q=100, o=o)
    assert (o[b.n:] == 7).all()
    chunks.Some(b, 2, (0,)).check(o, None, q, d ** -0.5, 100)
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
    """Pages beyond 32 bits of bytes: the same results as in a small cache."""
    d, heads, group, page, tokens = 256, 2, 32, 64, 150
    b = Batch(kda, [(tokens, 300), (1, 130)], heads, d, page)
    pages = (1 << 32) // (heads * page * d // 2) + 5000
    far = kda.KvCache.empty(pages, heads, d, page)
    table = torch.where(b.table >= 0, pages - 1 - 500 * b.table, b.table)
    cfg, r, w, rope = make_cfg(kda, group * heads, d), Rand(6), Rand(8).weight(d), make_rope(kda, 64)
    whole = torch.tensor([0, 300, 430], dtype=torch.int32, device="cuda")
    k, v = r(430, heads, d, dtype=BF), r(430, heads, d, dtype=BF)
    for cache, t in ((b.cache, b.table), (far, table)):
        kda.kda_append_kv(cfg, cache, whole, t, b.lengths, k, v, w, rope=rope)
    q = r(b.n, group * heads, d, dtype=BF)
    o = kda.kda_paged_attention(cfg, far, q, b.cu, table, b.lengths, max_q=tokens)
    assert torch.equal(kda.kda_paged_attention(cfg, b.cache, q, *b.where, max_q=tokens), o)
    check_attention(o, None, b, q, d ** -0.5)


@pytest.mark.parametrize("io,out", [(F32, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("d,heads", [(64, 260), (128, 260), (256, 40)])
def test_the_other_types_at_these_sizes(kda, d, heads, io, out):  # noqa: F811
    chunks.attend(kda, Batch(kda, [(257, 300)], heads, d, 64), 1, io, out, heads=(0, heads - 1), max_q=257)


@pytest.mark.parametrize("d,heads,group", [(64, 8, 32), (128, 8, 32), (256, 2, 16)])
def test_single_tokens_where_max_q_is_not_known(kda, d, heads, group):  # noqa: F811
    """The kernel of single tokens takes them: the same bits."""
    b = Batch(kda, [(1, 30 + i) for i in range(260)], heads, d, 64)
    b.fill()
    q = Rand(5)(b.n, heads * group, d, dtype=BF)
    cfg = make_cfg(kda, heads * group, d)
    o = kda.kda_paged_attention(cfg, b.cache, q, *b.where, max_q=1)
    assert torch.equal(kda.kda_paged_attention(cfg, b.cache, q, *b.where), o)
    assert torch.equal(kda.kda_paged_attention(cfg, b.cache, q, None, b.table, b.lengths), o)
