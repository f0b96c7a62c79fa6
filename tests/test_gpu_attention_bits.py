"""What attention over the paged cache holds of its inputs: which positions a token sees where a length passes the table,
small channels beside large ones, weights, and the log of their sum."""
import pytest
import torch

from tests import attention_bounds as ref
from tests.layer_reference import check
from tests.test_gpu_kv_cache import Batch
from tests.test_gpu_layer import BF, F32, Rand
from tests.test_gpu_rope import kda, make_cfg  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

# (d, key heads, query heads of each, tokens): rows of a key head of one sequence from one to thousands, so that every
# kernel and every number of row tiles takes some
SHAPES = [(64, 2, 4, 1), (64, 2, 4, 5), (64, 1, 5, 9), (64, 2, 2, 75), (64, 8, 52, 160), (128, 2, 4, 1), (128, 2, 3, 7),
          (128, 8, 52, 160), (256, 2, 8, 1), (256, 2, 4, 6), (256, 2, 16, 130), (256, 4, 16, 130)]
TYPES = [(BF, BF), (F32, BF), (BF, F32), (F32, F32)]


def compare(kda, b, cfg, q, sees, scale, max_q, note=""):  # noqa: F811
    """o and lse of the call against 64 bits; sees: a list of counts for each sequence."""
    lse = torch.empty(q.shape[:2], device="cuda")
    o = kda.kda_paged_attention(cfg, b.cache, q, *b.where, scale, max_q=max_q, lse=lse)
    heads = sorted({0, 1, q.shape[1] // 2, q.shape[1] - 1} & set(range(q.shape[1])))
    group = q.shape[1] // b.heads
    cu = b.cu.tolist()
    for i, s in enumerate(sees):
        if not s:
            continue
        k, v = (x[[h // group for h in heads]] for x in b.held(i))
        e, el, m, top = ref.attention(q[cu[i]:cu[i + 1]][:, heads].double().cpu(), k, v, s, scale)
        rel, rl = ref.bounds(b.d, max(s + [1]), top, o.dtype)
        check(o[cu[i]:cu[i + 1]][:, heads].cpu(), e, m, rel, f"{note} sequence {i}")
        g = lse[cu[i]:cu[i + 1]][:, heads].double().cpu()
        none = el.isinf()
        assert torch.equal(g.isinf(), none) and (g[none] < 0).all()
        ratio = ((g - el).abs() / (rl + 4 * 2.0 ** -24 * el.abs()))[~none]
        assert (ratio <= 1).all(), f"{note} lse of sequence {i}: {float(ratio.max())} of the bound"


@pytest.mark.parametrize("d,heads,group,tokens", SHAPES)
@pytest.mark.parametrize("io,out", TYPES)
def test_lengths_beyond_the_table(kda, d, heads, group, tokens, io, out):  # noqa: F811
    """Token j sees positions 0 .. length - tokens + j, those of them that the table has room for: all of its pages are held,
    lengths pass them by less than the tokens, by as much, and by far.  Queries of 0: the mean of what is seen, and the log of
    its count."""
    room = 256
    b = Batch(kda, [(tokens, room)] * 5, heads, d, 64)
    b.fill()
    beyond = [0, max(1, tokens // 2), tokens, tokens + room, 2**31 - 1 - room]
    b.lengths = torch.tensor([room + x for x in beyond], dtype=torch.int32, device="cuda")
    q = torch.zeros(b.n, heads * group, d, dtype=io, device="cuda")
    sees = [[min(room, room + x - tokens + j + 1) for j in range(tokens)] for x in beyond]
    for max_q in (tokens, 0):
        compare(kda, b, make_cfg(kda, heads * group, d, io, out), q, sees, d ** -0.5, max_q, f"max_q {max_q}")


@pytest.mark.parametrize("d,heads,group,tokens", SHAPES)
@pytest.mark.parametrize("io,out", TYPES)
@pytest.mark.parametrize("ratio", [2.0 ** 10, 2.0 ** 20, 2.0 ** 60])
def test_small_channels_beside_large_ones(kda, d, heads, group, tokens, io, out, ratio):  # noqa: F811
    """One channel in 32 of the queries is `ratio` times the others, and the keys are 0 there: scores are the others'."""
    b = Batch(kda, [(tokens, tokens + 90)], heads, d, 64)
    b.fill()
    b.cache.k[..., ::16] &= 0xf0       # the even channel of the first byte of each 32
    q = Rand(5)(b.n, heads * group, d, dtype=io, scale=2)
    q[..., ::32] *= ratio
    sees = [[91 + j for j in range(tokens)]]
    compare(kda, b, make_cfg(kda, heads * group, d, io, out), q, sees, d ** -0.5, tokens)


@pytest.mark.parametrize("d,heads,group,tokens", SHAPES)
@pytest.mark.parametrize("io,out", TYPES)
def test_weights_and_their_sum(kda, d, heads, group, tokens, io, out):  # noqa: F811
    """Scores that rise by a little at a time, so that a row's running maximum lags behind, and outputs far smaller than
    their terms."""
    n = tokens + 400
    b = Batch(kda, [(tokens, n)], heads, d, 64)
    b.fill()
    q = Rand(7)(b.n, heads * group, d, dtype=io)
    # half of a row's weight on one key: the scores' slope along the positions comes from the scales
    for p in range(n):
        b.cache.k_scale[int(b.table[0, p // 64]), :, :, p % 64] = 124 + (p * 5 // n)
    sees = [[401 + j for j in range(tokens)]]
    compare(kda, b, make_cfg(kda, heads * group, d, io, out), q, sees, 0.7 * d ** -0.5, tokens)


@pytest.mark.parametrize("io,out", TYPES)
@pytest.mark.parametrize("d,heads,group", [(64, 2, 4), (128, 2, 4), (256, 2, 8)])
def test_a_token_beside_others(kda, d, heads, group, io, out):  # noqa: F811
    """A decoding token is as near to 64 bits beside drafts and chunks as alone."""
    for tokens in (1, 5, 60):
        b = Batch(kda, [(1, 700), (tokens, 300)], heads, d, 64)
        b.fill()
        q = Rand(9)(b.n, heads * group, d, dtype=io, scale=2)
        sees = [[700], [301 - tokens + j for j in range(tokens)]]
        for max_q in (tokens, 0):
            compare(kda, b, make_cfg(kda, heads * group, d, io, out), q, sees, d ** -0.5, max_q, f"{tokens} tokens")
