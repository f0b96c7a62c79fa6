"""The paged 4-bit cache: appended rows against their definition in 64 bits, bit for bit."""
import pytest
import torch

from tests import attention_reference as ref
from tests.test_gpu_layer import BF, F32, Rand
from tests.test_gpu_rope import EPS, expected, kda, make_cfg, make_rope  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


class Batch:
    """Sequences (new tokens, tokens held with them) with pages in a random order, among pages of no one."""

    def __init__(self, kda, seqs, heads, d, page, seed=0, spare=3, extra=0):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.seqs, self.page, self.heads, self.d = seqs, page, heads, d
        held = [(n + page - 1) // page for _, n in seqs]
        pages = sum(held) + spare
        order = torch.randperm(pages, generator=self.g, device="cuda").int().cpu()
        self.table = torch.full((len(seqs), max(held + [0]) + extra), -1, dtype=torch.int32)
        at = 0
        for i, h in enumerate(held):
            self.table[i, :h] = order[at:at + h]
            at += h
        self.lengths = torch.tensor([n for _, n in seqs], dtype=torch.int32).cuda()
        self.cu = torch.tensor([0] + [q for q, _ in seqs]).cumsum(0).int().cuda()
        self.n = sum(q for q, _ in seqs)
        self.table = self.table.cuda()
        self.cache = kda.KvCache.empty(pages, heads, d, page)
        for t in (self.cache.k, self.cache.k_scale, self.cache.v, self.cache.v_scale):   # bytes of every kind
            t.copy_(torch.randint(0, 256, t.shape, generator=self.g, device="cuda", dtype=torch.uint8))

    @property
    def where(self):
        return self.cu, self.table, self.lengths

    def fill(self, seed=1, bad=False):
        """Everything that the sequences hold, of normal data."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        for vals, scales in ((self.cache.k, self.cache.k_scale), (self.cache.v, self.cache.v_scale)):
            x = torch.randn((*vals.shape[:3], self.d), generator=g, device="cuda") * 0.5
            code, e = ref.quantised(x)
            for i, (_, n) in enumerate(self.seqs):
                for p in range((n + self.page - 1) // self.page):
                    j, m = int(self.table[i, p]), min(self.page, n - p * self.page)
                    vals[j, :, :m] = (code[..., 0::2] | (code[..., 1::2] << 4))[j, :, :m]
                    scales[j, :, :, :m] = e[j, :, :m].transpose(-1, -2)

    def held(self, i):
        """Keys and values of a sequence in 64 bits on the CPU, [heads, length, d]."""
        n = self.seqs[i][1]
        return [ref.values(*ref.stored(p, self.table[i], n)).cpu()
                for p in ((self.cache.k, self.cache.k_scale), (self.cache.v, self.cache.v_scale))]


def positions_of(batch):
    return torch.cat([torch.arange(n - q, n) for q, n in batch.seqs]).int()


CASES = [([(1, 1)], 1, 64, 32, 64, 1, False), ([(1, 777), (1, 32), (1, 33), (1, 64)], 2, 256, 64, 64, 1, False),
         ([(5, 5), (0, 40), (31, 95), (1, 0), (64, 128), (3, 2)], 3, 64, 32, 48, 3, True),
         ([(300, 1000), (7, 7)], 8, 128, 128, 128, 1, False), ([(40, 513)], 2, 256, 256, 208, 2, False),
         ([(33, 66)], 5, 128, 32, 96, 4, False), ([(20, 20), (9, 300)], 1, 256, 64, 0, 1, False),
         ([(4100, 4200)], 8, 256, 64, 64, 1, True)]


@pytest.mark.parametrize("seqs,heads,d,page,rot,axes,inter", CASES)
@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("norm,given", [(True, False), (True, True), (False, True)])
def test_append(kda, seqs, heads, d, page, rot, axes, inter, io, norm, given):  # noqa: F811
    b = Batch(kda, seqs, heads, d, page, seed=d + page)
    r = Rand(5)
    k, v = r(b.n, heads, d, dtype=io, scale=3), r(b.n, heads, d, dtype=io)
    w, rope, cfg = r.weight(d) if norm else None, make_rope(kda, rot, axes, inter), make_cfg(kda, heads, d, io, F32)
    at = positions_of(b)
    pos = torch.randint(0, 100000, (axes, b.n), generator=r.g, device="cuda", dtype=torch.int32) if given else None
    before = [t.clone() for t in (b.cache.k, b.cache.k_scale, b.cache.v, b.cache.v_scale)]
    kda.kda_append_kv(cfg, b.cache, *b.where, k, v, w, EPS, rope=rope, positions=pos)
    ek, _ = expected(k, w, rope, pos if given else at[None].expand(axes, -1))
    # what should be there now, and everything else as it was
    seq = torch.repeat_interleave(torch.arange(len(seqs)), torch.tensor([q for q, _ in seqs]))
    ok = at >= 0
    pg, off = b.table.cpu()[seq[ok], at[ok].long() // page].long().cuda(), (at[ok].long() % page).cuda()
    for i, x in enumerate((ek.cuda(), v)):
        code, e = ref.quantised(x[ok])
        before[2 * i][pg, :, off] = code[..., 0::2] | (code[..., 1::2] << 4)
        before[2 * i + 1][pg, :, :, off] = e
        got, scale = (b.cache.k, b.cache.k_scale) if i == 0 else (b.cache.v, b.cache.v_scale)
        # (a zero's sign is the product's: both zeros are one value)
        same = lambda t: torch.stack((t & 15, t >> 4)).masked_fill_(torch.stack((t & 15, t >> 4)) == 8, 0)   # noqa: E731
        assert torch.equal(scale, before[2 * i + 1]), f"{'kv'[i]} scales"
        assert torch.equal(same(got), same(before[2 * i])), f"{'kv'[i]} values"
    ko, vo = kda.kda_read_kv(cfg, b.cache, *b.where, b.n)
    for i, got in enumerate((ko, vo)):
        code, e = ref.quantised((ek.cuda(), v)[i])
        val = ref.values(code, e)
        val[~ok] = 0
        assert torch.equal(got.double(), val.to(got.device)), "read back"


def test_every_boundary(kda):  # noqa: F811
    """Values at, just above and just below each boundary between two codes, maxima around 6 and 3 times powers of two,
    and blocks of zeros, subnormals, infinities, NaN and huge values."""
    rows = []
    for e in (-120, -20, 0, 40, 120):
        for top in (6.0, 3.0, 3.0000002, 5.9999995, 4.0, 6.0000005):
            x = torch.tensor([m + s * 1e-7 * m for m in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0) for s in (-1, 0, 1)])
            rows.append(torch.cat((x.clamp(max=top), torch.tensor([top]), -x[:10])) * 2.0 ** e)
    special = torch.zeros(6, 32)
    special[1, 3] = 1e-40
    special[2, 5] = float("inf")
    special[3, 6] = float("nan")
    special[4, 7] = 2.0 ** 127
    special[5, 8] = 1.9 * 2.0 ** 126
    x = torch.cat((torch.stack(rows), special)).cuda()
    x = torch.cat((x, torch.zeros(-len(x) % 2, 32, device="cuda"))).view(-1, 1, 64)
    n = len(x)
    b = Batch(kda, [(n, n)], 1, 64, 32)
    cfg = make_cfg(kda, 1, 64, F32, F32)
    kda.kda_append_kv(cfg, b.cache, *b.where, x, x)
    code, e = ref.quantised(x)
    for got in kda.kda_read_kv(cfg, b.cache, *b.where, n):
        assert torch.equal(torch.nan_to_num(got.double(), nan=7e77), torch.nan_to_num(ref.values(code, e), nan=7e77))


def test_rows_pages_and_lengths_that_hold_nothing(kda):  # noqa: F811
    """Negative and far page numbers, lengths beyond the table, padded rows: nothing is written, zeros are read, rows
    behind the last sequence stay as they were."""
    b = Batch(kda, [(4, 100), (4, 100), (4, 100)], 2, 64, 32)
    b.table[0, 3] = -5
    b.table[1, 3] = b.cache.k.shape[0]
    b.lengths[2] = 2**31 - 1
    r = Rand(1)
    x = r(b.n + 5, 2, 64)
    cfg = make_cfg(kda, 2, 64, F32, F32)
    before = [t.clone() for t in (b.cache.k, b.cache.k_scale, b.cache.v, b.cache.v_scale)]
    kda.kda_append_kv(cfg, b.cache, *b.where, x, x)
    assert all(torch.equal(t, u) for t, u in zip(before, (b.cache.k, b.cache.k_scale, b.cache.v, b.cache.v_scale)))
    out = torch.full((b.n + 5, 2, 64), 7.0, device="cuda")
    kda.kda_read_kv(cfg, b.cache, *b.where, b.n + 5, k=out, v=out.clone())
    assert (out[:b.n] == 0).all() and (out[b.n:] == 7).all()


def test_one_token_each_views_streams_and_graph(kda):  # noqa: F811
    """cu_seqlens None, k and v as views into a projection, another stream, and replays of a captured step whose lengths
    grow on the device."""
    b, c = (Batch(kda, [(1, n) for n in (1, 40, 64, 200)], 2, 128, 64, seed=9) for _ in range(2))
    r = Rand(4)
    wide = r(4, 5 * 128, dtype=BF)
    k, v = wide[:, :256].view(4, 2, 128), wide[:, 256:512].view(4, 2, 128)
    cfg, rope, w = make_cfg(kda, 2, 128, BF, BF), make_rope(kda, 64), r.weight(128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kda.kda_append_kv(cfg, b.cache, None, b.table, b.lengths, k, v, w, rope=rope, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    kda.kda_append_kv(cfg, c.cache, *c.where, k.contiguous(), v.contiguous(), w, rope=rope)
    assert torch.equal(b.cache.k, c.cache.k) and torch.equal(b.cache.v_scale, c.cache.v_scale)
    for x in (b, c):
        x.lengths.fill_(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_append_kv(cfg, b.cache, None, b.table, b.lengths, k, v, w, rope=rope)
        got = kda.kda_read_kv(cfg, b.cache, None, b.table, b.lengths, 4)
        b.lengths.add_(1)
    for i in range(1, 4):
        graph.replay()
        kda.kda_append_kv(cfg, c.cache, None, c.table, c.lengths, k, v, w, rope=rope)
        e = kda.kda_read_kv(cfg, c.cache, None, c.table, c.lengths, 4)
        c.lengths.add_(1)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, e)), i
        assert all(torch.equal(getattr(b.cache, t), getattr(c.cache, t)) for t in ("k", "k_scale", "v", "v_scale")), i
