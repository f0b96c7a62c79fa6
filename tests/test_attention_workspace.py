"""The workspace of paged attention (CPU only): one for a call is enough for every smaller call, and its size is as stated."""
import itertools

import pytest
import torch

from tests.test_abi import kda  # noqa: F401  (fixture)

BF, F32 = torch.bfloat16, torch.float32
TOKENS = [0, 1, 2, 3, 5, 8, 13, 16, 17, 33, 64, 100, 128, 161, 200, 256, 257, 300, 511, 512, 513, 700, 1000, 1024, 1500, 2048, 2304,
          3100, 4096, 5000, 8192, 16384, 32768, 131072]


@pytest.mark.parametrize("d,heads,group", [(64, 1, 1), (64, 8, 4), (128, 8, 4), (128, 2, 24), (256, 2, 8), (256, 1, 16), (256, 16, 1)])
@pytest.mark.parametrize("io,out", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
def test_a_workspace_is_enough_for_smaller_calls(kda, d, heads, group, io, out):  # noqa: F811
    cfg = kda.Config(None, None, None, None, None, heads * group, d, d, io, out)
    need = lambda N, n, q: kda.kda_paged_attention_workspace_bytes(cfg, heads, N, n, q)   # noqa: E731
    counts = [0, 1, 2, 3, 17, 180, 256, 1024, 4096]
    most = {}
    for N, n in itertools.product(counts, TOKENS):
        sizes = [need(N, n, q) for q in [*TOKENS[1:], 0]]
        assert sizes == sorted(sizes), (N, n)     # in max_q, 0 the most
        most[N, n] = sizes
    for i, N in enumerate(counts):
        for j, n in enumerate(TOKENS):
            for other in ([(counts[i - 1], n)] if i else []) + ([(N, TOKENS[j - 1])] if j else []):
                assert all(a <= b for a, b in zip(most[other], most[N, n])), (other, (N, n))


def test_its_size(kda):  # noqa: F811
    """As include/kda.h states it, and tens of MB where a call is short."""
    MB = 10 ** 6
    for d, heads, group, chunks in ((256, 2, 8, 204), (128, 8, 4, 103), (64, 8, 4, 52)):
        cfg = kda.Config(None, None, None, None, None, heads * group, d, d, BF, BF)
        need = lambda N, n, q: kda.kda_paged_attention_workspace_bytes(cfg, heads, N, n, q)   # noqa: E731
        assert max(need(N, N, 1) for N in (1, 64, 4096)) <= 18 * MB
        for N, n in ((1, 8192), (4, 32768), (4096, 131072)):
            units = (n * group // 256 + N) * heads
            assert need(N, n, 0) <= chunks * MB + 32 * units + 256
        assert need(1, 256, 256) <= 70 * MB and need(1, 512, 512) <= 70 * MB
