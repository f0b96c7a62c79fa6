"""Every kernel of the block-scaled product on dense data: alone, again on two
streams, and captured into a graph."""
import pytest
import torch

from tests import layer_reference as ref
from tests.product_shapes import BF16, FP32
from tests.test_gpu_layer import BF, F32, Rand, fp8_operands, guarded, kda, make_cfg, same  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

ALL = [(BF, s) for ss in BF16.values() for s in ss] + [(F32, s) for ss in FP32.values() for s in ss]


@pytest.mark.parametrize("out,size", ALL)
def test_product_of_every_kernel(kda, out, size):
    M, N, K = size
    r = Rand(M + N + K)
    a, sa, w, sw = fp8_operands(r, M, N, K)
    y, ok = guarded((M, N), out)
    kda.kda_fp8_matmul(make_cfg(kda, out=out), a, sa, w, sw, y=y)
    for i in range(0, M, 2048):
        ref.check_matmul(y, a, sa, w, sw, rows=slice(i, i + 2048))
    assert ok()


def products(kda, seed, stream=None):
    """A call of every kernel of the product; the outputs."""
    r = Rand(seed)
    given = [(make_cfg(kda, out=out), fp8_operands(r, *size)) for out, size in ALL]
    torch.cuda.synchronize()
    return lambda: [kda.kda_fp8_matmul(cfg, *ops, stream=stream) for cfg, ops in given]


def test_products_repeat_on_two_streams(kda):
    first = products(kda, 51)()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    calls = [products(kda, 51, s) for s in streams]
    outs = [c() for _ in range(3) for c in calls]
    torch.cuda.synchronize()
    for o in outs:
        assert same(first, o)


def test_products_in_a_graph(kda):
    call = products(kda, 52)
    expect = call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    for _ in range(3):
        for o in outs:
            o.view(torch.uint8).fill_(0xff)
        graph.replay()
        torch.cuda.synchronize()
        assert same(expect, outs)
        assert same(expect, call())   # eager work between the replays
