"""Which kernel the block-scaled product takes (CPU only): the library's own
rule, compiled on the host, has to give the sizes of tests/product_shapes.py
the kernels that they are there for, and every kernel has to have a size."""
import os
import re
import subprocess

import pytest

from tests.product_shapes import BF16, CUS, FP32

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_delta_rule_03_amd", "csrc")

ASK = r"""
#include <cstdio>
#include "fp8_matmul_choice.h"
int main() {
  for (const auto& c : kda::kChoicesBf16) std::printf("table 1 %d %d %d\n", c.outs, c.toks, c.split);
  for (const auto& c : kda::kChoicesFp32) std::printf("table 0 %d %d %d\n", c.outs, c.toks, c.split);
  int bf16, N, K;
  long long M;
  while (std::scanf("%d %lld %d %d", &bf16, &M, &N, &K) == 4) {
    const kda::Choice c = kda::choose_fp8_matmul(bf16 != 0, M, N, K, CUS);
    std::printf("size %d %d %d %lld\n", c.outs, c.toks, c.split, static_cast<long long>(CUS * kda::choice_per_cu(c)));
  }
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    """ask([(bf16, M, N, K)]) -> (the two tables, [(outputs, tokens, parts, workgroups at a time)])."""
    d = tmp_path_factory.mktemp("choice")
    (d / "ask.cpp").write_text(ASK)
    subprocess.check_call(["g++", "-std=c++17", "-Wall", "-Werror", f"-DCUS={CUS}", "-I", CSRC, str(d / "ask.cpp"), "-o",
                           str(d / "ask")])

    def run(sizes):
        text = "\n".join(" ".join(map(str, map(int, s))) for s in sizes)
        out = subprocess.run([str(d / "ask")], input=text, capture_output=True, text=True, check=True).stdout
        lines = [x.split() for x in out.splitlines()]
        ints = {w: [tuple(map(int, x[1:])) for x in lines if x[0] == w] for w in ("table", "size")}
        return {b: {t[1:] for t in ints["table"] if t[0] == b} for b in (0, 1)}, ints["size"]
    return run


@pytest.mark.parametrize("bf16,shapes", [(1, BF16), (0, FP32)])
def test_every_kernel_has_its_sizes(ask, bf16, shapes):
    flat = [(k, s) for k, ss in shapes.items() for s in ss]
    tables, got = ask([(bf16, *s) for _, s in flat])
    assert tables[bf16] == set(shapes)
    for (kernel, size), g in zip(flat, got):
        assert g[:3] == kernel, (size, g)


def test_sizes_with_several_tiles_a_workgroup(ask):
    """Both a whole-K kernel and one with K in parts walk more than one tile a workgroup."""
    sizes = [(1, 5337, 5563, 432), (1, 5400, 5600, 2192), (0, 346, 11063, 1024)]
    for (_, m, n, k), (outs, toks, split, slots) in zip(sizes, ask(sizes)[1]):
        assert -(-m // toks) * -(-n // outs) > slots, (m, n, k)
        assert split == (2 if m == 346 else 1)


def test_parts_of_k_are_equal_and_whole(ask):
    """A size takes parts of K only where they are equal numbers of whole scale blocks, four or more."""
    sizes = [(b, m, n, k) for b in (0, 1) for m in (17, 63, 200, 256, 700, 1024) for n in (16, 600, 1024, 4096)
             for k in (16, 496, 512, 1000 - 8, 1024, 1040, 1152, 2048, 4096, 4112, 7680)]
    for (_, m, n, k), (_, _, split, _) in zip(sizes, ask(sizes)[1]):
        assert split <= 1 or (k % (128 * split) == 0 and k // 128 >= 4 * split), (m, n, k)


def test_inline_assembly_names_m0():
    """Assembly that writes m0 says so to the compiler."""
    for name in sorted(os.listdir(CSRC)):
        src = open(os.path.join(CSRC, name)).read()
        for m in re.finditer(r"\basm(?: volatile)?\((.*?)\);", src, re.S):
            if "m0" in m.group(1) or "KDA_LDS_FIRST" in m.group(1):
                clobbers = m.group(1).rsplit(":", 1)[1]
                assert '"m0"' in clobbers, f"{name}: {m.group(0)[:90]}"
