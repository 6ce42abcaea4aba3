"""How the sort is cut into CTAs and warps, on the CPU, with the kernel's own
header: every id has one warp, and a device without room for a cluster of 16
CTAs gets one of 8."""

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "quantized_linear_gemm_b200", "csrc")
COUNTS = (0, 1, 31, 32, 33, 1024, 1025, 8191, 8192, 8193, 16385, 65536, 65537, 10 ** 6 + 7, 2 ** 31 - 1)
SUCCESS, NOT_SUPPORTED = 0, 801


@pytest.fixture(scope="module")
def shape(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    d = tmp_path_factory.mktemp("sort")
    src, exe = str(d / "shape.cpp"), str(d / "shape")
    with open(src, "w") as f:
        f.write('#include <cstdio>\n#include <cstdlib>\n#include "moe_sort_shape.h"\n'
                'int main(int argc, char** argv) {\n'
                '  const int widest = lq::sort_widest(std::atoi(argv[1]), std::atoi(argv[2]));\n'
                '  for (int i = 3; i < argc; ++i) {\n'
                '    const lq::SortShape s = lq::sort_shape(std::atoll(argv[i]), widest);\n'
                '    std::printf("%d %lld\\n", s.ctas, static_cast<long long>(s.seg));\n  }\n}\n')
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, "-o", exe, src], check=True)

    def run(error, fitting):
        r = subprocess.run([exe, str(error), str(fitting), *map(str, COUNTS)], capture_output=True, text=True, check=True)
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    return run


@pytest.mark.parametrize("error,fitting,widest", [(SUCCESS, 1, 16), (SUCCESS, 9, 16), (SUCCESS, 0, 8),
                                                  (NOT_SUPPORTED, 0, 8)])
def test_clusters(shape, error, fitting, widest):
    got = shape(error, fitting)
    assert max(c for c, _ in got) == widest
    for n, (ctas, seg) in zip(COUNTS, got):
        assert 1 <= ctas <= widest and ctas & (ctas - 1) == 0
        assert seg % 32 == 0 and ctas * 32 * seg >= n             # 32 warps per CTA cover every id
        assert ctas == widest or n <= ctas * 1024


def test_same_cut_as_far_as_both_fit(shape):
    wide, narrow = shape(SUCCESS, 1), shape(SUCCESS, 0)
    assert [w for n, w in zip(COUNTS, wide) if n <= 8192] == [w for n, w in zip(COUNTS, narrow) if n <= 8192]
