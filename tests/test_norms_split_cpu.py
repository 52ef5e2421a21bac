"""How the norms' launchers cut calls of very many rows, on the host: the launches are recorded, not made."""
import os
import subprocess

import pytest

from gated_delta_net_gb300 import build

HARNESS = r"""
#include <cstdio>
#include <cstdlib>
#include <type_traits>
#include "internal.cuh"

namespace gdn {
int sm_count() { return 152; }
template <typename P, typename = void>
struct Residual : std::false_type {};
template <typename P>
struct Residual<P, std::void_t<decltype(P::h)>> : std::true_type {};

// grid, rows a kernel counts to (0: a block a row), byte addresses of the first row of x, y, h, n
template <typename K, typename P, typename... R>
cudaError_t recorded(K, dim3 grid, unsigned, cudaStream_t, P p, R... rows) {
    if constexpr (Residual<P>::value)
        std::printf("%u %lld %llu %llu %llu %llu\n", grid.x, (0ll + ... + rows), (unsigned long long)p.x, (unsigned long long)p.y,
                    (unsigned long long)p.h, (unsigned long long)p.n);
    return cudaSuccess;
}
}  // namespace gdn

#define launch_early recorded
#include "norms.cu"

int main(int, char **v) {
    gdn_residual_norm_args a = {};
    a.total_tokens = std::atoi(v[1]);
    a.width = std::atoi(v[2]);
    a.dtype = std::atoi(v[3]);
    a.weight_dtype = GDN_F32;
    a.scale = 1.f;
    a.x_stride = std::atoll(v[4]);
    a.x = (void *)(1ull << 40); a.y = (void *)(2ull << 40); a.h = (void *)(3ull << 40); a.n = (void *)(4ull << 40);
    a.weight = a.post_weight = (void *)4096;
    return gdn::launch_residual_norm(a, nullptr);
}
"""


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    where = tmp_path_factory.mktemp("split")
    src, exe = where / "split.cu", where / "split"
    src.write_text(HARNESS)
    subprocess.run([build.nvcc(), "-std=c++17", "--expt-relaxed-constexpr", "-gencode", "arch=compute_103a,code=compute_103a",
                    "-I", build.CSRC, "-I", build.INCLUDE, str(src), "-o", str(exe)], check=True, capture_output=True)
    return lambda *args: subprocess.run([str(exe), *map(str, args)], check=True, capture_output=True, text=True).stdout


@pytest.mark.parametrize("tokens", [1, 1000, 2 ** 30, 2 ** 30 + 1, 2 ** 31 - 1])
@pytest.mark.parametrize("width,dtype,stride", [(8, 1, 0), (8, 1, 24), (4, 0, 0), (7, 1, 0), (1, 0, 3)])
def test_residual_norm_rows_stay_countable(harness, tokens, width, dtype, stride):
    size = 2 if dtype else 4
    at = 0
    for line in harness(tokens, width, dtype, stride).splitlines():
        grid, rows, *first = map(int, line.split())
        assert grid >= 1
        # a row's number and the one a grid further on are ints (a block a row has no such step)
        assert rows + grid < 2 ** 31
        rows = rows or grid
        row = [(stride or width) * size, width * size, width * size, width * size]
        assert first == [(i + 1 << 40) + at * r for i, r in enumerate(row)]
        at += rows
    assert at == tokens
