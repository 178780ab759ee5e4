"""What the library would launch, seen on the host: a small program links it and defines the
runtime's launch entry itself, so that sizes no test could hold in memory are checked too."""

import os
import shutil
import subprocess

import pytest

from gemv_int4_quantize_amd import LIB_PATH

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")

PROGRAM = r"""
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include "w8a8.h"
struct Dim { uint32_t x, y, z; };
static Dim g_grid, g_block;
extern "C" {
int __hipPushCallConfiguration(Dim grid, Dim block, size_t, void*) { g_grid = grid; g_block = block; return 0; }
int __hipPopCallConfiguration(Dim* grid, Dim* block, size_t* shared, void** stream) {
  *grid = g_grid; *block = g_block; *shared = 0; *stream = nullptr;
  return 0;
}
int hipLaunchKernel(const void*, Dim grid, Dim block, void** args, size_t, void*) {
  // scores: (TokArgs, parts, seg, workspace, ...), their gradient: (TokGradArgs, parts, seg)
  std::printf("launch %u %u %d %d\n", grid.x, block.x, *static_cast<int*>(args[1]), *static_cast<int*>(args[2]));
  return 0;
}
int hipGetLastError() { return 0; }
int hipGetDevice(int* d) { *d = 0; return 0; }
int hipDeviceGetAttribute(int* v, int, int) { *v = 0; return 1; }  // the built-in figures
}
int main(int argc, char** argv) {
  const int64_t M = std::atoll(argv[1]), V = std::atoll(argv[2]);
  const int top = std::atoi(argv[3]);
  size_t bytes = 0;
  if (tok_workspace_bytes(M, V, top, &bytes) != 0) return 1;
  char* p = reinterpret_cast<char*>(0x10000);
  float* f = reinterpret_cast<float*>(p);
  int64_t* i = reinterpret_cast<int64_t*>(p);
  std::printf("bytes %zu\n", bytes);
  if (tok_logprobs(p, W4_DT_BF16, M, V, V, i, -100, 1.0, top, f, f, f, f, i, bytes ? p : nullptr, bytes, nullptr) != 0) return 2;
  std::printf("gradient\n");
  if (tok_logprobs_grad(p, W4_DT_BF16, M, V, V, i, -100, 1.0, 0, f, f, nullptr, f, nullptr, nullptr, p + 64, V, nullptr) != 0) return 3;
  return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("launches")
    (d / "p.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", INCLUDE, str(d / "p.cpp"), LIB_PATH, "-rdynamic",
                    "-Wl,-rpath," + os.path.dirname(LIB_PATH), "-Wl,--allow-shlib-undefined", "-o", str(d / "p")], check=True)
    return str(d / "p")


@pytest.mark.parametrize("M,V,top", [(4, 128256, 20), (64, 9000, 0), (700, 16384, 5), ((1 << 23) + 10, 16384, 5),
                                     ((1 << 23) + 1023, 17000, 0), ((1 << 24) + 1, 8192, 1), (3 << 23, 16384, 0),
                                     ((1 << 25) + 3, 2, 1)])
def test_rows_and_workspace_of_the_scores(program, M, V, top):
    """All rows are covered, and a row is cut into parts only where the workspace has room for them."""
    out = subprocess.run([program, str(M), str(V), str(top)], check=True, capture_output=True, text=True).stdout
    forward, gradient = ([tuple(map(int, line.split()[1:])) for line in half.splitlines() if line.startswith("launch")]
                         for half in out.split("gradient"))
    size = int(out.split()[1])
    if size:  # one launch over all parts, one that joins them
        (grid, _, parts, seg), (join, _, of, _) = forward
        assert grid == M * parts and join == M and of == parts > 1
        assert (parts - 1) * seg < V <= parts * seg and size >= M * parts * (16 + 8 * top)
    else:
        assert all(parts == 1 and seg >= V for _, _, parts, seg in forward)
        assert sum(grid for grid, *_ in forward) == M
    for launches in (forward, gradient):
        assert all(grid * block < 1 << 32 for grid, block, *_ in launches)
    assert sum(grid // parts for grid, _, parts, _ in gradient) == M
    assert all((parts - 1) * seg < V <= parts * seg for _, _, parts, seg in gradient)
