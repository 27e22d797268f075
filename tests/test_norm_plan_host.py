"""The norm's grids: no more blocks than the multiprocessors' shared memory has room
for at once.  Host only (compiled, nothing is launched)."""
import os
import subprocess

import pytest

from moe_expert_layer_softmax_gb300 import _build

SOURCE = '''
#include <cstdio>
#include "norm.cuh"
using namespace moe;
namespace moe { const DeviceInfo* device_info() { static DeviceInfo i; i.sm_count = 152; i.ready = true; return &i; } }
template <int BYTES, int NV> void ring(int d) {
  const RowSplit split(d, NV, NV, kNormThreads);
  const int threads = split.threads(), bytes = RowRing<BYTES, NV>::kBytes;
  const int n = norm_resident(norm_blocks(true, NV, kNormThreads), kNormThreads, threads, bytes);
  printf("%d %d %d %d %d %d\\n", BYTES, NV, d, threads * bytes, n, row_blocks(1 << 20, split.group, threads, n));
}
int main() {
  for (int d : {6152, 7168, 7176, 8192}) { ring<64, 4>(d); ring<48, 4>(d); ring<32, 4>(d); }
  for (int d : {4104, 6144}) { ring<64, 3>(d); ring<32, 3>(d); }
  for (int d : {264, 4096}) { ring<64, 2>(d); ring<96, 2>(d); ring<32, 2>(d); }
}
'''


def test_blocks_fit_the_shared_memory(tmp_path):
    try:
        cc = _build.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    src, exe = tmp_path / "plan.cu", tmp_path / "plan"
    src.write_text(SOURCE)
    subprocess.run([cc, *_build.ARCH, "-std=c++17", "-I", _build.CSRC, "-I", os.path.join(_build.ROOT, "include"),
                    str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n")
    seen = set()
    for line in filter(None, lines):
        bytes_, nv, d, smem, n, grid = map(int, line.split())
        assert n >= 1 and n * (smem + 1024 + 512) <= 228 * 1024, line
        assert grid == 152 * n, line   # of a million rows
        seen.add((bytes_, d, n))
    assert (64, 8192, 1) in seen       # 128 KB a block
    assert (64, 7168, 2) in seen and (32, 8192, 2) in seen and (96, 4096, 2) in seen
