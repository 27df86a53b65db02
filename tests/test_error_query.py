"""The query of the device error words: a word that nothing was recorded in is read and not
written (each copy costs the caller microseconds, and there is a word a translation unit).  On the
CPU against fakes of the two CUDA copies; on the GPU an error is reported once."""
import glob
import os
import re
import subprocess

import pytest
import torch

from gated_deltanet_linear_13_gb300 import build_lib

PROGRAM = r'''
#include <cuda_runtime.h>
#include <cstdio>
#include <cstring>
static int reads, writes;
static unsigned word;
template <class W> cudaError_t fake_from(void* to, const W&, size_t n) {
  ++reads; memcpy(to, &word, n); return cudaSuccess;
}
template <class W> cudaError_t fake_to(const W&, const void* from, size_t n) {
  ++writes; memcpy(&word, from, n); return cudaSuccess;
}
#define cudaMemcpyFromSymbol fake_from
#define cudaMemcpyToSymbol fake_to
#include "common.cuh"
int main() {
  for (unsigned recorded : {0u, 1u, 2u, 3u}) {
    word = recorded; reads = writes = 0;
    const unsigned got = gdn::take_error(word);
    printf("%u %u %u %d %d\n", recorded, got, word, reads, writes);
  }
}
'''


def test_a_clean_word_is_only_read(tmp_path):
    src, exe = tmp_path / "query.cu", tmp_path / "query"
    src.write_text(PROGRAM)
    r = subprocess.run([build_lib.NVCC, *build_lib.ARCH, "-std=c++17", "-I", build_lib.INCLUDE, "-I",
                        build_lib.CSRC, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lines = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n")
    # recorded, returned, left, reads, writes
    assert lines[:4] == ["0 0 0 1 0", "1 1 0 1 1", "2 2 0 1 1", "3 3 0 1 1"]


def test_every_word_is_taken_so():
    words = 0
    for path in glob.glob(os.path.join(build_lib.CSRC, "*.cu")):
        with open(path) as f:
            text = f.read()
        assert "cudaMemcpyToSymbol" not in text, path
        words += len(re.findall(r"take_error\(g_err_\w+\)", text))
    assert words == 10


@pytest.mark.gpu
def test_a_recorded_error_is_reported_once():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_deltanet_linear_13_gb300 as gdn
    build_lib.build()
    gdn.load_library()
    kv = torch.zeros(1, 1, 16, 128, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(1, 1, 128, dtype=torch.bfloat16, device="cuda")
    slot = torch.tensor([16], dtype=torch.int32, device="cuda")
    for _ in range(2):
        gdn.gdn_kv_cache_append(x, x, kv, kv.clone(), slot)
        assert [gdn.gdn_get_device_error() for _ in range(3)] == [6, 0, 0]
