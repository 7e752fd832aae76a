"""The operators of a paged cache in 8 bits on the host where their checks end."""

import itertools
import os
import random
import subprocess

import pytest

torch = pytest.importorskip("torch")

import sparse_attention_indexer_fp32_gb300 as tk  # noqa: E402
from sparse_attention_indexer_fp32_gb300 import _cache  # noqa: E402
from sparse_attention_indexer_fp32_gb300 import build as cuda_build  # noqa: E402


def _elements(shape, strides, start=0):
    return {start + sum(i * s for i, s in zip(at, strides)) for at in itertools.product(*(range(n) for n in shape))}


def test_caches_that_share_an_element_are_found():
    """Whatever the strides: no two caches that share an element pass, parts side by side do."""

    def meet(shape, strides, second, gap):
        return _cache._meet((*shape[:3], shape[3]), (*strides, 1), (*strides, 1), second, gap, 1)

    # pages and heads 33 and 21 apart, entries 5: the element at 48 is reached by another way than the strides' order
    shape, strides = (2, 2, 3, 2), (5, 33, 21)
    shared = _elements(shape, (*strides, 1)) & _elements((*shape[:3], 1), (*strides, 1), 48)
    assert shared and meet(shape, strides, 1, 48)
    rng = random.Random(1)
    found = 0
    for _ in range(4000):
        shape = tuple(rng.randint(1, 4) for _ in range(4))
        strides = [rng.randint(1, 12) for _ in range(3)]
        if rng.random() < 0.5:  # strides of a tensor, its dimensions in any order
            order, step = rng.sample(range(3), 3), shape[3] + rng.randint(0, 4)
            for d in order:
                strides[d], step = step, step * shape[d] + rng.randint(0, 3)
        second, gap = rng.randint(1, 4), rng.randint(-40, 40)
        shared = _elements(shape, (*strides, 1)) & _elements((*shape[:3], second), (*strides, 1), gap)
        found += bool(shared)
        assert not shared or meet(shape, strides, second, gap), (shape, strides, second, gap)
    assert found > 500
    # what lies side by side in pages, entries, heads or the pool is let through
    for shape, strides, second, gap in (((5, 4, 3, 8), (192, 24, 8), 8, 96), ((5, 4, 3, 8), (192, 24, 8), 8, -96),
                                        ((5, 4, 3, 8), (240, 60, 20), 12, 8), ((5, 4, 3, 12), (240, 60, 20), 8, -8),
                                        ((5, 4, 3, 8), (96, 8, 32), 8, 480), ((3, 4, 3, 8), (96, 24, 8), 8, 288),
                                        ((3, 4, 3, 8), (192, 24, 8), 8, 96), ((1, 1, 1, 8), (7, 3, 5), 8, 8)):
        assert not _elements(shape, (*strides, 1)) & _elements((*shape[:3], second), (*strides, 1), gap)
        assert not meet(shape, strides, second, gap), (shape, strides, second, gap)


def test_spans_that_overlap():
    for size, spans, want in ((8, [(108, 120), (92, 100)], False), (8, [(107, 120)], True),
                              (8, [(90, 101)], True), (8, [(102, 104)], True), (8, [(90, 120)], True), (0, [(90, 120)], False),
                              (8, [(104, 104)], False), (8, [(100, 108)], True), (8, [(100, 104)], True), (8, [(104, 108)], True)):
        assert _cache._clash(100, size, spans) is want, (size, spans)


# ---- the registers that attention's warps trade ------------------------------------------------------

PROGRAM = r"""
#include <cstdio>
#include "step_launch.cuh"

__global__ void kernel(int* x) { *x = 1; }

extern int calls;

int main() {
  for (int i = 0; i < 5; ++i) std::printf("%d ", static_cast<int>(tki::has_registers<kernel>(64)));
  std::printf("%d\n", calls);
}
"""

FAKE = r"""
#include <cuda_runtime_api.h>

// The CUDA call, with answers of the test's: an error at first, then registers.
int calls = 0, answers[] = {-1, 40, 64, -1, 1};
cudaError_t CUDARTAPI cudaFuncGetAttributes(cudaFuncAttributes* f, const void*) {
  const int a = answers[calls++];
  f->numRegs = a;
  return a < 0 ? cudaErrorUnknown : cudaSuccess;
}
"""


def test_an_answer_that_did_not_come_is_asked_for_again(tmp_path):
    """A register count that CUDA fails to tell, or another one than was laid out for, refuses that call alone; once it
    was right it is not asked for again."""
    source, fake, program = tmp_path / "registers.cu", tmp_path / "fake.cpp", tmp_path / "registers"
    source.write_text(PROGRAM), fake.write_text(FAKE)
    libraries = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cuda_build.nvcc()))), "lib64")
    subprocess.run([cuda_build.nvcc(), *cuda_build.ARCH, "-std=c++17", "-cudart", "shared", "-I", cuda_build.INCLUDE, "-I",
                    cuda_build.CSRC, str(source), str(fake), "-o", str(program)], check=True, timeout=300)
    got = subprocess.run([str(program)], check=True, timeout=60, capture_output=True, text=True,
                         env={**os.environ, "LD_LIBRARY_PATH": libraries}).stdout.split()
    assert [int(x) for x in got] == [tk.Status.ECUDA, tk.Status.ECUDA, tk.Status.OK, tk.Status.OK, tk.Status.OK, 3]
