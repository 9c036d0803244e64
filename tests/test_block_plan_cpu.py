"""CPU: which kernel fp8_linear_block runs for a shape: the shapes of the GPU
tests reach every one.  linear_block_plan is built with the host compiler."""

import os
import shutil
import subprocess

import pytest

from block_tile_shapes import KERNEL_SHAPES, NO_K
from test_gpu_linear_block import SHAPES

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.fail("g++ is needed to build the host check")
    exe = str(tmp_path_factory.mktemp("plan") / "linear_block_plan")
    r = subprocess.run([gxx, "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-isystem", "/opt/rocm/include",
                        os.path.join(HERE, "host", "linear_block_plan.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(shapes):
        text = "\n".join("%d %d %d" % s for s in shapes)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=60)
        assert out.returncode == 0
        return out.stdout.splitlines()

    return run


@pytest.mark.parametrize("table", [KERNEL_SHAPES, NO_K])
def test_shapes_reach_their_kernels(plan, table):
    for kernel, shapes in table.items():
        assert plan(shapes) == [kernel] * len(shapes)


def test_both_kinds_of_columns():
    for kernel, shapes in KERNEL_SHAPES.items():
        assert {n % 4 == 0 for _, n, _ in shapes} == {True, False}, kernel


def test_every_kernel_has_products_against_the_formula(plan):
    # (256x128 in the test of workgroups that walk tiles)
    assert set(plan(SHAPES)) | {"256x128"} == set(KERNEL_SHAPES)
    assert plan([(1020, 16380, 2064)]) == ["256x128"]


def test_most_rows(plan):
    # beyond as many tiles as a launch can number threads for, the kernel that walks tiles
    assert plan([(2 ** 31 - 1, 3, 16), (4194304 * 128, 64, 128)]) == ["256x128"] * 2
