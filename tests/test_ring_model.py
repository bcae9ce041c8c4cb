"""Every order of the adapters' ring of stages, on the CPU: no wait takes one phase of its barrier for another, no slot is filled
before it is free, and everyone comes to the end."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not available")
    exe = str(tmp_path_factory.mktemp("ring") / "ring_model")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror", "-I",
                    os.path.join(ROOT, "combine_topk_ids_histogram_gb300", "csrc"), os.path.join(ROOT, "tests", "c", "ring_model.cpp"), "-o", exe], check=True)
    return lambda *a: subprocess.run([exe, *map(str, a)], capture_output=True, text=True).stdout.strip()


@pytest.mark.parametrize("first", range(9))
@pytest.mark.parametrize("second", [0, 1, 2, 3, 6])
def test_every_order(model, first, second):
    assert model(first, second) == "ok"


def test_the_model_finds_a_phase_that_is_passed_over(model):
    """With two barriers for finished products, stage 2's can end before a warp has looked for stage 0's."""
    assert model(6, 3, "two") == "a wait sees the parity of another phase"


@pytest.mark.parametrize("first", [15, 16, 17, 24, 25, 33, 41])
def test_chunks_of_sums(model, first):
    assert model(first, 2) == "ok"


@pytest.mark.parametrize("first,second", [(1, 1), (4, 3), (6, 6), (18, 2)])
def test_a_wait_that_runs_out(model, first, second):
    """Products that never finish: everyone comes to the end, and nobody fills a slot that they may still read.  Going on in the loop, as if
    the wait had ended, would."""
    for n in range(first + second + 1):
        assert model(first, second, "lost", n) == "ok"
    assert model(6, 6, "lost", 1, "on") == "a slot is filled before its products are done"


def test_the_kernel_goes_by_the_ring(model):
    """The kernel's barriers and phases are the ones that the model goes through."""
    with open(os.path.join(ROOT, "combine_topk_ids_histogram_gb300", "csrc", "ep_lora.cu")) as f:
        src = f.read()
    assert "s_full[kRing], s_free[kRing], s_done[kRing], s_taken[2];" in src
    for line in src.splitlines():
        if "wait(s_" in line or "tc_commit" in line:
            assert "slot" in line or "chunk_phase" in line, line
        if "wait(s_" in line and "stages1 > 0" not in line:     # (the last one of the first product, behind its loop)
            assert "break;" in line, line
