"""Which kernel answers a call (csrc/answer_way.h), compiled for the host and checked
without a GPU: that the GPU tests' sizes reach the kernels that they mean to test."""
import os
import shutil
import subprocess

import pytest

import test_gpu_answer_rescale
import test_gpu_answer_ways
import test_gpu_answer_weights

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "context_causal_attention_zigzag_gb300", "csrc")
CUDA_INCLUDE = "/usr/local/cuda/include"

PROGRAM = r"""
#include <stdio.h>
#include "answer_way.h"
using namespace cpattn;

int main() {
  TreeArgs a = {};
  while (scanf("%d %d %d %d %d %d %d", &a.N, &a.R, &a.H, &a.Hkv, &a.D, &a.Nk, &a.causal) == 7)
    printf("%d %d\n", (int)prompt_way(a, 152).by, prompt_way(a, 152).above);
  return 0;
}
"""
NAMES = ["small", "direct", "line", "sorted"]


@pytest.fixture(scope="module")
def way(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None or not os.path.exists(os.path.join(CUDA_INCLUDE, "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA headers")
    at = tmp_path_factory.mktemp("way")
    src, exe = at / "way.cpp", at / "way"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, "-I", os.path.join(ROOT, "include"), "-I", CUDA_INCLUDE,
                    str(src), "-o", str(exe)], check=True, capture_output=True, text=True)

    def ask(N, R, H, Hkv, D, Nk=None, causal=True):
        line = " ".join(str(int(x)) for x in (N, R, H, Hkv, D, N if Nk is None else Nk, causal))
        out = subprocess.run([str(exe)], input=line, capture_output=True, text=True, check=True).stdout.split()
        return NAMES[int(out[0])] + (f"+{out[1]}" if out[1] != "0" else "")
    return ask


def marks(test, names):
    """The parameter sets of a test's parametrization by `names`."""
    return [m.args[1] for m in test.pytestmark if m.name == "parametrize" and m.args[0] == names][0]


def test_planned_calls_are_sorted(way):
    for N, R, H, Hkv, D in test_gpu_answer_ways.PLANNED:
        assert way(N, R, H, Hkv, D) == "sorted"


def test_tests_of_shared_batches_share_them(way):
    from test_gpu_answer_ways import SHARE, SHARED
    for causal in (True, False):
        assert [way(sum(nq), len(nq), H, Hkv, D, sum(nk or nq), causal) for nq, nk, H, Hkv, D in SHARED] == \
            [f"small+{SHARE}"] * len(SHARED)
    assert way(463, 64, 32, 8, 128) == f"small+{SHARE}"


def test_tests_of_the_softmax_correction_reach_every_tensor_core_kernel(way):
    cases = marks(test_gpu_answer_rescale.test_rising_scores_in_prompts, "nq,nk,H,Hkv,D")
    want = ["sorted"] * 6 + ["direct"] * 2 + ["line"] * 3
    for causal in (True, False):
        assert [way(sum(nq), len(nq), H, Hkv, D, sum(nk), causal) for nq, nk, H, Hkv, D in cases] == want


def test_tests_of_weak_weights_reach_every_tensor_core_kernel(way):
    cases = marks(test_gpu_answer_weights.test_many_weak_keys_behind_a_strong_one_in_a_prompt, "nq,nk,R,H,Hkv,D")
    assert [way(nq * R, R, H, Hkv, D, nk * R, False) for nq, nk, R, H, Hkv, D in cases] == \
        ["sorted"] * 3 + ["line"] * 2


# sequences of nq queries and nk keys (None: nq), H, Hkv: the kernel; a number behind it:
# sequences of so many keys and more go to the cut line
UNEVEN = [
    ([400] + [1] * 63, None, 32, 8, "small+32"),
    ([400] + [0] * 63, None, 32, 8, "small+32"),
    ([2000] + [0] * 511, None, 32, 8, "small+32"),
    ([1] * 256, [16384] + [1] * 255, 32, 8, "small+256"),
    ([1] * 38, [19000] + [1] * 37, 8, 1, "line"),
    ([128] * 4, [4128] + [128] * 3, 32, 8, "line"),
]
EVEN = [
    ([77], None, 32, 8, "direct"),
    ([4] * 8, None, 32, 8, "small"),
    ([1] * 64, None, 32, 8, "small"),
    ([128] * 4, [500] * 4, 32, 8, "direct"),
    ([16] * 8, None, 32, 8, "direct"),
    ([16] * 64, None, 32, 8, "line"),
    ([1], [1001], 32, 8, "line"),
    ([1000] * 16, None, 32, 8, "sorted"),
]


@pytest.mark.parametrize("nq,nk,H,Hkv,want", UNEVEN + EVEN)
def test_the_longest_sequence_is_kept_in_mind(way, nq, nk, H, Hkv, want):
    """No kernel whose blocks walk a sequence alone takes a batch of which one sequence
    could hold nearly all keys."""
    assert way(sum(nq), len(nq), H, Hkv, 128, sum(nk or nq)) == want
