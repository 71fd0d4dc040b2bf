"""Which form of the cached-weights kernel takes a call (csrc/weights_line.h, compiled for the host)."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "context_causal_attention_zigzag_gb300", "csrc")
CUDA_INCLUDE = "/usr/local/cuda/include"

PROGRAM = r"""
#include <stdio.h>
#include "weights_line.h"
int main() {
  int R, N, G;
  while (scanf("%d %d %d", &R, &N, &G) == 3) printf("%d\n", cpattn::wline::keys_stream(R, N, G));
  return 0;
}
"""


@pytest.fixture(scope="module")
def keys_stream(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None or not os.path.exists(os.path.join(CUDA_INCLUDE, "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA headers")
    src, exe = (tmp_path_factory.mktemp("form") / n for n in ("form.cpp", "form"))
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O2", "-I", CSRC, "-I", os.path.join(ROOT, "include"), "-I", CUDA_INCLUDE,
                    str(src), "-o", str(exe)], check=True, capture_output=True, text=True)

    def ask(calls):
        out = subprocess.run([str(exe)], input="".join("%d %d %d\n" % c for c in calls), capture_output=True, text=True)
        return [line == "1" for line in out.stdout.split()]
    return ask


def test_single_tokens_and_prompts(keys_stream):
    #                       requests, tokens, query heads a kv head
    assert keys_stream([(64, 64, 4), (32, 32 * 30, 4), (8, 8, 128), (1 << 17, 1 << 17, 128)]) == [True] * 4
    assert keys_stream([(1, 500, 4), (32, 32 * 33, 4), (16, 16000, 4), (0, 1, 1)]) == [False] * 4


def test_no_call_outlasts_the_bounded_waits(keys_stream):
    """All rows may be one request's.  Where keys stream a tile of 128 rows takes 1.7 us at 1.9 GHz (2.2 at 1.5,
    twice that with rows from memory at worst) and waits last as long as all of them; they give up after 2 s."""
    rng = random.Random(1)
    calls = [(1 << 20, (1 << 27) // g, g) for g in (1, 3, 7, 8, 32, 65, 128)]
    for _ in range(20000):
        G = rng.choice([1, 2, 3, 4, 7, 8, 16, 32, 65, 100, 128])
        calls.append((rng.randint(1, 1 << rng.randint(0, 20)), rng.randint(1, (1 << rng.randint(0, 27)) // G + 1), G))
    calls = [(R, N, G) for R, N, G in calls if N * G <= 1 << 27]
    found = keys_stream(calls)
    assert len(found) == len(calls) and any(found)
    for (R, N, G), keys in zip(calls, found):
        if keys:
            tiles = -(-N // (128 // G))
            assert tiles * 4.4e-6 < 1.5, (R, N, G)
